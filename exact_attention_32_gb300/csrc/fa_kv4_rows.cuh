// Attention over a 4-bit cache for many rows a key head (part of fa_kv4_decode.cu; its shares, merge and notation).
//
// fa_kv4_decode_kernel leaves the codes as they are, since with few rows there is no time to decode them; it pays for that
// with every score: four products of 32 channels (K's scale differs between them) in two parts of q, and P in three parts.
// With many rows a key the score's work is what counts.  Here a warpgroup decodes each tile once for up to 48 rows:
//   S^T = K Q^T      K as halves, code times scale (exact: at most 6 significant bits), Q as halves under a power of two of its
//                    row (bf16's 8 bits: exact down to 2^-24 of the row's largest value, off by at most 2^-32 of that
//                    below); one value a score, summed in fp32
//   O^T += V^T P^T   V's codes as halves, P times V's scale as one half.  A row has one reference r, a whole number that
//                    stands in for its maximum (log2): p = 2^(x - r) in fp32 goes into the sum, p times the key's V scale into the
//                    product.  r keeps the largest such product so far between 2^8 and 2^15 (of a half's 2^-24 to
//                    2^16), and every p below 2^60 (of V rows that are all zeros).
// d = 64: V's rows of keys 0-63 and 64-127 of a tile lie side by side, so that the product has 128 rows; P's columns of
// the second half of the keys lie behind those of the first, and O is the sum of the two diagonal blocks.
//
// A tile is 128 keys; a CTA an SM.  A softmax warpgroup takes half of the rows, one thread a key.  Its steps hang on one
// another (scores, whether a row's reference grows, P), so two teams of two warpgroups take turns by tile, each with a
// reference, a sum and an O of its own, joined at the end of a segment: with one team a tile of 48 rows took 3430 cycles, of which
// the warps issued in 40 %, with two 2000 (60 %).  32 sequences of up to 8192, 8 key heads, 48 rows: 95 to 109 us from box to box, 1.4 to
// 1.6 TB/s of cache (22 us would be the bytes): the chain load, decode, S, P, O through pairs of buffers bounds it, no unit alone (without
// the conversions, the decoded tiles' stores or the exponentials a tile would take 3 % less).
// Roles (896 threads): warps 0-7 and 8-15 the teams; 16-19 decode K and 20-23 V; 24 loads K's codes and scales, 25 V's; 26 issues S's
// products and 27 O's (from one warp, in one order, each would wait for what the other waits for: 4000 cycles a tile).
// Launched with 72 registers a thread, of which the last twelve warps give some to the softmax of 48 rows.  Spilled all the same: 140 to
// 144 bytes stored and 132 to 136 loaded with 48 rows, 20 to 28 and 56 to 80 with 32.

constexpr int kRowsLaunchRegs = 72;
// A row's reference is set this far (log2) above what the largest term needs: with the decode kernel's 3 one of 24 rows grew in
// every sixth tile, at 5000 cycles each time.
constexpr float kRowsHeadroom = 6.f, kRowsTopLog2 = 15.f, kRowsSumLog2 = 60.f;
constexpr float kRowsNone = FLT_MAX;  // minus the reference of a row that has met no key
// What starting and ending an item costs, in tiles.  48 rows, 32 sequences of up to 8192: 6 134 us, 9 113, 13 104; 32 rows 100, 96,
// 100; 128 rows 296, 266, 246.
constexpr int kRowsItemUnits = 12;

template <int D, int NG>
struct RowCfg {
    static constexpr int N = 16 * NG, NH = 8 * NG;  // rows of a CTA, of a softmax warpgroup
    // 32 rows: with more for the softmax 100 us in place of 95 (32 sequences of up to 8192).  48 rows: as launched 111 us, this
    // split 101, others within 1 to 20 % above.
    static constexpr int kSoftmaxRegs = NG == 3 ? 88 : 72, kDecodeRegs = NG == 3 ? 48 : 72, kOtherRegs = NG == 3 ? 56 : 72;
    static_assert(4 * kSoftmaxRegs + 2 * kDecodeRegs + kOtherRegs <= 7 * kRowsLaunchRegs, "the warpgroups' shares are what the block has");
    static constexpr int kThreads = 896, kDecodeWarp = 16, kLoadWarp = 24, kMmaWarp = 26, kPvWarp = 27;
    static constexpr int TK = 128;
    static constexpr int kTile = TK * D * 2;
    static constexpr int kK = 0, kV = 2 * kTile;  // two each
    static constexpr int kQ = kV + 2 * kTile;
    static constexpr int kP = kQ + D / 64 * 8192;  // one a team
    static constexpr int kPBytes = 16384;
    // tiles as they lie in the pages: K's codes and scales; V's codes; V's scales and whether each run of 16 tokens is there
    // (which the softmax reads, later than the decoding warps read theirs)
    static constexpr int kStages = 2, kSmallStages = 4;
    static constexpr int kCodes = TK * D / 2, kRawKBytes = kCodes + TK * (D / 32), kSmallBytes = TK + 32;
    static constexpr int kRawK = kP + 2 * kPBytes, kRawV = kRawK + kStages * kRawKBytes, kSmall = kRawV + kStages * kCodes;
    // a softmax warpgroup's, per pair of rows: {mult, mult', -r, -r'}, {mult, mult', 0, 0}, {alpha, alpha'}; the rows' masks; a
    // failed wait
    static constexpr int kState = kSmall + kSmallStages * kSmallBytes;
    static constexpr int kSeen = 16 * (16 + 16 + 8), kFail = kSeen + 8 * 32, kStateBytes = kFail + 16;
    static constexpr int kRed = kState + 4 * kStateBytes;  // its reductions over warps: float [4][32]
    static constexpr int kMult = kRed + 4 * 512;           // of all rows
    static constexpr int kWalk = kMult + 4 * 48;
    static constexpr int kBar = kWalk + 64 + 8 * (kThreads / 32);
    static constexpr int kNumBars = 19 + 4 * kStages + 2 * kSmallStages;
    static constexpr int kSmemBytes = kBar + kNumBars * 8 + 16;
    static_assert(kSmemBytes <= 232448 && kRawKBytes % 16 == 0 && kStateBytes % 16 == 0 && kWalk % 16 == 0, "shared memory plan");
    static constexpr int kTmemCols = 512, kO = 128;  // S in columns [0, 64) and [64, 128), O behind them, 128 columns a team
};
// of the two buffers of a kind: + 0, + 1; then full and free of the stages of K, of V, and of V's scales
enum { R_K_READY = 0, R_K_FREE = 2, R_V_READY = 4, R_V_FREE = 6, R_S_FULL = 8, R_S_FREE = 10, R_P_READY = 12, R_PV_DONE = 14, R_Q_READY = 16,
       R_DONE, R_RAW = R_DONE + 2 };

// Joins V values of every lane over the warp: lane i (i < V) gets the i-th values', by halving: V + 32 / V exchanges, where
// one value after the other takes 5 V.
template <int V, typename F>
__device__ __forceinline__ float over_lanes(float (&v)[V], F join)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = V / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool upper = lane & o;
            const float mine = upper ? v[i + o] : v[i], theirs = upper ? v[i] : v[i + o];
            v[i] = join(mine, __shfl_xor_sync(0xffffffffu, theirs, o));
        }
    float x = v[0];
#pragma unroll
    for (int o = V; o < 32; o <<= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <int D, int NG>
__global__ void __launch_bounds__(RowCfg<D, NG>::kThreads, 1)
fa_kv4_rows_kernel(const DecodeArgs a)
{
    using C = RowCfg<D, NG>;
    constexpr int N = C::N, NH = C::NH, TK = C::TK, RS = C::kStages, XS = C::kSmallStages;
    constexpr int KRAW_FULL = R_RAW, KRAW_FREE = KRAW_FULL + RS, VRAW_FULL = KRAW_FREE + RS, VRAW_FREE = VRAW_FULL + RS, X_FULL = VRAW_FREE + RS,
                  X_FREE = X_FULL + XS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((sb & 1023u) != 0) {  // the swizzled tiles need a 1024-byte-aligned base
        if (tid == 0) kv4_timeout();
        return;
    }
    const uint32_t bar0 = sb + C::kBar;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBar + C::kNumBars * 8);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(R_K_READY + i), 4);
            mbar_init(BAR(R_K_FREE + i), 1);
            mbar_init(BAR(R_V_READY + i), 4);
            mbar_init(BAR(R_V_FREE + i), 1);
            mbar_init(BAR(R_S_FULL + i), 1);
            mbar_init(BAR(R_S_FREE + i), 8);
            mbar_init(BAR(R_P_READY + i), 8);
            mbar_init(BAR(R_PV_DONE + i), 1);
        }
        mbar_init(BAR(R_Q_READY), 16);
        mbar_init(BAR(R_DONE), 1);
        mbar_init(BAR(R_DONE + 1), 1);
        for (int s = 0; s < RS; ++s) {
            mbar_init(BAR(KRAW_FULL + s), 1);
            mbar_init(BAR(KRAW_FREE + s), 4);
            mbar_init(BAR(VRAW_FULL + s), 1);
            mbar_init(BAR(VRAW_FREE + s), 4);
        }
        for (int s = 0; s < XS; ++s) {
            mbar_init(BAR(X_FULL + s), 1);
            mbar_init(BAR(X_FREE + s), 8);
        }
        fence_mbar_init();
        // (one thread asks: the status may change while a block starts, and its roles have to agree)
        tmem_slot[1] = *reinterpret_cast<volatile int *>(&g_kv4_status) != FA_ERR_TIMEOUT;
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    Walk &start = *reinterpret_cast<Walk *>(smem + C::kWalk);
    const int64_t share = walk_begin<TK, C::kThreads>(a, start, reinterpret_cast<int64_t *>(smem + C::kWalk + 64));
    if (tid == 0) a.split[blockIdx.x].parts = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk w = start;
    if (tmem_slot[1] == 0) w.left = 0;

    if (warp >= C::kLoadWarp) {
        registers_to<kRowsLaunchRegs, C::kOtherRegs>();
        if (warp == C::kLoadWarp || warp == C::kLoadWarp + 1) {
            // ----------------------------------------------------------------- loads: K, or V and its scales
            const bool values = warp != C::kLoadWarp;
            const int bt = min(1 << a.c.log2_page, TK), n_boxes = TK / bt;  // tokens a lane loads: a page, or the tile's part of one
            // the table's entry for this lane's tokens, asked for a tile ahead
            auto entry = [&](int t) -> int {
                const int key = t * TK + lane * bt;
                return lane < n_boxes && key < w.len ? a.table[w.b * a.max_pages + (key >> a.c.log2_page)] : 0;
            };
            int n = 0;
            bool ok = true;
            while (w.left > 0 && w.t0 == w.t1) walk_next<TK>(w, a);
            int t = w.t0, next = w.left > 0 ? entry(t) : 0;
            for (; w.left > 0; ++n) {
                const int page = next, h = w.it / a.n_rc, key = t * TK + lane * bt;
                bool there = lane < n_boxes && key < w.len;
                if (there && static_cast<unsigned>(page) >= static_cast<unsigned>(a.c.n_pages)) {
                    kv4_report();
                    there = false;
                }
                const uint32_t boxes = __ballot_sync(0xffffffffu, there);
                if (++t == w.t1) {
                    do walk_next<TK>(w, a);
                    while (w.left > 0 && w.t0 == w.t1);
                    t = w.t0;
                }
                if (w.left > 0) next = entry(t);
                const int st = n % RS, xs = n % XS, tokens = __popc(boxes) * bt;
                const int64_t row = there ? kv4_row(a.c, page, h, key) : 0;
                // (rows that are left out keep stale bytes, as good as any: their weight is 0)
                if (!values) {
                    if (n >= RS && !(ok = mbar_wait_warp(BAR(KRAW_FREE + st), (n / RS - 1) & 1, kWaitLimitNs))) break;
                    const uint32_t to = sb + C::kRawK + st * C::kRawKBytes;
                    if (lane == 0) mbar_arrive_expect_tx(BAR(KRAW_FULL + st), tokens * (D / 2 + D / 32));
                    __syncwarp();
                    if (there) {
                        bulk_load(to + lane * bt * (D / 2), a.c.k + row * (D / 2), bt * (D / 2), BAR(KRAW_FULL + st));
                        bulk_load(to + C::kCodes + lane * bt * (D / 32), a.c.k_scale + row * (D / 32), bt * (D / 32), BAR(KRAW_FULL + st));
                    }
                } else {
                    if (n >= XS && !(ok = mbar_wait_warp(BAR(X_FREE + xs), (n / XS - 1) & 1, kWaitLimitNs))) break;
                    uint8_t *small = smem + C::kSmall + xs * C::kSmallBytes;
                    if (lane < TK / 16) reinterpret_cast<int *>(small + TK)[lane] = (boxes >> (lane * 16 / bt)) & 1u;
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(BAR(X_FULL + xs), tokens);
                    __syncwarp();
                    if (there) bulk_load(smem_u32(small) + lane * bt, a.c.v_scale + row, bt, BAR(X_FULL + xs));
                    if (n >= RS && !(ok = mbar_wait_warp(BAR(VRAW_FREE + st), (n / RS - 1) & 1, kWaitLimitNs))) {
                        ++n;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(BAR(VRAW_FULL + st), tokens * (D / 2));
                    __syncwarp();
                    if (there)
                        bulk_load(sb + C::kRawV + st * C::kCodes + lane * bt * (D / 2), a.c.v + row * (D / 2), bt * (D / 2), BAR(VRAW_FULL + st));
                }
            }
            if (!ok && lane == 0) kv4_timeout();
            // no copy in flight when the CTA ends
            const uint64_t lim = ok ? kWaitLimitNs : kCleanupLimitNs;
            for (int i = n > RS ? n - RS : 0; i < n; ++i) mbar_wait(BAR((values ? VRAW_FULL : KRAW_FULL) + i % RS), (i / RS) & 1, lim);
            for (int i = n > XS ? n - XS : 0; values && i < n; ++i) mbar_wait(BAR(X_FULL + i % XS), (i / XS) & 1, lim);
        } else if (warp == C::kMmaWarp) {
            // ------------------------------------------------------------- products of the scores
            constexpr uint32_t idS = idesc_f16_f32(128, N, false);
            const uint64_t d_kmaj = smem_desc_sw128(sb, 16, 1024);
            const uint32_t kmaj = lo32(d_kmaj), kmaj_hi = hi32(d_kmaj);
            bool ok = true;
            int n = 0, seg = 0;
            for (; w.left > 0 && ok; walk_next<TK>(w, a)) {
                if (w.t0 == w.t1) continue;
                if (!(ok = mbar_wait_warp(BAR(R_Q_READY), seg++ & 1, kWaitLimitNs))) break;
                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    const int buf = n & 1;
                    if (!(ok = n < 2 ? mbar_wait_warp(BAR(R_K_READY + buf), 0, kWaitLimitNs)
                                     : wait_both(BAR(R_K_READY + buf), (n >> 1) & 1, BAR(R_S_FREE + buf), ((n >> 1) - 1) & 1)))
                        break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss_lohi(tmem + buf * 64, kmaj + ((C::kK + buf * C::kTile + kk / 4 * 16384 + kk % 4 * 32) >> 4), kmaj_hi,
                                        kmaj + ((C::kQ + kk / 4 * 8192 + kk % 4 * 32) >> 4), kmaj_hi, idS, kk > 0 ? 1u : 0u);
                        mma_commit(BAR(R_S_FULL + buf));
                        mma_commit(BAR(R_K_FREE + buf));
                    }
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) kv4_timeout();
            if (elect_one()) mma_commit(BAR(R_DONE));
            __syncwarp();
            mbar_wait_warp(BAR(R_DONE), 0, ok ? kWaitLimitNs : kCleanupLimitNs);
        } else if (warp == C::kPvWarp) {
            // -------------------------------------------- products of the outputs: O^T (+)= V^T P^T
            constexpr uint32_t idO = idesc_f16_f32(128, D == 128 ? N : 2 * N, true, true);
            constexpr int kHalf = D == 128 ? 16384 : 8192;  // between V's (and P's) blocks of 64 columns
            const uint64_t d_mn = smem_desc_sw128(sb, kHalf, 1024);
            const uint32_t mn = lo32(d_mn), mn_hi = hi32(d_mn);
            bool ok = true;
            int n = 0;
            for (; w.left > 0 && ok; walk_next<TK>(w, a))
                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    const int buf = n & 1;
                    if (!(ok = wait_both(BAR(R_V_READY + buf), (n >> 1) & 1, BAR(R_P_READY + buf), (n >> 1) & 1))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < (D == 128 ? 8 : 4); ++kk)
                            mma_ss_lohi(tmem + C::kO + buf * 128, mn + ((C::kV + buf * C::kTile) >> 4) + kk * 128, mn_hi,
                                        mn + ((C::kP + buf * C::kPBytes) >> 4) + kk * 128, mn_hi, idO, t < w.t0 + 2 && kk == 0 ? 0u : 1u);
                        mma_commit(BAR(R_PV_DONE + buf));
                        mma_commit(BAR(R_V_FREE + buf));
                    }
                    __syncwarp();
                }
            if (!ok && lane == 0) kv4_timeout();
            if (elect_one()) mma_commit(BAR(R_DONE + 1));
            __syncwarp();
            mbar_wait_warp(BAR(R_DONE + 1), 0, ok ? kWaitLimitNs : kCleanupLimitNs);
        }
    } else if (warp >= C::kDecodeWarp) {
        registers_to<kRowsLaunchRegs, C::kDecodeRegs>();
        {
            // ------------------------------------------------ decoding: 32 channels of a key a thread at a time
            constexpr int PPR = D / 32, TURNS = TK * PPR / 128;
            bool ok = true;
            int n = 0;
            const bool values = warp >= C::kDecodeWarp + 4;  // V (else K)
            const int free = values ? R_V_FREE : R_K_FREE, ready = values ? R_V_READY : R_K_READY, full = values ? VRAW_FULL : KRAW_FULL,
                      raw_free = values ? VRAW_FREE : KRAW_FREE;
            for (; w.left > 0 && ok; walk_next<TK>(w, a))
                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    const int st = n % RS, buf = n & 1;
                    const uint8_t *raw = smem + (values ? C::kRawV + st * C::kCodes : C::kRawK + st * C::kRawKBytes);
                    if (!(ok = n < 2 ? mbar_wait_warp(BAR(full + st), (n / RS) & 1, kWaitLimitNs)
                                     : wait_both(BAR(full + st), (n / RS) & 1, BAR(free + buf), ((n >> 1) - 1) & 1)))
                        break;
                    // all of a thread's pieces ahead of its stores, which would hold the loads back
                    uint4 x[TURNS];
                    __half2 scale[TURNS];
#pragma unroll
                    for (int i = 0; i < TURNS; ++i) {
                        const int piece = i * 128 + (tid & 127);
                        x[i] = reinterpret_cast<const uint4 *>(raw)[piece];
                        if (!values) scale[i] = __half2half2(kv4_scale_half(raw[C::kCodes + piece]));
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(raw_free + st));
                    // piece i to its row, times a scale or as it is; pieces of the second 64 channels (d = 128) write the other
                    // half of theirs first, so that the eight lanes of a store meet in no bank
                    auto put = [&](int i, uint8_t *to, auto scaled) {
                        const int piece = i * 128 + (tid & 127), key = piece / PPR, p = piece % PPR;
                        const bool turn = p & 2;
                        const uint32_t word[4] = {turn ? x[i].z : x[i].x, turn ? x[i].w : x[i].y, turn ? x[i].x : x[i].z, turn ? x[i].y : x[i].w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t y[4];
                            kv4_decode8(word[u], y);
                            if constexpr (decltype(scaled)::value) {
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const __half2 v = __hmul2(half2_of(y[c]), scale[i]);
                                    y[c] = *reinterpret_cast<const uint32_t *>(&v);
                                }
                            }
                            *reinterpret_cast<uint4 *>(to + ((((p & 1) * 4 + (u ^ (p & 2))) ^ (key & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    };
#pragma unroll
                    for (int i = 0; i < TURNS; ++i) {
                        const int piece = i * 128 + (tid & 127), key = piece / PPR, p = piece % PPR;
                        if (values)
                            put(i, smem + C::kV + buf * C::kTile + (D == 128 ? (p >> 1) * 16384 + key * 128 : (key >> 6) * 8192 + (key & 63) * 128),
                                std::false_type{});
                        else
                            put(i, smem + C::kK + buf * C::kTile + (p >> 1) * 16384 + key * 128, std::true_type{});
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(ready + buf));
                }
            if (!ok && lane == 0) kv4_timeout();
        }
    } else {
        // --------------------- softmax: warpgroup (team, g) has rows g NH .. g NH + NH - 1 of the team's tiles
        registers_to<kRowsLaunchRegs, C::kSoftmaxRegs>();
        const int wg = warp >> 2, team = wg >> 1, g = wg & 1, wl = warp & 3, tl = tid & 127;  // tl: TMEM lane, the tile's key
        const uint32_t loff = static_cast<uint32_t>(wl * 32) << 16;
        uint8_t *const state = smem + C::kState + wg * C::kStateBytes;
        float4 *sm_ref = reinterpret_cast<float4 *>(state), *sm_raw = sm_ref + 16;  // [row pair]
        float2 *sm_alpha = reinterpret_cast<float2 *>(state + 32 * 16);
        volatile float *sm_fail = reinterpret_cast<volatile float *>(state + C::kFail);  // a wait gave up: the group leaves together
        uint64_t *sm_seen = reinterpret_cast<uint64_t *>(state + C::kSeen);
        float *sm_red = reinterpret_cast<float *>(smem + C::kRed + wg * 512);  // [warp][row]
        float *sm_mult = reinterpret_cast<float *>(smem + C::kMult);              // [row]: a product of its halves times this is the score
        auto sync = [&]() { group_sync(1 + wg); };
        auto both_sync = [&]() { asm volatile("barrier.cta.sync %0, 256;\n" ::"r"(5 + g) : "memory"); };  // both teams' warpgroups of these rows
        auto all_sync = [&]() { asm volatile("barrier.cta.sync 7, 512;\n" ::: "memory"); };
        constexpr int V = NH <= 16 ? 16 : 32;  // values that over_lanes joins
        // O's columns of this group's rows, for the tile's keys 0-63 and 64-127 (d = 64)
        auto o_col = [&](int half, int r) -> uint32_t { return tmem + loff + C::kO + team * 128 + half * N + g * NH + r; };
        int n = 0;  // tiles of all segments before this one
        bool ok = true;
        if (tl == 0) *sm_fail = 0.f;
        for (; w.left > 0 && ok; walk_next<TK>(w, a)) {
            if (w.t0 == w.t1) continue;
            const int h = w.it / a.n_rc, rc = w.it - h * a.n_rc;
            const int64_t bh = static_cast<int64_t>(w.b) * a.c.heads + h;
            const int row0 = rc * N + g * NH, n_rows = min(NH, a.R - row0);  // (0 or less: this group has padding only)
            int newest = min(a.n_q, w.len);  // the sequence's drafts
            if (a.n_new != nullptr) newest = min(max(a.n_new[w.b], 0), newest);
            // Q: 8 channels a thread, D / 8 threads a row; the teams share the rows out.
            constexpr int TPR = D / 8, TURNS = (N * TPR + 511) / 512;
            const int64_t q_row0 = bh * a.R + rc * N;
            uint4 u[TURNS];
#pragma unroll
            for (int i = 0; i < TURNS; ++i) {
                const int r = (i * 512 + tid) / TPR, ch = tid % TPR;
                u[i] = make_uint4(0, 0, 0, 0);
                if (r < N && rc * N + r < a.R) u[i] = *reinterpret_cast<const uint4 *>(a.q + (q_row0 + r) * D + ch * 8);
            }
#pragma unroll
            for (int i = 0; i < TURNS; ++i) {
                const int r = (i * 512 + tid) / TPR, ch = tid % TPR;
                const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
                for (int c = 0; c < 4; ++c) top = max(top, max((x[c] << 16) & 0x7FFFFFFFu, x[c] & 0x7FFF0000u));
#pragma unroll
                for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const bool bad = top >= 0x7F800000u;
                // its exponent, held where 2^(7 - e) and 2^(e - 7) are normal numbers
                const int e = top == 0 ? 7 : min(max(static_cast<int>(top >> 23) - 127, -100), 127);
                const float up = __uint_as_float(static_cast<uint32_t>(7 - e + 127) << 23);
                if (r < N && ch == 0) sm_mult[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 7 + 127) << 23);
                uint32_t y[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const __half2 z = __floats2half2_rn(__uint_as_float(x[c] << 16) * up, __uint_as_float(x[c] & 0xFFFF0000u) * up);
                    y[c] = *reinterpret_cast<const uint32_t *>(&z);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) y[c] = bad ? 0x7FFF7FFFu : y[c];  // a row with a NaN or an infinity is NaN
                if (r < N)
                    *reinterpret_cast<uint4 *>(smem + C::kQ + (ch >> 3) * 8192 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                        make_uint4(y[0], y[1], y[2], y[3]);
            }
            if (tl < NH) sm_seen[tl] = a.tree[static_cast<int64_t>(w.b) * a.n_q + (row0 + tl) % a.n_q];
            fence_proxy_async_smem();
            all_sync();
            if (lane == 0) mbar_arrive(BAR(R_Q_READY));
            if (tl < NH / 2) {
                const float2 mult = *reinterpret_cast<const float2 *>(sm_mult + g * NH + 2 * tl);
                sm_ref[tl] = make_float4(mult.x, mult.y, kRowsNone, kRowsNone);
                sm_raw[tl] = make_float4(mult.x, mult.y, 0.f, 0.f);
            }
            sync();
            float2 l[NG][4];
#pragma unroll
            for (int q = 0; q < NG; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) l[q][i] = make_float2(0.f, 0.f);

            const int tiles = w.t1 - w.t0, mine0 = (n & 1) == team ? 0 : 1;  // this team's tiles: mine0, mine0 + 2, ...
            for (int i = mine0; i < tiles; i += 2) {
                const int nn = n + i, xs = nn % XS, key = (w.t0 + i) * TK + tl;
                const uint32_t phase = (nn >> 1) & 1;
                const uint8_t *small = smem + C::kSmall + xs * C::kSmallBytes;
                ok = wait_both(BAR(X_FULL + xs), (nn / XS) & 1, BAR(R_S_FULL + team), phase);
                if (!ok) *sm_fail = 1.f;
                tc_fence_after();
                float vs = kv4_scale(small[tl]);
                const bool here = reinterpret_cast<const int *>(small + TK)[tl >> 4] != 0;
                // keys that a row does not admit, or that no page holds, leave it; what lies there may be anything
                const bool edge = (w.t0 + i) * TK + TK > w.len - newest || __any_sync(0xffffffffu, !here);
                const bool gone = key >= w.len || !here;
                if (gone) vs = 0.f;
                const float limit = fminf(kRowsTopLog2 - lg2(vs), kRowsSumLog2);  // x - r of this key stays below
                // this key's log2 scores less the rows' references; anew where a row's grows (always in its first tile, soon
                // seldom): first the scores themselves, then against what the references have become
                float2 x[NG][4];
                const float4 *from = i == mine0 ? sm_raw : sm_ref;
                // (the same rounded product both times, so its addend is one that is not known to be 0: mul and add are made one fma,
                // which is off by more than a reference allows where scores pass 2^28)
                const float zero = *reinterpret_cast<const volatile float *>(&sm_raw[0].z);
                for (bool grown = false;;) {
                    uint32_t s[NG][8];
#pragma unroll
                    for (int q = 0; q < NG; ++q) tmem_ld8(tmem + loff + team * 64 + g * NH + q * 8, s[q]);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 c = from[q * 4 + j];
                            const float2 p = fma2(make_float2(__uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1])), make_float2(c.x, c.y),
                                                  make_float2(zero, zero));
                            x[q][j] = add2(p, make_float2(c.z, c.w));
                        }
                    if (edge) {
                        const int draft = key - (w.len - newest), bit = draft & 63;
                        const uint32_t *seen = reinterpret_cast<const uint32_t *>(sm_seen) + (bit >> 5);
#pragma unroll
                        for (int q = 0; q < NG; ++q)
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                if (gone || (draft >= 0 && ((seen[2 * (q * 8 + r)] >> (bit & 31)) & 1u) == 0))
                                    (r & 1 ? x[q][r / 2].y : x[q][r / 2].x) = -INFINITY;
                    }
                    if (grown) break;
                    if (from == sm_ref) {
                        float top = -INFINITY;
#pragma unroll
                        for (int q = 0; q < NG; ++q)
#pragma unroll
                            for (int j = 0; j < 4; ++j) top = fmax3(top, x[q][j].x, x[q][j].y);
                        const bool grows = group_or(1 + wg, top > limit);
                        if (*sm_fail != 0.f) ok = false;
                        if (!grows || !ok) break;
                        from = sm_raw;
                        continue;
                    }
                    // of the warp's keys, what row `lane`'s reference has to be at least
                    float v[V];
#pragma unroll
                    for (int r = 0; r < V; ++r) {
                        const float xr = r < NH ? (r & 1 ? x[r / 8][r / 2 % 4].y : x[r / 8][r / 2 % 4].x) : 0.f;
                        v[r] = fmaxf(__fsub_ru(xr, limit), -FLT_MAX);  // (up: a reference below x - limit lets P pass a half's range)
                    }
                    const float need = over_lanes<V>(v, [](float p, float q) { return fmaxf(p, q); });
                    if (lane < NH) sm_red[wl * 32 + lane] = need;
                    sync();
                    if (tl < NH) {
                        const float most = fmaxf(fmaxf(sm_red[tl], sm_red[32 + tl]), fmaxf(sm_red[64 + tl], sm_red[96 + tl]));
                        float *minus_r = reinterpret_cast<float *>(sm_ref + (tl >> 1)) + 2 + (tl & 1);
                        const float old = -*minus_r, r = most > old ? ceilf(most + kRowsHeadroom) : old;
                        reinterpret_cast<float *>(sm_alpha)[tl] = ex2(old - r);
                        *minus_r = -r;
                    }
                    // O is complete so far
                    if (i > mine0 && !mbar_wait_warp(BAR(R_PV_DONE + team), phase ^ 1, kWaitLimitNs)) *sm_fail = 1.f;
                    sync();
                    if (*sm_fail != 0.f) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j) l[q][j] = mul2(l[q][j], sm_alpha[q * 4 + j]);
                    if (i > mine0) {
                        tc_fence_after();
#pragma unroll
                        for (int half = 0; half < 128 / D; ++half)
#pragma unroll
                            for (int q = 0; q < NG; ++q) {
                                uint32_t o[8];
                                tmem_ld8(o_col(half, q * 8), o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 8; j += 2) {
                                    const float2 y = mul2(make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), sm_alpha[q * 4 + j / 2]);
                                    o[j] = __float_as_uint(y.x);
                                    o[j + 1] = __float_as_uint(y.y);
                                }
                                tmem_st8(o_col(half, q * 8), o);
                            }
                        tmem_wait_st();
                    }
                    grown = true;
                    from = sm_ref;
                }
                if (!ok) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(BAR(R_S_FREE + team));
                    mbar_arrive(BAR(X_FREE + xs));
                }
                // P: the sum in fp32, the product's operand times V's scale
                uint32_t y[NG][4];
#pragma unroll
                for (int q = 0; q < NG; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 p = make_float2(ex2(x[q][j].x), ex2(x[q][j].y)), pv = mul2(p, make_float2(vs, vs));
                        l[q][j] = add2(l[q][j], p);
                        const __half2 z = __floats2half2_rn(pv.x, pv.y);
                        y[q][j] = *reinterpret_cast<const uint32_t *>(&z);
                    }
                if (edge) {  // a value that a row does not admit stays out of it, a NaN too
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            y[q][j] &= (x[q][j].x == -INFINITY ? 0u : 0xFFFFu) | (x[q][j].y == -INFINITY ? 0u : 0xFFFF0000u);
                }
                // the product of the team's tile before has read P
                if (nn > 1 && !mbar_wait_warp(BAR(R_PV_DONE + team), phase ^ 1, kWaitLimitNs)) *sm_fail = 1.f;
#pragma unroll
                for (int q = 0; q < NG; ++q) {
                    const int col = (D == 128 ? 0 : (tl >> 6) * N) + g * NH + q * 8, k = D == 128 ? tl : tl & 63;
                    *reinterpret_cast<uint4 *>(smem + C::kP + team * C::kPBytes + (col >> 6) * 8192 + k * 128 + ((((col & 63) >> 3) ^ (k & 7)) << 4)) =
                        make_uint4(y[q][0], y[q][1], y[q][2], y[q][3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(R_P_READY + team));
            }
            // (a group whose wait gave up still meets the others at the barriers below; all leave behind them)

            // ---------------------------------------------------- end of the segment
            const bool any = mine0 < tiles;  // this team had a tile
            const int last = n + mine0 + (tiles - 1 - mine0) / 2 * 2;
            if (any && ok && !mbar_wait_warp(BAR(R_PV_DONE + team), (last >> 1) & 1, kWaitLimitNs)) *sm_fail = 1.f;
            tc_fence_after();
            {
                float v[V];
#pragma unroll
                for (int r = 0; r < V; ++r) v[r] = r < NH ? (r & 1 ? l[r / 8][r / 2 % 4].y : l[r / 8][r / 2 % 4].x) : 0.f;
                const float sum = over_lanes<V>(v, [](float p, float q) { return p + q; });
                if (lane < NH) sm_red[wl * 32 + lane] = sum;
            }
            all_sync();
            bool failed = false;  // (all leave where one has to: they meet again at the barriers below)
#pragma unroll
            for (int i = 0; i < 4; ++i) failed |= *reinterpret_cast<const volatile float *>(smem + C::kState + i * C::kStateBytes + C::kFail) != 0.f;
            if (failed) {
                ok = false;
                break;
            }
            // A thread a row: what this team's O is multiplied with (to be under the larger of the teams' references, and over
            // the sum if the segment is the whole item), 0 where nothing is to come of it
            const bool whole = w.t0 == 0 && w.t1 == w.n_t;
            const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (n == 0 ? 0 : 1);
            float *sm_factor = reinterpret_cast<float *>(sm_alpha);
            if (tl < NH) {
                const float *state_other = reinterpret_cast<const float *>(smem + C::kState + (wg ^ 2) * C::kStateBytes);
                const float *red_other = reinterpret_cast<const float *>(smem + C::kRed + (wg ^ 2) * 512);
                const int at = (tl >> 1) * 4 + 2 + (tl & 1);
                const float own = -reinterpret_cast<const float *>(sm_ref)[at], other = -state_other[at], m = fmaxf(own, other);
                const float own_f = ex2(own - m);
                float ll = ((sm_red[tl] + sm_red[32 + tl]) + (sm_red[64 + tl] + sm_red[96 + tl])) * own_f +
                           ((red_other[tl] + red_other[32 + tl]) + (red_other[64 + tl] + red_other[96 + tl])) * ex2(other - m);
                float factor = any ? own_f : 0.f;
                if ((row0 + tl) % a.n_q >= newest) factor = ll = 0.f;  // no draft of this sequence
                if (whole) factor *= ll == 0.f ? 0.f : 1.f / ll;
                sm_factor[tl] = factor;
                if (team == 0 && tl < n_rows) {
                    if (whole)
                        a.lse[bh * a.R + row0 + tl] = ll == 0.f ? -INFINITY : (m + log2f(ll)) * kLn2;
                    else
                        a.part_ml[slot * N + g * NH + tl] = make_float2(m, ll);
                }
            }
            if (tid == 0 && w.t0 == 0 && !whole) {
                Split sp;
                sp.row = bh * a.R + row0;
                sp.n_rows = min(N, a.R - row0);
                sp.parts = 1 + static_cast<int>((w.n_t - w.t1 + share - 1) / share);
                sp.slot = static_cast<int>(slot);
                sp.pad = 0;
                a.split[blockIdx.x] = sp;
            }
            sync();
            const int half = D == 64 ? wl >> 1 : 0;  // d = 64: lanes 64-127 hold keys 64-127's part of channel lane - 64
            float y[NG][8];
            {
                uint32_t o[NG][8];
#pragma unroll
                for (int q = 0; q < NG; ++q) tmem_ld8(o_col(half, q * 8), o[q]);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < NG; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float f = sm_factor[q * 8 + j];
                        y[q][j] = f == 0.f ? 0.f : __uint_as_float(o[q][j]) * f;
                    }
            }
            tc_fence_before();
            // scratch: a P buffer of these rows', which the products have read; team 1's values, and (d = 64) lanes 64-127's of each
            // team
            float *sx = reinterpret_cast<float *>(smem + C::kP + g * C::kPBytes);
            if constexpr (D == 128) {
                if (team == 1)
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int j = 0; j < 8; ++j) sx[(q * 8 + j) * 128 + tl] = y[q][j];
            } else {
                if (half == 1)
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int j = 0; j < 8; ++j) sx[(team * NH + q * 8 + j) * 64 + tl - 64] = y[q][j];
                sync();
                if (half == 0) {
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[q][j] += sx[(team * NH + q * 8 + j) * 64 + tl];
                    if (team == 1)
#pragma unroll
                        for (int q = 0; q < NG; ++q)
#pragma unroll
                            for (int j = 0; j < 8; ++j) sx[(NH + q * 8 + j) * 64 + tl] = y[q][j];
                }
            }
            both_sync();
            if (team == 0 && (D == 128 || half == 0)) {
#pragma unroll
                for (int q = 0; q < NG; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[q][j] += sx[D == 128 ? (q * 8 + j) * 128 + tl : (NH + q * 8 + j) * 64 + tl];
#pragma unroll
                for (int q = 0; q < NG; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = q * 8 + j;
                        if (r >= n_rows) continue;
                        if (whole)
                            a.o[(bh * a.R + row0 + r) * D + tl] = __float2bfloat16_rn(y[q][j]);
                        else
                            a.part_o[(slot * N + g * NH + r) * D + tl] = y[q][j];
                    }
            }
            n += tiles;
            all_sync();  // before the next segment's Q and state take the place of these
        }
        if (!ok && lane == 0) kv4_timeout();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}
