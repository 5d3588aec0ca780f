// Exact attention forward of packed sequences with grouped heads (fa_fwd_packed): TMA + tcgen05 + TMEM.
//
// Per sequence (rows start .. start + len - 1 of the packed tensors), query head h and row i:
//   S_ij = scale q_i . k_j over the sequence's keys j (causal: j <= i) of key head h / (H / Hkv),
//   P = softmax(S),  O_i = sum_j P_ij v_j,  LSE_i = m_i + ln l_i
// in one pass over the keys with a running maximum, sum and numerator, as in fa_fwd_tc.cu, whose pipeline
// this is: two tiles of 128 query rows share one stream of K/V tiles of 128 keys; a warp loads (TMA), a warp
// issues the products (S = Q K^T from shared memory, O += P V with P from tensor memory), a warpgroup per tile takes
// the softmax with a row a thread.  What differs:
//   - The work list is the plan's (fa_packed.cuh), longest loops first; a persistent CTA takes its items in zigzag
//     order, which pairs long ones with short ones.
//   - With an even number of query heads a key head, the two tiles of an item are the same 128 rows of two heads (PAIR):
//     they end on the same key tile, and a sequence of up to 128 rows fills both.  Otherwise they are 256 rows of one
//     head; a tile behind the sequence's end is left out, and causal the first tile ends a key tile before the second.
//   - A 128-row tile that reaches behind its sequence holds rows of others.  Their keys' scores become -inf, their rows of V
//     zeros (zero_tail_rows, up to a step of the product), their rows of O stay in tensor memory: a whole warp's 32 rows
//     leave by TMA, the rows of a cut one by stores of their own.
//   - A thread finds its item in the list; the next one is asked for an item ahead.
//   - Where few long items leave SMs idle, a cluster of CTAs shares each (ranks_of).
// What bounds it is the chain S, softmax, P V of a tile, as in fa_fwd_tc.cu, and an item's start and end, about two tiles: 3
// sequences of up to 16384, 32 heads on 8, d = 128, causal, 1930 to 2070 us (1.59 to 1.49 PFLOP/s, by the power), 16 of 200 to 4096 320 to 340 us (1.30; the tensor pipe
// 62 % busy), 48 of 100 to 1000, 16 heads, d = 64, not causal 76 us (0.57, 35 %).
// Every mbarrier wait is bounded; a wait that gives up sets FA_ERR_TIMEOUT and the CTA winds down.
#include <math.h>

#include <type_traits>

#include "fa_packed.cuh"

using namespace sm100;

namespace {

constexpr int kTile = 128;    // query rows of a tile, keys of a K/V tile
// Three warpgroups: two of softmax, and the load and product warps' (two of its warps idle).  Launched with 168 registers a
// thread (what 384 threads may have); the third gives 64 of its own up, and the softmax, a row's 128 scores a thread, takes 32 more each
// (with 168 it spilled up to 250 bytes).  What ptxas spills is left of that: 16 to 36 bytes stored and 28 to 64 loaded, 44 and 96 to 124
// where a cluster shares an item.
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 200, kOtherRegs = 104;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "the warpgroups' shares are what the block has");
constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr float kRescaleLog2 = 8.0f;  // the numerator is rescaled when the row max grows by more than 2^8
constexpr float kHeavyShare = 0.25f;  // d = 128: see "heavy" in the softmax
constexpr uint64_t kWaitLimitNs = 1000000000ull;   // 1 s per pipeline wait
constexpr uint64_t kCleanupLimitNs = 20000000ull;  // 20 ms per wait while winding down

template <int D>
struct PCfg {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kAtoms = D / 64;                  // 128-byte-wide column blocks of a tile
    static constexpr int kStages = D == 128 ? 4 : 8;       // K/V ring slots
    static constexpr int kSSteps = D / 16;
    // d = 64: the P V product runs at N = 80 with a column of ones behind V's 64, so that column 64 of O is the sum of exactly the
    // rounded P that is multiplied
    static constexpr bool kOnesCol = D == 64;
    static constexpr int kPVN = kOnesCol ? 80 : D;
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kOnes = kRing + kStages * kTileBytes;
    static constexpr int kBar = kOnes + (kOnesCol ? kTile * 128 : 0);
    static constexpr int kNumBars = 9 + 2 * kStages;
    static constexpr int kStage = (kBar + kNumBars * 8 + 16 + 1023) / 1024 * 1024;  // O on its way out: 4 KB a softmax warp
    static constexpr int kSmemBytes = 1024 + kStage + 8 * 4096;
    static_assert(kSmemBytes <= 232448, "shared memory plan exceeds 227 KB");
};
enum { Q_FULL = 0, Q_EMPTY, S_FULL, P_FULL = S_FULL + 2, O_FULL = P_FULL + 2, MMA_DONE = O_FULL + 2, KV_FULL };

struct FwdArgs {
    PlanView plan;
    FaRows o;
    float *lse;
    int T, B, heads, units, group, fill;  // heads: H; units: items of a list entry; group: H / Hkv
    int ranks;                            // CTAs (a cluster) that share an item
    float scale, scale_log2;
};

// An item: up to two tiles of query rows against one key head's keys of a sequence.
struct Item {
    int start, len, row, head;
};

// First row (in the sequence) and head of tile t, and the key tiles it takes: none if it lies behind the sequence's end.
template <bool PAIR>
__device__ __forceinline__ int tile_row(const Item &w, int t) { return w.row + (PAIR ? 0 : t * kTile); }
template <bool PAIR>
__device__ __forceinline__ int tile_head(const Item &w, int t) { return w.head + (PAIR ? t : 0); }
template <bool CAUSAL, bool PAIR>
__device__ __forceinline__ int tile_keys(const Item &w, int t)
{
    const int row = tile_row<PAIR>(w, t);
    if (row >= w.len) return 0;
    return CAUSAL ? row / kTile + 1 : (w.len + kTile - 1) / kTile;
}

// The items of this CTA: in round r item r G + c of the grid's G CTAs, and in odd rounds r G + G - 1 - c.  The distance
// from one to the next alternates between two values, so the entry and the unit of an item (entry * units + unit) are
// carried along without a division (three of them took 600 cycles an item of every role's warp).
struct Items {
    const int4 *list;
    int left, units;  // items from this CTA's next on (at most 0: none), units of an entry
    int entry, unit;
    int step[2], step_entry[2], step_unit[2];
    int odd;
    int4 next;
    __device__ __forceinline__ Items(const int4 *l, int n_items, int n_units, int G, int c) : list(l), units(n_units), odd(0)
    {
        left = n_items - c;
        step[0] = 2 * (G - c) - 1;
        step[1] = 2 * c + 1;
        for (int i = 0; i < 2; ++i) {
            step_entry[i] = step[i] / units;
            step_unit[i] = step[i] - step_entry[i] * units;
        }
        entry = c / units;
        unit = c - entry * units;
        if (left > 0) next = __ldg(list + entry);
    }
    // The next item, if there is one; the one after it is asked for.
    template <bool PAIR>
    __device__ __forceinline__ bool take(Item &w)
    {
        if (left <= 0) return false;
        w.start = next.x;
        w.len = next.y;
        w.row = next.z * (PAIR ? kTile : 2 * kTile);
        w.head = PAIR ? 2 * unit : unit;
        left -= odd ? step[1] : step[0];
        entry += odd ? step_entry[1] : step_entry[0];
        unit += odd ? step_unit[1] : step_unit[0];
        odd ^= 1;
        if (unit >= units) {
            unit -= units;
            ++entry;
        }
        if (left > 0) next = __ldg(list + entry);
        return true;
    }
};

// Row max of a tile: eight independent chains of 3-input maxes.
__device__ __forceinline__ float row_max(const float (&s)[kTile])
{
    float mx[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        const int b = 16 * g;
        float a = fmax3(s[b], s[b + 1], s[b + 2]);
#pragma unroll
        for (int i = 3; i < 15; i += 2) a = fmax3(a, s[b + i], s[b + i + 1]);
        mx[g] = fmaxf(a, s[b + 15]);
    }
    return fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

// SHARED: there is a cluster of a.ranks CTAs for every item, each for its part of the key tiles; what they have of a row is joined
// through distributed shared memory, in the ranks' order.
template <int D, bool CAUSAL, bool PAIR, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
fa_packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const FwdArgs a)
{
    using C = PCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar0 = sb + C::kBar;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    auto FULL = [&](int s) { return BAR(KV_FULL + s); };
    auto EMPTY = [&](int s) { return BAR(KV_FULL + C::kStages + s); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBar + C::kNumBars * 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(BAR(Q_FULL), 1);
        mbar_init(BAR(Q_EMPTY), 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(BAR(S_FULL + t), 1);
            mbar_init(BAR(P_FULL + t), 4);  // one arrive per softmax warp
            mbar_init(BAR(O_FULL + t), 1);
        }
        mbar_init(BAR(MMA_DONE), 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(FULL(s), 1);
            mbar_init(EMPTY(s), 1);
        }
        fence_mbar_init();
    }
    if constexpr (C::kOnesCol) {
        // kTile rows of 128 bytes in V's swizzle: 1.0 in column 0 (16-byte piece 0 lies at piece r mod 8), zeros elsewhere
        for (int i = tid; i < kTile * 8; i += kThreads) {
            const int r = i >> 3, c = i & 7;
            reinterpret_cast<uint4 *>(smem + C::kOnes)[i] = make_uint4(c == (r & 7) ? 0x3F80u : 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // a plan of another T, B or mask, or a wait that gave up and nobody has read so yet: nothing is done (one thread asks: the
    // status may change while a block starts, and its roles have to agree)
    if (tid == 0) {
        const bool fits = plan_fits(a.plan.head, a.T, a.B, CAUSAL);
        if (!fits && blockIdx.x == 0) packed_bad_sequence();
        tmem_slot[1] = fits && *reinterpret_cast<volatile int *>(&g_packed_status) != FA_ERR_TIMEOUT;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool run = tmem_slot[1] != 0;
    const int n_items = run ? (PAIR ? a.plan.head->n_blocks : a.plan.head->n_pairs) * a.units : 0;
    const int ranks = SHARED ? a.ranks : 1, rank = SHARED ? blockIdx.x % ranks : 0;
    Items items(PAIR ? a.plan.blocks : a.plan.pairs, n_items, a.units, gridDim.x / ranks, blockIdx.x / ranks);
    Item w;
    // this CTA's key tiles [begin, end) of an item's n
    auto begin = [&](int n) { return SHARED ? n * rank / ranks : 0; };
    auto end = [&](int n) { return SHARED ? n * (rank + 1) / ranks : n; };

    if (warp >= kLoadWarp) {
        registers_down<kOtherRegs>();
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ loads
            if (lane == 0) {
                prefetch_tmap(&tm_q);
                prefetch_tmap(&tm_k);
                prefetch_tmap(&tm_v);
                bool ok = true;
                int it = 0, uc = 0;
                while (ok && items.take<PAIR>(w)) {
                    const int n0 = tile_keys<CAUSAL, PAIR>(w, 0), n1 = tile_keys<CAUSAL, PAIR>(w, 1), n_kv = max(n0, n1), j1 = end(n_kv);
                    if (SHARED && begin(n_kv) == j1) continue;
                    // the Q buffers are free once the item before has issued its last S
                    if (!(ok = mbar_wait(BAR(Q_EMPTY), (uc & 1) ^ 1, kWaitLimitNs))) break;
                    mbar_arrive_expect_tx(BAR(Q_FULL), (n1 > 0 ? 2 : 1) * C::kTileBytes);
                    for (int t = 0; t < (n1 > 0 ? 2 : 1); ++t)
                        for (int c = 0; c < C::kAtoms; ++c)
                            tma_load_3d(sb + t * C::kTileBytes + c * 16384, &tm_q, BAR(Q_FULL), c * 64, w.start + tile_row<PAIR>(w, t),
                                        tile_head<PAIR>(w, t));
                    ++uc;
                    const int kv = w.head / a.group;
                    for (int j = begin(n_kv); j < j1 && ok; ++j)
                        for (int kind = 0; kind < 2; ++kind, ++it) {
                            const int slot = it % C::kStages, use = it / C::kStages;
                            if (!(ok = mbar_wait(EMPTY(slot), (use & 1) ^ 1, kWaitLimitNs))) break;
                            mbar_arrive_expect_tx(FULL(slot), C::kTileBytes);
                            for (int c = 0; c < C::kAtoms; ++c)
                                tma_load_3d(sb + C::kRing + slot * C::kTileBytes + c * 16384, kind == 0 ? &tm_k : &tm_v, FULL(slot),
                                            c * 64, w.start + j * kTile, kv);
                        }
                }
                if (!ok) packed_timeout();
                // every copy this thread issued has landed before the CTA may exit
                const uint64_t lim = ok ? kWaitLimitNs : kCleanupLimitNs;
                if (uc > 0) mbar_wait(BAR(Q_FULL), (uc - 1) & 1, lim);
                for (int k = max(0, it - C::kStages); k < it; ++k) mbar_wait(FULL(k % C::kStages), (k / C::kStages) & 1, lim);
            }
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------------- products
            constexpr uint32_t idS = idesc_bf16_f32(kTile, kTile, false);
            constexpr uint32_t idO = idesc_bf16_f32(kTile, C::kPVN, true);
            const uint64_t dq = smem_desc_sw128(sb, 16, 1024);
            const uint64_t dk = smem_desc_sw128(sb + C::kRing, 16, 1024);
            const uint64_t dv = smem_desc_sw128(sb + C::kRing, C::kOnesCol ? C::kOnes - C::kRing : kTile * 128, 1024);
            const uint32_t dq_lo = static_cast<uint32_t>(dq), dq_hi = static_cast<uint32_t>(dq >> 32);
            const uint32_t dk_hi = static_cast<uint32_t>(dk >> 32), dv_hi = static_cast<uint32_t>(dv >> 32);
            constexpr uint32_t kTile16 = C::kTileBytes >> 4;
            // d = 64: the block behind V's 64 columns is the ones block, so the leading byte offset (bits 16..29) falls by what
            // the start address (bits 0..13) gains
            constexpr uint32_t kVSlot = C::kOnesCol ? kTile16 - (kTile16 << 16) : kTile16;
            bool ok = true;
            int it = 0, uc = 0;
            int sent[2] = {0, 0};  // S tiles sent to tile 0 / 1 (all items)
            while (ok && items.take<PAIR>(w)) {
                const int all = max(tile_keys<CAUSAL, PAIR>(w, 0), tile_keys<CAUSAL, PAIR>(w, 1)), j0 = begin(all), n_kv = end(all);
                const int n[2] = {min(tile_keys<CAUSAL, PAIR>(w, 0), n_kv), min(tile_keys<CAUSAL, PAIR>(w, 1), n_kv)};
                if (SHARED && j0 == n_kv) continue;
                const int last = (w.len - 1) / kTile, left = w.len - last * kTile;  // the sequence's last key tile, its keys
                if (!(ok = mbar_wait_warp(BAR(Q_FULL), uc & 1, kWaitLimitNs))) break;
                tc_fence_after();
                uint32_t v_lo = 0;  // V of the tile before
                int v_slot = -1, v_steps = kTile / 16;
                // O_t += P_t V of key tile j, and its end if it is the last
                auto pv = [&](int t, int j) -> bool {
                    if (!mbar_wait_warp(BAR(P_FULL + t), (sent[t] - 1) & 1, kWaitLimitNs)) return false;
                    tc_fence_after();
                    if (elect_one()) {
    #pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            if (kk < v_steps)
                                mma_ts_lohi(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, v_lo + kk * 128, dv_hi, idO,
                                            (j > j0 || kk > 0) ? 1u : 0u);
                        if (j == n[t] - 1) mma_commit(BAR(O_FULL + t));
                    }
                    __syncwarp();
                    return true;
                };
                for (int j = j0; j < n_kv && ok; ++j) {
                    const int kslot = it % C::kStages, kuse = it / C::kStages;
                    ++it;
                    const int vslot = it % C::kStages, vuse = it / C::kStages;
                    ++it;
                    if (!(ok = mbar_wait_warp(FULL(kslot), kuse & 1, kWaitLimitNs))) break;
                    tc_fence_after();
                    const uint32_t dk_lo = static_cast<uint32_t>(dk) + kslot * kTile16;
    #pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j > j0 && j <= n[t] && !(ok = pv(t, j - 1))) break;
                        if (j >= n[t]) continue;
                        if (elect_one()) {
    #pragma unroll
                            for (int kk = 0; kk < C::kSSteps; ++kk) {
                                const uint32_t koff = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                                mma_ss_lohi(tmem + t * 128, dq_lo + t * kTile16 + koff, dq_hi, dk_lo + koff, dk_hi, idS, kk > 0 ? 1u : 0u);
                            }
                            mma_commit(BAR(S_FULL + t));
                        }
                        __syncwarp();
                        ++sent[t];
                    }
                    if (!ok) break;
                    if (elect_one()) {
                        mma_commit(EMPTY(kslot));
                        if (j > j0) mma_commit(EMPTY(v_slot));
                        if (j == n_kv - 1) mma_commit(BAR(Q_EMPTY));  // the item's last reads of Q are issued
                    }
                    __syncwarp();
                    if (!(ok = mbar_wait_warp(FULL(vslot), vuse & 1, kWaitLimitNs))) break;
                    v_slot = vslot;
                    v_lo = static_cast<uint32_t>(dv) + vslot * kVSlot;
                    v_steps = kTile / 16;
                    if (j == last) {
                        v_steps = (left + 15) / 16;
                        if (left & 15) {
                            zero_tail_rows<D>(smem + C::kRing + vslot * C::kTileBytes, left, lane);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    tc_fence_after();
                }
    #pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (ok && n[t] == n_kv) ok = pv(t, n_kv - 1);
                if (!ok) break;
                if (elect_one()) mma_commit(EMPTY(v_slot));
                __syncwarp();
                ++uc;
            }
            if (!ok && lane == 0) packed_timeout();
            // no product of this CTA may still be running when tensor memory is freed
            if (elect_one()) mma_commit(BAR(MMA_DONE));
            __syncwarp();
            mbar_wait_warp(BAR(MMA_DONE), 0, ok ? kWaitLimitNs : kCleanupLimitNs);
        }
    } else {
        // --------------------------------------------------------------- softmax
        registers_up<kSoftmaxRegs>();
        const int t = warp >> 2;    // this warpgroup's tile
        const int row = tid & 127;  // row within the tile == TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * 128;
        const uint32_t tO = tmem + lane_off + 256 + t * 128;
        if (run && a.fill) {  // rows of no sequence
            const Outside out = outside(a.plan.head);
            const int64_t n = static_cast<int64_t>(out.n) * a.heads * (D / 8);
            for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + tid; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
                const int c = static_cast<int>(i % (D / 8)), h = static_cast<int>(i / (D / 8) % a.heads);
                const int r = out.row(static_cast<int>(i / (D / 8) / a.heads));
                reinterpret_cast<uint4 *>(packed_row(a.o, r, h))[c] = make_uint4(0, 0, 0, 0);
                if (c == 0) a.lse[static_cast<int64_t>(h) * a.T + r] = -INFINITY;
            }
        }
        bool ok = true;
        int jg = 0, uc = 0;
        const float c_u = a.scale_log2;
        float m_ref = -INFINITY;  // reference max, unscaled units
        float l = 0.f;            // exp-sum relative to m_ref (fp32 terms; gives LSE)
        float lr = 0.f;           // the divisor of O (d = 128)
        bool any = false;         // SHARED: this CTA has an item, and key tiles of it
        while (ok && items.take<PAIR>(w)) {
            const int all = SHARED ? max(tile_keys<CAUSAL, PAIR>(w, 0), tile_keys<CAUSAL, PAIR>(w, 1)) : 0;
            const int n_mine = tile_keys<CAUSAL, PAIR>(w, t), row0 = tile_row<PAIR>(w, t);
            const int j0 = begin(all), j1 = SHARED ? min(n_mine, end(all)) : n_mine;
            if (j1 <= j0) continue;
            const bool mine = row0 + row < w.len;
            m_ref = -INFINITY;
            l = lr = 0.f;
            // One key tile; `masked`: some row does not admit some of its keys (an item's last tile: the diagonal's, or one that
            // reaches behind the sequence's end).
            auto tile = [&](auto masked, int j) -> bool {
                if (!mbar_wait_warp(BAR(S_FULL + t), jg & 1, kWaitLimitNs)) return false;
                tc_fence_after();
                // S_t and its row max over the admitted keys: each 32-column piece's max comes with the load; a masked tile takes
                // the max again over the admitted ones
                float s[kTile], mt;
                int pieces = 4;  // with keys that some row of this warp admits
                {
                    float pm[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + c * 32, *reinterpret_cast<float(*)[32]>(&s[c * 32]), pm[c]);
                    tmem_wait_ld();
                    mt = fmax3(fmaxf(pm[0], pm[1]), pm[2], pm[3]);
                }
                if constexpr (decltype(masked)::value) {
                    const int k0 = j * kTile, hi = (CAUSAL ? min(w.len - 1, row0 + row) : w.len - 1) - k0;
                    pieces = min(((CAUSAL ? min(w.len - 1, row0 + (warp & 3) * 32 + 31) : w.len - 1) - k0) / 32 + 1, 4);
#pragma unroll
                    for (int i = 0; i < kTile; ++i)
                        if (i > hi) s[i] = -INFINITY;
                    mt = row_max(s);
                }
                const float m_new = fmaxf(m_ref, mt);
                const bool need = (m_new - m_ref) * c_u > kRescaleLog2;  // true while m_ref = -inf
                float alpha = 1.f;
                if (need) {
                    alpha = ex2((m_ref - m_new) * c_u);  // 0 on the first tile
                    m_ref = m_new;
                }
                const float mc = (m_ref == -INFINITY ? 0.f : m_ref) * c_u;
                // d = 128: O is divided by lr, the sum of the rounded P wherever one key can carry the row: the exact
                // rounded sum is taken in "heavy" tiles, where the tile's largest P exceeds kHeavyShare of the row's running sum;
                // over many comparable keys the roundings average out and the fp32 sum serves.  (d = 64: column 64 of O.)  Lanes
                // behind the sequence's end have no say: what lies there is another's.
                [[maybe_unused]] bool heavy = false;
                if constexpr (!C::kOnesCol) heavy = __any_sync(0xffffffffu, mine && ex2(fmaf(mt, c_u, -mc)) > kHeavyShare * (l * alpha));
                const float2 c2 = make_float2(c_u, c_u), nmc2 = make_float2(-mc, -mc);
                float2 lf[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
                    if (!decltype(masked)::value || c < pieces) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = fma2(make_float2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), c2, nmc2);
                            const float p0 = ex2(x.x), p1 = ex2(x.y);
                            p[i] = pack_bf16x2(p0, p1);
                            lf[c] = add2(lf[c], make_float2(p0, p1));
                        }
                    } else {  // (the product reads P up to the sequence's end; causal that is behind this warp's rows)
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[i] = 0;
                    }
                    tmem_st16(tS + c * 16, p);
                }
                const float2 lfs = add2(add2(lf[0], lf[1]), add2(lf[2], lf[3]));
                if constexpr (!C::kOnesCol) {
                    float add = lfs.x + lfs.y;
                    if (heavy) {
                        float lq[4] = {0.f, 0.f, 0.f, 0.f};
                        tmem_wait_st();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r[32];
                            tmem_ld32(tS + h * 32, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) lq[i & 3] = add_bf16x2(lq[i & 3], r[i]);
                        }
                        add = (lq[0] + lq[1]) + (lq[2] + lq[3]);
                    }
                    lr = lr * alpha + add;
                }
                l = l * alpha + (lfs.x + lfs.y);
                // the numerator rescaled (it holds P V up to the tile before: that product was issued ahead of this S)
                if (j > j0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t r[32];
                        tmem_ld32(tO + c * 32, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y = mul2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(alpha, alpha));
                            r[i] = __float_as_uint(y.x);
                            r[i + 1] = __float_as_uint(y.y);
                        }
                        tmem_st32(tO + c * 32, r);
                    }
                    if constexpr (C::kOnesCol) {
                        const float lc = __uint_as_float(tmem_ld1(tO + 64));
                        tmem_wait_ld();
                        tmem_st1(tO + 64, __float_as_uint(lc * alpha));
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(P_FULL + t));
                ++jg;
                return true;
            };
            const int plain = n_mine - (CAUSAL || n_mine * kTile > w.len ? 1 : 0);
            for (int j = j0; j < min(plain, j1) && ok; ++j) ok = tile(std::false_type{}, j);
            if (ok && plain < j1) ok = tile(std::true_type{}, plain);
            if (!ok || !(ok = mbar_wait_warp(BAR(O_FULL + t), uc & 1, kWaitLimitNs))) break;
            tc_fence_after();
            // O = u / lr in bf16, LSE from the fp32 sum.  The next item's first product over O_t is issued only after this
            // warpgroup's next arrive, so the reads here are safe.
            if constexpr (C::kOnesCol) {
                lr = __uint_as_float(tmem_ld1(tO + 64));
                tmem_wait_ld();
            }
            if constexpr (SHARED) {
                any = true;
                continue;
            }
            const float inv_l = lr > 0.f ? 1.f / lr : 0.f;
            const int head = tile_head<PAIR>(w, t), wrow = row0 + (warp & 3) * 32;  // this warp's first row
            const bool whole = wrow + 32 <= w.len;
            const uint32_t stage = sb + C::kStage + warp * 4096;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {  // 64 columns at a time: two pieces of 32 rows of 64 bytes
                uint32_t r[2][32];
                tmem_ld32(tO + c * 64, r[0]);
                tmem_ld32(tO + c * 64 + 32, r[1]);
                if (lane == 0) bulk_wait_read0();  // (what was stored before has left the staging buffers)
                tmem_wait_ld();
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 y[4];
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        const uint32_t *x = r[u] + q4 * 8;
                        y[q4].x = pack_bf16x2(__uint_as_float(x[0]) * inv_l, __uint_as_float(x[1]) * inv_l);
                        y[q4].y = pack_bf16x2(__uint_as_float(x[2]) * inv_l, __uint_as_float(x[3]) * inv_l);
                        y[q4].z = pack_bf16x2(__uint_as_float(x[4]) * inv_l, __uint_as_float(x[5]) * inv_l);
                        y[q4].w = pack_bf16x2(__uint_as_float(x[6]) * inv_l, __uint_as_float(x[7]) * inv_l);
                    }
                    if (whole) {  // in the 64-byte swizzle
                        const uint32_t buf = stage + u * 2048 + lane * 64;
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) st_shared_v4(buf + ((q4 ^ ((lane >> 1) & 3)) << 4), y[q4]);
                    } else if (mine) {
                        uint4 *to = reinterpret_cast<uint4 *>(packed_row(a.o, w.start + row0 + row, head) + c * 64 + u * 32);
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) to[q4] = y[q4];
                    }
                }
                if (whole) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&tm_o, stage, c * 64, w.start + wrow, head);
                        tma_store_3d(&tm_o, stage + 2048, c * 64 + 32, w.start + wrow, head);
                        bulk_commit();
                    }
                }
            }
            if (mine) a.lse[static_cast<int64_t>(head) * a.T + w.start + row0 + row] = l > 0.f ? m_ref * a.scale + logf(l) : -INFINITY;
            ++uc;
        }
        if (!ok) packed_timeout();
        if (lane == 0) bulk_wait0();  // every O store of this warp has completed
        if constexpr (SHARED) {
            // the sums and the unnormalised O where K and V were, once both tiles' products have read them: [tile][row][d] fp32, 16-byte
            // pieces at piece ^ (row mod 8)
            __syncwarp();
            asm volatile("barrier.cta.sync 1, 256;\n" ::: "memory");
            reinterpret_cast<float4 *>(smem + C::kStage)[tid] = any ? make_float4(m_ref, l, lr, 0.f) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            if (any) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld32(tO + c * 32, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(smem + C::kRing + tid * (D * 4) + (((c * 8 + i) ^ (row & 7)) << 4)) =
                            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                }
            }
        }
    }
    if constexpr (SHARED) {
        __syncwarp();
        cluster_sync();
        Items again(PAIR ? a.plan.blocks : a.plan.pairs, n_items, a.units, gridDim.x / ranks, blockIdx.x / ranks);
        if (warp < kLoadWarp && again.take<PAIR>(w)) {
            // each CTA takes its part of the item's 8-column pieces
            constexpr int kPieces = 2 * kTile * D / 8;
            for (int i = kPieces * rank / ranks + tid; i < kPieces * (rank + 1) / ranks; i += 256) {
                const int c = i % (D / 8), at = i / (D / 8), t = at / kTile, row = tile_row<PAIR>(w, t) + at % kTile, head = tile_head<PAIR>(w, t);
                if (row >= w.len) continue;
                float m = -INFINITY;
                for (int other = 0; other < ranks; ++other) m = fmaxf(m, ld_cluster_v4(sb + C::kStage + at * 16, other).x);
                float l = 0.f, lr = 0.f;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                const uint32_t from = sb + C::kRing + at * (D * 4), p0 = ((2 * c) ^ (at & 7)) << 4, p1 = ((2 * c + 1) ^ (at & 7)) << 4;
                for (int other = 0; other < ranks; ++other) {
                    const float4 part = ld_cluster_v4(sb + C::kStage + at * 16, other);
                    if (part.y == 0.f) continue;  // no keys of this row
                    const float4 u = ld_cluster_v4(from + p0, other), v = ld_cluster_v4(from + p1, other);
                    const float f = ex2((part.x - m) * a.scale_log2);
                    l = fmaf(f, part.y, l);
                    lr = fmaf(f, part.z, lr);
                    x = make_float4(fmaf(f, u.x, x.x), fmaf(f, u.y, x.y), fmaf(f, u.z, x.z), fmaf(f, u.w, x.w));
                    y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
                }
                const float inv = lr > 0.f ? 1.f / lr : 0.f;
                reinterpret_cast<uint4 *>(packed_row(a.o, w.start + row, head))[c] =
                    make_uint4(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv), pack_bf16x2(y.x * inv, y.y * inv),
                               pack_bf16x2(y.z * inv, y.w * inv));
                if (c == 0) a.lse[static_cast<int64_t>(head) * a.T + w.start + row] = l > 0.f ? m * a.scale + logf(l) : -INFINITY;
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA ends while others read its shared memory
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool CAUSAL, bool PAIR, bool SHARED>
cudaError_t launch(const FaPackedProblem &p, int ranks, cudaStream_t stream)
{
    using C = PCfg<D>;
    CUtensorMap mq, mk, mv, mo;
    if (!make_rows_map(&mq, p.q, p.T, p.H, D) || !make_rows_map(&mk, p.k, p.T, p.Hkv, D) ||
        !make_rows_map(&mv, p.v, p.T, p.Hkv, D) || !make_rows_map(&mo, p.o, p.T, p.H, D, true))
        return cudaErrorInvalidValue;
    const cudaError_t e = set_max_dynamic_smem<fa_packed_fwd_kernel<D, CAUSAL, PAIR, SHARED>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    FwdArgs a;
    a.plan = plan_view(p.plan, p.B, p.T);
    a.o = p.o;
    a.lse = p.lse;
    a.T = static_cast<int>(p.T);
    a.B = static_cast<int>(p.B);
    a.heads = static_cast<int>(p.H);
    a.units = static_cast<int>(PAIR ? p.H / 2 : p.H);
    a.group = static_cast<int>(p.H / p.Hkv);
    a.fill = p.fill;
    a.ranks = ranks;
    a.scale = p.scale;
    a.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    const int64_t most = (p.T / (PAIR ? 128 : 256) + p.B) * a.units;  // items, whatever the lengths are
    const int64_t grid = SHARED ? most * ranks : most < p.sm_count ? most : p.sm_count;
    auto kern = fa_packed_fwd_kernel<D, CAUSAL, PAIR, SHARED>;
    if constexpr (SHARED)
        return launch_with(kern, static_cast<unsigned>(grid), kThreads, C::kSmemBytes, stream, static_cast<unsigned>(ranks), false, mq, mk,
                           mv, mo, a);
    kern<<<static_cast<unsigned>(grid), kThreads, C::kSmemBytes, stream>>>(mq, mk, mv, mo, a);
    return cudaGetLastError();
}

template <int D, bool SHARED>
cudaError_t launch_d(const FaPackedProblem &p, int ranks, cudaStream_t s)
{
    if (p.H / p.Hkv % 2 == 0) return p.causal ? launch<D, true, true, SHARED>(p, ranks, s) : launch<D, false, true, SHARED>(p, ranks, s);
    return p.causal ? launch<D, true, false, SHARED>(p, ranks, s) : launch<D, false, false, SHARED>(p, ranks, s);
}

// How many CTAs share an item's key tiles: long loops of few items leave SMs idle, but joining them costs as much as 8 tiles.
// Measured (us, d = 128, one sequence, causal; 1, 2, 3 and 4 CTAs): 4096 rows, 4 heads on 4 (64 items) 54, 39, 45, 43; 12000, 3 on 1
// (141) 146, 99, 135, 135; 2048, 8 on 1 (64) 30, 27, 39, 37; 4096, 16 on 2 (256) 56, 102, 147, 164.
int ranks_of(const FaPackedProblem &p)
{
    const bool pair = p.H / p.Hkv % 2 == 0;
    const int64_t mean = (p.T / p.B + kTile - 1) / kTile, tiles = mean > 0 ? mean : 1;
    const int64_t n = p.B * (pair ? tiles * (p.H / 2) : (tiles + 1) / 2 * p.H);
    // (several sequences: their lengths differ as a rule, and the longest counts; causal it is taken for 2.5 times the mean.  5 of 50 to
    // 12000, 2 heads on 2, d = 64: 2 CTAs 64 us, 1 CTA 107; 3 of 100 to 8000, 4 on 2, d = 64: 55 and 74.  With 3 times 4 of 2048, 4
    // on 2, would take 42 in place of 31.)
    const double longest = static_cast<double>(tiles) * (p.B > 1 && p.causal ? 2.5 : 1);
    return cluster_ranks(static_cast<double>(n), longest, 1, 1, 8, p.causal);
}

}  // namespace

cudaError_t fa_launch_packed_fwd(const FaPackedProblem &p, cudaStream_t stream)
{
    const int ranks = ranks_of(p);
    if (ranks > 1) return p.d == 64 ? launch_d<64, true>(p, ranks, stream) : launch_d<128, true>(p, ranks, stream);
    return p.d == 64 ? launch_d<64, false>(p, 1, stream) : launch_d<128, false>(p, 1, stream);
}

int fa_packed_fwd_take_status(cudaStream_t stream) { return fa_take_status_word(g_packed_status, stream); }
