// Exact attention backward of packed sequences with grouped heads (fa_bwd_packed): TMA + tcgen05 + TMEM.
//
// Per sequence, with P = exp(scale q k^T - LSE) recomputed from the saved LSE and D_i = dO_i . O_i:
//   dV_j = sum over the key head's query heads and rows i of P_ij dO_i
//   dS_ij = P_ij (dO_i . v_j - D_i),   dQ_i = scale sum_j dS_ij k_j,   dK_j = scale sum dS_ij q_i
//
// Three launches, as in fa_bwd_tc.cu, whose pipeline the main one is:
//   pre   D and LSE log2 e of every row, in vectors padded to whole blocks of 128 rows (+inf and 0 behind a sequence's
//         end, so that P is 0 there); the fp32 dQ accumulator zeroed
//   main  a CTA per 128 keys of one key head of one sequence, the longest loops first (the plan's list), over the 128-row
//         query blocks (causal: from the diagonal) of each of the key head's query heads in turn: dK and dV, which
//         sum over those heads, stay in tensor memory through all of it; each block's part of dQ is added to
//         the accumulator by one bulk reduction
//   post  dQ = bf16(scale accumulator); zeros in rows of no sequence where they are asked for
// Per query block (S^T etc. are key-major: TMEM lane = key):
//   S^T  = K Q^T      SS product -> TMEM A
//   dP^T = V dO^T     SS product -> TMEM B
//   P^T  = exp2(S^T scale log2 e - LSE log2 e)   softmax warps, bf16 back into A
//   dV  += P^T dO     A from TMEM, B = dO MN-major -> TMEM C
//   dS^T = P^T (dP^T - D)                        softmax warps, bf16 into B and into shared memory
//   dK  += dS^T Q     A from TMEM -> TMEM D
//   dQ   = dS K       A = dS MN-major, B = K MN-major -> TMEM A, read into registers, staged in the Q / dO stage that the
//                     block no longer needs, and added to the accumulator by the load warp
// The accumulator is blocked: a 128 x d fp32 block per (query head, block), as the 8 warps' slices (warpgroup, 32
// rows) one behind the other, each 32 rows x d/2 columns with the 16-byte piece c of row l at piece c ^ (l mod d/8).
//
// A 128-row tile that reaches behind its sequence holds rows of others.  Sums over rows (dV, dK over queries, dQ over
// keys) step 16 rows at a time and end behind the sequence's last one; of that step the rows behind are made zeros in
// Q, dO, K and V (zero_tail_rows), so that their P, dP and dS are zeros too, whatever the tile held.  Rows past that
// step are lanes and columns of results that nothing reads.
// Roles (320 threads): warps 0-3 and 4-7 are two warpgroups that take query columns 0-63 and 64-127 of a block (and halves
// of dQ's, dK's and dV's columns); warp 8 loads; warp 9 issues the products and owns the tensor memory.
// Every mbarrier wait is bounded; a wait that gives up sets FA_ERR_TIMEOUT and the CTA winds down.
#include <math.h>

#include "fa_packed.cuh"

using namespace sm100;

namespace {

constexpr int kBlock = 128;  // keys per CTA, rows of a query block
constexpr int kThreads = 320;
constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr uint64_t kCleanupLimitNs = 20000000ull;

template <int D>
struct BCfg {
    static constexpr int kTile = kBlock * D * 2;
    static constexpr int kAtoms = D / 64;
    static constexpr int kK = 0;
    static constexpr int kV = kTile;
    static constexpr int kStage0 = 2 * kTile;  // stage s: Q at kStage0 + s * kStageBytes, dO behind it
    static constexpr int kStageBytes = 2 * kTile;
    static constexpr int kDS = kStage0 + 2 * kStageBytes;   // dS, 128 keys x 128 queries bf16, MN-major
    static constexpr int kVec = kDS + kBlock * kBlock * 2;  // per stage: LSE log2 e (512 B), D (512 B)
    static constexpr int kBar = kVec + 2 * 1024;
    static constexpr int kNumBars = 13;
    static constexpr int kSmemBytes = kBar + kNumBars * 8 + 16;
    static_assert(kSmemBytes <= 232448, "shared memory plan exceeds 227 KB");
};

enum { KV_FULL = 0, Q_FULL = 1, DQ_STAGED = 3, S_FULL = 5, DP_FULL = 6, P_READY = 7, DS_READY = 8, DQ_FULL = 9,
       DQ_CONSUMED = 10, DONE = 11, MMA_DONE = 12 };

struct BwdArgs {
    PlanView plan;
    FaRows dk, dv, dq, o, dout;
    const float *lse;               // [H][T]
    float *lse2, *dvec, *dq_acc;    // [H][nb * 128], the same, [H][nb][128 * D]
    int T, B, heads, kv_heads, group, fill;
    int nb;                         // blocks that the padded arrays have room for
    int heads_per_group;            // see the order of the CTAs
    float scale, scale_log2;
};

__device__ __forceinline__ uint32_t lo32(uint64_t x) { return static_cast<uint32_t>(x); }
__device__ __forceinline__ uint32_t hi32(uint64_t x) { return static_cast<uint32_t>(x >> 32); }

// TMEM column of the packed (bf16 pairs) 16-query step kk: warpgroup w packs its 64 queries into columns [64 w, 64 w + 32).
__device__ __forceinline__ uint32_t packed_col(int kk) { return kk < 4 ? kk * 8 : 64 + (kk - 4) * 8; }

template <int D, bool CAUSAL>
__global__ void __launch_bounds__(kThreads, 1)
fa_packed_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdArgs a)
{
    using C = BCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The grid has a CTA for every block that the lengths could make; those past the list end here, and all do for a plan
    // of another batch (which the pre kernel reports).
    if (!plan_fits(a.plan.head, a.T, a.B, CAUSAL)) return;
    const int n_blocks = a.plan.head->n_blocks;
    // The key heads go in groups, so that the CTAs resident at one time share a few heads' Q, dO and dQ blocks in L2; inside
    // a group the list's order, the longest loops first.
    const int64_t per_group = static_cast<int64_t>(a.heads_per_group) * n_blocks;
    if (blockIdx.x >= static_cast<int64_t>(a.kv_heads) * n_blocks) return;
    if ((sb & 1023u) != 0) {  // the swizzled tiles need a 1024-byte-aligned base
        if (tid == 0) packed_timeout();
        return;
    }
    const int grp = static_cast<int>(blockIdx.x / per_group), rem = static_cast<int>(blockIdx.x - grp * per_group);
    const int gsize = min(a.heads_per_group, a.kv_heads - grp * a.heads_per_group);
    const int kvh = grp * a.heads_per_group + rem % gsize;
    const int4 entry = a.plan.blocks[rem / gsize];
    const int start = entry.x, len = entry.y, blk0 = entry.w;
    const int n_seq = (len + kBlock - 1) / kBlock;
    // entries hold the number of a query block whose loop over keys is as long as this key block's over queries
    const int kb = CAUSAL ? n_seq - 1 - entry.z : entry.z;
    const int k0 = kb * kBlock, qb0 = CAUSAL ? kb : 0, nq = n_seq - qb0;
    const int n_it = nq * a.group;  // query blocks of all of the key head's query heads
    const int q_left = len - (n_seq - 1) * kBlock;           // rows of the sequence's last block
    const int k_rows = min(kBlock, len - k0);                // keys of this block
    const uint32_t bar0 = sb + C::kBar;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBar + C::kNumBars * 8);

    if (tid == 0) {
        mbar_init(BAR(KV_FULL), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(BAR(Q_FULL + s), 1);
            mbar_init(BAR(DQ_STAGED + s), 8);  // the softmax warps, once their dQ slices are staged
        }
        mbar_init(BAR(S_FULL), 1);
        mbar_init(BAR(DP_FULL), 1);
        mbar_init(BAR(P_READY), 8);
        mbar_init(BAR(DS_READY), 8);
        mbar_init(BAR(DQ_FULL), 1);
        mbar_init(BAR(DQ_CONSUMED), 8);
        mbar_init(BAR(DONE), 1);
        mbar_init(BAR(MMA_DONE), 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // (one thread asks: the status may change while a block starts, and its roles have to agree)
    if (tid == 0) tmem_slot[1] = *reinterpret_cast<volatile int *>(&g_packed_status) != FA_ERR_TIMEOUT;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool run = tmem_slot[1] != 0;  // no wait has given up that nobody has read so yet
    const uint32_t tA = tmem, tB = tmem + 128, tC = tmem + 256, tD = tmem + 384;

    if (!run) {
        // nothing to do
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            prefetch_tmap(&tm_do);
            mbar_arrive_expect_tx(BAR(KV_FULL), 2 * C::kTile);
            for (int c = 0; c < C::kAtoms; ++c) {
                tma_load_3d(sb + C::kK + c * 16384, &tm_k, BAR(KV_FULL), c * 64, start + k0, kvh);
                tma_load_3d(sb + C::kV + c * 16384, &tm_v, BAR(KV_FULL), c * 64, start + k0, kvh);
            }
            // (query head, block) of iteration i
            auto place = [&](int i, int &h, int &qb) {
                h = kvh * a.group + i / nq;
                qb = qb0 + i % nq;
            };
            // add the dQ block that iteration j staged in stage j & 1 to the accumulator
            auto flush = [&](int j) -> bool {
                if (!mbar_wait(BAR(DQ_STAGED + (j & 1)), (j >> 1) & 1, kWaitLimitNs)) return false;
                int h, qb;
                place(j, h, qb);
                bulk_reduce_add_f32(a.dq_acc + (static_cast<int64_t>(h) * a.nb + blk0 + qb) * (kBlock * D),
                                    sb + C::kStage0 + (j & 1) * C::kStageBytes, kBlock * D * 4);
                bulk_commit();
                return true;
            };
            bool ok = true;
            int issued = 0;
            for (int i = 0; i < n_it; ++i) {
                const int st = i & 1;
                if (i >= 2) {  // the stage is free once the block staged in it two iterations ago is read out
                    if (!(ok = flush(i - 2))) break;
                    bulk_wait_read0();
                }
                int h, qb;
                place(i, h, qb);
                const int row = start + qb * kBlock;
                const uint32_t sq = sb + C::kStage0 + st * C::kStageBytes, sdo = sq + C::kTile;
                mbar_arrive_expect_tx(BAR(Q_FULL + st), 2 * C::kTile + 1024);
                for (int c = 0; c < C::kAtoms; ++c) {
                    tma_load_3d(sq + c * 16384, &tm_q, BAR(Q_FULL + st), c * 64, row, h);
                    tma_load_3d(sdo + c * 16384, &tm_do, BAR(Q_FULL + st), c * 64, row, h);
                }
                const int64_t vo = (static_cast<int64_t>(h) * a.nb + blk0 + qb) * kBlock;
                bulk_load(sb + C::kVec + st * 1024, a.lse2 + vo, 512, BAR(Q_FULL + st));
                bulk_load(sb + C::kVec + st * 1024 + 512, a.dvec + vo, 512, BAR(Q_FULL + st));
                ++issued;
            }
            for (int j = n_it >= 2 ? n_it - 2 : 0; j < n_it && ok; ++j) ok = flush(j);
            bulk_wait0();  // the accumulator additions complete before the CTA ends
            if (!ok) packed_timeout();
            const uint64_t lim = ok ? kWaitLimitNs : kCleanupLimitNs;
            mbar_wait(BAR(KV_FULL), 0, lim);
            for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i) mbar_wait(BAR(Q_FULL + (i & 1)), (i >> 1) & 1, lim);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------- products
        constexpr uint32_t idS = idesc_bf16_f32(kBlock, kBlock, false);   // S^T, dP^T: K-major operands
        constexpr uint32_t idAcc = idesc_bf16_f32(kBlock, D, true);       // dV, dK: A in TMEM, B MN-major
        constexpr uint32_t idQ = idesc_bf16_f32(kBlock, D, true, true);   // dQ: A and B MN-major
        constexpr uint32_t kStage16 = C::kStageBytes >> 4, kTile16 = C::kTile >> 4;
        const uint64_t d_k_kmaj = smem_desc_sw128(sb + C::kK, 16, 1024);
        const uint64_t d_v_kmaj = smem_desc_sw128(sb + C::kV, 16, 1024);
        const uint64_t d_k_mn = smem_desc_sw128(sb + C::kK, 16384, 1024);
        const uint64_t d_ds_mn = smem_desc_sw128(sb + C::kDS, 16384, 1024);
        const uint64_t d_q_kmaj = smem_desc_sw128(sb + C::kStage0, 16, 1024);
        const uint64_t d_q_mn = smem_desc_sw128(sb + C::kStage0, 16384, 1024);
        const int k_steps = (k_rows + 15) / 16, tail_steps = (q_left + 15) / 16;
        bool ok = mbar_wait_warp(BAR(KV_FULL), 0, kWaitLimitNs);
        if (ok && (k_rows & 15)) {
            zero_tail_rows<D>(smem + C::kK, k_rows, lane);
            zero_tail_rows<D>(smem + C::kV, k_rows, lane);
            fence_proxy_async_smem();
            __syncwarp();
        }
        int block = 0;  // of the query head's nq
        for (int i = 0; i < n_it && ok; ++i) {
            const int st = i & 1;
            if (!(ok = mbar_wait_warp(BAR(Q_FULL + st), (i >> 1) & 1, kWaitLimitNs))) break;
            const bool tail = ++block == nq;
            if (tail) {
                block = 0;
                if (q_left & 15) {
                    zero_tail_rows<D>(smem + C::kStage0 + st * C::kStageBytes, q_left, lane);
                    zero_tail_rows<D>(smem + C::kStage0 + st * C::kStageBytes + C::kTile, q_left, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            const int q_steps = tail ? tail_steps : kBlock / 16;
            if (i > 0 && !(ok = mbar_wait_warp(BAR(DQ_CONSUMED), (i - 1) & 1, kWaitLimitNs))) break;
            tc_fence_after();
            const uint32_t q_lo = lo32(d_q_kmaj) + st * kStage16, do_lo = q_lo + kTile16;
            const uint32_t qmn_lo = lo32(d_q_mn) + st * kStage16, domn_lo = qmn_lo + kTile16;
            // S^T = K Q^T and dP^T = V dO^T
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t koff = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                    mma_ss_lohi(tA, lo32(d_k_kmaj) + koff, hi32(d_k_kmaj), q_lo + koff, hi32(d_q_kmaj), idS, kk > 0 ? 1u : 0u);
                }
                mma_commit(BAR(S_FULL));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t koff = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                    mma_ss_lohi(tB, lo32(d_v_kmaj) + koff, hi32(d_v_kmaj), do_lo + koff, hi32(d_q_kmaj), idS, kk > 0 ? 1u : 0u);
                }
                mma_commit(BAR(DP_FULL));
            }
            __syncwarp();
            // dV += P^T dO
            if (!(ok = mbar_wait_warp(BAR(P_READY), i & 1, kWaitLimitNs))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    if (kk < q_steps)
                        mma_ts_lohi(tC, tA + packed_col(kk), domn_lo + kk * 128, hi32(d_q_mn), idAcc, (i > 0 || kk > 0) ? 1u : 0u);
            }
            __syncwarp();
            // dK += dS^T Q, then dQ = dS K
            if (!(ok = mbar_wait_warp(BAR(DS_READY), i & 1, kWaitLimitNs))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    if (kk < q_steps)
                        mma_ts_lohi(tD, tB + packed_col(kk), qmn_lo + kk * 128, hi32(d_q_mn), idAcc, (i > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    if (kk < k_steps)
                        mma_ss_lohi(tA, lo32(d_ds_mn) + kk * 128, hi32(d_ds_mn), lo32(d_k_mn) + kk * 128, hi32(d_k_mn), idQ,
                                    kk > 0 ? 1u : 0u);
                mma_commit(BAR(DQ_FULL));
            }
            __syncwarp();
        }
        if (!ok && lane == 0) packed_timeout();
        if (elect_one()) {
            if (ok) mma_commit(BAR(DONE));
            mma_commit(BAR(MMA_DONE));
        }
        __syncwarp();
        mbar_wait_warp(BAR(MMA_DONE), 0, ok ? kWaitLimitNs : kCleanupLimitNs);
    } else {
        // ------------------------------------------------ softmax-side warpgroups
        const int wg = warp >> 2;              // query columns [64 wg, 64 wg + 64); d columns [wg D/2, (wg + 1) D/2)
        const int r = (warp & 3) * 32 + lane;  // TMEM lane
        const uint32_t loff = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int key = k0 + r;
        bool ok = true;
        int block = 0;
        for (int i = 0; i < n_it && ok; ++i) {
            const int st = i & 1;
            const int q0 = (qb0 + block) * kBlock;
            const bool diagonal = CAUSAL && block == 0;
            if (++block == nq) block = 0;
            if (!mbar_wait_warp(BAR(Q_FULL + st), (i >> 1) & 1, kWaitLimitNs) || !mbar_wait_warp(BAR(S_FULL), i & 1, kWaitLimitNs)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float *lse2_s = reinterpret_cast<const float *>(smem + C::kVec + st * 1024) + wg * 64;
            const float *d_s = lse2_s + kBlock;
            // P^T = exp2(S^T scale log2 e - LSE log2 e); 0 for keys behind the sequence and, causal, keys after the query
            float p[64];
            {
                uint32_t a0[32], a1[32];
                tmem_ld32(tA + loff + wg * 64, a0);
                tmem_ld32(tA + loff + wg * 64 + 32, a1);
                tmem_wait_ld();
                const float2 sl = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 l0 = *reinterpret_cast<const float2 *>(lse2_s + j);
                    const float2 l1 = *reinterpret_cast<const float2 *>(lse2_s + 32 + j);
                    const float2 x0 = fma2(make_float2(__uint_as_float(a0[j]), __uint_as_float(a0[j + 1])), sl, make_float2(-l0.x, -l0.y));
                    const float2 x1 = fma2(make_float2(__uint_as_float(a1[j]), __uint_as_float(a1[j + 1])), sl, make_float2(-l1.x, -l1.y));
                    p[j] = ex2(x0.x);
                    p[j + 1] = ex2(x0.y);
                    p[32 + j] = ex2(x1.x);
                    p[32 + j + 1] = ex2(x1.y);
                }
            }
            if (key >= len) {
#pragma unroll
                for (int j = 0; j < 64; ++j) p[j] = 0.f;
            } else if (diagonal) {
                const int qb = q0 + wg * 64;  // query qb + j admits key iff key <= qb + j
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (key > qb + j) p[j] = 0.f;
            }
            {
                uint32_t pk[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(p[h * 32 + 2 * j], p[h * 32 + 2 * j + 1]);
                    tmem_st16(tA + loff + wg * 64 + h * 16, pk);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(P_READY));

            // dS^T = P^T (dP^T - D)
            if (!mbar_wait_warp(BAR(DP_FULL), i & 1, kWaitLimitNs)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t dsk[32];
            {
                uint32_t b0[32], b1[32];
                tmem_ld32(tB + loff + wg * 64, b0);
                tmem_ld32(tB + loff + wg * 64 + 32, b1);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 dd0 = *reinterpret_cast<const float2 *>(d_s + j);
                    const float2 dd1 = *reinterpret_cast<const float2 *>(d_s + 32 + j);
                    dsk[j / 2] = pack_bf16x2(p[j] * (__uint_as_float(b0[j]) - dd0.x), p[j + 1] * (__uint_as_float(b0[j + 1]) - dd0.y));
                    dsk[16 + j / 2] = pack_bf16x2(p[32 + j] * (__uint_as_float(b1[j]) - dd1.x),
                                                  p[32 + j + 1] * (__uint_as_float(b1[j + 1]) - dd1.y));
                }
            }
            {
                uint32_t h0[16], h1[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    h0[j] = dsk[j];
                    h1[j] = dsk[16 + j];
                }
                tmem_st16(tB + loff + wg * 64, h0);
                tmem_st16(tB + loff + wg * 64 + 16, h1);
            }
            // dS^T's row (this key) into the MN-major dS tile: column block wg, 16-byte piece c (queries 8c .. 8c+7) at
            // piece c ^ (key row mod 8)
            uint8_t *row_base = smem + C::kDS + wg * 16384 + r * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4 *>(row_base + ((c ^ (r & 7)) * 16)) =
                    make_uint4(dsk[4 * c], dsk[4 * c + 1], dsk[4 * c + 2], dsk[4 * c + 3]);
            fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(DS_READY));

            // this block's part of dQ (TMEM lane = query row): into registers, TMEM A released, then staged in this
            // block's Q / dO stage (every product that read it has completed by DQ_FULL) for the load warp's reduction
            if (!mbar_wait_warp(BAR(DQ_FULL), i & 1, kWaitLimitNs)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t x0[32], x1[32];
            tmem_ld32(tA + loff + wg * (D / 2), x0);
            if constexpr (D == 128) tmem_ld32(tA + loff + wg * (D / 2) + 32, x1);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(DQ_CONSUMED));
            constexpr int kPieces = D / 8;  // of 16 bytes, in a row of the warp's slice
            constexpr int kSliceBytes = 32 * (D / 2) * 4;
            const int slot = wg * 4 + (warp & 3);
            uint8_t *srow = smem + C::kStage0 + st * C::kStageBytes + slot * kSliceBytes + lane * (D * 2);
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const uint32_t *x = c < 8 ? x0 : x1;
                const int cl = c & 7;
                *reinterpret_cast<uint4 *>(srow + ((c ^ (lane & (kPieces - 1))) * 16)) =
                    make_uint4(x[4 * cl], x[4 * cl + 1], x[4 * cl + 2], x[4 * cl + 3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(DQ_STAGED + st));
        }
        if (ok) ok = mbar_wait_warp(BAR(DONE), 0, kWaitLimitNs);
        if (!ok) packed_timeout();
        tc_fence_after();
        // dV (TMEM C) and scale dK (TMEM D), this warpgroup's half of the columns; every lane takes part in the loads
        if (ok) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const uint32_t tsrc = (which == 0 ? tC : tD) + loff + wg * (D / 2);
                const float mul = which == 0 ? 1.f : a.scale;
                __nv_bfloat16 *out = packed_row(which == 0 ? a.dv : a.dk, start + key, kvh) + wg * (D / 2);
#pragma unroll
                for (int cc = 0; cc < D / 64; ++cc) {
                    uint32_t x[32];
                    tmem_ld32(tsrc + cc * 32, x);
                    tmem_wait_ld();
                    if (key >= len) continue;
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint4 v4;
                        v4.x = pack_bf16x2(__uint_as_float(x[8 * q4 + 0]) * mul, __uint_as_float(x[8 * q4 + 1]) * mul);
                        v4.y = pack_bf16x2(__uint_as_float(x[8 * q4 + 2]) * mul, __uint_as_float(x[8 * q4 + 3]) * mul);
                        v4.z = pack_bf16x2(__uint_as_float(x[8 * q4 + 4]) * mul, __uint_as_float(x[8 * q4 + 5]) * mul);
                        v4.w = pack_bf16x2(__uint_as_float(x[8 * q4 + 6]) * mul, __uint_as_float(x[8 * q4 + 7]) * mul);
                        *reinterpret_cast<uint4 *>(out + cc * 32 + 8 * q4) = v4;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// D_i = dO_i . O_i and LSE_i log2 e of every row of every block (0 and +inf behind a sequence's end); the block's dQ
// accumulator zeroed.  A block of threads per 128 rows of a head, two rows a warp at a time.  Memory-bound.
template <int D>
__global__ void __launch_bounds__(256)
fa_packed_pre_kernel(const BwdArgs a, int causal)
{
    constexpr int TPR = D / 8;  // threads a row, 8 channels each
    if (!plan_fits(a.plan.head, a.T, a.B, causal)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) packed_bad_sequence();
        return;
    }
    const int t = threadIdx.x % TPR, r0 = threadIdx.x / TPR;
    const int64_t n = static_cast<int64_t>(a.plan.head->n_blocks) * a.heads;
    for (int64_t it = blockIdx.x; it < n; it += gridDim.x) {
        const int4 e = a.plan.blocks[it / a.heads];
        const int h = static_cast<int>(it % a.heads);
        const int64_t block = static_cast<int64_t>(h) * a.nb + e.w + e.z;
#pragma unroll 4
        for (int r = r0; r < kBlock; r += 256 / TPR) {
            const int row = e.z * kBlock + r;
            float acc = 0.f;
            if (row < e.y) {
                const uint4 x = reinterpret_cast<const uint4 *>(packed_row(a.o, e.x + row, h))[t];
                const uint4 y = reinterpret_cast<const uint4 *>(packed_row(a.dout, e.x + row, h))[t];
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc = fmaf(__uint_as_float(xs[c] << 16), __uint_as_float(ys[c] << 16), acc);
                    acc = fmaf(__uint_as_float(xs[c] & 0xFFFF0000u), __uint_as_float(ys[c] & 0xFFFF0000u), acc);
                }
            }
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (t == 0) {
                a.dvec[block * kBlock + r] = acc;
                a.lse2[block * kBlock + r] = row < e.y ? a.lse[static_cast<int64_t>(h) * a.T + e.x + row] * 1.4426950408889634f : INFINITY;
            }
        }
        float4 *z = reinterpret_cast<float4 *>(a.dq_acc + block * (kBlock * D));
#pragma unroll 8
        for (int i = threadIdx.x; i < kBlock * D / 4; i += 256) z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// dQ = bf16(scale accumulator), a block of threads per 128 rows of a head, four elements a thread at a time; zeros in rows of
// no sequence.  Memory-bound.
template <int D>
__global__ void __launch_bounds__(256)
fa_packed_post_kernel(const BwdArgs a, int causal)
{
    constexpr int kPieces = D / 8;  // of 4 floats, in half a row
    if (!plan_fits(a.plan.head, a.T, a.B, causal)) return;
    const int64_t n = static_cast<int64_t>(a.plan.head->n_blocks) * a.heads;
    for (int64_t it = blockIdx.x; it < n; it += gridDim.x) {
        const int4 e = a.plan.blocks[it / a.heads];
        const int h = static_cast<int>(it % a.heads);
        const float4 *acc = reinterpret_cast<const float4 *>(a.dq_acc + (static_cast<int64_t>(h) * a.nb + e.w + e.z) * (kBlock * D));
#pragma unroll 4
        for (int i = threadIdx.x; i < kBlock * D / 4; i += 256) {
            const int rr = i / (D / 4), c4 = i % (D / 4), row = e.z * kBlock + rr;
            if (row >= e.y) break;
            const int slot = (c4 / kPieces) * 4 + rr / 32, l = rr % 32, c = c4 % kPieces;
            const float4 x = acc[slot * (32 * kPieces) + l * kPieces + (c ^ (l & (kPieces - 1)))];
            reinterpret_cast<uint2 *>(packed_row(a.dq, e.x + row, h))[c4] =
                make_uint2(pack_bf16x2(x.x * a.scale, x.y * a.scale), pack_bf16x2(x.z * a.scale, x.w * a.scale));
        }
    }
    if (!a.fill) return;
    const Outside out = outside(a.plan.head);
    const int all = a.heads + 2 * a.kv_heads;
    const int64_t pieces = static_cast<int64_t>(out.n) * all * (D / 8);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < pieces; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int c = static_cast<int>(i % (D / 8)), h = static_cast<int>(i / (D / 8) % all);
        const int r = out.row(static_cast<int>(i / (D / 8) / all));
        __nv_bfloat16 *to = h < a.heads ? packed_row(a.dq, r, h)
                                        : h < a.heads + a.kv_heads ? packed_row(a.dk, r, h - a.heads)
                                                                   : packed_row(a.dv, r, h - a.heads - a.kv_heads);
        reinterpret_cast<uint4 *>(to)[c] = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------------ host side

template <int D, bool CAUSAL>
cudaError_t launch(const FaPackedProblem &p, const BwdArgs &a, cudaStream_t s)
{
    using C = BCfg<D>;
    CUtensorMap mq, mk, mv, mdo;
    if (!make_rows_map(&mq, p.q, p.T, p.H, D) || !make_rows_map(&mk, p.k, p.T, p.Hkv, D) ||
        !make_rows_map(&mv, p.v, p.T, p.Hkv, D) || !make_rows_map(&mdo, p.dout, p.T, p.H, D))
        return cudaErrorInvalidValue;
    cudaError_t e = set_max_dynamic_smem<fa_packed_bwd_kernel<D, CAUSAL>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(a.nb) * p.H, cap = static_cast<int64_t>(p.sm_count) * 8;
    const unsigned around = static_cast<unsigned>(rows < cap ? rows : cap);
    fa_packed_pre_kernel<D><<<around, 256, 0, s>>>(a, CAUSAL);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    fa_packed_bwd_kernel<D, CAUSAL><<<static_cast<unsigned>(a.nb * p.Hkv), kThreads, C::kSmemBytes, s>>>(mq, mk, mv, mdo, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    fa_packed_post_kernel<D><<<around, 256, 0, s>>>(a, CAUSAL);
    return cudaGetLastError();
}

}  // namespace

int64_t fa_packed_bwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d)
{
    (void)Hkv;
    return (T / 128 + B) * H * 128 * (d + 2) * 4;
}

cudaError_t fa_launch_packed_bwd(const FaPackedProblem &p, void *workspace, cudaStream_t s)
{
    BwdArgs a;
    a.plan = plan_view(p.plan, p.B, p.T);
    a.dk = p.dk;
    a.dv = p.dv;
    a.dq = p.dq;
    a.o = p.o;
    a.dout = p.dout;
    a.lse = p.lse;
    a.nb = static_cast<int>(p.T / kBlock + p.B);
    const int64_t rows = p.H * a.nb * kBlock;
    a.dq_acc = static_cast<float *>(workspace);
    a.lse2 = a.dq_acc + rows * p.d;
    a.dvec = a.lse2 + rows;
    a.T = static_cast<int>(p.T);
    a.B = static_cast<int>(p.B);
    a.heads = static_cast<int>(p.H);
    a.kv_heads = static_cast<int>(p.Hkv);
    a.group = static_cast<int>(p.H / p.Hkv);
    a.fill = p.fill;
    // about 256 CTAs per group of key heads (at least one head)
    const int64_t hpg = a.nb >= 256 ? 1 : 256 / a.nb;
    a.heads_per_group = static_cast<int>(hpg < p.Hkv ? hpg : p.Hkv);
    a.scale = p.scale;
    a.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    if (p.d == 64) return p.causal ? launch<64, true>(p, a, s) : launch<64, false>(p, a, s);
    return p.causal ? launch<128, true>(p, a, s) : launch<128, false>(p, a, s);
}

int fa_packed_bwd_take_status(cudaStream_t stream) { return packed_take_status_here(stream); }
