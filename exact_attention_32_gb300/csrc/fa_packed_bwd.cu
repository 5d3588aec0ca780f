// Exact attention backward of packed sequences with grouped heads (fa_bwd_packed): TMA + tcgen05 + TMEM.
//
// Per sequence, with P = exp(scale q k^T - LSE) recomputed from the saved LSE and D_i = dO_i . O_i:
//   dV_j = sum over the key head's query heads and rows i of P_ij dO_i
//   dS_ij = P_ij (dO_i . v_j - D_i),   dQ_i = scale sum_j dS_ij k_j,   dK_j = scale sum dS_ij q_i
//
// Three launches:
//   pre   D and LSE log2 e of every row, in vectors padded to whole blocks of 128 rows (+inf and 0 behind a sequence's
//         end, so that P is 0 there); the fp32 dQ accumulator zeroed
//   main  a CTA per 128 keys of one key head of one sequence, the longest loops first (the plan's list), over the 128-row
//         query blocks (causal: from the diagonal) of each of the key head's query heads in turn: dK and dV, which
//         sum over those heads, stay in tensor memory through all of it; each block's part of dQ is added to
//         the accumulator in L2.  Where that leaves SMs idle, a cluster of CTAs shares the loop (ranks_of) and adds its dK and dV
//         through distributed shared memory in the ranks' order.
//   post  dQ = bf16(scale accumulator); zeros in rows of no sequence where they are asked for
// Per query block i (S^T etc. are key-major: TMEM lane = key):
//   S^T  = K Q^T      SS product -> TMEM A
//   P^T  = exp2(S^T scale log2 e - LSE log2 e)   softmax warps, bf16 back into A
//   dP^T = V dO^T     SS product -> TMEM B
//   dS^T = P^T (dP^T - D)                        softmax warps, bf16 into B and into shared memory
//   dV  += P^T dO     A from TMEM, B = dO MN-major -> TMEM C
//   dK  += dS^T Q     A from TMEM -> TMEM D
//   dQ   = dS K       A = dS MN-major, B = K MN-major -> TMEM B, read into registers, added to the accumulator
// The products are issued so that one block's last overlap the next one's softmax:
//   dP_i  dV_i  S_i+1  dK_i  dQ_i  (dQ_i read out)  dP_i+1 ...
// S_i+1 takes A's place behind dV_i, which read P_i there, and while dK_i and dQ_i run the softmax warps take P_i+1;
// dQ_i takes B's place behind dK_i, which read dS_i there.  (In the order S_i dP_i dV_i dK_i dQ_i, with dQ in A, the tensor
// pipe waited for both halves of the softmax of every block.)
// The accumulator is blocked: a 128 x d fp32 block per (query head, block), as pieces of 32 rows x 32 columns, 4 KB each: its
// 8 groups of 4 columns one behind the other, in each the 32 rows next to one another.  A warpgroup of its own reads dQ
// out, stages it piece by piece and adds each by a bulk reduction of 8 KB (by softmax warps between a block's P and its dS: 5 %
// slower; reductions of 2 KB 5 %, of 512 bytes 11 %; plain vector reductions, more).  This is what bounds the kernel: 64 KB a
// block and tile leave an SM at about 15 bytes a cycle, reduced or only stored.  32 heads of 16384, causal: 4370 us, without the
// additions 3950; 8 sequences of 700 to 4096, 32 heads on 8: 844 us of 985, 0.87 PFLOP/s over all three kernels, the tensor
// pipe 53 % busy.
//
// A 128-row tile that reaches behind its sequence holds rows of others.  Sums over rows (dV, dK over queries, dQ over
// keys) step 16 rows at a time and end behind the sequence's last one; of that step the rows behind are made zeros in
// Q, dO, K and V (zero_tail_rows, by a warp of its own), so that their P, dP and dS are zeros too, whatever the tile
// held.  Rows past that step are lanes and columns of results that nothing reads.
// Roles: warps 0-3 and 4-7 are two warpgroups that take query columns 0-63 and 64-127 of a block (and halves of dK's
// and dV's columns at the end); warps 8-11 add dQ; warp 12 loads; warp 13 issues the products and owns the tensor memory;
// warp 14 zeroes tails.
// Every mbarrier wait is bounded; a wait that gives up sets FA_ERR_TIMEOUT and the CTA winds down.
#include <math.h>

#include <type_traits>

#include "fa_packed.cuh"

using namespace sm100;

namespace {

constexpr int kBlock = 128;  // keys per CTA, rows of a query block
// Launched with 128 registers a thread (what 512 threads may have): the softmax, which holds a block's P until its dP is
// there, takes 32 more each of what the others give up (without, it spilled).
constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 160, kAddRegs = 88, kOtherRegs = 104;
static_assert(2 * kSoftmaxRegs + kAddRegs + kOtherRegs <= 4 * kLaunchRegs, "the warpgroups' shares are what the block has");
constexpr int kAddWarp = 8;
constexpr int kLoadWarp = 12;
constexpr int kMmaWarp = 13;
constexpr int kTailWarp = 14;
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr uint64_t kCleanupLimitNs = 20000000ull;

template <int D>
struct BCfg {
    static constexpr int kTile = kBlock * D * 2;
    static constexpr int kAtoms = D / 64;
    static constexpr int kK = 0;
    static constexpr int kV = kTile;
    // Q in two buffers, dO in one: dO_i+1 has S_i+1, dK_i and dQ_i to arrive in
    static constexpr int kQ = 2 * kTile;
    static constexpr int kDO = kQ + 2 * kTile;
    static constexpr int kDS = kDO + kTile;                 // dS, 128 keys x 128 queries bf16, MN-major
    static constexpr int kDQ = kDS + kBlock * kBlock * 2;   // dQ on its way out: two pieces a warp
    static constexpr int kVec = kDQ + 4 * 8192;             // per Q buffer: LSE log2 e (512 B), D (512 B)
    static constexpr int kBar = kVec + 2 * 1024;
    static constexpr int kNumBars = 18;
    static constexpr int kSmemBytes = kBar + kNumBars * 8 + 16;
    static_assert(kSmemBytes <= 232448, "shared memory plan exceeds 227 KB");
};

enum { KV_FULL = 0, Q_FULL = 1, Q_FREE = 3, DO_FULL = 5, DO_FREE, S_FULL, DP_FULL, P_READY, DS_READY, DQ_FULL, DQ_CONSUMED, KV_TAIL,
       Q_TAIL, DO_TAIL = Q_TAIL + 2, DONE, MMA_DONE };

struct BwdArgs {
    PlanView plan;
    FaRows dk, dv, dq, o, dout;
    const float *lse;               // [H][T]
    float *lse2, *dvec, *dq_acc;    // [H][nb * 128], the same, [H][nb][128 * D]
    int T, B, heads, kv_heads, group, fill;
    int nb;                         // blocks that the padded arrays have room for
    int heads_per_group;            // see the order of the CTAs
    int ranks;                      // CTAs (a cluster) that share a key block
    float scale, scale_log2;
};

__device__ __forceinline__ uint32_t lo32(uint64_t x) { return static_cast<uint32_t>(x); }
__device__ __forceinline__ uint32_t hi32(uint64_t x) { return static_cast<uint32_t>(x >> 32); }

// TMEM column of the packed (bf16 pairs) 16-query step kk: warpgroup w packs its 64 queries into columns [64 w, 64 w + 32).
__device__ __forceinline__ uint32_t packed_col(int kk) { return kk < 4 ? kk * 8 : 64 + (kk - 4) * 8; }

// SHARED: a.ranks CTAs share a key block (compiled apart: with the code for it the plain kernel took 1014 us in place of 988).
template <int D, bool CAUSAL, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
fa_packed_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdArgs a)
{
    using C = BCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The grid has a CTA for every block that the lengths could make; those past the list end here, and all do for a plan
    // of another T, B or mask (which the pre kernel reports); not before the pre kernel, which the post kernel does not wait for.
    // (The post kernel is not let in early from here: its blocks, waiting beside the last CTAs, took 1017 us in place of 988.)
    const bool fits = plan_fits(a.plan.head, a.T, a.B, CAUSAL);
    const int n_blocks = fits ? a.plan.head->n_blocks : 0;
    // The key heads go in groups, so that the CTAs resident at one time share a few heads' Q, dO and dQ blocks in L2; inside
    // a group the list's order, the longest loops first.
    const int64_t per_group = static_cast<int64_t>(a.heads_per_group) * n_blocks;
    const unsigned ranks = SHARED ? a.ranks : 1, work = blockIdx.x / ranks, rank = blockIdx.x % ranks;  // (a cluster's CTAs have one `work`)
    if (work >= static_cast<int64_t>(a.kv_heads) * n_blocks) {
        wait_for_the_one_before();
        return;
    }
    if ((sb & 1023u) != 0) {  // the swizzled tiles need a 1024-byte-aligned base
        if (tid == 0) packed_timeout();
        return;
    }
    const int grp = static_cast<int>(work / per_group), rem = static_cast<int>(work - grp * per_group);
    const int gsize = min(a.heads_per_group, a.kv_heads - grp * a.heads_per_group);
    const int kvh = grp * a.heads_per_group + rem % gsize;
    const int4 entry = a.plan.blocks[rem / gsize];
    const int start = entry.x, len = entry.y, blk0 = entry.w;
    const int n_seq = (len + kBlock - 1) / kBlock;
    // entries hold the number of a query block whose loop over keys is as long as this key block's over queries
    const int kb = CAUSAL ? n_seq - 1 - entry.z : entry.z;
    const int k0 = kb * kBlock, qb0 = CAUSAL ? kb : 0, nq = n_seq - qb0;
    // query blocks of all of the key head's query heads, from which this CTA takes n_it behind the first it0
    const int all_it = nq * a.group, it0 = SHARED ? static_cast<int>(static_cast<int64_t>(all_it) * rank / ranks) : 0,
              n_it = SHARED ? static_cast<int>(static_cast<int64_t>(all_it) * (rank + 1) / ranks) - it0 : all_it;
    const int h0 = kvh * a.group + (SHARED ? it0 / nq : 0), block0 = SHARED ? it0 % nq : 0;  // the first one's head, and its number among the head's
    const int q_left = len - (n_seq - 1) * kBlock;           // rows of the sequence's last block
    const int k_rows = min(kBlock, len - k0);                // keys of this block
    const uint32_t bar0 = sb + C::kBar;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBar + C::kNumBars * 8);

    if (tid == 0) {
        mbar_init(BAR(KV_FULL), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(BAR(Q_FULL + s), 1);
            mbar_init(BAR(Q_FREE + s), 1);
            mbar_init(BAR(Q_TAIL + s), 1);
        }
        mbar_init(BAR(DO_FULL), 1);
        mbar_init(BAR(DO_FREE), 1);
        mbar_init(BAR(DO_TAIL), 1);
        mbar_init(BAR(S_FULL), 1);
        mbar_init(BAR(DP_FULL), 1);
        mbar_init(BAR(P_READY), 8);
        mbar_init(BAR(DS_READY), 8);
        mbar_init(BAR(DQ_FULL), 1);
        mbar_init(BAR(DQ_CONSUMED), 4);
        mbar_init(BAR(KV_TAIL), 1);
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
    wait_for_the_one_before();  // (D, LSE and the accumulator's zeros)
    const uint32_t tA = tmem, tB = tmem + 128, tC = tmem + 256, tD = tmem + 384;

    if (!run) {
        // nothing to do
    } else if (warp >= kLoadWarp) {
        registers_down<kOtherRegs>();
        if (warp == kLoadWarp && lane == 0) {
            // ------------------------------------------------------------ loads
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            prefetch_tmap(&tm_do);
            if (n_it > 0) {
                mbar_arrive_expect_tx(BAR(KV_FULL), 2 * C::kTile);
                for (int c = 0; c < C::kAtoms; ++c) {
                    tma_load_3d(sb + C::kK + c * 16384, &tm_k, BAR(KV_FULL), c * 64, start + k0, kvh);
                    tma_load_3d(sb + C::kV + c * 16384, &tm_v, BAR(KV_FULL), c * 64, start + k0, kvh);
                }
            }
            bool ok = true;
            int i = 0, n_do = 0;
            for (int h = h0, qb = qb0 + block0; i < n_it; ++i) {
                const int st = i & 1;
                if (i >= 2 && !(ok = mbar_wait(BAR(Q_FREE + st), ((i >> 1) - 1) & 1, kWaitLimitNs))) break;
                const int row = start + qb * kBlock;
                mbar_arrive_expect_tx(BAR(Q_FULL + st), C::kTile + 1024);
                for (int c = 0; c < C::kAtoms; ++c)
                    tma_load_3d(sb + C::kQ + st * C::kTile + c * 16384, &tm_q, BAR(Q_FULL + st), c * 64, row, h);
                const int64_t vo = (static_cast<int64_t>(h) * a.nb + blk0 + qb) * kBlock;
                bulk_load(sb + C::kVec + st * 1024, a.lse2 + vo, 512, BAR(Q_FULL + st));
                bulk_load(sb + C::kVec + st * 1024 + 512, a.dvec + vo, 512, BAR(Q_FULL + st));
                if (i >= 1 && !(ok = mbar_wait(BAR(DO_FREE), (i - 1) & 1, kWaitLimitNs))) {
                    ++i;
                    break;
                }
                mbar_arrive_expect_tx(BAR(DO_FULL), C::kTile);
                for (int c = 0; c < C::kAtoms; ++c) tma_load_3d(sb + C::kDO + c * 16384, &tm_do, BAR(DO_FULL), c * 64, row, h);
                ++n_do;
                if (++qb == n_seq) {
                    qb = qb0;
                    ++h;
                }
            }
            if (!ok) packed_timeout();
            // every copy this thread issued has landed before the CTA may exit
            const uint64_t lim = ok ? kWaitLimitNs : kCleanupLimitNs;
            if (n_it > 0) mbar_wait(BAR(KV_FULL), 0, lim);
            for (int j = i > 2 ? i - 2 : 0; j < i; ++j) mbar_wait(BAR(Q_FULL + (j & 1)), (j >> 1) & 1, lim);
            if (n_do > 0) mbar_wait(BAR(DO_FULL), (n_do - 1) & 1, lim);
        } else if (warp == kTailWarp) {
            // -------------------------------------------------- rows behind the sequence's end
            bool ok = true;
            if ((k_rows & 15) && n_it > 0) {
                ok = mbar_wait_warp(BAR(KV_FULL), 0, kWaitLimitNs);
                zero_tail_rows<D>(smem + C::kK, k_rows, lane);
                zero_tail_rows<D>(smem + C::kV, k_rows, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(KV_TAIL));
            }
            if (q_left & 15) {  // every block's tiles go by this warp then (a wait for some of a barrier's phases can mistake one for another)
                int block = block0;
                for (int i = 0; i < n_it && ok; ++i) {
                    const int st = i & 1;
                    const bool tail = ++block == nq;
                    if (tail) block = 0;
                    auto pass = [&](int from, uint32_t phase, int to, uint8_t *tile) -> bool {
                        if (!mbar_wait_warp(BAR(from), phase, kWaitLimitNs)) return false;
                        if (tail) {
                            zero_tail_rows<D>(tile, q_left, lane);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive(BAR(to));
                        return true;
                    };
                    ok = pass(Q_FULL + st, (i >> 1) & 1, Q_TAIL + st, smem + C::kQ + st * C::kTile) &&
                         pass(DO_FULL, i & 1, DO_TAIL, smem + C::kDO);
                }
            }
            if (!ok && lane == 0) packed_timeout();
        } else if (warp == kMmaWarp && lane == 0) {
            // ------------------------------------------------------------- products
            constexpr uint32_t idS = idesc_bf16_f32(kBlock, kBlock, false);   // S^T, dP^T: K-major operands
            constexpr uint32_t idAcc = idesc_bf16_f32(kBlock, D, true);       // dV, dK: A in TMEM, B MN-major
            constexpr uint32_t idQ = idesc_bf16_f32(kBlock, D, true, true);   // dQ: A and B MN-major
            constexpr uint32_t kTile16 = C::kTile >> 4;
            const uint64_t d_kmaj = smem_desc_sw128(sb, 16, 1024), d_mn = smem_desc_sw128(sb, 16384, 1024);
            const uint32_t kmaj_hi = hi32(d_kmaj), mn_hi = hi32(d_mn);
            const uint32_t kmaj = lo32(d_kmaj), mn = lo32(d_mn);
            const uint32_t k_kmaj = kmaj + (C::kK >> 4), v_kmaj = kmaj + (C::kV >> 4), k_mn = mn + (C::kK >> 4), ds_mn = mn + (C::kDS >> 4),
                           q_kmaj = kmaj + (C::kQ >> 4), q_mn = mn + (C::kQ >> 4), do_kmaj = kmaj + (C::kDO >> 4), do_mn = mn + (C::kDO >> 4);
            const int k_steps = (k_rows + 15) / 16, tail_steps = (q_left + 15) / 16;
            int block = block0;  // of the query head's nq
            const int q_there = (q_left & 15) ? Q_TAIL : Q_FULL, do_there = (q_left & 15) ? DO_TAIL : DO_FULL;
            // block i's tile is there, and its rows behind the end are zeros; S_i = K Q_i^T
            auto scores = [&](int i) -> bool {
                const int st = i & 1;
                if (!mbar_wait(BAR(q_there + st), (i >> 1) & 1, kWaitLimitNs)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t koff = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                    mma_ss_lohi(tA, k_kmaj + koff, kmaj_hi, q_kmaj + st * kTile16 + koff, kmaj_hi, idS, kk > 0 ? 1u : 0u);
                }
                mma_commit(BAR(S_FULL));
                return true;
            };
            bool ok = n_it == 0 || (mbar_wait(BAR(KV_FULL), 0, kWaitLimitNs) &&
                                    (!(k_rows & 15) || mbar_wait(BAR(KV_TAIL), 0, kWaitLimitNs)) && scores(0));
            for (int i = 0; i < n_it && ok; ++i) {
                const int st = i & 1;
                const bool tail = ++block == nq;
                if (tail) block = 0;
                const int q_steps = tail ? tail_steps : kBlock / 16;
                // dP^T = V dO^T, once B's dQ of the block before has been read
                if (!(ok = mbar_wait(BAR(do_there), i & 1, kWaitLimitNs))) break;
                if (i > 0 && !(ok = mbar_wait(BAR(DQ_CONSUMED), (i - 1) & 1, kWaitLimitNs))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t koff = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                    mma_ss_lohi(tB, v_kmaj + koff, kmaj_hi, do_kmaj + koff, kmaj_hi, idS, kk > 0 ? 1u : 0u);
                }
                mma_commit(BAR(DP_FULL));
                // dV += P^T dO
                if (!(ok = mbar_wait(BAR(P_READY), i & 1, kWaitLimitNs))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    if (kk < q_steps) mma_ts_lohi(tC, tA + packed_col(kk), do_mn + kk * 128, mn_hi, idAcc, (i > 0 || kk > 0) ? 1u : 0u);
                mma_commit(BAR(DO_FREE));
                if (i + 1 < n_it && !(ok = scores(i + 1))) break;
                // dK += dS^T Q, then dQ = dS K
                if (!(ok = mbar_wait(BAR(DS_READY), i & 1, kWaitLimitNs))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    if (kk < q_steps) mma_ts_lohi(tD, tB + packed_col(kk), q_mn + st * kTile16 + kk * 128, mn_hi, idAcc, (i > 0 || kk > 0) ? 1u : 0u);
                mma_commit(BAR(Q_FREE + st));
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    if (kk < k_steps) mma_ss_lohi(tB, ds_mn + kk * 128, mn_hi, k_mn + kk * 128, mn_hi, idQ, kk > 0 ? 1u : 0u);
                mma_commit(BAR(DQ_FULL));
            }
            if (!ok) packed_timeout();
            if (ok) mma_commit(BAR(DONE));
            mma_commit(BAR(MMA_DONE));
            mbar_wait(BAR(MMA_DONE), 0, ok ? kWaitLimitNs : kCleanupLimitNs);
        }
        __syncwarp();
    } else if (warp >= kAddWarp) {
        // ---------------------------------------------------------------- dQ (TMEM lane = query row)
        registers_down<kAddRegs>();
        const int q = warp - kAddWarp;  // this warp's 32 rows
        const uint32_t tQ = tB + (static_cast<uint32_t>(q * 32) << 16);
        uint8_t *stage = smem + C::kDQ + q * 8192;
        bool ok = true;
        int h = h0, qb = qb0 + block0;
        for (int i = 0; i < n_it; ++i) {
            float *acc = a.dq_acc + (static_cast<int64_t>(h) * a.nb + blk0 + qb) * (kBlock * D) + q * (32 * D);
            if (!(ok = mbar_wait_warp(BAR(DQ_FULL), i & 1, kWaitLimitNs))) break;
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
                uint32_t x[2][32];
                tmem_ld32(tQ + half * 64, x[0]);
                tmem_ld32(tQ + half * 64 + 32, x[1]);
                tmem_wait_ld();
                if (half == D / 64 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(DQ_CONSUMED));
                }
                if (lane == 0) bulk_wait_read0();  // (what was added before has left the buffers)
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4 *>(stage + u * 4096 + (c * 32 + lane) * 16) =
                            make_uint4(x[u][4 * c], x[u][4 * c + 1], x[u][4 * c + 2], x[u][4 * c + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bulk_reduce_add_f32(acc + half * 2048, smem_u32(stage), 8192);
                    bulk_commit();
                }
            }
            if (++qb == n_seq) {
                qb = qb0;
                ++h;
            }
        }
        if (!ok && lane == 0) packed_timeout();
        if (lane == 0) bulk_wait0();  // the additions have completed before the CTA ends
    } else {
        // ------------------------------------------------ softmax-side warpgroups
        registers_up<kSoftmaxRegs>();
        const int wg = warp >> 2;              // query columns [64 wg, 64 wg + 64); d columns [wg D/2, (wg + 1) D/2)
        const int r = (warp & 3) * 32 + lane;  // TMEM lane
        const uint32_t loff = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int key = k0 + r;
        bool ok = true;
        int block = block0;
        for (int i = 0; i < n_it && ok; ++i) {
            const int st = i & 1;
            const int qb = qb0 + block;
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
            const float2 sl = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[32], pk[16];
                tmem_ld32(tA + loff + wg * 64 + h * 32, x);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(lse2_s + h * 32 + j);
                    const float2 y = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), sl, make_float2(-l.x, -l.y));
                    const float2 z = fma2(make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), sl, make_float2(-l.z, -l.w));
                    p[h * 32 + j] = ex2(y.x);
                    p[h * 32 + j + 1] = ex2(y.y);
                    p[h * 32 + j + 2] = ex2(z.x);
                    p[h * 32 + j + 3] = ex2(z.y);
                }
                if (key >= len || diagonal) {  // query q0 + j admits key iff key <= q0 + j
                    const int q0 = key >= len ? -64 : qb * kBlock + wg * 64 + h * 32;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (key > q0 + j) p[h * 32 + j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(p[h * 32 + 2 * j], p[h * 32 + 2 * j + 1]);
                tmem_st16(tA + loff + wg * 64 + h * 16, pk);
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
            uint8_t *row_base = smem + C::kDS + wg * 16384 + r * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t b[32], dsk[16];
                tmem_ld32(tB + loff + wg * 64 + h * 32, b);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 dd = *reinterpret_cast<const float4 *>(d_s + h * 32 + j);
                    const float2 y = mul2(make_float2(p[h * 32 + j], p[h * 32 + j + 1]),
                                          add2(make_float2(__uint_as_float(b[j]), __uint_as_float(b[j + 1])), make_float2(-dd.x, -dd.y)));
                    const float2 z = mul2(make_float2(p[h * 32 + j + 2], p[h * 32 + j + 3]),
                                          add2(make_float2(__uint_as_float(b[j + 2]), __uint_as_float(b[j + 3])), make_float2(-dd.z, -dd.w)));
                    dsk[j / 2] = pack_bf16x2(y.x, y.y);
                    dsk[j / 2 + 1] = pack_bf16x2(z.x, z.y);
                }
                // (columns [32 h, 32 h + 16) of this warpgroup's 64: the first half's lie in columns that have been read)
                tmem_st16(tB + loff + wg * 64 + h * 16, dsk);
                // dS^T's row (this key) into the MN-major dS tile: column block wg, 16-byte piece c (queries 8c .. 8c+7) at
                // piece c ^ (key row mod 8)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4 *>(row_base + (((h * 4 + c) ^ (r & 7)) * 16)) =
                        make_uint4(dsk[4 * c], dsk[4 * c + 1], dsk[4 * c + 2], dsk[4 * c + 3]);
            }
            fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(DS_READY));
        }
        if (ok) ok = mbar_wait_warp(BAR(DONE), 0, kWaitLimitNs);
        if (!ok) packed_timeout();
        tc_fence_after();
        // dV (TMEM C) and scale dK (TMEM D), this warpgroup's half of the columns; every lane takes part in the loads.  Shared with other
        // CTAs, in fp32 into the place of K, V and Q, which the products have read: [dV, dK][key][d], 16-byte pieces at
        // piece ^ (key mod 8)
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
                    if constexpr (SHARED) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<float4 *>(smem + (which * kBlock + r) * (D * 4) + (((wg * (D / 8) + cc * 8 + c) ^ (r & 7)) << 4)) =
                                n_it == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)  // (there is nothing in tensor memory)
                                          : make_float4(__uint_as_float(x[4 * c]) * mul, __uint_as_float(x[4 * c + 1]) * mul,
                                                        __uint_as_float(x[4 * c + 2]) * mul, __uint_as_float(x[4 * c + 3]) * mul);
                        continue;
                    }
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
    if constexpr (SHARED) {
        __syncwarp();
        cluster_sync();
        if (warp < kAddWarp) {  // rank by rank, in their order; each CTA takes its part of the result's 8-column pieces
            constexpr int kPieces = 2 * kBlock * D / 8;
            const int end = kPieces * static_cast<int>(rank + 1) / static_cast<int>(ranks);
            for (int i = kPieces * static_cast<int>(rank) / static_cast<int>(ranks) + tid; i < end; i += kAddWarp * 32) {
                const int c = i % (D / 8), r = i / (D / 8) % kBlock, which = i / (D / 8) / kBlock;
                if (k0 + r >= len) continue;
                const uint32_t from = sb + (which * kBlock + r) * (D * 4), p0 = ((2 * c) ^ (r & 7)) << 4, p1 = ((2 * c + 1) ^ (r & 7)) << 4;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                for (unsigned other = 0; other < ranks; ++other) {
                    const float4 u = ld_cluster_v4(from + p0, other), v = ld_cluster_v4(from + p1, other);
                    x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
                    y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
                }
                reinterpret_cast<uint4 *>(packed_row(which == 0 ? a.dv : a.dk, start + k0 + r, kvh))[c] =
                    make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
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

// D_i = dO_i . O_i and LSE_i log2 e of every row of every block (0 and +inf behind a sequence's end); the block's dQ
// accumulator zeroed.  A block of threads per 128 rows of a head, two rows a warp at a time.  Memory-bound: 83 us for 15600 rows
// of 32 heads, d = 128 (480 MB, 5.8 TB/s; by 8 blocks an SM in turns 97).
template <int D>
__global__ void __launch_bounds__(256)
fa_packed_pre_kernel(const BwdArgs a, int causal)
{
    constexpr int TPR = D / 8;  // threads a row, 8 channels each
    let_the_next_one_start();
    if (!plan_fits(a.plan.head, a.T, a.B, causal)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) packed_bad_sequence();
        return;
    }
    const int t = threadIdx.x % TPR, r0 = threadIdx.x / TPR;
    const int64_t n = static_cast<int64_t>(a.plan.head->n_blocks) * a.heads;
    const int64_t it = blockIdx.x;
    if (it >= n) return;
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

// dQ = bf16(scale accumulator), a block of threads per 128 rows of a head, 8 columns a thread at a time: a warp reads 4 whole lines
// and writes 64 bytes of 8 rows.  Memory-bound: 58 us for 15600 rows of 32 heads, d = 128 (360 MB, 6.2 TB/s; half a row a thread,
// whose stores lie a row apart, took 145).  Zeros in rows of no sequence.
template <int D>
__global__ void __launch_bounds__(256)
fa_packed_post_kernel(const BwdArgs a, int causal)
{
    const bool fits = plan_fits(a.plan.head, a.T, a.B, causal);
    wait_for_the_one_before();
    if (!fits) return;
    const int64_t n = static_cast<int64_t>(a.plan.head->n_blocks) * a.heads;
    const int64_t it = blockIdx.x;
    if (it < n) {
        const int4 e = a.plan.blocks[it / a.heads];
        const int h = static_cast<int>(it % a.heads);
        const float4 *acc = reinterpret_cast<const float4 *>(a.dq_acc + (static_cast<int64_t>(h) * a.nb + e.w + e.z) * (kBlock * D));
#pragma unroll
        for (int u = 0; u < kBlock * D / 8 / 256; ++u) {
            const int i = u * 256 + threadIdx.x, pair = i & 3, r = (i >> 2) & 31, piece = i >> 7;  // (a piece: 32 rows x 32 columns)
            const int row = e.z * kBlock + piece / (D / 32) * 32 + r;
            if (row >= e.y) continue;
            const float4 x = acc[piece * 256 + pair * 64 + r], y = acc[piece * 256 + pair * 64 + 32 + r];
            reinterpret_cast<uint4 *>(packed_row(a.dq, e.x + row, h))[piece % (D / 32) * 4 + pair] =
                make_uint4(pack_bf16x2(x.x * a.scale, x.y * a.scale), pack_bf16x2(x.z * a.scale, x.w * a.scale),
                           pack_bf16x2(y.x * a.scale, y.y * a.scale), pack_bf16x2(y.z * a.scale, y.w * a.scale));
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

template <int D, bool CAUSAL, bool SHARED>
cudaError_t launch(const FaPackedProblem &p, const BwdArgs &a, cudaStream_t s)
{
    using C = BCfg<D>;
    CUtensorMap mq, mk, mv, mdo;
    if (!make_rows_map(&mq, p.q, p.T, p.H, D) || !make_rows_map(&mk, p.k, p.T, p.Hkv, D) ||
        !make_rows_map(&mv, p.v, p.T, p.Hkv, D) || !make_rows_map(&mdo, p.dout, p.T, p.H, D))
        return cudaErrorInvalidValue;
    cudaError_t e = set_max_dynamic_smem<fa_packed_bwd_kernel<D, CAUSAL, SHARED>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const unsigned around = static_cast<unsigned>(static_cast<int64_t>(a.nb) * p.H);
    fa_packed_pre_kernel<D><<<around, 256, 0, s>>>(a, CAUSAL);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_with(fa_packed_bwd_kernel<D, CAUSAL, SHARED>, static_cast<unsigned>(a.nb * p.Hkv * a.ranks), kThreads, C::kSmemBytes, s,
                    static_cast<unsigned>(a.ranks), true, mq, mk, mv, mdo, a);
    if (e != cudaSuccess) return e;
    return launch_with(fa_packed_post_kernel<D>, around, 256, 0, s, 1, true, a, static_cast<int>(CAUSAL));
}

// How many CTAs share a key block's loop over query blocks: with one, few key heads and long groups leave most SMs idle.  Measured
// (us, a sequence where not said otherwise, causal; the one chosen here first; 5 and 7 are never the best):
//   500 rows, 8 heads on 1    8 35   4 42   1 92     2048, 8 on 1   8 64    6 77   4 99    1 313
//   2048, 16 on 2             6 80   4 101  1 316    4096, 16 on 2  4 187   3 236  8 274   1 621
//   8192, 8 on 1              4 336  6 385  1 1216   4096, 4 on 4   2 67    1 93   3 91
//   3000, 24 on 3             4 169  3 185  1 475    10 of 300, 8 on 2   2 37  1 47  4 48
//   3 of 1024, 8 on 8         1 39   2 60            2000 and 1500, 6 on 2, d = 64, not causal   2 54  4 60  1 88
// Lengths differ as a rule, and what counts then is the longest: causal it is taken for twice the mean (by the mean alone 4 of 1 to
// 3077, 4 on 4, d = 64, took 51 in place of 37, 20 of 20 to 1000, 8 on 2, 64 in place of 42).
int ranks_of(const FaPackedProblem &p)
{
    const int64_t mean = (p.T / p.B + kBlock - 1) / kBlock, blocks = mean > 0 ? mean : 1;
    const double group = static_cast<double>(p.H / p.Hkv), longest = static_cast<double>(blocks) * (p.B > 1 && p.causal ? 2 : 1);
    return cluster_ranks(static_cast<double>(p.B * blocks * p.Hkv), group * longest, group, 4, 4, p.causal);
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
    // Key heads in groups of about 512 CTAs, of equal size: fewer in one leave SMs without work at its end (8 sequences of 700
    // to 4096 rows, 8 key heads, 130 blocks: groups of 1 head 1160 us, of 2 1094, of 4 1011), more share less of L2 (of 8 1060).
    const int64_t most = a.nb < 512 ? 512 / a.nb : 1, groups = p.Hkv > most ? (p.Hkv + most - 1) / most : 1;
    a.heads_per_group = static_cast<int>((p.Hkv + groups - 1) / groups);
    a.ranks = ranks_of(p);
    a.scale = p.scale;
    a.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    auto run = [&](auto shared) {
        constexpr bool SHARED = decltype(shared)::value;
        if (p.d == 64) return p.causal ? launch<64, true, SHARED>(p, a, s) : launch<64, false, SHARED>(p, a, s);
        return p.causal ? launch<128, true, SHARED>(p, a, s) : launch<128, false, SHARED>(p, a, s);
    };
    return a.ranks > 1 ? run(std::true_type{}) : run(std::false_type{});
}

int fa_packed_bwd_take_status(cudaStream_t stream) { return fa_take_status_word(g_packed_status, stream); }
