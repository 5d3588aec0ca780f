// Accumulated attention weight of a prompt's keys (fa_key_weights):
//     w_j = sum over the heads of key head j's group and the queries i of
//           exp(scale q_i . k_j - LSE_i),
// the column sums of the softmax matrix, recomputed from the forward's LSE as the
// backward recomputes it, never stored.
//
// One CTA takes 256 keys of one (b, key head) as two tiles of 128 and goes over
// the group's queries 128 at a time (causal: from the diagonal).  Per query block
// and key tile S^T = K Q^T is one 128 x 128 x d tcgen05 product with the key as the
// TMEM lane, so a thread owns a key: it takes exp2(S scale log2e - LSE log2e) of 128
// queries and adds them up in fp32, with nothing to exchange between threads.
//
// What bounds it: at d = 128 a tile's product and its 16384 exponentials (32 a clock and SM) take 512 cycles each, side by
// side, at d = 64 the product half of that.  32 heads of 16384 queries, causal, take 850 us (1.29 PFLOP/s, 67 % of the
// measured bf16 rate; 790 to 870, as the card's power allows), and with an eighth of the exponentials still 630 to 690.
// A product whose operands both come from shared memory
// at N = 128 would need all of its 128 bytes a clock, so K lies in tensor memory
// as the A operand (2 x d/2 columns, for the CTA's life) and only Q streams
// through shared memory (TMA, 128-byte swizzle, four stages); a Q block is used for
// both key tiles.  The other columns hold three 128 x 128 accumulators in turn,
// so the pipe runs on while the warpgroups read theirs.
// Roles (608 threads): warps 0-15 four warpgroups, two per key tile, each with half of a
// block's queries (one per tile took 831 us, two 842, both with the products issued by lane 0); warp 16 loads Q, warp 17
// issues the products, from an elected lane (829 -> 774 us), and owns the tensor memory, warp 18 loads LSE log2 e.
// Measured and not kept, against 774: exp2 by a polynomial for a share of the scores; the two warpgroups of a tile in
// turns (900); two issuing warps (774); an accumulator given back before its scores are used (823).
//
// Every mbarrier wait is bounded; one that gives up sets FA_ERR_TIMEOUT in this
// file's status word and the CTA winds down.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "fa_fwd_common.cuh"

using namespace sm100;

namespace {

constexpr int kKeyTile = 128, kKeys = 256, kQBlock = 128;
constexpr int kKwThreads = 608, kKwLoad = 16, kKwMma = 17, kKwLse = 18;
constexpr int kStages = 4;  // Q blocks in shared memory
constexpr int kMaxRanks = 8;
constexpr int kBufs = 3;    // accumulators in tensor memory

__device__ int g_key_weights_status;
__device__ __forceinline__ void kw_report(int code) { atomicExch(&g_key_weights_status, code); }

template <int D>
struct KwCfg {
    static constexpr int kStageBytes = kQBlock * D * 2;
    static constexpr int kLse = kStages * kStageBytes;  // per stage: 128 floats
    static constexpr int kSum = kLse + kStages * kQBlock * 4;  // rank 0: [rank][key] sums of its cluster
    static constexpr int kOut = kSum + kMaxRanks * kKeys * 4;  // per stage: does it hold a query that adds nothing?
    static constexpr int kBar = kOut + kStages * 4;
    static constexpr int kNumBars = 4 * kStages + 4 * kBufs + 2;
    static constexpr int kSmemBytes = kBar + kNumBars * 8 + 16;
};
// barriers: Q_FULL, Q_FREE (both key tiles' products read it), LSE_FULL, LSE_FREE per stage; S_FULL, S_FREE per
// (buffer, warpgroup).  Product n (query block n / 2, key tile n % 2) goes to buffer n % 3, so a warpgroup takes a
// buffer every sixth product; with a barrier of its own it sees every phase of it.
enum { KW_Q_FULL = 0, KW_Q_FREE = kStages, KW_LSE_FULL = 2 * kStages, KW_LSE_FREE = 3 * kStages,
       KW_S_FULL = 4 * kStages, KW_S_FREE = 4 * kStages + 2 * kBufs, KW_K_READY = 4 * kStages + 4 * kBufs,
       KW_MMA_DONE = KW_K_READY + 1 };
static_assert(kBufs == 3, "the phases below count a warpgroup's uses of a buffer as n / 6");
__device__ __forceinline__ int kw_slot(int n) { return 2 * (n % kBufs) + (n & 1); }

struct KwArgs {
    const __nv_bfloat16 *k;
    const float *lse;
    float *weights;
    int N, H, heads, n_kblocks, n_qblocks, first, ranks;
    float scale_log2;
};

// A CTA's query blocks: every ranks-th of its key block's, heads one after the other.
struct KwWalk {
    int left, qb, qh;  // blocks still to come; block within the head; (b, head) slice
    int qb0, n_qblocks, step;
    __device__ __forceinline__ void next()
    {
        --left;
        qb += step;
        while (qb >= n_qblocks) {
            qb -= n_qblocks - qb0;
            ++qh;
        }
    }
};

// Address of another rank's shared memory in the cluster, a store to it, and the cluster's barrier.
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float x)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

template <int D, bool CAUSAL>
__global__ void __launch_bounds__(kKwThreads, 1)
fa_key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const KwArgs a)
{
    using C = KwCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((sb & 1023u) != 0) {  // the swizzled tiles need a 1024-byte-aligned base
        if (tid == 0) kw_report(FA_ERR_LAUNCH);
        return;
    }
    const uint32_t bar0 = sb + C::kBar;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBar + C::kNumBars * 8);

    // key-block major: causal CTAs with many query blocks (small kb) start first.  Where there are too few key blocks for
    // the SMs, the `ranks` CTAs of a cluster share one: rank r takes the query blocks r, r + ranks, ...
    const int BHkv = static_cast<int>(gridDim.x) / (a.n_kblocks * a.ranks);
    const int unit = blockIdx.x / a.ranks, rank = blockIdx.x % a.ranks;
    const int kb = unit / BHkv, bhk = unit % BHkv;
    const int k0 = kb * kKeys;
    const int G = a.H / a.heads;
    const int qh0 = bhk * G;  // (b, query head) slices of the group: b * H + hkv * G = bhk * G
    const int qb0 = max(CAUSAL ? k0 / kQBlock : 0, a.first / kQBlock);
    const int per_head = a.n_qblocks - qb0;
    const int nq_all = per_head * G;
    const int nq = nq_all > rank ? (nq_all - rank + a.ranks - 1) / a.ranks : 0;
    KwWalk walk;
    walk.left = nq;
    walk.qb = qb0 + rank % per_head;
    walk.qh = qh0 + rank / per_head;
    walk.qb0 = qb0;
    walk.n_qblocks = a.n_qblocks;
    walk.step = a.ranks;
    const bool run = *reinterpret_cast<volatile int *>(&g_key_weights_status) == 0;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(BAR(KW_Q_FULL + s), 1);
            mbar_init(BAR(KW_Q_FREE + s), 1);
            mbar_init(BAR(KW_LSE_FULL + s), 1);
            mbar_init(BAR(KW_LSE_FREE + s), 16);
        }
        for (int s = 0; s < 2 * kBufs; ++s) {
            mbar_init(BAR(KW_S_FULL + s), 1);
            mbar_init(BAR(KW_S_FREE + s), 8);
        }
        mbar_init(BAR(KW_K_READY), 16);
        mbar_init(BAR(KW_MMA_DONE), 1);
        fence_mbar_init();
    }
    if (warp == kKwMma) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (a.ranks > 1) cluster_sync();  // rank 0's shared memory is there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tK = tmem + kBufs * 128;  // K tile w at columns tK + w * 64

    if (!run) {
        // nothing to do
    } else if (warp == kKwLoad) {
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            bool ok = true;
            int issued = 0;
            for (int i = 0; i < nq; ++i, walk.next()) {
                const int st = i % kStages;
                if (i >= kStages && !(ok = mbar_wait(BAR(KW_Q_FREE + st), (i / kStages - 1) & 1, kWaitLimitNs))) break;
                mbar_arrive_expect_tx(BAR(KW_Q_FULL + st), C::kStageBytes);
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(sb + st * C::kStageBytes + c * 16384, &tm_q, BAR(KW_Q_FULL + st), c * 64, walk.qb * kQBlock,
                                walk.qh);
                ++issued;
            }
            if (!ok) kw_report(FA_ERR_TIMEOUT);
            // no copy in flight when the CTA ends
            for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                mbar_wait(BAR(KW_Q_FULL + i % kStages), (i / kStages) & 1, ok ? kWaitLimitNs : kCleanupLimitNs);
        }
    } else if (warp == kKwLse) {
        // -LSE log2 e of each query; +inf for those past N, before first or without a key, which add nothing whatever their
        // scores are (a NaN in them, or in the key): a block that has some goes through the guarded sum
        bool ok = true;
        for (int i = 0; i < nq && ok; ++i, walk.next()) {
            const int st = i % kStages, q0 = walk.qb * kQBlock;
            if (i >= kStages && !(ok = mbar_wait_warp(BAR(KW_LSE_FREE + st), (i / kStages - 1) & 1, kWaitLimitNs))) break;
            const float *src = a.lse + static_cast<int64_t>(walk.qh) * a.N;
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = src[min(q0 + j * 32 + lane, a.N - 1)];  // (without branches: the loads go out together)
            float *dst = reinterpret_cast<float *>(smem + C::kLse) + st * kQBlock;
            bool out = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = q0 + j * 32 + lane;
                if (q < a.first || q >= a.N) x[j] = -INFINITY;
                out |= x[j] == -INFINITY;
                dst[j * 32 + lane] = x[j] * -1.4426950408889634f;
            }
            out = __any_sync(0xffffffffu, out);
            if (lane == 0) reinterpret_cast<int *>(smem + C::kOut)[st] = out;
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(KW_LSE_FULL + st));
        }
        if (!ok && lane == 0) kw_report(FA_ERR_TIMEOUT);
    } else if (warp == kKwMma) {
        constexpr uint32_t id = idesc_bf16_f32(kKeyTile, kQBlock, false);
        const uint64_t dq = smem_desc_sw128(sb, 16, 1024);
        const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
        bool ok = mbar_wait_warp(BAR(KW_K_READY), 0, kWaitLimitNs);
        tc_fence_after();
        int n = 0;  // products so far
        for (int i = 0; i < nq && ok; ++i) {
            const int st = i % kStages;
            if (!(ok = mbar_wait_warp(BAR(KW_Q_FULL + st), (i / kStages) & 1, kWaitLimitNs))) break;
            const uint32_t b_lo = q_lo + st * (C::kStageBytes >> 4);
            for (int w = 0; w < 2; ++w, ++n) {
                const int buf = n % kBufs;
                const int last = n - kBufs;  // the buffer's product before this one
                if (last >= 0 && !(ok = mbar_wait_warp(BAR(KW_S_FREE + kw_slot(last)), (last / 6) & 1, kWaitLimitNs))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ts_lohi(tS + buf * 128, tK + w * 64 + kk * 8,
                                    b_lo + (((kk / 4) * 16384 + (kk % 4) * 32) >> 4), q_hi, id, kk > 0 ? 1u : 0u);
                    mma_commit(BAR(KW_S_FULL + kw_slot(n)));
                    if (w == 1) mma_commit(BAR(KW_Q_FREE + st));
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) kw_report(FA_ERR_TIMEOUT);
        if (elect_one()) mma_commit(BAR(KW_MMA_DONE));
        __syncwarp();
        mbar_wait_warp(BAR(KW_MMA_DONE), 0, ok ? kWaitLimitNs : kCleanupLimitNs);
    } else {
        // --------------------------- two warpgroups per key tile, a thread per key and half of each query block
        const int w = warp >> 3, half = (warp >> 2) & 1;
        const int key = k0 + w * kKeyTile + (warp & 3) * 32 + lane;
        const uint32_t loff = static_cast<uint32_t>((warp & 3) * 32) << 16;
        // this half of the K row into tensor memory: bf16 pairs, channels 2c, 2c + 1 in column c
        {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.k + (static_cast<int64_t>(bhk) * a.N + key) * D) +
                               half * (D / 16);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t x[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (key < a.N) u = src[c * 4 + j];
                    x[4 * j] = u.x;
                    x[4 * j + 1] = u.y;
                    x[4 * j + 2] = u.z;
                    x[4 * j + 3] = u.w;
                }
                tmem_st16(tK + w * 64 + loff + half * (D / 4) + c * 16, x);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(KW_K_READY));
        }
        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
        float total = 0.f;
        bool ok = true;
        for (int i = 0; i < nq && ok; ++i, walk.next()) {
            const int st = i % kStages, n = 2 * i + w, buf = n % kBufs;
            const int q0 = walk.qb * kQBlock;
            {
                const uint32_t b0 = BAR(KW_LSE_FULL + st), b1 = BAR(KW_S_FULL + kw_slot(n)), f0 = (i / kStages) & 1, f1 = (n / 6) & 1;
                const bool there0 = mbar_try_wait(b0, f0), there1 = mbar_try_wait(b1, f1);  // (one vote where both are)
                if (!__all_sync(0xffffffffu, there0 && there1) &&
                    !(ok = mbar_wait_warp(b0, f0, kWaitLimitNs) && mbar_wait_warp(b1, f1, kWaitLimitNs)))
                    break;
            }
            const bool out = reinterpret_cast<volatile int *>(smem + C::kOut)[st] != 0;
            tc_fence_after();
            const float *ls = reinterpret_cast<const float *>(smem + C::kLse) + st * kQBlock + half * 64;
            const uint32_t src = tS + buf * 128 + loff + half * 64;
            // 16 queries of this key: their scores in x, their sum added to s0, s1 (the tile's sums in registers of
            // their own first: 64 terms, then one addition to the total)
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
            auto take = [&](const uint32_t (&x)[16], int c, auto guard) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(ls + c * 16 + j);
                    const float2 y0 = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), sc,
                                           make_float2(l.x, l.y));
                    const float2 y1 = fma2(make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), sc,
                                           make_float2(l.z, l.w));
                    float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
                    if constexpr (decltype(guard)::value) {
                        const int q = CAUSAL ? q0 + half * 64 + c * 16 + j : key;
                        if (key > q || l.x == INFINITY) p0.x = 0.f;
                        if (key > q + 1 || l.y == INFINITY) p0.y = 0.f;
                        if (key > q + 2 || l.z == INFINITY) p1.x = 0.f;
                        if (key > q + 3 || l.w == INFINITY) p1.y = 0.f;
                    }
                    s0 = add2(s0, p0);
                    s1 = add2(s1, p1);
                }
            };
            // the next 16 scores are on their way from tensor memory while the last are used (in pieces of 32: 119 in place of 114 us
            // for 2 x 32 heads on 8 of 4096; all 64 before the first is used, and the accumulator given back then: 127)
            auto tile = [&](auto guard) {
                uint32_t x0[16], x1[16];
                tmem_ld16(src, x0);
                tmem_wait_ld();
                tmem_ld16(src + 16, x1);
                take(x0, 0, guard);
                tmem_wait_ld();
                tmem_ld16(src + 32, x0);
                take(x1, 1, guard);
                tmem_wait_ld();
                tmem_ld16(src + 48, x1);
                take(x0, 2, guard);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(KW_S_FREE + kw_slot(n)));
                take(x1, 3, guard);
            };
            if ((CAUSAL && q0 < k0 + w * kKeyTile + kKeyTile - 1) || out)
                tile(std::true_type{});
            else
                tile(std::false_type{});
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(KW_LSE_FREE + st));
            total += (s0.x + s0.y) + (s1.x + s1.y);
        }
        if (!ok && lane == 0) kw_report(FA_ERR_TIMEOUT);
        // the halves' sums, through the LSE stages (their last readers are behind the barrier)
        float *sum = reinterpret_cast<float *>(smem + C::kLse);
        asm volatile("barrier.cta.sync 1, 512;\n" ::: "memory");
        if (half == 1) sum[w * kKeyTile + (warp & 3) * 32 + lane] = total;
        asm volatile("barrier.cta.sync 1, 512;\n" ::: "memory");
        if (half == 0) {
            const int i = w * kKeyTile + (warp & 3) * 32 + lane;
            total += sum[i];
            if (a.ranks == 1) {
                if (ok && key < a.N) a.weights[static_cast<int64_t>(bhk) * a.N + key] = total;
            } else {
                st_cluster_f32(mapa(sb + C::kSum + (rank * kKeys + i) * 4, 0), ok ? total : NAN);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kKwMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    __syncwarp();
    if (a.ranks > 1) {  // every thread of the cluster; the ranks' sums are added in their order
        cluster_sync();
        if (rank == 0 && run && tid < kKeys && k0 + tid < a.N) {
            const float *sum = reinterpret_cast<const float *>(smem + C::kSum);
            float total = 0.f;
            for (int r = 0; r < a.ranks; ++r) total += sum[r * kKeys + tid];
            a.weights[static_cast<int64_t>(bhk) * a.N + k0 + tid] = total;
        }
    }
}

// CTAs a key block (1, 2, 4 or 8): those with the shortest time by the longest CTA, the SMs' share of all query blocks, and
// what a CTA costs besides (8 blocks' time: 7.5 us, from launch to the last sum).  Only where the key blocks do not fill the SMs:
// 5 key heads of 5414 keys, 20 of queries, causal: 110 CTAs 154 us, 220 84, 440 85, 880 126; 2 key heads of 6281, 16 of queries from 3140
// on: 50 CTAs 188 us, 100 101, 200 70, 400 85; 32 of 700, d = 64, 96 CTAs 27, 192 33.
int fewest_rounds(const KwArgs &a, int64_t units, int64_t G, bool causal, int sm_count)
{
    if (units >= sm_count) return 1;
    const int64_t b0 = a.first / kQBlock;
    int64_t all = 0;  // query blocks of a (b, key head)
    for (int64_t kb = 0; kb < a.n_kblocks; ++kb) {
        const int64_t from = kb * (kKeys / kQBlock);
        all += (a.n_qblocks - (causal && from > b0 ? from : b0)) * G;
    }
    const int64_t longest = (a.n_qblocks - b0) * G, total = all * (units / a.n_kblocks);
    int best = 1;
    int64_t best_time = 0;
    for (int r = 1; r <= kMaxRanks && (r == 1 || longest >= 2 * r); r *= 2) {
        const int64_t rounds = (units * r + sm_count - 1) / sm_count, own = (longest + r - 1) / r;
        const int64_t shared = causal ? total / sm_count : rounds * own;
        const int64_t time = 8 * rounds + (own > shared ? own : shared);
        if (r == 1 || time < best_time) {
            best = r;
            best_time = time;
        }
    }
    return best;
}

template <int D, bool CAUSAL>
cudaError_t launch_kw(const FaKeyWeightsProblem &p, cudaStream_t s)
{
    using C = KwCfg<D>;
    CUtensorMap mq;
    if (!make_map(&mq, p.q, p.B * p.H, p.N, D)) return cudaErrorInvalidValue;
    cudaError_t e = set_max_dynamic_smem<fa_key_weights_kernel<D, CAUSAL>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    KwArgs a;
    a.k = static_cast<const __nv_bfloat16 *>(p.k);
    a.lse = p.lse;
    a.weights = p.weights;
    a.N = static_cast<int>(p.N);
    a.H = static_cast<int>(p.H);
    a.heads = static_cast<int>(p.Hkv);
    a.n_kblocks = static_cast<int>((p.N + kKeys - 1) / kKeys);
    a.n_qblocks = static_cast<int>((p.N + kQBlock - 1) / kQBlock);
    a.first = static_cast<int>(p.first_query);
    a.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    const int64_t units = p.B * p.Hkv * a.n_kblocks;
    a.ranks = fewest_rounds(a, units, p.H / p.Hkv, CAUSAL, p.sm_count);
    const int64_t grid = units * a.ranks;
    if (grid > 0x7fffffffLL || p.B * p.H > 0x7fffffffLL || (p.H / p.Hkv) * a.n_qblocks > 0x3fffffffLL)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kKwThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(a.ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fa_key_weights_kernel<D, CAUSAL>, mq, a);
}

}  // namespace

cudaError_t fa_launch_key_weights(const FaKeyWeightsProblem &p, cudaStream_t s)
{
    if (p.d == 64) return p.causal ? launch_kw<64, true>(p, s) : launch_kw<64, false>(p, s);
    return p.causal ? launch_kw<128, true>(p, s) : launch_kw<128, false>(p, s);
}

int fa_key_weights_take_status(cudaStream_t stream)
{
    int h = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&h, g_key_weights_status, sizeof(int), 0, cudaMemcpyDeviceToHost, stream) !=
            cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_key_weights_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream) !=
            cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_LAUNCH;
    }
    return h;
}
