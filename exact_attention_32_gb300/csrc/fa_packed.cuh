// The plan of a packed batch (fa_packed_plan), as the kernels that follow it see it, and what
// the forward and the backward of packed sequences share.
//
// A plan is a header, then two lists of work and the sequences themselves, all int4:
//   blocks  every 128-row block of every sequence {first row, length, block, first block}: the
//           sequence's first row in the packed tensors, its length, the block's number in it, and the
//           number of its first block among all sequences' blocks (what padded arrays go by)
//   pairs   every 256-row unit, likewise
//   seqs    {first row, length, first block, 0}
// Both lists have the longest loops first (causal: a block's loop ends at its diagonal), so that
// what a CTA takes last is short.  The lists have room for T / 128 + B and T / 256 + B entries,
// what the host can know without reading the lengths.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"
#include "sm100_ptx.cuh"

namespace {

// Sticky status of this translation unit's kernels: FA_ERR_BAD_SEQUENCE (offsets that do not ascend inside the tensors, or a
// plan of another T, B or mask), FA_ERR_TIMEOUT once a bounded wait gave up (which the other does not overwrite).
__device__ int g_packed_status;

__device__ __forceinline__ void packed_bad_sequence() { atomicCAS(&g_packed_status, 0, FA_ERR_BAD_SEQUENCE); }
__device__ __forceinline__ void packed_timeout() { atomicExch(&g_packed_status, FA_ERR_TIMEOUT); }

struct PlanHead {
    int magic, T, B, causal;
    int n_blocks, n_pairs;  // entries of the two lists
    int first, last;        // rows [first, last) belong to sequences
};
constexpr int kPlanMagic = 0x46415031;
constexpr int64_t kPlanHeadBytes = 128;

struct PlanView {
    PlanHead *head;
    int4 *blocks, *pairs, *seqs;
};

__host__ __device__ inline PlanView plan_view(void *plan, int64_t B, int64_t T)
{
    PlanView v;
    char *p = static_cast<char *>(plan);
    v.head = reinterpret_cast<PlanHead *>(p);
    v.blocks = reinterpret_cast<int4 *>(p + kPlanHeadBytes);
    v.pairs = v.blocks + (T / 128 + B);
    v.seqs = v.pairs + (T / 256 + B);
    return v;
}

// Whether the plan in memory was made for this T, B and mask; every length in it then lies inside the tensors.  (Whether they are this
// batch's lengths is the caller's to know.)
__device__ __forceinline__ bool plan_fits(const PlanHead *h, int T, int B, int causal)
{
    return h->magic == kPlanMagic && h->T == T && h->B == B && h->causal == causal;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn packed_encode_fn()
{
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        cudaGetLastError();
        return EncodeTiledFn(nullptr);
    }();
    return fn;
}

// A packed tensor [T][heads][d] of any strides as (d, T, heads).  Loads: boxes of 64 columns (the 128-byte swizzle's
// width) x 128 rows; stores: 32 columns x 32 rows, 64-byte swizzle.
inline bool make_rows_map(CUtensorMap *m, const FaRows &r, int64_t T, int64_t heads, int d, bool store = false)
{
    const EncodeTiledFn fn = packed_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(r.token_stride) * 2, static_cast<cuuint64_t>(r.head_stride) * 2};
    const cuuint32_t load[3] = {64, 128, 1}, put[3] = {32, 32, 1}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, strides, store ? put : load, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, store ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              store ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [n, n rounded up to 16) of a 128-row tile of D columns (128-byte swizzle: the swizzle stays inside a row) to
// zeros, by `lanes` threads of a warp; a fence makes it visible to the products that follow.  The tile is loaded 128 rows at a time, so behind a
// sequence's last row it holds the next sequence's, or whatever lies behind the last one; a product over these rows
// has weight 0 for them, which keeps them out only as long as they are finite.  Products step 16 rows at a time and end
// behind the last step that has a row of the sequence, so no more rows than these matter.
template <int D>
__device__ __forceinline__ void zero_tail_rows(uint8_t *tile, int n, int lane, int lanes = 32)
{
    constexpr int kPieces = D / 8;  // of 16 bytes, in a row
    const int rows = ((n + 15) & ~15) - n;
    for (int i = lane; i < rows * kPieces; i += lanes) {
        const int r = n + i / kPieces, c = i % kPieces;
        *reinterpret_cast<uint4 *>(tile + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// A kernel behind another whose results it needs: launched before that one has ended, so that its launch and what it does
// first overlap it, it waits for the end itself.  (The plan is not among those results: it is older.)
__device__ __forceinline__ void wait_for_the_one_before() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// In the kernel before: once all its CTAs have come here (or ended), the next one's may take what room there is.
__device__ __forceinline__ void let_the_next_one_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// In clusters of `cluster` CTAs; behind: with the launch above.
template <typename... P, typename... A>
cudaError_t launch_with(void (*kern)(P...), unsigned grid, int threads, int smem, cudaStream_t s, unsigned cluster, bool behind, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attrs[2] = {};
    cfg.attrs = attrs;
    if (behind) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs].val.clusterDim.x = cluster;
        attrs[cfg.numAttrs].val.clusterDim.y = attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Four floats at an address of this CTA's shared memory in the cluster's CTA `rank`; the cluster's barrier.
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr, uint32_t rank)
{
    float4 x;
    asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %4, %5;\nld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return x;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// How many CTAs (a cluster) share a loop: the least by an estimate of the time, in steps of the loop, for sequences of equal lengths.
// n loops, the longest of `loop` steps, which go `step` at a time; a CTA costs `alone` besides its steps, in a cluster `fixed`.
// Where not all are resident at one time: causal, with the longest loops first, the work over the SMs and the last ones' end (an
// eighth more for clusters, as measured), else whole turns.
inline int cluster_ranks(double n, double loop, double step, double alone, double fixed, bool causal)
{
    // CTAs, in clusters of that many, that the GPU's groups of SMs hold at one time, with one CTA an SM
    constexpr struct {
        int ranks, resident;
    } kClusters[] = {{1, 152}, {2, 152}, {3, 138}, {4, 144}, {6, 138}, {8, 120}};
    int best = 1;
    double least = 0;
    for (const auto &c : kClusters) {
        if (c.ranks > 1 && c.ranks > loop) break;
        const double cost = c.ranks == 1 ? alone : fixed;
        const double share = cost + ceil(loop / c.ranks), turns = ceil(n * c.ranks / c.resident);
        double t = share * turns;
        if (turns > 1 && causal) {
            t = fmax(share, n * (loop / 2 + cost * c.ranks) / c.resident + cost + step / c.ranks);
            if (c.ranks > 1) t *= 1.125;
        }
        if (c.ranks == 1 || t < least) {
            least = t;
            best = c.ranks;
        }
    }
    return best;
}

// Rows of no sequence: [0, first) and [last, T).  n of them; the i-th.
struct Outside {
    int first, last, n;
    __device__ __forceinline__ int row(int i) const { return i < first ? i : last + (i - first); }
};
__device__ __forceinline__ Outside outside(const PlanHead *h) { return {h->first, h->last, h->first + (h->T - h->last)}; }

// Row `row` of head `head` of a packed bf16 tensor.
__device__ __forceinline__ __nv_bfloat16 *packed_row(const FaRows &r, int64_t row, int head)
{
    return static_cast<__nv_bfloat16 *>(r.p) + row * r.token_stride + head * r.head_stride;
}

}  // namespace
