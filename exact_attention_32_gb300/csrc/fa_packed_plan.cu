// The plan of a packed batch (format: fa_packed.cuh), made on the device from the sequences' offsets, so that no
// length is read back by the host and a captured step can run with new ones.
//
// One block: a plan is small (an entry per 128 rows) and made once a batch for all layers and both directions; 7 to 8 us, most of it
// barriers, for 3 to 48 sequences.  The
// offsets are held to an ascending run inside [0, T] (a prefix maximum), the lists are sorted by the
// length of their loops by counting (1024 bins; past 1023 tiles a bin holds several lengths, which only loosens the order).
#include "fa_packed.cuh"

namespace {

constexpr int kThreads = 1024, kBins = 1024;

// Inclusive scan over the block, starting from `carry`; `scan` holds 32 partial results.
template <bool MAX>
__device__ __forceinline__ int block_scan(int x, int carry, int *scan)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto join = [](int a, int b) { return MAX ? max(a, b) : a + b; };
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = join(x, y);
    }
    __syncthreads();  // (the one before has been read)
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = carry;
    for (int i = 0; i < warp; ++i) before = join(before, scan[i]);
    return join(x, before);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

__global__ void __launch_bounds__(kThreads)
fa_packed_plan_kernel(const int32_t *__restrict__ cu, int B, int T, int causal, PlanView v)
{
    __shared__ int scan[32];
    __shared__ int bins[2][kBins];
    __shared__ int carry[3], most;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = false;
    if (tid == 0) {
        const int c0 = cu[0];
        bad = c0 < 0 || c0 > T;
        carry[0] = min(max(c0, 0), T);
        carry[1] = carry[2] = most = 0;
        v.head->first = carry[0];
    }
    bins[0][tid] = bins[1][tid] = 0;
    __syncthreads();
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + tid, end0 = carry[0], blk0 = carry[1], pairs0 = carry[2];
        const int raw = b < B ? cu[b + 1] : 0;
        const int end = block_scan<true>(min(max(raw, 0), T), end0, scan);
        bad |= b < B && raw != end;
        int start = __shfl_up_sync(0xffffffffu, end, 1);
        __syncthreads();
        if (lane == 31) scan[warp] = end;
        __syncthreads();
        if (lane == 0) start = warp == 0 ? end0 : scan[warp - 1];
        const int len = b < B ? end - start : 0, n = ceil_div(len, 128);
        const int upto = block_scan<false>(n, blk0, scan), pairs = block_scan<false>(ceil_div(len, 256), pairs0, scan);
        if (b < B) v.seqs[b] = make_int4(start, len, upto - n, 0);
        atomicMax(&most, n);
        __syncthreads();
        if (tid == kThreads - 1) {  // (a thread past the last sequence has its end, and counts nothing)
            carry[0] = end;
            carry[1] = upto;
            carry[2] = pairs;
        }
        __syncthreads();
    }
    int shift = 0;
    while ((most >> shift) >= kBins) ++shift;
    // a warp a sequence: its blocks' loops counted, then (the bins' places known) the entries put there
    auto walk = [&](auto place) {
        for (int b = warp; b < B; b += kThreads / 32) {
            const int4 s = v.seqs[b];
            const int n = ceil_div(s.y, 128), n2 = ceil_div(s.y, 256);
            for (int m = lane; m < n; m += 32) place(0, (causal ? m + 1 : n) >> shift, make_int4(s.x, s.y, m, s.z));
            for (int m = lane; m < n2; m += 32) place(1, (causal ? min(n, 2 * m + 2) : n) >> shift, make_int4(s.x, s.y, m, s.z));
        }
    };
    walk([&](int list, int bin, int4) { atomicAdd(&bins[list][bin], 1); });
    __syncthreads();
    for (int list = 0; list < 2; ++list) {  // places from the last bin down
        const int mine = bins[list][kBins - 1 - tid];
        const int at = block_scan<false>(mine, 0, scan) - mine;
        bins[list][kBins - 1 - tid] = at;
        __syncthreads();
    }
    walk([&](int list, int bin, int4 e) { (list == 0 ? v.blocks : v.pairs)[atomicAdd(&bins[list][bin], 1)] = e; });
    if (tid == 0) {
        v.head->magic = kPlanMagic;
        v.head->T = T;
        v.head->B = B;
        v.head->causal = causal;
        v.head->n_blocks = carry[1];
        v.head->n_pairs = carry[2];
        v.head->last = carry[0];
    }
    if (bad) packed_bad_sequence();
}

}  // namespace

int64_t fa_packed_plan_size(int64_t B, int64_t T)
{
    return kPlanHeadBytes + 16 * ((T / 128 + B) + (T / 256 + B) + B);
}

cudaError_t fa_launch_packed_plan(const int32_t *cu_seqlens, int64_t B, int64_t T, int causal, void *plan, cudaStream_t stream)
{
    fa_packed_plan_kernel<<<1, kThreads, 0, stream>>>(cu_seqlens, static_cast<int>(B), static_cast<int>(T), causal,
                                                      plan_view(plan, B, T));
    return cudaGetLastError();
}

int fa_packed_plan_take_status(cudaStream_t stream) { return fa_take_status_word(g_packed_status, stream); }
