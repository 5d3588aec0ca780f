// Moving tokens and pages of the 4-bit KV cache (format: fa_kv4.cuh): the accepted path of a tree of drafts to the
// front of the drafts, and whole pages to other ones.  Bytes are moved as they are.
#include "fa_kv4.cuh"

namespace {

// ----------------------------------------------------------------------- keep

constexpr int kMostDrafts = 64;

// A block per (sequence, key head), D / 16 threads a draft (half for K, half for V), 16 bytes each.  Every
// row is read before any is written: a path is moved over drafts that it passes.  A call is a few rows of 137 bytes a head,
// so its time is latency: lengths and path, the page, the row, the store, one behind the other, and nothing else (with an append
// before and a read behind it, in a graph: 16 drafts of 1 sequence 6.0 us, 32 drafts of 64 sequences 9.8).
template <int D>
__global__ void __launch_bounds__(kMostDrafts * D / 16)
fa_kv4_keep_kernel(const Kv4KeepProblem p)
{
    constexpr int TPR = D / 16, HALF = TPR / 2;
    const Kv4Cache &c = p.cache;
    const int tid = threadIdx.x, i = tid / TPR, t = tid % TPR;
    const int64_t b = blockIdx.x / c.heads;
    const int h = static_cast<int>(blockIdx.x - b * c.heads);
    const int32_t *path = p.path + b * p.n_draft;
    const int mine = i < p.n_draft ? path[i] : 0, before = i > 0 && i < p.n_draft ? path[i - 1] : -1;
    const int len = kv4_length(p.lens, b, p.max_pages << c.log2_page);
    int drafts = min(p.n_draft, len);
    if (p.n_new != nullptr) drafts = min(max(p.n_new[b], 0), drafts);
    int m = min(max(p.n_path[b], 0), drafts);
    // the first entry that does not ascend, or is no draft, ends the path
    __shared__ int end;
    if (tid == 0) end = kMostDrafts;
    __syncthreads();
    if (i < m && (mine <= before || mine >= drafts)) atomicMin(&end, i);
    __syncthreads();
    bool bad = end < m;
    m = min(m, end);
    const int first = len - drafts;
    if (h == 0 && tid == 0) p.new_lens[b] = first + m;
    const bool go = i < m && mine != i;
    uint4 x = make_uint4(0, 0, 0, 0);
    uint32_t y = 0;
    int64_t to = -1;
    if (go) {
        bool from_there, to_there;
        const int ps = kv4_page_quiet(c, p.table, b, p.max_pages, first + mine, &from_there);
        const int pd = kv4_page_quiet(c, p.table, b, p.max_pages, first + i, &to_there);
        const int64_t from = kv4_row(c, ps, h, first + mine);
        if (from_there) {  // (a draft that no page holds leaves zeros without weight)
            x = reinterpret_cast<const uint4 *>(t < HALF ? c.k : c.v)[from * HALF + t % HALF];
            // the row's small parts, one a thread: K's scales, V's scale, the weight
            if (t == 0)
                y = D == 128 ? reinterpret_cast<const uint32_t *>(c.k_scale)[from] : reinterpret_cast<const uint16_t *>(c.k_scale)[from];
            if (t == 1) y = c.v_scale[from];
            if (t == 2 && c.weights != nullptr) y = reinterpret_cast<const uint32_t *>(c.weights)[from];
        }
        if (to_there) to = kv4_row(c, pd, h, first + i);
        bad |= !from_there || !to_there;
    }
    __syncthreads();
    if (to >= 0) {
        reinterpret_cast<uint4 *>(t < HALF ? c.k : c.v)[to * HALF + t % HALF] = x;
        if (t == 0) {
            if (D == 128)
                reinterpret_cast<uint32_t *>(c.k_scale)[to] = y;
            else
                reinterpret_cast<uint16_t *>(c.k_scale)[to] = static_cast<uint16_t>(y);
        }
        if (t == 1) c.v_scale[to] = static_cast<uint8_t>(y);
        if (t == 2 && c.weights != nullptr) reinterpret_cast<uint32_t *>(c.weights)[to] = y;
    }
    if (bad) kv4_report();
}

// ----------------------------------------------------------------------- copy

constexpr int kCopyThreads = 256, kCopyTurns = 4;  // 16-byte pieces a thread has under way

// A page is five runs of bytes, one in each array, each a multiple of 16 bytes; a block takes kCopyThreads
// kCopyTurns pieces of one page.  Memory-bound: 262 MB each way, 8 key heads, d = 128, pages of 64, 88 us (6.0 TB/s).
__global__ void __launch_bounds__(kCopyThreads)
fa_kv4_copy_kernel(Kv4Cache from, Kv4Cache to, const int32_t *__restrict__ pages, const int32_t *__restrict__ to_pages, int64_t items,
                   int slices)
{
    const int rows = from.heads << from.log2_page;       // token-heads of a page
    const int codes = rows / 16 * (from.d / 2), k_scales = rows / 16 * (from.d / 32), v_scales = rows / 16;
    const int weights = to.weights != nullptr ? rows / 4 : 0;
    const int all = 2 * codes + k_scales + v_scales + weights;
    bool bad = false;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t pair = it / slices;
        const int src = pages[pair], dst = to_pages[pair];
        if (src < 0 || dst < 0) continue;
        if (src >= from.n_pages || dst >= to.n_pages) {
            bad = true;
            continue;
        }
        const int at0 = static_cast<int>(it - pair * slices) * (kCopyThreads * kCopyTurns) + threadIdx.x;
        uint4 x[kCopyTurns];
        uint4 *out[kCopyTurns];
#pragma unroll
        for (int u = 0; u < kCopyTurns; ++u) {
            int at = at0 + u * kCopyThreads;
            x[u] = make_uint4(0, 0, 0, 0);
            out[u] = nullptr;
            if (at >= all) continue;
            const uint8_t *a = from.k;
            uint8_t *z = to.k;
            int run = codes;
            if (at >= codes) {
                at -= codes, a = from.v, z = to.v;
                if (at >= codes) {
                    at -= codes, a = from.k_scale, z = to.k_scale, run = k_scales;
                    if (at >= k_scales) {
                        at -= k_scales, a = from.v_scale, z = to.v_scale, run = v_scales;
                        if (at >= v_scales) {
                            at -= v_scales, run = weights;
                            a = reinterpret_cast<const uint8_t *>(from.weights), z = reinterpret_cast<uint8_t *>(to.weights);
                        }
                    }
                }
            }
            out[u] = reinterpret_cast<uint4 *>(z) + static_cast<int64_t>(dst) * run + at;
            if (a != nullptr) x[u] = reinterpret_cast<const uint4 *>(a)[static_cast<int64_t>(src) * run + at];
        }
#pragma unroll
        for (int u = 0; u < kCopyTurns; ++u)
            if (out[u] != nullptr) *out[u] = x[u];
    }
    if (bad) kv4_report();
}

}  // namespace

cudaError_t fa_launch_kv4_keep(const Kv4KeepProblem &p, cudaStream_t stream)
{
    const int64_t bh = p.B * p.cache.heads;
    if (bh > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // (whole warps for the drafts that there may be)
    const int threads = (p.n_draft * (p.cache.d / 16) + 31) / 32 * 32;
    if (p.cache.d == 128)
        fa_kv4_keep_kernel<128><<<static_cast<unsigned>(bh), threads, 0, stream>>>(p);
    else
        fa_kv4_keep_kernel<64><<<static_cast<unsigned>(bh), threads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t fa_launch_kv4_copy(const Kv4Cache &from, const int32_t *pages, const Kv4Cache &to, const int32_t *to_pages, int64_t n,
                               int sm_count, cudaStream_t stream)
{
    const int64_t rows = static_cast<int64_t>(from.heads) << from.log2_page;
    const int64_t all = rows / 16 * (from.d + from.d / 32 + 1) + (to.weights != nullptr ? rows / 4 : 0);
    const int64_t slices = (all + kCopyThreads * kCopyTurns - 1) / (kCopyThreads * kCopyTurns);
    const int64_t items = n * slices, cap = static_cast<int64_t>(sm_count) * 8 * 16;
    fa_kv4_copy_kernel<<<static_cast<unsigned>(items < cap ? items : cap), kCopyThreads, 0, stream>>>(from, to, pages, to_pages, items,
                                                                                                  static_cast<int>(slices));
    return cudaGetLastError();
}

int fa_kv4_move_take_status(cudaStream_t stream) { return fa_take_status_word(g_kv4_status, stream); }
