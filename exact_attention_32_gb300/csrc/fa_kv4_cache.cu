// Writing, reading back and evicting from the 4-bit KV cache (format: fa_kv4.cuh).
#include <math.h>

#include "fa_kv4.cuh"

namespace {

// --------------------------------------------------------------------- append

// amax / 6 on the scale grid (to nearest even), as a byte; 255 for a block with a NaN or an infinity.
// amax is a bf16 value, so amax / 6 either is a middle of two grid values exactly or
// lies at least 2^-9 (relative) from one: the rounded fp32 quotient falls on the
// same side as the exact one.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax)
{
    if (!(amax < INFINITY)) return 255u;
    const float s = fminf(__fdiv_rn(amax, 6.f), 10240.f);
    if (s < 6.103515625e-05f)  // below 2^-14: multiples of 2^-17 (adding 96 rounds to its last place)
        return __float2uint_rn(__fsub_rn(__fadd_rn(s, 96.f), 96.f) * 131072.f);
    uint32_t b = __float_as_uint(s);
    b += 0x7FFFFu + ((b >> 20) & 1u);  // four significant bits, to nearest even
    return (b >> 20) - (112u << 3);
}

// Four bytes of codes of eight values under the scale of `byte`.  x is a bf16
// value and the scale has four significant bits, so x / s meets a middle of two
// E2M1 values exactly or not within 2^-9 of it: the rounded quotient keeps the side.
__device__ __forceinline__ uint32_t kv4_codes(const float (&x)[8], uint32_t byte)
{
    const float s = kv4_scale(byte);
    if (byte == 0u || byte == 255u) return 0u;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], s);
    return kv4_encode8(y);
}

// amax that keeps a NaN (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float unpack8(uint4 u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        m = max_nan(m, max_nan(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
    return m;
}

// D / 8 threads a row, eight channels each: one 16-byte load of K and of V, the
// maxima over 4 threads (a K block) and over the row (V) by shuffles, four bytes of
// codes out.  Memory-bound: 4 d bytes in and d + d/32 + 1 out a row.
template <int D>
__global__ void __launch_bounds__(256)
fa_kv4_append_kernel(Kv4Cache c, const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                     const float *__restrict__ w_new, const int32_t *__restrict__ n_new,
                     const int32_t *__restrict__ lens, const int32_t *__restrict__ table, int64_t rows, int64_t S,
                     int64_t max_pages)
{
    constexpr int TPR = D / 8;
    const int t = threadIdx.x % TPR;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (256 / TPR);
    // whole warps stay in the loop together: rows past the end are computed on row 0's data and not stored
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * (256 / TPR); r0 < rows; r0 += stride) {
        const int64_t r = r0 + threadIdx.x / TPR;
        const int64_t rr = r < rows ? r : 0;
        const int64_t bh = rr / S;
        const int i = static_cast<int>(rr - bh * S);
        const int64_t b = bh / c.heads;
        const int h = static_cast<int>(bh - b * c.heads);
        int n = n_new != nullptr ? n_new[b] : static_cast<int>(S);
        n = n < 0 ? 0 : (n > S ? static_cast<int>(S) : n);
        const int len = kv4_length(lens, b, max_pages << c.log2_page);
        const int pos = len - n + i;
        const bool mine = r < rows && i < n;
        int page = -1;
        if (mine) {
            if (pos >= 0)
                page = kv4_page(c, table, b, max_pages, pos);
            else if (t == 0)
                kv4_report();
        }
        float xk[8], xv[8];
        float mk = 0.f, mv = 0.f;
        if (page >= 0) {
            mk = unpack8(k_new[rr * TPR + t], xk);
            mv = unpack8(v_new[rr * TPR + t], xv);
        }
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) {
            if (o < 4) mk = max_nan(mk, __shfl_xor_sync(0xffffffffu, mk, o));
            mv = max_nan(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        }
        if (page < 0) continue;
        const int64_t row = kv4_row(c, page, h, pos);
        const uint32_t bk = kv4_scale_byte(mk), bv = kv4_scale_byte(mv);
        reinterpret_cast<uint32_t *>(c.k)[row * TPR + t] = kv4_codes(xk, bk);
        reinterpret_cast<uint32_t *>(c.v)[row * TPR + t] = kv4_codes(xv, bv);
        if ((t & 3) == 0) c.k_scale[row * (D / 32) + (t >> 2)] = static_cast<uint8_t>(bk);
        if (t == 0) {
            c.v_scale[row] = static_cast<uint8_t>(bv);
            if (c.weights != nullptr) c.weights[row] = w_new != nullptr ? w_new[rr] : 0.f;
        }
    }
}

// ----------------------------------------------------------------------- read

// Eight bf16 values of four bytes of codes times a scale (exact).
__device__ __forceinline__ uint4 kv4_bf16x8(uint32_t codes, float s)
{
    uint32_t h[4], y[4];
    kv4_decode8(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        const __nv_bfloat162 p = __floats2bfloat162_rn(f.x * s, f.y * s);
        y[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
}

// D / 8 threads a row, eight channels each of K and V.  Memory-bound by the 4 d bytes written a row.
template <int D>
__global__ void __launch_bounds__(256)
fa_kv4_read_kernel(Kv4Cache c, const int32_t *__restrict__ first, const int32_t *__restrict__ lens,
                   const int32_t *__restrict__ table, int64_t rows, int64_t T, int64_t max_pages,
                   uint4 *__restrict__ k_out, uint4 *__restrict__ v_out)
{
    constexpr int TPR = D / 8;
    const int t = threadIdx.x % TPR;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (256 / TPR);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR; r < rows; r += stride) {
        const int64_t bh = r / T;
        const int64_t b = bh / c.heads;
        const int h = static_cast<int>(bh - b * c.heads);
        const int64_t pos = (r - bh * T) + (first != nullptr ? first[b] : 0);
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (pos >= 0 && pos < kv4_length(lens, b, max_pages << c.log2_page)) {
            const int page = kv4_page(c, table, b, max_pages, static_cast<int>(pos));
            if (page >= 0) {
                const int64_t row = kv4_row(c, page, h, static_cast<int>(pos));
                k = kv4_bf16x8(reinterpret_cast<const uint32_t *>(c.k)[row * TPR + t],
                               kv4_scale(c.k_scale[row * (D / 32) + (t >> 2)]));
                v = kv4_bf16x8(reinterpret_cast<const uint32_t *>(c.v)[row * TPR + t], kv4_scale(c.v_scale[row]));
            }
        }
        k_out[r * TPR + t] = k;
        v_out[r * TPR + t] = v;
    }
}

// ---------------------------------------------------------------------- evict

constexpr int kSelThreads = 1024;

// An order-preserving image of a weight: larger float, larger key; -0 and 0 alike; a NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (isnan(w)) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Which tokens of one (sequence, key head) stay.  The candidates are the tokens
// before the protected last ones; `need` of them stay.  The need-th largest key is
// found bit by bit from the top: a bit is set where at least `need` candidates reach
// the value with it.  Above it all stay, at it the lowest positions.
__global__ void __launch_bounds__(kSelThreads)
fa_kv4_select_kernel(Kv4Cache c, const int32_t *__restrict__ lens, const int32_t *__restrict__ table,
                     int64_t max_pages, int keep, int recent, int32_t *__restrict__ kept,
                     int32_t *__restrict__ new_lens)
{
    __shared__ int warp_sum[2][32];
    __shared__ int warp_gt[32], warp_eq[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t bh = blockIdx.x, b = bh / c.heads;
    const int h = static_cast<int>(bh - b * c.heads);
    const int len = kv4_length(lens, b, max_pages << c.log2_page);
    const int m = len < keep ? len : keep;
    const int cand = len - (recent < len ? recent : len);
    const int need = m - (len - cand);  // >= 0: recent <= keep
    int32_t *out = kept + bh * keep;
    if (h == 0 && tid == 0) new_lens[b] = m;
    for (int i = m + tid; i < keep; i += kSelThreads) out[i] = -1;
    if (need == cand) {
        for (int i = tid; i < m; i += kSelThreads) out[i] = i;
        return;
    }
    for (int i = tid; i < len - cand; i += kSelThreads) out[need + i] = cand + i;
    if (need == 0) return;

    auto key_at = [&](int j) -> uint32_t {
        const int page = kv4_page(c, table, b, max_pages, j);
        return page < 0 ? 0u : weight_key(c.weights[kv4_row(c, page, h, j)]);
    };
    uint32_t at = 0;
    for (int bit = 31, turn = 0; bit >= 0; --bit, turn ^= 1) {
        const uint32_t v = at | (1u << bit);
        int n = 0;
        for (int j = tid; j < cand; j += kSelThreads) n += key_at(j) >= v;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) warp_sum[turn][warp] = n;
        __syncthreads();
        if (__reduce_add_sync(0xffffffffu, warp_sum[turn][lane]) >= need) at = v;
    }
    // how many lie above it
    int n = 0;
    for (int j = tid; j < cand; j += kSelThreads) n += key_at(j) > at;
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (lane == 0) warp_sum[0][warp] = n;
    __syncthreads();
    const int ties = need - __reduce_add_sync(0xffffffffu, warp_sum[0][lane]);
    // positions in order, a block of 1024 at a time
    int gt0 = 0, eq0 = 0;
    for (int j0 = 0; j0 < cand; j0 += kSelThreads) {
        const int j = j0 + tid;
        const uint32_t key = j < cand ? key_at(j) : 0u;
        const bool gt = j < cand && key > at, eq = j < cand && key == at;
        const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        __syncthreads();
        if (lane == 0) {
            warp_gt[warp] = __popc(bg);
            warp_eq[warp] = __popc(be);
        }
        __syncthreads();
        const int wg = warp_gt[lane], we = warp_eq[lane];
        const uint32_t below = (1u << lane) - 1u;
        const int gt_before = gt0 + __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0) + __popc(bg & below);
        const int eq_before = eq0 + __reduce_add_sync(0xffffffffu, lane < warp ? we : 0) + __popc(be & below);
        if (gt || (eq && eq_before < ties)) out[gt_before + (eq_before < ties ? eq_before : ties)] = j;
        gt0 += __reduce_add_sync(0xffffffffu, wg);
        eq0 += __reduce_add_sync(0xffffffffu, we);
    }
}

// The kept rows to their new pages: D / 16 threads a row (half for K, half for V),
// 16 bytes each.
template <int D>
__global__ void __launch_bounds__(256)
fa_kv4_move_kernel(Kv4Cache from, Kv4Cache to, const int32_t *__restrict__ table, int64_t max_pages,
                   const int32_t *__restrict__ to_table, int64_t to_max_pages, const int32_t *__restrict__ kept,
                   int64_t rows, int keep)
{
    constexpr int TPR = D / 16, HALF = TPR / 2;
    const int t = threadIdx.x % TPR;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (256 / TPR);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR; r < rows; r += stride) {
        const int src = kept[r];
        if (src < 0) continue;
        const int64_t bh = r / keep, b = bh / from.heads;
        const int h = static_cast<int>(bh - b * from.heads), dst = static_cast<int>(r - bh * keep);
        const int ps = kv4_page(from, table, b, max_pages, src), pd = kv4_page(to, to_table, b, to_max_pages, dst);
        if (ps < 0 || pd < 0) continue;
        const int64_t rs = kv4_row(from, ps, h, src), rd = kv4_row(to, pd, h, dst);
        const int i = t % HALF;
        const uint4 x = reinterpret_cast<const uint4 *>(t < HALF ? from.k : from.v)[rs * HALF + i];
        reinterpret_cast<uint4 *>(t < HALF ? to.k : to.v)[rd * HALF + i] = x;
        if (t == 0) {
            if (D == 128)
                reinterpret_cast<uint32_t *>(to.k_scale)[rd] = reinterpret_cast<const uint32_t *>(from.k_scale)[rs];
            else
                reinterpret_cast<uint16_t *>(to.k_scale)[rd] = reinterpret_cast<const uint16_t *>(from.k_scale)[rs];
        } else if (t == 1) {
            to.v_scale[rd] = from.v_scale[rs];
        } else if (t == 2) {
            to.weights[rd] = from.weights[rs];
        }
    }
}

// Blocks of 256 threads for `rows` rows of `per` threads, at most 16 blocks an SM in one wave.
unsigned row_grid(int64_t rows, int per, int sm_count)
{
    const int64_t want = (rows + 256 / per - 1) / (256 / per), cap = static_cast<int64_t>(sm_count) * 16;
    return static_cast<unsigned>(want < cap ? want : cap);
}

}  // namespace

cudaError_t fa_launch_kv4_append(const Kv4Cache &c, const void *k_new, const void *v_new, const float *w_new,
                                 const int32_t *n_new, const int32_t *lens, const int32_t *table, int64_t B, int64_t S,
                                 int64_t max_pages, int sm_count, cudaStream_t stream)
{
    const int64_t rows = B * c.heads * S;
    auto *kern = c.d == 128 ? fa_kv4_append_kernel<128> : fa_kv4_append_kernel<64>;
    kern<<<row_grid(rows, c.d / 8, sm_count), 256, 0, stream>>>(c, static_cast<const uint4 *>(k_new),
                                                                static_cast<const uint4 *>(v_new), w_new, n_new, lens,
                                                                table, rows, S, max_pages);
    return cudaGetLastError();
}

cudaError_t fa_launch_kv4_read(const Kv4Cache &c, const int32_t *first, const int32_t *lens, const int32_t *table,
                               int64_t B, int64_t max_pages, int64_t T, void *k_out, void *v_out, int sm_count,
                               cudaStream_t stream)
{
    const int64_t rows = B * c.heads * T;
    auto *kern = c.d == 128 ? fa_kv4_read_kernel<128> : fa_kv4_read_kernel<64>;
    kern<<<row_grid(rows, c.d / 8, sm_count), 256, 0, stream>>>(c, first, lens, table, rows, T, max_pages,
                                                                static_cast<uint4 *>(k_out),
                                                                static_cast<uint4 *>(v_out));
    return cudaGetLastError();
}

cudaError_t fa_launch_kv4_evict(const Kv4EvictProblem &p, cudaStream_t stream)
{
    const int64_t bh = p.B * p.from.heads, rows = bh * p.keep;
    if (bh > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    fa_kv4_select_kernel<<<static_cast<unsigned>(bh), kSelThreads, 0, stream>>>(
        p.from, p.lens, p.table, p.max_pages, static_cast<int>(p.keep), static_cast<int>(p.recent), p.kept, p.new_lens);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    auto *kern = p.from.d == 128 ? fa_kv4_move_kernel<128> : fa_kv4_move_kernel<64>;
    kern<<<row_grid(rows, p.from.d / 16, p.sm_count), 256, 0, stream>>>(p.from, p.to, p.table, p.max_pages, p.to_table,
                                                                        p.to_max_pages, p.kept, rows,
                                                                        static_cast<int>(p.keep));
    return cudaGetLastError();
}

int fa_kv4_cache_take_status(cudaStream_t stream) { return kv4_take_status_here(stream); }
