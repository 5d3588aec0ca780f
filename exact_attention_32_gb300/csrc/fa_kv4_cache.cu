// Writing, reading back and evicting from the 4-bit KV cache (format: fa_kv4.cuh).
#include <math.h>

#include "fa_kv4.cuh"

namespace {

// --------------------------------------------------------------------- append

// amax / 6 on the scale grid (to nearest even), as a byte, from amax's bf16 bits; 255 for a block with a NaN or an
// infinity.  amax = X 2^a (X < 256) and a middle of two scales is M 2^b (M < 32), so amax / 6 is a middle exactly or
// differs from it by at least 1 part in 255 (X 2^k against 3 M).  From 2^-14 on, the product with the rounded 1/6,
// rounded to a half (2^-11), is the middle where the quotient is one and keeps the side where it is not; the byte is
// that half's upper bits, to nearest even.  Below, a half's steps are too coarse for the same argument: there the
// rounded quotient (2^-24) is taken to multiples of 2^-17 (adding 96 rounds to its last place).
__device__ __forceinline__ uint32_t kv4_scale_byte(uint32_t amax)
{
    if (amax >= 0x7F80u) return 255u;
    const float x = __uint_as_float(amax << 16);
    const float s = fminf(x * 0.16666667163372039794921875f, 10240.f);
    if (s < 6.2e-05f) {  // (a little above 2^-14, where both ways agree)
        const float q = __fdiv_rn(x, 6.f);
        if (q < 6.103515625e-05f) return __float2uint_rn(__fsub_rn(__fadd_rn(q, 96.f), 96.f) * 131072.f);
    }
    const uint32_t h = __half_as_ushort(__float2half_rn(s));
    return (h + 63u + ((h >> 7) & 1u)) >> 7;
}

// Four bytes of codes of eight values under the scale of `byte`.  x is a bf16 value X 2^a (X < 256), the scale
// n 2^b (n < 16), a middle of two E2M1 values M 2^c (M <= 7), so x / s is a middle exactly or differs from it by at
// least 1 part in 255 (X 2^k against n M <= 105, both whole or X < 256).  The product with 1 / s (rcp.approx, 2^-23) is
// within 2^-22 of x / s, and rounding it to a half (2^-11) gives the middle where x / s is one and keeps the side
// where it is not: the codes are those of the exact quotient, for a third of a division's instructions.
__device__ __forceinline__ uint32_t kv4_codes(const float (&x)[8], uint32_t byte)
{
    if (byte == 0u || byte == 255u) return 0u;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(kv4_scale(byte)));
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 q = __floats2half2_rn(x[2 * i] * r, x[2 * i + 1] * r);
        y[i] = *reinterpret_cast<const uint32_t *>(&q);
    }
    return kv4_encode8(y);
}

// Larger of two pairs of unsigned 16-bit values.  The bits of |x| order bf16 values, infinities and NaNs (above all).
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight bf16 values as fp32; returns the bits of the largest |x|, in both halves.
__device__ __forceinline__ uint32_t unpack8(uint4 u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    const uint32_t m = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                 max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max_u16x2(m, __byte_perm(m, m, 0x1032));
}

// n / d and n % d of row indices, in 32 bits where all of them fit (a 64-bit division costs as much as the rest of a row).
__device__ __forceinline__ int64_t row_div(int64_t n, int64_t d, int64_t rows, int64_t *rest)
{
    if (rows <= 0x7fffffffLL) {
        const uint32_t q = static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
        *rest = static_cast<uint32_t>(n) - q * static_cast<uint32_t>(d);
        return q;
    }
    const int64_t q = n / d;
    *rest = n - q * d;
    return q;
}

// D / 16 threads a row, 16 channels of K and of V each: the maxima over 2 threads (a K
// block) and over the row (V) by shuffles, eight bytes of codes out of each.  4 d bytes in and d + d/32 + 1 out a row;
// with eight channels a thread the work of finding a row's place, done by all of its threads, bound it (43 us in
// place of 32 for 8 x 8 heads of up to 4096 tokens, 104 MB: 3.3 TB/s, two thirds of the issue slots).  The values are asked
// for before the row's page is known.  A division a row and thread, for its place and for x / s, cost 63 us.
template <int D>
__global__ void __launch_bounds__(256)
fa_kv4_append_kernel(Kv4Cache c, const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                     const float *__restrict__ w_new, const int32_t *__restrict__ n_new,
                     const int32_t *__restrict__ lens, const int32_t *__restrict__ table, int64_t rows, int64_t S,
                     int64_t max_pages)
{
    constexpr int TPR = D / 16, kStep = 256 / TPR;  // rows of a block at a time
    const int t = threadIdx.x % TPR;
    bool bad = false;
    // whole warps stay in the loop together
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kStep; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kStep) {
        const int64_t r = r0 + threadIdx.x / TPR, rr = r < rows ? r : 0;
        int64_t at, h;
        const int64_t bh = row_div(rr, S, rows, &at), b = row_div(bh, c.heads, rows, &h);
        int n = n_new != nullptr ? n_new[b] : static_cast<int>(S);
        n = n < 0 ? 0 : (n > S ? static_cast<int>(S) : n);
        const bool mine = r < rows && at < n;
        if (!__any_sync(0xffffffffu, mine)) continue;  // (past the tokens of a short sequence)
        uint4 uk[2], uv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uk[i] = uv[i] = make_uint4(0, 0, 0, 0);
            if (mine) {
                uk[i] = k_new[(rr * TPR + t) * 2 + i];
                uv[i] = v_new[(rr * TPR + t) * 2 + i];
            }
        }
        const float w = mine && t == 0 && w_new != nullptr ? w_new[rr] : 0.f;
        // the place is made of the length as it is given: held to the table, a length past it would put the tokens over others
        const int64_t place = at - n + lens[b];
        const bool in = mine && place >= 0 && place < (max_pages << c.log2_page);
        const int pos = in ? static_cast<int>(place) : 0;  // (a thread without a place looks up position 0's page, and drops it)
        bool valid;
        const int page = kv4_page_quiet(c, table, b, max_pages, pos, &valid);
        valid = valid && in;
        bad |= mine && !valid;
        float xk[2][8], xv[2][8];
        uint32_t mk = max_u16x2(unpack8(uk[0], xk[0]), unpack8(uk[1], xk[1]));
        uint32_t mv = max_u16x2(unpack8(uv[0], xv[0]), unpack8(uv[1], xv[1]));
        mk = max_u16x2(mk, __shfl_xor_sync(0xffffffffu, mk, 1));
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) mv = max_u16x2(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        if (!mine || !valid) continue;
        const int64_t row = kv4_row(c, page, static_cast<int>(h), pos);
        const uint32_t bk = kv4_scale_byte(mk & 0xFFFFu), bv = kv4_scale_byte(mv & 0xFFFFu);
        reinterpret_cast<uint2 *>(c.k)[row * TPR + t] = make_uint2(kv4_codes(xk[0], bk), kv4_codes(xk[1], bk));
        reinterpret_cast<uint2 *>(c.v)[row * TPR + t] = make_uint2(kv4_codes(xv[0], bv), kv4_codes(xv[1], bv));
        if ((t & 1) == 0) c.k_scale[row * (D / 32) + (t >> 1)] = static_cast<uint8_t>(bk);
        if (t == 0) {
            c.v_scale[row] = static_cast<uint8_t>(bv);
            if (c.weights != nullptr) c.weights[row] = w;
        }
    }
    if (bad) kv4_report();
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

// D / 8 threads a row, eight channels each of K and V.  Memory-bound by the 4 d bytes written a row: 4 x 8 heads of 16384
// tokens, 338 MB, in 54 us (6.3 TB/s; the copy's rate would take 50).  16 channels a thread, whose stores then leave gaps, took
// 75 us; two or four rows a thread under way, or a block for each 16 rows without a loop, were no faster or up to 15 % slower.
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
        int64_t at, head;
        const int64_t bh = row_div(r, T, rows, &at), b = row_div(bh, c.heads, rows, &head);
        const int h = static_cast<int>(head);
        const int64_t pos = at + (first != nullptr ? first[b] : 0);
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

// The `need` (1 .. cand - 1) candidates with the largest keys, ties to the lowest position, to out[0 .. need) in order.
// Thread t has the keys of positions i 1024 + t (those past 1024 KPT are read again each time).  The need-th largest
// key is found 11 bits at a time from the top: a histogram of the digit over the keys that share the digits so far,
// and the digit at which its sums from above reach what is still needed.  Above the key all stay, at it the first
// `ties`.  (Bit by bit, with the keys counted against 32 bounds, 15360 candidates took 30 us; with digits of 8 bits 22 us:
// the first is nearly the exponent, and a warp's additions meet on few counters.  With 11 bits it takes 19 us for 16 x 8 heads
// of up to 15360 candidates: one block each, so latency; the weights themselves are 6 MB.)
constexpr int kBins = 2048;
struct SelectShared {
    uint32_t counts[kBins];  // the histogram, then the places
    int warp_sum[32];
    int digit, rest;
};

template <int KPT, bool MORE, typename KeyAt>
__device__ __forceinline__ void select_top(KeyAt key_at, int cand, int need, int32_t *out, SelectShared &sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t (&counts)[kBins] = sh.counts;
    uint32_t key[KPT];
#pragma unroll
    for (int i = 0; i < KPT; ++i) key[i] = key_at(min(i * kSelThreads + tid, cand - 1));
    uint32_t at = 0, mask = 0;
    int ties = need;
    for (int turn = 0; turn < 3; ++turn) {
        const int shift = turn == 0 ? 21 : turn == 1 ? 10 : 0;
        const uint32_t bins = turn == 2 ? 1024u : 2048u;
        counts[tid] = 0;
        counts[tid + 1024] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KPT; ++i)
            if (i * kSelThreads + tid < cand && (key[i] & mask) == at) atomicAdd(&counts[(key[i] >> shift) & (bins - 1u)], 1u);
        for (int j = KPT * kSelThreads + tid; MORE && j < cand; j += kSelThreads) {
            const uint32_t k = key_at(j);
            if ((k & mask) == at) atomicAdd(&counts[(k >> shift) & (bins - 1u)], 1u);
        }
        __syncthreads();
        // thread t: digits 2047 - 2t and 2046 - 2t, and the sum from the top down to them
        const int c0 = static_cast<int>(counts[2047 - 2 * tid]), c1 = static_cast<int>(counts[2046 - 2 * tid]);
        int sum = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) sh.warp_sum[warp] = sum;
        __syncthreads();
        sum += __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0);
        const int before0 = sum - c0 - c1, before1 = sum - c1;
        if (sum >= ties && before0 < ties) {
            const bool first = before1 >= ties;
            sh.digit = first ? 2047 - 2 * tid : 2046 - 2 * tid;
            sh.rest = ties - (first ? before0 : before1);
        }
        __syncthreads();
        at |= static_cast<uint32_t>(sh.digit) << shift;
        mask |= (bins - 1u) << shift;
        ties = sh.rest;
    }
    __syncthreads();
    // positions in order, in rounds of up to 1024 KPT: how many above and at the bound each warp has in each block of 1024,
    // their prefix sums (16 bits each), and each thread's place
    int gt0 = 0, eq0 = 0;
    const uint32_t below = (1u << lane) - 1u;
    for (int j0 = 0; j0 < cand; j0 += KPT * kSelThreads) {
        uint32_t bg[KPT], be[KPT];
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int j = j0 + i * kSelThreads + tid;
            if (MORE && j0 > 0) key[i] = j < cand ? key_at(j) : 0u;
            bg[i] = __ballot_sync(0xffffffffu, j < cand && key[i] > at);
            be[i] = __ballot_sync(0xffffffffu, j < cand && key[i] == at);
            if (lane == 0) counts[i * 32 + warp] = __popc(bg[i]) | (__popc(be[i]) << 16);
        }
        __syncthreads();
        const uint32_t own = tid < KPT * 32 ? counts[tid] : 0u;
        uint32_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) sh.warp_sum[warp] = static_cast<int>(sum);
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (int i = 0; i < KPT; ++i) {  // (the first KPT warps hold the counts)
            const uint32_t n = static_cast<uint32_t>(sh.warp_sum[i]);
            if (i < warp) before += n;
            all += n;
        }
        if (tid < KPT * 32) counts[tid] = before + sum - own;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int j = j0 + i * kSelThreads + tid;
            const uint32_t n = counts[i * 32 + warp];
            const int gt = gt0 + static_cast<int>(n & 0xFFFFu) + __popc(bg[i] & below);
            const int eq = eq0 + static_cast<int>(n >> 16) + __popc(be[i] & below);
            if (((bg[i] >> lane) & 1u) || (((be[i] >> lane) & 1u) && eq < ties)) out[gt + (eq < ties ? eq : ties)] = j;
        }
        gt0 += all & 0xFFFFu;
        eq0 += all >> 16;
        __syncthreads();  // before the next round's counts
    }
}

// Which tokens of one (sequence, key head) stay: a block each.
__global__ void __launch_bounds__(kSelThreads)
fa_kv4_select_kernel(Kv4Cache c, const int32_t *__restrict__ lens, const int32_t *__restrict__ table,
                     int64_t max_pages, int keep, int recent, int32_t *__restrict__ kept,
                     int32_t *__restrict__ new_lens)
{
    __shared__ SelectShared sh;
    const int tid = threadIdx.x;
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
    bool bad = false;
    auto key_at = [&](int j) -> uint32_t {  // (no branch: a thread's loads go out together)
        bool valid;
        const int page = kv4_page_quiet(c, table, b, max_pages, j, &valid);
        const float w = c.weights[kv4_row(c, page, h, j)];
        bad |= !valid;
        return valid ? weight_key(w) : 0u;
    };
    if (cand <= 4 * kSelThreads)
        select_top<4, false>(key_at, cand, need, out, sh);
    else if (cand <= 16 * kSelThreads)
        select_top<16, false>(key_at, cand, need, out, sh);
    else
        select_top<16, true>(key_at, cand, need, out, sh);
    if (bad) kv4_report();
}

// The kept rows to their new pages: D / 16 threads a row (half for K, half for V),
// 16 bytes each.  Memory-bound; a row waits for its position, then the pages, then the row,
// so a thread has two rows under way.  16 x 8 heads of 4096 rows kept of up to 16384, 146 MB in pieces of 64 bytes and
// less: 35 us (4.2 TB/s).
template <int D>
__global__ void __launch_bounds__(256)
fa_kv4_move_kernel(Kv4Cache from, Kv4Cache to, const int32_t *__restrict__ table, int64_t max_pages,
                   const int32_t *__restrict__ to_table, int64_t to_max_pages, const int32_t *__restrict__ kept,
                   int64_t rows, int keep)
{
    constexpr int TPR = D / 16, HALF = TPR / 2, U = 2;
    const int t = threadIdx.x % TPR, i = t % HALF;
    constexpr int kStep = 256 / TPR;  // rows of a block at a time
    bool bad = false;
    kv4_wait_for_the_one_before();  // (the selection)
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * (U * kStep) + threadIdx.x / TPR; r0 < rows;
         r0 += static_cast<int64_t>(gridDim.x) * (U * kStep)) {
        int src[U];
        int64_t rs[U], rd[U];
        uint4 x[U];
        uint32_t y[U];
        bool go[U], there[U];
#pragma unroll
        for (int u = 0; u < U; ++u) src[u] = r0 + u * kStep < rows ? kept[r0 + u * kStep] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int64_t dst, h;
            const int64_t bh = row_div(min(r0 + u * kStep, rows - 1), keep, rows, &dst), b = row_div(bh, from.heads, rows, &h);
            bool vd;
            const int ps = kv4_page_quiet(from, table, b, max_pages, max(src[u], 0), &there[u]);
            const int pd = kv4_page_quiet(to, to_table, b, to_max_pages, static_cast<int>(dst), &vd);
            rs[u] = kv4_row(from, ps, static_cast<int>(h), max(src[u], 0));
            rd[u] = kv4_row(to, pd, static_cast<int>(h), static_cast<int>(dst));
            go[u] = src[u] >= 0 && vd;
            bad |= src[u] >= 0 && !(there[u] && vd);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = reinterpret_cast<const uint4 *>(t < HALF ? from.k : from.v)[rs[u] * HALF + i];
            // the row's small parts, one a thread: K's scales, V's scale, the weight
            y[u] = 0;
            if (t == 0)
                y[u] = D == 128 ? reinterpret_cast<const uint32_t *>(from.k_scale)[rs[u]]
                                : reinterpret_cast<const uint16_t *>(from.k_scale)[rs[u]];
            if (t == 1) y[u] = from.v_scale[rs[u]];
            if (t == 2) y[u] = reinterpret_cast<const uint32_t *>(from.weights)[rs[u]];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!go[u]) continue;
            if (!there[u]) {  // a token that no page holds: zeros without weight, not what lies in the new page
                x[u] = make_uint4(0, 0, 0, 0);
                y[u] = 0;
            }
            reinterpret_cast<uint4 *>(t < HALF ? to.k : to.v)[rd[u] * HALF + i] = x[u];
            if (t == 0) {
                if (D == 128)
                    reinterpret_cast<uint32_t *>(to.k_scale)[rd[u]] = y[u];
                else
                    reinterpret_cast<uint16_t *>(to.k_scale)[rd[u]] = static_cast<uint16_t>(y[u]);
            }
            if (t == 1) to.v_scale[rd[u]] = static_cast<uint8_t>(y[u]);
            if (t == 2) reinterpret_cast<uint32_t *>(to.weights)[rd[u]] = y[u];
        }
    }
    if (bad) kv4_report();
}

// Blocks of 256 threads for `rows` rows of `per` threads, `turns` rows a thread; at most `waves` x 8 blocks an SM (then
// a block takes several turns).
unsigned row_grid(int64_t rows, int per, int turns, int sm_count, int waves = 2)
{
    const int64_t step = 256 / per * turns, want = (rows + step - 1) / step, cap = static_cast<int64_t>(sm_count) * 8 * waves;
    return static_cast<unsigned>(want < cap ? want : cap);
}

}  // namespace

cudaError_t fa_launch_kv4_append(const Kv4Cache &c, const void *k_new, const void *v_new, const float *w_new,
                                 const int32_t *n_new, const int32_t *lens, const int32_t *table, int64_t B, int64_t S,
                                 int64_t max_pages, int sm_count, cudaStream_t stream)
{
    const int64_t rows = B * c.heads * S;
    auto *kern = c.d == 128 ? fa_kv4_append_kernel<128> : fa_kv4_append_kernel<64>;
    kern<<<row_grid(rows, c.d / 16, 1, sm_count, 64), 256, 0, stream>>>(c, static_cast<const uint4 *>(k_new),
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
    kern<<<row_grid(rows, c.d / 8, 1, sm_count), 256, 0, stream>>>(c, first, lens, table, rows, T, max_pages,
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
    return kv4_launch_behind(kern, dim3(row_grid(rows, p.from.d / 16, 2, p.sm_count, 64)), 256, stream, p.from, p.to, p.table, p.max_pages,
                             p.to_table, p.to_max_pages, p.kept, rows, static_cast<int>(p.keep));
}

int fa_kv4_cache_take_status(cudaStream_t stream) { return kv4_take_status_here(stream); }
