// Attention of the newest tokens over a 4-bit KV cache (fa_fwd_kv4).
//
// For each (sequence, key head) the R = H / Hkv * n_q query rows that share its
// keys go together, so a key's 4-bit row is read and decoded once for all of them:
//     S = scale q K^T,  O = softmax(S) V,  LSE = ln sum exp S
// with one pass over the keys, a running maximum m and sum l per row, and O
// rescaled when m grows.  The keys are cut into chunks; every CTA takes one chunk
// of one (sequence, key head) and up to 32 rows, its warps take 32 keys a step, and
// nothing is exchanged until the end: the warps' (m, l, O) are merged in shared
// memory, the chunks' in a second kernel (O = sum 2^(m_s - m) O_s / sum 2^(m_s - m) l_s).
//
// What bounds it is the bytes of the cache (133 a key and head at d = 128), so
// the K and V codes go from global memory straight into registers in the layout
// of the warp-level MMA (m16n8k16, f16 in, fp32 out), where the decoded halves are
// its A operand: a tile's 16 keys (K) or 16 channels (V) are its M, eight query
// rows its N.  Per pair of values that costs one conversion and, for K, one multiply
// by the scale, for V one byte permute; there is no shared-memory traffic in the
// loop and no barrier.  Both products are exact in what they multiply: q is bf16
// scaled by a power of two into a half (its maximum at 2^14, so only values 2^28
// below the row's maximum lose bits), a K value is exact in a half, a V code is
// too.  P is rounded once, to a half: p <= 1 times V's scale times 4 (at most
// 40960), relative error 2^-11, below bf16's 2^-8 of the output; the sum l takes
// the unrounded p in fp32.
#include <math.h>

#include "fa_kv4.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kStep = 32;                  // keys a warp takes at a time
constexpr int kChunkUnit = kWarps * kStep;  // chunks are a multiple of this
constexpr int kMaxChunk = 4096;
constexpr float kLn2 = 0.69314718055994531f;

struct DecodeArgs {
    Kv4Cache c;
    const __nv_bfloat16 *q;
    const int32_t *lens, *table;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o;    // [rows][n_splits][D], unnormalised
    float2 *part_ml;  // [rows][n_splits]: running maximum (log2), sum
    float *scores;    // [B][heads][R][max_tokens] log2 scores, or null
    float2 *row_ml;   // [rows]: maximum (log2), 1 / sum; with scores
    int64_t max_pages;
    int R, n_q, n_rc, n_splits, chunk;
    float scale_log2;
};

__device__ __forceinline__ float ex2f(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of halves held a row per quad (two columns a lane).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Streaming loads: each byte of the cache is read once by one SM.
template <int WORDS>
__device__ __forceinline__ void ld_stream(const void *p, uint32_t (&r)[WORDS])
{
    if constexpr (WORDS == 4)
        asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
            : "l"(p));
    else if constexpr (WORDS == 2)
        asm("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
    else
        asm("ld.global.nc.L1::no_allocate.u32 %0, [%1];\n" : "=r"(r[0]) : "l"(p));
}

// 16 keys of K as one lane holds them: of keys g and g + 8 (g = lane / 4) the D/4
// channels from t * D/4 (t = lane % 4), and the scales of those channels' block.
template <int D>
struct KTile {
    uint32_t x[2][D / 32];
    uint32_t s[2];
};
// 16 keys of V: of keys 2t, 2t+1, 2t+8, 2t+9 the D/8 channels from g * D/8; the
// scales of keys g and g + 8.
template <int D>
struct VTile {
    uint32_t x[4][D / 64];
    uint32_t s[2];
};

template <int D, int RT, bool SCORES>
__global__ void __launch_bounds__(kWarps * 32, RT == 1 ? 4 : RT == 2 ? 3 : 2)
fa_kv4_decode_kernel(const DecodeArgs a)
{
    constexpr int ROWS = 8 * RT;
    constexpr int KW = D / 32, VW = D / 64, MT = D / 16;
    extern __shared__ __align__(16) float sm_o[];  // [kWarps][ROWS][D], for the warps' merge
    __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
    __shared__ int sm_page[kMaxChunk / 16 + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

    const int split = blockIdx.x % a.n_splits;
    const int64_t item = blockIdx.x / a.n_splits;
    const int rc = static_cast<int>(item % a.n_rc);
    const int64_t bh = item / a.n_rc, b = bh / a.c.heads;
    const int h = static_cast<int>(bh - b * a.c.heads);
    const int row0 = rc * ROWS, n_rows = min(ROWS, a.R - row0);
    const int len = kv4_length(a.lens, b, a.max_pages << a.c.log2_page);
    const int k_begin = split * a.chunk;
    if (k_begin >= len && split > 0) return;  // (the merge counts the chunks from the length)
    const int k_end = min(len, k_begin + a.chunk);

    // pages of this chunk
    const int page0 = k_begin >> a.c.log2_page;
    const int n_pg = k_end > k_begin ? ((k_end - 1) >> a.c.log2_page) - page0 + 1 : 0;
    for (int i = tid; i < n_pg; i += kWarps * 32)
        sm_page[i] = kv4_page(a.c, a.table, b, a.max_pages, (page0 + i) << a.c.log2_page);

    // Q as the MMA's B operand: lane (g, t) holds row g's channels from t * D/4, in halves
    uint32_t qb[RT][MT][2];
    float mult[RT][2];  // log2 score of rows 2t, 2t + 1 per unit of the product
    int limit[RT][2];   // keys those rows admit
    {
        const __nv_bfloat16 *q0 = a.q + (bh * a.R + row0) * D;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            uint32_t x[MT][2];
            float amax = 0.f;
            const bool live = rt * 8 + g < n_rows;
#pragma unroll
            for (int i = 0; i < MT / 2; ++i) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live) u = *reinterpret_cast<const uint4 *>(q0 + (rt * 8 + g) * D + t * (D / 4) + i * 8);
                x[2 * i][0] = u.x;
                x[2 * i][1] = u.y;
                x[2 * i + 1][0] = u.z;
                x[2 * i + 1][1] = u.w;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[i][j] << 16)),
                                             fabsf(__uint_as_float(x[i][j] & 0xFFFF0000u))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // exponent of the row's maximum, held where 2^(14 - e) and 2^(e - 14) are normal numbers
            int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
            e = amax == 0.f || e > 127 ? 14 : max(e, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    qb[rt][i][j] = pack_h2(__uint_as_float(x[i][j] << 16) * up,
                                           __uint_as_float(x[i][j] & 0xFFFF0000u) * up);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int er = __shfl_sync(0xffffffffu, e, (2 * t + j) * 4);
                mult[rt][j] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(er - 14 + 127) << 23);
                limit[rt][j] = len - a.n_q + 1 + (row0 + rt * 8 + 2 * t + j) % a.n_q;
            }
        }
    }
    __syncthreads();

    float m[RT][2], l[RT][2], acc[RT][MT][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[rt][j] = -INFINITY;
            l[rt][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[rt][i][j] = 0.f;
    }

    // row of the pool that holds the first of 16 keys from `key`, or -1 (nothing to read)
    auto row_of = [&](int key) -> int64_t {
        if (key >= k_end) return -1;
        const int page = sm_page[(key >> a.c.log2_page) - page0];
        return page < 0 ? -1 : kv4_row(a.c, page, h, key);
    };
    auto load_k = [&](KTile<D> &kt, int64_t row) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            kt.s[j] = 0;
#pragma unroll
            for (int i = 0; i < KW; ++i) kt.x[j][i] = 0;
            if (row >= 0) {
                const int64_t r = row + g + 8 * j;
                ld_stream<KW>(a.c.k + r * (D / 2) + t * (D / 8), kt.x[j]);
                kt.s[j] = __ldg(a.c.k_scale + r * (D / 32) + t * (D / 32) / 4);
            }
        }
    };
    auto load_v = [&](VTile<D> &vt, int64_t row) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < VW; ++i) vt.x[j][i] = 0;
            if (row >= 0) ld_stream<VW>(a.c.v + (row + 2 * t + (j & 1) + 8 * (j >> 1)) * (D / 2) + g * (D / 16), vt.x[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) vt.s[j] = row >= 0 ? __ldg(a.c.v_scale + row + g + 8 * j) : 0;
    };

    KTile<D> kt[2];
    VTile<D> vt[2];
    int key = k_begin + warp * kStep;
    int64_t rows[2] = {row_of(key), row_of(key + 16)};
#pragma unroll
    for (int u = 0; u < 2; ++u) load_k(kt[u], rows[u]);
#pragma unroll
    for (int u = 0; u < 2; ++u) load_v(vt[u], rows[u]);

    for (; key < k_end; key += kChunkUnit) {
        const int64_t next[2] = {row_of(key + kChunkUnit), row_of(key + kChunkUnit + 16)};
        float x[RT][2][4];  // scores of keys g, g + 8 of each tile: (g, 2t), (g, 2t+1), (g+8, 2t), (g+8, 2t+1)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t s0 = (kt[u].s[0] << 7) * 0x10001u, s1 = (kt[u].s[1] << 7) * 0x10001u;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[rt][u][i] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t r0[4], r1[4];
                kv4_decode8(kt[u].x[0][w], r0);
                kv4_decode8(kt[u].x[1][w], r1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r0[i] = mul_h2(r0[i], s0);
                    r1[i] = mul_h2(r1[i], s1);
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    mma16816(x[rt][u], r0[0], r1[0], r0[1], r1[1], qb[rt][2 * w][0], qb[rt][2 * w][1]);
                    mma16816(x[rt][u], r0[2], r1[2], r0[3], r1[3], qb[rt][2 * w + 1][0], qb[rt][2 * w + 1][1]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) load_k(kt[u], next[u]);

        // log2 scores; keys that a row does not admit, or that no page holds, leave it
        float vs[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) vs[u][j] = kv4_scale(vt[u].s[j]) * 4.f;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[rt][u][i] *= mult[rt][i & 1];
        const bool edge = key + kStep > len - a.n_q + 1 || key + kStep > k_end || rows[0] < 0 || rows[1] < 0;
        if (edge) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int kk = key + 16 * u + g + 8 * j;
                    const bool gone = rows[u] < 0 || kk >= k_end;
                    if (gone) vs[u][j] = 0.f;  // what lies behind the length may be anything
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (gone || kk >= limit[rt][i]) x[rt][u][2 * j + i] = -INFINITY;
                }
        }
        if constexpr (SCORES) {
            const int64_t cap = a.max_pages << a.c.log2_page;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = rt * 8 + 2 * t + i;
                    if (r < n_rows) {
                        float *s = a.scores + (bh * a.R + row0 + r) * cap + key + g;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (key + 16 * u + g + 8 * j < k_end) s[16 * u + 8 * j] = x[rt][u][2 * j + i];
                    }
                }
        }
        // the running maximum: grown only where some key passes it, which soon is rare
        bool grows = false;
        float mx[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[rt][i] = fmaxf(fmaxf(x[rt][0][i], x[rt][0][2 + i]), fmaxf(x[rt][1][i], x[rt][1][2 + i]));
                grows |= mx[rt][i] > m[rt][i];
            }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float al[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = mx[rt][i];
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    v = fmaxf(v, m[rt][i]);
                    al[i] = m[rt][i] == -INFINITY ? 0.f : ex2f(m[rt][i] - v);  // (nothing yet: l and O are 0)
                    if (m[rt][i] == v) al[i] = 1.f;
                    m[rt][i] = v;
                    l[rt][i] *= al[i];
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[rt][i][j] *= al[j & 1];
            }
        }
        // P: the sum in fp32, the MMA's operand as halves times V's scale times 4
        uint32_t pb[RT][2][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float m0 = m[rt][0] == -INFINITY ? 0.f : m[rt][0], m1 = m[rt][1] == -INFINITY ? 0.f : m[rt][1];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p0 = ex2f(x[rt][u][2 * j] - m0), p1 = ex2f(x[rt][u][2 * j + 1] - m1);
                    l[rt][0] += p0;
                    l[rt][1] += p1;
                    float y0 = p0 * vs[u][j], y1 = p1 * vs[u][j];
                    if (edge) {  // a value that a row does not admit stays out of it, a NaN too
                        if (x[rt][u][2 * j] == -INFINITY) y0 = 0.f;
                        if (x[rt][u][2 * j + 1] == -INFINITY) y1 = 0.f;
                    }
                    pb[rt][u][j] = movmatrix_trans(pack_h2(y0, y1));
                }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                uint32_t r[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kv4_decode8(vt[u].x[j][w], r[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = __byte_perm(r[0][i], r[1][i], 0x5410), a1 = __byte_perm(r[0][i], r[1][i], 0x7632);
                    const uint32_t a2 = __byte_perm(r[2][i], r[3][i], 0x5410), a3 = __byte_perm(r[2][i], r[3][i], 0x7632);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) mma16816(acc[rt][4 * w + i], a0, a1, a2, a3, pb[rt][u][0], pb[rt][u][1]);
                }
            }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            load_v(vt[u], next[u]);
            rows[u] = next[u];
        }
    }

    // the warps' states: l over the lanes, then all through shared memory
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v = l[rt][i];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            if (g == 0) {
                sm_m[warp][rt * 8 + 2 * t + i] = m[rt][i];
                sm_l[warp][rt * 8 + 2 * t + i] = v;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                *reinterpret_cast<float2 *>(sm_o + (warp * ROWS + rt * 8 + 2 * t + i) * D + g * (D / 8) + 2 * mt) =
                    make_float2(acc[rt][mt][i], acc[rt][mt][2 + i]);
        }
    }
    __syncthreads();
    for (int e = tid; e < n_rows * (D / 4); e += kWarps * 32) {
        const int r = e / (D / 4), ch = (e % (D / 4)) * 4;
        float mm = sm_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][r]);
        float ll = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_m[w][r] == -INFINITY && !isnan(sm_l[w][r]) ? 0.f : ex2f(sm_m[w][r] - mm);
            const float4 v = *reinterpret_cast<const float4 *>(sm_o + (w * ROWS + r) * D + ch);
            ll = fmaf(f, sm_l[w][r], ll);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        o.x *= 0.25f;  // P carried a factor of 4
        o.y *= 0.25f;
        o.z *= 0.25f;
        o.w *= 0.25f;
        const int64_t row = bh * a.R + row0 + r;
        if (a.n_splits > 1) {
            *reinterpret_cast<float4 *>(a.part_o + (row * a.n_splits + split) * D + ch) = o;
            if (ch == 0) a.part_ml[row * a.n_splits + split] = make_float2(mm, ll);
        } else {
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            uint2 y;
            const __nv_bfloat162 y0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), y1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
            y.x = *reinterpret_cast<const uint32_t *>(&y0);
            y.y = *reinterpret_cast<const uint32_t *>(&y1);
            *reinterpret_cast<uint2 *>(a.o + row * D + ch) = y;
            if (ch == 0) {
                a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
                if (SCORES) a.row_ml[row] = make_float2(ll == 0.f ? 0.f : mm, inv);
            }
        }
    }
}

// Merge of a row's chunks: one warp a row, D/32 channels a lane.
template <int D>
__global__ void __launch_bounds__(128)
fa_kv4_merge_kernel(const DecodeArgs a, int64_t rows)
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int64_t b = row / a.R / a.c.heads;
    const int len = kv4_length(a.lens, b, a.max_pages << a.c.log2_page);
    const int parts = max(1, (len + a.chunk - 1) / a.chunk);
    const float2 *ml = a.part_ml + row * a.n_splits;
    float m = -INFINITY;
    for (int s = lane; s < parts; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = 0.f;
    const float *po = a.part_o + row * a.n_splits * D + lane * PER;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
        const float2 v = ml[s];
        const float f = v.x == -INFINITY && !isnan(v.y) ? 0.f : ex2f(v.x - m);
        l = fmaf(f, v.y, l);
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = fmaf(f, po[static_cast<int64_t>(s) * D + i], x[i]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < PER; i += 2)
        *reinterpret_cast<__nv_bfloat162 *>(a.o + row * D + lane * PER + i) = __floats2bfloat162_rn(x[i] * inv, x[i + 1] * inv);
    if (lane == 0) {
        a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        if (a.scores != nullptr) a.row_ml[row] = make_float2(l == 0.f ? 0.f : m, inv);
    }
}

// weights[key] += sum over the rows of exp2(score - m) / l: one thread a key.
__global__ void __launch_bounds__(256)
fa_kv4_weights_kernel(const DecodeArgs a, int blocks)
{
    const int64_t bh = blockIdx.x / blocks, b = bh / a.c.heads;
    const int h = static_cast<int>(bh - b * a.c.heads);
    const int64_t cap = a.max_pages << a.c.log2_page;
    const int len = kv4_length(a.lens, b, cap);
    for (int key = blockIdx.x % blocks * 256 + threadIdx.x; key < len; key += blocks * 256) {
        const int page = kv4_page(a.c, a.table, b, a.max_pages, key);
        if (page < 0) continue;
        const float *s = a.scores + bh * a.R * cap + key;
        const float2 *ml = a.row_ml + bh * a.R;
        float w = 0.f;
#pragma unroll 4
        for (int r = 0; r < a.R; ++r) w = fmaf(ex2f(s[r * cap] - ml[r].x), ml[r].y, w);
        a.c.weights[kv4_row(a.c, page, h, key)] += w;
    }
}

// ------------------------------------------------------------------ host side

struct Geometry {
    int rt, n_rc, n_splits, chunk;
    int64_t part_o, part_ml, scores, row_ml, total;  // byte offsets in the workspace
};

// The split of the keys, from the sizes alone (152 SMs, 4 CTAs each, four waves of
// them where the keys allow: sequences are seldom of equal length).
Geometry geometry(int64_t B, int64_t H, int64_t heads, int64_t n_q, int64_t d, int64_t max_tokens, int accumulate)
{
    Geometry g;
    const int64_t R = H / heads * n_q, rows = B * H * n_q;
    g.rt = R <= 8 ? 1 : R <= 16 ? 2 : 4;
    g.n_rc = static_cast<int>((R + 8 * g.rt - 1) / (8 * g.rt));
    const int64_t items = B * heads * g.n_rc, want = 152 * 4 * 4;
    int64_t splits = (want + items - 1) / items;
    int64_t chunk = (max_tokens + splits - 1) / splits;
    if (chunk < 2 * kChunkUnit) chunk = 2 * kChunkUnit;
    if (chunk > kMaxChunk) chunk = kMaxChunk;
    chunk = (chunk + kChunkUnit - 1) / kChunkUnit * kChunkUnit;
    g.chunk = static_cast<int>(chunk);
    g.n_splits = static_cast<int>((max_tokens + chunk - 1) / chunk);
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    int64_t at = 0;
    g.part_o = at;
    if (g.n_splits > 1) at = up(at + rows * g.n_splits * d * 4);
    g.part_ml = at;
    if (g.n_splits > 1) at = up(at + rows * g.n_splits * 8);
    g.scores = at;
    if (accumulate) at = up(at + rows * max_tokens * 4);
    g.row_ml = at;
    if (accumulate) at = up(at + rows * 8);
    g.total = at < 256 ? 256 : at;
    return g;
}

template <int D, int RT, bool SCORES>
cudaError_t launch(const DecodeArgs &a, int64_t ctas, cudaStream_t s)
{
    constexpr int kSmem = kWarps * 8 * RT * D * 4;
    cudaError_t e = set_max_dynamic_smem<fa_kv4_decode_kernel<D, RT, SCORES>>(kSmem);
    if (e != cudaSuccess) return e;
    fa_kv4_decode_kernel<D, RT, SCORES><<<static_cast<unsigned>(ctas), kWarps * 32, kSmem, s>>>(a);
    return cudaGetLastError();
}

template <int D, bool SCORES>
cudaError_t launch_rt(const DecodeArgs &a, int rt, int64_t ctas, cudaStream_t s)
{
    return rt == 1 ? launch<D, 1, SCORES>(a, ctas, s)
                   : rt == 2 ? launch<D, 2, SCORES>(a, ctas, s) : launch<D, 4, SCORES>(a, ctas, s);
}

}  // namespace

int64_t fa_kv4_decode_workspace(int64_t B, int64_t H, int64_t heads, int64_t n_q, int64_t d, int64_t max_tokens,
                                int accumulate)
{
    return geometry(B, H, heads, n_q, d, max_tokens, accumulate).total;
}

cudaError_t fa_launch_kv4_decode(const Kv4DecodeProblem &p, void *workspace, cudaStream_t stream)
{
    const int64_t cap = p.max_pages << p.cache.log2_page, heads = p.cache.heads;
    const Geometry g = geometry(p.B, p.H, heads, p.n_q, p.cache.d, cap, p.accumulate);
    const int64_t rows = p.B * p.H * p.n_q, ctas = p.B * heads * g.n_rc * g.n_splits;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    char *ws = static_cast<char *>(workspace);
    DecodeArgs a;
    a.c = p.cache;
    a.q = static_cast<const __nv_bfloat16 *>(p.q);
    a.lens = p.lens;
    a.table = p.table;
    a.o = static_cast<__nv_bfloat16 *>(p.o);
    a.lse = p.lse;
    a.part_o = reinterpret_cast<float *>(ws + g.part_o);
    a.part_ml = reinterpret_cast<float2 *>(ws + g.part_ml);
    a.scores = p.accumulate ? reinterpret_cast<float *>(ws + g.scores) : nullptr;
    a.row_ml = reinterpret_cast<float2 *>(ws + g.row_ml);
    a.max_pages = p.max_pages;
    a.R = static_cast<int>(p.H / heads * p.n_q);
    a.n_q = static_cast<int>(p.n_q);
    a.n_rc = g.n_rc;
    a.n_splits = g.n_splits;
    a.chunk = g.chunk;
    a.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    cudaError_t e;
    if (p.cache.d == 128)
        e = p.accumulate ? launch_rt<128, true>(a, g.rt, ctas, stream) : launch_rt<128, false>(a, g.rt, ctas, stream);
    else
        e = p.accumulate ? launch_rt<64, true>(a, g.rt, ctas, stream) : launch_rt<64, false>(a, g.rt, ctas, stream);
    if (e != cudaSuccess) return e;
    if (g.n_splits > 1) {
        const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
        if (p.cache.d == 128)
            fa_kv4_merge_kernel<128><<<grid, 128, 0, stream>>>(a, rows);
        else
            fa_kv4_merge_kernel<64><<<grid, 128, 0, stream>>>(a, rows);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (p.accumulate) {
        int64_t blocks = (cap + 255) / 256;
        if (blocks > 512) blocks = 512;
        if (blocks * p.B * heads > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        fa_kv4_weights_kernel<<<static_cast<unsigned>(blocks * p.B * heads), 256, 0, stream>>>(a, static_cast<int>(blocks));
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int fa_kv4_decode_take_status(cudaStream_t stream) { return kv4_take_status_here(stream); }
