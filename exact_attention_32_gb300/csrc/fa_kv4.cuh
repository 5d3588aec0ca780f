// The 4-bit KV cache's format and page addressing, shared by the kernels that
// write it, read it and attend to it (fa_kv4_cache.cu, fa_kv4_decode.cu).
//
// A row is one token of one key head: d E2M1 codes, two a byte, the even channel
// in the low nibble.  K has one scale per 32 channels, V one per row.  A scale is
// the sign-less top byte of a half: five exponent bits and three mantissa bits,
// half(byte << 7), so 0xE2 = 10240 is the largest scale whose multiples (up to
// 6 x) stay finite in a half, and 0xFF is a NaN: a block that held a NaN or an
// infinity reads back as NaN instead of as some finite value.
// code * scale has at most 6 significant bits and is a multiple of 2^-18, so it
// is exact in a half and in bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"

namespace {

// Sticky status of this translation unit's kernels: FA_ERR_BAD_PAGE once a
// kernel met a page index or a length outside its cache (it left that part out),
// FA_ERR_TIMEOUT once a bounded wait gave up (which a bad page does not overwrite).
__device__ int g_kv4_status;

__device__ __forceinline__ void kv4_report() { atomicCAS(&g_kv4_status, 0, FA_ERR_BAD_PAGE); }

int kv4_take_status_here(cudaStream_t stream)
{
    int h = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&h, g_kv4_status, sizeof(int), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_kv4_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_LAUNCH;
    }
    return h;
}

// Length of sequence b, held inside [0, capacity]; a length outside is reported.
__device__ __forceinline__ int kv4_length(const int32_t *lens, int64_t b, int64_t capacity)
{
    const int n = lens[b];
    if (n >= 0 && n <= capacity) return n;
    kv4_report();
    return n < 0 ? 0 : static_cast<int>(capacity);
}

// Page that holds token `pos` of sequence b, or -1 (reported) if the table's entry is no page of the pool.
__device__ __forceinline__ int kv4_page(const Kv4Cache &c, const int32_t *table, int64_t b, int64_t max_pages, int pos)
{
    const int page = table[b * max_pages + (pos >> c.log2_page)];
    if (page >= 0 && page < c.n_pages) return page;
    kv4_report();
    return -1;
}

// The same without the report and without a branch, for loops that keep several rows under way: page 0 where the
// entry is no page, and whether it is one.
__device__ __forceinline__ int kv4_page_quiet(const Kv4Cache &c, const int32_t *table, int64_t b, int64_t max_pages,
                                              int pos, bool *valid)
{
    const int page = table[b * max_pages + (pos >> c.log2_page)];
    *valid = static_cast<unsigned>(page) < static_cast<unsigned>(c.n_pages);
    return *valid ? page : 0;
}

// Row of the pool that holds token `pos` of head h in `page`: the index into
// k, v (rows of d/2 bytes), k_scale (d/32 bytes), v_scale (one byte) and weights.
__device__ __forceinline__ int64_t kv4_row(const Kv4Cache &c, int page, int h, int pos)
{
    return ((static_cast<int64_t>(page) * c.heads + h) << c.log2_page) + (pos & ((1 << c.log2_page) - 1));
}

// The scale that a byte stands for.
__device__ __forceinline__ __half kv4_scale_half(uint32_t byte)
{
    return __ushort_as_half(static_cast<unsigned short>(byte << 7));
}
__device__ __forceinline__ float kv4_scale(uint32_t byte) { return __half2float(kv4_scale_half(byte)); }

// Four bytes of codes as eight halves: r[i] = channels (2i, 2i + 1).
__device__ __forceinline__ void kv4_decode8(uint32_t x, uint32_t (&r)[4])
{
    asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(x));
}

// Eight halves as four bytes of codes: to nearest, ties to the even code, at most 6 in magnitude.
__device__ __forceinline__ uint32_t kv4_encode8(const uint32_t (&y)[4])
{
    uint32_t r;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f16x2 a, %1;\ncvt.rn.satfinite.e2m1x2.f16x2 b, %2;\n"
        "cvt.rn.satfinite.e2m1x2.f16x2 c, %3;\ncvt.rn.satfinite.e2m1x2.f16x2 d, %4;\n"
        "mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]));
    return r;
}

// A kernel behind another whose results it needs: launched before that one has ended, so that its launch overlaps it, it
// waits for the end itself.
__device__ __forceinline__ void kv4_wait_for_the_one_before() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t kv4_launch_behind(void (*kern)(P...), dim3 grid, int threads, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace
