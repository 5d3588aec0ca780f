// Attention over the 4-bit cache with its status word set from the host: the kernels' own source, and calls that
// set the word, launch and read it back (tests/test_kv4_status.py).
#include "fa_kv4_decode.cu"

extern "C" int kv4_status_set(int code)
{
    return static_cast<int>(cudaMemcpyToSymbol(g_kv4_status, &code, sizeof(int)));
}

extern "C" int kv4_status_take() { return fa_kv4_decode_take_status(nullptr); }

extern "C" int kv4_status_decode(void *k, void *v, void *k_scale, void *v_scale, float *weights, int n_pages, int heads,
                                 int log2_page, int d, const void *q, const int32_t *lens, const int32_t *table, void *o,
                                 float *lse, int64_t B, int64_t H, int64_t n_q, int64_t max_pages, float scale,
                                 int accumulate, void *workspace)
{
    Kv4DecodeProblem p = {};
    p.cache = {static_cast<uint8_t *>(k), static_cast<uint8_t *>(v), static_cast<uint8_t *>(k_scale),
               static_cast<uint8_t *>(v_scale), weights, n_pages, heads, log2_page, d};
    p.q = q;
    p.lens = lens;
    p.table = table;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.H = H;
    p.n_q = n_q;
    p.max_pages = max_pages;
    p.scale = scale;
    p.accumulate = accumulate;
    return static_cast<int>(fa_launch_kv4_decode(p, workspace, nullptr));
}
