// C ABI of packed sequences: argument validation and dispatch, in the order of fa_api.cu
// (sizes, then device, pointers, overlaps).  The operations and every argument are documented in include/fa.h.
#include <math.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"

namespace {

constexpr int64_t kMost = (int64_t(1) << 31) - 512;  // rows: a tile past the last one still has a 31-bit number
constexpr int64_t kMostSequences = (int64_t(1) << 31) - 2048;  // which the plan's block takes 1024 at a time, numbered likewise

int check_batch(int64_t B, int64_t T)
{
    return B >= 1 && T >= 1 && B <= kMostSequences && T <= kMost ? FA_OK : FA_ERR_INVALID_ARG;
}

int check_sizes(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d)
{
    if (check_batch(B, T) != FA_OK || H < 1 || Hkv < 1 || d < 1) return FA_ERR_INVALID_ARG;
    if (H > (int64_t(1) << 20) || H % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    // work items (a block of 128 rows of a head) are counted in 31 bits; elements of a tensor and of the workspace in 41
    if (T / 128 + B > kMost / H || T * H > (int64_t(1) << 40) / d) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

int check_softmax(float scale, int causal, int fill)
{
    if ((causal != 0 && causal != 1) || (fill != 0 && fill != 1)) return FA_ERR_INVALID_ARG;
    return scale > 0.f && isfinite(scale) ? FA_OK : FA_ERR_INVALID_ARG;
}

// A packed tensor of `heads` heads: what the kernels take of it, and the bytes from its first element to its last.
struct Rows {
    FaRows r;
    int64_t heads, d;
    uint64_t bytes;
    bool by_token;  // a token's heads lie together (else a head's tokens do)
};

// Strides of an axis of one element mean nothing and become the others' natural ones.  A stride fits a tensor map
// (16-byte multiples below 2^40 bytes); rows of an output do not meet.
int check_rows(const fa_rows *in, int64_t T, int64_t heads, int64_t d, bool output, Rows *out)
{
    if (in == nullptr) return FA_ERR_INVALID_ARG;
    int64_t ts = in->token_stride, hs = in->head_stride;
    if (heads == 1) hs = T == 1 ? d : ts;
    if (T == 1) ts = heads == 1 ? d : hs;
    for (const int64_t s : {ts, hs})
        if (s < d || s % 8 != 0 || s >= int64_t(1) << 38) return FA_ERR_INVALID_ARG;
    if (ts > (int64_t(1) << 42) / T || hs > (int64_t(1) << 42) / heads) return FA_ERR_INVALID_ARG;
    out->by_token = heads == 1 || (T > 1 && ts >= (heads - 1) * hs + d);
    const bool by_head = T == 1 || (heads > 1 && hs >= (T - 1) * ts + d);
    if (output && !out->by_token && !by_head) return FA_ERR_INVALID_ARG;
    out->r = {in->p, ts, hs};
    out->heads = heads;
    out->d = d;
    out->bytes = static_cast<uint64_t>((T - 1) * ts + (heads - 1) * hs + d) * 2u;
    return FA_OK;
}

// Whether two tensors share an element, as far as the layout tells: their ranges meet, and they are not slices of
// the same rows.
bool rows_meet(const Rows &a, const Rows &b)
{
    if (!fa_ranges_overlap(a.r.p, a.bytes, b.r.p, b.bytes)) return false;
    if (!a.by_token || !b.by_token || a.r.token_stride != b.r.token_stride) return true;
    const int64_t ts = a.r.token_stride;
    const int64_t wa = (a.heads - 1) * a.r.head_stride + a.d, wb = (b.heads - 1) * b.r.head_stride + b.d;
    int64_t at = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.r.p)) - static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.r.p))) / 2 % ts;
    if (at < 0) at += ts;
    return !(at >= wa && at + wb <= ts);
}
bool meets(const Rows &a, const void *p, uint64_t bytes) { return fa_ranges_overlap(a.r.p, a.bytes, p, bytes); }

}  // namespace

extern "C" int64_t fa_packed_plan_bytes(int64_t B, int64_t T)
{
    return check_batch(B, T) == FA_OK ? fa_packed_plan_size(B, T) : -1;
}

extern "C" int fa_packed_plan(const int32_t *cu_seqlens, int64_t B, int64_t T, int causal, void *plan, int64_t plan_bytes,
                              void *stream)
{
    int st = check_batch(B, T);
    if (st != FA_OK) return st;
    const int64_t need = fa_packed_plan_size(B, T);
    if ((causal != 0 && causal != 1) || plan_bytes < need) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK || (st = fa_check_device_pointer(cu_seqlens, dev, 4)) != FA_OK ||
        (st = fa_check_device_pointer(plan, dev, 16)) != FA_OK)
        return st;
    if (fa_ranges_overlap(plan, static_cast<uint64_t>(need), cu_seqlens, static_cast<uint64_t>(B + 1) * 4u)) return FA_ERR_INVALID_ARG;
    return fa_launch_packed_plan(cu_seqlens, B, T, causal, plan, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

extern "C" int fa_fwd_packed(const fa_rows *q, const fa_rows *k, const fa_rows *v, const fa_rows *o, float *lse,
                             const void *plan, int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, float scale,
                             int causal, int fill, void *stream)
{
    int st = check_sizes(B, T, H, Hkv, d);
    if (st != FA_OK || (st = check_softmax(scale, causal, fill)) != FA_OK) return st;
    Rows rq, rk, rv, ro;
    if ((st = check_rows(q, T, H, d, false, &rq)) != FA_OK || (st = check_rows(k, T, Hkv, d, false, &rk)) != FA_OK ||
        (st = check_rows(v, T, Hkv, d, false, &rv)) != FA_OK || (st = check_rows(o, T, H, d, true, &ro)) != FA_OK)
        return st;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(q->p), static_cast<const void *>(k->p), static_cast<const void *>(v->p),
                          static_cast<const void *>(o->p), plan})
        if ((st = fa_check_device_pointer(p, dev, 16)) != FA_OK) return st;
    if ((st = fa_check_device_pointer(lse, dev, 4)) != FA_OK) return st;
    const uint64_t lbytes = static_cast<uint64_t>(H * T) * 4u, pbytes = static_cast<uint64_t>(fa_packed_plan_size(B, T));
    for (const Rows *in : {&rq, &rk, &rv})
        if (rows_meet(ro, *in) || meets(*in, lse, lbytes)) return FA_ERR_INVALID_ARG;
    if (meets(ro, lse, lbytes) || meets(ro, plan, pbytes) || fa_ranges_overlap(lse, lbytes, plan, pbytes)) return FA_ERR_INVALID_ARG;
    FaPackedProblem p = {};
    p.q = rq.r;
    p.k = rk.r;
    p.v = rv.r;
    p.o = ro.r;
    p.lse = lse;
    p.plan = const_cast<void *>(plan);
    p.B = B;
    p.T = T;
    p.H = H;
    p.Hkv = Hkv;
    p.d = static_cast<int>(d);
    p.scale = scale;
    p.causal = causal;
    p.fill = fill;
    p.sm_count = sm_count;
    return fa_launch_packed_fwd(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

extern "C" int64_t fa_bwd_packed_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d)
{
    return check_sizes(B, T, H, Hkv, d) == FA_OK ? fa_packed_bwd_workspace_size(B, T, H, Hkv, d) : -1;
}

extern "C" int fa_bwd_packed(const fa_rows *q, const fa_rows *k, const fa_rows *v, const fa_rows *o, const float *lse,
                             const fa_rows *dout, const fa_rows *dq, const fa_rows *dk, const fa_rows *dv, const void *plan,
                             int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, float scale, int causal, int fill,
                             void *workspace, int64_t workspace_bytes, void *stream)
{
    int st = check_sizes(B, T, H, Hkv, d);
    if (st != FA_OK || (st = check_softmax(scale, causal, fill)) != FA_OK) return st;
    const int64_t need = fa_packed_bwd_workspace_size(B, T, H, Hkv, d);
    if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
    const fa_rows *tensors[8] = {q, k, v, o, dout, dq, dk, dv};
    const int64_t heads[8] = {H, Hkv, Hkv, H, H, H, Hkv, Hkv};
    Rows r[8];
    for (int i = 0; i < 8; ++i)
        if ((st = check_rows(tensors[i], T, heads[i], d, i >= 5, &r[i])) != FA_OK) return st;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK) return st;
    for (const fa_rows *t : tensors)
        if ((st = fa_check_device_pointer(t->p, dev, 16)) != FA_OK) return st;
    for (const void *p : {plan, static_cast<const void *>(workspace)})
        if ((st = fa_check_device_pointer(p, dev, 16)) != FA_OK) return st;
    if ((st = fa_check_device_pointer(lse, dev, 4)) != FA_OK) return st;
    const uint64_t lbytes = static_cast<uint64_t>(H * T) * 4u, pbytes = static_cast<uint64_t>(fa_packed_plan_size(B, T)),
                   wbytes = static_cast<uint64_t>(need);
    for (int i = 0; i < 8; ++i) {
        if (meets(r[i], workspace, wbytes)) return FA_ERR_INVALID_ARG;
        if (i < 5) continue;
        if (meets(r[i], lse, lbytes) || meets(r[i], plan, pbytes)) return FA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (rows_meet(r[i], r[j])) return FA_ERR_INVALID_ARG;
    }
    if (fa_ranges_overlap(workspace, wbytes, lse, lbytes) || fa_ranges_overlap(workspace, wbytes, plan, pbytes)) return FA_ERR_INVALID_ARG;
    FaPackedProblem p = {};
    p.q = r[0].r;
    p.k = r[1].r;
    p.v = r[2].r;
    p.o = r[3].r;
    p.dout = r[4].r;
    p.dq = r[5].r;
    p.dk = r[6].r;
    p.dv = r[7].r;
    p.lse = const_cast<float *>(lse);
    p.plan = const_cast<void *>(plan);
    p.B = B;
    p.T = T;
    p.H = H;
    p.Hkv = Hkv;
    p.d = static_cast<int>(d);
    p.scale = scale;
    p.causal = causal;
    p.fill = fill;
    p.sm_count = sm_count;
    return fa_launch_packed_bwd(p, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}
