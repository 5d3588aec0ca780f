// Attention of the newest tokens over a 4-bit KV cache (fa_fwd_kv4).
//
// For each (sequence, key head) the R = H / Hkv * n_q query rows that share its
// keys go together (up to 32 at a time), so a key's row is read once for all of them:
//     S = scale q K^T,  O = softmax(S) V,  LSE = ln sum exp S
// in one pass over the keys with a running maximum m and sum l per row.
//
// What bounds it is the bytes of the cache (133 a key and head at d = 128), at
// which an SM has 2.8 instruction slots for every cached value: too few to decode them
// in registers for warp-level products (that form of this kernel spent 2.9, and
// reached 62 % of the copy bandwidth).  So the codes are never decoded: E2M1 is an
// operand type of tcgen05.mma (kind::f8f6f4), and the TMA spreads each 8 bytes of codes
// over the 16-byte slot that the tensor core reads them from (16U4_ALIGN16B).
//   S^T = K Q^T      A = K as stored (128 rows, K-major), B = Q in E4M3.  One product per 32
//                    channels, into columns of its own: K's scale differs per 32 channels
//                    and is applied to the sums, one thread per key.
//   O^T += V^T P^T   A = V as stored, MN-major; B = P times V's scale, in E5M2.
// What is not 4-bit goes in as several parts, each 8 to 32 times what the ones before leave, in columns next to one
// another (a product's time is A's, so they cost nothing).  q (bf16, eight bits, scaled by a power of
// two to a maximum in [128, 256)) is two parts of E4M3, four bits each: exact down to 2^-13 of the row's maximum, and
// to 2^-21 of it below.  P s (s: V's scale) spans far more, since a key of a thousandth of another's weight counts where there
// are thousands of them, or where the other's V is small: it is rounded to a half, under a power of two of its row
// that keeps the largest p s so far between 2^11 and 2^15, and goes in as three parts of E5M2 (a half's exponents, three bits
// each).  So it is off by at most 2^-11 of itself down to 2^-24 of that largest term, and by 2^-34 of the term below (two
// parts of E4M3 under one factor for all rows lost the keys behind a heavy one: O of 16384 keys was off by half).
// l is summed in fp32.  The products are exact and added in fp32.
//
// Work: a tile is 128 rows of 128 values: 128 keys at d = 128, 256 at d = 64 (keys 2i and
// 2i + 1 side by side, as they lie in the page).  All tiles of all (sequence, head, row chunk) items in a row
// are cut into equal shares, one a CTA, so lengths may differ as they like; a CTA
// takes its share as segments of items.  A segment that is a whole item is finished in
// place; the others leave (m, l, O) in the workspace, which a second kernel merges
// (O = sum 2^(m_s - m) O_s / sum 2^(m_s - m) l_s).
// Roles: a softmax warpgroup per 8 rows (1, 2 or 4), one thread a TMEM lane; three warps that load (K, V, the scales), a lane
// a page (or the part of a page in the tile); a warp that issues the products.  A copy takes its warp 77 cycles to issue,
// so one warp for all copies was too slow where pages are small (32 sequences of 8192 in pages of 16: 86 us, two warps 70,
// three 66; in pages of 1024 60).  A softmax takes about 2000 cycles a tile, waits between
// its steps for the most part, so an SM needs several at work to keep up with the 720 cycles that a tile's bytes
// take: three CTAs of 8 rows, two of 16, one of 32.  K and V have stages of their own, K's free as soon as S is there.
// What a softmax needs to begin, K and the scales, comes ahead of V, which it needs at its end: with the scales behind V's
// barrier 64 sequences of 16384 (8 key heads, 8 rows each, 1.12 GB) took 208 us, so 190, 5.9 TB/s (the copies alone 6.9).
// Copies of 8 bytes a lane by the load warps (cp.async) in the TMA's place took 3500 cycles
// to issue a tile, two and a half times what all of the tile may take; TMA copies from an elected lane, box by box, more
// than those of several lanes in one instruction (pages of 16: 102 us against 87).  Softmax code for 4 rows instead of 8, where
// no more are live, gained 1 to 2 % only: its time is latency.
#include <algorithm>
#include <cuda.h>
#include <float.h>
#include <math.h>

#include <mutex>
#include <type_traits>

#include "fa_kv4.cuh"
#include "sm100_ptx.cuh"

using namespace sm100;

namespace {

constexpr int kMinShare = 4;   // units: a shorter share costs more in merging than it saves
constexpr int kItemUnits = 3;  // what starting and ending an item costs, in tiles (4 to 6 us beside 1.4 us a tile)
constexpr int kWholeTiles = 4;  // tables of so few tiles: items go to CTAs whole, and nothing is merged
constexpr int kSms = 152;
// A row's reference is set this far (log2) above the largest score when one passes it: with the maximum itself some of a
// tile's 8 or 16 rows grow in nearly every one of the first dozens of tiles, at 1300 cycles each time.
constexpr float kHeadroom = 3.f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint64_t kWaitLimitNs = 1000000000ull;   // 1 s per pipeline wait
constexpr uint64_t kCleanupLimitNs = 20000000ull;  // 20 ms while winding down

__device__ __forceinline__ void kv4_timeout() { atomicExch(&g_kv4_status, FA_ERR_TIMEOUT); }

// An item in several shares: its rows, its parts (0: this CTA holds no first part) and the first part's slot; the
// others are slot 0 of the CTAs that follow.
struct Split {
    int64_t row;
    int n_rows, parts, slot, pad;
};

struct DecodeArgs {
    Kv4Cache c;
    const __nv_bfloat16 *q;
    const int32_t *lens, *table;
    const uint64_t *tree;  // [B][n_q] which drafts a row admits, and how many a sequence has (or null); TREE only
    const int32_t *n_new;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o;     // [CTA][2][RP][D], unnormalised; slot 0: the segment that starts its share, 1: that ends it
    float2 *part_ml;   // [CTA][2][RP]: running maximum (log2), sum
    struct Split *split;  // [CTA]: the item whose first part is this CTA's, for the merge
    float *scores;     // [B][heads][max_tokens][Rs] log2 scores, or null
    float2 *row_ml;    // [rows]: maximum (log2), 1 / sum; with scores
    int64_t max_pages;
    int B, R, Rs, n_q, n_rc, whole;
    int item_cost;  // what starting and ending an item costs, in tiles
    float scale_log2;
};

template <int D, int RT>
struct DecCfg {
    static constexpr int RP = 8 * RT;          // rows a CTA takes
    static constexpr int kLoadWarp = 4 * RT, kMmaWarp = kLoadWarp + 3, kWarps = kLoadWarp + 4, kThreads = 32 * kWarps;
    static constexpr int N = 16 * RT;          // columns of S: per 8 rows, 8 high parts and 8 rests of q
    static constexpr int KPT = 128 / D;        // keys a thread (and a 128-byte row) holds
    static constexpr int U = KPT * RT;         // 8 rows of every KPT-th key: P and O have 24 columns of each, parts 1 and 2 of
    static constexpr int kPart3 = 16 * U;      // all of them first, then the parts 3
    static constexpr int NP = (24 * U + 15) / 16 * 16;  // (a product's N is a multiple of 16: of a last odd 8, 8 more that hold anything)
    static constexpr int TK = 128 * KPT;       // keys a tile
    static constexpr int NG = TK / 16;         // runs of 16 tokens, each in one page
    static constexpr int kHalf = 16384;        // K or V of a tile
    static constexpr int kPerSm = RT == 1 ? 3 : RT == 2 ? 2 : 1;   // CTAs an SM
    static constexpr int kStages = RT == 1 ? 2 : RT == 2 ? 3 : 5;  // of K
    static constexpr int kStagesV = RT == 2 && D == 64 ? 2 : kStages;  // of V
    // What fits kPerSm CTAs an SM.  d = 64, 8 rows, with two buffers: two CTAs an SM, 64 sequences of 16384 194 us in place of 133;
    // d = 128, 16 rows, with two stages of V and two buffers: 32 of 8192 56 us in place of 55.
    static constexpr int kPBufs = RT == 1 || (RT == 2 && D == 128) ? 1 : 2;
    static constexpr int kV = kStages * kHalf;
    static constexpr int kQ = kV + kStagesV * kHalf;
    static constexpr int kP = kQ + N * 128;
    static constexpr int kPBytes = 128 * NP;
    static constexpr int kScale = kP + kPBufs * kPBytes;         // a tile's K scales 512, V scales 256, page flags 64
    static constexpr int kScaleBytes = 512 + 256 + 64;
    static constexpr int kScales = kStages + 1;                  // of these
    static constexpr int kFloat = kScale + kScales * kScaleBytes;
    static constexpr int kGroupFloats = 6 * 8 + 8;  // mult, m, alpha, top, f, o_alpha [8]; fail
    static constexpr int kWalk = kFloat + RT * kGroupFloats * 4;  // the share's start, the scan's sums
    static constexpr int kBar = kWalk + 64 + 8 * kWarps;
    static constexpr int kNumBars = 2 * (kStages + kStagesV + kScales) + 8;
    static constexpr int kSmemBytes = kBar + kNumBars * 8 + 16;
    static constexpr int kSCols = 4 * N, kOCols = NP;
    static constexpr int kTmemCols = kSCols + kOCols <= 128 ? 128 : kSCols + kOCols <= 256 ? 256 : 512;
    // The grid's equal shares are for kPerSm CTAs on every SM at once; a second round for those that do not fit would double its
    // time.  (228 KB of shared memory an SM, 1 KB of it for each CTA, and 512 columns of tensor memory.)
    static_assert(kPerSm * (kSmemBytes + 1024) <= 228 * 1024 && kPerSm * kTmemCols <= 512, "kPerSm CTAs fit an SM");
};
// P_READY is a barrier a buffer: a group may have tile n + 1's P written while another still works on tile n's, and its
// arrival must not count for tile n.  (It reaches tile n + 2 only behind the product of tile n.)
enum { D_S_FULL = 0, D_S_FREE, D_P_READY, D_P_READY1, D_PV_DONE, D_PV_DONE1, D_Q_READY, D_DONE, D_STAGES };
// then K_FULL, K_FREE, V_FULL, V_FREE of the stages and X_FULL, X_FREE of the scales

__host__ __device__ inline int tile_keys(int d) { return 128 * (128 / d); }

// Tiles of one (sequence, head, row chunk): at least one, so that an empty sequence's rows are written too.
__device__ __forceinline__ int tiles_of(int len, int tk) { return len <= tk ? 1 : (len + tk - 1) / tk; }
// Units of it: its tiles behind item_cost for its start and end; one where items go whole.
__device__ __forceinline__ int item_units(const DecodeArgs &a, int n_t) { return a.whole ? 1 : n_t + a.item_cost; }

// A CTA's way through its share: segments [t0, t1) of the n_t tiles of item `it` (head * n_rc + chunk) of sequence b.
// The segment that a share begins or ends with may lie in an item's first units and hold no tile.
struct Walk {
    int64_t left;  // units of the share still to come
    int b, it, at, t0, t1, n_t, len;  // at: unit of the item where the segment begins
};

template <int TK>
__device__ __forceinline__ void walk_open(Walk &w, const DecodeArgs &a)
{
    w.len = kv4_length(a.lens, w.b, a.max_pages << a.c.log2_page);
    w.n_t = tiles_of(w.len, TK);
}
// The segment from unit w.at on, as far as the share or the item goes.
__device__ __forceinline__ void walk_clip(Walk &w, const DecodeArgs &a)
{
    if (a.whole) {
        w.t0 = 0;
        w.t1 = w.n_t;
        return;
    }
    const int end = static_cast<int>(min(static_cast<int64_t>(w.n_t + a.item_cost), w.at + w.left));
    w.t0 = max(0, w.at - a.item_cost);
    w.t1 = max(0, end - a.item_cost);
}

template <int TK>
__device__ __forceinline__ void walk_next(Walk &w, const DecodeArgs &a)
{
    w.left -= item_units(a, w.n_t) - w.at;
    w.at = 0;
    if (w.left <= 0) return;
    if (++w.it == a.c.heads * a.n_rc) {
        w.it = 0;
        ++w.b;
        walk_open<TK>(w, a);
    }
    walk_clip(w, a);
}

// The share of this CTA (returned: its units), by all of its THREADS threads: units before each sequence by a scan over the
// lengths, a thread each at a time; `start`, where it begins, is there behind the next barrier.  `scan` holds a value a warp.
template <int TK, int THREADS>
__device__ __forceinline__ int64_t walk_begin(const DecodeArgs &a, Walk &start, int64_t *scan)
{
    constexpr int kWarps = THREADS / 32;
    static_assert(sizeof(Walk) <= 64, "fits before the scan");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t cap = a.max_pages << a.c.log2_page;
    const int items = a.c.heads * a.n_rc;
    auto units_of = [&](int b) -> int64_t {
        return b < a.B ? static_cast<int64_t>(item_units(a, tiles_of(kv4_length(a.lens, b, cap), TK))) * items : 0;
    };
    int64_t total = 0;
    const int64_t units0 = units_of(tid);  // (most batches have no more sequences than this)
    {
        int64_t n = units0;
        for (int b = tid + THREADS; b < a.B; b += THREADS) n += units_of(b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == 0) scan[warp] = n;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) total += scan[i];
    }
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    if (!a.whole && share < kMinShare) share = kMinShare;
    const int64_t u0 = blockIdx.x * share;
    if (tid == 0) start.left = 0;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B && base <= u0; b0 += THREADS) {
        const int b = b0 + tid;
        const int64_t mine = b0 == 0 ? units0 : units_of(b);
        int64_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        int64_t all = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) x += scan[i];
            all += scan[i];
        }
        const int64_t before = base + x - mine;
        if (b < a.B && u0 >= before && u0 < before + mine) {
            Walk w;
            w.b = b;
            w.left = min(share, total - u0);
            walk_open<TK>(w, a);
            const int units = item_units(a, w.n_t);
            w.it = static_cast<int>((u0 - before) / units);
            w.at = static_cast<int>((u0 - before) % units);
            walk_clip(w, a);
            start = w;
        }
        base += all;
    }
    return share;
}

// Two fp32 -> two E4M3 bytes (`lo` in the low one), and back, exactly.
__device__ __forceinline__ uint32_t e4m3x2(float2 v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;\n" : "=h"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Two halves of at most 2^15 as E5M2 three times: y = a + b / 8 + c / 256.  An E5M2 value is the top byte of a half, with three of
// its eleven bits; what rounding leaves fits three bits twice more, so this is exact from 2^-13 on (below, off by at most 2^-24: the
// smallest halves).  a and b are rounded to nearest on the bits, in the upper byte of each half (conversions back and forth took 2 % of
// the kernel at 32 rows); a NaN, 0x7FFF here, comes out of c.
__device__ __forceinline__ uint32_t round3(__half2 y) { return (*reinterpret_cast<const uint32_t *>(&y) + 0x00800080u) & 0xFF00FF00u; }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ void e5m2_parts(__half2 y, uint32_t &a, uint32_t &b, uint32_t &c)
{
    a = round3(y);
    const __half2 y1 = __hmul2(__hsub2(y, half2_of(a)), __float2half2_rn(8.f));
    b = round3(y1);
    const __half2 y2 = __hmul2(__hsub2(y1, half2_of(b)), __float2half2_rn(32.f));
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&y2)));
    c = r;
}
// 1 / x of a power of two
__device__ __forceinline__ float inverse_pow2(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

// Barrier of a softmax warpgroup; with an OR over its threads.
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;\n" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_or(int id, bool x)
{
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, %2, 128, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x)), "r"(id)
        : "memory");
    return r != 0;
}

// Maximum of finite floats over the warp.
__device__ __forceinline__ float warp_max(float x)
{
    int i = __float_as_int(x);
    i ^= (i >> 31) & 0x7FFFFFFF;
    i = __reduce_max_sync(0xffffffffu, i);
    i ^= (i >> 31) & 0x7FFFFFFF;
    return __int_as_float(i);
}

// Waits of a whole warp for several barriers (bounded): asked one after the other, answered by one vote; a wait each costs
// 170 cycles where nothing is left to wait for.
__device__ __forceinline__ bool wait_both(uint32_t bar0, uint32_t phase0, uint32_t bar1, uint32_t phase1)
{
    const bool a = mbar_try_wait(bar0, phase0), b = mbar_try_wait(bar1, phase1);
    if (__all_sync(0xffffffffu, a && b)) return true;
    return mbar_wait_warp(bar0, phase0, kWaitLimitNs) && mbar_wait_warp(bar1, phase1, kWaitLimitNs);
}
__device__ __forceinline__ uint32_t lo32(uint64_t x) { return static_cast<uint32_t>(x); }
__device__ __forceinline__ uint32_t hi32(uint64_t x) { return static_cast<uint32_t>(x >> 32); }

// TREE: the newest tokens are drafts, and which of them a row admits is a bit mask; the tokens before them everyone admits.
template <int D, int RT, bool SCORES, bool TREE>
__global__ void __launch_bounds__(DecCfg<D, RT>::kThreads, DecCfg<D, RT>::kPerSm)
fa_kv4_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a)
{
    using C = DecCfg<D, RT>;
    constexpr int RP = C::RP, N = C::N, KPT = C::KPT, TK = C::TK, ST = C::kStages, SV = C::kStagesV;
    constexpr int kLoadWarp = C::kLoadWarp, kMmaWarp = C::kMmaWarp, kDecThreads = C::kThreads;
    constexpr int K_FULL = D_STAGES, K_FREE = K_FULL + ST, V_FULL = K_FREE + ST, V_FREE = V_FULL + SV,
                  XS = C::kScales, X_FULL = V_FREE + SV, X_FREE = X_FULL + XS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((sb & 1023u) != 0) {  // the swizzled tiles need a 1024-byte-aligned base
        if (tid == 0) kv4_timeout();
        return;
    }
    const uint32_t bar0 = sb + C::kBar;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBar + C::kNumBars * 8);
    const int64_t cap = a.max_pages << a.c.log2_page;

    if (tid == 0) {
        for (int s = 0; s < 2 * (ST + SV + XS); ++s) mbar_init(BAR(D_STAGES + s), 1);
        mbar_init(BAR(D_S_FULL), 1);
        mbar_init(BAR(D_S_FREE), 4 * RT);
        mbar_init(BAR(D_P_READY), 4 * RT);
        mbar_init(BAR(D_P_READY1), 4 * RT);
        mbar_init(BAR(D_PV_DONE), 1);
        mbar_init(BAR(D_PV_DONE1), 1);
        mbar_init(BAR(D_Q_READY), 4 * RT);
        mbar_init(BAR(D_DONE), 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }


    Walk &start = *reinterpret_cast<Walk *>(smem + C::kWalk);
    const int64_t share = walk_begin<TK, kDecThreads>(a, start, reinterpret_cast<int64_t *>(smem + C::kWalk + 64));
    if (tid == 0) a.split[blockIdx.x].parts = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tO = tmem + C::kSCols;
    // P's buffer of tile n, and the barriers and phase of its writing and its product
    auto pbuf = [&](int n) { return C::kPBufs == 2 ? n & 1 : 0; };
    auto pv_bar = [&](int n) { return BAR(D_PV_DONE + pbuf(n)); };
    auto pv_phase = [&](int n) -> uint32_t { return (C::kPBufs == 2 ? n >> 1 : n) & 1; };
    const bool run = *reinterpret_cast<volatile int *>(&g_kv4_status) != FA_ERR_TIMEOUT;
    Walk w = start;
    if (!run) w.left = 0;

    if (warp >= kLoadWarp && warp < kMmaWarp) {
        // -------------------------------------------------------------------- loads: K, V, scales
        const int role = warp - kLoadWarp, depth = role == 0 ? ST : role == 1 ? SV : XS;
        const CUtensorMap *map = role == 0 ? &tm_k : &tm_v;
        if (lane == 0 && role < 2) prefetch_tmap(map);
        const int bt = min(1 << a.c.log2_page, TK), n_boxes = TK / bt;  // tokens a box: a page, or the tile's part of one
        const int in_page = (1 << a.c.log2_page) - 1;
        const uint32_t dst = sb + (role == 0 ? 0 : C::kV) + lane * bt / KPT * 128;
        const int full = role == 0 ? K_FULL : role == 1 ? V_FULL : X_FULL, free = role == 0 ? K_FREE : role == 1 ? V_FREE : X_FREE;
        // the table's entry for this lane's box, asked for a tile ahead
        auto entry = [&](int t) -> int {
            const int key = t * TK + lane * bt;
            return lane < n_boxes && key < w.len ? a.table[w.b * a.max_pages + (key >> a.c.log2_page)] : 0;
        };
        int n = 0;
        bool ok = true;
        while (w.left > 0 && w.t0 == w.t1) walk_next<TK>(w, a);  // (a segment without a tile falls through every role)
        int t = w.t0, next = w.left > 0 ? entry(t) : 0;
        for (; w.left > 0; ++n) {
            const int page = next, h = w.it / a.n_rc, slot = (t * TK & in_page) / KPT;  // (a tile begins a page, or lies in one)
            bool there = lane < n_boxes && t * TK + lane * bt < w.len;
            if (there && static_cast<unsigned>(page) >= static_cast<unsigned>(a.c.n_pages)) {
                kv4_report();
                there = false;
            }
            const uint32_t boxes = __ballot_sync(0xffffffffu, there);
            const uint32_t tokens = __popc(boxes) * bt;
            if (++t == w.t1) {
                do walk_next<TK>(w, a);
                while (w.left > 0 && w.t0 == w.t1);
                t = w.t0;
            }
            if (w.left > 0) next = entry(t);
            const int st = n % depth;
            if (n >= depth && !(ok = mbar_wait_warp(BAR(free + st), (n / depth - 1) & 1, kWaitLimitNs))) break;
            uint8_t *scale = smem + C::kScale + st * C::kScaleBytes;
            if (role == 2 && lane < C::NG) reinterpret_cast<int *>(scale + 768)[lane] = (boxes >> (lane * 16 / bt)) & 1u;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(BAR(full + st), tokens * (role == 2 ? D / 32 + 1 : D / 2));
            __syncwarp();
            // (rows of a box that is left out keep stale codes, as good as any: their weight is 0)
            if (there && role < 2) tma_load_4d(dst + st * C::kHalf, map, BAR(full + st), 0, slot, h, page);
            if (there && role == 2) {
                const int64_t row = kv4_row(a.c, page, h, slot * KPT);
                bulk_load(smem_u32(scale) + lane * bt * (D / 32), a.c.k_scale + row * (D / 32), bt * (D / 32), BAR(full + st));
                bulk_load(smem_u32(scale) + 512 + lane * bt, a.c.v_scale + row, bt, BAR(full + st));
            }
        }
        if (!ok && lane == 0) kv4_timeout();
        // no copy in flight when the CTA ends
        const uint64_t lim = ok ? kWaitLimitNs : kCleanupLimitNs;
        for (int i = n > depth ? n - depth : 0; i < n; ++i) mbar_wait(BAR(full + i % depth), (i / depth) & 1, lim);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------------- products
        constexpr uint32_t idS = idesc_e2m1_f8_f32(128, N, false, false, kE4M3);
        constexpr uint32_t idO = idesc_e2m1_f8_f32(128, C::NP, true, true, kE5M2);
        const uint64_t dA = smem_desc_sw128(sb, 16, 1024);  // K tiles, and V tiles read the other way
        const uint64_t dQ = smem_desc_sw128(sb + C::kQ, 16, 1024);
        const uint64_t dP = smem_desc_plain(sb + C::kP, 128, 2048);
        bool ok = true;
        int n = 0, seg = 0;
        auto pv = [&](int m, bool first) -> bool {  // O^T (+)= V^T P^T of tile m
            if (!wait_both(BAR(V_FULL + m % SV), (m / SV) & 1, BAR(D_P_READY + pbuf(m)), pv_phase(m))) return false;
            tc_fence_after();
            const uint32_t v = lo32(dA) + ((C::kV + m % SV * C::kHalf) >> 4);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss_f8_lohi(tO, v + kk * 256, hi32(dA), lo32(dP) + pbuf(m) * (C::kPBytes >> 4) + kk * 32, hi32(dP), idO,
                                   first && kk == 0 ? 0u : 1u);
                mma_commit(pv_bar(m));
                mma_commit(BAR(V_FREE + m % SV));
            }
            __syncwarp();
            return true;
        };
        for (; w.left > 0 && ok; walk_next<TK>(w, a)) {
            if (w.t0 == w.t1) continue;
            if (!(ok = mbar_wait_warp(BAR(D_Q_READY), seg++ & 1, kWaitLimitNs))) break;
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const int st = n % ST;
                if (!(ok = n == 0 ? mbar_wait_warp(BAR(K_FULL), 0, kWaitLimitNs)
                                  : wait_both(BAR(K_FULL + st), (n / ST) & 1, BAR(D_S_FREE), (n - 1) & 1)))
                    break;
                tc_fence_after();
                const uint32_t k = lo32(dA) + st * (C::kHalf >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_ss_f8_lohi(tS + i * N, k + i * 2, hi32(dA), lo32(dQ) + (D == 128 ? i : i & 1) * 2, hi32(dQ), idS, 0u);
                    mma_commit(BAR(D_S_FULL));
                    mma_commit(BAR(K_FREE + st));
                    if (n > 0) mbar_arrive(BAR(X_FREE + (n - 1) % XS));  // (the scales were read before the scores)
                }
                __syncwarp();
                if (t > w.t0 && !(ok = pv(n - 1, t - 1 == w.t0))) break;
            }
            if (!ok || !(ok = pv(n - 1, w.t1 - 1 == w.t0))) break;
        }
        if (!ok && lane == 0) kv4_timeout();
        if (elect_one()) mma_commit(BAR(D_DONE));
        __syncwarp();
        mbar_wait_warp(BAR(D_DONE), 0, ok ? kWaitLimitNs : kCleanupLimitNs);
    } else {
        // ------------------------------------------------- softmax: warpgroup g has rows 8 g .. 8 g + 7
        const int g = warp >> 2, wl = warp & 3, tl = tid & 127;  // tl: TMEM lane
        const uint32_t loff = static_cast<uint32_t>(wl * 32) << 16;
        float *sm_mult = reinterpret_cast<float *>(smem + C::kFloat) + g * C::kGroupFloats;
        float *sm_m = sm_mult + 8, *sm_alpha = sm_m + 8, *sm_top = sm_alpha + 8, *sm_f = sm_top + 8, *sm_oalpha = sm_f + 8;
        volatile float *sm_fail = sm_oalpha + 8;  // a warp's wait gave up: all of the group leave at the next barrier
        // reductions over the group's warps, in its own part of P's first buffer where the products have read all of P
        float *sm_red = reinterpret_cast<float *>(smem + C::kP + ((KPT - 1) * RT + g) * 2048);
        auto unit = [&](int k) { return k * RT + g; };  // its columns of P and O
        auto sync = [&]() { group_sync(1 + g); };
        int n = 0;
        bool ok = true;
        if (tl == 0) *sm_fail = 0.f;
        for (; w.left > 0 && ok; walk_next<TK>(w, a)) {
            if (w.t0 == w.t1) continue;
            const int h = w.it / a.n_rc, rc = w.it - h * a.n_rc;
            const int64_t bh = static_cast<int64_t>(w.b) * a.c.heads + h;
            const int row0 = rc * RP + g * 8, n_rows = min(8, a.R - row0);  // (0 or less: this group has padding only)
            // newest tokens that not every row admits: all n_q, whatever the length is, or the sequence's drafts
            int newest = a.n_q;
            uint2 seen = make_uint2(0, 0);  // the drafts that row row0 + lane % 8 admits
            if constexpr (TREE) {
                newest = min(newest, w.len);
                if (a.n_new != nullptr) newest = min(max(a.n_new[w.b], 0), newest);
                const uint64_t s = a.tree[static_cast<int64_t>(w.b) * a.n_q + (row0 + (lane & 7)) % a.n_q];
                seen = make_uint2(static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32));
            }
            // Q: 8 channels a thread, D / 8 threads a row
            constexpr int TPR = D / 8;
            if (tl < 8 * TPR) {
                const int r = tl / TPR, ch = tl % TPR;
                uint4 u = make_uint4(0, 0, 0, 0);
                if (r < n_rows) u = *reinterpret_cast<const uint4 *>(a.q + (bh * a.R + row0 + r) * D + ch * 8);
                const uint32_t x[4] = {u.x, u.y, u.z, u.w};
                float2 f[4];
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
                    amax = fmaxf(amax, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
                }
#pragma unroll
                for (int o = 1; o < TPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                // exponent of the row's maximum, held where 2^(7 - e) and 2^(e - 7) are normal numbers
                int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
                e = amax == 0.f ? 7 : min(max(e, -100), 127);
                const float up = __uint_as_float(static_cast<uint32_t>(7 - e + 127) << 23);
                uint32_t hb[4], lb[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i].x *= up;
                    f[i].y *= up;
                    hb[i] = e4m3x2(f[i]);
                    const float2 v = e4m3x2_f32(hb[i]);
                    lb[i] = e4m3x2(make_float2((f[i].x - v.x) * 16.f, (f[i].y - v.y) * 16.f));
                }
                // row r's high part in column g * 16 + r, its rest 8 columns on
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const int col = g * 16 + r + part * 8;
                    const uint32_t *y = part ? lb : hb;
                    *reinterpret_cast<uint2 *>(smem + C::kQ + col * 128 + (((ch >> 1) ^ (col & 7)) << 4) + (ch & 1) * 8) =
                        make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
                }
                if (ch == 0) {
                    sm_mult[r] = !(amax < INFINITY) ? NAN : a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 7 + 127) << 23);
                    sm_m[r] = -FLT_MAX;
                    sm_top[r] = -FLT_MAX;
                    sm_f[r] = 1.f;
                }
            }
            fence_proxy_async_smem();
            sync();
            if (lane == 0) mbar_arrive(BAR(D_Q_READY));
            float2 l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] = make_float2(0.f, 0.f);
            // this thread's scores: an address carried along (made anew each tile it spilled 44 bytes: 12 rows with weights 76 us for 71)
            float *sc = SCORES ? a.scores + (bh * cap + w.t0 * TK + tl * KPT) * a.Rs + row0 : nullptr;

            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const int xs = n % XS;
                const uint8_t *scale = smem + C::kScale + xs * C::kScaleBytes;
                const int key0 = t * TK;
                ok = wait_both(BAR(X_FULL + xs), (n / XS) & 1, BAR(D_S_FULL), n & 1);
                if (!ok) *sm_fail = 1.f;
                tc_fence_after();
                // log2 scores of this thread's keys
                float2 x[KPT][4];
                float ks[4], vs[KPT];
                {
                    const uint32_t b = *reinterpret_cast<const uint32_t *>(scale + tl * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) ks[i] = kv4_scale((b >> (8 * i)) & 255u);
#pragma unroll
                    for (int k = 0; k < KPT; ++k) vs[k] = kv4_scale(scale[512 + tl * KPT + k]);
                }
                const bool here = reinterpret_cast<const int *>(scale + 768)[tl * KPT >> 4] != 0;
                {
                    uint32_t s[4][16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld16(tS + loff + i * N + g * 16, s[i]);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(D_S_FREE));
#pragma unroll
                    for (int k = 0; k < KPT; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float2 hi = make_float2(0.f, 0.f), lo = hi;
#pragma unroll
                            for (int i = 0; i < 4 / KPT; ++i) {
                                const int q = k * (4 / KPT) + i;
                                const float2 f = make_float2(ks[q], ks[q]);
                                const float2 sh = make_float2(__uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1]));
                                const float2 sl = make_float2(__uint_as_float(s[q][8 + 2 * j]), __uint_as_float(s[q][9 + 2 * j]));
                                hi = i == 0 ? mul2(f, sh) : fma2(f, sh, hi);
                                lo = i == 0 ? mul2(f, sl) : fma2(f, sl, lo);
                            }
                            const float2 m = *reinterpret_cast<const float2 *>(sm_mult + 2 * j);
                            x[k][j] = mul2(fma2(lo, make_float2(0.0625f, 0.0625f), hi), m);
                        }
                }
                // keys that a row does not admit, or that no page holds, leave it; what lies there may be anything
                const bool edge = key0 + TK > w.len - newest + (TREE ? 0 : 1) || __any_sync(0xffffffffu, !here);
                if (edge) {
#pragma unroll
                    for (int k = 0; k < KPT; ++k) {
                        const int key = key0 + tl * KPT + k;
                        const bool gone = key >= w.len || !here;
                        if (gone) vs[k] = 0.f;
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            bool out = gone;
                            if constexpr (TREE) {
                                const int draft = key - (w.len - newest);
                                const uint32_t lo = __shfl_sync(0xffffffffu, seen.x, r), hi = __shfl_sync(0xffffffffu, seen.y, r);
                                out |= draft >= 0 && (((draft & 32 ? hi : lo) >> (draft & 31)) & 1u) == 0;
                            } else {
                                out |= key >= w.len - a.n_q + 1 + (row0 + r) % a.n_q;
                            }
                            if (out) (r & 1 ? x[k][r / 2].y : x[k][r / 2].x) = -INFINITY;
                        }
                    }
                }
                if constexpr (SCORES) {
#pragma unroll
                    for (int k = 0; k < KPT; ++k) {
                        const int key = key0 + tl * KPT + k;
                        if (key < w.len) {
                            float *s = sc + k * a.Rs;
                            if (a.R <= 2) {
                                if (n_rows > 0) s[0] = x[k][0].x;
                                if (n_rows > 1) s[1] = x[k][0].y;
                            } else {
#pragma unroll
                                for (int r = 0; r < 2; ++r)
                                    if (4 * r < n_rows)
                                        *reinterpret_cast<float4 *>(s + 4 * r) =
                                            make_float4(x[k][2 * r].x, x[k][2 * r].y, x[k][2 * r + 1].x, x[k][2 * r + 1].y);
                            }
                        }
                    }
                }
                if (SCORES) sc += TK * a.Rs;
                // does a key pass its row's maximum, or its term the row's largest?  Soon that is rare.  (Terms are held against
                // the largest relative to the maximum: a large score's step may pass a scale's log2.)
                bool grows = false;
                float lv[KPT];  // log2 of V's scale
#pragma unroll
                for (int k = 0; k < KPT; ++k) lv[k] = lg2(vs[k]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float2 m = *reinterpret_cast<const float2 *>(sm_m + 2 * r), top = *reinterpret_cast<const float2 *>(sm_top + 2 * r);
#pragma unroll
                    for (int k = 0; k < KPT; ++k) {
                        const float2 y = make_float2(x[k][r].x - m.x, x[k][r].y - m.y), z = add2(y, make_float2(lv[k], lv[k]));
                        grows |= y.x > 0.f || y.y > 0.f || z.x > top.x || z.y > top.y;
                    }
                }
                grows = group_or(1 + g, grows);
                if (*sm_fail != 0.f) {
                    ok = false;
                    break;
                }
                if (grows) {
                    // O is complete so far, where it will be rescaled, and P's buffers are free
                    if (t > w.t0 && !mbar_wait_warp(pv_bar(n - 1), pv_phase(n - 1), kWaitLimitNs)) *sm_fail = 1.f;
                    // of the warp's keys, each row's maximum and its largest term over that
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        float v = -FLT_MAX, z = -FLT_MAX;
#pragma unroll
                        for (int k = 0; k < KPT; ++k) v = fmaxf(v, r & 1 ? x[k][r / 2].y : x[k][r / 2].x);
                        v = warp_max(v);
#pragma unroll
                        for (int k = 0; k < KPT; ++k) z = fmaxf(z, ((r & 1 ? x[k][r / 2].y : x[k][r / 2].x) - v) + lv[k]);
                        z = warp_max(z);
                        if (lane == 0) *reinterpret_cast<float2 *>(sm_red + (wl * 8 + r) * 2) = make_float2(v, z);
                    }
                    sync();
                    if (*sm_fail != 0.f) {
                        ok = false;
                        break;
                    }
                    if (tl < 8) {
                        const float old = sm_m[tl], f = sm_f[tl];
                        float2 y[4];
                        float v = old, z = -FLT_MAX;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            y[i] = *reinterpret_cast<const float2 *>(sm_red + (i * 8 + tl) * 2);
                            v = fmaxf(v, y[i].x);
                        }
                        if (v > old) v += kHeadroom;
#pragma unroll
                        for (int i = 0; i < 4; ++i) z = fmaxf(z, (y[i].x - v) + y[i].y);
                        const float rel = (old - v) + sm_top[tl];  // the row's largest term so far
                        z = z > rel ? z + kHeadroom : rel;
                        const float alpha = ex2(old - v);
                        // the power of two that keeps the terms up to 2^15; held at 2^100 where p itself is next to nothing
                        const int e = min(max(__float2int_rd(15.f - z), -100), 100);
                        const float now = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                        sm_m[tl] = v;
                        sm_top[tl] = z;
                        sm_alpha[tl] = alpha;
                        sm_f[tl] = now;
                        sm_oalpha[tl] = alpha * (now * inverse_pow2(f));
                    }
                    sync();
#pragma unroll
                    for (int r = 0; r < 4; ++r) l[r] = mul2(l[r], *reinterpret_cast<const float2 *>(sm_alpha + 2 * r));
                    if (t > w.t0) {
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < KPT; ++k) {
#pragma unroll
                            for (int part = 0; part < 3; ++part) {
                                const uint32_t at = tO + loff + (part < 2 ? unit(k) * 16 + part * 8 : C::kPart3 + unit(k) * 8);
                                uint32_t o[8];
                                tmem_ld8(at, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sm_oalpha[j]);
                                tmem_st8(at, o);
                            }
                        }
                        tmem_wait_st();
                    }
                }
                // has P's buffer been read?  (asked ahead; a wait where nothing is left to wait for takes 170 cycles)
                const bool free = n < C::kPBufs || mbar_test_wait(pv_bar(n), pv_phase(n - C::kPBufs));
                // P: the sum in fp32; the product's operand times V's scale and the row's factor, in three parts
                __half2 y[KPT][4];
#pragma unroll
                for (int k = 0; k < KPT; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 m = *reinterpret_cast<const float2 *>(sm_m + 2 * j), f = *reinterpret_cast<const float2 *>(sm_f + 2 * j);
                        const float2 xx = x[k][j];
                        const float2 p = make_float2(ex2(xx.x - m.x), ex2(xx.y - m.y));
                        l[j] = add2(l[j], p);
                        float2 pv = mul2(p, mul2(f, make_float2(vs[k], vs[k])));
                        if (edge) {  // a value that a row does not admit stays out of it, a NaN too
                            if (xx.x == -INFINITY) pv.x = 0.f;
                            if (xx.y == -INFINITY) pv.y = 0.f;
                        }
                        y[k][j] = __floats2half2_rn(pv.x, pv.y);
                    }
                if (!__all_sync(0xffffffffu, free) && !mbar_wait_warp(pv_bar(n), pv_phase(n - C::kPBufs), kWaitLimitNs)) *sm_fail = 1.f;
#pragma unroll
                for (int k = 0; k < KPT; ++k) {
                    uint32_t pa[4], pb[4], pc[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) e5m2_parts(y[k][j], pa[j], pb[j], pc[j]);
                    uint8_t *to = smem + C::kP + pbuf(n) * C::kPBytes + tl * 16;
                    *reinterpret_cast<uint4 *>(to + unit(k) * 2048) =
                        make_uint4(__byte_perm(pa[0], pa[1], 0x7531), __byte_perm(pa[2], pa[3], 0x7531),
                                   __byte_perm(pb[0], pb[1], 0x7531), __byte_perm(pb[2], pb[3], 0x7531));
                    *reinterpret_cast<uint2 *>(to + (C::U + unit(k) / 2) * 2048 + unit(k) % 2 * 8) =
                        make_uint2(pc[0] | (pc[1] << 16), pc[2] | (pc[3] << 16));
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(D_P_READY + pbuf(n)));
            }
            if (!ok) break;

            // ---------------------------------------------------- end of the segment
            if (!mbar_wait_warp(pv_bar(n - 1), pv_phase(n - 1), kWaitLimitNs)) *sm_fail = 1.f;
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float v = r & 1 ? l[r / 2].y : l[r / 2].x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) sm_red[wl * 8 + r] = v;
            }
            // this lane's channel of every row: the three parts' sums, the row's factor taken out
            float y[8];
            const int half = D == 64 ? wl >> 1 : 0;  // d = 64: lanes 64-127 hold the odd keys' part of channel lane - 64
            {
                uint32_t o[16], o3[8];
                tmem_ld16(tO + loff + unit(half) * 16, o);
                tmem_ld8(tO + loff + C::kPart3 + unit(half) * 8, o3);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = fmaf(__uint_as_float(o3[j]), 0x1p-8f, fmaf(__uint_as_float(o[8 + j]), 0.125f, __uint_as_float(o[j]))) *
                           inverse_pow2(sm_f[j]);
            }
            tc_fence_before();
            float *sx = reinterpret_cast<float *>(smem + C::kP) + g * 8 * 64;  // (the products have read P)
            if (D == 64 && half == 1) {
#pragma unroll
                for (int r = 0; r < 8; ++r) sx[r * 64 + tl - 64] = y[r];
            }
            sync();
            if (*sm_fail != 0.f) {
                ok = false;
                break;
            }
            if (D == 128 || half == 0) {
                const bool whole = w.t0 == 0 && w.t1 == w.n_t;
                const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (n == w.t1 - w.t0 ? 0 : 1);
                if (tid == 0 && w.t0 == 0 && !whole) {
                    Split sp;
                    sp.row = bh * a.R + row0;
                    sp.n_rows = min(RP, a.R - row0);
                    sp.parts = 1 + static_cast<int>((w.n_t - w.t1 + share - 1) / share);
                    sp.slot = static_cast<int>(slot);
                    sp.pad = 0;
                    a.split[blockIdx.x] = sp;
                }
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (r >= n_rows) break;
                    float v = y[r];
                    if (D == 64) v += sx[r * 64 + tl];
                    float ll = (sm_red[r] + sm_red[8 + r]) + (sm_red[16 + r] + sm_red[24 + r]);
                    const int64_t row = bh * a.R + row0 + r;
                    if (TREE && (row0 + r) % a.n_q >= newest) v = ll = 0.f;  // no draft of this sequence
                    if (whole) {
                        const float inv = ll == 0.f ? 0.f : 1.f / ll;
                        a.o[row * D + tl] = __float2bfloat16_rn(v * inv);
                        if (tl == 0) {
                            a.lse[row] = ll == 0.f ? -INFINITY : (sm_m[r] + log2f(ll)) * kLn2;
                            if (SCORES) a.row_ml[row] = make_float2(ll == 0.f ? 0.f : sm_m[r], inv);
                        }
                    } else {
                        a.part_o[(slot * RP + g * 8 + r) * D + tl] = v;
                        if (tl == 0) a.part_ml[slot * RP + g * 8 + r] = make_float2(sm_m[r], ll);
                    }
                }
            }
            sync();  // before the next segment's Q and state take the place of these
        }
        if (!ok && lane == 0) kv4_timeout();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

#include "fa_kv4_rows.cuh"

// Merge of the items that lie in several shares: a block per CTA of the kernel before, for the item whose first part that
// CTA holds; its warps over the item's rows and each row's parts.  Where there are few items, and so many parts of each, a
// block for every row of an item (gridDim.y).
constexpr int kMergeWarps = 16;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
fa_kv4_merge_kernel(const DecodeArgs a, int RP)
{
    constexpr int PER = D / 32;
    __shared__ float sm_l[kMergeWarps], sm_m[kMergeWarps];
    __shared__ float sm_x[kMergeWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    kv4_wait_for_the_one_before();
    const Split sp = a.split[blockIdx.x];
    if (sp.parts == 0) return;
    auto slot = [&](int i) -> int64_t { return i == 0 ? sp.slot : (static_cast<int64_t>(blockIdx.x) + i) * 2; };
    const int rows = (sp.n_rows + gridDim.y - 1) / gridDim.y;  // of this block
    const int row_end = min(sp.n_rows, static_cast<int>(blockIdx.y + 1) * rows);
    const int per_row = max(1, kMergeWarps / rows);  // warps a row
    for (int r0 = blockIdx.y * rows; r0 < row_end; r0 += kMergeWarps / per_row) {
        const int rr = r0 + warp / per_row, w = warp % per_row;
        const bool live = rr < row_end;
        float m = -FLT_MAX, l = 0.f, x[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = 0.f;
        constexpr int kBatch = 8;  // parts whose loads go out together, against a maximum of their own
        for (int i0 = live ? w : sp.parts; i0 < sp.parts; i0 += kBatch * per_row) {
            float2 v[kBatch];
            float y[kBatch][PER], mb = m;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * per_row;
                const int64_t s = slot(min(i, sp.parts - 1)) * RP + rr;
                const float *po = a.part_o + s * D + lane * PER;
                v[u] = a.part_ml[s];
                if constexpr (PER == 4)
                    *reinterpret_cast<float4 *>(y[u]) = *reinterpret_cast<const float4 *>(po);
                else
                    *reinterpret_cast<float2 *>(y[u]) = *reinterpret_cast<const float2 *>(po);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) mb = fmaxf(mb, v[u].x);
            const float back = ex2(m - mb);
            m = mb;
            l *= back;
#pragma unroll
            for (int j = 0; j < PER; ++j) x[j] *= back;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (i0 + u * per_row >= sp.parts) break;
                const float f = ex2(v[u].x - m);
                l = fmaf(f, v[u].y, l);
#pragma unroll
                for (int j = 0; j < PER; ++j) x[j] = fmaf(f, y[u][j], x[j]);
            }
        }
        if (per_row > 1) {
            if (lane == 0) {
                sm_l[warp] = l;
                sm_m[warp] = m;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) sm_x[warp][lane * PER + j] = x[j];
            __syncthreads();  // (with several warps a row all rows go in one turn)
            if (live && w == 0) {
                float mt = m;
                for (int i = 1; i < per_row; ++i) mt = fmaxf(mt, sm_m[warp + i]);
                const float back = ex2(m - mt);
                l *= back;
#pragma unroll
                for (int j = 0; j < PER; ++j) x[j] *= back;
                m = mt;
                for (int i = 1; i < per_row; ++i) {
                    const float f = ex2(sm_m[warp + i] - m);
                    l = fmaf(f, sm_l[warp + i], l);
#pragma unroll
                    for (int j = 0; j < PER; ++j) x[j] = fmaf(f, sm_x[warp + i][lane * PER + j], x[j]);
                }
            }
        }
        if (!live || w != 0) continue;
        const int64_t row = sp.row + rr;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int j = 0; j < PER; j += 2)
            *reinterpret_cast<__nv_bfloat162 *>(a.o + row * D + lane * PER + j) = __floats2bfloat162_rn(x[j] * inv, x[j + 1] * inv);
        if (lane == 0) {
            a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            if (a.scores != nullptr) a.row_ml[row] = make_float2(l == 0.f ? 0.f : m, inv);
        }
    }
}

// weights[key] += sum over the rows of exp2(score - m) / l.  Memory-bound by the scores, 4 Rs bytes a key.  L lanes read a key's
// rows, 4 C each (C = 0: one or two rows, a thread a key), and add them up; a warp has 32 U keys under way, 32 / L a turn, and
// each lane ends with the sums of U of them.  A thread a key is as fast up to 12 rows (24 sequences of 8 key heads with 12 rows: the
// whole call 71 us, with four lanes 2 more), but reads 16 bytes of a line at a time: with 32 rows 52 us for 67 MB of scores where
// eight lanes take 20; with 16 the whole call 63 us, with four lanes 59.
template <int L, int C, int U>
__global__ void __launch_bounds__(256)
fa_kv4_weights_kernel(const DecodeArgs a, int blocks)
{
    constexpr int KEYS = 32 / L, CC = C == 0 ? 1 : C;  // keys of a turn
    const int64_t bh = blockIdx.x / blocks, b = bh / a.c.heads;
    const int h = static_cast<int>(bh - b * a.c.heads), lane = threadIdx.x & 31, sub = lane % L;
    const int64_t cap = a.max_pages << a.c.log2_page;
    const int len = kv4_length(a.lens, b, cap);
    kv4_wait_for_the_one_before();
    // A wait gave up, in this call or in one before, and nobody has read so yet: the scores are not all there, and weights, which
    // a caller cannot compute again from what it has, stay as they are.  (An ordinary load, held against the store only: volatile
    // ones of every warp meet in one place of L2 and took 4 us of 61.)
    const bool off = g_kv4_status == FA_ERR_TIMEOUT;
    const float2 *ml = a.row_ml + bh * a.R;
    for (int key0 = blockIdx.x % blocks * 256 * U + (threadIdx.x & ~31); key0 < len; key0 += blocks * 256 * U) {
        int64_t row[U];
        float old[U], v[U][L][CC][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int own = key0 + u * 256 + sub * KEYS + lane / L;  // the key whose sum this lane takes
            bool valid;
            const int page = kv4_page_quiet(a.c, a.table, b, a.max_pages, min(own, len - 1), &valid);
            row[u] = kv4_row(a.c, page, h, min(own, len - 1));
            old[u] = a.c.weights[row[u]];
            if (!valid || own >= len) row[u] = -1;  // (a bad page is reported by the kernel before)
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int key = min(key0 + u * 256 + i * KEYS + lane / L, len - 1);
                const float *s = a.scores + (bh * cap + key) * a.Rs;
                if constexpr (C == 0) {
                    v[u][i][0][0] = s[0];
                    v[u][i][0][1] = a.R == 2 ? s[1] : 0.f;
                    v[u][i][0][2] = v[u][i][0][3] = 0.f;
                } else {
#pragma unroll
                    for (int c = 0; c < CC; ++c)
                        *reinterpret_cast<float4 *>(v[u][i][c]) = *reinterpret_cast<const float4 *>(s + min(4 * (sub + c * L), a.Rs - 4));
                }
            }
        float mine[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < L; ++i) {
                // with the guard a key that a row does not admit (score -infinity) has no weight in it, whatever the row's sum is
                auto sum = [&](auto guard) {
                    float w = 0.f;
                    auto add = [&](float x, float2 p) {
                        const float e = ex2(x - p.x);
                        if (!decltype(guard)::value || e != 0.f) w = fmaf(e, p.y, w);
                    };
#pragma unroll
                    for (int c = 0; c < CC; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 4 * (sub + c * L) + j;
                            if (r < a.R) add(v[u][i][c][j], ml[r]);  // (what lies behind the last row may be anything)
                        }
                    if constexpr (L * C == 16) {  // more than 64 rows
                        const float *s = a.scores + (bh * cap + min(key0 + u * 256 + i * KEYS + lane / L, len - 1)) * a.Rs;
                        for (int r0 = 4 * (C * L + sub); r0 < a.R; r0 += 4 * L) {
                            const float4 f = *reinterpret_cast<const float4 *>(s + r0);
                            const float y[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (r0 + j < a.R) add(y[j], ml[r0 + j]);
                        }
                    }
                    return w;
                };
                float w = sum(std::false_type{});
                if (w != w) w = sum(std::true_type{});  // (asked of every term 216 us became 237, for 80 rows)
#pragma unroll
                for (int o = 1; o < L; o <<= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
                if (sub == i) mine[u] = w;
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row[u] >= 0 && !off) a.c.weights[row[u]] = old[u] + mine[u];
    }
}

// ------------------------------------------------------------------ host side

struct Geometry {
    int rt, ng, rows, n_rc, ctas, whole, Rs;  // rows: of a chunk
    int64_t part_o, part_ml, split, scores, row_ml, total;  // byte offsets in the workspace
};

// The CTAs and the workspace's layout of items of g.n_rc chunks of g.rows rows.
void lay_out(Geometry &g, int64_t B, int64_t H, int64_t heads, int64_t n_q, int64_t d, int64_t max_tokens, int accumulate)
{
    const int64_t R = H / heads * n_q, rows = B * H * n_q;
    const int64_t tk = g.ng > 0 ? 128 : tile_keys(static_cast<int>(d));
    const int64_t items = B * heads * g.n_rc, tiles = (max_tokens + tk - 1) / tk;
    g.whole = tiles <= kWholeTiles;
    g.Rs = static_cast<int>(R <= 2 ? R : (R + 3) / 4 * 4);
    const int64_t ctas = kSms * (g.ng > 0 ? 1 : g.rt == 1 ? 3 : g.rt == 2 ? 2 : 1);
    const int64_t need = g.whole ? items : (items * (tiles + (g.ng > 0 ? kRowsItemUnits : kItemUnits)) + kMinShare - 1) / kMinShare;
    g.ctas = static_cast<int>(need < ctas ? need : ctas);
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    int64_t at = 0;
    g.part_o = at;
    at = up(at + g.ctas * 2 * g.rows * d * 4);
    g.part_ml = at;
    at = up(at + g.ctas * 2 * g.rows * 8);
    g.split = at;
    at = up(at + g.ctas * static_cast<int64_t>(sizeof(Split)));
    g.scores = at;
    if (accumulate) at = up(at + B * heads * g.Rs * max_tokens * 4);
    g.row_ml = at;
    if (accumulate) at = up(at + rows * 8);
    g.total = at;
}

// tree: for fa_fwd_kv4_tree, whose items of many rows a key head go to fa_kv4_rows_kernel (g.ng > 0) or, where there is little work,
// in smaller chunks.  Up to 8 rows it has the chain's chunks and shares, and so its bits.
Geometry geometry(int64_t B, int64_t H, int64_t heads, int64_t n_q, int64_t d, int64_t max_tokens, int accumulate, bool tree)
{
    Geometry g;
    const int64_t R = H / heads * n_q;
    g.ng = 0;
    // 32 sequences of 8192, 4 key heads: a chunk of 16 rows takes 39 to 41 us among others, one of 32 74 (32 rows in one CTA 85, in
    // two of 16 89; 40 rows in two of 32 144, in three of 16 123; 1 key head: 80 rows 67 and 62, 96 rows 67 and 71, 176 even)
    g.rt = R <= 8 ? 1 : R <= 16 || (R + 15) / 16 * 7 < (R + 31) / 32 * 13 ? 2 : 4;
    if (tree && R > 8) {
        // Units (tiles, and kItemUnits an item) for each CTA that the SMs hold, in chunks of 8 and of 16 rows.
        // Few: chunks of 8.  1 sequence of 700, 4 key heads, 64 rows, d = 64 (0.3 units): chunks of 8 11.1 us, of 16 12.2, the other
        // kernel 19.3; 1 of 4000, 8 key heads, 48 rows, d = 128 (3.7) 23.0, 22.9, 27.6; 2 of 2000, 64 rows (5.3) 20.8, 18.6, 21.7; 1 of
        // 4000, 4 key heads, 16 rows (0.6) 13.9 and 15.1.
        // Many: the other kernel, whose first tile takes 15 us more and the others less.  8 key heads, 48 rows, d = 128, chunks
        // of 16 and the other kernel: 4 sequences of up to 4000 (11 units) 21.7 and 30.3; 1 of 30000 (18.8) 46.7 and 42.7; 32 of up
        // to 8192 (169) 160 and 101, 24 rows 101 and 89, 32 rows 108 and 95, 64 rows 186 and 156, 128 rows 350 and 245; d = 64,
        // 48 rows 124 and 106, 64 rows 140 and 145, 128 rows 268 and 237, but 24 rows (in one chunk of 32) 81 and 89, 32 rows 77
        // and 82.  Short tables, 128 sequences, d = 128, 48 rows: of 640 tokens 129 and 117, 512 122 and 99, 384 109 and 104, 272 107 and 103; of
        // 256, where the first tile is half of an item, 95 and 106, of 128 79 and 90 (128 rows 231 and 321, 188 and 259; d = 64, 48 rows 92
        // and 100, 91 and 86): there the rule, which looks at the work alone, takes the slower one.
        const int64_t tiles = (max_tokens + tile_keys(static_cast<int>(d)) - 1) / tile_keys(static_cast<int>(d));
        auto work = [&](int64_t rows, int64_t per_sm) { return B * heads * ((R + rows - 1) / rows) * (tiles + kItemUnits) / (kSms * per_sm); };
        if (work(8, 3) < 2) {
            g.rt = 1;
        } else if (R <= 16 || work(16, 2) < 14) {
            g.rt = 2;
        } else if (d == 128 || R > 32) {
            g.n_rc = static_cast<int>((R + 47) / 48);
            g.ng = static_cast<int>(((R + g.n_rc - 1) / g.n_rc + 15) / 16);
        }
    }
    if (g.ng == 0) g.n_rc = static_cast<int>((R + 8 * g.rt - 1) / (8 * g.rt));
    g.rows = g.ng > 0 ? 16 * g.ng : 8 * g.rt;
    lay_out(g, B, H, heads, n_q, d, max_tokens, accumulate);
    return g;
}

// Bytes for fa_fwd_kv4_tree with at most so many sequences, drafts and tokens of a table: the most over the forms that geometry
// may choose for any such call.  (Of each the CTAs grow with the items and the tiles, up to what the SMs hold; it is the choice
// that does not: 6 drafts of 32 heads on 8, d = 128, tables of 8192, go in chunks of 16 rows for 3 sequences, of 32 for 16, in less.)
int64_t tree_workspace(int64_t B, int64_t H, int64_t heads, int64_t n_q, int64_t d, int64_t max_tokens)
{
    const int64_t R = H / heads * n_q;
    int64_t most = 0;
    auto form = [&](int rt, int ng, int rows) {
        Geometry g;
        g.rt = rt;
        g.ng = ng;
        g.rows = rows;
        g.n_rc = static_cast<int>((R + rows - 1) / rows);
        lay_out(g, B, H, heads, n_q, d, max_tokens, 0);
        most = std::max(most, g.total);
    };
    form(1, 0, 8);
    if (R > 8) form(2, 0, 16);
    if (R > 16 && d == 64) form(4, 0, 32);
    if (R > 16 && (d == 128 || R > 32)) form(4, 3, 48);  // (in even chunks of at most 48)
    return most;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

// The pool's codes as [page][head][row][128 values], a row being one token (d = 128) or two (d = 64); a box is
// one page's rows of one head, at most a tile's.
bool make_code_map(CUtensorMap *m, const Kv4Cache &c, void *base)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t rows = (cuuint64_t(1) << c.log2_page) * c.d / 128;
    const cuuint64_t dims[4] = {128, rows, static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.n_pages)};
    const cuuint64_t strides[3] = {64, rows * 64, rows * 64 * c.heads};
    const cuuint32_t box[4] = {128, static_cast<cuuint32_t>(rows < 128 ? rows : 128), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RT, bool SCORES, bool TREE>
cudaError_t launch(const DecodeArgs &a, int ctas, cudaStream_t s)
{
    using C = DecCfg<D, RT>;
    CUtensorMap mk, mv;
    if (!make_code_map(&mk, a.c, a.c.k) || !make_code_map(&mv, a.c, a.c.v)) return cudaErrorInvalidValue;
    cudaError_t e = set_max_dynamic_smem<fa_kv4_decode_kernel<D, RT, SCORES, TREE>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    fa_kv4_decode_kernel<D, RT, SCORES, TREE><<<static_cast<unsigned>(ctas), C::kThreads, C::kSmemBytes, s>>>(mk, mv, a);
    return cudaGetLastError();
}

template <int D, bool SCORES, bool TREE>
cudaError_t launch_rt(const DecodeArgs &a, int rt, int ctas, cudaStream_t s)
{
    if (rt == 1) return launch<D, 1, SCORES, TREE>(a, ctas, s);
    if constexpr (!TREE || D == 64)  // (d = 128: trees go in chunks of 8 or 16, or to the other kernel)
        if (rt == 4) return launch<D, 4, SCORES, TREE>(a, ctas, s);
    return launch<D, 2, SCORES, TREE>(a, ctas, s);
}

template <int D, int NG>
cudaError_t launch_rows(const DecodeArgs &a, int ctas, cudaStream_t s)
{
    using C = RowCfg<D, NG>;
    const cudaError_t e = set_max_dynamic_smem<fa_kv4_rows_kernel<D, NG>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    fa_kv4_rows_kernel<D, NG><<<static_cast<unsigned>(ctas), C::kThreads, C::kSmemBytes, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_kind(const DecodeArgs &a, int rt, int ng, int ctas, cudaStream_t s)
{
    if (ng > 0)
        return ng == 2 ? launch_rows<D, 2>(a, ctas, s) : launch_rows<D, 3>(a, ctas, s);
    if (a.tree != nullptr) return launch_rt<D, false, true>(a, rt, ctas, s);
    return a.scores != nullptr ? launch_rt<D, true, false>(a, rt, ctas, s) : launch_rt<D, false, false>(a, rt, ctas, s);
}

}  // namespace

int64_t fa_kv4_decode_workspace(int64_t B, int64_t H, int64_t heads, int64_t n_q, int64_t d, int64_t max_tokens,
                                int accumulate, bool tree)
{
    return tree ? tree_workspace(B, H, heads, n_q, d, max_tokens) : geometry(B, H, heads, n_q, d, max_tokens, accumulate, false).total;
}

cudaError_t fa_launch_kv4_decode(const Kv4DecodeProblem &p, void *workspace, cudaStream_t stream)
{
    const int64_t cap = p.max_pages << p.cache.log2_page, heads = p.cache.heads;
    const Geometry g = geometry(p.B, p.H, heads, p.n_q, p.cache.d, cap, p.accumulate, p.tree != nullptr);
    const int64_t rows = p.B * p.H * p.n_q;
    if (rows > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    char *ws = static_cast<char *>(workspace);
    DecodeArgs a;
    a.c = p.cache;
    a.q = static_cast<const __nv_bfloat16 *>(p.q);
    a.lens = p.lens;
    a.table = p.table;
    a.tree = p.tree;
    a.n_new = p.n_new;
    a.o = static_cast<__nv_bfloat16 *>(p.o);
    a.lse = p.lse;
    a.part_o = reinterpret_cast<float *>(ws + g.part_o);
    a.part_ml = reinterpret_cast<float2 *>(ws + g.part_ml);
    a.split = reinterpret_cast<Split *>(ws + g.split);
    a.scores = p.accumulate ? reinterpret_cast<float *>(ws + g.scores) : nullptr;
    a.row_ml = reinterpret_cast<float2 *>(ws + g.row_ml);
    a.max_pages = p.max_pages;
    a.B = static_cast<int>(p.B);
    a.R = static_cast<int>(p.H / heads * p.n_q);
    a.n_q = static_cast<int>(p.n_q);
    a.n_rc = g.n_rc;
    a.Rs = g.Rs;
    a.whole = g.whole;
    a.item_cost = g.ng > 0 ? kRowsItemUnits : kItemUnits;
    a.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    cudaError_t e = p.cache.d == 128 ? launch_kind<128>(a, g.rt, g.ng, g.ctas, stream)
                                        : launch_kind<64>(a, g.rt, g.ng, g.ctas, stream);
    if (e != cudaSuccess) return e;
    if (!g.whole && g.ctas > 1) {
        // few items of many parts: 8 of 57 parts and 4 rows took 12.3 us with a block an item, 9.2 with one a row
        const int64_t items = p.B * heads * g.n_rc;
        const int rows = a.R < g.rows ? a.R : g.rows;
        int parts_of_rows = items * 8 <= g.ctas ? rows : 1;
        // (trees of more than 8 rows, whose sums are in an order of their own: no more blocks than are resident at one time; 1
        // sequence of 4000, 8 key heads, 48 rows, 23.0 -> 18.5 us for the call, of 30000 42.8 -> 37.0; 8 of up to 4000, 4 key heads,
        // 16 rows, 22.6 -> 16.8)
        if (a.tree != nullptr && a.R > 8) parts_of_rows = std::min(parts_of_rows, std::max(1, 4 * kSms / g.ctas));
        const dim3 grid(static_cast<unsigned>(g.ctas), parts_of_rows);
        e = p.cache.d == 128 ? kv4_launch_behind(fa_kv4_merge_kernel<128>, grid, kMergeWarps * 32, stream, a, g.rows)
                             : kv4_launch_behind(fa_kv4_merge_kernel<64>, grid, kMergeWarps * 32, stream, a, g.rows);
        if (e != cudaSuccess) return e;
    }
    if (p.accumulate) {
        int64_t blocks = (cap + 511) / 512, most = 0x7fffffffLL / (p.B * heads);
        if (blocks > 512) blocks = 512;
        if (blocks > most) blocks = most;  // (at least 1: the rows fit 31 bits)
        auto *kern = a.R <= 2 ? fa_kv4_weights_kernel<1, 0, 2> : a.Rs <= 4 ? fa_kv4_weights_kernel<1, 1, 2>
                     : a.Rs <= 8 ? fa_kv4_weights_kernel<1, 2, 2> : a.Rs <= 12 ? fa_kv4_weights_kernel<1, 3, 1>
                     : a.Rs <= 16 ? fa_kv4_weights_kernel<4, 1, 1> : a.Rs <= 32 ? fa_kv4_weights_kernel<8, 1, 1>
                     : a.Rs <= 48 ? fa_kv4_weights_kernel<4, 3, 1> : fa_kv4_weights_kernel<8, 2, 1>;
        e = kv4_launch_behind(kern, dim3(static_cast<unsigned>(blocks * p.B * heads)), 256, stream, a, static_cast<int>(blocks));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int fa_kv4_decode_take_status(cudaStream_t stream) { return fa_take_status_word(g_kv4_status, stream); }
