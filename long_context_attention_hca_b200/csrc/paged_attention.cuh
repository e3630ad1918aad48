// paged_attention.cuh -- what the paged attention kernels share: parameters,
// the map from a CTA to a request's rows, the visible keys, page lookups.
#pragma once

#include "common.cuh"

namespace hca {
namespace paged {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;
constexpr int TK = 64;                       // keys per tile
constexpr int MAX_SPLITS = 64;

struct Params {
    const uint16_t* q;          // [n_rows][H][D] bf16
    int64_t n_rows;
    int H, B;
    const int32_t* row_start;   // [B + 1]
    const int32_t* ctx;         // [B] tokens cached before this step
    // compressed entries (m = 0: none)
    int m;
    const uint8_t* codes;
    const float* scales;
    const uint16_t* rope;
    int64_t e_pages;
    uint32_t e_size;            // entries per page
    const int32_t* e_table;     // [B][e_width]
    uint32_t e_width;
    // raw tokens
    const uint16_t* tok;
    int64_t t_pages;
    uint32_t t_size;
    const int32_t* t_table;
    uint32_t t_width;
    int W, n_first;
    float scale_log2;
    int n_splits;
    uint16_t* out;
    uint16_t* part_o;           // [tiles][splits][rows][D] fp16: O / l of the split
    float* part_ml;             // [tiles][splits][2][rows]: running max (base 2), l
    // section 9 extras (each null when off)
    const float* q_norm_w;
    float norm_eps;
    const float* sink;
    const float* inv_freq;
};

// Tiles of R rows, a row = (new token, head) flattened inside a request, so
// that a tile never mixes two requests' keys.  Request b owns the tile numbers
// floor(row_start[b] H / R) + b .. floor(row_start[b+1] H / R) + b: at least
// ceil(new H / R) of them, disjoint and ascending in b, and computable from
// row_start alone (no tile list to build, none to wait for).  The search is
// 32 candidates wide, one round for up to 32 requests.
__device__ __forceinline__ int64_t tile0(const Params& p, int b, int R) {
    return static_cast<int64_t>(p.row_start[b]) * p.H / R + b;
}

// The largest b in [0, n) with at_most(b), which holds up to some b >= 0 and for
// none after; whole warps.
template <class F>
__device__ __forceinline__ int last_at_most(int n, F at_most) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int c = lo + lane * step;
        const unsigned mask = __ballot_sync(0xffffffffu, c < hi && (lane == 0 || at_most(c)));
        lo += (31 - __clz(mask)) * step;
        if (lo + step < hi) hi = lo + step;
    }
    return lo;
}

__device__ __forceinline__ int find_tile_req(const Params& p, int64_t t, int R) {
    return last_at_most(p.B, [&](int b) { return tile0(p, b, R) <= t; });
}

// One tile's rows and keys.  Key slots in order: entries [0, n_e), first
// tokens [0, n_f), window tokens [w_lo, w_lo + n_w).
struct Tile {
    int b;
    int64_t row0;               // first row of the tile in q / out: (row_start[b] H + ...)
    int r0, rows;               // first row inside the request, rows that hold a query
    int64_t ctx;
    int n_new;
    int64_t w_lo;
    int n_e, n_f, n_w, n_tot;
};

__device__ __forceinline__ int64_t entries_before(const Params& p, int64_t pos) {
    if (p.m <= 0) return 0;
    // positions stay below 2^31
    const int64_t e = static_cast<uint32_t>(pos + 1) / static_cast<uint32_t>(p.m);
    const int64_t cap = static_cast<int64_t>(p.e_width) * p.e_size;
    return e < cap ? e : cap;
}

// false: the tile has no rows here.  Called by whole warps.
__device__ __forceinline__ bool make_tile(const Params& p, int64_t t, int R, Tile& T) {
    const int b = find_tile_req(p, t, R);
    const int64_t s = p.row_start[b];
    int64_t e = p.row_start[b + 1];
    if (e > p.n_rows) e = p.n_rows;
    T.b = b;
    T.n_new = s < 0 || e < s ? 0 : static_cast<int>(e - s);
    const int64_t r0 = (t - tile0(p, b, R)) * R;
    const int64_t left = static_cast<int64_t>(T.n_new) * p.H - r0;
    if (left <= 0 || r0 < 0) return false;
    T.r0 = static_cast<int>(r0);
    T.rows = static_cast<int>(left < R ? left : R);
    T.row0 = s * p.H + r0;
    T.ctx = p.ctx[b] > 0 ? p.ctx[b] : 0;
    const int64_t p_lo = T.ctx + T.r0 / p.H, p_hi = T.ctx + (T.r0 + T.rows - 1) / p.H;
    T.w_lo = p_lo - (p.W - 1) > 0 ? p_lo - (p.W - 1) : 0;
    T.n_e = static_cast<int>(entries_before(p, p_hi));
    T.n_f = static_cast<int>(p.n_first < T.w_lo ? p.n_first : T.w_lo);
    T.n_w = static_cast<int>(p_hi - T.w_lo + 1);
    T.n_tot = T.n_e + T.n_f + T.n_w;
    return true;
}

// The slots that a query at position pos sees: slot < e_lim, or n_e <= slot <=
// w_hi with (slot >= w_from or slot < f_to).
struct RowKeys { int e_lim, w_from, w_hi, f_to; };

__device__ __forceinline__ RowKeys row_keys(const Params& p, const Tile& T, int64_t pos) {
    RowKeys k;
    const int w0 = T.n_e + T.n_f;
    const int64_t from = pos - (p.W - 1) > T.w_lo ? pos - (p.W - 1) : T.w_lo;
    k.e_lim = static_cast<int>(entries_before(p, pos));
    k.w_from = w0 + static_cast<int>(from - T.w_lo);
    k.w_hi = w0 + static_cast<int>(pos - T.w_lo);
    // first tokens: all n_f of them, and those that lie inside the tile's window range
    const int64_t f = T.w_lo < p.n_first ? static_cast<int64_t>(p.n_first) : T.n_f;
    k.f_to = T.n_e + static_cast<int>(f < T.n_f + T.n_w ? f : T.n_f + T.n_w);
    return k;
}

__device__ __forceinline__ bool sees(const RowKeys& k, int n_e, int slot) {
    return slot < k.e_lim || (slot >= n_e && slot <= k.w_hi && (slot >= k.w_from || slot < k.f_to));
}

// Row of a slot's key in its pool, or -1: no such slot, a page number outside
// the pool, or a column outside the table (the key is then not visible).
__device__ __forceinline__ int64_t entry_row(const Params& p, int b, uint32_t e) {
    const uint32_t pg = e / p.e_size;
    if (pg >= p.e_width) return -1;
    const int64_t id = __ldg(p.e_table + static_cast<size_t>(b) * p.e_width + pg);
    return id >= 0 && id < p.e_pages ? id * p.e_size + e % p.e_size : -1;
}
__device__ __forceinline__ int64_t token_row(const Params& p, int b, uint32_t t) {
    const uint32_t pg = t / p.t_size;
    if (pg >= p.t_width) return -1;
    const int64_t id = __ldg(p.t_table + static_cast<size_t>(b) * p.t_width + pg);
    return id >= 0 && id < p.t_pages ? id * p.t_size + t % p.t_size : -1;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Whether any of these fp16 pairs holds an infinity or a NaN: x * 0 is then a
// NaN and stays one in the sum, and +-0 otherwise.
template <int N>
__device__ __forceinline__ bool any_bad(const uint32_t (&h)[N]) {
    uint32_t z = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(h[i]), "r"(0u));
    return (z & 0x7FFF7FFFu) != 0;
}

// 16 FP8 codes x their scale -> fp16.  A scale in fp16's normal range is
// rounded to fp16 (half a step, 2^-11) and each product once more (2^-11): one
// conversion and one multiplication per pair, where products in fp32 take four
// conversions per pair, at a quarter of the rate.  Any other scale: fp32
// products, rounded once.
__device__ __forceinline__ void dequant16(const uint4& cv, float sc, uint32_t (&h)[8]) {
    const uint32_t cw[4] = {cv.x, cv.y, cv.z, cv.w};
    if (sc >= 6.103515625e-05f && sc <= 65504.0f) {
        const uint32_t s2 = pack_half2(sc, sc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[2 * i] = hmul2(e4m3x2_to_f16x2(static_cast<uint16_t>(cw[i] & 0xFFFFu)), s2);
            h[2 * i + 1] = hmul2(e4m3x2_to_f16x2(static_cast<uint16_t>(cw[i] >> 16)), s2);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = unpack_half2(e4m3x2_to_f16x2(static_cast<uint16_t>(cw[i] & 0xFFFFu)));
            const float2 b = unpack_half2(e4m3x2_to_f16x2(static_cast<uint16_t>(cw[i] >> 16)));
            h[2 * i] = pack_half2(a.x * sc, a.y * sc);
            h[2 * i + 1] = pack_half2(b.x * sc, b.y * sc);
        }
    }
}

// cos / sin of RoPE pair i at position t, fp32 out.  The angle t f_i is an fp64
// product (exact below position 2^29: 29 + 24 bits); its whole half turns are
// taken off there, and the rest, in [-1/2, 1/2] half turns, goes to sincospif.
// u = t f_i / pi is off by three roundings (the angle, 1 / pi, the product), 3 x
// 2^-53 of itself: for f_i <= 1 below 2^-24 of a half turn up to position 2^29
// and 2^-22 at 2^31, where the query's rounding to fp16 is 2^-11.  An fp64 sincos
// costs 16K clocks of latency here, more than the query's load.
__device__ __forceinline__ float2 rope_cs(const float* inv_freq, int i, int64_t t) {
    const double u = static_cast<double>(t) * static_cast<double>(__ldg(inv_freq + i)) * 0.31830988618379067154;
    const double k = rint(u);
    float sn, cs;
    sincospif(static_cast<float>(u - k), &sn, &cs);
    if (static_cast<long long>(k) & 1) { sn = -sn; cs = -cs; }
    return make_float2(cs, sn);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace paged
}  // namespace hca
