// paged_cache.cu -- the paged cache's bookkeeping and its writes: block tables
// and slot maps of a step from request lengths, raw tokens into their pages,
// pooled entries into theirs.
//
// "DeepSeek V4 ..." reading note, section 11: a classical cache of compressed
// entries plus a state cache of the recent window and the uncompressed tail of
// the block not yet complete.  Here both live in pages that requests of
// different lengths share, and each request advances by its own number of new
// tokens per step.  The stored bits are those of the contiguous calls: the
// same fixed fp32 sequences (pooling.cuh, include/hca.h).
#include "pooling.cuh"

namespace hca {
namespace {

// ---------------------------------------------------------------- page plan
// Request b owns items [lo, hi) = [ctx / m, (ctx + new) / m) of this step
// (tokens for m = 1, entries of m tokens otherwise).  Two exclusive prefix
// sums over the requests decide everything else: rows (hi - lo) and new pages
// (ceil(hi / P) - ceil(lo / P)).
//
// Bound: latency (16 B written per row; 46K rows are 0.7 MB).  So one launch:
// every CTA scans the requests for itself into shared memory (8 B each, L2
// hits) instead of waiting for another CTA's scan, then finds each of its rows'
// request by binary search there.  Nothing that a CTA reads is written by
// another: fresh pages are computed from the free list, old ones are read from
// table columns that this step does not write, and the free count left is a
// separate output.  Measured (in a graph): 32 requests of one token 3.5 us, 192
// requests with 46K rows 4.6 us.
//
// Pages missing: new ones that the stack or the table's width does not give, and
// pages begun in an earlier step that got none then, where this step has an item
// in them (no fresh page takes their place: the page's earlier items are lost,
// and a page that lacks them must not become visible).
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 16384;            // the C ABI's bound

struct PlanArgs {
    const int32_t* ctx;
    const int32_t* nnew;
    int B, m, P;
    int32_t* table;
    int width;
    const int32_t* free_pages;
    const int32_t* free_count;
    int free_cap;
    int64_t max_rows;
    int32_t *row_start, *row_req, *row_pos;
    int64_t* slot;
    int32_t *missing, *free_left;
};

struct Span { uint32_t lo, hi; };

// lengths below zero count as zero; positions end at 2^31 - 1
__device__ __forceinline__ Span plan_span(const PlanArgs& a, int b) {
    const int64_t c = max(a.ctx[b], 0);
    const int64_t e = min(c + static_cast<int64_t>(max(a.nnew[b], 0)), static_cast<int64_t>(0x7FFFFFFF));
    return {static_cast<uint32_t>(c) / static_cast<uint32_t>(a.m), static_cast<uint32_t>(e) / static_cast<uint32_t>(a.m)};
}

__device__ __forceinline__ uint32_t pages_of(uint32_t n, uint32_t P) { return n / P + (n % P != 0); }

// largest b in [0, n) with s[b] <= v (s ascending, s[0] <= v)
__device__ __forceinline__ int find_req(const int32_t* s, int n, int32_t v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanArgs a) {
    extern __shared__ int32_t sh[];
    int32_t* s_row = sh;                    // [B + 1]
    int32_t* s_page = sh + a.B + 1;         // [B + 1]
    __shared__ int64_t s_warp[3][kPlanThreads / 32];
    __shared__ int64_t s_carry[3];          // rows, pages inside the table, pages wanted
    __shared__ int s_gone;                  // pages begun earlier that the step needs and no one has
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t P = a.P, width = a.width;
    if (tid < 3) s_carry[tid] = 0;
    if (tid == 0) s_gone = 0;
    __syncthreads();
    // counted by the last CTA, which has the fewest rows; a load is waited for in the next round, or at the end
    const bool counts = blockIdx.x == gridDim.x - 1;
    int gone = 0;
    int32_t held = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int64_t v[3] = {0, 0, 0};
        if (b < a.B) {
            const Span s = plan_span(a, b);
            const uint32_t have = pages_of(s.lo, P), want = pages_of(s.hi, P);
            v[0] = s.hi - s.lo;
            v[1] = min(want, width) - min(have, width);
            v[2] = want - have;
            if (counts) {
                gone += held < 0;
                held = 0;
                if (s.hi > s.lo && s.lo % P != 0)
                    held = have > width ? -1 : a.table[static_cast<size_t>(b) * width + have - 1];
            }
        }
        int64_t inc[3] = {v[0], v[1], v[2]};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, inc[k], o);
                if (lane >= o) inc[k] += x;
            }
            if (lane == 31) s_warp[k][warp] = inc[k];
        }
        __syncthreads();
        int64_t base[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            base[k] = s_carry[k];
            for (int w = 0; w < warp; ++w) base[k] += s_warp[k][w];
        }
        if (b < a.B) {
            // a running total beyond 2^31 - 1 stays there (no such row exists)
            s_row[b] = static_cast<int32_t>(min(base[0] + inc[0] - v[0], static_cast<int64_t>(0x7FFFFFFF)));
            s_page[b] = static_cast<int32_t>(min(base[1] + inc[1] - v[1], static_cast<int64_t>(0x7FFFFFFF)));
        }
        __syncthreads();
        if (tid == kPlanThreads - 1)
            for (int k = 0; k < 3; ++k) s_carry[k] = base[k] + inc[k];
        __syncthreads();
    }
    if (tid == 0) {
        s_row[a.B] = static_cast<int32_t>(min(s_carry[0], static_cast<int64_t>(0x7FFFFFFF)));
        s_page[a.B] = static_cast<int32_t>(min(s_carry[1], static_cast<int64_t>(0x7FFFFFFF)));
    }
    __syncthreads();
    const int F = max(min(*a.free_count, a.free_cap), 0);
    const int64_t gtid = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    const int64_t gsz = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    // the k-th new page of the step comes from the top of the free stack
    auto fresh = [&](int64_t k) -> int32_t { return k < F ? a.free_pages[F - 1 - k] : -1; };
    const int64_t rows = min(static_cast<int64_t>(s_row[a.B]), a.max_rows);
    for (int64_t r = gtid; r < rows; r += gsz) {
        const int b = find_req(s_row, a.B, static_cast<int32_t>(r));
        const uint32_t lo = static_cast<uint32_t>(max(a.ctx[b], 0)) / static_cast<uint32_t>(a.m);
        const uint32_t pos = lo + static_cast<uint32_t>(r - s_row[b]);
        const uint32_t pi = pos / P, have = pages_of(lo, P);
        int32_t id = -1;
        if (pi < width)
            id = pi < have ? a.table[static_cast<size_t>(b) * width + pi]
                           : fresh(static_cast<int64_t>(s_page[b]) + (pi - min(have, width)));
        a.row_req[r] = b;
        a.row_pos[r] = static_cast<int32_t>(pos);
        a.slot[r] = id >= 0 ? static_cast<int64_t>(id) * P + pos % P : -1;
    }
    const int64_t pages = s_page[a.B];
    for (int64_t k = gtid; k < pages; k += gsz) {
        const int b = find_req(s_page, a.B, static_cast<int32_t>(k));
        const uint32_t lo = static_cast<uint32_t>(max(a.ctx[b], 0)) / static_cast<uint32_t>(a.m);
        const uint32_t pi = min(pages_of(lo, P), width) + static_cast<uint32_t>(k - s_page[b]);
        a.table[static_cast<size_t>(b) * width + pi] = fresh(k);
    }
    for (int64_t b = gtid; b <= a.B; b += gsz) a.row_start[b] = s_row[b];
    if (!counts) return;
    gone += held < 0;
    if (gone) atomicAdd(&s_gone, gone);
    __syncthreads();
    if (tid == 0) {
        const int64_t granted = min(s_carry[1], static_cast<int64_t>(F));
        *a.missing = static_cast<int32_t>(min(s_carry[2] - granted + s_gone, static_cast<int64_t>(0x7FFFFFFF)));
        *a.free_left = F - static_cast<int32_t>(granted);
    }
}

// ---------------------------------------------------------------- token store
// One warp per token, 16 (d = 512) or 4 (d = 128) consecutive channels per
// lane: the RMSNorm's pairwise tree closes inside the warp (no block barrier),
// and each lane computes the fp64 angle of ONE RoPE pair (the d_rope / 2 pairs
// over the lanes), where a thread that owns 8 channels would compute four in a
// row.  Bytes: 4 d + 12 a token.  Measured (in a graph): 14K tokens of d = 512
// with RMSNorm and RoPE 10.0 us, 2.9 TB/s (44% of a copy); 32 tokens 3.0 us, a
// load, the tree and a store in a row.
template <int D>
__global__ void __launch_bounds__(256)
page_store_kernel(const uint16_t* __restrict__ x, int64_t n_rows, const int32_t* __restrict__ n_live,
                  const int32_t* __restrict__ pos, const int64_t* __restrict__ slot, int d_rope,
                  const float* __restrict__ norm_w, float norm_eps, const float* __restrict__ inv_freq,
                  uint16_t* __restrict__ pages, int64_t n_slots) {
    constexpr int C = D / 32;
    __shared__ float s_rope[8][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp;
    if (t >= n_rows) return;
    // everything the token needs is asked for at once; whether it is to be stored is known later
    const int live = *n_live;
    const int64_t to = slot[t];
    const int ch = lane * C;
    const uint16_t* src = x + static_cast<size_t>(t) * D + ch;
    const bool pair = inv_freq && 2 * lane < d_rope;
    const int32_t at = inv_freq ? pos[t] : 0;
    const float fr = pair ? __ldg(inv_freq + lane) : 0.0f;
    uint32_t w[C / 2];
    if constexpr (C >= 8) {
#pragma unroll
        for (int i = 0; i < C / 8; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = __ldg(reinterpret_cast<const uint4*>(src) + i);
    } else {
        *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(src));
    }
    if (t >= live || to < 0 || to >= n_slots) return;
    uint16_t* dst = pages + static_cast<size_t>(to) * D + ch;
    if (norm_w || inv_freq) {
        CosSin cs = {1.0, 0.0};
        if (pair) cs = rope_cos_sin(at, fr);
        float y[C];
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            y[2 * i] = __uint_as_float(w[i] << 16);
            y[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        if (norm_w) {
            float sq[C];
#pragma unroll
            for (int i = 0; i < C; ++i) sq[i] = __fmul_rn(y[i], y[i]);
#pragma unroll
            for (int o = 1; o < C; o <<= 1)
#pragma unroll
                for (int i = 0; i < C; i += 2 * o) sq[i] = __fadd_rn(sq[i], sq[i + o]);
            float s = sq[0];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
            const float r = __fsqrt_rn(__fadd_rn(__fdiv_rn(s, static_cast<float>(D)), norm_eps));
#pragma unroll
            for (int i = 0; i < C; i += 4) {
                const float4 nw = __ldg(reinterpret_cast<const float4*>(norm_w + ch + i));
                y[i] = __fmul_rn(__fdiv_rn(y[i], r), nw.x);
                y[i + 1] = __fmul_rn(__fdiv_rn(y[i + 1], r), nw.y);
                y[i + 2] = __fmul_rn(__fdiv_rn(y[i + 2], r), nw.z);
                y[i + 3] = __fmul_rn(__fdiv_rn(y[i + 3], r), nw.w);
            }
        }
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
        const int dn = D - d_rope;
        if (inv_freq) {
            if (ch >= dn)
#pragma unroll
                for (int i = 0; i < C; ++i) s_rope[warp][ch - dn + i] = y[i];
            __syncwarp();
            if (pair) {
                const float2 ab = *reinterpret_cast<const float2*>(&s_rope[warp][2 * lane]);
                const uint32_t r = rotate_to_bf16(ab.x, ab.y, cs);
                *reinterpret_cast<uint32_t*>(pages + static_cast<size_t>(to) * D + dn + 2 * lane) = r;
            }
            if (ch >= dn) return;
        }
    }
    if constexpr (C >= 8) {
#pragma unroll
        for (int i = 0; i < C / 8; ++i) *(reinterpret_cast<uint4*>(dst) + i) = *reinterpret_cast<uint4*>(w + 4 * i);
    } else {
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(w);
    }
}

// ---------------------------------------------------------------- entry compressors
// One work item per new entry, and one per request for a step that completes
// no block of it.  The sums run over the tokens in ascending order, as the C
// ABI fixes them; the maximum has no order, nor has the computing of the terms.
// The tail is read and written in place by the same thread (m = 4) or the same
// CTA with a barrier between (m = 128), channel by channel, so that nothing
// else has to be waited for.  Bytes: 4 d a token in.
struct CompArgs {
    const uint16_t* x;
    const uint16_t* gate;
    int64_t n_tok;
    const int32_t *tok_start, *ctx;
    int B;
    const float* bias;
    const int32_t *ent_start, *ent_req, *ent_pos;
    const int64_t* ent_slot;
    int64_t max_ent;
    uint16_t *tail_x, *tail_gate;
    int d_rope, g;
    uint8_t* codes;
    float* scales;
    uint16_t* rope;
    int64_t n_slots;
    const float* norm_w;
    float norm_eps;
    const float* inv_freq;
};

__device__ __forceinline__ float2 bf2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// What an item is: an entry (of request b, tokens e M .. e M + M - 1), or a
// request whose step completes no block (entry = false).
struct CompItem {
    bool entry, tail;           // pool the entry; write the request's new tail (after reading the old one)
    int b;
    int64_t e, ctx, q0, end;    // entry; tokens [ctx, end) are the step's, token t at row q0 + t - ctx of x
};

template <int M>
__device__ __forceinline__ CompItem comp_item(const CompArgs& a, int64_t it) {
    CompItem c = {};
    const int64_t n_ent = min(static_cast<int64_t>(a.ent_start[a.B]), a.max_ent);
    const bool entry = it < n_ent;
    c.b = -1;
    if (entry) c.b = a.ent_req[it];
    else if (it >= a.max_ent && it < a.max_ent + a.B) c.b = static_cast<int>(it - a.max_ent);
    if (c.b < 0 || c.b >= a.B) { c.b = -1; return c; }
    c.ctx = max(a.ctx[c.b], 0);
    c.q0 = a.tok_start[c.b];
    c.end = c.ctx + max(min(static_cast<int64_t>(a.tok_start[c.b + 1]), a.n_tok) - c.q0, static_cast<int64_t>(0));
    if (entry) {
        c.e = a.ent_pos[it];
        c.entry = c.e >= c.ctx / M && (c.e + 1) * M <= c.end;
        c.tail = c.entry && c.e == c.ctx / M;
    } else {
        c.tail = c.end > c.ctx && c.ctx / M == c.end / M;       // no block of b completes
    }
    return c;
}

// m = 128: few entries complete per step (16K tokens are 120), so an item is
// spread over a cluster of d / 64 CTAs of 64 channels each, and inside a CTA
// over the tokens: warp w takes tokens w, w + 8, ... (16 of them, every load of
// gate and x in flight at once), e_i and x_i go through shared memory, and one
// thread per channel adds e_i and e_i x_i up in order.  One thread per two
// channels for all 128 tokens (the form of m = 4) took 40 us for 16K tokens of d
// = 512, a round trip to DRAM for every batch of loads; this takes 24.7 us (1.4
// TB/s), bound by issue (the exponentials) and the ordered sums, for which one warp
// pair of eight is at work.  x as stored in shared memory and 64 registers let four
// CTAs share an SM (e_i x_i there and 80 registers: three, 30.3 us).  With RMSNorm
// the CTAs' sums of squares meet through distributed shared memory, in the C ABI's
// tree.
template <int D>
__global__ void __cluster_dims__(D / 64, 1, 1) __launch_bounds__(256, 4)
page_compress128_kernel(CompArgs a) {
    constexpr int M = 128, G = D / 64, TW = M / 8;
    extern __shared__ float terms[];            // [M][64] e_i, then [M][64] x_i as stored
    uint16_t* const xs = reinterpret_cast<uint16_t*>(terms + M * 64);
    __shared__ float s_max[8][64];
    __shared__ float s_sum[2], s_all[G];
    __shared__ CosSin s_cs[32];                 // of the entry's position, in the CTA that holds the RoPE dims
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = blockIdx.x % G;
    const int64_t it = blockIdx.x / G;
    const CompItem c = comp_item<M>(a, it);     // the same in every CTA of the cluster
    if (!c.entry && !c.tail) return;
    // a CTA's shared memory may be written by another once it is known to have started; waited for where that is
    const bool meet = c.entry && a.norm_w;
    if (meet) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int ch0 = grp * 64, ch = ch0 + 2 * lane;
    if (c.entry) {
        const int64_t t0 = c.e * M;             // token i is in the tail while t0 + i < ctx
        const size_t toff = static_cast<size_t>(c.b) * M * D + ch;
        uint32_t gz[TW], xv[TW];
#pragma unroll
        for (int j = 0; j < TW; ++j) {
            const int i = warp + 8 * j;
            const bool old = t0 + i < c.ctx;
            const size_t off = old ? toff + static_cast<size_t>(i) * D : static_cast<size_t>(c.q0 + t0 + i - c.ctx) * D + ch;
            gz[j] = *reinterpret_cast<const uint32_t*>((old ? a.tail_gate : a.gate) + off);
            xv[j] = *reinterpret_cast<const uint32_t*>((old ? a.tail_x : a.x) + off);
        }
#pragma unroll
        for (int j = 0; j < TW; ++j) *reinterpret_cast<uint32_t*>(xs + (warp + 8 * j) * 64 + 2 * lane) = xv[j];
        float2 z[TW];
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < TW; ++j) {
            const float2 bv = __ldg(reinterpret_cast<const float2*>(a.bias + static_cast<size_t>(warp + 8 * j) * D + ch));
            const float2 gv = bf2(gz[j]);
            z[j] = make_float2(__fadd_rn(gv.x, bv.x), __fadd_rn(gv.y, bv.y));
            m0 = fmaxf(m0, z[j].x);
            m1 = fmaxf(m1, z[j].y);
        }
        *reinterpret_cast<float2*>(&s_max[warp][2 * lane]) = make_float2(m0, m1);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float2 o = *reinterpret_cast<const float2*>(&s_max[w][2 * lane]);
            m0 = fmaxf(m0, o.x);
            m1 = fmaxf(m1, o.y);
        }
#pragma unroll
        for (int j = 0; j < TW; ++j) {
            const float e0 = cw_exp_neg(__fsub_rn(z[j].x, m0)), e1 = cw_exp_neg(__fsub_rn(z[j].y, m1));
            *reinterpret_cast<float2*>(&terms[(warp + 8 * j) * 64 + 2 * lane]) = make_float2(e0, e1);
        }
        __syncthreads();                        // (the tail rows have been read, too)
        float y = 0.0f;
        if (warp == 2 && a.inv_freq && lane < a.d_rope / 2 && grp == G - 1)      // (beside the sums)
            s_cs[lane] = rope_cos_sin(t0, __ldg(a.inv_freq + lane));
        if (tid < 64) {
            float S = 0.0f, N = 0.0f;
#pragma unroll 16
            for (int i = 0; i < M; ++i) {
                const float e = terms[i * 64 + tid];
                S = __fadd_rn(S, e);
                N = __fadd_rn(N, __fmul_rn(e, __uint_as_float(static_cast<uint32_t>(xs[i * 64 + tid]) << 16)));
            }
            y = __fdiv_rn(N, S);
        }
        if (meet) {                             // uniform over the cluster
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
            if (tid < 64) {
                float s = __fmul_rn(y, y);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
                if (lane == 0) s_sum[warp] = s;
            }
            __syncthreads();
            if (tid < G) {
                // this CTA's sum into every CTA of the cluster
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at)
                             : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&s_all[grp]))), "r"(tid));
                asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(at), "f"(__fadd_rn(s_sum[0], s_sum[1])) : "memory");
            }
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            float s;
            if constexpr (G == 8)
                s = __fadd_rn(__fadd_rn(__fadd_rn(s_all[0], s_all[1]), __fadd_rn(s_all[2], s_all[3])),
                              __fadd_rn(__fadd_rn(s_all[4], s_all[5]), __fadd_rn(s_all[6], s_all[7])));
            else
                s = __fadd_rn(s_all[0], s_all[1]);
            const float r = __fsqrt_rn(__fadd_rn(__fdiv_rn(s, static_cast<float>(D)), a.norm_eps));
            if (tid < 64) y = __fmul_rn(__fdiv_rn(y, r), __ldg(a.norm_w + ch0 + tid));
        }
        // storage: thread = channel; FP8 groups of one warp (g = 32) or both (g = 64), or RoPE dims
        const int dn = D - a.d_rope, my = ch0 + tid;
        const int64_t to = a.ent_slot[it];
        float amax = fabsf(y);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (tid < 64 && lane == 0) s_max[0][warp] = amax;
        __syncthreads();
        if (a.g == 64) amax = fmaxf(s_max[0][0], s_max[0][1]);
        if (tid < 64 && to >= 0 && to < a.n_slots) {
            const float other = __shfl_xor_sync(0xffffffffu, y, 1);      // the pair's other channel
            if (my < dn) {
                const float scale = __fdiv_rn(amax, 448.0f);
                if ((tid & 1) == 0)
                    *reinterpret_cast<uint16_t*>(a.codes + to * dn + my) =
                        amax != 0.0f ? f32x2_to_e4m3x2(__fdiv_rn(y, scale), __fdiv_rn(other, scale)) : 0;
                if (my % a.g == 0) a.scales[to * (dn / a.g) + my / a.g] = scale;
            } else if ((tid & 1) == 0) {
                uint32_t w;
                if (a.inv_freq) {
                    w = rotate_to_bf16(y, other, s_cs[(my - dn) / 2]);
                } else {
                    __nv_bfloat162 h = __floats2bfloat162_rn(y, other);
                    w = *reinterpret_cast<uint32_t*>(&h);
                }
                *reinterpret_cast<uint32_t*>(a.rope + to * a.d_rope + (my - dn)) = w;
            }
        }
    }
    if (c.tail) {
        const int64_t t1 = max(c.ctx, c.end / M * M);
        const int n = static_cast<int>(c.end - t1);              // < M
        const size_t from = static_cast<size_t>(c.q0 + t1 - c.ctx) * D + ch;
        const size_t to = (static_cast<size_t>(c.b) * M + static_cast<size_t>(t1 % M)) * D + ch;
#pragma unroll 8
        for (int i = warp; i < n; i += 8) {
            const uint32_t xw = __ldg(reinterpret_cast<const uint32_t*>(a.x + from + static_cast<size_t>(i) * D));
            const uint32_t gw = __ldg(reinterpret_cast<const uint32_t*>(a.gate + from + static_cast<size_t>(i) * D));
            *reinterpret_cast<uint32_t*>(a.tail_x + to + static_cast<size_t>(i) * D) = xw;
            *reinterpret_cast<uint32_t*>(a.tail_gate + to + static_cast<size_t>(i) * D) = gw;
        }
    }
}

// m = 4: many entries, so a thread owns 2 channels of an entry (D / 2 threads),
// its four tokens' loads in flight at once.
template <int M, int D>
__global__ void __launch_bounds__(256)
page_compress_kernel(CompArgs a) {
    constexpr int TPE = D / 2;              // threads per entry
    constexpr int IPB = 256 / TPE;          // items per block
    __shared__ float s_part[8];
    const int ch = (threadIdx.x % TPE) * 2;
    const int64_t it = static_cast<int64_t>(blockIdx.x) * IPB + threadIdx.x / TPE;
    const CompItem c = comp_item<M>(a, it);
    // every thread of the block stays for the norm's barriers
    if (__syncthreads_or(c.entry)) {
        const int64_t t0 = c.e * M;
        const size_t toff = static_cast<size_t>(max(c.b, 0)) * M * D + ch;
        uint32_t gz[M], xv[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            gz[i] = xv[i] = 0;
            if (c.entry) {
                const bool old = t0 + i < c.ctx;
                const size_t off = old ? toff + static_cast<size_t>(i) * D : static_cast<size_t>(c.q0 + t0 + i - c.ctx) * D + ch;
                gz[i] = *reinterpret_cast<const uint32_t*>((old ? a.tail_gate : a.gate) + off);
                xv[i] = *reinterpret_cast<const uint32_t*>((old ? a.tail_x : a.x) + off);
            }
        }
        float2 z[M];
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float2 gv = bf2(gz[i]), bv = __ldg(reinterpret_cast<const float2*>(a.bias + ch + static_cast<size_t>(i) * D));
            z[i] = make_float2(__fadd_rn(gv.x, bv.x), __fadd_rn(gv.y, bv.y));
            m0 = fmaxf(m0, z[i].x);
            m1 = fmaxf(m1, z[i].y);
        }
        float S0 = 0.0f, S1 = 0.0f, N0 = 0.0f, N1 = 0.0f;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float2 v = bf2(xv[i]);
            const float e0 = cw_exp_neg(__fsub_rn(z[i].x, m0)), e1 = cw_exp_neg(__fsub_rn(z[i].y, m1));
            S0 = __fadd_rn(S0, e0);
            S1 = __fadd_rn(S1, e1);
            N0 = __fadd_rn(N0, __fmul_rn(e0, v.x));
            N1 = __fadd_rn(N1, __fmul_rn(e1, v.y));
        }
        float y0 = __fdiv_rn(N0, S0), y1 = __fdiv_rn(N1, S1);
        if (a.norm_w) {                     // uniform over the grid
            float s = __fadd_rn(__fmul_rn(y0, y0), __fmul_rn(y1, y1));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
            const int wv = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) s_part[wv] = s;
            __syncthreads();
            if (D == 512) {
                s = __fadd_rn(__fadd_rn(__fadd_rn(s_part[0], s_part[1]), __fadd_rn(s_part[2], s_part[3])),
                              __fadd_rn(__fadd_rn(s_part[4], s_part[5]), __fadd_rn(s_part[6], s_part[7])));
            } else {
                s = __fadd_rn(s_part[wv & ~1], s_part[wv | 1]);
            }
            const float r = __fsqrt_rn(__fadd_rn(__fdiv_rn(s, static_cast<float>(D)), a.norm_eps));
            const float2 nw = __ldg(reinterpret_cast<const float2*>(a.norm_w + ch));
            y0 = __fmul_rn(__fdiv_rn(y0, r), nw.x);
            y1 = __fmul_rn(__fdiv_rn(y1, r), nw.y);
        }
        const int dn = D - a.d_rope;
        float amax = fmaxf(fabsf(y0), fabsf(y1));
        for (int o = 1; o < a.g / 2; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int64_t to = c.entry ? a.ent_slot[it] : -1;
        if (to >= 0 && to < a.n_slots) {
            if (ch < dn) {
                const float scale = __fdiv_rn(amax, 448.0f);
                const uint16_t w = amax != 0.0f ? f32x2_to_e4m3x2(__fdiv_rn(y0, scale), __fdiv_rn(y1, scale)) : 0;
                *reinterpret_cast<uint16_t*>(a.codes + to * dn + ch) = w;
                if (ch % a.g == 0) a.scales[to * (dn / a.g) + ch / a.g] = scale;
            } else {
                uint32_t w;
                if (a.inv_freq) {
                    w = rotate_to_bf16(y0, y1, rope_cos_sin(t0, __ldg(a.inv_freq + (ch - dn) / 2)));
                } else {
                    __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
                    w = *reinterpret_cast<uint32_t*>(&h);
                }
                *reinterpret_cast<uint32_t*>(a.rope + to * a.d_rope + (ch - dn)) = w;
            }
        }
    }
    if (c.tail) {
        const int64_t t1 = max(c.ctx, c.end / M * M);
        const int n = static_cast<int>(c.end - t1);              // < M
        const size_t from = static_cast<size_t>(c.q0 + t1 - c.ctx) * D + ch;
        const size_t to = (static_cast<size_t>(c.b) * M + static_cast<size_t>(t1 % M)) * D + ch;
#pragma unroll
        for (int i = 0; i < M - 1; ++i)
            if (i < n) {
                *reinterpret_cast<uint32_t*>(a.tail_x + to + static_cast<size_t>(i) * D) =
                    __ldg(reinterpret_cast<const uint32_t*>(a.x + from + static_cast<size_t>(i) * D));
                *reinterpret_cast<uint32_t*>(a.tail_gate + to + static_cast<size_t>(i) * D) =
                    __ldg(reinterpret_cast<const uint32_t*>(a.gate + from + static_cast<size_t>(i) * D));
            }
    }
}

}  // namespace

int page_plan_launch(const int32_t* ctx, const int32_t* nnew, int B, int m, int P, int32_t* table, int width,
                     const int32_t* free_pages, const int32_t* free_count, int free_cap, int64_t max_rows,
                     int32_t* row_start, int32_t* row_req, int32_t* row_pos, int64_t* slot, int32_t* missing,
                     int32_t* free_left, cudaStream_t st) {
    PlanArgs a = {ctx, nnew, B, m, P, table, width, free_pages, free_count, free_cap, max_rows,
                  row_start, row_req, row_pos, slot, missing, free_left};
    const size_t smem = 2 * (static_cast<size_t>(B) + 1) * sizeof(int32_t);
    if (smem > 48 * 1024) {
        // (the largest B's, so that two threads' calls cannot lower it under each other's launch)
        const cudaError_t e = allow_smem<page_plan_kernel>(2 * (kPlanMaxB + 1) * static_cast<int>(sizeof(int32_t)));
        if (e != cudaSuccess) { set_last_cuda_error(static_cast<int>(e)); return HCA_ERR_CUDA; }
    }
    // a thread per row until every SM has a CTA; beyond that a CTA's scan costs more than further rows
    int64_t grid = ceil_div(max_rows > B ? max_rows : B + 1, kPlanThreads);
    if (grid > sm_count()) grid = sm_count();
    page_plan_kernel<<<static_cast<unsigned>(grid), kPlanThreads, smem, st>>>(a);
    HCA_CHECK_LAUNCH();
    return HCA_OK;
}

int page_store_launch(const uint16_t* x, int64_t n_rows, const int32_t* n_live, const int32_t* pos,
                      const int64_t* slot, const hca_kv_layout& L, const hca_entry_extras* ex, uint16_t* pages,
                      int64_t n_slots, cudaStream_t st) {
    const float* nw = ex ? ex->norm_w : nullptr;
    const float* fq = ex ? ex->inv_freq : nullptr;
    const float eps = ex ? ex->norm_eps : 0.0f;
    const unsigned grid = static_cast<unsigned>(ceil_div(n_rows, 8));
    if (L.d == 512)
        page_store_kernel<512><<<grid, 256, 0, st>>>(x, n_rows, n_live, pos, slot, L.d_rope, nw, eps, fq, pages, n_slots);
    else
        page_store_kernel<128><<<grid, 256, 0, st>>>(x, n_rows, n_live, pos, slot, L.d_rope, nw, eps, fq, pages, n_slots);
    HCA_CHECK_LAUNCH();
    return HCA_OK;
}

int page_compress_launch(int m, const uint16_t* x, const uint16_t* gate, int64_t n_tok, const int32_t* tok_start,
                         const int32_t* ctx, int B, const float* bias, const int32_t* ent_start, const int32_t* ent_req,
                         const int32_t* ent_pos, const int64_t* ent_slot, int64_t max_ent, uint16_t* tail_x,
                         uint16_t* tail_gate, const hca_kv_layout& L, const hca_kv_cache& pool, int64_t n_slots,
                         const hca_entry_extras* ex, cudaStream_t st) {
    CompArgs a = {x, gate, n_tok, tok_start, ctx, B, bias, ent_start, ent_req, ent_pos, ent_slot, max_ent, tail_x,
                  tail_gate, L.d_rope, L.scale_group, pool.codes, pool.scales, pool.rope, n_slots,
                  ex ? ex->norm_w : nullptr, ex ? ex->norm_eps : 0.0f, ex ? ex->inv_freq : nullptr};
    const int64_t items = max_ent + B;
    if (m == 4) {
        const unsigned grid = static_cast<unsigned>(ceil_div(items, 256 / (L.d / 2)));
        if (L.d == 512) page_compress_kernel<4, 512><<<grid, 256, 0, st>>>(a);
        else page_compress_kernel<4, 128><<<grid, 256, 0, st>>>(a);
    } else {
        constexpr int smem = 128 * 64 * (sizeof(float) + sizeof(uint16_t));
        auto kern = L.d == 512 ? page_compress128_kernel<512> : page_compress128_kernel<128>;
        const cudaError_t e = L.d == 512 ? allow_smem<page_compress128_kernel<512>>(smem) : allow_smem<page_compress128_kernel<128>>(smem);
        if (e != cudaSuccess) { set_last_cuda_error(static_cast<int>(e)); return HCA_ERR_CUDA; }
        kern<<<static_cast<unsigned>(items * (L.d / 64)), 256, smem, st>>>(a);
    }
    HCA_CHECK_LAUNCH();
    return HCA_OK;
}

}  // namespace hca
