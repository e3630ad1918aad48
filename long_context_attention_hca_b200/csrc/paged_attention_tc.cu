// paged_attention_tc.cu -- attention over paged caches on the sm_100a tensor
// cores, d = 512 (paged_attention.cu holds the attention rule, the kernel for d
// = 128 and the choice between the two).
//
// Two kernels.  The first writes each request's keys once, dequantised to fp16,
// into rows of the workspace (entries, then first tokens and window tokens in
// position order): every one of the request's tokens reads them, so that a page
// lookup, a dequantisation and a check for non-finite values per key is paid
// once and the second kernel is fed by TMA alone.
//
// The second runs on CTA pairs (cta_group::2): 128 rows (tokens x heads,
// flattened), 64 in each CTA, against tiles of 128 keys.
//   S = Q K^T    M = 128, N = 128, K = 512: each CTA holds its 64 rows of Q and
//                64 of the tile's keys
//   O += P V     M = 128, N = 2 x 256, K = 128: each CTA holds its 64 rows of P
//                and half of the dims of all 128 keys
// Why pairs: a CTA's O is 64 rows x 512 dims of fp32, half of its TMEM, and an
// M = 128 instruction over two CTAs keeps the tensor pipe at its full rate
// where M = 64 in one CTA runs at half; and each CTA reads half of B.
// TMEM (every row on two lanes: lane r holds the first half of an
// instruction's N, lane 64 + r the second): S in 2 buffers of 64 columns, O in
// 2 x 128 columns.
//
// Per 128-key tile and CTA: 48 instructions, 2048 clocks at the tensor pipe's
// rate; shared memory moves 128 KB for QK's operands (1024 clocks at 128 B), 96
// KB for PV's (768) and 128 KB in.  The K and the V part of a tile arrive as four
// 16 KB pieces each, every piece with its own slot, so that a piece of the next
// tile is on its way as soon as its predecessor is multiplied; one TMA a piece
// and one issuing thread for K and one for V (one thread for both, four copies a
// piece, spent 3.3K clocks a tile on issuing).  The softmax of tile i runs beside
// QK(i + 1).  Measured: 2.2K clocks a tile; 4096 tokens x 64 heads after 131072
// (entries of 128 tokens and the window) in 596 us alone, 1.05 PFLOP/s, 63% of a
// large library product's burst rate; what is missing is 6-11K clocks an item (its
// query conversion and first tile, its output) against some ten tiles.
//
// The pairs are persistent: the grid is one pair per two SMs, and a pair takes
// (tile, split of its keys) items from a counter until none is left, so that an
// item's query load, first keys and first QK run beside the item before (its
// last softmax, its output), and long and short items even out.  Splits are for
// steps of few rows: their partial outputs are joined by the combine kernel.
//
// Warps: 0-7 softmax and output (two groups of four, tiles in turn; a row of a
// tile is shared by two threads, one TMEM lane each), 8 K copies (in the first
// CTA also the item counter), 9 QK issue, 10 PV issue (the first CTA's only),
// 11-14 query rows to fp16, 15 V copies.  The online softmax is in base 2; O is rescaled only when
// a row's maximum grows by more than 2^8 (P <= 2^8 in fp16).  Every wait is
// bounded: one that gives up sets the device error word, and the pair, which
// still meets at the end, makes the rows NaN of every item that it was at and of
// those that no pair has taken (fail_items).
#include <cuda.h>

#include "paged_attention.cuh"

namespace hca {

__device__ int g_paged_device_error = 0;

namespace paged {
namespace tcp {

constexpr int D = 512;
constexpr int PAIR = 128;                    // rows of a CTA pair
constexpr int ROWS = 64;                     // rows of one CTA
constexpr int HALF = 64;                     // keys of a half tile (one CTA's K)
constexpr int NSLOT = 8, SLOT = 16384;       // K pieces 0-3, V pieces 4-7
constexpr int Q_OFF = 0;                     // 8 column blocks (64 dims) of 64 rows x 128 B
constexpr int P_OFF = 65536;                 // 2 buffers of 2 column blocks (64 keys) of 64 rows x 128 B
constexpr int R_OFF = P_OFF + 2 * 16384;
constexpr int CTRL_OFF = R_OFF + NSLOT * SLOT;
constexpr int SMEM = 232448;                 // all that a CTA may have: the rest is Ctrl's
constexpr int NSOFT = 8, NQ = 4, NTHREADS = (12 + NQ) * 32;
constexpr uint32_t S_COL = 0, O_COL = 128, TMEM_COLS = 512;
constexpr float GROW = 8.0f;                 // log2 units
constexpr int DR = 64, DN = D - DR;
constexpr long long WAIT_CLOCKS = 2000000000ll;   // about a second

struct Stage {
    uint16_t* rows;             // [bound][512] fp16
    uint8_t* flags;             // [bound]: 1 not visible, 2 non-finite
    int64_t per_req;            // rows of a request besides its new tokens
    int64_t bound;              // rows of the workspace
    float2* cs;                 // [n_rows][32]: cos / sin of each new token's RoPE pairs (with inv_freq)
    int* next;                  // the item counter
    int n_items;                // tiles x splits
    int pairs;                  // CTA pairs of the launch: their first items are 0 .. pairs - 1
};

// Request b's staged rows start at b per_req + row_start[b]: entries (padded
// with zeros to a multiple of 64), first tokens [0, f), tokens from w0 on, and
// 64 rows of zeros (a half tile may reach past its last key; V must be finite).
struct Region {
    int64_t base, w0;
    int n_e, n_e64, f;
};

__device__ __forceinline__ Region region(const Params& p, const Stage& s, int b, int64_t ctx, int n_new) {
    Region r;
    r.base = b * s.per_req + p.row_start[b];
    r.n_e = static_cast<int>(entries_before(p, ctx + n_new - 1));
    r.n_e64 = (r.n_e + 63) & ~63;
    r.w0 = ctx - (p.W - 1) > 0 ? ctx - (p.W - 1) : 0;
    r.f = static_cast<int>(p.n_first < r.w0 ? p.n_first : r.w0);
    return r;
}

// ------------------------------------------------------------------ staging
// A warp takes 8 consecutive staged rows: lane l < 8 finds where row l comes
// from (request, page, pool row), then the warp loads, converts and stores the
// rows, 16 dims a lane, four rows' loads in flight.  Bound: DRAM and L2 (604 or
// 1024 B in, 1 KB out a row); one row a warp took 18 us for 33K rows, most of it
// the chain search -> table -> row of every warp.  Few fat blocks also leave
// room on the SMs for the attention's CTAs to start beside them.  Now 33K rows
// take 15.8 us cold (54 MB in and out, 3.4 TB/s) and 5K rows 8 us, the chain of
// dependent loads (request, page number, row).
constexpr int STAGE_ROWS = 8;                   // a warp

__global__ void __launch_bounds__(256) stage_kernel(Params p, Stage s) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    pdl_trigger();                              // the attention's prologue may start
    if (w == 0 && lane == 0) *s.next = s.pairs;
    const int64_t g0 = w * STAGE_ROWS, stage_warps = (s.bound + STAGE_ROWS - 1) / STAGE_ROWS;
    if (w >= stage_warps) {
        // the new tokens' RoPE table, lane = pair: once here, where every row's conversion and output would go through
        // sincos again (7K clocks an item there, most of them instruction fetches)
        const int64_t n0 = (w - stage_warps) * STAGE_ROWS;
        if (p.inv_freq == nullptr || n0 >= p.n_rows || n0 >= p.row_start[p.B]) return;
        int b = last_at_most(p.B, [&](int c) { return p.row_start[c] <= n0; });
        for (int64_t n = n0; n < n0 + STAGE_ROWS && n < p.n_rows && n < p.row_start[p.B]; ++n) {
            while (b + 1 < p.B && p.row_start[b + 1] <= n) ++b;
            s.cs[n * 32 + lane] = rope_cs(p.inv_freq, lane, (p.ctx[b] > 0 ? p.ctx[b] : 0) + n - p.row_start[b]);
        }
        return;
    }
    // the request of row g0: the largest b with b per_req + row_start[b] <= g0
    const int b0 = last_at_most(p.B, [&](int c) { return c * s.per_req + p.row_start[c] <= g0; });
    int64_t from = -1;                          // pool row, -1: a row of zeros
    int kind = 0;                               // 0: nothing staged here, 1: entry, 2: token
    const int64_t g = g0 + lane;
    if (lane < STAGE_ROWS && g < s.bound) {
        int b = b0;
        while (b + 1 < p.B && (b + 1) * s.per_req + p.row_start[b + 1] <= g) ++b;
        const int64_t st = p.row_start[b];
        const int64_t en = p.row_start[b + 1] < p.n_rows ? p.row_start[b + 1] : p.n_rows;
        const int n_new = st < 0 || en < st ? 0 : static_cast<int>(en - st);
        if (n_new > 0) {
            const int64_t ctx = p.ctx[b] > 0 ? p.ctx[b] : 0;
            const Region r = region(p, s, b, ctx, n_new);
            int64_t i = g - r.base;
            if (i >= 0 && i < r.n_e64) {
                kind = 1;
                if (i < r.n_e) from = entry_row(p, b, static_cast<uint32_t>(i));
            } else if (i >= r.n_e64) {
                i -= r.n_e64;
                const int64_t n_t = ctx + n_new - r.w0;
                if (i < r.f + n_t + HALF) {
                    kind = 2;
                    if (i < r.f + n_t) from = token_row(p, b, static_cast<uint32_t>(i < r.f ? i : r.w0 + (i - r.f)));
                }
            }
        }
    }
    const int d0 = lane * 16;
#pragma unroll 1
    for (int k0 = 0; k0 < STAGE_ROWS; k0 += 4) {
        int64_t row[4];
        int kd[4];
        uint4 c0[4], c1[4];
        float sc[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            row[k] = __shfl_sync(0xffffffffu, from, k0 + k);
            kd[k] = __shfl_sync(0xffffffffu, kind, k0 + k);
            c0[k] = c1[k] = make_uint4(0, 0, 0, 0);
            sc[k] = 0.0f;
            if (row[k] < 0) continue;
            if (kd[k] == 1 && d0 < DN) {
                c0[k] = __ldg(reinterpret_cast<const uint4*>(p.codes + row[k] * DN + d0));
                sc[k] = __ldg(p.scales + row[k] * (DN / 64) + d0 / 64);
            } else {
                const uint4* src = reinterpret_cast<const uint4*>(kd[k] == 1 ? p.rope + row[k] * DR + (d0 - DN) : p.tok + row[k] * D + d0);
                c0[k] = __ldg(src);
                c1[k] = __ldg(src + 1);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (kd[k] == 0) continue;
            uint32_t h[8];
            if (kd[k] == 1 && d0 < DN) {
                dequant16(c0[k], sc[k], h);
            } else {
                const uint32_t v[8] = {c0[k].x, c0[k].y, c0[k].z, c0[k].w, c1[k].x, c1[k].y, c1[k].z, c1[k].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = pack_half2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
            }
            const bool bad = __any_sync(0xffffffffu, any_bad(h));
            const uint32_t keep = bad ? 0u : 0xffffffffu;
            uint4* dst = reinterpret_cast<uint4*>(s.rows + (g0 + k0 + k) * D + d0);
            dst[0] = make_uint4(h[0] & keep, h[1] & keep, h[2] & keep, h[3] & keep);
            dst[1] = make_uint4(h[4] & keep, h[5] & keep, h[6] & keep, h[7] & keep);
            if (lane == 0) s.flags[g0 + k0 + k] = row[k] < 0 ? 1 : (bad ? 2 : 0);
        }
    }
}

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {     // the same address in the pair's first CTA
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
// Arrival at a barrier of either CTA.  What it announces (operands in this CTA's shared memory, TMEM that has been read)
// is ordered by the proxy and tcgen05 fences in front of it; a release at cluster scope would wait for every memory
// operation of the thread, 1-2K clocks each time.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
// ... and one that publishes this thread's plain stores to the other CTA
__device__ __forceinline__ void mbar_arrive_release(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
// staged rows into this CTA, 64-dim column blocks one after the other, the bytes counted at the barrier of the pair's
// first CTA
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int row, int block, uint32_t bar_first) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(0), "r"(row), "r"(block), "r"(bar_first) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 :: "l"(map), "r"(x), "r"(y), "r"(src) : "memory");
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// arrives at `bar` of both CTAs once this thread's MMAs so far have completed
__device__ __forceinline__ void commit2(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// pairs of floats in one register pair (two operations an instruction)
__device__ __forceinline__ uint64_t pair64(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
                   "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(a));
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 :: "r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                    "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                    "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}
// shared-memory matrix descriptor, 128-byte swizzle (sm_100 format)
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// instruction descriptor, kind::f16: fp16 A and B, fp32 accumulator
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
// byte offset of (row, 16-byte chunk c in 0..7) inside a column block of 128-byte rows (128-byte swizzle)
__device__ __forceinline__ uint32_t sw128(int row, int c) {
    return static_cast<uint32_t>((row >> 3) * 1024 + (row & 7) * 128 + ((c ^ (row & 7)) << 4));
}

// Bounded wait of a whole warp, the same answer for all its lanes.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    bool done = mbar_try(bar, parity);
    if (!__all_sync(0xffffffffu, done)) {
        const long long t0 = clock64();
        while (!done && !*abort_flag && clock64() - t0 < WAIT_CLOCKS) done = mbar_try(bar, parity);
        if (!__all_sync(0xffffffffu, done)) {
            *abort_flag = 1;
            atomicExch(&g_paged_device_error, 1);
            return false;
        }
    }
    return true;
}

// One item: a tile's rows and the key tiles [k0, k0 + n) of its split.
struct Item {
    Tile T;
    int index;                  // tile x splits + split; -1: no more items
    int k0, n;
    int h_e, h_f, n_half;       // half tiles of 64 staged rows: entries, first tokens, all
    int64_t ent0, tok0, win0;   // staged rows of the first entry, first token, first window token
    int64_t tok_row;            // row of the request's first new token
};

// A pair's items that may not be out yet: item j is drawn once j - 1 is posted, that is once all have taken j - 3, and
// the softmax warps take an item ahead of the output of the one before: j - 4 .. j at most.
constexpr int RECENT = 8;

struct Ctrl {
    uint64_t full[NSLOT], empty[NSLOT], s_full[2], s_free[2], p_full[2], pv_done[2], q_full, q_free, o_free;
    uint64_t item_full[2], item_free[2], drain;
    Item item[2];
    float mx[2][2][ROWS];       // [group][key half][row]: a tile's largest raw logit; at the end each thread's l
    float m[2][ROWS];           // [tile parity]: the running maximum (base 2) after the tile
    Item soft_item[2];          // the softmax warps' copy, by item parity
    int recent[RECENT];         // the first CTA's: the items with keys that it drew last, in turn (-1: none)
    uint32_t tmem;
    int abort_flag;
};
static_assert(CTRL_OFF + sizeof(Ctrl) <= SMEM, "shared memory");
// warps that take an item from the mailbox: softmax (one for all), QK, PV and the query warps of the first CTA;
// softmax, K and the query warps of the second; V of both
constexpr int TAKERS = 3 + NQ + 2 + NQ + 2;

__device__ __forceinline__ bool make_item(const Params& p, const Stage& s, int item, Item& I) {
    const int t = item / p.n_splits, split = item - t * p.n_splits;
    I.index = item;
    if (!make_tile(p, t, PAIR, I.T)) return false;
    const Region rg = region(p, s, I.T.b, I.T.ctx, I.T.n_new);
    I.h_e = (I.T.n_e + HALF - 1) / HALF;
    I.h_f = (I.T.n_f + HALF - 1) / HALF;
    I.n_half = I.h_e + I.h_f + (I.T.n_w + HALF - 1) / HALF;
    const int tiles = (I.n_half + 1) / 2;
    I.k0 = static_cast<int>(static_cast<int64_t>(tiles) * split / p.n_splits);
    I.n = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / p.n_splits) - I.k0;
    I.ent0 = rg.base;
    I.tok_row = p.row_start[I.T.b];
    I.tok0 = rg.base + rg.n_e64;
    I.win0 = I.tok0 + rg.f + (I.T.w_lo - rg.w0);
    return true;
}

// One thread: the four pieces of a key tile's K (slots 0-3, dims 128 j .., all rows from y) or V (slots 4-7, 32 keys
// each: rows y, y + 32 of the tile's first half, y2, y2 + 32 of its second; dims of column blocks from `block`).  u: key
// tiles before.  Waits for each slot, announces both CTAs' bytes (first CTA), copies.
__device__ __forceinline__ bool copy_pieces(Ctrl& c, int slot0, int u, bool first, uint32_t dst, const CUtensorMap* map, int y,
                                            int blocks, volatile int* abort_flag, int y2, int block) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t full = smem_u32(&c.full[slot0 + j]), empty = smem_u32(&c.empty[slot0 + j]);
        if (u > 0 && !mbar_try(empty, (u - 1) & 1)) {
            const long long t0 = clock64();
            while (!mbar_try(empty, (u - 1) & 1))
                if (*abort_flag || clock64() - t0 >= WAIT_CLOCKS) {
                    *abort_flag = 1;
                    atomicExch(&g_paged_device_error, 1);
                    return false;
                }
        }
        if (first) mbar_expect(full, 2 * SLOT);
        if (blocks == 2) tma_3d(dst + j * SLOT, map, y, 2 * j, in_first(full));
        else tma_3d(dst + j * SLOT, map, (j & 2 ? y2 : y) + (j & 1) * 32, block, in_first(full));
    }
    return true;
}

// After a wait has given up (both CTAs' writes are done): NaN for all rows of the items that the pair drew last, done or
// not, and of those left on the counter.  Whole warps, each an item at a time.
__device__ __forceinline__ void fail_items(const Params& p, const Stage& s, const int* recent) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();                                     // (the counter is set)
    for (bool own = warp < RECENT;; own = false) {
        int it = 0;
        if (own) {
            it = recent[warp];
            if (it < 0) continue;
        } else {
            if (lane == 0) it = atomicAdd(s.next, 1);
            it = __shfl_sync(0xffffffffu, it, 0);
            if (it >= s.n_items) break;
        }
        Item I;
        if (!make_item(p, s, it, I)) continue;
        if (p.n_splits > 1) {
            // (a weight of NaN: the combine makes the row NaN, whatever else it joins)
            float* ml = p.part_ml + static_cast<int64_t>(it) * 2 * PAIR;
            for (int r = lane; r < PAIR; r += 32) {
                ml[r] = 0.0f;
                ml[PAIR + r] = __int_as_float(0x7fc00000);
            }
        } else {
            uint4* row = reinterpret_cast<uint4*>(p.out + I.T.row0 * D);
            for (int i = lane; i < I.T.rows * (D / 8); i += 32) row[i] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        }
    }
}

// first staged row of a half tile (past the last: finite rows that no query sees)
__device__ __forceinline__ int64_t half_row(const Item& I, int h) {
    if (h < I.h_e) return I.ent0 + h * HALF;
    if (h < I.h_e + I.h_f) return I.tok0 + (h - I.h_e) * HALF;
    return h < I.n_half ? I.win0 + (h - I.h_e - I.h_f) * HALF : I.win0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
paged_tc_kernel(Params p, Stage s, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ CUtensorMap o_map, const __grid_constant__ CUtensorMap p_map) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl& c = *reinterpret_cast<Ctrl*>(smem + CTRL_OFF);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cta_rank();
    const uint32_t sbase = smem_u32(smem);
    volatile int* abort_flag = &c.abort_flag;

    if (tid == 0) {
        for (int i = 0; i < NSLOT; ++i) { mbar_init(smem_u32(&c.full[i]), 1); mbar_init(smem_u32(&c.empty[i]), 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c.s_full[i]), 1);
            mbar_init(smem_u32(&c.s_free[i]), NSOFT);   // the four warps of the tile's group, in both CTAs
            mbar_init(smem_u32(&c.p_full[i]), NSOFT);
            mbar_init(smem_u32(&c.pv_done[i]), 1);
            mbar_init(smem_u32(&c.item_full[i]), 1);
            mbar_init(smem_u32(&c.item_free[i]), TAKERS);
        }
        mbar_init(smem_u32(&c.q_full), 2 * NQ);
        mbar_init(smem_u32(&c.q_free), 1);
        mbar_init(smem_u32(&c.o_free), 2 * NSOFT);
        mbar_init(smem_u32(&c.drain), 2);               // both issuing threads
        for (int i = 0; i < RECENT; ++i) c.recent[i] = -1;
        c.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(&c.tmem)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    cluster_sync();                                 // barriers and TMEM of both CTAs are ready
    fence_after();
    const uint32_t tmem = c.tmem;
    // From here until a warp's own pdl_wait() the staging kernel may still be running.  It was launched plainly, so that
    // everything before it is complete: lengths and queries may be read, what it writes (staged rows, flags, RoPE table,
    // the item counter) not yet.  A pair's first item is its own number; later ones come from the counter.
    bool ok = true;
    const int rbase = rank * ROWS;                  // first row of this CTA in a tile

    // item k from the mailbox (false: no more); whole warps
    auto take_item = [&](int k, Item& I) -> bool {
        if (!wait_bar(smem_u32(&c.item_full[k & 1]), (k >> 1) & 1, abort_flag)) { ok = false; I.index = -1; return false; }
        asm volatile("fence.acq_rel.cluster;" ::: "memory");       // the words came from the first CTA
        I = c.item[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive_release(in_first(smem_u32(&c.item_free[k & 1])));
        return I.index >= 0;
    };

    if (warp == 8) {
        // ------------------------------------------------------------ K copies, items
        const bool leader = elect_one();
        // the next item with rows and keys, posted to both CTAs: where and how much is worked out once, here
        auto post_next = [&](int k, Item& J) {
            for (bool own = k == 0;; own = false) {
                int it = blockIdx.x >> 1;
                if (!own) {
                    if (k == 0) pdl_wait();          // (the counter is set)
                    if (lane == 0) it = atomicAdd(s.next, 1);
                    it = __shfl_sync(0xffffffffu, it, 0);
                }
                J.index = -1;
                if (it >= s.n_items) break;
                if (!make_item(p, s, it, J)) continue;
                if (J.n > 0) {
                    if (lane == 0) c.recent[k & (RECENT - 1)] = it;
                    break;
                }
                // no key tile left for this split: its rows' partials weigh nothing
                for (int r = lane; r < PAIR; r += 32) {
                    p.part_ml[static_cast<int64_t>(it) * 2 * PAIR + r] = -INFINITY;
                    p.part_ml[static_cast<int64_t>(it) * 2 * PAIR + PAIR + r] = 0.0f;
                }
            }
            if (k >= 2 && ok) ok = wait_bar(smem_u32(&c.item_free[k & 1]), ((k >> 1) & 1) ^ 1, abort_flag);
            if (!ok) return;
            if (lane == 0) c.item[k & 1] = J;
            __syncwarp();
            // lane w: word w into the second CTA
            constexpr int WORDS = sizeof(Item) / 4;
            static_assert(WORDS <= 32 && sizeof(Item) % 4 == 0, "one word a lane");
            if (lane < WORDS) {
                const uint32_t at = smem_u32(&c.item[k & 1]) + lane * 4;
                uint32_t far, w;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
                asm volatile("mapa.shared::cluster.u32 %0, %1, 1;" : "=r"(far) : "r"(at));
                asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(far), "r"(w) : "memory");
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
            }
            __syncwarp();
            if (lane < 2) {
                uint32_t bar;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&c.item_full[k & 1])), "r"(lane));
                mbar_arrive_release(bar);
            }
            __syncwarp();
        };
        Item I, J;
        int u = 0;                                   // key tiles so far: each uses every K slot once
        if (rank == 0) post_next(0, I); else take_item(0, I);
        pdl_wait();
        for (int k = 0; I.index >= 0 && ok; ++k) {
            for (int i = 0; i < I.n && ok; ++i, ++u) {
                const int y = static_cast<int>(half_row(I, 2 * (I.k0 + i) + rank));
                if (leader) ok = copy_pieces(c, 0, u, rank == 0, sbase + R_OFF, &k_map, y, 2, abort_flag, 0, 0);
                ok = __all_sync(0xffffffffu, ok);
                if (i == 0 && rank == 0 && ok) post_next(k + 1, J);      // behind the item's first keys
            }
            if (rank == 0) I = J; else take_item(k + 1, I);
        }
        // gave up: copies in flight land within microseconds, before this CTA's memory may go to another
        if (!ok) for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    } else if (warp == 15) {
        // ------------------------------------------------------------ V copies
        pdl_wait();
        const bool leader = elect_one();
        Item I;
        int u = 0;
        for (int k = 0; ok; ++k) {
            if (!take_item(k, I)) break;
            for (int i = 0; i < I.n && ok; ++i, ++u) {
                // keys 32 j .. of the tile: half tile j / 2, its rows 32 (j & 1) ..
                const int h = 2 * (I.k0 + i);
                if (leader)
                    ok = copy_pieces(c, 4, u, rank == 0, sbase + R_OFF + 4 * SLOT, &v_map, static_cast<int>(half_row(I, h)), 4,
                                     abort_flag, static_cast<int>(half_row(I, h + 1)), rank * 4);
                ok = __all_sync(0xffffffffu, ok);
            }
        }
        if (!ok) for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    } else if (warp == 9 && rank == 0) {
        // ------------------------------------------------------------ QK issue
        const bool leader = elect_one();
        constexpr uint32_t id = idesc_f16(128, 128, 0);
        const uint64_t qd = sdesc(sbase + Q_OFF, 16, 1024);
        int u = 0, uses[2] = {0, 0};                 // key tiles and uses of each S buffer so far
        Item I;
        for (int k = 0; ok; ++k) {
            if (!take_item(k, I)) break;
            ok = wait_bar(smem_u32(&c.q_full), k & 1, abort_flag);
            for (int i = 0; i < I.n && ok; ++i, ++u) {
                const int b = i & 1, use = (b ? uses[1] : uses[0]) + (i >> 1);
                if (use > 0) ok = wait_bar(smem_u32(&c.s_free[b]), (use - 1) & 1, abort_flag);     // S's last use has been read
                for (int j = 0; j < 4 && ok; ++j) {
                    const int sl = j;
                    ok = wait_bar(smem_u32(&c.full[sl]), u & 1, abort_flag);
                    if (!ok) break;
                    fence_after();
                    const uint64_t kd = sdesc(sbase + R_OFF + sl * SLOT, 16, 1024);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)   // 16 dims a step: column block kk / 4, 32 bytes a step inside it
                            mma2(tmem + S_COL + b * 64, qd + static_cast<uint32_t>(((2 * j + (kk >> 2)) * 8192 + (kk & 3) * 32) >> 4),
                                 kd + static_cast<uint32_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), id, (j > 0 || kk > 0) ? 1u : 0u);
                        commit2(smem_u32(&c.empty[sl]));
                        if (j == 3) commit2(smem_u32(&c.s_full[b]));
                        if (j == 3 && i == I.n - 1) commit2(smem_u32(&c.q_free));
                    }
                    __syncwarp();
                }
            }
            uses[0] += (I.n + 1) / 2;
            uses[1] += I.n / 2;
        }
        if (leader) commit2(smem_u32(&c.drain));
    } else if (warp == 10 && rank == 0) {
        // ------------------------------------------------------------ PV issue
        const bool leader = elect_one();
        constexpr uint32_t id = idesc_f16(128, 256, 1);
        const uint64_t pd = sdesc(sbase + P_OFF, 16, 1024);
        int u = 0, uses[2] = {0, 0};
        Item I;
        for (int k = 0; ok; ++k) {
            if (!take_item(k, I)) break;
            if (k > 0) ok = wait_bar(smem_u32(&c.o_free), (k - 1) & 1, abort_flag);               // O of the item before is out
            for (int i = 0; i < I.n && ok; ++i, ++u) {
                const int b = i & 1, use = (b ? uses[1] : uses[0]) + (i >> 1);
                ok = wait_bar(smem_u32(&c.p_full[b]), use & 1, abort_flag);
                for (int j = 0; j < 4 && ok; ++j) {
                    const int sl = 4 + j;
                    ok = wait_bar(smem_u32(&c.full[sl]), u & 1, abort_flag);
                    if (!ok) break;
                    fence_after();
                    // V: dims are contiguous (MN-major), 64-dim column blocks 4096 B apart, 8 keys 1024 B
                    const uint64_t vd = sdesc(sbase + R_OFF + sl * SLOT, 4096, 1024);
                    if (leader) {
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {
                            const int kk = 2 * j + k2;   // 16 keys a step
                            const uint64_t a = pd + static_cast<uint32_t>((b * 16384 + (kk >> 2) * 8192 + (kk & 3) * 32) >> 4);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                mma2(tmem + O_COL + h * 128, a, vd + static_cast<uint32_t>((h * 8192 + k2 * 2048) >> 4), id,
                                     (i > 0 || kk > 0) ? 1u : 0u);
                        }
                        commit2(smem_u32(&c.empty[sl]));
                        if (j == 3) commit2(smem_u32(&c.pv_done[b]));
                    }
                    __syncwarp();
                }
            }
            uses[0] += (I.n + 1) / 2;
            uses[1] += I.n / 2;
        }
        if (leader) commit2(smem_u32(&c.drain));
    } else if (warp >= 11) {
        // ------------------------------------------------------------ query rows
        // 16 rows a warp, copied as stored (bf16) to where the fp16 values go, then converted in place, each lane what
        // it copied itself; RMSNorm and RoPE in fp32.  Rolled loops: an unrolled form of this (8 rows in registers)
        // took 14K clocks an item, most of them waiting for instructions.
        const int w0 = (warp - 11) * (ROWS / NQ);
        uint8_t* const my = smem + Q_OFF + (lane >> 2) * 8192;       // dims 16 lane .. + 15: two chunks of column block lane / 4
        const int ch = (lane & 3) * 2;
        const uint32_t q_first = in_first(smem_u32(&c.q_full));
        // (in registers: with all of the SM's memory shared there is no L1 to speak of, and a load of the weights per
        // row cost 0.7K clocks each)
        uint64_t nw[8];
        if (p.q_norm_w)
#pragma unroll
            for (int i = 0; i < 8; ++i)              // (volatile: not to be loaded again in the loop)
                asm volatile("ld.global.nc.b64 %0, [%1];" : "=l"(nw[i]) : "l"(p.q_norm_w + lane * 16 + 2 * i));
        Item I;
        for (int k = 0; ok; ++k) {
            if (!take_item(k, I)) break;
            const Tile& T = I.T;
            const int rows = min(max(T.rows - rbase, 0), ROWS);
            const uint16_t* src = p.q + (T.row0 + rbase + w0) * D + lane * 16;
            // the rows on their way to L2 while the item before still uses the buffer
            if (k > 0) {
                if (lane < 8)
#pragma unroll 1
                    for (int r = 0; r < ROWS / NQ; ++r)
                        if (w0 + r < rows) asm volatile("prefetch.global.L2 [%0];" :: "l"(src + static_cast<int64_t>(r) * D + lane * 48));
                ok = wait_bar(smem_u32(&c.q_free), (k - 1) & 1, abort_flag);
            }
#pragma unroll 4
            for (int r = 0; r < ROWS / NQ; ++r) {
                const uint32_t d0 = smem_u32(my + sw128(w0 + r, ch)), d1 = smem_u32(my + sw128(w0 + r, ch + 1));
                if (w0 + r < rows) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(d0), "l"(src + static_cast<int64_t>(r) * D) : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(d1), "l"(src + static_cast<int64_t>(r) * D + 8) : "memory");
                } else {
                    *reinterpret_cast<uint4*>(my + sw128(w0 + r, ch)) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(my + sw128(w0 + r, ch + 1)) = make_uint4(0, 0, 0, 0);
                }
            }
            if (k == 0 && p.inv_freq) pdl_wait();    // (the RoPE table)
            asm volatile("cp.async.wait_all;" ::: "memory");
            // token of a row, counted up: a division per item instead of one per row
            int tok = (T.r0 + rbase + w0) / p.H, head = (T.r0 + rbase + w0) - tok * p.H, cs_tok = tok;
            float2 cs[8];                            // of this lane's pairs (lanes that hold RoPE dims), at the row's position
            auto load_cs = [&](int tk) {
                if (lane * 16 >= DN && tk < T.n_new) {
                    const float4* from = reinterpret_cast<const float4*>(s.cs + (I.tok_row + tk) * 32 + (lane * 16 - DN) / 2);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 c2 = from[i];
                        cs[2 * i] = make_float2(c2.x, c2.y);
                        cs[2 * i + 1] = make_float2(c2.z, c2.w);
                    }
                }
            };
            if (p.inv_freq) load_cs(tok);
            // one warp issues an instruction every two or three clocks here, so the arithmetic is on pairs (f32x2)
#pragma unroll 1
            for (int r = w0; r < w0 + ROWS / NQ && r < rows; ++r) {
                uint4* const c0 = reinterpret_cast<uint4*>(my + sw128(r, ch));
                uint4* const c1 = reinterpret_cast<uint4*>(my + sw128(r, ch + 1));
                const uint4 a0 = *c0, a1 = *c1;
                const uint32_t v[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
                uint64_t f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = pair64(v[i] << 16, v[i] & 0xFFFF0000u);
                if (p.q_norm_w) {
                    uint64_t s0 = 0, s1 = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s0 = fma2(f[i], f[i], s0);
                        s1 = fma2(f[i + 4], f[i + 4], s1);
                    }
                    const float2 sa = unpair(s0), sb = unpair(s1);
                    float ss = (sa.x + sa.y) + (sb.x + sb.y);
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float rr = rsqrtf(ss * (1.0f / D) + p.norm_eps);
                    const uint64_t r2 = pair64(__float_as_uint(rr), __float_as_uint(rr));
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = mul2(mul2(f[i], r2), nw[i]);
                }
                if (p.inv_freq) {
                    if (tok != cs_tok) {
                        cs_tok = tok;
                        load_cs(tok);
                    }
                    if (lane * 16 >= DN)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 ab = unpair(f[i]);
                            f[i] = pair64(__float_as_uint(ab.x * cs[i].x - ab.y * cs[i].y), __float_as_uint(ab.x * cs[i].y + ab.y * cs[i].x));
                        }
                    if (++head == p.H) { head = 0; ++tok; }
                }
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) { const float2 ab = unpair(f[i]); h[i] = pack_half2(ab.x, ab.y); }
                *c0 = make_uint4(h[0], h[1], h[2], h[3]);
                *c1 = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(q_first);
        }
    } else if (warp < NSOFT) {
        // ------------------------------------------------------------ softmax
        // Group g (4 warps) takes the tiles of parity g, so that a tile's
        // exponentials and its P stores run beside the next tile's; only the
        // running maximum passes from tile to tile.
        const int qd = warp & 3, g = warp >> 2;
        const int hk = qd >> 1;                      // which half of the tile's keys
        const int r = (qd & 1) * 32 + lane;          // row of this CTA
        const uint32_t lb = tmem + (static_cast<uint32_t>(qd * 32) << 16);
        int uses[2] = {0, 0};                        // of each parity's buffers, so far
        // one warp takes an item for all eight (they meet at barriers: all go on, or none), the next one ahead of the
        // output of this one: the fence in there would wait for the output's stores
        auto take_for_all = [&](int k) {
            if (warp == 0) {
                Item J;
                take_item(k, J);
                if (lane == 0) c.soft_item[k & 1] = J;
            }
        };
        take_for_all(0);
        bar_sync(5, NSOFT * 32);
        pdl_wait();                                  // (the flags of the staged rows)
        for (int kk = 0;; ++kk) {
            const Item& I = c.soft_item[kk & 1];     // (read where needed: its fields in registers would spill others)
            const int it = I.index;
            if (it < 0) break;
            const Tile& T = I.T;
            const RowKeys rk = row_keys(p, T, T.ctx + (T.r0 + min(rbase + r, T.rows - 1)) / p.H);
            float m_l = -INFINITY, l_run = 0.0f;     // this thread's share of l, and the maximum it is relative to
            uint32_t fl[2];
            auto flags_of = [&](int i) {
                const uint8_t* f = s.flags + (i < I.n ? half_row(I, 2 * (I.k0 + i) + hk) : I.ent0) + lane;
                fl[0] = f[0];
                fl[1] = f[32];
            };
            flags_of(g);
            for (int i = g; i < I.n; i += 2) {
                const int h = 2 * (I.k0 + i) + hk, use = uses[g] + (i >> 1);
                if (ok) ok = wait_bar(smem_u32(&c.s_full[g]), use & 1, abort_flag);
                fence_after();
                float v[64];
                {
                    uint32_t sr[32];
                    tmem_ld32(lb + S_COL + g * 64, sr);
                    uint32_t s2[32];
                    tmem_ld32(lb + S_COL + g * 64 + 32, s2);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) { v[j] = __uint_as_float(sr[j]); v[32 + j] = __uint_as_float(s2[j]); }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(in_first(smem_u32(&c.s_free[g])));            // S may be overwritten
                // keys that this row sees among the half tile's 64, as bits
                auto below = [](int k) -> unsigned { return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u); };
                unsigned vis[2], bad = 0;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const unsigned gone = __ballot_sync(0xffffffffu, fl[z] & 1u), nf = __ballot_sync(0xffffffffu, fl[z] & 2u);
                    if (h < I.h_e) {
                        vis[z] = below(rk.e_lim - (h * HALF + z * 32));
                    } else if (h < I.h_e + I.h_f) {
                        vis[z] = below(T.n_f - ((h - I.h_e) * HALF + z * 32));
                    } else {
                        const int k0 = T.n_e + T.n_f + (h - I.h_e - I.h_f) * HALF + z * 32;   // slot of the first of these keys
                        vis[z] = h < I.n_half ? below(rk.w_hi + 1 - k0) & (~below(rk.w_from - k0) | below(rk.f_to - k0)) : 0u;
                    }
                    vis[z] &= ~gone;
                    bad |= vis[z] & nf;
                }
                flags_of(i + 2);
                if (!__all_sync(0xffffffffu, (vis[0] & vis[1]) == 0xffffffffu))
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] = ((vis[j >> 5] >> (j & 31)) & 1u) ? v[j] : -INFINITY;
                float t[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) t[j] = fmaxf(fmaxf(v[j], v[j + 16]), fmaxf(v[j + 32], v[j + 48]));
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                    for (int j = 0; j < w; ++j) t[j] = fmaxf(t[j], t[j + w]);
                c.mx[g][hk][r] = t[0];
                bar_sync(1 + g, 128);
                // the scale is positive: the largest raw logit scaled is the largest logit
                const float m_tile = fmaxf(t[0], c.mx[g][hk ^ 1][r]) * p.scale_log2;
                // the maximum after tile i - 1, from the other group
                // (a barrier of this group either way, before c.mx is written again)
                if (i > 0) bar_sync(3 + (i & 1), 256); else bar_sync(1 + g, 128);
                const float m_old = i > 0 ? c.m[(i - 1) & 1][r] : -INFINITY;
                bool resc = false;
                float m_new = m_old;
                if (m_old == -INFINITY) {
                    m_new = m_tile;                  // nothing seen before: O and l are zero
                } else if (m_tile > m_old + GROW) {
                    resc = true;
                    m_new = m_tile;
                }
                if (hk == 0) c.m[i & 1][r] = m_new;
                if (i + 1 < I.n) asm volatile("bar.arrive %0, 256;" :: "r"(3 + ((i + 1) & 1)) : "memory");
                const float ref = m_new == -INFINITY ? 0.0f : m_new;
                uint32_t pk[32];
                // l sums the probabilities in fp32 as they are; PV uses them rounded to fp16, which weighs a key by at
                // most half a step (2^-11) more or less
                uint64_t ps[4] = {0, 0, 0, 0};
                const uint64_t sc2 = pair64(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
                const uint64_t rf2 = pair64(__float_as_uint(-ref), __float_as_uint(-ref));
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float2 x = unpair(fma2(pair64(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1])), sc2, rf2));
                    const float e0 = ex2(x.x), e1 = ex2(x.y);
                    pk[j] = pack_half2(e0, e1);
                    ps[j & 3] = add2(ps[j & 3], pair64(__float_as_uint(e0), __float_as_uint(e1)));
                }
                const float2 pt = unpair(add2(add2(ps[0], ps[1]), add2(ps[2], ps[3])));
                l_run = (m_l == -INFINITY ? l_run : l_run * ex2(m_l - m_new)) + (pt.x + pt.y);
                m_l = m_new;
                // a visible key that is not finite; or a query that is not, and all its logits so far -inf
                if (bad || (m_new == -INFINITY && (vis[0] | vis[1]))) l_run = __int_as_float(0x7fc00000);
                if (use > 0 && ok) ok = wait_bar(smem_u32(&c.pv_done[g]), (use - 1) & 1, abort_flag);   // P's buffer is free
                if (__any_sync(0xffffffffu, resc)) {
                    // O must hold still: PV(i - 1) complete (the barrier's phase before belongs to a PV that completed
                    // ahead of the one just waited for; PV(i) waits for this P)
                    if (ok) ok = wait_bar(smem_u32(&c.pv_done[g ^ 1]), (uses[g ^ 1] + ((i - 1) >> 1)) & 1, abort_flag);
                    fence_after();
                    const float alpha = resc ? ex2(m_old - m_new) : 1.0f;
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
                        uint32_t o[32];
                        const uint32_t a = lb + O_COL + q * 32;
                        tmem_ld32(a, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        tmem_st32(a, o);
                    }
                    tmem_wait_st();
                }
                uint8_t* pb = smem + P_OFF + g * 16384 + hk * 8192;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(pb + sw128(r, j)) = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
                fence_async();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(in_first(smem_u32(&c.p_full[g])));
            }
            take_for_all(kk + 1);
            const int rows = min(max(T.rows - rbase, 0), ROWS);
            const int rt = min(rbase + r, T.rows - 1);
            const int tok = (T.r0 + rt) / p.H;
            // ---- the item's output.  The last tile's group waits for the last PV (it has seen the phase before; the
            // other group may not have)
            if (g == ((I.n - 1) & 1) && ok) ok = wait_bar(smem_u32(&c.pv_done[g]), (uses[g] + ((I.n - 1) >> 1)) & 1, abort_flag);
            uses[0] += (I.n + 1) / 2;
            uses[1] += I.n / 2;
            bar_sync(5, NSOFT * 32);
            fence_after();
            const float m_used = c.m[(I.n - 1) & 1][r];
            c.mx[g][hk][r] = m_l == -INFINITY ? l_run : l_run * ex2(m_l - m_used);
            bar_sync(5, NSOFT * 32);
            float l = c.mx[0][0][r] + c.mx[0][1][r] + c.mx[1][0][r] + c.mx[1][1][r];
            const bool parts = p.n_splits > 1;
            if (parts && hk == 0 && g == 0) {
                float* ml = p.part_ml + static_cast<int64_t>(it) * 2 * PAIR + rbase + r;
                ml[0] = m_used;
                ml[PAIR] = l;
            }
            if (!parts && p.sink && (m_used != -INFINITY || l != l)) l += ex2(__ldg(p.sink + (T.r0 + rt) % p.H) * LOG2E - m_used);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            // RoPE back: pair `lane` at this row's position, when the warp's rows are one token's
            const bool rot = !parts && p.inv_freq && hk == 1 && g == 1;      // this warp holds the RoPE dims
            const bool one_tok = __all_sync(0xffffffffu, tok == __shfl_sync(0xffffffffu, tok, 0));
            float2 cs = make_float2(1.0f, 0.0f);
            const float2* row_cs = s.cs + (I.tok_row + tok) * 32;
            if (rot && one_tok) cs = row_cs[lane];
            const int64_t row_out = (parts ? static_cast<int64_t>(it) * PAIR : T.row0) + rbase;
            // c.mx is read: the next item may write it; and so is this item (soft_item), whose place the item after the
            // next one takes: with few rows and short key lists no barrier of all eight warps comes before that
            bar_sync(5, NSOFT * 32);
            // O: row r, dims 256 hk + 128 g .. + 127, 32 of them at a time.  64 rows (always, with 64 heads; partials
            // always): through the P buffers (free now) in turn, four blocks of 64 rows x 32 dims (64-byte swizzle) each
            // stored by one TMA copy while the next 32 dims are read and rounded.  Fewer rows: straight from registers,
            // 32 bytes (a sector) a store where the output allows it (for all rows, that kept the load/store unit busy
            // for 4K clocks an item, and the next item's query conversion waiting).
            const bool whole = parts || rows == ROWS;
            uint16_t* dst = (parts ? p.part_o : p.out) + (row_out + r) * D + hk * 256 + g * 128;
            uint8_t* seg = smem + P_OFF + (hk * 2 + g) * 4096 + r * 64;
            const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;     // (the same for every row)
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t w[32];                      // O, then its rounded pairs in the first half
                tmem_ld32(lb + O_COL + g * 128 + q * 32, w);
                tmem_wait_ld();
                if (q == 3) {                        // O has been read
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(in_first(smem_u32(&c.o_free)));
                }
                const bool turn = rot && q >= 2;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float x = __uint_as_float(w[2 * j]) * inv, y = __uint_as_float(w[2 * j + 1]) * inv;
                    if (turn) {
                        float zx = __shfl_sync(0xffffffffu, cs.x, (q & 1) * 16 + j), zy = __shfl_sync(0xffffffffu, cs.y, (q & 1) * 16 + j);
                        if (!one_tok) {              // few heads: the neighbours are other tokens' rows
                            const float2 z = row_cs[(q & 1) * 16 + j];
                            zx = z.x;
                            zy = z.y;
                        }
                        const float x2 = x * zx + y * zy;
                        y = y * zx - x * zy;
                        x = x2;
                    }
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(x, y);
                    w[j] = parts ? pack_half2(x, y) : *reinterpret_cast<const uint32_t*>(&b2);
                }
                if (whole) {
                    if (q > 0) bar_sync(5, NSOFT * 32);      // this round's buffer has been read
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(seg + (q & 1) * 16384 + ((k ^ ((r >> 1) & 3)) << 4)) =
                            make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    fence_async();
                    bar_sync(5, NSOFT * 32);
                    if (warp == 0) {
                        if (elect_one()) {
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                tma_store_2d(parts ? &p_map : &o_map, sbase + P_OFF + (q & 1) * 16384 + z * 4096, z * 128 + q * 32,
                                             static_cast<int>(row_out));
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                            if (q < 3) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                            else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        }
                        __syncwarp();
                    }
                    if (q == 3) bar_sync(5, NSOFT * 32);     // P may be written again
                } else if (r < rows) {
                    if (wide) {
                        st_global_32(dst + q * 32, w);
                        st_global_32(dst + q * 32 + 16, w + 8);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4*>(dst + q * 32 + k * 8) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    }
                }
            }
        }
        if (warp == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        fence_before();
    }
    __syncwarp();
    // every issued MMA has completed before TMEM is freed and before either CTA's memory goes
    if (warp == 9) {
        const long long t0 = clock64();
        while (!mbar_try(smem_u32(&c.drain), 0) && clock64() - t0 < WAIT_CLOCKS) {}
        __syncwarp();
    }
    // (what this thread has set, the first CTA knows after the barrier)
    if (*abort_flag) asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(in_first(smem_u32(&c.abort_flag))), "r"(1) : "memory");
    __syncwarp();
    cluster_sync();
    if (rank == 0 && *abort_flag) fail_items(p, s, c.recent);
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &q, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(q);
        return nullptr;
    }();
    return fn;
}

// The staged rows as [column block of 64 dims][row][64]: a copy of several blocks lays them one after the other.
static bool make_map(CUtensorMap* m, uint16_t* rows, int64_t bound, uint32_t box_rows, uint32_t box_blocks) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dim[3] = {64, static_cast<cuuint64_t>(bound), D / 64};
    const cuuint64_t stride[2] = {D * 2, 128};
    const cuuint32_t box[3] = {64, box_rows, box_blocks}, ones[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, rows, dim, stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of 512 16-bit values (the output, the partials) in blocks of 64 rows x 32 dims.
static bool make_row_map(CUtensorMap* m, uint16_t* rows, int64_t n) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dim[2] = {D, static_cast<cuuint64_t>(n)};
    const cuuint64_t stride[1] = {D * 2};
    const cuuint32_t box[2] = {32, ROWS}, ones[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, rows, dim, stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tcp

// Workspace: staged rows (fp16), the new tokens' RoPE table, a flag byte a staged row, the item counter.
static int64_t stage_per_req(int64_t max_entries, int W, int n_first) {
    return ((max_entries + 63) & ~int64_t(63)) + n_first + W + 63;
}
int64_t tc_stage_rows(int64_t n_rows, int B, int64_t max_entries, int W, int n_first) {
    return B * stage_per_req(max_entries, W, n_first) + n_rows;
}
size_t tc_stage_bytes(int64_t rows, int64_t n_rows) {
    return (static_cast<size_t>(rows) * (tcp::D * 2 + 1) + static_cast<size_t>(n_rows) * 256 + 32 + 255) & ~size_t(255);
}

int tc_chunk_launch(const Params& p, int64_t tiles, int64_t max_entries, void* ws, cudaStream_t st) {
    tcp::Stage s;
    s.per_req = stage_per_req(max_entries, p.W, p.n_first);
    s.bound = tc_stage_rows(p.n_rows, p.B, max_entries, p.W, p.n_first);
    s.rows = static_cast<uint16_t*>(ws);
    s.cs = reinterpret_cast<float2*>(s.rows + s.bound * tcp::D);
    s.flags = reinterpret_cast<uint8_t*>(s.cs + p.n_rows * 32);
    s.next = reinterpret_cast<int*>(s.flags + ((s.bound + 15) & ~int64_t(15)));
    s.n_items = static_cast<int>(tiles * p.n_splits);
    CUtensorMap km, vm, om, pm;
    if (!tcp::make_row_map(&om, p.out, p.n_rows * p.H)) return HCA_ERR_CUDA;
    pm = om;
    if (p.n_splits > 1 && !tcp::make_row_map(&pm, p.part_o, tiles * p.n_splits * tcp::PAIR)) return HCA_ERR_CUDA;
    if (!tcp::make_map(&km, s.rows, s.bound, tcp::HALF, 2) || !tcp::make_map(&vm, s.rows, s.bound, 32, 4)) return HCA_ERR_CUDA;
    cudaError_t e = allow_smem<tcp::paged_tc_kernel>(tcp::SMEM);
    if (e != cudaSuccess) { set_last_cuda_error(static_cast<int>(e)); return HCA_ERR_CUDA; }
    const int64_t pairs = sm_count() / 2 < s.n_items ? sm_count() / 2 : s.n_items;
    s.pairs = static_cast<int>(pairs);
    const int64_t warps = ceil_div(s.bound, tcp::STAGE_ROWS) + (p.inv_freq ? ceil_div(p.n_rows, tcp::STAGE_ROWS) : 0);
    tcp::stage_kernel<<<static_cast<unsigned>(ceil_div(warps, 8)), 256, 0, st>>>(p, s);
    HCA_CHECK_LAUNCH();
    e = launch_pdl(tcp::paged_tc_kernel, dim3(static_cast<unsigned>(2 * pairs)), dim3(tcp::NTHREADS), tcp::SMEM, st, p, s, km, vm, om, pm);
    if (e != cudaSuccess) { set_last_cuda_error(static_cast<int>(e)); return HCA_ERR_CUDA; }
    HCA_CHECK_LAUNCH();
    return HCA_OK;
}

}  // namespace paged

// Reads and clears the device error word of the chunk kernel.  Synchronous.
int paged_take_device_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_device_error, sizeof(int)) != cudaSuccess) return -1;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_paged_device_error, &z, sizeof(int));
    }
    return v;
}

}  // namespace hca
