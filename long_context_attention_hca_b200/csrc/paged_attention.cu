// paged_attention.cu -- attention of each request's new tokens over its paged
// cache: the compressed entries of complete blocks, the sliding window of its
// raw tokens and, where asked, its first tokens, under one softmax; requests of
// any length, from one new token (decode) to a prefill chunk.
//
// "DeepSeek V4 ..." reading note, sections 7 and 8 (shared key-value MQA, the
// window branch, dense attention over every compressed entry), 9 (FP8 entries
// with BF16 RoPE dims; query RMSNorm, partial RoPE, sink) and the section 8
// table (ratio 0: window only).
//
//   o_h(p) = sum_j w_j k_j / (sum_j w_j [+ e^sink_h]),  w_j = e^(scale q_h.k_j)
//   over j: entries e < (p + 1) / m, tokens max(0, p - W + 1) .. p, tokens
//   below n_first; key = value, shared by every head.
#include "paged_attention.cuh"

namespace hca {
namespace paged {

int64_t tc_stage_rows(int64_t n_rows, int B, int64_t max_entries, int W, int n_first);
size_t tc_stage_bytes(int64_t rows, int64_t n_rows);
int tc_chunk_launch(const Params& p, int64_t tiles, int64_t max_entries, void* ws, cudaStream_t st);

// ---------------------------------------------------------------- row kernel
// One CTA = one tile of R rows (tokens x heads, flattened inside a request) and
// one split of its keys.  8 warps: R / 16 row groups x KG key groups; warp
// (rg, kg) computes S for 16 rows and its TK / KG keys over all D dims (mma.sync,
// fp16 operands, fp32 sums), the groups share row maxima and P through shared
// memory, and warp (rg, kg) then accumulates its D / KG dims of O in registers.
// Keys cross from their pages as stored and become fp16 in shared memory.  With
// R = 128 (d = 128 only: O of 16 rows and all dims fits a warp) there is one key
// group: nothing of the softmax is shared, and a key is converted for twice as
// many rows.
//
// Bound at d = 128: latency and issue, not bytes.  A 64-key tile of R = 128 takes
// 9.3K clocks with one CTA an SM (1.5K converting keys, 1.1K queueing copies,
// 2.1K S, 4.1K softmax and O) and 11K with two, 4096 tokens x 64 heads over 64K
// take 493 us, 178 TFLOP/s; 33 single tokens of 8 heads, 10.4 us cold.  Converting
// from registers a tile ahead and four-warp CTAs, three an SM, were no faster.
//
// A key that holds an infinity or a NaN (or a value beyond fp16's range) is
// stored as zeros and marked: a query that sees it gets NaN, one that does not
// see it is untouched (0 x NaN would not be).  A query with such a value is NaN
// throughout: as an infinity it could leave all its logits at -inf, and the row
// would look like one without keys.
template <int D, int R>
struct Rows {
    static constexpr int RG = R / 16, KG = 8 / RG;
    static constexpr int KEYS = TK / KG;         // keys of a warp's S
    static constexpr int NT = KEYS / 8;          // its n-tiles
    static constexpr int DW = D / KG;            // output dims of a warp
    static constexpr int NO = DW / 8;            // their n-tiles
    static constexpr int DR = D == 512 ? 64 : 32;
    static constexpr int G = D == 512 ? 64 : 32;
    static constexpr int DN = D - DR;
    static constexpr size_t Q_BYTES = size_t(R) * D * 2;
    static constexpr size_t K_BYTES = size_t(TK) * D * 2;
    static constexpr size_t P_BYTES = KG > 1 ? size_t(R) * TK * 2 : 0;
    static constexpr size_t CS_BYTES = size_t(R) * (DR / 2) * 8;     // cos / sin of each row's position
    static constexpr size_t RAW_BYTES = size_t(TK) * D * 2;          // the next tile's keys as stored
    static constexpr size_t SC_BYTES = size_t(TK) * 8 * 4;           // and their scales
    static constexpr size_t SMEM = Q_BYTES + K_BYTES + P_BYTES + CS_BYTES + RAW_BYTES + SC_BYTES;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// row-major fp16 tile, 16-byte chunks XOR-swizzled by row (conflict-free ldmatrix)
template <int W2>
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
    return static_cast<uint32_t>(row * W2 + ((chunk ^ (row & 7)) << 4));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v) {
    return pack_half2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

template <int D, int R>
__global__ void __launch_bounds__(256, D == 512 ? 1 : 2) paged_rows_kernel(Params p) {
    using C = Rows<D, R>;
    extern __shared__ __align__(128) char smem[];
    char* qs = smem;
    char* ks = smem + C::Q_BYTES;
    char* ps = ks + C::K_BYTES;
    float2* s_cs = reinterpret_cast<float2*>(ps + C::P_BYTES);
    char* raw = ps + C::P_BYTES + C::CS_BYTES;
    float* s_sc = reinterpret_cast<float*>(raw + C::RAW_BYTES);      // [key][8]
    __shared__ float s_max[8][16];               // [warp][row of its group]
    __shared__ float s_l[8][16];
    __shared__ int64_t s_row[2][TK];             // [tile parity]: a key's row of its pool, -1: not visible
    __shared__ float s_add[TK];                  // -inf: no such key; NaN: the key holds a non-finite value
    const uint32_t qa = static_cast<uint32_t>(__cvta_generic_to_shared(qs));
    const uint32_t ka = static_cast<uint32_t>(__cvta_generic_to_shared(ks));
    const uint32_t pa = static_cast<uint32_t>(__cvta_generic_to_shared(ps));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = warp / C::KG, kg = warp % C::KG;
    const int split = blockIdx.y;

    Tile T;
    if (!make_tile(p, blockIdx.x, R, T)) return;
    const int n_tiles = (T.n_tot + TK - 1) / TK;
    const int t_begin = static_cast<int>(static_cast<int64_t>(n_tiles) * split / p.n_splits);
    const int t_end = static_cast<int>(static_cast<int64_t>(n_tiles) * (split + 1) / p.n_splits);

    // ---- queries as stored, to where their fp16 rows go (converted in place, row by row); a lane copies what it will
    // convert
    constexpr int CL = D / 32;                   // consecutive dims of a lane
    const uint32_t raw_a = static_cast<uint32_t>(__cvta_generic_to_shared(raw));
    const uint32_t sc_a = static_cast<uint32_t>(__cvta_generic_to_shared(s_sc));
#pragma unroll 2
    for (int r = warp; r < T.rows; r += 8) {
        const uint16_t* src = p.q + (T.row0 + r) * D + lane * CL;
        if constexpr (CL >= 8) {
            cp16(qa + r * (D * 2) + lane * 32, src);
            cp16(qa + r * (D * 2) + lane * 32 + 16, src + 8);
        } else {
            cp8(qa + r * (D * 2) + lane * 8, src);
        }
    }
    cp_commit();

    // ---- keys: 64 threads look up the pool rows of a tile's keys, one tile ahead of the copies; a thread copies
    // 16-dim unit u of keys kr + KPP k as stored (cp.async), and later converts just what it copied itself, so that
    // the copies of a tile fly while the tile before is computed.  The loops stay rolled: a CTA runs through them a
    // few times only, and straight-line code would wait for its own instructions (a convert phase of 64 keys took
    // 12K clocks the first time and 7K later when unrolled, with the lookups in every lane).
    constexpr int UPK = D / 16;                  // 16-dim units of a key
    constexpr int KPP = 256 / UPK;               // keys per pass
    const int u = tid % UPK, kr = tid / UPK, d0 = u * 16;
    auto look_up = [&](int t) {
        if (tid < TK) {
            const int slot = t * TK + tid;
            int64_t row = -1;
            if (t < t_end && slot < T.n_tot) {
                if (slot < T.n_e) {
                    row = entry_row(p, T.b, static_cast<uint32_t>(slot));
                } else {
                    const int j = slot - T.n_e;
                    row = token_row(p, T.b, static_cast<uint32_t>(j < T.n_f ? j : T.w_lo + (j - T.n_f)));
                }
            }
            s_row[t & 1][tid] = row;
        }
    };
    auto copy_tile = [&](int t) {
#pragma unroll 2
        for (int k = 0; k < TK / KPP; ++k) {
            const int key = kr + k * KPP;
            const int64_t row = s_row[t & 1][key];
            if (row < 0) continue;
            const uint32_t dst = raw_a + key * (D * 2) + u * 32;
            const void* src;
            if (t * TK + key >= T.n_e) {
                src = p.tok + row * D + d0;
            } else if (d0 < C::DN) {
                cp16(dst, p.codes + row * C::DN + d0);
                if (u % (C::G / 16) == 0) cp4(sc_a + (key * 8 + u / (C::G / 16)) * 4, p.scales + row * (C::DN / C::G) + u / (C::G / 16));
                continue;
            } else {
                src = p.rope + row * C::DR + (d0 - C::DN);
            }
            cp16(dst, src);
            cp16(dst + 16, static_cast<const char*>(src) + 16);
        }
        cp_commit();
    };
    look_up(t_begin);
    look_up(t_begin + 1);

    // ---- queries -> fp16 (rows past the last are zero); RMSNorm and RoPE in fp32
    if (p.inv_freq) {
        for (int w = tid; w < T.rows * (C::DR / 2); w += 256) {
            const int r = w / (C::DR / 2);
            // one table row per token: rows of the same token read the first one's
            if (r == 0 || (T.r0 + r) % p.H == 0)
                s_cs[w] = rope_cs(p.inv_freq, w % (C::DR / 2), T.ctx + (T.r0 + r) / p.H);
        }
    }
    __syncthreads();                             // the pool rows and the RoPE table
    copy_tile(t_begin);
    cp_wait<1>();                                // this lane's query parts
#pragma unroll 1
    for (int r = warp; r < R; r += 8) {
        uint32_t v[CL / 2];
#pragma unroll
        for (int i = 0; i < CL / 2; ++i) v[i] = 0;
        if (r < T.rows) {
            if constexpr (CL >= 8) {
#pragma unroll
                for (int i = 0; i < CL / 8; ++i)
                    *reinterpret_cast<uint4*>(v + 4 * i) = *reinterpret_cast<const uint4*>(qs + r * (D * 2) + lane * 32 + i * 16);
            } else {
                *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(qs + r * (D * 2) + lane * 8);
            }
        }
        __syncwarp();                            // the row has been read
        float f[CL];
#pragma unroll
        for (int i = 0; i < CL / 2; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
        if (p.q_norm_w && r < T.rows) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < CL; ++i) ss += f[i] * f[i];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rr = rsqrtf(ss / static_cast<float>(D) + p.norm_eps);
#pragma unroll
            for (int i = 0; i < CL; ++i) f[i] = f[i] * rr * __ldg(p.q_norm_w + lane * CL + i);
        }
        if (p.inv_freq && r < T.rows && lane * CL >= C::DN) {
            const int h = (T.r0 + r) % p.H;
            const float2* cs = s_cs + max(r - h, 0) * (C::DR / 2) + (lane * CL - C::DN) / 2;
#pragma unroll
            for (int i = 0; i < CL / 2; ++i) {
                const float a = f[2 * i], b = f[2 * i + 1];
                f[2 * i] = a * cs[i].x - b * cs[i].y;
                f[2 * i + 1] = a * cs[i].y + b * cs[i].x;
            }
        }
        uint32_t h2[CL / 2];
#pragma unroll
        for (int i = 0; i < CL / 2; ++i) h2[i] = pack_half2(f[2 * i], f[2 * i + 1]);
        if (__any_sync(0xffffffffu, any_bad(h2)))
#pragma unroll
            for (int i = 0; i < CL / 2; ++i) h2[i] = 0x7FFF7FFFu;
        if constexpr (CL >= 8) {
#pragma unroll
            for (int i = 0; i < CL / 8; ++i)
                *reinterpret_cast<uint4*>(qs + swz<D * 2>(r, lane * (CL / 8) + i)) = *reinterpret_cast<uint4*>(h2 + 4 * i);
        } else {
            *reinterpret_cast<uint2*>(qs + swz<D * 2>(r, lane / 2) + (lane & 1) * 8) = *reinterpret_cast<uint2*>(h2);
        }
    }

    // this thread's rows of S: g8 and g8 + 8 of its row group
    const int g8 = lane >> 2, q4 = lane & 3;
    RowKeys rk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = min(rg * 16 + g8 + 8 * i, T.rows - 1);
        rk[i] = row_keys(p, T, T.ctx + (T.r0 + r) / p.H);
    }
    float o[C::NO][4];
#pragma unroll
    for (int j = 0; j < C::NO; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m_r[2] = {-INFINITY, -INFINITY}, l_r[2] = {0.0f, 0.0f};
    const int e_all = static_cast<int>(entries_before(p, T.ctx + T.r0 / p.H));       // entries that every row sees

    for (int t = t_begin; t < t_end; ++t) {
        cp_wait<0>();
        __syncthreads();                         // the last tile's keys and P are read
        bool flagged = false;
#pragma unroll 2
        for (int k = 0; k < TK / KPP; ++k) {
            const int key = kr + k * KPP;
            const int slot = t * TK + key;
            const bool here = s_row[t & 1][key] >= 0;
            uint32_t h[8];
            const uint4 r0 = *reinterpret_cast<const uint4*>(raw + key * (D * 2) + u * 32);
            if (slot < T.n_e && d0 < C::DN) {
                dequant16(r0, s_sc[key * 8 + u / (C::G / 16)], h);
            } else {
                const uint4 r1 = *reinterpret_cast<const uint4*>(raw + key * (D * 2) + u * 32 + 16);
                const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = bf16x2_to_f16x2(w[i]);
            }
            const bool bad = here && any_bad(h);
            // the UPK lanes of a key are one warp's (8 or 32 consecutive lanes)
            const unsigned bm = __ballot_sync(0xffffffffu, bad) >> (UPK == 32 ? 0 : (lane / UPK) * UPK);
            const bool kbad = (bm & (UPK == 32 ? 0xffffffffu : (1u << (UPK & 31)) - 1u)) != 0;
            if (kbad || !here)
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = 0;
            // (the upper half of the units stores its chunks in the other order: eight lanes, eight bank groups)
            const int sw = (u >> 2) & 1;
            const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
            *reinterpret_cast<uint4*>(ks + swz<D * 2>(key, 2 * u + sw)) = sw ? hi : lo;
            *reinterpret_cast<uint4*>(ks + swz<D * 2>(key, 2 * u + 1 - sw)) = sw ? lo : hi;
            if (u == 0) s_add[key] = !here ? -INFINITY : (kbad ? __int_as_float(0x7fc00000) : 0.0f);
            flagged = flagged || kbad || (!here && slot < T.n_tot);
        }
        copy_tile(t + 1);                        // (no rows past the last tile: nothing is copied)
        flagged = __syncthreads_or(flagged);
        look_up(t + 2);

        const int mi = lane >> 3;
        if constexpr (C::KG == 1) {
            // A row's softmax stays in its warp: 32 keys at a time (S of 64 would not fit the registers beside O), P
            // from registers straight into the second product, no mask where every row sees the whole tile.
            const bool masked = flagged || (t + 1) * TK > e_all;
#pragma unroll 1
            for (int k0 = 0; k0 < TK; k0 += 32) {
                float s[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a[4];
                    ldsm4(qa + swz<D * 2>(rg * 16 + (lane & 7) + 8 * (mi & 1), 2 * kk + (mi >> 1)), a);
#pragma unroll
                    for (int nt = 0; nt < 4; nt += 2) {
                        uint32_t b[4];
                        ldsm4(ka + swz<D * 2>(k0 + nt * 8 + (lane & 7) + 8 * (mi >> 1), 2 * kk + (mi & 1)), b);
                        mma16816(s[nt], a, b[0], b[1]);
                        mma16816(s[nt + 1], a, b[2], b[3]);
                    }
                }
                if (masked)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = k0 + j * 8 + q4 * 2 + (i & 1);
                            // (no such key: -inf for a query of NaN, too)
                            const float add = s_add[key];
                            s[j][i] = sees(rk[i >> 1], T.n_e, t * TK + key) && add != -INFINITY ? s[j][i] + add : -INFINITY;
                        }
                float alpha[2], ref[2], rs[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * i], s[j][2 * i + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m_r[i], mx * p.scale_log2);
                    alpha[i] = mn == -INFINITY ? 1.0f : ex2(m_r[i] - mn);
                    m_r[i] = mn;
                    ref[i] = mn == -INFINITY ? 0.0f : mn;
                }
                uint32_t pr[4][2];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        pr[j][i] = pack_half2(ex2(fmaf(s[j][2 * i], p.scale_log2, -ref[i])), ex2(fmaf(s[j][2 * i + 1], p.scale_log2, -ref[i])));
                        const float2 f = unpack_half2(pr[j][i]);     // l sums the probabilities as PV uses them
                        rs[i] += f.x + f.y;
                    }
                l_r[0] = l_r[0] * alpha[0] + rs[0];
                l_r[1] = l_r[1] * alpha[1] + rs[1];
                if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f))
#pragma unroll
                    for (int j = 0; j < C::NO; ++j) {
                        o[j][0] *= alpha[0]; o[j][1] *= alpha[0];
                        o[j][2] *= alpha[1]; o[j][3] *= alpha[1];
                    }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const uint32_t a[4] = {pr[2 * kk][0], pr[2 * kk][1], pr[2 * kk + 1][0], pr[2 * kk + 1][1]};
#pragma unroll
                    for (int nt = 0; nt < C::NO; nt += 2) {
                        uint32_t b[4];
                        ldsm4t(ka + swz<D * 2>(k0 + kk * 16 + (lane & 7) + 8 * (mi & 1), nt + (mi >> 1)), b);
                        mma16816(o[nt], a, b[0], b[1]);
                        mma16816(o[nt + 1], a, b[2], b[3]);
                    }
                }
            }
        } else {
            // ---- S = Q K^T for 16 rows and this warp's keys
            float s[C::NT][4];
#pragma unroll
            for (int j = 0; j < C::NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll 8
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t a[4];
                ldsm4(qa + swz<D * 2>(rg * 16 + (lane & 7) + 8 * (mi & 1), 2 * kk + (mi >> 1)), a);
                if constexpr (C::NT >= 2) {
#pragma unroll
                    for (int nt = 0; nt < C::NT; nt += 2) {
                        uint32_t b[4];
                        ldsm4(ka + swz<D * 2>(kg * C::KEYS + nt * 8 + (lane & 7) + 8 * (mi >> 1), 2 * kk + (mi & 1)), b);
                        mma16816(s[nt], a, b[0], b[1]);
                        mma16816(s[nt + 1], a, b[2], b[3]);
                    }
                } else {
                    // 8 keys: one x4 load brings two k-steps; the odd step uses the pair loaded with the even one
                    uint32_t b[4];
                    ldsm4(ka + swz<D * 2>(kg * 8 + (lane & 7), (2 * (kk & ~1) + mi)), b);
                    mma16816(s[0], a, (kk & 1) ? b[2] : b[0], (kk & 1) ? b[3] : b[1]);
                }
            }
            // ---- logits (base 2), masks, row maxima over the key groups
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < C::NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = kg * C::KEYS + j * 8 + q4 * 2 + (i & 1);
                    float v = s[j][i] * p.scale_log2;
                    if (flagged) v = s_add[key] == -INFINITY ? -INFINITY : v + s_add[key];
                    if (!sees(rk[i >> 1], T.n_e, t * TK + key)) v = -INFINITY;
                    s[j][i] = v;
                    mx[i >> 1] = fmaxf(mx[i >> 1], v);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            }
            if (q4 == 0) { s_max[warp][g8] = mx[0]; s_max[warp][g8 + 8] = mx[1]; }
            __syncthreads();
            float alpha[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mn = m_r[i];
#pragma unroll
                for (int k = 0; k < C::KG; ++k) mn = fmaxf(mn, s_max[rg * C::KG + k][g8 + 8 * i]);
                // nothing seen yet: any finite reference does (every term is 0)
                alpha[i] = mn == -INFINITY ? 1.0f : ex2(m_r[i] - mn);
                m_r[i] = mn;
            }
            float rs[2] = {0.0f, 0.0f};
            const float ref[2] = {m_r[0] == -INFINITY ? 0.0f : m_r[0], m_r[1] == -INFINITY ? 0.0f : m_r[1]};
#pragma unroll
            for (int j = 0; j < C::NT; ++j) {
                const uint32_t lo = pack_half2(ex2(s[j][0] - ref[0]), ex2(s[j][1] - ref[0]));
                const uint32_t hi = pack_half2(ex2(s[j][2] - ref[1]), ex2(s[j][3] - ref[1]));
                // l sums the probabilities as PV uses them: fp16, at most half a step off each
                const float2 fl = unpack_half2(lo), fh = unpack_half2(hi);
                rs[0] += fl.x + fl.y;
                rs[1] += fh.x + fh.y;
                const int col = kg * C::KEYS + j * 8 + q4 * 2;
                const int r = rg * 16 + g8;
                *reinterpret_cast<uint32_t*>(ps + swz<TK * 2>(r, col >> 3) + (col & 7) * 2) = lo;
                *reinterpret_cast<uint32_t*>(ps + swz<TK * 2>(r + 8, col >> 3) + (col & 7) * 2) = hi;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) l_r[i] = l_r[i] * alpha[i] + rs[i];
#pragma unroll
            for (int j = 0; j < C::NO; ++j) {
                o[j][0] *= alpha[0]; o[j][1] *= alpha[0];
                o[j][2] *= alpha[1]; o[j][3] *= alpha[1];
            }
            __syncthreads();                         // P is complete
            // ---- O += P V (the same tile), this warp's dims
#pragma unroll
            for (int kk = 0; kk < TK / 16; ++kk) {
                uint32_t a[4];
                ldsm4(pa + swz<TK * 2>(rg * 16 + (lane & 7) + 8 * (mi & 1), 2 * kk + (mi >> 1)), a);
#pragma unroll
                for (int nt = 0; nt < C::NO; nt += 2) {
                    uint32_t b[4];
                    ldsm4t(ka + swz<D * 2>(kk * 16 + (lane & 7) + 8 * (mi & 1), kg * (C::DW / 8) + nt + (mi >> 1)), b);
                    mma16816(o[nt], a, b[0], b[1]);
                    mma16816(o[nt + 1], a, b[2], b[3]);
                }
            }
        }
    }

    // ---- l over the key groups
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l_r[i] += __shfl_xor_sync(0xffffffffu, l_r[i], 1);
        l_r[i] += __shfl_xor_sync(0xffffffffu, l_r[i], 2);
    }
    if (q4 == 0) { s_l[warp][g8] = l_r[0]; s_l[warp][g8 + 8] = l_r[1]; }
    __syncthreads();
    float inv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = rg * 16 + g8 + 8 * i;
        float l = 0.0f;
#pragma unroll
        for (int k = 0; k < C::KG; ++k) l += s_l[rg * C::KG + k][g8 + 8 * i];
        l_r[i] = l;
        if (p.n_splits == 1 && p.sink && r < T.rows) {
            // no key seen: the sink alone, the output is 0
            if (m_r[i] != -INFINITY || l != l) l += ex2(__ldg(p.sink + (T.r0 + r) % p.H) * LOG2E - m_r[i]);
        }
        inv[i] = l == 0.0f ? 0.0f : 1.0f / l;
    }
    const int64_t part = static_cast<int64_t>(blockIdx.x) * p.n_splits + split;
    if (p.n_splits > 1 && kg == 0 && q4 == 0) {
        float* ml = p.part_ml + part * 2 * R + rg * 16 + g8;
        ml[0] = m_r[0]; ml[8] = m_r[1];
        ml[R] = l_r[0]; ml[R + 8] = l_r[1];
    }
    const int r0 = rg * 16 + g8;
    if (p.n_splits > 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (r0 + 8 * i >= T.rows) continue;
            uint16_t* dst = p.part_o + (part * R + r0 + 8 * i) * D + kg * C::DW + q4 * 2;
#pragma unroll
            for (int j = 0; j < C::NO; ++j)
                *reinterpret_cast<uint32_t*>(dst + j * 8) = pack_half2(o[j][2 * i] * inv[i], o[j][2 * i + 1] * inv[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r0 + 8 * i;
            if (r >= T.rows) continue;
            const int h = (T.r0 + r) % p.H;
            const float2* cs = s_cs + max(r - h, 0) * (C::DR / 2);
            uint16_t* dst = p.out + (T.row0 + r) * D + kg * C::DW + q4 * 2;
#pragma unroll
            for (int j = 0; j < C::NO; ++j) {
                const int d = kg * C::DW + j * 8 + q4 * 2;
                float x = o[j][2 * i] * inv[i], y = o[j][2 * i + 1] * inv[i];
                if (p.inv_freq && d >= C::DN) {
                    const float2 c = cs[(d - C::DN) / 2];
                    const float x2 = x * c.x + y * c.y;
                    y = y * c.x - x * c.y;
                    x = x2;
                }
                *reinterpret_cast<__nv_bfloat162*>(dst + j * 8) = __floats2bfloat162_rn(x, y);
            }
        }
    }
}

// ---------------------------------------------------------------- combine
// Joins a tile's splits: out = sum_s 2^(m_s - M) l_s o_s / (sum_s 2^(m_s - M)
// l_s [+ sink]), o_s = O_s / l_s in fp16 (half the traffic of fp32; 2^-11
// relative, an eighth of the output's bf16 step).  Bound: the latency of the
// loads, so four warps share a row: each takes every fourth split, its lanes
// over the dims, eight splits' loads in flight; the four sums meet in shared
// memory.  Lane s of every warp holds split s's weight (twice for S > 32).
// Measured: 4 tokens x 64 heads in 18 splits 6.7 us, 33 x 8 in 6 splits 5 us (cold).
template <int D, int R>
__global__ void __launch_bounds__(256) paged_combine_kernel(Params p) {
    constexpr int DR = D == 512 ? 64 : 32, DN = D - DR, CL = D / 32;
    __shared__ float s_acc[8][CL][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3;
    pdl_wait();                                  // the partials are complete
    Tile T;
    if (!make_tile(p, blockIdx.x, R, T)) return;
    const int r = blockIdx.y * 2 + (warp >> 2);
    if (blockIdx.y * 2 >= T.rows) return;        // both rows of the block
    const bool row = r < T.rows;
    const int S = p.n_splits;
    const int64_t part = static_cast<int64_t>(blockIdx.x) * S;
    float m[2], l[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int s = lane + 32 * k;
        m[k] = row && s < S ? p.part_ml[(part + s) * 2 * R + r] : -INFINITY;
        l[k] = row && s < S ? p.part_ml[(part + s) * 2 * R + R + r] : 0.0f;
    }
    float M = fmaxf(m[0], m[1]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float w[2], L = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        // a split that saw nothing has l = 0 and an O that is not read; l = NaN stays NaN
        w[k] = l[k] == 0.0f ? 0.0f : (M == -INFINITY ? l[k] : ex2(m[k] - M) * l[k]);
        L += w[k];
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float acc[CL];
#pragma unroll
    for (int i = 0; i < CL; ++i) acc[i] = 0.0f;
    constexpr int BS = 8;                        // splits whose loads fly together
#pragma unroll 1
    for (int s0 = quarter; s0 < S; s0 += 4 * BS) {
        uint32_t v[BS][CL / 2];
        float ws[BS];
#pragma unroll
        for (int j = 0; j < BS; ++j) {
            const int s = s0 + 4 * j;
            const float a = __shfl_sync(0xffffffffu, w[0], s & 31), b = __shfl_sync(0xffffffffu, w[1], s & 31);
            ws[j] = s < S ? (s < 32 ? a : b) : 0.0f;
#pragma unroll
            for (int i = 0; i < CL / 2; ++i) v[j][i] = 0;
            if (ws[j] != 0.0f) {                 // (an empty split's O was not written)
                const uint16_t* src = p.part_o + ((part + s) * R + r) * D + lane * CL;
                if constexpr (CL >= 8) {
#pragma unroll
                    for (int i = 0; i < CL / 8; ++i)
                        *reinterpret_cast<uint4*>(v[j] + 4 * i) = *(reinterpret_cast<const uint4*>(src) + i);
                } else {
                    *reinterpret_cast<uint2*>(v[j]) = *reinterpret_cast<const uint2*>(src);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < BS; ++j)
#pragma unroll
            for (int i = 0; i < CL / 2; ++i) {
                const float2 f = unpack_half2(v[j][i]);
                acc[2 * i] += ws[j] * f.x;
                acc[2 * i + 1] += ws[j] * f.y;
            }
    }
#pragma unroll
    for (int i = 0; i < CL; ++i) s_acc[warp][i][lane] = acc[i];
    __syncthreads();
    if (quarter != 0 || !row) return;
    const int h = (T.r0 + r) % p.H;
    if (p.sink && (M != -INFINITY || L != L)) L += ex2(__ldg(p.sink + h) * LOG2E - M);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int i = 0; i < CL; ++i)
        acc[i] = (acc[i] + s_acc[warp + 1][i][lane] + s_acc[warp + 2][i][lane] + s_acc[warp + 3][i][lane]) * inv;
    if (p.inv_freq && lane * CL >= DN) {
        const int64_t pos = T.ctx + (T.r0 + r) / p.H;
#pragma unroll
        for (int i = 0; i < CL / 2; ++i) {
            const float2 cs = rope_cs(p.inv_freq, (lane * CL - DN) / 2 + i, pos);
            const float x = acc[2 * i], y = acc[2 * i + 1];
            acc[2 * i] = x * cs.x + y * cs.y;
            acc[2 * i + 1] = y * cs.x - x * cs.y;
        }
    }
    uint32_t v[CL / 2];
#pragma unroll
    for (int i = 0; i < CL / 2; ++i) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    uint16_t* dst = p.out + (T.row0 + r) * D + lane * CL;
    if constexpr (CL >= 8) {
#pragma unroll
        for (int i = 0; i < CL / 8; ++i) *(reinterpret_cast<uint4*>(dst) + i) = *reinterpret_cast<uint4*>(v + 4 * i);
    } else {
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(v);
    }
}

// ---------------------------------------------------------------- host side
// Staged keys take 1 KB each: at most 2 GB of workspace, by the tables' widths
// (the lengths are on the device); beyond that (64 requests whose entry tables
// reach 4M tokens, or 255 that reach 1M) the row kernel serves d = 512 too: 4096
// tokens after 131072 in 4.24 ms where the pairs take 0.59, 13 mixed requests 1.11
// and 0.21 ms, 4 single tokens after 1M 49 and 37 us.
constexpr int64_t MAX_STAGE_ROWS = 2ll << 20;
constexpr int PAIR_ROWS = 128;

// Rows of a row kernel's tile: 16 when no request can fill more (a small head
// count at decode); 128 when such tiles give every SM one (500 tokens x 64 heads
// over 64K: 73 us, with 64 rows 95; 4096 tokens 493 and 660; between one and two
// tiles an SM either is ahead by turns, 4 x 170 window tokens 47 and 46 us); else
// 64 (64 tokens over 128K: 35 us; 32 single tokens 22, splits included).  What
// counts is the rows that can hold a query: a padded step has many others.
inline int tile_rows(int64_t n_rows, int B, int64_t max_new, int H) {
    if (max_new * H <= 16) return 16;
    const int64_t live = n_rows < B * max_new ? n_rows : B * max_new;
    return live * H / 128 >= sm_count() ? 128 : 64;
}
inline int64_t tile_count(int64_t n_rows, int H, int B, int R) { return n_rows * H / R + B; }

// Splits: enough work for every SM (pair) when the tiles alone are too few, but
// at least two key tiles for each (max_keys: the longest key list there can be)
// and only where that shortens a tile's chain by more than the combine costs
// (join, in key tiles: a pair takes 1.15 us a tile and the combine 6 us; 32
// requests of 6 tiles took 44 us in two splits and 30 us whole, 4 requests of 65
// tiles take 36 us in 18 splits where one pair's 65 tiles alone would be 75).
inline int split_count(int64_t slots, int64_t tiles, int64_t max_keys, int tile_keys, int join) {
    const int64_t keys = ceil_div(max_keys, tile_keys);
    int64_t s = slots / (tiles > 0 ? tiles : 1);
    if (s > ceil_div(keys, 2)) s = ceil_div(keys, 2);
    if (s > MAX_SPLITS) s = MAX_SPLITS;
    if (s <= 1 || keys - ceil_div(keys, s) <= join) return 1;
    return static_cast<int>(s);
}

struct Plan { bool pairs; int R, splits; int64_t tiles; size_t stage_bytes; };

static Plan make_plan(int64_t n_rows, int B, int H, int D, int64_t max_new, int64_t max_entries, int W, int n_first) {
    Plan k = {};
    // the longest key list of a tile: entries, first tokens, the window and the tile's own tokens
    const int64_t max_keys = max_entries + W + n_first + 64;
    const int64_t stage_rows = tc_stage_rows(n_rows, B, max_entries, W, n_first);
    const int64_t reqs = n_rows < B ? n_rows : B;      // requests that can have a new token
    k.pairs = D == 512 && stage_rows <= MAX_STAGE_ROWS;
    k.R = k.pairs ? PAIR_ROWS : (D == 512 ? 64 : tile_rows(n_rows, B, max_new, H));
    k.tiles = tile_count(n_rows, H, B, k.R);
    // tiles that can hold rows: one a request when no request fills more
    const int64_t busy = max_new * H <= k.R ? reqs : n_rows * H / k.R + reqs;
    if (k.pairs) {
        k.stage_bytes = tc_stage_bytes(stage_rows, n_rows);
        k.splits = split_count(sm_count() / 2, busy, max_keys, 128, 5);
    } else if (k.R == 128) {
        k.splits = 1;       // taken only where the tiles alone give every SM one: there is no combine of such tiles
    } else {
        // d = 128: two CTAs fit an SM, where that gives shorter chains and not the same work twice as thin (32 single
        // tokens x 64 heads over 64K: 22.4 us with both slots counted, 26.1 with one; 100 over 32K: 37 and 30 us, so
        // not for 64-row tiles that fill more than half the SMs; with 8 heads 15.9 and 20.4)
        const bool both = D == 128 && (k.R == 16 || 2 * busy <= sm_count());
        k.splits = split_count(both ? 2 * sm_count() : sm_count(), busy, max_keys, TK, 2);
    }
    return k;
}

static size_t part_bytes(const Plan& k, int D) {
    if (k.splits <= 1) return 0;
    return static_cast<size_t>(k.tiles) * k.splits * k.R * (static_cast<size_t>(D) * 2 + 2 * sizeof(float)) + 256;
}

template <int D, int R>
static int launch_combine(const Params& p, const Plan& k, cudaStream_t st) {
    if (k.splits <= 1) return HCA_OK;
    const cudaError_t e = launch_pdl(paged_combine_kernel<D, R>, dim3(static_cast<unsigned>(k.tiles), R / 2), dim3(256), 0, st, p);
    if (e != cudaSuccess) { set_last_cuda_error(static_cast<int>(e)); return HCA_ERR_CUDA; }
    HCA_CHECK_LAUNCH();
    return HCA_OK;
}

template <int D, int R>
static int launch_rows(const Params& p, const Plan& k, cudaStream_t st) {
    auto kern = paged_rows_kernel<D, R>;
    const cudaError_t e = allow_smem<paged_rows_kernel<D, R>>(static_cast<int>(Rows<D, R>::SMEM));
    if (e != cudaSuccess) { set_last_cuda_error(static_cast<int>(e)); return HCA_ERR_CUDA; }
    kern<<<dim3(static_cast<unsigned>(k.tiles), k.splits), 256, Rows<D, R>::SMEM, st>>>(p);
    HCA_CHECK_LAUNCH();
    if constexpr (R == 128) return HCA_OK;       // (one split: make_plan)
    else return launch_combine<D, R>(p, k, st);
}

}  // namespace paged

size_t paged_attn_ws_bytes(int64_t n_rows, int B, int H, int D, int64_t max_new, int64_t max_entries, int W, int n_first) {
    const paged::Plan k = paged::make_plan(n_rows, B, H, D, max_new, max_entries, W, n_first);
    return k.stage_bytes + paged::part_bytes(k, D);
}

int paged_attn_launch(paged::Params p, int D, int64_t max_new, int64_t max_entries, void* ws, size_t ws_bytes,
                      cudaStream_t st) {
    const paged::Plan k = paged::make_plan(p.n_rows, p.B, p.H, D, max_new, max_entries, p.W, p.n_first);
    const size_t need = k.stage_bytes + paged::part_bytes(k, D);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return HCA_ERR_WORKSPACE;
    p.n_splits = k.splits;
    if (k.splits > 1) {
        p.part_o = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + k.stage_bytes);
        p.part_ml = reinterpret_cast<float*>(p.part_o + static_cast<size_t>(k.tiles) * k.splits * k.R * D);
    }
    if (k.pairs) {
        const int rc = paged::tc_chunk_launch(p, k.tiles, max_entries, ws, st);
        return rc == HCA_OK ? paged::launch_combine<512, paged::PAIR_ROWS>(p, k, st) : rc;
    }
    if (D == 512) return paged::launch_rows<512, 64>(p, k, st);
    if (k.R == 128) return paged::launch_rows<128, 128>(p, k, st);
    return k.R == 16 ? paged::launch_rows<128, 16>(p, k, st) : paged::launch_rows<128, 64>(p, k, st);
}

}  // namespace hca
