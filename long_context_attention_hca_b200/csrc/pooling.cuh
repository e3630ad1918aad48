// pooling.cuh -- device helpers of the compressors' fixed fp32 sequences,
// shared by the contiguous compressors (compress.cu) and the paged ones
// (paged_cache.cu): the same operations in the same order on both, so that an
// entry's bits do not depend on where it is stored.
#pragma once

#include "common.cuh"

namespace hca {

// E(z) ~= e^z for z <= 0: Cody & Waite argument reduction with a two-part
// ln 2, the Taylor series of e^r to degree 7 (Horner, fused multiply-adds),
// then the exact scale 2^n.  Constants: RN(1/ln 2); ln 2 rounded to fp32
// with its 9 low mantissa bits cleared (so n*LN2_HI is exact for |n| < 2^7);
// RN(ln 2 - LN2_HI); RN(1/k!) for k = 0..7.
__device__ __forceinline__ float cw_exp_neg(float z) {
    if (!(z >= -87.0f)) return 0.0f;
    const float kL2E = __uint_as_float(0x3FB8AA3Bu);
    const float kLn2Hi = __uint_as_float(0x3F317200u);
    const float kLn2Lo = __uint_as_float(0x35BFBE8Eu);
    float nf = rintf(__fmul_rn(z, kL2E));
    float r = __fmaf_rn(-nf, kLn2Hi, z);
    r = __fmaf_rn(-nf, kLn2Lo, r);
    float p = __uint_as_float(0x39500D01u);                 // 1/7!
    p = __fmaf_rn(p, r, __uint_as_float(0x3AB60B61u));      // 1/6!
    p = __fmaf_rn(p, r, __uint_as_float(0x3C088889u));      // 1/5!
    p = __fmaf_rn(p, r, __uint_as_float(0x3D2AAAABu));      // 1/4!
    p = __fmaf_rn(p, r, __uint_as_float(0x3E2AAAABu));      // 1/3!
    p = __fmaf_rn(p, r, 0.5f);                              // 1/2!
    p = __fmaf_rn(p, r, 1.0f);                              // 1/1!
    p = __fmaf_rn(p, r, 1.0f);                              // 1/0!
    const int n = static_cast<int>(nf);                     // -126 <= n <= 0
    return __fmul_rn(p, __uint_as_float(static_cast<uint32_t>(n + 127) << 23));
}

__device__ __forceinline__ void load8_bf16(const uint16_t* p, float (&v)[8]) {
    uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load8_f32(const float* p, float (&v)[8]) {
    float4 a = __ldg(reinterpret_cast<const float4*>(p));
    float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// One RoPE pair (a, b) rotated to position pos by the angle pos * f (the fp64
// product, exact below position 2^29), in fp64 with every product and sum rounded
// (no FMA), each result rounded once to bf16 (a in the low half).
__device__ __forceinline__ uint32_t rope_pair_to_bf16(float a_, float b_, int64_t pos, float f) {
    const double ang = __dmul_rn(static_cast<double>(pos), static_cast<double>(f));
    double sn, cs;
    sincos(ang, &sn, &cs);
    const double a = a_, b = b_;
    const double x0 = __dsub_rn(__dmul_rn(a, cs), __dmul_rn(b, sn));
    const double x1 = __dadd_rn(__dmul_rn(a, sn), __dmul_rn(b, cs));
    const uint32_t lo = __bfloat16_as_ushort(__double2bfloat16(x0));
    const uint32_t hi = __bfloat16_as_ushort(__double2bfloat16(x1));
    return lo | (hi << 16);
}

// cos and sin, each within a few 2^-53, of the fp64 product pos * f, which is the
// angle (exact below position 2^29, rounded beyond, as in rope_pair_to_bf16): u =
// angle / pi is reduced to r in [-1/2, 1/2] by one fused multiply-add (1 / pi in
// two parts: its nearest double and the rest), and sincospi has no large
// arguments to look after.  The rotated pair is that of rope_pair_to_bf16 to
// about 2^-51 (|a| + |b|), so that its bf16 values are the same unless one lies
// that near to the middle between two of them; at a fraction of the latency.
struct CosSin { double c, s; };
__device__ __forceinline__ CosSin rope_cos_sin(int64_t pos, float f) {
    const double ang = __dmul_rn(static_cast<double>(pos), static_cast<double>(f));
    const double ip = 0.31830988618379069, ip_lo = -1.9678676675182486e-17;
    const double k = rint(ang * ip);
    const double r = fma(ang, ip, -k) + ang * ip_lo;
    CosSin v;
    sincospi(r, &v.s, &v.c);
    if (static_cast<long long>(k) & 1) { v.c = -v.c; v.s = -v.s; }
    return v;
}
__device__ __forceinline__ uint32_t rotate_to_bf16(float a_, float b_, const CosSin& v) {
    const double a = a_, b = b_;
    const double x0 = __dsub_rn(__dmul_rn(a, v.c), __dmul_rn(b, v.s));
    const double x1 = __dadd_rn(__dmul_rn(a, v.s), __dmul_rn(b, v.c));
    const uint32_t lo = __bfloat16_as_ushort(__double2bfloat16(x0));
    const uint32_t hi = __bfloat16_as_ushort(__double2bfloat16(x1));
    return lo | (hi << 16);
}

}  // namespace hca
