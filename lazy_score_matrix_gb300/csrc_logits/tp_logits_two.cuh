// Two-word fp32 arithmetic for the list's part of a row: a value h + l with |l| at most half a step of h. A loss
// near zero is the difference of logarithms that agree to several digits, which one fp32 word does not hold,
// and fp64 has two lanes a clock per SM here: a warp's dozen fp64 exponentials and logarithms took longer than
// a row's reduction. exp and ln are the table-driven methods of P. T. P. Tang (ACM Trans. Math. Softw. 15(2),
// 1989; 16(4), 1990) with the leading terms in two words; errors at most 2.2e-9 (exp, relative; from e^-70 down
// its second word falls under fp32's smallest step, 6e-8 at the worst) and 3.7e-9 (ln, absolute).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tp {
namespace rows {

struct Two {
    float h, l;
};

__device__ __forceinline__ Two two_sum(float a, float b) {  // Knuth: exact
    const float s = a + b, t = s - a;
    return Two{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two add(const Two& a, const Two& b) {
    const Two s = two_sum(a.h, b.h);
    const float l = s.l + (a.l + b.l), h = s.h + l;
    return Two{h, l - (h - s.h)};
}
__device__ __forceinline__ Two neg(const Two& a) { return Two{-a.h, -a.l}; }
__device__ __forceinline__ Two mul(const Two& a, const Two& b) {
    const float p = a.h * b.h;
    return Two{p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h)};
}
__device__ __forceinline__ Two warp_add(Two v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = add(v, Two{__shfl_xor_sync(~0u, v.h, o), __shfl_xor_sync(~0u, v.l, o)});
    return v;
}

// 2^(j/32) in two words; the CPU test recomputes both tables in decimal arithmetic
static __device__ const float2 kExpTab[32] = {
    {0x1p+0f, 0x0p+0f},
    {0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f},
    {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f},
    {0x1.29e9ep+0f, -0x1.5c0424p-25f},
    {0x1.306fep+0f, 0x1.4636e2p-25f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f},
    {0x1.3dea64p+0f, 0x1.824684p-25f},
    {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f},
    {0x1.5342b6p+0f, -0x1.2c561p-25f},
    {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.6247ecp+0f, -0x1.f8b55p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f},
    {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.7a1148p+0f, -0x1.829fdp-25f},
    {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.93737cp+0f, -0x1.e64744p-25f},
    {0x1.9c4918p+0f, 0x1.51f848p-27f},
    {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f},
    {0x1.b7f77p+0f, -0x1.a09438p-25f},
    {0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f},
    {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f},
    {0x1.f50766p+0f, -0x1.246ebp-26f},
};
// c = 1/(1 + (i + 1/2)/32) rounded to a multiple of 2^-9, and -ln c in two words
static __device__ const float4 kLnTab[32] = {
    {0x1.f8p-1f, 0x1.020566p-6f, -0x1.db29eep-32f, 0.f},
    {0x1.e9p-1f, 0x1.788596p-5f, -0x1.72a212p-31f, 0.f},
    {0x1.dbp-1f, 0x1.333d8p-4f, -0x1.f9f02ep-30f, 0.f},
    {0x1.cep-1f, 0x1.a4e764p-4f, 0x1.63787p-33f, 0.f},
    {0x1.c1p-1f, 0x1.0ce7ecp-3f, 0x1.b99852p-28f, 0.f},
    {0x1.b5p-1f, 0x1.4462bap-3f, -0x1.1b2612p-30f, 0.f},
    {0x1.aap-1f, 0x1.7898d8p-3f, 0x1.51131cp-29f, 0.f},
    {0x1.9fp-1f, 0x1.ae2ca6p-3f, 0x1.ece57ap-28f, 0.f},
    {0x1.95p-1f, 0x1.e020ccp-3f, 0x1.88d6aep-29f, 0.f},
    {0x1.8bp-1f, 0x1.09aa58p-2f, -0x1.a32726p-27f, 0.f},
    {0x1.82p-1f, 0x1.214456p-2f, 0x1.a1d71ap-27f, 0.f},
    {0x1.79p-1f, 0x1.396ce4p-2f, -0x1.4c8816p-27f, 0.f},
    {0x1.7p-1f, 0x1.522aep-2f, 0x1.ce28f6p-28f, 0.f},
    {0x1.68p-1f, 0x1.68ac84p-2f, -0x1.6395ecp-30f, 0.f},
    {0x1.6p-1f, 0x1.7fafa4p-2f, -0x1.09fabap-28f, 0.f},
    {0x1.59p-1f, 0x1.944144p-2f, -0x1.6bf9b4p-27f, 0.f},
    {0x1.52p-1f, 0x1.a93ed4p-2f, -0x1.ba930ep-29f, 0.f},
    {0x1.4bp-1f, 0x1.beacdap-2f, -0x1.d8e52ep-30f, 0.f},
    {0x1.44p-1f, 0x1.d49024p-2f, 0x1.b7be9ap-28f, 0.f},
    {0x1.3ep-1f, 0x1.e7b42cp-2f, 0x1.eed6bap-29f, 0.f},
    {0x1.38p-1f, 0x1.fb358ap-2f, 0x1.ef491p-27f, 0.f},
    {0x1.32p-1f, 0x1.078bfp-1f, 0x1.4cf15ap-27f, 0.f},
    {0x1.2dp-1f, 0x1.0ffb54p-1f, 0x1.09d23ap-28f, 0.f},
    {0x1.27p-1f, 0x1.1a4a74p-1f, -0x1.d2173p-27f, 0.f},
    {0x1.22p-1f, 0x1.230b0ep-1f, -0x1.d050dap-27f, 0.f},
    {0x1.1dp-1f, 0x1.2bf2ap-1f, -0x1.9ef8f2p-27f, 0.f},
    {0x1.18p-1f, 0x1.35028ap-1f, 0x1.b3b19p-26f, 0.f},
    {0x1.13p-1f, 0x1.3e3c44p-1f, -0x1.b9c224p-27f, 0.f},
    {0x1.0fp-1f, 0x1.45bcc4p-1f, 0x1.93224ep-27f, 0.f},
    {0x1.0ap-1f, 0x1.4f45a8p-1f, 0x1.ad270cp-28f, 0.f},
    {0x1.06p-1f, 0x1.5707a2p-1f, 0x1.aee31ap-27f, 0.f},
    {0x1.02p-1f, 0x1.5ee82ap-1f, 0x1.448324p-26f, 0.f},
};

// e^x; 0 below -87 (what is smaller does not count beside the largest term, which is near 1), +inf above 88.
__device__ __forceinline__ Two exp_two(const Two& x) {
    // ln2/32 in words of 11, 11 and 24 bits: n times the first two is exact for |n| < 2^12
    constexpr float kL1 = 0x1.62cp-6f, kL2 = 0x1.214p-17f, kL3 = 0x1.fbe8e8p-28f;
    if (!(x.h >= -87.f)) return Two{x.h == x.h ? 0.f : x.h, 0.f};
    if (x.h > 88.f) return Two{__int_as_float(0x7f800000), 0.f};
    const float n = rintf(x.h * 46.166241f);
    const int k = (int)n;
    const float r = fmaf(-n, kL2, fmaf(-n, kL1, x.h)) + fmaf(-n, kL3, x.l);
    const float p = fmaf(r * r, fmaf(r, fmaf(r, 1.f / 24.f, 1.f / 6.f), 0.5f), r);  // e^r - 1
    const float2 t = __ldg(kExpTab + (k & 31));
    const Two y = two_sum(t.x, fmaf(t.x, p, t.y));
    const float s = __int_as_float(((k >> 5) + 127) << 23);  // k >> 5 in [-126, 126]
    return Two{y.h * s, y.l * s};
}

// ln z for positive normal z.h; NaN and +inf come back.
__device__ __forceinline__ Two ln_two(const Two& z) {
    constexpr float kLn2Hi = 0x1.62ep-1f, kLn2Lo = 0x1.0bfbe8p-15f;  // 14 bits: e times it is exact
    if (!(z.h < __int_as_float(0x7f800000))) return Two{z.h, 0.f};
    const int b = __float_as_int(z.h), e = (b >> 23) - 127;
    const float f = __int_as_float((b & 0x007fffff) | 0x3f800000);
    const float4 t = __ldg(kLnTab + ((b >> 18) & 31));
    const float r = fmaf(f, t.x, -1.f) + z.l / z.h;  // |r| < 2^-6
    const float p = fmaf(r * r, fmaf(r, fmaf(r, fmaf(r, 0.2f, -0.25f), 1.f / 3.f), -0.5f), r);  // ln(1 + r)
    const Two s = two_sum((float)e * kLn2Hi, t.y);
    const float l = s.l + fmaf((float)e, kLn2Lo, t.z) + p, h = s.h + l;
    return Two{h, l - (h - s.h)};
}

}  // namespace rows
}  // namespace tp
