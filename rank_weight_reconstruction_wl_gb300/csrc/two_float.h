// two_float.h -- numbers as the sum of two floats, and exponentials of logits in
// them.  Plain C++: the host compiles it as well, to check its precision.
#pragma once

#ifdef __CUDACC__
#define WL_FF __device__ __forceinline__
#else
#include <cmath>
#include <cstring>
#define WL_FF inline
#endif

namespace wl {

#ifdef __CUDACC__
WL_FF int ff_bits(float f) { return __float_as_int(f); }
WL_FF float ff_float(int i) { return __int_as_float(i); }
#else
using std::fmaf;
WL_FF int ff_bits(float f)
{
    int i;
    std::memcpy(&i, &f, 4);
    return i;
}
WL_FF float ff_float(int i)
{
    float f;
    std::memcpy(&f, &i, 4);
    return f;
}
#endif

// 2^(j/32) as two floats, in two tables: 32 entries of 4 bytes are 32 banks, so that lanes never collide (128 pairs of
// floats took six accesses a warp).
#ifdef __CUDACC__
__constant__
#else
const
#endif
    float kExp2High[32] = {
    0x1.0p+0f, 0x1.059b0ep+0f, 0x1.0b5586p+0f, 0x1.11301ep+0f, 0x1.172b84p+0f, 0x1.1d4874p+0f,
    0x1.2387a6p+0f, 0x1.29e9ep+0f, 0x1.306fep+0f, 0x1.371a74p+0f, 0x1.3dea64p+0f, 0x1.44e086p+0f,
    0x1.4bfdaep+0f, 0x1.5342b6p+0f, 0x1.5ab07ep+0f, 0x1.6247ecp+0f, 0x1.6a09e6p+0f, 0x1.71f75ep+0f,
    0x1.7a1148p+0f, 0x1.82589ap+0f, 0x1.8ace54p+0f, 0x1.93737cp+0f, 0x1.9c4918p+0f, 0x1.a5503cp+0f,
    0x1.ae89fap+0f, 0x1.b7f77p+0f, 0x1.c199bep+0f, 0x1.cb720ep+0f, 0x1.d5818ep+0f, 0x1.dfc974p+0f,
    0x1.ea4afap+0f, 0x1.f50766p+0f};
#ifdef __CUDACC__
__constant__
#else
const
#endif
    float kExp2Low[32] = {
    0x0.0p+0f, -0x1.9d4f52p-25f, 0x1.9f3122p-25f, -0x1.fdb496p-25f, -0x1.c15742p-27f, -0x1.d2e8cap-25f,
    0x1.ceac48p-25f, -0x1.5c0424p-25f, 0x1.4636e2p-25f, -0x1.18aac6p-25f, 0x1.824684p-25f, 0x1.8624b4p-30f,
    -0x1.593abcp-25f, -0x1.2c561p-25f, -0x1.5bd5ecp-27f, -0x1.f8b55p-25f, 0x1.9fcef4p-26f, 0x1.1d8beep-25f,
    -0x1.829fdp-25f, -0x1.accc7cp-26f, 0x1.15506ep-27f, -0x1.e64744p-25f, 0x1.51f848p-27f, -0x1.b83b54p-25f,
    -0x1.a94b14p-26f, -0x1.a09438p-25f, -0x1.3d56b2p-27f, -0x1.8837ccp-27f, -0x1.822dbcp-27f, -0x1.908c94p-25f,
    0x1.52486cp-27f, -0x1.246ebp-26f};

struct FF {
    float h, l;
};

WL_FF FF ff_add(FF a, FF b)
{
    const float s = a.h + b.h, t = s - a.h;
    const float e = (a.h - (s - t)) + (b.h - t);  // Knuth's two-sum: exact
    return FF{s, e + (a.l + b.l)};
}

// The same with l below half a step of h, so that two of them compare by h, then l.
WL_FF FF ff_norm(FF a)
{
    const float s = a.h + a.l;
    return FF{s, a.l - (s - a.h)};
}
// A running sum's next.  Without ff_norm the low parts of thousands of equal terms grow until their own roundings matter:
// 2^-27 of a sum of 32768 (2^-38 so).
WL_FF FF ff_sum(FF sum, FF x) { return ff_norm(ff_add(sum, x)); }
WL_FF FF ff_mul(FF a, float f)
{
    const float p = a.h * f;
    return ff_norm(FF{p, fmaf(a.h, f, -p) + a.l * f});
}
WL_FF bool ff_less(FF a, FF b)  // false where one is NaN
{
    return a.h < b.h || (a.h == b.h && a.l < b.l);
}
WL_FF FF ff_mul(FF a, FF b)
{
    const float p = a.h * b.h;
    return FF{p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h)};
}
WL_FF double ff_double(FF a) { return (double)a.h + (double)a.l; }
WL_FF FF ff_of(double d)
{
    const float h = (float)d;
    return FF{h, (float)(d - (double)h)};
}

// 2^((l - m) c), l <= m, right to 2^-36.8 of itself down to 2^-32, to 2^-34.4 below (the worst of 12 million arguments); 0
// below 2^-100 and where l is -infinity (rows with a NaN do not come here).  The low part is up to 2^-17 of the high one.
// table: kExp2High, then kExp2Low.
WL_FF FF weight(float l, float m, FF c, const float *table)
{
    const float d = l - m, t = d - l;
    const float dl = (l - (d - t)) - (m + t);  // what d has lost
    const float y = fmaxf(d * c.h, -128.0f);
    const float yl = fmaf(dl, c.h, fmaf(d, c.l, fmaf(d, c.h, -y)));
    // y + yl = k/32 + f + yl, |f| <= 1/64
    const float magic = 12582912.0f;  // 1.5 * 2^23
    const float z = fmaf(y, 32.0f, magic);
    const float f = fmaf(z - magic, -0.03125f, y);
    // 2^f - 1 = g + gl = f ln2 + (f ln2)^2 / 2 + (f ln2)^3 / 6 + (f ln2)^4 / 24, the next term below 2^-39.  Of the first term
    // all is kept; what follows is below 2^-14, so that its roundings are below 2^-37.  One float for g left 2^-28.8.
    const float r = f * f * fmaf(f, fmaf(f, 0x1.3b2ab6p-7f, 0x1.c6b08ep-5f), 0x1.ebfbep-3f);
    const float g = fmaf(f, 0x1.62e43p-1f, r);
    const float gl = fmaf(f, -0x1.05c61p-29f, fmaf(f, 0x1.62e43p-1f, -g) + r);
    const int j = ff_bits(z) & 31;
    const float Th = table[j], Tl = table[32 + j];
    // 2^k by its bits: z's integer part from bit 5 on
    const float s = ff_float(((ff_bits(z) & ~31) << 18) + 0x3f800000);
    // (Th + Tl) (1 + g + gl) = Th + q + ..., all of it times 1 + yl ln2
    const float q = Th * g, h = Th + q;
    const float low = (q - (h - Th)) + (fmaf(Th, gl, fmaf(Th, g, -q)) + fmaf(Tl, g, Tl));
    const float more = fmaf(h, yl * 0x1.62e43p-1f, low);
    return y > -100.0f ? FF{h * s, more * s} : FF{0.0f, 0.0f};
}

// max(R - S q, 0)
WL_FF FF residual(FF R, float q, FF S)
{
    const float p = q * S.h;
    const float pl = fmaf(q, S.h, -p) + q * S.l;
    const float s = R.h - p, t = s - R.h;
    const float e = (R.h - (s - t)) - (p + t) + (R.l - pl);
    const float h = s + e;
    return h > 0.0f ? FF{h, e - (h - s)} : FF{0.0f, 0.0f};
}

}  // namespace wl
