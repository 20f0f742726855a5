// Rotary positions: device code shared by the rotation kernel (rope.cu) and the append to
// the 4-bit cache (kv4.cu).
//
// Pair i of the first `rot` channels of a head, at position p, is rotated by the angle
// p f_i: y0 = x0 c - x1 s, y1 = x1 c + x0 s, with c = cos(p f_i) m and s = sin(p f_i) m.
// The angle, its sine and its cosine are 64-bit (p f_i reaches 10^6 and more, where a
// 32-bit angle is wrong by 0.06 and more) and rounded once to 32 bits with the factor m;
// the rotation itself is four 32-bit products and two sums, each rounded on its own (no
// fused multiply-add), so that the codes the cache gets from it are defined bit for bit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace sage {

// Eight 16-bit elements of a 16-byte word to fp32 and back (round to nearest even).
template <typename T>
__device__ __forceinline__ void load8(const uint4 &u, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<__half>(const uint4 &u, float (&f)[8])
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 t = __half22float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const uint4 &u, float (&f)[8])
{
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 store8(const float (&f)[8]);
template <>
__device__ __forceinline__ uint4 store8<__half>(const float (&f)[8])
{
    uint4 u;
    __half2 *h = reinterpret_cast<__half2 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++)
        h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    return u;
}
template <>
__device__ __forceinline__ uint4 store8<__nv_bfloat16>(const float (&f)[8])
{
    uint4 u;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++)
        h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return u;
}

// (cos, sin) of position * freq, times mscale, rounded once to fp32.
//
// The angle x = RN(position freq), |x| < 2^31, is reduced by the nearest multiple k of pi/2
// (Cody and Waite's method: pi/2 in two pieces). x - k P1 is exact: it is a multiple of 2^-52
// below 1. Sine and cosine of the rest, at most pi/4, are their Taylor sums to the 17th and 18th
// power, whose next terms are below 2^-60: what is left are a few roundings of 2^-53.
__device__ __forceinline__ float2 rope_cos_sin(int position, double freq, double mscale,
                                               bool inverse)
{
    const double x = (double)position * freq;
    const double kd = rint(x * 0.6366197723675814);    // 2 / pi
    const int k = (int)(long long)kd;
    double r = fma(kd, -1.5707963267948966, x);        // pi / 2: its 53 leading bits, then the next
    r = fma(kd, -6.123233995736766e-17, r);
    const double z = r * r;
    double s = 1.0 / 355687428096000.0, c = -1.0 / 6402373705728000.0;   // 1/17!, -1/18!
    s = fma(s, z, -1.0 / 1307674368000.0);
    c = fma(c, z, 1.0 / 20922789888000.0);
    s = fma(s, z, 1.0 / 6227020800.0);
    c = fma(c, z, -1.0 / 87178291200.0);
    s = fma(s, z, -1.0 / 39916800.0);
    c = fma(c, z, 1.0 / 479001600.0);
    s = fma(s, z, 1.0 / 362880.0);
    c = fma(c, z, -1.0 / 3628800.0);
    s = fma(s, z, -1.0 / 5040.0);
    c = fma(c, z, 1.0 / 40320.0);
    s = fma(s, z, 1.0 / 120.0);
    c = fma(c, z, -1.0 / 720.0);
    s = fma(s, z, -1.0 / 6.0);
    c = fma(c, z, 1.0 / 24.0);
    c = fma(c, z, -0.5);
    s = fma(s * z, r, r);
    c = fma(c, z, 1.0);
    const double sn = k & 1 ? c : s, cn = k & 1 ? s : c;     // quadrant
    const float sf = (float)((k & 2 ? -sn : sn) * mscale);
    return make_float2((float)(((k + 1) & 2 ? -cn : cn) * mscale), inverse ? -sf : sf);
}

// A head's d channels are worked on in units of 16: eight pairs of a rotated unit, or 16
// plain channels. Unit u of the half layout holds channels 8u .. 8u+7 and rot/2 + 8u ..
// rot/2 + 8u + 7 (the pairs' two halves); of the interleaved layout, and past rot, 16
// consecutive channels. a0 and a1 are the channels where its two 8-channel chunks start.
struct RopeUnit {
    int a0, a1;
    bool rotated;
};
__device__ __forceinline__ RopeUnit rope_unit(int u, int rot, bool interleaved)
{
    const bool r = u < rot / 16;
    if (r && !interleaved)
        return RopeUnit{8 * u, rot / 2 + 8 * u, true};
    return RopeUnit{16 * u, 16 * u + 8, r};
}

// a - b on packed pairs: one exactly rounded subtraction each.
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

// Cosines and sines of a unit's eight pairs.
struct RopeAngles {
    float2 c[4], s[4];
    __device__ void load(const float *cos, const float *sin)
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            c[i] = reinterpret_cast<const float2 *>(cos)[i];
            s[i] = reinterpret_cast<const float2 *>(sin)[i];
        }
    }
};

// Rotates a pair: a <- a c - b s, b <- b c + a s. (Packed pairs of these lose the rounding of
// the products: mul and add of f32x2 were fused on the way, one result in 2^14 differed.)
__device__ __forceinline__ void rope_pair(float &a, float &b, float c, float s)
{
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// Rotates a unit's two chunks in place.
__device__ __forceinline__ void rope_rotate(float (&x)[8], float (&y)[8], const RopeAngles &cs,
                                            bool interleaved)
{
    if (interleaved) {                                 // pairs side by side, the unit's 16 channels in a row
#pragma unroll
        for (int i = 0; i < 2; i++) {
            rope_pair(x[4 * i], x[4 * i + 1], cs.c[i].x, cs.s[i].x);
            rope_pair(x[4 * i + 2], x[4 * i + 3], cs.c[i].y, cs.s[i].y);
            rope_pair(y[4 * i], y[4 * i + 1], cs.c[2 + i].x, cs.s[2 + i].x);
            rope_pair(y[4 * i + 2], y[4 * i + 3], cs.c[2 + i].y, cs.s[2 + i].y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            rope_pair(x[2 * i], y[2 * i], cs.c[i].x, cs.s[i].x);
            rope_pair(x[2 * i + 1], y[2 * i + 1], cs.c[i].y, cs.s[i].y);
        }
    }
}

// Arguments of the rotation kernel: tensors [B, H, N, d] with their own strides (elements).
struct RopeTensor {
    const void *in;
    void *out;
    int H;
    int64_t in_b, in_n, in_h, out_b, out_n, out_h;
};
struct RopeArgs {
    RopeTensor q, k;
    const int32_t *positions;   // [B, N] (pos_b apart), or nullptr: 0 .. N-1
    int64_t pos_b;
    const double *freqs;        // [rot / 2]
    double mscale;
    int B, N, d, rot, interleaved, inverse, bf16;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st);

}  // namespace sage
