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
__device__ __forceinline__ float2 rope_cos_sin(int position, double freq, double mscale,
                                               bool inverse)
{
    double s, c;
    sincos((double)position * freq, &s, &c);
    const float sf = (float)(s * mscale);
    return make_float2((float)(c * mscale), inverse ? -sf : sf);
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

// Rotates a unit's two chunks in place; cs: the (cos, sin) of its eight pairs.
__device__ __forceinline__ void rope_rotate(float (&x)[8], float (&y)[8], const float2 *cs,
                                            bool interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 e = cs[i], f = cs[4 + i];
            const float a = x[2 * i], b = x[2 * i + 1], c = y[2 * i], d = y[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, e.x), __fmul_rn(b, e.y));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(b, e.x), __fmul_rn(a, e.y));
            y[2 * i] = __fsub_rn(__fmul_rn(c, f.x), __fmul_rn(d, f.y));
            y[2 * i + 1] = __fadd_rn(__fmul_rn(d, f.x), __fmul_rn(c, f.y));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 e = cs[i];
            const float a = x[i], b = y[i];
            x[i] = __fsub_rn(__fmul_rn(a, e.x), __fmul_rn(b, e.y));
            y[i] = __fadd_rn(__fmul_rn(b, e.x), __fmul_rn(a, e.y));
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
