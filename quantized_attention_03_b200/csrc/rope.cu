// Rotary positions of queries and keys, in one launch: every element is read once, rotated
// and written once, so the pass is bound by HBM (4 bytes per element; 537 MB in 86 us, 6.2 TB/s).
//
// One CTA takes a few neighbouring tokens with their heads, so that a token's 64-bit sines and
// cosines (one per pair, 64 at d = 128) are computed once. A thread keeps one place, 16 channels
// of one token (both halves of eight pairs, so a rotation in place is safe), holds their sines
// and cosines in registers and walks over the heads, two at a time with all loads in flight.
// (Four at a time cost the registers of two more CTAs an SM: 95 against 87 us for 537 MB.)
#include <algorithm>

#include "rope.cuh"
#include "sage_common.cuh"
#include "sm100_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;

template <typename T, int D, int TOKENS>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeArgs p, int heads_per_cta)
{
    constexpr int kUnits = D / 16, kStep = kThreads / (TOKENS * kUnits), kUnroll = 2;
    // cosines and sines, [TOKENS][rot / 2]
    __shared__ __align__(16) float s_c[TOKENS * D / 2], s_s[TOKENS * D / 2];
    griddep_launch_dependents();
    griddep_wait();
    const int half = p.rot / 2, all = p.B * p.N, t0 = blockIdx.x * TOKENS;
    for (int i = threadIdx.x; i < TOKENS * half; i += kThreads) {
        const int t = min(t0 + i / half, all - 1), b = t / p.N, n = t - b * p.N;
        const int pos = p.positions ? p.positions[b * p.pos_b + n] : n;
        const float2 cs = rope_cos_sin(pos, p.freqs[i % half], p.mscale, p.inverse);
        s_c[i] = cs.x;
        s_s[i] = cs.y;
    }
    __syncthreads();
    // unit fastest, then token, then head: a token's neighbours of one head lie side by side
    const int u = threadIdx.x % kUnits, tl = threadIdx.x / kUnits % TOKENS;
    const int t = t0 + tl, b = t / p.N, n = t - b * p.N;
    if (t >= all)
        return;
    const RopeUnit ru = rope_unit(u, p.rot, p.interleaved);
    RopeAngles cs;
    if (ru.rotated)
        cs.load(s_c + tl * half + 8 * u, s_s + tl * half + 8 * u);
    const int h0 = blockIdx.y * heads_per_cta, h1 = h0 + heads_per_cta;
    auto walk = [&](const RopeTensor &x, int first, int last) {
        const T *in = static_cast<const T *>(x.in) + b * x.in_b + n * x.in_n;
        T *out = static_cast<T *>(x.out) + b * x.out_b + n * x.out_n;
        if (!ru.rotated && x.in == x.out)
            return;
        for (int h = first + threadIdx.x / (TOKENS * kUnits); h < last; h += kStep * kUnroll) {
            uint4 w[kUnroll][2];
#pragma unroll
            for (int i = 0; i < kUnroll; i++) {
                const T *a = in + (h + i * kStep) * x.in_h;
                if (h + i * kStep < last) {
                    w[i][0] = *reinterpret_cast<const uint4 *>(a + ru.a0);
                    w[i][1] = *reinterpret_cast<const uint4 *>(a + ru.a1);
                }
            }
#pragma unroll
            for (int i = 0; i < kUnroll; i++) {
                if (h + i * kStep >= last)
                    break;
                if (ru.rotated) {
                    float f0[8], f1[8];
                    load8<T>(w[i][0], f0);
                    load8<T>(w[i][1], f1);
                    rope_rotate(f0, f1, cs, p.interleaved);
                    w[i][0] = store8<T>(f0);
                    w[i][1] = store8<T>(f1);
                }
                T *o = out + (h + i * kStep) * x.out_h;
                *reinterpret_cast<uint4 *>(o + ru.a0) = w[i][0];
                *reinterpret_cast<uint4 *>(o + ru.a1) = w[i][1];
            }
        }
    };
    if (h0 < p.q.H)
        walk(p.q, h0, min(h1, p.q.H));
    if (h1 > p.q.H)
        walk(p.k, max(0, h0 - p.q.H), min(h1 - p.q.H, p.k.H));
}

template <typename T, int D, int TOKENS>
cudaError_t launch(const RopeArgs &a, cudaStream_t st)
{
    const int gx = (int)(((int64_t)a.B * a.N + TOKENS - 1) / TOKENS), heads = a.q.H + a.k.H;
    // few tokens: their heads spread over more CTAs
    const int gy = std::max(1, std::min((heads + 15) / 16, 296 / gx));
    const int hpc = (heads + gy - 1) / gy;
    return launch_overlapped(rope_kernel<T, D, TOKENS>, dim3(gx, (heads + hpc - 1) / hpc), kThreads, 0, st, a, hpc);
}
template <typename T>
cudaError_t launch(const RopeArgs &a, cudaStream_t st)
{
    // with many tokens, a few in a CTA: 64+64 heads of d = 128 take 8.2 us one a CTA and 8.9 four a
    // CTA for 1024 tokens, 16.6 and 11.6 for 2048
    if ((int64_t)a.B * a.N >= 8 * 148)
        return a.d == 128 ? launch<T, 128, 4>(a, st) : launch<T, 64, 8>(a, st);
    return a.d == 128 ? launch<T, 128, 1>(a, st) : launch<T, 64, 1>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st)
{
    return a.bf16 ? launch<__nv_bfloat16>(a, st) : launch<__half>(a, st);
}

}  // namespace sage
