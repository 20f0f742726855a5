// Rotary positions of queries and keys, in one launch: every element is read once, rotated
// and written once, so the pass is bound by HBM (4 bytes per element).
//
// One CTA takes a few tokens with all their heads, so that a token's 64-bit sines and
// cosines (one per pair, 64 at d = 128) are computed once and shared by its heads; a thread
// takes 16 channels of one head at a time (two 16-byte loads, two 16-byte stores) and holds
// both halves of its pairs, so that a rotation in place is safe.
#include <algorithm>

#include "rope.cuh"
#include "sage_common.cuh"
#include "sm100_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs p, int tokens_per_cta,
                                                        int heads_per_cta)
{
    __shared__ float2 s_cs[kThreads];                 // [tokens_per_cta][rot / 2]
    griddep_wait();
    const int half = p.rot / 2, units = p.d / 16;
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta, all = (int64_t)p.B * p.N;
    const int tokens = (int)min((int64_t)tokens_per_cta, all - t0);
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int64_t t = t0 + i / half;
        const int n = (int)(t % p.N);
        const int pos = p.positions ? __ldg(p.positions + t / p.N * p.pos_b + n) : n;
        s_cs[i] = rope_cos_sin(pos, __ldg(p.freqs + i % half), p.mscale, p.inverse);
    }
    __syncthreads();
    const int heads = p.q.H + p.k.H;
    const int h0 = blockIdx.y * heads_per_cta, nh = min(heads_per_cta, heads - h0);
    // unit fastest, then token, then head: a token's neighbours of one head lie side by side
    for (int i = threadIdx.x; i < nh * tokens * units; i += kThreads) {
        const int u = i % units, tl = i / units % tokens, h = h0 + i / (units * tokens);
        const RopeTensor &x = h < p.q.H ? p.q : p.k;
        const int hh = h < p.q.H ? h : h - p.q.H;
        const int64_t t = t0 + tl, b = t / p.N, n = t % p.N;
        const T *in = static_cast<const T *>(x.in) + b * x.in_b + n * x.in_n + hh * x.in_h;
        T *out = static_cast<T *>(x.out) + b * x.out_b + n * x.out_n + hh * x.out_h;
        const RopeUnit ru = rope_unit(u, p.rot, p.interleaved);
        if (!ru.rotated && in == out)
            continue;
        uint4 w0 = *reinterpret_cast<const uint4 *>(in + ru.a0);
        uint4 w1 = *reinterpret_cast<const uint4 *>(in + ru.a1);
        if (ru.rotated) {
            float f0[8], f1[8];
            load8<T>(w0, f0);
            load8<T>(w1, f1);
            rope_rotate(f0, f1, s_cs + tl * half + 8 * u, p.interleaved);
            w0 = store8<T>(f0);
            w1 = store8<T>(f1);
        }
        *reinterpret_cast<uint4 *>(out + ru.a0) = w0;
        *reinterpret_cast<uint4 *>(out + ru.a1) = w1;
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st)
{
    const int64_t tokens = (int64_t)a.B * a.N;
    const int heads = a.q.H + a.k.H;
    const int tpc = tokens >= 4 * 148 ? std::max(1, 2 * kThreads / a.rot) : 1;
    const int64_t gx = (tokens + tpc - 1) / tpc;
    // few tokens: their heads spread over more CTAs
    const int gy = (int)std::max<int64_t>(1, std::min<int64_t>((heads + 15) / 16, 296 / gx));
    const int hpc = (heads + gy - 1) / gy;
    const dim3 grid((unsigned)gx, (unsigned)((heads + hpc - 1) / hpc));
    if (a.bf16)
        rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, tpc, hpc);
    else
        rope_kernel<__half><<<grid, kThreads, 0, st>>>(a, tpc, hpc);
    return cudaGetLastError();
}

}  // namespace sage
