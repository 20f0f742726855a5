// Append to and gather from the paged 4-bit cache (format: kv4.cuh).
//
// Append reads new keys, values (and queries), rotates keys and queries by their positions,
// quantizes keys and values and writes their codes and params where the block table puts
// them. Gather is the way back: tokens of the cache as 16-bit tensors. Both read and write
// every byte once and are bound by HBM when the tokens are many, by latency when few.
#include <algorithm>

#include "kv4.cuh"
#include "quant_codes.cuh"
#include "rope.cuh"
#include "sm100_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;    // tokens one CTA takes at most

// Last sequence whose first row is at or before row t (cu non-decreasing), found by a whole
// warp: each round looks at 32 spread places at once, so 1024 sequences take two rounds.
__device__ int find_sequence(const Kv4Seqs &s, int t)
{
    if (s.cu == nullptr)
        return min(t / (s.total / s.nseq), s.nseq - 1);
    const int lane = threadIdx.x % 32;
    int lo = 0, n = s.nseq;                            // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = lane * step < n && __ldg(s.cu + i) <= t;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// Where the CTA's tokens live: row t0 + i is token pos[i] of a sequence, in row slot of the
// page whose first byte (of head 0) is at base[i]; base < 0: nothing to do with its cache
// row (a bad page), pos < 0: nothing to do with the token at all.
struct Places {
    int64_t base[kMaxTokens];
    int pos[kMaxTokens];
};
__device__ void find_places(const Kv4Seqs &s, int t0, int tokens, int64_t page_bytes, Places &w)
{
    // the first CTA looks at every sequence, so that malformed lengths are reported whatever
    // sequence the search below finds for a row
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int a, b, len;
        for (int i = threadIdx.x; i < s.nseq; i += kThreads)
            s.rows(i, a, b, len);
    }
    const int warp = threadIdx.x / 32;
    for (int i = warp; i < tokens; i += kThreads / 32) {
        const int t = t0 + i, seq = find_sequence(s, t);
        int a, b, len, pos = -1;
        int64_t base = -1;
        // rows past the last sequence belong to nobody and are left alone
        if (s.rows(seq, a, b, len) && t >= a && t < b) {
            pos = len - (b - t);
            if (pos < 0) {
                atomicOr(s.status, status_bit(SAGE_ERR_BAD_SEQLENS));
                pos = -1;
            } else {
                const int page = s.page(seq, pos);
                if (page >= 0)
                    base = (int64_t)page * s.Hkv * page_bytes;
            }
        }
        if (threadIdx.x % 32 == 0) {
            w.base[i] = base;
            w.pos[i] = pos;
        }
    }
}

__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Codes of eight channels, channel i in bits 4i .. 4i+3. round((x - low) / step) with the
// product by r = fl(1 / step) in place of the quotient: clamped to [-1, 16] first, the two
// differ by less than 2^-17, so they round alike unless the product is within 2^-15 of a
// half-integer; those take the division itself.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float step, float low, float r)
{
    if (step == 0.0f)
        return 0u;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float d = __fsub_rn(x[i], low);
        const float q = fminf(fmaxf(d * r, -1.0f), 16.0f);
        float n = rintf(q);
        if (fabsf(q - n) > 0.5f - 3.0517578125e-05f)
            n = rintf(__fdiv_rn(d, step));
        w |= (uint32_t)max(0, min(15, __float2int_rn(n))) << (4 * i);
    }
    return w;
}

// One CTA: a few tokens. Threads first rotate the queries, 16 channels each; then d/16
// neighbouring lanes take one head of keys or values (the keys rotated like the queries),
// reduce the groups' extremes over their lanes and write the codes.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4AppendArgs p, int tokens_per_cta,
                                                              int q_ctas)
{
    constexpr int kUnits = D / 16, kGroups = D / kKv4Group;
    __shared__ float2 s_cs[2 * kThreads];             // [tokens][rot / 2]
    __shared__ Places s_w;
    griddep_wait();
    const int t0 = blockIdx.x * tokens_per_cta;
    const int tokens = min(tokens_per_cta, p.s.total - t0);
    const int64_t page_bytes = kv4_page_bytes(p.s.page_size(), D);
    find_places(p.s, t0, tokens, page_bytes, s_w);
    __syncthreads();
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < tokens * half; i += kThreads)
        s_cs[i] = rope_cos_sin(s_w.pos[i / half], __ldg(p.freqs + i % half), p.mscale, false);
    __syncthreads();

    if ((int)blockIdx.y < q_ctas) {
        const int hpc = (p.Hq + q_ctas - 1) / q_ctas, h0 = blockIdx.y * hpc;
        const int nh = min(hpc, p.Hq - h0);
        for (int i = threadIdx.x; i < tokens * nh * kUnits; i += kThreads) {
            const int u = i % kUnits, h = h0 + i / kUnits % nh, tl = i / (kUnits * nh);
            if (s_w.pos[tl] < 0)
                continue;
            const T *in = static_cast<const T *>(p.q) + (t0 + tl) * p.q_tok + h * p.q_head;
            T *out = static_cast<T *>(p.q_out) + (t0 + tl) * p.qo_tok + h * p.qo_head;
            const RopeUnit ru = rope_unit(u, p.rot, p.interleaved);
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
    if (blockIdx.y + 1 != gridDim.y)
        return;
    const int items = tokens * 2 * p.s.Hkv * kUnits;
    const int whole = (items + 31) / 32 * 32;         // whole warps reach the shuffles
    for (int i = threadIdx.x; i < whole; i += kThreads) {
        const int u = i % kUnits, hv = i / kUnits % (2 * p.s.Hkv);
        const int tl = i / (kUnits * 2 * p.s.Hkv);
        const bool is_v = hv >= p.s.Hkv;
        const int h = is_v ? hv - p.s.Hkv : hv;
        const bool on = i < items && s_w.base[min(tl, tokens - 1)] >= 0;
        const RopeUnit ru = rope_unit(u, is_v ? 0 : p.rot, p.interleaved);
        float f0[8] = {}, f1[8] = {};
        if (on) {
            const T *in = is_v ? static_cast<const T *>(p.v) + (t0 + tl) * p.v_tok + h * p.v_head
                               : static_cast<const T *>(p.k) + (t0 + tl) * p.k_tok + h * p.k_head;
            load8<T>(*reinterpret_cast<const uint4 *>(in + ru.a0), f0);
            load8<T>(*reinterpret_cast<const uint4 *>(in + ru.a1), f1);
            if (ru.rotated)
                rope_rotate(f0, f1, s_cs + tl * half + 8 * u, p.interleaved);
            if (!is_v && p.k_mean) {
                const float *m = p.k_mean + h * D;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    f0[j] = __fsub_rn(f0[j], __ldg(m + ru.a0 + j));
                    f1[j] = __fsub_rn(f1[j], __ldg(m + ru.a1 + j));
                }
            }
        }
        // extremes of each group over the head's lanes
        float lo[kGroups], hi[kGroups];
        {
            float l0 = f0[0], x0 = f0[0], l1 = f1[0], x1 = f1[0];
#pragma unroll
            for (int j = 1; j < 8; j++) {
                l0 = min_nan(l0, f0[j]);
                x0 = max_nan(x0, f0[j]);
                l1 = min_nan(l1, f1[j]);
                x1 = max_nan(x1, f1[j]);
            }
#pragma unroll
            for (int g = 0; g < kGroups; g++) {
                const bool in0 = ru.a0 / kKv4Group == g, in1 = ru.a1 / kKv4Group == g;
                lo[g] = min_nan(in0 ? l0 : INFINITY, in1 ? l1 : INFINITY);
                hi[g] = max_nan(in0 ? x0 : -INFINITY, in1 ? x1 : -INFINITY);
#pragma unroll
                for (int o = kUnits / 2; o > 0; o >>= 1) {
                    lo[g] = min_nan(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], o));
                    hi[g] = max_nan(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], o));
                }
            }
        }
        if (!on)
            continue;
        __half step[kGroups], low[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; g++) {
            step[g] = __float2half_rn(__fmul_rn(__fsub_rn(hi[g], lo[g]), 1.0f / 15.0f));
            low[g] = __float2half_rn(lo[g]);
        }
        const int ps = p.s.page_size(), row = s_w.pos[tl] & (ps - 1);
        uint8_t *page = p.s.cache + s_w.base[tl] + h * page_bytes;
        uint8_t *codes = page + (is_v ? ps * (D / 2) : 0) + row * (D / 2);
        __half2 *params = reinterpret_cast<__half2 *>(page + ps * D + (is_v ? ps * kGroups * 4 : 0)) +
                          row * kGroups;
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const int a = c ? ru.a1 : ru.a0;
            const int g = kGroups == 1 ? 0 : a / kKv4Group;
            const float sf = __half2float(kGroups > 1 && g ? step[kGroups - 1] : step[0]);
            const float lf = __half2float(kGroups > 1 && g ? low[kGroups - 1] : low[0]);
            *reinterpret_cast<uint32_t *>(codes + a / 2) = codes8(c ? f1 : f0, sf, lf, __frcp_rn(sf));
        }
        if (u < kGroups)
            params[u] = __halves2half2(u ? step[kGroups - 1] : step[0], u ? low[kGroups - 1] : low[0]);
    }
}

// One CTA: a few tokens; a thread turns one 32-bit word of codes (8 channels) into 16 bytes.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4GatherArgs p, int tokens_per_cta)
{
    constexpr int kWords = D / 8, kGroups = D / kKv4Group;
    __shared__ Places s_w;
    griddep_wait();
    const int t0 = blockIdx.x * tokens_per_cta;
    const int tokens = min(tokens_per_cta, p.s.total - t0);
    const int ps = p.s.page_size();
    const int64_t page_bytes = kv4_page_bytes(ps, D);
    find_places(p.s, t0, tokens, page_bytes, s_w);
    __syncthreads();
    const int items = tokens * p.s.Hkv * kWords;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int wd = i % kWords, h = i / kWords % p.s.Hkv, tl = i / (kWords * p.s.Hkv);
        if (s_w.base[tl] < 0)
            continue;
        const int row = s_w.pos[tl] & (ps - 1);
        const uint8_t *page = p.s.cache + s_w.base[tl] + h * page_bytes;
        const int64_t o = ((int64_t)(t0 + tl) * p.s.Hkv + h) * p.rep * D + wd * 8;
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(page + x * ps * (D / 2) +
                                                                   row * (D / 2) + wd * 4);
            const __half2 sl = *(reinterpret_cast<const __half2 *>(page + ps * D + x * ps * kGroups * 4) +
                                 row * kGroups + wd / 8);
            const float step = __low2float(sl), low = __high2float(sl);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                f[j] = __fadd_rn(__fmul_rn((float)((w >> (4 * j)) & 15u), step), low);
            const uint4 u = store8<T>(f);
            T *out = static_cast<T *>(x ? p.v_out : p.k_out) + o;
            for (int r = 0; r < p.rep; r++)
                *reinterpret_cast<uint4 *>(out + r * D) = u;
        }
    }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, cudaStream_t st)
{
    // as many tokens as fill the threads with angles, once there are enough CTAs
    const int tpc = a.s.total >= 4 * 148 ? 4 : 1;
    const int gx = (a.s.total + tpc - 1) / tpc;
    const int q_ctas = a.q ? std::max(1, std::min((a.Hq + 31) / 32, 296 / gx)) : 0;
    const int gy = q_ctas + (gx < 296 || q_ctas == 0 ? 1 : 0);   // few tokens: keys and values apart
    const dim3 grid(gx, gy);
    auto go = [&](auto kern) { kern<<<grid, kThreads, 0, st>>>(a, tpc, q_ctas); };
    if (a.bf16)
        a.d == 128 ? go(kv4_append_kernel<__nv_bfloat16, 128>) : go(kv4_append_kernel<__nv_bfloat16, 64>);
    else
        a.d == 128 ? go(kv4_append_kernel<__half, 128>) : go(kv4_append_kernel<__half, 64>);
    return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs &a, cudaStream_t st)
{
    const int tpc = a.s.total >= 8 * 4 * 148 ? 8 : 1;
    const int grid = (a.s.total + tpc - 1) / tpc;
    auto go = [&](auto kern) { kern<<<grid, kThreads, 0, st>>>(a, tpc); };
    if (a.bf16)
        a.d == 128 ? go(kv4_gather_kernel<__nv_bfloat16, 128>) : go(kv4_gather_kernel<__nv_bfloat16, 64>);
    else
        a.d == 128 ? go(kv4_gather_kernel<__half, 128>) : go(kv4_gather_kernel<__half, 64>);
    return cudaGetLastError();
}

}  // namespace sage
