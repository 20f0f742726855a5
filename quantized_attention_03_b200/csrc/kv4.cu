// Append to and gather from the paged 4-bit cache (format: kv4.cuh).
//
// Append reads new keys, values (and queries), rotates keys and queries by their positions,
// quantizes keys and values and writes their codes and params where the block table puts
// them. Gather is the way back: tokens of the cache as 16-bit tensors. Both read and write
// every byte once. With many tokens gather is bound by HBM (16384 tokens of 8 heads, each written
// 4 times: 48 us, 5.9 TB/s), append half by HBM and half by the quantization (19357 tokens of
// 32 + 16 heads: 97 us for 418 MB); with few tokens both by the latency of finding their places.
#include <algorithm>
#include <type_traits>

#include "kv4.cuh"
#include "quant_codes.cuh"
#include "rope.cuh"
#include "sm100_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256, kAppendThreads = 128;   // of gather, and of append
constexpr int kMaxTokens = 8;     // tokens one CTA takes at most, a warp each to find their places

// The last sequence whose first row is at or before row t (cu non-decreasing), its rows a .. b-1
// and its length, found by a whole warp: each round looks at 32 spread places at once, and the
// last loads what goes with them, so up to 32 sequences take one round trip and 1024 two.
__device__ int find_sequence(const Kv4Seqs &s, int t, int &a, int &b, int &len)
{
    if (s.cu == nullptr) {
        const int n = s.total / s.nseq, seq = min(t / n, s.nseq - 1);
        a = seq * n;
        b = a + n;
        len = s.kv_lens[seq];
        return seq;
    }
    const int lane = threadIdx.x % 32;
    int lo = 0, n = s.nseq;                            // the answer is in [lo, lo + n)
    while (n > 32) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && s.cu[lo + lane * step] <= t;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        lo += last * step;
        n = min(step, n - last * step);
    }
    const int i = lo + min(lane, n - 1);
    a = s.cu[i];
    b = s.cu[i + 1];
    len = s.kv_lens[i];
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, lane < n && a <= t) | 1u);
    a = __shfl_sync(0xffffffffu, a, last);
    b = __shfl_sync(0xffffffffu, b, last);
    len = __shfl_sync(0xffffffffu, len, last);
    return lo + last;
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
        for (int i = threadIdx.x; i < s.nseq; i += blockDim.x)
            s.rows(i, a, b, len);
    }
    const int warp = threadIdx.x / 32;
    for (int i = warp; i < tokens; i += blockDim.x / 32) {
        int a, b, len, pos = -1;
        const int t = t0 + i, seq = find_sequence(s, t, a, b, len);
        int64_t base = -1;
        // rows past the last sequence belong to nobody and are left alone
        if (s.sound(a, b, len) && t >= a && t < b) {
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

__device__ __forceinline__ float min_nan(float a, float b, float c)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Least and greatest of eight.
__device__ __forceinline__ float min8(const float (&x)[8])
{
    return min_nan(min_nan(x[0], x[1], x[2]), min_nan(x[3], x[4], x[5]), min_nan(x[6], x[7]));
}
__device__ __forceinline__ float max8(const float (&x)[8])
{
    return max_nan(max_nan(x[0], x[1], x[2]), max_nan(x[3], x[4], x[5]), max_nan(x[6], x[7]));
}

// Codes of eight channels, channel i in bits 4i .. 4i+3: round((x - low) / step), clamped. The
// product with r = fl(1 / step) stands in for the quotient: where it is below 16 the two differ
// by less than 2^-17, so they round alike unless the product is within 2^-15 of a half-integer;
// then the division itself is taken (2^-14 of the elements). Adding 1.5 2^23 rounds to an
// integer in the low bits of the sum; the constant parts of eight such sums are taken off the
// packed word together.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float step, float low, float r)
{
    if (step == 0.0f)
        return 0u;
    float d[8], b[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 e = add2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(-low, -low));
        const float2 q = mul2(e, make_float2(r, r));
        const float2 n = add2(q, make_float2(kRound, kRound));
        const float2 t = fma2(add2(n, make_float2(-kRound, -kRound)), make_float2(-1.0f, -1.0f), q);
        d[2 * i] = e.x;
        d[2 * i + 1] = e.y;
        b[2 * i] = n.x;
        b[2 * i + 1] = n.y;
        far = fmaxf(far, fmaxf(fabsf(t.x), fabsf(t.y)));
    }
    if (far > 0.5f - 3.0517578125e-05f) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            b[i] = kRound + rintf(fminf(fmaxf(__fdiv_rn(d[i], step), -1.0f), 16.0f));
    }
    uint32_t w = 0;
#pragma unroll
    for (int i = 7; i >= 0; i--)                       // a NaN becomes the lower bound: code 0
        w = (w << 4) + __float_as_uint(fminf(fmaxf(b[i], kRound), kRound + 15.0f));
    return w - (uint32_t)kRoundBits * 0x11111111u;
}

// A thread keeps one place of one token, 16 channels (unit u), and walks over the heads of its
// CTA, a slice (blockIdx.y) of the queries' and of the keys' and values'. Its first rows are
// under way while the tokens' places, sines and cosines are worked out, each next one while one
// is computed. Keys and values: the d/16 neighbouring lanes of a head reduce their groups'
// extremes together and write the codes.
template <typename T, int D, int TOKENS>
__global__ void __launch_bounds__(kAppendThreads, TOKENS == 1 ? 4 : 6) kv4_append_kernel(const Kv4AppendArgs p, int q_heads, int kv_heads)
{
    constexpr int kUnits = D / 16, kGroups = D / kKv4Group, kStep = kAppendThreads / (TOKENS * kUnits);
    // cosines and sines, [TOKENS][rot / 2]
    __shared__ __align__(16) float s_c[TOKENS * D / 2], s_s[TOKENS * D / 2];
    __shared__ Places s_w;
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * TOKENS, tokens = min(TOKENS, p.s.total - t0);
    const int64_t page_bytes = kv4_page_bytes(p.s.page_size(), D);
    const int u = threadIdx.x % kUnits, tl = threadIdx.x / kUnits % TOKENS, hl = threadIdx.x / (kUnits * TOKENS);
    const bool here = tl < tokens;
    const int t = t0 + tl;
    const int q0 = blockIdx.y * q_heads, q1 = p.q ? min(p.Hq, q0 + q_heads) : 0;
    const int k0 = blockIdx.y * kv_heads, k1 = min(p.s.Hkv, k0 + kv_heads);
    const RopeUnit ru = rope_unit(u, p.rot, p.interleaved), vu = rope_unit(u, 0, 0);
    uint4 wq[2], wk[2], wv[2];
    auto load = [&](uint4 (&w)[2], const void *x, int64_t tok, int64_t head, int h, const RopeUnit &unit) {
        const T *in = static_cast<const T *>(x) + t * tok + h * head;
        w[0] = *reinterpret_cast<const uint4 *>(in + unit.a0);
        w[1] = *reinterpret_cast<const uint4 *>(in + unit.a1);
    };
    if (here && q0 + hl < q1)
        load(wq, p.q, p.q_tok, p.q_head, q0 + hl, ru);
    if (here && k0 + hl < k1) {
        load(wk, p.k, p.k_tok, p.k_head, k0 + hl, ru);
        load(wv, p.v, p.v_tok, p.v_head, k0 + hl, vu);
    }
    find_places(p.s, t0, tokens, page_bytes, s_w);
    __syncthreads();
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < tokens * half; i += kAppendThreads) {
        const int k = i / half;
        const float2 cs = rope_cos_sin(s_w.pos[k], p.freqs[i - k * half], p.mscale, false);
        s_c[i] = cs.x;
        s_s[i] = cs.y;
    }
    __syncthreads();
    RopeAngles cs;
    if (ru.rotated && here)
        cs.load(s_c + tl * half + 8 * u, s_s + tl * half + 8 * u);

    if (here && s_w.pos[tl] >= 0) {
        const T *in = static_cast<const T *>(p.q) + t * p.q_tok + (q0 + hl) * p.q_head;
        T *out = static_cast<T *>(p.q_out) + t * p.qo_tok + (q0 + hl) * p.qo_head;
        for (int h = q0 + hl; h < q1; h += kStep, out += kStep * p.qo_head) {
            uint4 w0 = wq[0], w1 = wq[1];
            in += kStep * p.q_head;
            if (h + kStep < q1) {
                wq[0] = *reinterpret_cast<const uint4 *>(in + ru.a0);
                wq[1] = *reinterpret_cast<const uint4 *>(in + ru.a1);
            }
            if (ru.rotated) {
                float f0[8], f1[8];
                load8<T>(w0, f0);
                load8<T>(w1, f1);
                rope_rotate(f0, f1, cs, p.interleaved);
                w0 = store8<T>(f0);
                w1 = store8<T>(f1);
            }
            *reinterpret_cast<uint4 *>(out + ru.a0) = w0;
            *reinterpret_cast<uint4 *>(out + ru.a1) = w1;
        }
    }
    const bool on = here && s_w.base[min(tl, tokens - 1)] >= 0;
    const int ps = p.s.page_size(), row = here ? s_w.pos[tl] & (ps - 1) : 0;
    uint8_t *const at = p.s.cache + (on ? s_w.base[tl] : 0);
    // keys, then values; whole warps reach the shuffles
    auto walk = [&](auto values, uint4 (&w)[2], const void *x, int64_t tok, int64_t head) {
        constexpr bool is_v = decltype(values)::value;
        const RopeUnit &unit = is_v ? vu : ru;
        const int a0 = unit.a0, a1 = unit.a1;
        for (int top = hl / (32 / kUnits) * (32 / kUnits); k0 + top < k1; top += kStep) {
            const int h = k0 + top + hl % (32 / kUnits);
            const bool act = on && h < k1;
            float f0[8] = {}, f1[8] = {};
            if (act) {
                load8<T>(w[0], f0);
                load8<T>(w[1], f1);
                if (h + kStep < k1)
                    load(w, x, tok, head, h + kStep, unit);
            }
            if (act && !is_v) {
                if (ru.rotated)
                    rope_rotate(f0, f1, cs, p.interleaved);
                if (p.k_mean) {
                    const float2 *m0 = reinterpret_cast<const float2 *>(p.k_mean + h * D + a0);
                    const float2 *m1 = reinterpret_cast<const float2 *>(p.k_mean + h * D + a1);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float2 x = sub2(make_float2(f0[2 * j], f0[2 * j + 1]), m0[j]);
                        const float2 y = sub2(make_float2(f1[2 * j], f1[2 * j + 1]), m1[j]);
                        f0[2 * j] = x.x;
                        f0[2 * j + 1] = x.y;
                        f1[2 * j] = y.x;
                        f1[2 * j + 1] = y.y;
                    }
                }
            }
            // extremes of the groups of this lane's two chunks, over the lanes that share them:
            // values have both chunks in one group, four lanes a group
            float lo0 = min8(f0), hi0 = max8(f0), lo1 = min8(f1), hi1 = max8(f1);
            if constexpr (is_v) {
                lo0 = min_nan(lo0, lo1);
                hi0 = max_nan(hi0, hi1);
#pragma unroll
                for (int o = 2; o > 0; o >>= 1) {
                    lo0 = min_nan(lo0, __shfl_xor_sync(0xffffffffu, lo0, o));
                    hi0 = max_nan(hi0, __shfl_xor_sync(0xffffffffu, hi0, o));
                }
                lo1 = lo0;
                hi1 = hi0;
            } else {
                float lo[kGroups], hi[kGroups];
#pragma unroll
                for (int g = 0; g < kGroups; g++) {
                    const bool in0 = a0 / kKv4Group == g, in1 = a1 / kKv4Group == g;
                    lo[g] = min_nan(in0 ? lo0 : INFINITY, in1 ? lo1 : INFINITY);
                    hi[g] = max_nan(in0 ? hi0 : -INFINITY, in1 ? hi1 : -INFINITY);
#pragma unroll
                    for (int o = kUnits / 2; o > 0; o >>= 1) {
                        lo[g] = min_nan(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], o));
                        hi[g] = max_nan(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], o));
                    }
                }
                const bool s0 = kGroups > 1 && a0 / kKv4Group, s1 = kGroups > 1 && a1 / kKv4Group;
                lo0 = s0 ? lo[kGroups - 1] : lo[0];
                hi0 = s0 ? hi[kGroups - 1] : hi[0];
                lo1 = s1 ? lo[kGroups - 1] : lo[0];
                hi1 = s1 ? hi[kGroups - 1] : hi[0];
            }
            if (!act)
                continue;
            uint8_t *page = at + h * page_bytes;
            uint8_t *codes = page + (is_v ? ps * (D / 2) : 0) + row * (D / 2);
            __half2 *params = reinterpret_cast<__half2 *>(page + ps * D + (is_v ? ps * kGroups * 4 : 0)) +
                              row * kGroups;
            auto word = [&](const float (&f)[8], int a, float lo, float hi) {
                const __half step = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
                const __half low = __float2half_rn(lo);
                const float sf = __half2float(step);
                if (a % kKv4Group == 0)                // the chunk that begins a group writes its params
                    params[a / kKv4Group] = __halves2half2(step, low);
                return codes8(f, sf, __half2float(low), __frcp_rn(sf));
            };
            const uint32_t w0 = word(f0, a0, lo0, hi0), w1 = word(f1, a1, lo1, hi1);
            if (is_v || a1 == a0 + 8) {
                *reinterpret_cast<uint2 *>(codes + a0 / 2) = make_uint2(w0, w1);
            } else {
                *reinterpret_cast<uint32_t *>(codes + a0 / 2) = w0;
                *reinterpret_cast<uint32_t *>(codes + a1 / 2) = w1;
            }
        }
    };
    walk(std::false_type{}, wk, p.k, p.k_tok, p.k_head);
    walk(std::true_type{}, wv, p.v, p.v_tok, p.v_head);
}

// One CTA: a few tokens. A thread keeps one 32-bit word of codes (8 channels) and walks over the
// tokens' heads, keys and values together.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4GatherArgs p, int tokens_per_cta)
{
    constexpr int kWords = D / 8, kGroups = D / kKv4Group, kStep = kThreads / kWords, kUnroll = 2;
    __shared__ Places s_w;
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * tokens_per_cta;
    const int tokens = min(tokens_per_cta, p.s.total - t0);
    const int ps = p.s.page_size(), Hkv = p.s.Hkv;
    const int64_t page_bytes = kv4_page_bytes(ps, D);
    find_places(p.s, t0, tokens, page_bytes, s_w);
    __syncthreads();
    const int wd = threadIdx.x % kWords;
    const int dt = kStep / Hkv, dh = kStep % Hkv;      // a step to the thread's next (token, head)
    int tl = threadIdx.x / kWords / Hkv, h = threadIdx.x / kWords % Hkv;
    while (tl < tokens) {
        uint32_t w[kUnroll][2];
        __half2 sl[kUnroll][2];
        int64_t o[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; i++) {
            o[i] = -1;
            if (tl < tokens && s_w.base[tl] >= 0) {
                const int row = s_w.pos[tl] & (ps - 1);
                const uint8_t *page = p.s.cache + s_w.base[tl] + h * page_bytes;
                o[i] = ((int64_t)(t0 + tl) * Hkv + h) * p.rep * D + wd * 8;
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    w[i][x] = reinterpret_cast<const uint32_t *>(page + (x * ps + row) * (D / 2))[wd];
                    sl[i][x] = *(reinterpret_cast<const __half2 *>(page + ps * D + (x * ps + row) * (kGroups * 4)) +
                                     wd / 8);
                }
            }
            tl += dt;
            h += dh;
            if (h >= Hkv) {
                h -= Hkv;
                tl++;
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; i++) {
            if (o[i] < 0)
                continue;
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const float step = __low2float(sl[i][x]), low = __high2float(sl[i][x]);
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; j++)            // the product is exact: 11 bits times 4
                    f[j] = fmaf((float)((w[i][x] >> (4 * j)) & 15u), step, low);
                const uint4 v = store8<T>(f);
                T *out = static_cast<T *>(x ? p.v_out : p.k_out) + o[i];
                for (int r = 0; r < p.rep; r++)
                    *reinterpret_cast<uint4 *>(out + r * D) = v;
            }
        }
    }
}

}  // namespace

namespace {
template <typename T, int D, int TOKENS>
cudaError_t launch_append(const Kv4AppendArgs &a, cudaStream_t st)
{
    const int gx = (a.s.total + TOKENS - 1) / TOKENS;
    // few tokens: their heads spread over more CTAs
    const int gy = std::max(1, std::min({((a.q ? a.Hq : 0) + 15) / 16, (a.s.Hkv + 3) / 4, 296 / gx}));
    return launch_overlapped(kv4_append_kernel<T, D, TOKENS>, dim3(gx, gy), kAppendThreads, 0, st, a, (a.Hq + gy - 1) / gy,
                             (a.s.Hkv + gy - 1) / gy);
}
template <typename T>
cudaError_t launch_append(const Kv4AppendArgs &a, cudaStream_t st)
{
    // with many tokens, a few in a CTA: 32 + 16 heads of d = 128 take 13 us one a CTA and 18 four a
    // CTA for 1024 tokens, 50 and 43 for 4096
    if (a.s.total >= 16 * 148)
        return a.d == 128 ? launch_append<T, 128, 4>(a, st) : launch_append<T, 64, 8>(a, st);
    return a.d == 128 ? launch_append<T, 128, 1>(a, st) : launch_append<T, 64, 1>(a, st);
}
}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, cudaStream_t st)
{
    return a.bf16 ? launch_append<__nv_bfloat16>(a, st) : launch_append<__half>(a, st);
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs &a, cudaStream_t st)
{
    // tokens of a CTA: about 2048 stores of 16 bytes, but at least 2 CTAs an SM. 16384 tokens of 8
    // heads, each written 4 times: 48 us with 2 tokens, 51 with 8; once: 26 and 20
    const int stores = a.s.Hkv * (a.d / 8) * a.rep * 2;   // Hkv rep is at most 65535
    const int tpc = std::max(1, std::min({kMaxTokens, std::max(2, 2048 / stores), a.s.total / 592}));
    const int grid = (a.s.total + tpc - 1) / tpc;
    auto go = [&](auto kern) { return launch_overlapped(kern, dim3(grid), kThreads, 0, st, a, tpc); };
    if (a.bf16)
        return a.d == 128 ? go(kv4_gather_kernel<__nv_bfloat16, 128>) : go(kv4_gather_kernel<__nv_bfloat16, 64>);
    return a.d == 128 ? go(kv4_gather_kernel<__half, 128>) : go(kv4_gather_kernel<__half, 64>);
}

}  // namespace sage
