// C-ABI entry points of the rotary positions and the paged 4-bit cache: argument checks,
// then one launch (two for the attention) on the caller's stream.
#include <climits>
#include <cmath>

#include "kv4.cuh"
#include "rope.cuh"

using namespace sage;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool strides_ok(const int64_t *s, int n)
{
    for (int i = 0; i < n; i++)
        if (s[i] % 8 != 0)
            return false;
    return true;
}

// Strides that an output may have over dimensions of n places: none 0, which would put several
// elements in one place; those of the input where it is the input.
bool out_strides_ok(const void *in, const int64_t *si, const void *out, const int64_t *so, const int *n, int dims)
{
    for (int i = 0; i < dims; i++)
        if (n[i] > 1 && (so[i] == 0 || (in == out && si[i] != so[i])))
            return false;
    return true;
}

sage_status_t check_rot(int rot_dim, int d, const double *freqs, int flags, int known_flags)
{
    if (flags & ~known_flags)
        return SAGE_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > d || (rot_dim > 0 && !freqs))
        return SAGE_ERR_INVALID_ARG;
    return rot_dim % 16 ? SAGE_ERR_UNSUPPORTED : SAGE_OK;
}

// Sizes shared by the cache's entry points.
sage_status_t check_seqs(int dtype, int nseq, int total, int Hkv, int d, int page_size,
                         int num_pages, int max_pages, const int32_t *cu_seqlens)
{
    if ((dtype != SAGE_F16 && dtype != SAGE_BF16) || nseq < 0 || total < 0 || Hkv < 0 ||
        num_pages < 0 || max_pages < 0)
        return SAGE_ERR_INVALID_ARG;
    if (d != 64 && d != 128)
        return SAGE_ERR_UNSUPPORTED;
    if (Hkv > 65535 || nseq > 65535)
        return SAGE_ERR_UNSUPPORTED;
    if (page_size < kKv4MinPage || page_size > kKv4MaxPage || (page_size & (page_size - 1)))
        return SAGE_ERR_UNSUPPORTED;
    if ((!cu_seqlens && nseq > 0 && total % nseq) || (num_pages == 0 && nseq > 0 && total > 0))
        return SAGE_ERR_INVALID_ARG;
    return SAGE_OK;
}

Kv4Seqs seqs(const void *cache, const int32_t *block_table, const int32_t *kv_lens,
             const int32_t *cu_seqlens, int nseq, int total, int Hkv, int page_size,
             int num_pages, int max_pages, int *status)
{
    int log2 = 0;
    while ((1 << log2) < page_size)
        log2++;
    return Kv4Seqs{static_cast<uint8_t *>(const_cast<void *>(cache)), block_table, kv_lens,
                   cu_seqlens, nseq, total, Hkv, num_pages, max_pages, log2, status};
}

}  // namespace

extern "C" {

sage_status_t sage_rope_freqs(double *freqs, double *mscale, int rot_dim, double base,
                              int scaling, double factor, double original_len, double beta_fast,
                              double beta_slow)
{
    if (!freqs || rot_dim < 2 || rot_dim % 2 || !(base > 1.0))
        return SAGE_ERR_INVALID_ARG;
    if (scaling < SAGE_ROPE_PLAIN || scaling > SAGE_ROPE_PARTS ||
        (scaling != SAGE_ROPE_PLAIN && !(factor >= 1.0)) ||
        (scaling == SAGE_ROPE_BASE && rot_dim < 4) ||
        (scaling == SAGE_ROPE_PARTS &&
         !(original_len > 0.0 && beta_slow > 0.0 && beta_fast > beta_slow)))
        return SAGE_ERR_INVALID_ARG;
    if (scaling == SAGE_ROPE_BASE)
        base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    double lo = 0.0, hi = 0.0;
    if (scaling == SAGE_ROPE_PARTS) {
        // pair i turns original_len f_i / 2 pi times over the trained positions; the pair
        // (not whole) that turns `turns` times
        const double two_pi = 6.283185307179586;
        auto pair = [&](double turns) {
            return rot_dim * std::log(original_len / (turns * two_pi)) / (2.0 * std::log(base));
        };
        lo = std::fmax(std::floor(pair(beta_fast)), 0.0);
        hi = std::fmin(std::ceil(pair(beta_slow)), rot_dim - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; i++) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == SAGE_ROPE_LINEAR)
            f /= factor;
        if (scaling == SAGE_ROPE_PARTS) {
            const double r = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
            f = f * (1.0 - r) + f / factor * r;
        }
        freqs[i] = f;
    }
    if (mscale)
        *mscale = scaling == SAGE_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return SAGE_OK;
}

sage_status_t sage_rope(const void *q, void *q_out, const void *k, void *k_out,
                        const int32_t *positions, const double *freqs, int dtype, int B, int N,
                        int Hq, int Hk, int d, int rot_dim, int64_t pos_stride,
                        const int64_t *strides, double mscale, int flags, sage_stream_t stream)
{
    if ((dtype != SAGE_F16 && dtype != SAGE_BF16) || B < 0 || N < 0 || Hq < 0 || Hk < 0)
        return SAGE_ERR_INVALID_ARG;
    if (d != 64 && d != 128)
        return SAGE_ERR_UNSUPPORTED;
    if (Hq > 65535 || Hk > 65535 || (int64_t)B * N > INT_MAX)
        return SAGE_ERR_UNSUPPORTED;
    if (rot_dim == 0)
        return SAGE_ERR_INVALID_ARG;
    sage_status_t r = check_rot(rot_dim, d, freqs, flags, SAGE_ROPE_INTERLEAVED | SAGE_ROPE_INVERSE);
    if (r != SAGE_OK)
        return r;
    if (B == 0 || N == 0 || Hq + Hk == 0)
        return SAGE_OK;
    if ((Hq > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out)))
        return SAGE_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out) ||
        (strides && !strides_ok(strides, 12)))
        return SAGE_ERR_MISALIGNED;
    const int nq[3] = {B, Hq, N}, nk[3] = {B, Hk, N};
    if (strides && ((Hq > 0 && !out_strides_ok(q, strides, q_out, strides + 3, nq, 3)) ||
                    (Hk > 0 && !out_strides_ok(k, strides + 6, k_out, strides + 9, nk, 3))))
        return SAGE_ERR_INVALID_ARG;
    auto tensor = [&](const void *in, void *out, int H, const int64_t *s) {
        const int64_t b = (int64_t)H * N * d, h = (int64_t)N * d;
        if (!s)
            return RopeTensor{in, out, H, b, d, h, b, d, h};
        return RopeTensor{in, out, H, s[0], s[2], s[1], s[3], s[5], s[4]};
    };
    const RopeArgs a{tensor(q, q_out, Hq, strides), tensor(k, k_out, Hk, strides ? strides + 6 : nullptr),
                     positions, pos_stride, freqs, mscale, B, N, d, rot_dim,
                     (flags & SAGE_ROPE_INTERLEAVED) ? 1 : 0, (flags & SAGE_ROPE_INVERSE) ? 1 : 0,
                     dtype == SAGE_BF16};
    const cudaError_t e = launch_rope(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SAGE_OK : cuda_fail(e);
}

size_t sage_kv4_page_bytes(int page_size, int d)
{
    if (page_size < kKv4MinPage || page_size > kKv4MaxPage || (page_size & (page_size - 1)) ||
        (d != 64 && d != 128))
        return 0;
    return (size_t)kv4_page_bytes(page_size, d);
}

sage_status_t sage_kv4_append(void *cache, const int32_t *block_table, const int32_t *kv_lens,
                              const int32_t *cu_seqlens, const void *k, const void *v,
                              const void *q, void *q_out, const double *freqs,
                              const float *k_mean, int dtype, int nseq, int total, int Hq,
                              int Hkv, int d, int page_size, int num_pages, int max_pages,
                              int rot_dim, const int64_t *strides, double mscale, int flags,
                              sage_stream_t stream)
{
    sage_status_t r = check_seqs(dtype, nseq, total, Hkv, d, page_size, num_pages, max_pages, cu_seqlens);
    if (r != SAGE_OK)
        return r;
    if (Hq < 0)
        return SAGE_ERR_INVALID_ARG;
    if (Hq > 65535)
        return SAGE_ERR_UNSUPPORTED;
    if ((r = check_rot(rot_dim, d, freqs, flags, SAGE_ROPE_INTERLEAVED)) != SAGE_OK)
        return r;
    if (nseq == 0 || total == 0 || Hkv == 0)
        return SAGE_OK;
    if (!cache || !block_table || !kv_lens || !k || !v || (q && !q_out) || (q && Hq == 0))
        return SAGE_ERR_INVALID_ARG;
    if (!aligned16(cache) || !aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) ||
        !aligned16(k_mean) || (strides && !strides_ok(strides, 8)))
        return SAGE_ERR_MISALIGNED;
    const int nq[2] = {total, Hq};
    if (strides && q && !out_strides_ok(q, strides + 4, q_out, strides + 6, nq, 2))
        return SAGE_ERR_INVALID_ARG;
    int *status = status_ptr(&r);
    if (!status)
        return r;
    const int64_t kv = (int64_t)Hkv * d, qs = (int64_t)Hq * d;
    const int64_t dense[8] = {kv, d, kv, d, qs, d, qs, d};
    const int64_t *s = strides ? strides : dense;
    const Kv4AppendArgs a{seqs(cache, block_table, kv_lens, cu_seqlens, nseq, total, Hkv, page_size,
                               num_pages, max_pages, status),
                          k, v, q, q_out, s[0], s[1], s[2], s[3], s[4], s[5], s[6], s[7], freqs,
                          k_mean, mscale, Hq, d, rot_dim, (flags & SAGE_ROPE_INTERLEAVED) ? 1 : 0,
                          dtype == SAGE_BF16};
    const cudaError_t e = launch_kv4_append(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SAGE_OK : cuda_fail(e);
}

sage_status_t sage_kv4_gather(const void *cache, const int32_t *block_table,
                              const int32_t *kv_lens, const int32_t *cu_seqlens, void *k_out,
                              void *v_out, int dtype, int nseq, int total, int Hkv, int rep, int d,
                              int page_size, int num_pages, int max_pages, sage_stream_t stream)
{
    sage_status_t r = check_seqs(dtype, nseq, total, Hkv, d, page_size, num_pages, max_pages, cu_seqlens);
    if (r != SAGE_OK)
        return r;
    if (rep < 1)
        return SAGE_ERR_INVALID_ARG;
    if ((int64_t)Hkv * rep > 65535)
        return SAGE_ERR_UNSUPPORTED;
    if (nseq == 0 || total == 0 || Hkv == 0)
        return SAGE_OK;
    if (!cache || !block_table || !kv_lens || !k_out || !v_out)
        return SAGE_ERR_INVALID_ARG;
    if (!aligned16(cache) || !aligned16(k_out) || !aligned16(v_out))
        return SAGE_ERR_MISALIGNED;
    int *status = status_ptr(&r);
    if (!status)
        return r;
    const Kv4GatherArgs a{seqs(cache, block_table, kv_lens, cu_seqlens, nseq, total, Hkv, page_size,
                               num_pages, max_pages, status),
                          k_out, v_out, d, rep, dtype == SAGE_BF16};
    const cudaError_t e = launch_kv4_gather(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SAGE_OK : cuda_fail(e);
}

size_t sage_attn_kv4_workspace_size(int Hq, int Hkv, int max_q, int d)
{
    if (Hkv <= 0 || Hq <= 0 || Hq % Hkv || max_q <= 0 || max_q > SAGE_DECODE_MAX_Q ||
        (d != 64 && d != 128))
        return 0;
    return kv4_attn_workspace(Hq, Hkv, max_q, d);
}

sage_status_t sage_attn_kv4(const void *q, const void *cache, const int32_t *block_table,
                            const int32_t *kv_lens, const int32_t *cu_seqlens, void *out,
                            float *lse, int dtype, int nseq, int total, int max_q, int Hq, int Hkv,
                            int d, int page_size, int num_pages, int max_pages, int causal,
                            float sm_scale, const int64_t *q_strides, void *workspace,
                            size_t ws_bytes, sage_stream_t stream)
{
    sage_status_t r = check_seqs(dtype, nseq, total, Hkv, d, page_size, num_pages, max_pages, cu_seqlens);
    if (r != SAGE_OK)
        return r;
    if (Hq < 0 || max_q < 0 || (Hkv == 0 ? Hq > 0 : Hq % Hkv != 0))
        return SAGE_ERR_INVALID_ARG;
    if (Hq > 65535 || max_q > SAGE_DECODE_MAX_Q)
        return SAGE_ERR_UNSUPPORTED;
    if (nseq == 0 || total == 0 || Hq == 0 || Hkv == 0)
        return SAGE_OK;
    // a null cu_seqlens gives every sequence total / nseq queries
    if (max_q == 0 || (!cu_seqlens && total / nseq > max_q))
        return SAGE_ERR_INVALID_ARG;
    if (!q || !cache || !block_table || !kv_lens || !out || !workspace)
        return SAGE_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned16(workspace) ||
        (q_strides && !strides_ok(q_strides, 2)))
        return SAGE_ERR_MISALIGNED;
    if (ws_bytes < kv4_attn_workspace(Hq, Hkv, max_q, d))
        return SAGE_ERR_WORKSPACE;
    int *status = status_ptr(&r);
    if (!status)
        return r;
    const Kv4AttnArgs a{seqs(cache, block_table, kv_lens, cu_seqlens, nseq, total, Hkv, page_size,
                             num_pages, max_pages, status),
                        q, q_strides ? q_strides[0] : (int64_t)Hq * d, q_strides ? q_strides[1] : d,
                        out, lse, workspace, Hq, d, max_q, causal ? 1 : 0, dtype == SAGE_BF16,
                        sm_scale > 0.0f ? sm_scale : 1.0f / std::sqrt((float)d)};
    const cudaError_t e = launch_kv4_attn(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SAGE_OK : cuda_fail(e);
}

}  // extern "C"
