// The paged 4-bit key/value cache: its layout, and declarations of its kernels (append and
// gather in kv4.cu, attention in kv4_attn.cu).
//
// Every token of a key or value head is cut into groups of 64 channels. With lo and hi a
// group's least and greatest value: step = fp16((hi - lo) fl(1/15)), low = fp16(lo), code =
// round-half-even((x - low) / step) clamped to 0..15 (0 where step is 0), and the group
// stands for low + code * step. All of it in fp32, the quotient an IEEE division. A group
// that holds a NaN, an infinity or a value past fp16's range stands for non-finite values.
//
// One page holds page_size tokens of one head, [key codes | value codes | key params |
// value params]: codes [page_size][d/2] with channel 2i in the low half of byte i, params
// [page_size][d/64] of (step, low) as fp16. A run of tokens of a page is therefore four
// contiguous pieces. Pages lie as [num_pages][Hkv][page bytes].
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "sage_common.cuh"

namespace sage {

constexpr int kKv4Group = 64;       // channels per (step, low)
constexpr int kKv4MinPage = 16;     // tokens per page: a power of two from here ...
constexpr int kKv4MaxPage = 256;    // ... to here

__host__ __device__ constexpr int64_t kv4_page_bytes(int page_size, int d)
{
    return (int64_t)page_size * (d + 2 * 4 * (d / kKv4Group));
}

// A paged cache with its sequences: sequence s holds kv_lens[s] tokens, token j of it in
// row j % page_size of page block_table[s][j / page_size]; its new tokens (its queries)
// are rows cu[s] .. cu[s+1]-1 of the packed tensors, the last of its tokens. cu == nullptr:
// every sequence has total / nseq of them.
struct Kv4Seqs {
    uint8_t *cache;
    const int32_t *block_table;   // [nseq, max_pages]
    const int32_t *kv_lens;       // [nseq]
    const int32_t *cu;            // [nseq + 1] or nullptr
    int nseq, total, Hkv, num_pages, max_pages, page_log2;
    int *status;

    __device__ int page_size() const { return 1 << page_log2; }
    // Rows a..b-1 of sequence s; false (and a status bit) if cu_seqlens or kv_lens is malformed.
    __device__ bool rows(int s, int &a, int &b, int &len) const
    {
        if (cu) {
            a = cu[s];
            b = cu[s + 1];
        } else {
            const int n = total / nseq;
            a = s * n;
            b = a + n;
        }
        len = kv_lens[s];
        if (sound(a, b, len))
            return true;
        a = b = len = 0;
        return false;
    }
    __device__ bool sound(int a, int b, int len) const
    {
        if (a >= 0 && b >= a && b <= total && len >= 0 && (int64_t)len <= ((int64_t)max_pages << page_log2))
            return true;
        atomicOr(status, status_bit(SAGE_ERR_BAD_SEQLENS));
        return false;
    }
    // Page of token j of sequence s, or -1 (and a status bit) if the table's entry is not one.
    __device__ int page(int s, int j) const
    {
        const int id = block_table[(int64_t)s * max_pages + (j >> page_log2)];
        if (id < 0 || id >= num_pages) {
            atomicOr(status, status_bit(SAGE_ERR_BAD_PAGE));
            return -1;
        }
        return id;
    }
};

struct Kv4AppendArgs {
    Kv4Seqs s;
    const void *k, *v, *q;        // q may be nullptr
    void *q_out;
    int64_t k_tok, k_head, v_tok, v_head, q_tok, q_head, qo_tok, qo_head;
    const double *freqs;          // [rot / 2]; unused when rot == 0
    const float *k_mean;          // [Hkv, d] or nullptr
    double mscale;
    int Hq, d, rot, interleaved, bf16;
};
cudaError_t launch_kv4_append(const Kv4AppendArgs &a, cudaStream_t st);

struct Kv4GatherArgs {
    Kv4Seqs s;
    void *k_out, *v_out;          // [total, Hkv * rep, d]
    int d, rep, bf16;
};
cudaError_t launch_kv4_gather(const Kv4GatherArgs &a, cudaStream_t st);

struct Kv4AttnArgs {
    Kv4Seqs s;
    const void *q;
    int64_t q_tok, q_head;
    void *out;                    // [total, Hq, d]
    float *lse;                   // [total, Hq] or nullptr
    void *workspace;
    int Hq, d, max_q, causal, bf16;
    float sm_scale;
};
size_t kv4_attn_workspace(int Hq, int Hkv, int max_q, int d);
cudaError_t launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t st);

}  // namespace sage
