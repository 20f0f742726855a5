// Attention of a few queries per sequence over the paged 4-bit cache (format: kv4.cuh).
//
// For a query row q and a cached key k = low + step n (n the codes of a 64-channel group)
//   t_j = sm_scale log2(e) (sum_g step_g (q_g . n_g) + low_g sum(q_g)),  p_j = 2^(t_j - m),
//   O = sum_j p_j v_j / sum_j p_j,  v_j = (low' + step n'),  n' = n - 8, low' = low + 8 step,
// so neither keys nor values are ever written out: the codes themselves are the operands of
// two 16-bit tensor-core products and the params scale their 32-bit results (keys) or the
// probabilities (values).
//
// What bounds it: the cache is read once from HBM, 0.5625 bytes per element (B8 H32 over 32768
// keys of d 128: 1.21 GB, 185 us at the copy bandwidth, which the copies alone reach), and each
// element has to be turned from 4 bits into a 16-bit operand: the instructions are the bound,
// 231 us for that cache without its copies, 246 us in all (4.9 TB/s; 272 us in a loop of calls that
// lasts, at the lower clock of that).
//   - A code masked in place is an fp16 subnormal, n 2^-24 or 16 n 2^-24, which the tensor core
//     takes as it is; one AND makes two operands. The queries of the second kind of channel are
//     divided by 16 beforehand, the outputs at the end. Sums of such products are good to 2^-18 of
//     their terms' absolute sum; fp16 outputs over random keys are 2.1e-4 from 64-bit results, as
//     those rounded to fp16 are.
//   - Values are centred (n - 8), because the sum of p n' stays near the size of its result;
//     uncentred it would be the difference of two sums 100 times larger over a long cache, in
//     which the accumulator's own rounding shows. One product with constant codes -8 gives what
//     a tile has to be lessened by, the same for all channels (centring the codes themselves,
//     an addition for every two, took 260 us).
//   - Probabilities times step are split into two fp16 terms, high and low, each with its own
//     product: one term alone would round every p to 11 bits, as much error again as the
//     rounding of the 16-bit output. They are scaled by a power of two of their group's largest
//     step so far, whose product with p = 1 then is 8 or more: two terms are good to 2^-21 of the
//     product or to 2^-25, which is 2^-28 of the largest step, whichever is more. (One scale for
//     both groups of d = 128 left a group whose values were 10^6 times smaller 7 bits; two cost the
//     longest cache 1.2 us of 245.0 and saved the ragged sequences below 0.8 of 81.4.)
// Queries are the 8-wide side of mma.m16n8k16 and keys (or channels) the 16-wide one, so a
// group of up to 8 query rows that share a key head costs one pass, and a masked word of codes is
// an operand where it was loaded. tcgen05 was not tried: with keys on its 128-row side and 8 to 32
// rows of queries as N its tiles would be full, but its operands lie in shared or tensor memory, so
// the codes would first be expanded and written there.
//
// Work split: all (sequence, key head, row block, tile) of the call form one list, cut into
// equal shares whatever the sequences' lengths (which only the device knows), one per team: a
// warp where there are many such segments, else a CTA, whose warps take its tiles in turn. Each
// warp fetches its tiles through a ring of its own, up to two ahead and across segments; a CTA's
// warps are merged at the end of every segment. What a team began or left unfinished goes to two
// partial slots of the workspace and a second kernel merges those in order, so results do not
// depend on timing.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv4.cuh"
#include "rope.cuh"
#include "sm100_ptx.cuh"

namespace sage {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMergeWarps = 8;
constexpr int kSMs = 148;
// Places that the start of a segment takes in the list of work, in tiles: what it costs a CTA
// to start on one (queries, pages, first tile, merge), or a warp that works alone. Without it, a
// CTA that gets many short sequences is the last to end: 64 sequences of 1 to 8192 tokens took
// 122 us with 0, 101 with 8, 93 with 16, 95 with 24.
constexpr int kTeamCost = 16, kSoloCost = 2;
// From so many segments on, every warp works alone on its own share (64 such sequences 84 against
// 95 us, 256 of up to 200 tokens 31 against 42); below, the warps of a CTA share one, since the
// partial rows of all warps for one segment would cost more than its keys (8 segments of 32768
// keys: 53 against 23 us).
constexpr int kSoloSegments = kSMs;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// D: head dim. NT: 8-row query tiles per pass (rows of one key head). FOLD (NT = 1): at most 4
// rows, twice in the tile: the high terms of P in columns 0-3 and the low ones in 4-7, so that
// one value product takes both.
template <int D, int NT, bool FOLD>
struct Cfg {
    static constexpr int kTile = 4096 / D;             // keys per warp tile
    static constexpr int kGroups = D / kKv4Group;
    static constexpr int kStages = 2;                  // of 32 or 64 keys: 55 KB an SM in flight
    // 12 warps of 168 registers or 8 of 255 (50 to 80 bytes of spills a thread at d = 128); 16 of
    // 128 registers (200 to 220 bytes): 98 against 86 us over the ragged sequences below
    static constexpr int kCtasPerSM = NT == 1 ? 3 : 2;
    static constexpr int kRows = FOLD ? 4 : 8 * NT;
    static constexpr int kParBytes = kTile * kGroups * 4;          // params of a tile's keys
    static constexpr int kStageBytes = kTile * D + 2 * kParBytes;   // 4608: the other stage is an XOR away
    static constexpr int kPitch = D + 4;               // floats of a partial row: sums, reference, weight
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kFloats = kTile * kGroups * 2;   // a tile's params in fp32, keys' or values'
    static constexpr int kSmem = kRing + kWarps * (kRows * kPitch + 2 * kFloats) * 4;
};

// What a team that begins a (sequence, head, row block) and does not finish it leaves for the
// merge: the last team that works on it (-1: nothing to merge) and whose rows they are.
struct Tail {
    int last, row0, n, kvh, rb;
};

struct Params {
    Kv4AttnArgs a;
    int *solo;            // whether warps work alone, for the merge
    float *part;          // [teams][2][rows][D + 4]: sums, then reference and weight
    Tail *tail;           // [teams]
    int group;            // query heads per key head
    float sc_log2;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with no sum to add to.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// 8x8 transpose of 16-bit elements over the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t b) { return *reinterpret_cast<__half2 *>(&b); }

// 16-byte asynchronous copy, global to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// -8 and -128 times 2^-24, twice: what centres the codes of the two kinds of channel.
constexpr uint32_t kMinus8 = 0x80088008u, kMinus128 = 0x80808080u;

// A key's or value's two numbers for each of its groups, as the warp wrote them (below).
template <int G>
__device__ __forceinline__ void load_params(const float *at, float2 (&p)[G])
{
    if constexpr (G == 2) {
        const float4 u = *reinterpret_cast<const float4 *>(at);
        p[0] = make_float2(u.x, u.y);
        p[1] = make_float2(u.z, u.w);
    } else {
        p[0] = *reinterpret_cast<const float2 *>(at);
    }
}

// N channels from `ch` on of an output row, acc / L, and with the first of them its lse.
template <int N>
__device__ __forceinline__ void write_row(const Kv4AttnArgs &a, int64_t row, int head, int d, int ch, float M, float L,
                                          const float *acc)
{
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int64_t at = (row * a.Hq + head) * d + ch;
    uint32_t u[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; i++)
        if (a.bf16)
            *reinterpret_cast<__nv_bfloat162 *>(u + i) = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
        else
            u[i] = pack_half2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    uint16_t *out = static_cast<uint16_t *>(a.out) + at;
    if constexpr (N == 4)
        *reinterpret_cast<uint2 *>(out) = make_uint2(u[0], u[1]);
    else
        *reinterpret_cast<uint32_t *>(out) = u[0];
    if (ch == 0 && a.lse)
        a.lse[row * a.Hq + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// A query row's operands for the key product: this lane holds 16 channels of each group, u[g]
// the 16-bit input. Operand 0 of an 8-channel word is channels (0, 4), 1 is (1, 5) / 16, 2 is
// (2, 6), 3 is (3, 7) / 16, as the masked codes have them. The row is scaled by a power of two
// so that its largest element is in [2^14, 2^15); returned is what a product's units are worth,
// 2^24 over that factor (the codes are 2^-24), and in those units the row's sum over each group
// (in fp32: products of subnormals keep 2^-18 of their size, too little for the one term that
// all keys share).
template <int G>
__device__ __forceinline__ float query_row(const uint4 (&u)[G][2], int bf16, uint32_t (&qf)[G][2][4], float (&sum)[G])
{
    float big;
    if (bf16) {
        __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll
        for (int i = 0; i < G * 8; i++)
            m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 *>(&u[i / 8][i / 4 % 2])[i % 4]));
        big = fmaxf(__low2float(m), __high2float(m));
    } else {
        __half2 m = __float2half2_rn(0.0f);
#pragma unroll
        for (int i = 0; i < G * 8; i++)
            m = __hmax2(m, __habs2(reinterpret_cast<const __half2 *>(&u[i / 8][i / 4 % 2])[i % 4]));
        big = fmaxf(__low2float(m), __high2float(m));
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const int e = max(-100, min(100, (int)(__float_as_uint(big) >> 23) - 127));
    const float scale = __uint_as_float((uint32_t)(127 + 14 - e) << 23), s16 = scale * 0.0625f;
    // 2^(24 - 14 + e) and its reciprocal
    const float unit = __uint_as_float((uint32_t)(127 + 10 + e) << 23);
    const float per = __uint_as_float((uint32_t)(127 - 10 - e) << 23);
#pragma unroll
    for (int gr = 0; gr < G; gr++) {
        sum[gr] = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            float w[8];
            if (bf16)
                load8<__nv_bfloat16>(u[gr][j], w);
            else
                load8<__half>(u[gr][j], w);
            qf[gr][j][0] = pack_half2(w[0] * scale, w[4] * scale);
            qf[gr][j][1] = pack_half2(w[1] * s16, w[5] * s16);
            qf[gr][j][2] = pack_half2(w[2] * scale, w[6] * scale);
            qf[gr][j][3] = pack_half2(w[3] * s16, w[7] * s16);
            sum[gr] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
        }
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
        sum[gr] = (sum[gr] + __shfl_xor_sync(0xffffffffu, sum[gr], 2)) * per;
    }
    return unit;
}

// Segments of a sequence (key heads x row blocks) and tiles of each; at least one tile where it
// has queries, so that queries without keys are written too.
template <int D, int NT, bool FOLD>
__device__ __forceinline__ int sequence(const Params &p, int s, int &row0, int &n, int &len, int &nt, int &nrb)
{
    using C = Cfg<D, NT, FOLD>;
    int a, b;
    nt = nrb = 0;
    if (!p.a.s.rows(s, a, b, len))
        return 0;
    row0 = a;
    n = b - a;
    if (n == 0)
        return 0;
    if (n > p.a.max_q) {
        atomicOr(p.a.s.status, status_bit(SAGE_ERR_BAD_SEQLENS));
        return 0;
    }
    nt = max(1, (int)(((uint32_t)len + C::kTile - 1) / C::kTile));   // (len may be 2^31 - 1)
    nrb = (n * p.group + C::kRows - 1) / C::kRows;
    return nrb * p.a.s.Hkv;
}

// A walk over the segments (sequence, key head, row block, range of tiles) of a share [from, to)
// of the list, in which a segment is `cost` places of start-up and its tiles.
template <int D, int NT, bool FOLD>
struct Walk {
    int64_t x, to;                    // where the segment begins in the list, and the share ends
    int cost, s, row0, n, len, nt, nrb;   // the sequence
    int kvh, rb, t0, t1;              // the segment; t0 == t1: nothing of it is in the share
    bool live;                        // there is a segment

    __device__ void start(const Params &p, int start_cost, int64_t from, int64_t end, int seq, int64_t offset)
    {
        cost = start_cost;
        to = end;
        s = seq;
        sequence<D, NT, FOLD>(p, s, row0, n, len, nt, nrb);
        const int each = nt + cost, h = (int)(offset / each), at = (int)(offset % each);
        x = from - at;
        kvh = h / nrb;
        rb = h % nrb;
        t0 = max(0, at - cost);
        t1 = (int)min((int64_t)nt, max((int64_t)t0, to - x - cost));
        live = true;
        if (t0 >= t1)
            next(p);
    }
    __device__ void next(const Params &p)
    {
        x += nt + cost;
        live = false;
        if (x + cost >= to)
            return;
        if (++rb == nrb) {
            rb = 0;
            if (++kvh == p.a.s.Hkv) {
                kvh = 0;
                do {
                    if (++s >= p.a.s.nseq)
                        return;
                } while (sequence<D, NT, FOLD>(p, s, row0, n, len, nt, nrb) == 0);
            }
        }
        t0 = 0;
        t1 = (int)min((int64_t)nt, to - x - cost);
        live = true;
    }
};

__device__ __forceinline__ int64_t block_sum_scan(int64_t v, int64_t *s_warp, int64_t &total)
{
    // inclusive scan over the CTA
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += u;
    }
    __syncthreads();
    if (lane == 31)
        s_warp[warp] = v;
    __syncthreads();
    total = 0;
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < warp)
            before += s_warp[w];
        total += s_warp[w];
    }
    return v + before;
}

template <int D, int NT, bool FOLD>
__global__ void __launch_bounds__(kThreads, (Cfg<D, NT, FOLD>::kCtasPerSM)) kv4_attn_kernel(const Params p)
{
    using C = Cfg<D, NT, FOLD>;
    constexpr int kG = C::kGroups, kKB = C::kTile / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[kWarps];
    __shared__ int64_t s_x[kWarps + 1], s_from[kWarps];
    __shared__ int s_seq[kWarps], s_segments;
    __shared__ Walk<D, NT, FOLD> s_walk[2 * kWarps];
    float *s_o = reinterpret_cast<float *>(smem + C::kRing);
    float *kpar = s_o + kWarps * C::kRows * C::kPitch + threadIdx.x / 32 * (2 * C::kFloats);   // this warp's
    float *vpar = kpar + C::kFloats;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t4 = lane % 4;
    const int cta = blockIdx.x;
    if (tid == 0)
        s_segments = 0;
    __syncthreads();
    griddep_wait();

    // ---- the list of work: how many segments, how long, and this CTA's or warp's share
    const Kv4Seqs &sq = p.a.s;
    int row0, n, len, nt0 = 0, nt, nrb, segs0 = 0;
    for (int i = tid; i < sq.nseq; i += kThreads) {
        const int segs = sequence<D, NT, FOLD>(p, i, row0, n, len, nt, nrb);
        if (i == tid) {
            segs0 = segs;
            nt0 = nt;
        }
        if (segs)
            atomicAdd(&s_segments, min(segs, kSoloSegments));
    }
    __syncthreads();
    const bool solo = s_segments >= kSoloSegments;
    const int cost = solo ? kSoloCost : kTeamCost;
    auto places = [&](int i) -> int64_t {
        if (i == tid)
            return (int64_t)segs0 * (nt0 + cost);
        if (i >= sq.nseq)
            return 0;
        const int segs = sequence<D, NT, FOLD>(p, i, row0, n, len, nt, nrb);
        return (int64_t)segs * (nt + cost);
    };
    int64_t total = 0;
    for (int base = 0; base < sq.nseq; base += kThreads) {
        int64_t all;
        block_sum_scan(places(base + tid), s_scan, all);
        total += all;
    }
    const int64_t teams = max((int64_t)1, min((int64_t)gridDim.x * (solo ? kWarps : 1),
                                              total / (solo ? 1 + kSoloCost : kWarps)));
    const int team = solo ? cta * kWarps + warp : cta;
    if (tid <= kWarps) {
        const int64_t t = solo ? cta * kWarps + tid : cta + (tid > 0);
        s_x[tid] = t < teams ? total * t / teams : total;
    }
    if (cta == 0 && tid == 0)
        *p.solo = solo;
    __syncthreads();
    if (s_x[0] >= s_x[kWarps]) {
        if (lane == 0 && (solo || warp == 0))
            p.tail[team].last = -1;
        return;
    }
    int64_t sum = 0;
    for (int base = 0; base < sq.nseq; base += kThreads) {
        int64_t all;
        const int64_t v = places(base + tid), end = sum + block_sum_scan(v, s_scan, all);
#pragma unroll
        for (int w = 0; w < kWarps; w++)
            if (end - v <= s_x[w] && s_x[w] < end) {
                s_seq[w] = base + tid;
                s_from[w] = end - v;
            }
        sum += all;
    }
    __syncthreads();
    griddep_launch_dependents();

    // the walks live in shared memory: what a warp (solo) or the CTA works on, [0] and in turn
    // [1] there, then what each warp fetches, which is up to kStages tiles ahead
    const int step = solo ? 1 : kWarps, place = solo ? 0 : warp;   // of the tiles, this warp's
    Walk<D, NT, FOLD> *now = s_walk + (solo ? warp : 0);
    Tail tail{-1, 0, 0, 0, 0};
    if (lane == 0 && (solo || warp == 0)) {
        now->live = false;
        if (s_x[warp] < s_x[warp + 1])
            now->start(p, cost, s_x[warp], s_x[warp + 1], s_seq[warp], s_x[warp] - s_from[warp]);
    }
    __syncthreads();

    // ---- the warp's ring of tiles, filled by 16-byte asynchronous copies of all its lanes (bulk
    // copies take their operands from the warp, so lanes that copy a page each issue in turn: 6%
    // slower)
    uint8_t *ring = smem + warp * (C::kStages * C::kStageBytes);
    const uint32_t ring_at = smem_u32(ring) + lane * 16;
    const int ps = sq.page_size();
    const int64_t page_bytes = kv4_page_bytes(ps, D);
    const uint32_t page_stride = (uint32_t)(sq.Hkv * page_bytes);   // at most 65535 heads of 36864 bytes
    const int slice = min(ps, C::kTile);               // keys of a tile that one page holds
    const int slice_log2 = 31 - __clz(slice);
    // this lane's 16 bytes of a page's first rows (256 / D of a row's codes), and of its
    // params (lanes 0-15 the keys', 16-31 the values')
    constexpr int kRowStep = 1024 / D;                 // rows of codes that 512 bytes hold
    const int code_row = lane / (D / 32), par_row = lane % 16 * (4 / kG);
    const int par_off = ps * D + (lane / 16) * (ps * kG * 4) + lane % 16 * 16 - lane * 16;
    const uint8_t *const cache_at = sq.cache + lane * 16;
    const uint8_t *head;                               // this lane's part of the segment's head in page 0
    const int32_t *table;                              // of the segment's sequence
    int next_tile, end_tile, keys, ids = 0, stage_in = 0;
    bool more = true;
    auto enter = [&](const Walk<D, NT, FOLD> &w) {
        more = w.live;
        next_tile = w.t0 + place;
        end_tile = w.t1;
        keys = w.len;
        table = sq.block_table + (int64_t)w.s * sq.max_pages;
        head = cache_at + w.kvh * page_bytes;
    };
    // steps to the warp's next tile and looks up its pages (lane i: the i-th), one tile ahead
    // of their use
    auto advance = [&]() {
        if (next_tile >= end_tile) {
            Walk<D, NT, FOLD> w = s_walk[kWarps + warp];
            do {
                w.next(p);
                enter(w);
            } while (more && next_tile >= end_tile);
            __syncwarp();
            if (lane == 0)
                s_walk[kWarps + warp] = w;
            __syncwarp();
        }
        const int key = next_tile * C::kTile + lane * slice;
        ids = 0;
        if (more && lane * slice < C::kTile && key < keys)
            ids = table[key >> sq.page_log2];
    };
    auto issue = [&]() {
        if (more) {
            const int k0 = next_tile * C::kTile, left = keys - k0;
            const uint32_t dst = ring_at + stage_in;
            // a table entry that is no page: its status bit is set and page 0 read in its place
            if ((uint32_t)ids >= (uint32_t)sq.num_pages) {
                atomicOr(sq.status, status_bit(SAGE_ERR_BAD_PAGE));
                ids = 0;
            }
            if (left >= C::kTile && slice == C::kTile) {       // a whole tile of one page
                const int row = k0 & (ps - 1);
                const uint8_t *src = head + (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, ids, 0) * page_stride;
                const uint8_t *kc = src + row * (D / 2), *vc = kc + ps * (D / 2);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    copy16(dst + i * 512, kc + i * 512);
                    copy16(dst + C::kTile * (D / 2) + i * 512, vc + i * 512);
                }
                copy16(dst + C::kTile * D, src + par_off + row * (kG * 4));
            } else {
                // of whole pages (slice < kTile), or the sequence's last rows: copy i holds rows
                // i kRowStep to (i + 1) kRowStep - 1, all in slice i kRowStep / slice
                const int row0 = k0 & (ps - 1);                // not 0 only where slice == kTile
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t id = __shfl_sync(0xffffffffu, ids, i * kRowStep >> slice_log2);
                    const uint8_t *kc = head + (uint64_t)id * page_stride + (row0 + (i * kRowStep & (slice - 1))) * (D / 2);
                    if (i * kRowStep + code_row < left) {
                        copy16(dst + i * 512, kc);
                        copy16(dst + C::kTile * (D / 2) + i * 512, kc + ps * (D / 2));
                    }
                }
                const uint32_t id = __shfl_sync(0xffffffffu, ids, par_row >> slice_log2);
                if (par_row < left)
                    copy16(dst + C::kTile * D, head + (uint64_t)id * page_stride + par_off +
                                                   (row0 - (par_row & ~(slice - 1))) * (kG * 4));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        stage_in ^= C::kStageBytes;
        next_tile += step;
        if (more)
            advance();
    };
    if (lane == 0)
        s_walk[kWarps + warp] = *now;
    __syncwarp();
    enter(*now);
    if (more)
        advance();
#pragma unroll 1
    for (int i = 0; i < C::kStages; i++)
        issue();
    int stage_out = 0;

    while (now->live) {
        const Walk<D, NT, FOLD> &seg = *now;
        const int end = seg.t1, len = seg.len;
        // ---- the segment's queries: row r of the block is query r / group, head r % group
        const int r0 = seg.rb * C::kRows, nrows = min(C::kRows, seg.n * p.group - r0);
        uint32_t qf[NT][kG][2][4];
        float f[NT][2], qs[NT][kG][2];
        int lim[NT][2];
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const int r = FOLD ? g % 4 : i * 8 + g;
            const int qi = (r0 + r) / p.group, hh = (r0 + r) % p.group;
            const uint16_t *src = static_cast<const uint16_t *>(p.a.q) + (int64_t)(seg.row0 + qi) * p.a.q_tok +
                                  (int64_t)(seg.kvh * p.group + hh) * p.a.q_head + t4 * 16;
            uint4 u[kG][2];
#pragma unroll
            for (int gr = 0; gr < kG; gr++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    u[gr][j] = r < nrows ? reinterpret_cast<const uint4 *>(src + gr * 64)[j]
                                         : make_uint4(0u, 0u, 0u, 0u);
            float sum[kG];
            f[i][0] = f[i][1] = query_row<kG>(u, p.a.bf16, qf[i], sum);
#pragma unroll
            for (int gr = 0; gr < kG; gr++) {
                qs[i][gr][0] = __shfl_sync(0xffffffffu, sum[gr], t4 * 8);
                qs[i][gr][1] = __shfl_sync(0xffffffffu, sum[gr], t4 * 8 + 4);
            }
            // not 0, however small the row and the scale: a hidden score, -inf, times 0 is NaN
            const float least = __uint_as_float(1u << 23);
            f[i][0] = fmaxf(__shfl_sync(0xffffffffu, f[i][0], t4 * 8) * p.sc_log2, least);
            f[i][1] = fmaxf(__shfl_sync(0xffffffffu, f[i][1], t4 * 8 + 4) * p.sc_log2, least);
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const int rr = FOLD ? (2 * t4 + c) % 4 : i * 8 + 2 * t4 + c;
                lim[i][c] = p.a.causal && rr < nrows ? len - seg.n + (r0 + rr) / p.group : len - 1;
            }
        }
        // keys up to here are seen by every row of the block
        const int seen = p.a.causal ? min(len - 1, len - seg.n + r0 / p.group) : len - 1;

        float nm[NT][2], l[NT][2], o2[NT][kG][2], o[NT][kG][4][4];   // nm: -m
#pragma unroll
        for (int i = 0; i < NT; i++) {
#pragma unroll
            for (int c = 0; c < 2; c++) {
                nm[i][c] = INFINITY;
                l[i][c] = 0.0f;
            }
#pragma unroll
            for (int gr = 0; gr < kG; gr++) {
                o2[i][gr][0] = o2[i][gr][1] = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        o[i][gr][j][c] = 0.0f;
            }
        }
        const float2 low_sel = t4 < 2 ? make_float2(0.0f, 0.0f) : make_float2(-1.0f, -1.0f);
        // what the value products are scaled by, for each group of channels, so that a group of small
        // values keeps its bits beside one of large ones, and the steps (as fp16 bits) from which on
        // they are too large for it: 4 exponents above the one it is made for; 0: for none yet
        uint32_t vlimit[kG];
        float vscale[kG];
#pragma unroll
        for (int gr = 0; gr < kG; gr++) {
            vlimit[gr] = 0;
            vscale[gr] = 1.0f;
        }

        for (int t = seg.t0 + place; t < end; t += step) {
            const int k0 = t * C::kTile;
            const uint8_t *st = ring + stage_out;
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
            __syncwarp();                              // every lane's part has landed
            auto tile = [&](auto hides) {
                constexpr bool masked = decltype(hides)::value;

                // ---- scores, S^T: rows are keys, columns query rows; s f is the base-2 logit
                float s[kKB][NT][4];
                // the keys' params to fp32, two groups a lane, for the four lanes that share a key
                {
                    const uint2 u = reinterpret_cast<const uint2 *>(st + C::kTile * D)[lane];
                    const float2 x = __half22float2(bits_h2(u.x)), y = __half22float2(bits_h2(u.y));
                    reinterpret_cast<float4 *>(kpar)[lane] = make_float4(x.x, x.y, y.x, y.y);
                    __syncwarp();
                }
#pragma unroll
                for (int kb = 0; kb < kKB; kb++) {
                    const uint8_t *r0p = st + (kb * 16 + g) * (D / 2) + t4 * 8;
                    const uint8_t *r1p = r0p + 8 * (D / 2);
                    float2 p0[kG], p1[kG];
                    load_params<kG>(kpar + (kb * 16 + g) * (2 * kG), p0);
                    load_params<kG>(kpar + (kb * 16 + g + 8) * (2 * kG), p1);
#pragma unroll
                    for (int gr = 0; gr < kG; gr++) {
                        const uint2 w0 = *reinterpret_cast<const uint2 *>(r0p + gr * 32);
                        const uint2 w1 = *reinterpret_cast<const uint2 *>(r1p + gr * 32);
                        float acc[NT][4];
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            uint32_t u0 = j ? w0.y : w0.x, u1 = j ? w1.y : w1.x;
#pragma unroll
                            for (int hf = 0; hf < 2; hf++) {
                                const uint32_t a0 = u0 & 0x000F000Fu, a1 = u1 & 0x000F000Fu;
                                const uint32_t a2 = u0 & 0x00F000F0u, a3 = u1 & 0x00F000F0u;
#pragma unroll
                                for (int i = 0; i < NT; i++)
                                    if (j == 0 && hf == 0)
                                        mma16816_first(acc[i], a0, a1, a2, a3, qf[i][gr][0][0], qf[i][gr][0][1]);
                                    else
                                        mma16816(acc[i], a0, a1, a2, a3, qf[i][gr][j][2 * hf],
                                                 qf[i][gr][j][2 * hf + 1]);
                                u0 >>= 8;
                                u1 >>= 8;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < NT; i++)
#pragma unroll
                            for (int c = 0; c < 4; c++) {
                                const float2 pr = c < 2 ? p0[gr] : p1[gr];
                                const float sum = qs[i][gr][c & 1];
                                const float low = gr == 0 ? pr.y * sum : fmaf(pr.y, sum, s[kb][i][c]);
                                s[kb][i][c] = fmaf(pr.x, acc[i][c], low);
                            }
                    }
                }
                uint32_t hidden = 0;                       // of this lane's scores, bit kb*NT*4 + ...
                if (masked) {
#pragma unroll
                    for (int kb = 0; kb < kKB; kb++)
#pragma unroll
                        for (int i = 0; i < NT; i++)
#pragma unroll
                            for (int c = 0; c < 4; c++)
                                if (k0 + kb * 16 + g + (c >> 1) * 8 > lim[i][c & 1]) {
                                    s[kb][i][c] = -INFINITY;
                                    hidden |= 1u << ((kb * NT + i) * 4 + c);
                                }
                }

                // ---- the reference m that probabilities are taken relative to moves only when a
                // logit is more than 8 above it, so p <= 2^8
                float x[NT][2];
                bool move = false;
#pragma unroll
                for (int i = 0; i < NT; i++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        x[i][c] = fmaxf(s[0][i][c], s[0][i][c + 2]);
#pragma unroll
                        for (int kb = 1; kb < kKB; kb++)
                            x[i][c] = fmaxf(x[i][c], fmaxf(s[kb][i][c], s[kb][i][c + 2]));
                        move |= fmaf(x[i][c], f[i][c], nm[i][c]) > 8.0f;
                    }
                // ---- the tile's largest value steps: products p * step are scaled by a power of two
                // that keeps them below 2^15, whatever V's size. In a masked tile, rows behind the last
                // token and non-finite steps do not count (elsewhere every row sees every step)
                const uint2 vraw = reinterpret_cast<const uint2 *>(st + C::kTile * D + C::kParBytes)[lane];
                uint2 vs = make_uint2(vraw.x & 0x7FFFu, vraw.y & 0x7FFFu);
                if (masked) {
                    if (vs.x >= 0x7C00u || k0 + 2 * lane / kG >= len)
                        vs.x = 0;
                    if (vs.y >= 0x7C00u || k0 + (2 * lane + 1) / kG >= len)
                        vs.y = 0;
                }
                // this lane's two steps: the groups of one key, or two keys' (D = 64)
                const uint32_t vtop[2] = {kG == 2 ? vs.x : max(vs.x, vs.y), kG == 2 ? vs.y : 0u};
                if (__any_sync(0xffffffffu, move || vtop[0] >= vlimit[0] || (kG == 2 && vtop[1] >= vlimit[kG - 1]))) {
                    float shift[kG];
#pragma unroll
                    for (int gr = 0; gr < kG; gr++) {
                        const int texp = (int)(__reduce_max_sync(0xffffffffu, vtop[gr]) >> 10);
                        shift[gr] = 1.0f;
                        const int vexp = (int)(vlimit[gr] >> 10) - 4;
                        if (texp > vexp + 3) {
                            shift[gr] = vexp < 0 ? 0.0f : __uint_as_float((uint32_t)(127 + vexp - texp) << 23);
                            vlimit[gr] = (uint32_t)(texp + 4) << 10;
                            vscale[gr] = __uint_as_float((uint32_t)(127 + 18 - texp) << 23);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NT; i++)
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            float y = x[i][c], alpha = 1.0f;
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16)) * f[i][c];
                            if (y > -nm[i][c]) {           // (rows that have seen no key: -inf on both sides)
                                alpha = ex2_approx(-nm[i][c] - y);
                                nm[i][c] = -y;
                            }
                            l[i][c] *= alpha;
#pragma unroll
                            for (int gr = 0; gr < kG; gr++) {
                                o2[i][gr][c] *= alpha;
#pragma unroll
                                for (int j = 0; j < 4; j++) {
                                    o[i][gr][j][c] *= alpha * shift[gr];
                                    o[i][gr][j][c + 2] *= alpha * shift[gr];
                                }
                            }
                        }
                }

                // the values' params: step so scaled, and the middle low + 8 step
                {
                    const float2 x = __half22float2(bits_h2(vraw.x)), y = __half22float2(bits_h2(vraw.y));
                    reinterpret_cast<float4 *>(vpar)[lane] =
                        make_float4(x.x * vscale[0], fmaf(8.0f, x.x, x.y), y.x * vscale[kG - 1], fmaf(8.0f, y.x, y.y));
                    __syncwarp();
                }

                // ---- probabilities and O^T += V^T P^T: rows are channels, columns query rows
                float centre[NT][kG][4];
#pragma unroll
                for (int kb = 0; kb < kKB; kb++) {
#pragma unroll
                    for (int i = 0; i < NT; i++) {
                        const float2 ff = make_float2(f[i][0], f[i][1]);
                        // a row that has seen no key yet: 2^(-inf + 0)
                        const float2 nn = make_float2(nm[i][0] == INFINITY ? 0.0f : nm[i][0],
                                                      nm[i][1] == INFINITY ? 0.0f : nm[i][1]);
                        const float2 ta = fma2(make_float2(s[kb][i][0], s[kb][i][1]), ff, nn);
                        const float2 tb = fma2(make_float2(s[kb][i][2], s[kb][i][3]), ff, nn);
                        s[kb][i][0] = ex2_approx(ta.x);
                        s[kb][i][1] = ex2_approx(ta.y);
                        s[kb][i][2] = ex2_approx(tb.x);
                        s[kb][i][3] = ex2_approx(tb.y);
                        const float2 ls = add2(make_float2(s[kb][i][0], s[kb][i][1]),
                                               make_float2(s[kb][i][2], s[kb][i][3]));
                        const float2 lt = add2(make_float2(l[i][0], l[i][1]), ls);
                        l[i][0] = lt.x;
                        l[i][1] = lt.y;
                    }
                    const uint8_t *vr = st + (C::kTile + kb * 16 + 2 * t4) * (D / 2) + g * 4;
                    float2 p0[kG], p1[kG];
                    load_params<kG>(vpar + (kb * 16 + g) * (2 * kG), p0);
                    load_params<kG>(vpar + (kb * 16 + g + 8) * (2 * kG), p1);
#pragma unroll
                    for (int gr = 0; gr < kG; gr++) {
                        const float step0 = p0[gr].x, step1 = p1[gr].x, mid0 = p0[gr].y, mid1 = p1[gr].y;
                        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
                        for (int i = 0; i < NT; i++) {
                            float pv[4];
#pragma unroll
                            for (int c = 0; c < 4; c++)
                                pv[c] = s[kb][i][c] * (c < 2 ? step0 : step1);
                            if (masked) {                  // 0 times what lies in a hidden place is 0
#pragma unroll
                                for (int c = 0; c < 4; c++) {
                                    const bool hid = hidden >> ((kb * NT + i) * 4 + c) & 1;
                                    pv[c] = hid ? 0.0f : pv[c];
                                    o2[i][gr][c & 1] = hid ? o2[i][gr][c & 1]
                                                           : fmaf(s[kb][i][c], c < 2 ? mid0 : mid1, o2[i][gr][c & 1]);
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < 4; c++)
                                    o2[i][gr][c & 1] = fmaf(s[kb][i][c], c < 2 ? mid0 : mid1, o2[i][gr][c & 1]);
                            }
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const float2 v = make_float2(pv[2 * h], pv[2 * h + 1]);
                                const __half2 a = __floats2half2_rn(v.x, v.y);
                                // FOLD: this lane's columns take the high term (0) or the low one (-1)
                                const float2 d = fma2(__half22float2(a), FOLD ? low_sel : make_float2(-1.0f, -1.0f), v);
                                hi[i][h] = transpose8x8(FOLD ? pack_half2(d.x, d.y) : h2_bits(a));
                                if (!FOLD)
                                    lo[i][h] = transpose8x8(pack_half2(d.x, d.y));
                            }
                        }
                        // keys 2t, 2t+1 (A, B) and 2t+8, 2t+9 (C, D) of the block; 8 channels each
                        const uint32_t wa = *reinterpret_cast<const uint32_t *>(vr + gr * 32);
                        const uint32_t wb = *reinterpret_cast<const uint32_t *>(vr + gr * 32 + D / 2);
                        const uint32_t wc = *reinterpret_cast<const uint32_t *>(vr + gr * 32 + 8 * (D / 2));
                        const uint32_t wd = *reinterpret_cast<const uint32_t *>(vr + gr * 32 + 9 * (D / 2));
                        // minus 8 (and 128) for every code of the block, into sums of their own
#pragma unroll
                        for (int i = 0; i < NT; i++) {
                            if (kb == 0)
                                mma16816_first(centre[i][gr], kMinus8, kMinus128, kMinus8, kMinus128, hi[i][0],
                                               hi[i][1]);
                            else
                                mma16816(centre[i][gr], kMinus8, kMinus128, kMinus8, kMinus128, hi[i][0], hi[i][1]);
                            if (!FOLD)
                                mma16816(centre[i][gr], kMinus8, kMinus128, kMinus8, kMinus128, lo[i][0], lo[i][1]);
                        }
#pragma unroll
                        for (int q = 0; q < 2; q++) {      // channels 0-3, then 4-7 of the word
                            uint32_t ab = __byte_perm(wa, wb, q ? 0x7632 : 0x5410);
                            uint32_t cd = __byte_perm(wc, wd, q ? 0x7632 : 0x5410);
#pragma unroll
                            for (int e = 0; e < 2; e++) {
                                const uint32_t a0 = ab & 0x000F000Fu, a1 = ab & 0x00F000F0u;
                                const uint32_t a2 = cd & 0x000F000Fu, a3 = cd & 0x00F000F0u;
#pragma unroll
                                for (int i = 0; i < NT; i++) {
                                    mma16816(o[i][gr][2 * q + e], a0, a1, a2, a3, hi[i][0], hi[i][1]);
                                    if (!FOLD)
                                        mma16816(o[i][gr][2 * q + e], a0, a1, a2, a3, lo[i][0], lo[i][1]);
                                }
                                ab >>= 8;
                                cd >>= 8;
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; i++)
#pragma unroll
                    for (int gr = 0; gr < kG; gr++)
#pragma unroll
                        for (int j = 0; j < 4; j++)
#pragma unroll
                            for (int c = 0; c < 4; c += 2) {
                                const float2 y = add2(make_float2(o[i][gr][j][c], o[i][gr][j][c + 1]),
                                                      make_float2(centre[i][gr][c], centre[i][gr][c + 1]));
                                o[i][gr][j][c] = y.x;
                                o[i][gr][j][c + 1] = y.y;
                            }
            };
            if (k0 + C::kTile - 1 > seen)
                tile(std::true_type{});
            else
                tile(std::false_type{});
            __syncwarp();                              // the stage is read
            stage_out ^= C::kStageBytes;
            issue();
        }

        const bool whole = seg.t0 == 0 && seg.t1 == seg.nt;
        if (!whole && seg.t0 == 0) {
            // the list's place behind the segment's last tile lies in the share of team
            // ceil(place teams / total) - 1
            const int64_t last = seg.x + cost + seg.nt;
            tail = Tail{(int)((last * teams + total - 1) / total) - 1, seg.row0, seg.n, seg.kvh, seg.rb};
        }
        float unscale[kG];
#pragma unroll
        for (int gr = 0; gr < kG; gr++)
            unscale[gr] = vlimit[gr] == 0 ? 0.0f : __uint_as_float((127u + 2 + (vlimit[gr] >> 10)) << 23);
        float *const part = p.part + (int64_t)(team * 2 + (seg.t0 == 0)) * (C::kRows * C::kPitch);
#pragma unroll
        for (int i = 0; i < NT; i++) {
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const int r = FOLD ? (2 * t4 + c) % 4 : i * 8 + 2 * t4 + c;
                float lw = l[i][c], ow[kG];
#pragma unroll
                for (int gr = 0; gr < kG; gr++)
                    ow[gr] = o2[i][gr][c];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    lw += __shfl_xor_sync(0xffffffffu, lw, x);
#pragma unroll
                    for (int gr = 0; gr < kG; gr++)
                        ow[gr] += __shfl_xor_sync(0xffffffffu, ow[gr], x);
                }
                // FOLD: the low terms' columns (t4 >= 2) join the high ones'
                float v[kG][8];
#pragma unroll
                for (int gr = 0; gr < kG; gr++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            float y = o[i][gr][j][c + 2 * e];
                            if (FOLD)
                                y += __shfl_xor_sync(0xffffffffu, y, 2);
                            v[gr][2 * j + e] = fmaf(y, e ? unscale[gr] * 0.0625f : unscale[gr], ow[gr]);
                        }
                if (r >= nrows || (FOLD && t4 >= 2))
                    continue;
                if (solo && whole) {
                    const float inv = lw == 0.0f ? 0.0f : 1.0f / lw;
                    const int64_t row = seg.row0 + (r0 + r) / p.group;
                    const int hh = seg.kvh * p.group + (r0 + r) % p.group;
                    uint16_t *out = static_cast<uint16_t *>(p.a.out) + (row * p.a.Hq + hh) * D + g * 8;
#pragma unroll
                    for (int gr = 0; gr < kG; gr++) {
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            v[gr][e] *= inv;
                        *reinterpret_cast<uint4 *>(out + gr * 64) =
                            p.a.bf16 ? store8<__nv_bfloat16>(v[gr]) : store8<__half>(v[gr]);
                    }
                    if (g == 0 && p.a.lse)
                        p.a.lse[row * p.a.Hq + hh] = lw == 0.0f ? -INFINITY : (log2f(lw) - nm[i][c]) * kLn2;
                } else {
                    // to the workspace, or (CTA) to shared memory, where the warps are merged
                    float *dst = solo ? part + r * C::kPitch : s_o + (warp * C::kRows + r) * C::kPitch;
#pragma unroll
                    for (int gr = 0; gr < kG; gr++)
#pragma unroll
                        for (int h = 0; h < 2; h++)
                            *reinterpret_cast<float4 *>(dst + gr * 64 + g * 8 + 4 * h) =
                                make_float4(v[gr][4 * h], v[gr][4 * h + 1], v[gr][4 * h + 2], v[gr][4 * h + 3]);
                    if (g == 0)
                        *reinterpret_cast<float2 *>(dst + D) = make_float2(-nm[i][c], lw);
                }
            }
        }
        if (solo) {
            __syncwarp();
            if (lane == 0)
                now->next(p);
            __syncwarp();
            continue;
        }
        __syncthreads();
        Walk<D, NT, FOLD> *const then = s_walk + (now == s_walk);
        if (tid == kThreads - 1) {
            *then = seg;
            then->next(p);
        }
        for (int e = tid; e < nrows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c4 = e % (D / 4) * 4;
            const float *at = s_o + r * C::kPitch;
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; w++)
                M = fmaxf(M, at[w * C::kRows * C::kPitch + D]);
            const float b = M == -INFINITY ? 0.0f : M;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float *x = at + w * C::kRows * C::kPitch;
                const float2 ml = *reinterpret_cast<const float2 *>(x + D);
                const float4 v = *reinterpret_cast<const float4 *>(x + c4);
                const float wt = ex2_approx(ml.x - b);
                L = fmaf(wt, ml.y, L);
                acc.x = fmaf(wt, v.x, acc.x);
                acc.y = fmaf(wt, v.y, acc.y);
                acc.z = fmaf(wt, v.z, acc.z);
                acc.w = fmaf(wt, v.w, acc.w);
            }
            if (whole) {
                const int64_t row = seg.row0 + (r0 + r) / p.group;
                write_row<4>(p.a, row, seg.kvh * p.group + (r0 + r) % p.group, D, c4, M, L,
                             reinterpret_cast<const float *>(&acc));
            } else {
                *reinterpret_cast<float4 *>(part + r * C::kPitch + c4) = acc;
                if (c4 == 0)
                    *reinterpret_cast<float2 *>(part + r * C::kPitch + D) = make_float2(M, L);
            }
        }
        __syncthreads();                               // the merge buffer is free again
        now = then;
    }
    if (lane == 0 && (solo || warp == 0))
        p.tail[team] = tail;
}

// Merge of what several teams share: a CTA takes the segment that team blockIdx.x began and did
// not finish, or, where teams are warps and rows at most 8, each half of it one such segment; a
// segment of many CTAs has several CTAs here, a slice of the rows each.
// Its warps take the rows, several a row where the rows are few, eight partials at a time (all
// their loads in flight together), always in the same order.
template <int D, int NT, bool FOLD>
__global__ void __launch_bounds__(kMergeWarps * 32) kv4_attn_merge(const Params p)
{
    using C = Cfg<D, NT, FOLD>;
    constexpr int kC = D / 32, kChunk = 8;             // channels of a lane, partials at a time
    __shared__ __align__(16) float s_part[kMergeWarps][D];
    __shared__ float2 s_ml[kMergeWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32, slot_warp = threadIdx.x / 32;
    const bool solo = *p.solo != 0;
    const int mine = solo && C::kRows <= 8 ? kMergeWarps / 2 : kMergeWarps;   // warps of a segment
    const int teams = C::kCtasPerSM * kSMs;            // of CTAs; their rows go to several CTAs each
    const int team = solo ? blockIdx.x * (kMergeWarps / mine) + slot_warp / mine : blockIdx.x % teams;
    const int warp = slot_warp % mine;
    const Tail t = p.tail[team];
    if (t.last < 0)
        return;
    const int r0 = t.rb * C::kRows;
    int first = 0, nrows = min(C::kRows, t.n * p.group - r0);
    if (!solo) {
        const int slices = gridDim.x / teams, rows = (nrows + slices - 1) / slices;
        first = blockIdx.x / teams * rows;
        nrows = min(nrows, first + rows);
    }
    const int count = nrows - first;
    if (count <= 0)
        return;
    const int split = count <= mine / 8 ? 8 : count <= mine / 4 ? 4 : count <= mine / 2 ? 2 : 1;   // warps of a row
    const int each = (t.last - team + split) / split, part = warp % split;
    const int c0 = team + part * each, c1 = min(t.last + 1, c0 + each);
    for (int base = first; base < nrows; base += mine / split) {
        const int r = base + warp / split;
        float M = -INFINITY, L = 0.0f, acc[kC] = {};
        for (int c = c0; r < nrows && c < c1; c += kChunk) {
            float2 ml[kChunk];
            float v[kChunk][kC];
#pragma unroll
            for (int i = 0; i < kChunk; i++) {
                const bool in = c + i < c1;
                const float *x = p.part + ((int64_t)((in ? c + i : c) * 2 + (c + i == team)) * C::kRows + r) * C::kPitch;
                ml[i] = *reinterpret_cast<const float2 *>(x + D);
                if (!in)
                    ml[i] = make_float2(-INFINITY, 0.0f);
                if constexpr (kC == 4) {
                    *reinterpret_cast<float4 *>(v[i]) = *reinterpret_cast<const float4 *>(x + lane * 4);
                } else {
                    *reinterpret_cast<float2 *>(v[i]) = *reinterpret_cast<const float2 *>(x + lane * 2);
                }
            }
            float m = M;
#pragma unroll
            for (int i = 0; i < kChunk; i++)
                m = fmaxf(m, ml[i].x);
            const float b = m == -INFINITY ? 0.0f : m, scale = ex2_approx(M - b);
            M = m;
            L *= scale;
#pragma unroll
            for (int k = 0; k < kC; k++)
                acc[k] *= scale;
#pragma unroll
            for (int i = 0; i < kChunk; i++) {
                const float w = ex2_approx(ml[i].x - b);
                L = fmaf(w, ml[i].y, L);
#pragma unroll
                for (int k = 0; k < kC; k++)           // a slot read in place of one past the end: no part
                    acc[k] = fmaf(w, c + i < c1 ? v[i][k] : 0.0f, acc[k]);
            }
        }
        if (split > 1) {                               // and then the loop ends here: one barrier is enough
            s_ml[slot_warp] = make_float2(M, L);
#pragma unroll
            for (int k = 0; k < kC; k++)
                s_part[slot_warp][lane * kC + k] = acc[k];
            named_bar_sync(1 + slot_warp / mine, mine * 32);
            if (part)
                continue;
            for (int w = slot_warp + 1; w < slot_warp + split; w++) {
                const float2 o = s_ml[w];
                const float m = fmaxf(M, o.x), b = m == -INFINITY ? 0.0f : m;
                const float sa = ex2_approx(M - b), sb = ex2_approx(o.x - b);
                M = m;
                L = fmaf(sb, o.y, sa * L);
#pragma unroll
                for (int k = 0; k < kC; k++)
                    acc[k] = fmaf(sb, s_part[w][lane * kC + k], sa * acc[k]);
            }
        }
        if (r < nrows)
            write_row<kC>(p.a, t.row0 + (r0 + r) / p.group, t.kvh * p.group + (r0 + r) % p.group, D, lane * kC, M, L,
                          acc);
    }
}

// What takes a call's rows per key head: the folded tile up to 4, else passes of one tile or of
// two, whichever are the fewer at 1.68 times the cost. Of the longest cache below, one row takes
// 252 us folded and 284 in a plain tile; of 64 ragged sequences, 16 rows take 147 us in one pass
// of two tiles and 175 in two of one, 24 rows 268 in two of two and 249 in three of one.
int variant(int Hq, int Hkv, int max_q)
{
    const int rows = max_q * (Hq / Hkv);
    const int ones = (rows + 7) / 8, twos = (rows + 15) / 16;
    return rows <= 4 ? 0 : 100 * ones >= 168 * twos ? 2 : 1;
}
int ctas(int var) { return (var < 2 ? 3 : 2) * kSMs; }
int rows_of(int var) { return 4 << var; }

template <int D, int NT, bool FOLD>
cudaError_t launch(const Params &p, cudaStream_t st)
{
    using C = Cfg<D, NT, FOLD>;
    // once per device: setting it costs a microsecond of every call
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kv4_attn_kernel<D, NT, FOLD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess)
            return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    const int n = C::kCtasPerSM * kSMs;
    e = launch_overlapped(kv4_attn_kernel<D, NT, FOLD>, dim3(n), kThreads, C::kSmem, st, p);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kv4_attn_merge<D, NT, FOLD>, dim3(C::kRows <= 8 ? n * kWarps / 2 : n * kWarps),
                             kMergeWarps * 32, 0, st, p);
}

// [whether solo | tails], then the partial rows, of as many teams as there are warps
size_t tail_bytes(int var) { return (256 + sizeof(Tail) * kWarps * ctas(var) + 255) / 256 * 256; }

}  // namespace

size_t kv4_attn_workspace(int Hq, int Hkv, int max_q, int d)
{
    const int var = variant(Hq, Hkv, max_q);
    return tail_bytes(var) + (size_t)kWarps * ctas(var) * 2 * rows_of(var) * (d + 4) * sizeof(float);
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t st)
{
    const int var = variant(a.Hq, a.s.Hkv, a.max_q);
    Params p;
    p.a = a;
    p.solo = static_cast<int *>(a.workspace);
    p.tail = reinterpret_cast<Tail *>(static_cast<char *>(a.workspace) + 256);
    p.part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + tail_bytes(var));
    p.group = a.Hq / a.s.Hkv;
    p.sc_log2 = a.sm_scale * kLog2e;
    if (a.d == 128)
        return var == 0   ? launch<128, 1, true>(p, st)
               : var == 1 ? launch<128, 1, false>(p, st)
                          : launch<128, 2, false>(p, st);
    return var == 0 ? launch<64, 1, true>(p, st) : var == 1 ? launch<64, 1, false>(p, st) : launch<64, 2, false>(p, st);
}

}  // namespace sage
