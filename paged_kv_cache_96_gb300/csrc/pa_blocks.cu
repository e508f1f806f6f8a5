// pa_blocks.cu -- which blocks of a long context a query row attends: 8-bit bounds
// of every block's keys, and the blocks whose bounds allow the largest score, for
// sm_103a.  An addition to paged attention ("PagedAttention & Continuous Batching"
// §1.4 block table, §1.6, §2.4 decode is memory-bound): a row then reads its selected
// blocks (pa_list_decode.cu) and, of every other block, 2 d + 4 bytes a KV head.
//
// Bounds of block b and KV head kh over its n keys (positions below the context):
//     lo_d = min_p K[p][d], hi_d = max_p K[p][d], a = max_d max(|lo_d|, |hi_d|)
//     code(x) = rint(x * (127 / a)), scale = a * (1 / 127)        (fp32, IEEE)
// a not finite: codes 0, scale +inf; a < 2^-40: codes 0, scale 0.
//
// Score of block b for the row's G query heads, their elements coded the same way
// (codes c_h, scale s_h, each head by itself):
//     I_h = sum_d max(c_h,d lo_d, c_h,d hi_d) = sum_d min(c, 0) lo_d + max(c, 0) hi_d
//     score = max_h fl(s_h I_h) * scale
// the largest q . k that a key within the bounds could have, up to the codes'
// rounding.  I_h is a whole number of magnitude <= 128 * 127^2 < 2^21, so it is exact
// in any order, and with the two rounded fp32 products the score is one number however
// it is computed: what is selected does not depend on tiles or clusters.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include <cooperative_groups.h>

#include "pa_decode_common.cuh"
#include "pa_topk.cuh"

namespace cg = cooperative_groups;

namespace pa {

constexpr float kTiny = 0x1p-40f;  // amplitudes below it count as zero

__device__ __forceinline__ bool finite(float x)
{
    return (__float_as_uint(x) & 0x7fffffffu) < 0x7f800000u;
}

// The codes' factor and the scale of values of amplitude `top` (finite).
struct CodeScale {
    float inv, scale;
};
__device__ __forceinline__ CodeScale code_scale(float top)
{
    if (top < kTiny)
        return {0.f, 0.f};
    return {__fdiv_rn(127.f, top), __fmul_rn(top, 1.f / 127.f)};
}

// ---- bounds ---------------------------------------------------------------------
//
// What bounds it: HBM, each key of a touched block read once (128 contexts, 904 MB of
// keys: 153 us, 93 % of the measured copy rate).  A warp takes one
// (block, KV head): its rows of d keys are runs of 64 to 256 bytes, so a group of
// lanes has one row and the warp several, 16 bytes a lane, eight loads in flight;
// minima and maxima are taken on packed pairs in the pools' own type (FP8 codes as
// the fp16 values they are), which rounds nothing.  Consecutive warps take a block's
// consecutive heads.  The blocks that the step wrote to are numbered through all
// sequences by a scan in every CTA, so that one long prompt among decode rows is
// spread over the device.
struct SummaryParams {
    int8_t *codes;   // [num_blocks][num_kv_heads][2][head_dim]
    float *scales;   // [num_blocks][num_kv_heads]
    const void *key_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;  // [S + 1], or null: whole contexts
    int32_t *error_word;
    int max_blocks_per_seq, num_seqs, num_blocks, block_shift, num_kv_heads;
};

constexpr int kSumThreads = 256;
// Resident CTAs of an SM, which the grid fills once (5, with spilled registers: 160 us).
constexpr int kSumCtas = 4;
constexpr int kSumSeqs = 2 * kSumThreads;  // sequences numbered at once

// First block and number of blocks that the new tokens of sequence s are in.
struct Touched {
    int first, count, ctx;
};
__device__ __forceinline__ Touched touched_blocks(const SummaryParams &p, int s, bool flag)
{
    const int bs = 1 << p.block_shift;
    const long long cap = (long long)p.max_blocks_per_seq << p.block_shift;
    const int limit = (int)min(cap, (long long)INT32_MAX - bs);
    int c = p.context_lens[s];
    bool bad = c < 0 || c > limit;
    c = c < 0 ? 0 : min(c, limit);
    int n = c;
    if (p.query_start != nullptr) {
        const long long rows = (long long)p.query_start[s + 1] - p.query_start[s];
        bad |= rows < 0 || rows > c;
        n = (int)min(max(rows, 0ll), (long long)c);
    }
    if (bad && flag)
        flag_error(p.error_word, PA_DEVERR_CONTEXT_RANGE);
    if (n == 0)
        return {0, 0, c};
    const int first = (c - n) >> p.block_shift;
    return {first, ((c + bs - 1) >> p.block_shift) - first, c};
}

// Packed minimum and maximum that pass a NaN on.
__device__ __forceinline__ __half2 pair_min(__half2 a, __half2 b) { return __hmin2_nan(a, b); }
__device__ __forceinline__ __half2 pair_max(__half2 a, __half2 b) { return __hmax2_nan(a, b); }
__device__ __forceinline__ __nv_bfloat162 pair_min(__nv_bfloat162 a, __nv_bfloat162 b)
{
    return __hmin2_nan(a, b);
}
__device__ __forceinline__ __nv_bfloat162 pair_max(__nv_bfloat162 a, __nv_bfloat162 b)
{
    return __hmax2_nan(a, b);
}
__device__ __forceinline__ float2 pair_float(__half2 x) { return __half22float2(x); }
__device__ __forceinline__ float2 pair_float(__nv_bfloat162 x) { return __bfloat1622float2(x); }

// KV: __half, __nv_bfloat16, or uint8_t (e4m3 codes).
template <typename KV, int D>
__global__ void __launch_bounds__(kSumThreads, kSumCtas)
    summarize_kernel(const __grid_constant__ SummaryParams p)
{
    constexpr bool kFp8 = sizeof(KV) == 1;
    constexpr int kRowBytes = D * (int)sizeof(KV);
    constexpr int kLanes = kRowBytes / 16;  // lanes of a row
    constexpr int kRows = 32 / kLanes;      // rows of a warp's load
    constexpr int kElems = 16 / (int)sizeof(KV);  // elements of a lane
    constexpr int kPairs = kElems / 2;
    constexpr int kBatch = kFp8 ? 4 : 8;    // loads in flight
    using P = typename std::conditional<std::is_same<KV, __nv_bfloat16>::value, __nv_bfloat162,
                                        __half2>::type;
    __shared__ int pref[kSumSeqs + 1], first[kSumSeqs], len[kSumSeqs];
    __shared__ int warp_sum[kSumThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs = 1 << p.block_shift;
    const int part = lane % kLanes, row0 = lane / kLanes;
    pdl_wait_primary();
    pdl_launch_dependents();

    for (int s0 = 0; s0 < p.num_seqs; s0 += kSumSeqs) {
        const int seqs = min(kSumSeqs, p.num_seqs - s0);
        int carry = 0;
        for (int c = 0; c < seqs; c += kSumThreads) {
            const int k = c + tid;
            int n = 0;
            if (k < seqs) {
                const Touched t = touched_blocks(p, s0 + k, blockIdx.x == 0);
                first[k] = t.first;
                len[k] = t.ctx;
                n = t.count;
            }
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o)
                    x += y;
            }
            if (lane == 31)
                warp_sum[warp] = x;
            __syncthreads();
            int before = carry, all = 0;
#pragma unroll
            for (int w = 0; w < kSumThreads / 32; ++w) {
                before += w < warp ? warp_sum[w] : 0;
                all += warp_sum[w];
            }
            if (k < seqs)
                pref[k] = before + x - n;
            carry += all;
            __syncthreads();
        }
        if (tid == 0)
            pref[seqs] = carry;
        __syncthreads();

        // this warp's blocks and heads, in turn: the q-th block of all, KV head kh; the next
        // one's pool block is on its way while one is read
        struct Item {
            int q, kh, live, phys;
        };
        const int K = p.num_kv_heads;
        const int warps = gridDim.x * (kSumThreads / 32);
        const int step_q = warps / K, step_kh = warps - step_q * K;
        auto look_up = [&](Item &x) {
            if (x.q >= carry)
                return;
            int lo_s = 0, n_s = seqs;  // the last sequence with pref <= q
            while (n_s > 1) {
                const int half = n_s >> 1;
                if (pref[lo_s + half] <= x.q) {
                    lo_s += half;
                    n_s -= half;
                } else {
                    n_s = half;
                }
            }
            const int blk = first[lo_s] + x.q - pref[lo_s];
            x.phys = p.block_tables[(size_t)(s0 + lo_s) * p.max_blocks_per_seq + blk];
            x.live = min(bs, len[lo_s] - (blk << p.block_shift));
        };
        auto after = [&](Item x) {
            x.q += step_q;
            x.kh += step_kh;
            if (x.kh >= K) {
                x.kh -= K;
                ++x.q;
            }
            look_up(x);
            return x;
        };
        const int w0 = blockIdx.x * (kSumThreads / 32) + warp;
        Item next{w0 / K, w0 % K, 0, 0};
        look_up(next);
        while (next.q < carry) {
            const Item it = next;
            next = after(it);
            const int kh = it.kh, live = it.live, phys = it.phys;
            if (phys < 0 || phys >= p.num_blocks) {
                if (lane == 0)
                    flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                continue;
            }
            const size_t pitch = (size_t)p.num_kv_heads * kRowBytes;  // token to token
            const uint8_t *at = static_cast<const uint8_t *>(p.key_cache) +
                                ((size_t)phys << p.block_shift) * pitch +
                                (size_t)kh * kRowBytes + part * 16;
            P lo[kPairs], hi[kPairs];
            for (int r = row0; r < live + row0; r += kBatch * kRows) {
                uint4 w[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u)  // (rows past the end repeat the last one)
                    w[u] = *reinterpret_cast<const uint4 *>(
                        at + (size_t)min(r + u * kRows, live - 1) * pitch);
                if (r == row0) {
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        const uint32_t *x = reinterpret_cast<const uint32_t *>(&w[0]);
                        uint32_t v;
                        if constexpr (kFp8)
                            v = e4m3x2_to_f16x2((uint16_t)(x[e / 2] >> (16 * (e & 1))));
                        else
                            v = x[e];
                        lo[e] = hi[e] = *reinterpret_cast<const P *>(&v);
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const uint32_t *x = reinterpret_cast<const uint32_t *>(&w[u]);
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        uint32_t v;
                        if constexpr (kFp8)
                            v = e4m3x2_to_f16x2((uint16_t)(x[e / 2] >> (16 * (e & 1))));
                        else
                            v = x[e];
                        const P y = *reinterpret_cast<const P *>(&v);
                        lo[e] = pair_min(lo[e], y);
                        hi[e] = pair_max(hi[e], y);
                    }
                }
            }
            // the amplitude as 16 bits without a sign, which order finite values, infinities
            // and NaN in this order, in pairs
            uint32_t top2 = 0;
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1) {
                    lo[e] = pair_min(lo[e], __shfl_xor_sync(kFull, lo[e], o));
                    hi[e] = pair_max(hi[e], __shfl_xor_sync(kFull, hi[e], o));
                }
                const uint32_t a = *reinterpret_cast<const uint32_t *>(&lo[e]) & 0x7fff7fffu;
                const uint32_t b = *reinterpret_cast<const uint32_t *>(&hi[e]) & 0x7fff7fffu;
                top2 = __vmaxu2(top2, __vmaxu2(a, b));
            }
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                top2 = __vmaxu2(top2, __shfl_xor_sync(kFull, top2, o));
            const uint32_t bits = max(top2 & 0xffffu, top2 >> 16);
            const uint32_t both = bits | bits << 16;
            const float top = pair_float(*reinterpret_cast<const P *>(&both)).x;
            const bool ok = finite(top);
            const CodeScale cs = ok ? code_scale(top) : CodeScale{0.f, INFINITY};
            const size_t unit = (size_t)phys * p.num_kv_heads + kh;
            if (lane == 0)
                p.scales[unit] = cs.scale;
            if (row0 < 2) {  // the first rows' lanes write lo, the second's hi
                uint32_t out[kElems / 4];
#pragma unroll
                for (int e = 0; e < kPairs; e += 2) {
                    const float2 a0 = pair_float(lo[e]), a1 = pair_float(hi[e]);
                    const float2 b0 = pair_float(lo[e + 1]), b1 = pair_float(hi[e + 1]);
                    const float v[4] = {row0 ? a1.x : a0.x, row0 ? a1.y : a0.y,
                                        row0 ? b1.x : b0.x, row0 ? b1.y : b0.y};
                    uint32_t bytes = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int code = ok ? __float2int_rn(__fmul_rn(v[j], cs.inv)) : 0;
                        bytes |= ((uint32_t)code & 0xffu) << (8 * j);
                    }
                    out[e / 2] = bytes;
                }
                int8_t *dst = p.codes + (unit * 2 + row0) * D + part * kElems;
                if constexpr (kFp8)
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
                else
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0], out[1]);
            }
        }
        __syncthreads();
    }
}

// ---- selection ------------------------------------------------------------------
//
// One CTA, or a cluster of them, per (row, KV head).  What bounds it: the chain of
// dependent trips to memory -- the row's position, its table row, the blocks' codes -- and
// the selection behind it; with many long contexts HBM (2 d + 4 bytes a block).
//  * The candidates' pool blocks are looked up all at once, while the query is coded.  CTAs
//    are small, several on an SM, so that one's selection hides behind the others' loads
//    (copies into rings of shared memory in place of loads to registers leave room for
//    fewer, and a second tile's registers cost what they bring).
//  * The score product runs on the tensor cores as blocks x heads, on the codes as they
//    are (mma m16n8k32 on signed bytes).  A lane's 16 bytes are taken in the order in which
//    they lie (the sum over d is in a permuted order, which whole numbers allow) and
//    multiplied with the coded heads, kept in shared memory in the lanes' order.  Widened
//    to fp16 the same products took as long (21.3 us for 128 decode rows and 33.0 for 24
//    long ones, against 22.0 and 32.3 now) in twice the instructions: they are not the limit.
//  * Each CTA selects from its own candidates as many as are wanted of all, by one warp
//    from its registers where they are few; the first CTA of a cluster selects from those
//    lists, which come to its shared memory.
struct SelectParams {
    int32_t *selected;  // [T][Hkv][top_k]
    const void *query;
    const int8_t *codes;
    const float *scales;
    const int32_t *block_tables;
    const int32_t *token_seq, *token_pos;
    int32_t *error_word;
    int max_blocks_per_seq, num_seqs, num_blocks, block_shift, max_context_len;
    int num_heads, num_kv_heads, group, top_k, num_first, num_last;
};

// Threads of a CTA and CTAs that an SM holds.  Without clusters: 6 of 128 threads 22.0 us
// for 128 decode rows, 4 of 256 21.5 (with the products in fp16 21.2 and 22.1), 8 of 128
// (which spill) 22.8; in clusters, whose first CTA selects from more: 4 of 256 32.3 us for
// 24 rows of up to 4,096 blocks, 6 of 128 37.8.
__host__ __device__ constexpr int sel_threads(bool clusters) { return clusters ? 256 : 128; }
__host__ __device__ constexpr int sel_resident(bool clusters) { return clusters ? 4 : 6; }
// Shared memory of an SM in percent: the L1 takes the loads under way, and a larger share
// than the CTAs need cuts them short (128 decode rows 35 us with all of it, long ones 38).
constexpr int kSelCarveout = 50;
constexpr int kSelWarp = 512;    // candidates of which one warp selects by itself
constexpr int kSelCluster = 8;   // CTAs of a row and KV head, at most
constexpr int kSelShare = 256;   // candidates of a CTA in a cluster, at least

// Keys in the scores' order.  -0 (a negative product beside a scale of 0) is +0: they are
// equal scores, of which the lower block goes first.
__device__ __forceinline__ uint32_t score_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u == 0x80000000u ? u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// d[16 x 8] += a[16 x 32] b[32 x 8] on signed bytes, in 32 bits.
__device__ __forceinline__ void mma_bytes(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct SelectShared {
    float q_scale[16];
    TopkShared<8> topk;
    int above[8], ties[8];
};

// emit(i, place) for each of a warp's 32 keys from i = base on that is selected, in order;
// `above` and `ties` count the ones before.
template <typename Emit>
__device__ __forceinline__ void emit_run(const Threshold &cut, uint32_t key, int base, int end,
                                         int &above, int &ties, const Emit &emit)
{
    const int lane = threadIdx.x & 31, i = base + lane;
    const uint32_t below = (1u << lane) - 1, v = cut.level(key);
    const bool over = i < end && v > cut.prefix, tie = i < end && v == cut.prefix;
    const uint32_t over_m = __ballot_sync(kFull, over), tie_m = __ballot_sync(kFull, tie);
    const int my_ties = ties + __popc(tie_m & below);
    if (over || (tie && my_ties < cut.rest))
        emit(i, above + __popc(over_m & below) + min(my_ties, cut.rest));
    above += __popc(over_m);
    ties += __popc(tie_m);
}

// A warp's selection from at most 32 PER keys.
template <int PER, typename Emit>
__device__ __forceinline__ void warp_select(const uint32_t *keys, int n, int want,
                                            const Emit &emit)
{
    const int lane = threadIdx.x & 31;
    uint32_t key[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j)
        key[j] = 32 * j + lane < n ? keys[32 * j + lane] : 0u;
    const Threshold cut = warp_threshold(key, n, want);
    int above = 0, ties = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j)
        emit_run(cut, key[j], 32 * j, n, above, ties, emit);
}

// emit(i, place) for the `want` largest of keys [0, n), the lower of equal ones, in order
// of i.  By the whole CTA, behind a barrier; its threads come back at their own time.
template <int THREADS, typename Emit>
__device__ __forceinline__ void cta_select(SelectShared &sh, const uint32_t *keys, int n, int want,
                                           const Emit &emit)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (n <= kSelWarp) {
        if (warp == 0 && n <= kSelWarp / 2)
            warp_select<kSelWarp / 64>(keys, n, want, emit);
        else if (warp == 0)
            warp_select<kSelWarp / 32>(keys, n, want, emit);
        return;
    }
    const Threshold cut =
        top_threshold<THREADS, 8>(sh.topk, [&](int i) { return keys[i]; }, n, want);
    const int run = (n + THREADS - 1) / THREADS * 32;  // keys of a warp
    const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
    int above = 0, ties = 0;
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t v = cut.level(keys[i]);
        above += v > cut.prefix;
        ties += v == cut.prefix;
    }
    above = __reduce_add_sync(kFull, above);
    ties = __reduce_add_sync(kFull, ties);
    if (lane == 0) {
        sh.above[warp] = above;
        sh.ties[warp] = ties;
    }
    __syncthreads();
    above = ties = 0;
    for (int w = 0; w < warp; ++w) {
        above += sh.above[w];
        ties += sh.ties[w];
    }
    for (int b = i0; b < i1; b += 32)
        emit_run(cut, b + lane < i1 ? keys[b + lane] : 0u, b, i1, above, ties, emit);
}

// Shared memory of a CTA: the keys of its candidates and, in a cluster's first CTA, the
// lists of all of them.
static size_t select_bytes(int share, int ctas, int want)
{
    return 4 * (size_t)share + (ctas > 1 ? 8 * (size_t)ctas * want : 0);
}

// T: the query's type; NT: heads of a KV head in eights.  kClusters: for clusters of
// several CTAs.
template <typename T, int D, int NT, bool kClusters>
__global__ void __launch_bounds__(sel_threads(kClusters), sel_resident(kClusters) / NT)
    select_kernel(const __grid_constant__ SelectParams p)
{
    constexpr int kSegs = 2 * D / 64;  // 64-byte runs of a block's codes
    constexpr int kThreads = sel_threads(kClusters), kWarps = kThreads / 32;
    int rank = 0, ctas = 1;
    if constexpr (kClusters) {
        rank = (int)cg::this_cluster().block_rank();
        ctas = (int)cg::this_cluster().num_blocks();
    }
    __shared__ SelectShared sh;
    // B fragments of the coded heads: head 8 nt + g, codes 64 seg + 16 t4 .. + 15 of a
    // block's 2 D for the lane (g, t4)
    __shared__ __align__(16) uint4 qf[NT][kSegs][32];
    extern __shared__ uint32_t keys[];  // of this CTA's candidates; first, pool blocks
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    const int unit = (int)blockIdx.x / ctas;
    const int t = unit / p.num_kv_heads, kh = unit - t * p.num_kv_heads;
    const int G = p.group, top_k = p.top_k;
    if constexpr (kClusters)
        cg::this_cluster().sync();  // the first CTA's shared memory is there to be written
    pdl_wait_primary();
    pdl_launch_dependents();

    // ---- the row's context ----------------------------------------------------------
    const int s = p.token_seq[t], pos = p.token_pos[t];
    constexpr int kHeadsPerWarp = 8 * NT / kWarps;
    float x[kHeadsPerWarp][D / 32];
#pragma unroll
    for (int r = 0; r < kHeadsPerWarp; ++r) {
        const int h = r * kWarps + warp;
        const T *row = static_cast<const T *>(p.query) +
                       ((size_t)t * p.num_heads + (size_t)kh * G + (h < G ? h : 0)) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            x[r][e] = h < G ? (float)row[e * 32 + lane] : 0.f;
    }
    const bool whole = rank == 0 && tid == 0 && kh == 0;  // reports for the row
    int ctx = 0;
    if (s >= 0) {
        const long long cap = (long long)p.max_blocks_per_seq << p.block_shift;
        if (s >= p.num_seqs || pos < 0 || pos >= cap) {
            if (whole)
                flag_error(p.error_word, PA_DEVERR_TOKEN_RANGE);
        } else {
            if (pos >= p.max_context_len && whole)
                flag_error(p.error_word, PA_DEVERR_CONTEXT_RANGE);
            ctx = min(pos, p.max_context_len - 1) + 1;
        }
    }
    const int nb = (int)(((long long)ctx + (1 << p.block_shift) - 1) >> p.block_shift);
    int32_t *out = p.selected + (size_t)unit * top_k;
    if (nb <= top_k) {
        if (rank == 0)
            for (int i = tid; i < top_k; i += kThreads)
                out[i] = i < nb ? i : -1;
        return;
    }
    const int first = p.num_first, tail = nb - p.num_last;
    const int want = top_k - p.num_first - p.num_last;
    const int n = tail - first;  // candidates, more than are wanted
    // this CTA's candidates [c0, c0 + own), in tiles of 16
    const int share = ((n + 15) / 16 + ctas - 1) / ctas * 16;
    const int c0 = min(n, rank * share), own = min(n, c0 + share) - c0;
    const int tiles = (own + 15) / 16;
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq + first + c0;
    for (int i = tid; i < own; i += kThreads)
        keys[i] = (uint32_t)__ldg(table + i);

    // ---- the query heads' codes ------------------------------------------------------
#pragma unroll
    for (int r = 0; r < kHeadsPerWarp; ++r) {
        const int h = r * kWarps + warp;
        float top = 0.f;
        bool ok = true;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            ok &= finite(x[r][e]);
            top = fmaxf(top, fabsf(x[r][e]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        ok = __all_sync(kFull, ok);
        const CodeScale cs = ok ? code_scale(top) : CodeScale{0.f, 0.f};
        // element k = 32 e + lane of a side: run k / 64, lane 4 (h % 8) + k % 64 / 16
        int8_t *frag = reinterpret_cast<int8_t *>(&qf[h / 8][0][4 * (h & 7) + (lane >> 4)]) +
                       (lane & 15);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            const int code = ok ? __float2int_rn(__fmul_rn(x[r][e], cs.inv)) : 0;
            int8_t *at = frag + e / 2 * 512 + e % 2 * 32;
            at[0] = (int8_t)min(code, 0);
            at[D / 64 * 512] = (int8_t)max(code, 0);
        }
        if (lane == 0)
            sh.q_scale[h] = cs.scale;
    }
    __syncthreads();

    // ---- scores, 16 blocks a warp ----------------------------------------------------
    float q_scale[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        q_scale[nt][0] = sh.q_scale[nt * 8 + 2 * t4];
        q_scale[nt][1] = sh.q_scale[nt * 8 + 2 * t4 + 1];
    }
    for (int tile = warp; tile < tiles; tile += kWarps) {
        uint4 w[2][kSegs];
        float scale[2];
        bool ok[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = tile * 16 + g + 8 * r;
            int phys = i < own ? (int)keys[i] : 0;
            ok[r] = phys >= 0 && phys < p.num_blocks;
            phys = ok[r] ? phys : 0;
            const size_t at = (size_t)phys * p.num_kv_heads + kh;
            const uint4 *src = reinterpret_cast<const uint4 *>(p.codes + at * 2 * D) + t4;
#pragma unroll
            for (int sg = 0; sg < kSegs; ++sg)
                w[r][sg] = __ldg(src + sg * 4);
            scale[r] = __ldg(p.scales + at);
        }
        int acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0;
#pragma unroll
        for (int sg = 0; sg < kSegs; ++sg) {
            const uint4 a = w[0][sg], b = w[1][sg];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 q = qf[nt][sg][lane];
                mma_bytes(acc[nt], a.x, b.x, a.y, b.y, q.x, q.y);
                mma_bytes(acc[nt], a.z, b.z, a.w, b.w, q.z, q.w);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float best = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (nt * 8 + 2 * t4 + e < G)
                        best = fmaxf(best, __fmul_rn((float)acc[nt][2 * r + e],
                                                     q_scale[nt][e]));
            best = fmaxf(best, __shfl_xor_sync(kFull, best, 1));
            best = fmaxf(best, __shfl_xor_sync(kFull, best, 2));
            const int i = tile * 16 + g + 8 * r;
            if (t4 == 0 && i < own) {
                if (!ok[r])
                    flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                const float score = __float_as_uint(scale[r]) == 0x7f800000u
                                        ? scale[r] : __fmul_rn(best, scale[r]);
                keys[i] = ok[r] ? score_key(score) : 0u;
            }
        }
    }
    __syncthreads();

    // ---- the list, in ascending order ------------------------------------------------
    if (rank == 0) {
        for (int i = tid; i < first; i += kThreads)
            out[i] = i;
        for (int i = tid; i < p.num_last; i += kThreads)
            out[top_k - p.num_last + i] = tail + i;
    }
    if constexpr (!kClusters) {
        cta_select<kThreads>(sh, keys, n, want, [&](int i, int at) { out[first + at] = first + i; });
    } else {
        // the CTAs' lists come behind one another, keys and candidates
        cg::cluster_group cluster = cg::this_cluster();
        const int list0 = rank * min(want, share);  // (all CTAs before this one have `share`)
        uint32_t *all_keys = keys + share;          // in the first CTA
        uint32_t *all_ids = all_keys + (size_t)ctas * want;
        uint32_t *to_keys = cluster.map_shared_rank(all_keys, 0) + list0;
        uint32_t *to_ids = cluster.map_shared_rank(all_ids, 0) + list0;
        const int mine = min(want, own);
        if (mine == own) {
            for (int i = tid; i < own; i += kThreads) {
                to_keys[i] = keys[i];
                to_ids[i] = (uint32_t)(c0 + i);
            }
        } else {
            cta_select<kThreads>(sh, keys, own, mine, [&](int i, int at) {
                to_keys[at] = keys[i];
                to_ids[at] = (uint32_t)(c0 + i);
            });
        }
        cluster.sync();
        if (rank != 0)
            return;
        int total = 0;
        for (int r = 0; r < ctas; ++r)
            total += min(want, min(n, (r + 1) * share) - min(n, r * share));
        cta_select<kThreads>(sh, all_keys, total, want,
                   [&](int i, int at) { out[first + at] = first + (int)all_ids[i]; });
    }
}

// ---- host side -------------------------------------------------------------------

static bool pool_block(int block_size, int head_dim)
{
    return (head_dim == 64 || head_dim == 128) && block_size >= kTileTokens &&
           block_size <= 256 && (block_size & (block_size - 1)) == 0;
}

static pa_status current_device(int *dev, DeviceInfo *info)
{
    const cudaError_t e = cudaGetDevice(dev);
    return e != cudaSuccess ? record_cuda(e) : device_info(*dev, info);
}

template <typename KV>
static pa_status launch_summary(const SummaryParams &p, int head_dim, int sms,
                                cudaStream_t stream)
{
    // CTAs that the device holds at once, or a warp for every block that there can be
    const long long most = (long long)p.num_seqs * p.max_blocks_per_seq * p.num_kv_heads;
    const long long warps = kSumThreads / 32;
    const int grid = (int)std::min<long long>(kSumCtas * (long long)sms, (most + warps - 1) / warps);
    return head_dim == 128
               ? launch_pdl(summarize_kernel<KV, 128>, dim3(grid), dim3(kSumThreads), 0, stream, p)
               : launch_pdl(summarize_kernel<KV, 64>, dim3(grid), dim3(kSumThreads), 0, stream, p);
}

template <typename T, int D, int NT>
static pa_status launch_select(const SelectParams &p, int num_tokens, cudaStream_t stream)
{
    static size_t enabled_for[2][kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    DeviceInfo info;
    const pa_status st = current_device(&dev, &info);
    if (st != PA_OK)
        return st;
    const size_t room = (size_t)info.optin - (sizeof(SelectShared) + 16 * NT * D + 1024);
    const int bs = 1 << p.block_shift;
    // candidates of a row, at most
    const int most = (int)std::min<long long>(p.max_blocks_per_seq,
                                              ((long long)p.max_context_len + bs - 1) / bs);
    const int want = p.top_k - p.num_first - p.num_last;
    auto bytes = [&](int ctas) {
        return select_bytes(((most + 15) / 16 + ctas - 1) / ctas * 16, ctas, want);
    };
    // Clusters where the rows and KV heads leave SMs with fewer CTAs than they hold and
    // contexts are long, or where one CTA's memory does not hold their keys.
    const long long units = (long long)num_tokens * p.num_kv_heads;
    int ctas = 1;
    while (ctas < kSelCluster && units * ctas < sel_resident(true) * info.sms &&
           most >= 2 * ctas * kSelShare && bytes(2 * ctas) <= room)
        ctas *= 2;
    while (ctas < kSelCluster && bytes(ctas) > room)
        ctas *= 2;
    const size_t smem = bytes(ctas);
    if (smem > room || units * ctas > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    auto kernel = ctas > 1 ? select_kernel<T, D, NT, true> : select_kernel<T, D, NT, false>;
    {
        std::lock_guard<std::mutex> lock(mu);
        size_t *enabled = enabled_for[ctas > 1];
        if (smem > enabled[dev]) {
            cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         kSelCarveout);
            if (e != cudaSuccess)
                return record_cuda(e);
            enabled[dev] = smem;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * ctas));
    cfg.blockDim = dim3(sel_threads(ctas > 1));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return record_cuda(cudaLaunchKernelEx(&cfg, kernel, p));
}

template <typename T>
static pa_status select_as(const SelectParams &p, int head_dim, int num_tokens,
                           cudaStream_t stream)
{
    const bool wide = p.group > 8;
    if (head_dim == 128)
        return wide ? launch_select<T, 128, 2>(p, num_tokens, stream)
                    : launch_select<T, 128, 1>(p, num_tokens, stream);
    return wide ? launch_select<T, 64, 2>(p, num_tokens, stream)
                : launch_select<T, 64, 1>(p, num_tokens, stream);
}

} // namespace pa

using namespace pa;

extern "C" pa_status pa_summarize_blocks(int8_t *summaries, float *summary_scales,
                                         const void *key_cache, const int32_t *block_tables,
                                         int max_blocks_per_seq, const int32_t *context_lens,
                                         const int32_t *query_start, int num_seqs,
                                         int num_blocks, int block_size, int num_kv_heads,
                                         int head_dim, pa_dtype dtype, int32_t *error_word,
                                         void *stream)
{
    if (num_seqs < 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 ||
        (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_FP8_E4M3))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0)
        return PA_OK;
    if (!summaries || !summary_scales || !key_cache || !block_tables || !context_lens ||
        !aligned16(summaries) || !aligned16(key_cache))
        return PA_ERR_INVALID_ARG;
    if (!pool_block(block_size, head_dim) || (long long)num_blocks * block_size >= (1ll << 31) ||
        (long long)num_seqs * max_blocks_per_seq >= (1ll << 31) - (1 << 20))
        return PA_ERR_UNSUPPORTED;
    SummaryParams p{};
    p.codes = summaries;
    p.scales = summary_scales;
    p.key_cache = key_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.error_word = error_word;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_blocks = num_blocks;
    p.block_shift = __builtin_ctz((unsigned)block_size);
    p.num_kv_heads = num_kv_heads;
    int dev = 0;
    DeviceInfo info;
    const pa_status st = current_device(&dev, &info);
    if (st != PA_OK)
        return st;
    cudaStream_t q = as_stream(stream);
    return dtype == PA_FP8_E4M3 ? launch_summary<uint8_t>(p, head_dim, info.sms, q)
           : dtype == PA_BF16   ? launch_summary<__nv_bfloat16>(p, head_dim, info.sms, q)
                                : launch_summary<__half>(p, head_dim, info.sms, q);
}

extern "C" pa_status pa_select_blocks(int32_t *selected, int top_k, const void *query,
                                      const int8_t *summaries, const float *summary_scales,
                                      const int32_t *block_tables, int max_blocks_per_seq,
                                      const int32_t *token_seq, const int32_t *token_pos,
                                      int max_context_len, int num_first, int num_last,
                                      int num_tokens, int num_seqs, int num_heads,
                                      int num_kv_heads, int head_dim, int block_size,
                                      int num_blocks, pa_dtype dtype, int32_t *error_word,
                                      void *stream)
{
    if (num_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 ||
        max_context_len < 0 || top_k <= 0 || num_first < 0 || num_last < 0 ||
        num_first > top_k || num_last > top_k - num_first ||
        (dtype != PA_F16 && dtype != PA_BF16) || num_heads % num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return PA_OK;
    if (!selected || !query || !summaries || !summary_scales || !block_tables || !token_seq ||
        !token_pos || !aligned16(query) || !aligned16(summaries))
        return PA_ERR_INVALID_ARG;
    if (!pool_block(block_size, head_dim) || num_heads / num_kv_heads > 16 ||
        (long long)num_blocks * block_size >= (1ll << 31) ||
        (long long)max_blocks_per_seq * block_size >= (1ll << 31))
        return PA_ERR_UNSUPPORTED;
    SelectParams p{};
    p.selected = selected;
    p.query = query;
    p.codes = summaries;
    p.scales = summary_scales;
    p.block_tables = block_tables;
    p.token_seq = token_seq;
    p.token_pos = token_pos;
    p.error_word = error_word;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_blocks = num_blocks;
    p.block_shift = __builtin_ctz((unsigned)block_size);
    p.max_context_len = max_context_len;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    p.top_k = top_k;
    p.num_first = num_first;
    p.num_last = num_last;
    return dtype == PA_BF16
               ? select_as<__nv_bfloat16>(p, head_dim, num_tokens, as_stream(stream))
               : select_as<__half>(p, head_dim, num_tokens, as_stream(stream));
}
