// pa_window.cuh -- launch parameters and device helpers of the windowed
// chunked-attention kernel.
#pragma once

#include <type_traits>

#include "pa_decode_common.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

struct WindowMqParams {
    void *out;          // [T][H][D]
    const void *query;  // [T][H][D]
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;  // [S + 1]
    int32_t *error_word;
    uint64_t wait_ns;   // limit of one stage wait (PA_DEVERR_TIMEOUT past it)
    int withhold_fill;  // test hook: each CTA's key warp never issues its first fill
    int num_segments;   // sequences
    int num_heads, num_kv_heads, group;
    int max_blocks_per_seq, num_blocks, block_size, block_shift, max_context_len;
    int window, num_sinks;
    int sink_tokens;    // num_sinks rounded up to whole boxes
    float scale_log2;   // scale * log2(e) (times the K scale for FP8 pools)
    float out_scale;    // applied to the output (the V scale for FP8 pools)
    const void *key_cache, *value_cache;  // (for rows computed anew)
    int num_tokens;     // rows of query and out (T)
    int ordered;        // units numbered longest first
    int max_units;      // units of a KV head that query_start in order can give
};

// ---- fp32 helpers for the softmax ---------------------------------------------

// Maximum of three (max.f32 with three sources; a NaN source is ignored as
// in fmaxf).
__device__ __forceinline__ float fmax3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two fp32 values in one 64-bit register, and packed fp32 FMA / add on them
// (fma.rn.f32x2 / add.rn.f32x2: each lane rounds as its scalar form).
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t ffma_f32x2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t fadd_f32x2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 3-D tiled bulk tensor load global -> shared, completion on an mbarrier.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, uint32_t bar,
                                            int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Context length of a sequence, clamped like the decode pass.
__device__ __forceinline__ int window_context(const WindowMqParams &p, int s)
{
    const int limit = min(p.max_context_len, p.max_blocks_per_seq * p.block_size);
    int c = p.context_lens[s];
    if (c < 0 || c > limit) {
        flag_error(p.error_word, PA_DEVERR_CONTEXT_RANGE);
        c = c < 0 ? 0 : limit;
    }
    return c;
}

// First position of the window of the row at `pos` (of a row before the first
// position too, where pos + 1 - window would pass the 32 bits).
__device__ __forceinline__ int window_low(int pos, int window)
{
    return max(0, max(pos, -1) + 1 - window);
}

// First row of sequence s, kept inside the query; offsets that are not are
// flagged by the caller that passes `flag`.
__device__ __forceinline__ int window_row0(const WindowMqParams &p, int s, bool flag)
{
    const int r = p.query_start[s];
    if (flag && (r < 0 || r > p.num_tokens))
        flag_error(p.error_word, PA_DEVERR_TOKEN_RANGE);
    return min(max(r, 0), p.num_tokens);
}

// Rows of one sequence's chunk (none where its offsets decrease).
__device__ __forceinline__ int window_rows(const WindowMqParams &p, int s, bool flag = false)
{
    const int rows = window_row0(p, s + 1, flag) - window_row0(p, s, flag);
    if (flag && rows < 0)
        flag_error(p.error_word, PA_DEVERR_TOKEN_RANGE);
    return max(0, rows);
}

// Key tiles (of 64) a sequence's last row sees: the order of the deal.
__device__ __forceinline__ int window_order_key(const WindowMqParams &p, int s, int buckets)
{
    const int ctx = window_context(p, s);
    const unsigned keys = min((unsigned)ctx, (unsigned)min(p.sink_tokens, ctx) +
                                                 (unsigned)min(p.window, ctx));
    return buckets - 1 - (int)min((keys + 63) / 64, (unsigned)buckets - 1);
}

// ---- rows that a hidden value made non-finite -----------------------------------
//
// The tensor cores multiply a key that is hidden from a row by a weight of 0,
// which is not 0 when its value is infinite or NaN, and a value row that some
// row of the tile sees cannot be zeroed.  So a row that comes out non-finite is
// looked at again, by one warp.  Only values of keys that are hidden from it and seen
// by another row of its unit can have done that: the keys after its own position
// and those that its window has just left, as many of both as the unit has tokens
// at most.  If one of them is non-finite where the row is, the row is computed anew
// from what it sees, 32 keys at a time, 8 pool rows in flight (unless it sees a NaN
// there itself; the newest are read first).  So rows that are not numbers by what
// they see -- their query, a key, a value -- cost one look at the hidden values of
// their unit, and none where their sum of weights is NaN (64 rows of a context of
// 40,000, all NaN by an old key or an old value: 230 and 243 us, clean 230; reading
// again what each row sees took 472 and 265 ms).

template <typename T> __device__ __forceinline__ float window_float(T x)
{
    if constexpr (std::is_same<T, __half>::value)
        return __half2float(x);
    else
        return __bfloat162float(x);
}

// This lane's E = D / 32 elements of a pool row, as numbers.
template <typename T, int E, bool kFp8>
__device__ __forceinline__ void window_pool_row(const void *pool, size_t elem, float (&x)[E])
{
    if constexpr (kFp8) {
        const uint8_t *c = static_cast<const uint8_t *>(pool) + elem;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const uint32_t w = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(c + e));
            x[e] = __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
            x[e + 1] = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
        }
    } else {
        const T *v = static_cast<const T *>(pool) + elem;
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[e] = window_float<T>(v[e]);
    }
}

// A finite test that fast-math arithmetic does not fold away.
__device__ __forceinline__ bool window_finite(float x)
{
    return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
}

// The places in the pools of the keys of one sequence and KV head.
struct WindowKeys {
    const WindowMqParams &p;
    const int32_t *table;
    int kh;
    // elements before position t's row (-2: a table entry outside the pool)
    __device__ __forceinline__ long long at(int t, int head_dim) const
    {
        const int b = table[t >> p.block_shift];
        if (b < 0 || b >= p.num_blocks)
            return -2;
        return (((long long)b * p.block_size + (t & (p.block_size - 1))) * p.num_kv_heads + kh) *
               head_dim;
    }
};

constexpr int kWindowBatch = 8;  // pool rows in flight

// This lane's elements of rows u .. u + 7 of the 32 whose places the lanes hold
// (negative places: none, zeros).
template <typename T, int E, bool kFp8>
__device__ __forceinline__ void window_pool_rows(const void *pool, long long at, int u,
                                                 float (&x)[kWindowBatch][E])
{
#pragma unroll
    for (int k = 0; k < kWindowBatch; ++k) {
        const long long a = __shfl_sync(kFull, at, u + k);
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[k][e] = 0.f;
        if (a >= 0)
            window_pool_row<T, E, kFp8>(pool, a + (threadIdx.x & 31) * E, x[k]);
    }
}

// This lane's elements (bits) at which one of the values of positions [a0, a1)
// and [b0, b1) is non-finite, by a warp.
template <typename T, int D, bool kFp8>
__device__ __noinline__ unsigned window_non_finite(WindowKeys keys, const void *values,
                                                   int a0, int a1, int b0, int b1)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, na = max(0, a1 - a0), n = na + max(0, b1 - b0);
    unsigned hot = 0;
    for (int i = 0; i < n; i += 32) {
        const int j = i + lane;
        const long long at = j < n ? keys.at(j < na ? a0 + j : b0 + j - na, D) : -1;
#pragma unroll 1
        for (int u = 0; u < min(32, n - i); u += kWindowBatch) {
            float v[kWindowBatch][E];
            window_pool_rows<T, E, kFp8>(values, at, u, v);
#pragma unroll
            for (int k = 0; k < kWindowBatch; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (!window_finite(v[k][e]))
                        hot |= 1u << e;
        }
    }
    return hot;
}

// One row (position pos of the sequence with this table, KV head kh), by a
// warp: out and query are its D elements; unit: the first position that its
// unit's rows have, and one past the last.
template <typename T, int D, bool kFp8>
__device__ __noinline__ void window_mend_row(WindowKeys keys, const void *key_cache,
                                             const void *value_cache, int pos, int unit0,
                                             int unit1, const T *query, T *out)
{
    constexpr int E = D / 32, kBatch = kWindowBatch;
    const WindowMqParams &p = keys.p;
    const int lane = threadIdx.x & 31;
    const int low = window_low(pos, p.window);      // [low, pos] and [0, first) are seen
    const int first = min(p.num_sinks, low);
    const int seen = pos + 1 - low + first;
    // elements that are non-finite where a hidden value is
    unsigned open = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (!window_finite(window_float<T>(out[lane * E + e])))
            open |= 1u << e;
    if (!__any_sync(kFull, open != 0))
        return;
    open &= window_non_finite<T, D, kFp8>(keys, value_cache, pos + 1, unit1,
                                          max(window_low(unit0, p.window), p.num_sinks), low);
    if (!__any_sync(kFull, open != 0))
        return;
    // the i-th key seen, newest first: its place in the pools (-1: none)
    auto place = [&](int i) -> long long {
        return i >= seen ? -1
                         : keys.at(i <= pos - low ? pos - i : first - 1 - (i - (pos + 1 - low)), D);
    };
    auto rows = [&](const void *pool, long long at, int u, float (&x)[kBatch][E]) {
        window_pool_rows<T, E, kFp8>(pool, at, u, x);
    };
    // a NaN that the row sees accounts for its element
    for (int i = 0; i < seen; i += 32) {
        const long long at = place(i + lane);
        if (__any_sync(kFull, at == -2))
            return;  // (flagged; the row is undefined)
#pragma unroll 1
        for (int u = 0; u < 32; u += kBatch) {
            float v[kBatch][E];
            rows(value_cache, at, u, v);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if ((__float_as_uint(v[k][e]) & 0x7fffffffu) > 0x7f800000u)
                        open &= ~(1u << e);
        }
        if (!__any_sync(kFull, open != 0))
            return;
    }
    float q[E], o[E], m = -INFINITY, l = 0.f;  // (l: of this lane's keys)
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = window_float<T>(query[lane * E + e]);
        o[e] = 0.f;
    }
    for (int i = 0; i < seen; i += 32) {
        const long long at = place(i + lane);
        float mine = -INFINITY;  // the score of key i + lane
#pragma unroll 1
        for (int u = 0; u < 32; u += kBatch) {
            float k[kBatch][E];
            rows(key_cache, at, u, k);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    s = fmaf(q[e], k[b][e], s);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    s += __shfl_xor_sync(kFull, s, off);
                if (lane == u + b && at >= 0)
                    mine = s * p.scale_log2;
            }
        }
        float top = mine;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        const float mn = fmaxf(m, top);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - ref);  // (0 at first)
        const float w = exp2f(mine - ref);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] *= a;
#pragma unroll 1
        for (int u = 0; u < 32; u += kBatch) {
            float v[kBatch][E];
            rows(value_cache, at, u, v);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float wk = __shfl_sync(kFull, w, u + k);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    o[e] += wk * v[k][e];
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        l += __shfl_xor_sync(kFull, l, off);
    const float inv = p.out_scale / l;
#pragma unroll
    for (int e = 0; e < E; ++e)
        out[lane * E + e] = MmaOp<T>::from_float(o[e] * inv);
}

// Rows `todo` of the calling warp's 32 of a unit (those that it has), computed anew
// from what they see (nothing, at a negative position).  Out of line, like what it
// calls: within the output warps' code it slowed their loop down (8,192 rows over FP8
// pools 606 us for 580).
template <typename T, int D, bool kFp8>
__device__ __noinline__ void window_mend_unit(const WindowMqParams &p, int seq, int row0, int kh,
                                              int count, int pos0, unsigned todo)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.group;
    const WindowKeys keys{p, p.block_tables + (size_t)seq * p.max_blocks_per_seq, kh};
    __syncwarp();
    // whether a value hidden from one row and seen by another is non-finite
    const int end = pos0 + count;
    const bool hot =
        __any_sync(kFull, window_non_finite<T, D, kFp8>(
                              keys, p.value_cache, max(pos0, 0) + 1, end,
                              max(window_low(pos0, p.window), p.num_sinks),
                              window_low(end - 1, p.window)) != 0);
    for (; todo != 0; todo &= todo - 1) {
        const int rr = 32 * (warp & 3) + __ffs(todo) - 1;
        const int tk = rr / G;
        if (tk >= count)
            continue;
        const long long at =
            (((long long)row0 + tk) * p.num_heads + kh * G + rr - tk * G) * D;
        T *out = static_cast<T *>(p.out) + at;
        if (pos0 + tk < 0)
            for (int e = lane; e < D / 2; e += 32)
                reinterpret_cast<uint32_t *>(out)[e] = 0;
        else if (hot)
            window_mend_row<T, D, kFp8>(keys, p.key_cache, p.value_cache, pos0 + tk, pos0, end,
                                        static_cast<const T *>(p.query) + at, out);
    }
}

// Sequences of one launch (their unit counts are kept in shared memory).
constexpr int kWindowMaxSeqs = 5120;

// dtype: the query's, the output's and (unless fp8: e4m3 codes) the pools'.
pa_status launch_window_tiles(const WindowMqParams &prm, pa_dtype dtype, bool fp8, int head_dim,
                             cudaStream_t stream);

}  // namespace pa
