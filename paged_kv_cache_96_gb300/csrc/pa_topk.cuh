// pa_topk.cuh -- the `want` largest of n 32-bit keys, by one CTA: the threshold that
// separates them, found digit by digit over the bits in which the keys differ.
#pragma once

#include "pa_common.cuh"

namespace pa {

// Digits of BITS bits: a histogram of 2^BITS counters.  8 bits keep a small CTA's passes
// short; 11 spread keys that differ in their exponents most over more counters, whose
// additions queue up otherwise.
template <int BITS> struct TopkShared {
    int hist[1 << BITS];
    uint32_t lo[32], hi[32];
    int sums[32];
    int bin, rest, whole;
};

// Selected are the keys whose difference to `lo`, shifted right by `shift`, is above
// `prefix`, and of those at it the first `rest` (ties in the caller's order).
struct Threshold {
    uint32_t lo, prefix;
    int shift, rest;
    __device__ __forceinline__ uint32_t level(uint32_t key) const
    {
        return (uint32_t)((unsigned long long)(key - lo) >> shift);
    }
};

// key(i): the key of i in [0, n), 0 <= want <= n, n > 0.  All of the CTA's THREADS
// threads call it, with the keys visible to them; a digit costs a pass over the keys,
// into a histogram in shared memory, and a scan of its bins.
template <int THREADS, int BITS, typename Key>
__device__ __forceinline__ Threshold top_threshold(TopkShared<BITS> &sh, const Key &key, int n,
                                                   int want)
{
    constexpr int kWarps = THREADS / 32;
    constexpr int kBins = 1 << BITS, kOwn = kBins / THREADS;
    static_assert(kBins % THREADS == 0, "whole bins per thread");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int i = tid; i < n; i += THREADS) {
        const uint32_t k = key(i);
        lo = min(lo, k);
        hi = max(hi, k);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        sh.lo[warp] = lo;
        sh.hi[warp] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        lo = min(lo, sh.lo[w]);
        hi = max(hi, sh.hi[w]);
    }
    Threshold t{lo, 0u, 32 - __clz((int)(hi - lo)), want};
    while (t.shift > 0 && t.rest > 0) {
        const int width = min(BITS, t.shift);
        t.shift -= width;
#pragma unroll
        for (int b = 0; b < kOwn; ++b)
            sh.hist[b * THREADS + tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += THREADS) {
            const uint32_t v = t.level(key(i));
            if (((unsigned long long)v >> width) == t.prefix)
                atomicAdd(&sh.hist[v & ((1u << width) - 1)], 1);
        }
        __syncthreads();
        // thread t has bins kOwn t and on; counts from the top bin down
        int own[kOwn], sum = 0;
#pragma unroll
        for (int b = 0; b < kOwn; ++b) {
            own[b] = sh.hist[tid * kOwn + b];
            sum += own[b];
        }
        int above = sum;  // of this thread's bins and those of higher lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_down_sync(0xffffffffu, above, o);
            if (lane + o < 32)
                above += y;
        }
        if (lane == 0)
            sh.sums[warp] = above;
        __syncthreads();
        int over = above - sum;  // of higher threads' bins
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            over += w > warp ? sh.sums[w] : 0;
#pragma unroll
        for (int b = kOwn - 1; b >= 0; --b) {
            if (over < t.rest && over + own[b] >= t.rest) {
                sh.bin = tid * kOwn + b;
                sh.rest = t.rest - over;
                sh.whole = own[b] == t.rest - over;
            }
            over += own[b];
        }
        __syncthreads();
        t.prefix = (t.prefix << width) | (uint32_t)sh.bin;
        t.rest = sh.rest;
        const bool whole = sh.whole != 0;  // every key at the prefix is selected
        __syncthreads();
        if (whole)
            break;
    }
    return t;
}

// The same for at most 32 PER keys, by one warp with the keys in registers: key j of
// lane l is that of 32 j + l.  One bit of the threshold at a time, with a count over
// the warp, and no barrier of the CTA.
template <int PER>
__device__ __forceinline__ Threshold warp_threshold(const uint32_t (&key)[PER], int n, int want)
{
    const int lane = threadIdx.x & 31;
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (32 * j + lane < n) {
            lo = min(lo, key[j]);
            hi = max(hi, key[j]);
        }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    // (the keys that are not there are as low as any, and no bit counts them)
    uint32_t v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j)
        v[j] = 32 * j + lane < n ? key[j] - lo : 0u;
    auto count = [&](uint32_t least) {
        int c = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            c += v[j] >= least;
        return __reduce_add_sync(0xffffffffu, c);
    };
    Threshold t{lo, 0u, 0, want};
    for (int b = 31 - __clz((int)(hi - lo)); b >= 0; --b) {
        const uint32_t least = t.prefix | (1u << b);
        const int c = count(least);
        if (c >= want)
            t.prefix = least;
        if (c == want)
            break;
    }
    t.rest = want - (t.prefix == 0xffffffffu ? 0 : count(t.prefix + 1));
    return t;
}

} // namespace pa
