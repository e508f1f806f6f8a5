// pa_topk.cuh -- the `want` largest of n 32-bit keys, by one CTA: the threshold that
// separates them, found digit by digit over the bits in which the keys differ.
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int kTopkBins = 256;

struct TopkShared {
    int hist[kTopkBins];
    uint32_t lo[32], hi[32];
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
// threads call it, with the keys visible to them; digits of 8 bits at a time, each a
// histogram in shared memory, so that a pass over the keys is all that a digit costs.
template <int THREADS, typename Key>
__device__ __forceinline__ Threshold top_threshold(TopkShared &sh, const Key &key, int n, int want)
{
    constexpr int kWarps = THREADS / 32;
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
        const int width = min(8, t.shift);
        t.shift -= width;
        for (int b = tid; b < kTopkBins; b += THREADS)
            sh.hist[b] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += THREADS) {
            const uint32_t v = t.level(key(i));
            if (((unsigned long long)v >> width) == t.prefix)
                atomicAdd(&sh.hist[v & ((1u << width) - 1)], 1);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l has bins 8 l .. 8 l + 7; counts from the top bin down
            int own[8], sum = 0;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                own[b] = sh.hist[lane * 8 + b];
                sum += own[b];
            }
            int above = sum;  // of this lane's bins and those of higher lanes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_down_sync(0xffffffffu, above, o);
                if (lane + o < 32)
                    above += y;
            }
            int over = above - sum;  // of higher lanes' bins
#pragma unroll
            for (int b = 7; b >= 0; --b) {
                if (over < t.rest && over + own[b] >= t.rest) {
                    sh.bin = lane * 8 + b;
                    sh.rest = t.rest - over;
                    sh.whole = own[b] == t.rest - over;
                }
                over += own[b];
            }
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

} // namespace pa
