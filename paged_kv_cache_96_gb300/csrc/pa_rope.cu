// pa_rope.cu -- rotary positions with one or more axes, fused with the paged
// cache write ("PagedAttention & Continuous Batching" §1.5: the new tokens'
// K/V go to their slots; the rotation before it is not on the pages).
//
// For token t and rotary pair i (R = rot_dim, pair i turns two elements u, v
// of every query and key head):
//     phi = positions[axis_of_pair[i]][t] * inv_freq[i]
//     u' = u cos(phi) - v sin(phi),   v' = v cos(phi) + u sin(phi)
// with (u, v) = elements (i, i + R / 2), or (2i, 2i + 1) when interleaved;
// elements from R on pass through.  Products and sums are fp32, rounded once:
// to the 16-bit type for the query and 16-bit pools, to the e4m3 code of
// x * (1 / scale) for FP8 pools.
//
// What bounds it: memory.  Every element of q, k and v is read and written
// once, and the angles cost little next to that if they are computed once a
// token: a CTA takes one token, its first threads compute the R / 2 sines and
// cosines into shared memory while the first rows' loads are in flight, and
// every head reuses them (4 tokens 2.0 us a call in a graph, 128 tokens into FP8
// pools 2.8).  Long batches stream through persistent warps instead (below:
// 16,381 tokens of 20 KB 111 us, 6.06 TB/s).  A cosine table over positions would have to be
// read instead (R * 4 bytes a token and axis, and as long as the longest
// context); the angle itself costs about 40 instructions a pair.
//
// Far positions: phi / 2 pi grows to 10^5 turns and more, where an fp32
// product keeps no correct digit of the fraction.  The frequency is taken in
// turns, f / 2 pi, as an unevaluated sum of two fp32 numbers (48 bits), the
// position is split into two parts that fp32 holds exactly, the product's
// rounding error is recovered with a fused multiply-add, and only then are
// whole turns dropped.  The two fractions of up to half a turn are added in fp32, which
// rounds by 2^-24 of a turn (6 10^-8: the worst of 2 10^6 phases below a million);
// the frequency's 48 bits pass that from about 10^7 positions on (8 10^-8 at 2^24,
// 4.3 10^-6 at 2^31, frequencies up to 1).
#include <algorithm>
#include <cmath>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_decode_common.cuh"

namespace pa {

constexpr int kRopeMaxPairs = 128;  // head_dim up to 256
constexpr int kRopeMaxThreads = 256;
constexpr int kAhead = 3;  // rotary items of a thread whose loads go out first
// the streaming kernel: warps of a CTA (one an SM), bytes of a unit, units ahead
constexpr int kRingWarps = 24;
constexpr int kRingUnit = 2560;
constexpr int kRingDepth = 3;
// Batches that stream: rows of 4 KB (query, key and value) and 64 MB of them.  64 + 8
// + 8 heads of 128: 16,381 tokens 111 us (a CTA a token: 123), 4,096 tokens 33.2
// (33.7), 2,048 tokens 20.5 (18.0); 16 + 2 + 2 heads: 16,381 tokens 36.8 (51.5),
// 8,192 tokens 22.1 (26.5), 4,096 tokens 13.7 (13.5); rows of 3 KB, 8 + 8 + 8 heads of
// 64, 16,381 tokens 29.2 (22.9): a warp's own angles are most of its work there.
constexpr long long kRingRowBytes = 4096;
constexpr long long kRingBytes = 64ll << 20;

struct RopeParams {
    void *query_out;
    const void *query, *key, *value;
    void *key_cache, *value_cache;
    const int32_t *slot_mapping, *positions;
    const float *inv_freq;
    int32_t *error_word;
    long long q_stride, k_stride, v_stride, qo_stride;  // elements from token to token
    long long num_slots;
    int num_tokens, num_heads, num_kv_heads, head_dim, rot_dim;
    float k_inv_scale, v_inv_scale;  // FP8 pools
    uint64_t wait_ns;                // streaming kernel: limit of one wait
    int withhold_fill;               // its test hook: warp 0's first unit is never asked for
    int parts, part_heads;           // its units of a token, heads of one
    uint8_t axis[kRopeMaxPairs];     // axis of each rotary pair
};

// Fraction of a turn of pos * f / (2 pi), in about [-0.5, 0.5].
__device__ __forceinline__ float rope_turns(int pos, float f)
{
    // 1 / (2 pi) = kHi + kLo to 48 bits
    constexpr float kHi = 0.15915493667125702f;
    constexpr float kLo = 6.4206382432985265e-09f;
    const float fh = __fmul_rn(f, kHi);
    const float fl = __fmaf_rn(f, kLo, __fmaf_rn(f, kHi, -fh));
    // 19 high bits and 12 low bits of the position, each exact in fp32
    const float ph = (float)(pos & ~0xfff), pl = (float)(pos & 0xfff);
    const float a = __fmul_rn(ph, fh), b = __fmul_rn(pl, fh);
    const float ea = __fmaf_rn(ph, fh, -a), eb = __fmaf_rn(pl, fh, -b);
    float r = __fadd_rn(__fsub_rn(a, rintf(a)), __fsub_rn(b, rintf(b)));
    r = __fadd_rn(r, __fadd_rn(__fadd_rn(ea, eb), __fmul_rn(__fadd_rn(ph, pl), fl)));
    return __fsub_rn(r, rintf(r));
}

__device__ __forceinline__ float rope_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float rope_float(__half x) { return __half2float(x); }

// A 16-byte word that is read once: not kept in L1.
__device__ __forceinline__ uint4 load_word(const void *p)
{
    uint4 w;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(p)
                 : "memory");
    return w;
}

template <typename T> __device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8])
{
    const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = rope_float(e[i]);
}

template <typename T> __device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(MmaOp<T>::pack(x[0], x[1]), MmaOp<T>::pack(x[2], x[3]),
                      MmaOp<T>::pack(x[4], x[5]), MmaOp<T>::pack(x[6], x[7]));
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv)
{
    uint2 c;
    c.x = (uint32_t)f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) |
          ((uint32_t)f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16);
    c.y = (uint32_t)f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) |
          ((uint32_t)f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16);
    return c;
}

// Eight pairs turned: words wu and wv hold (u, v), or, interleaved, pairs 0-3 and 4-7.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void rope_turn(const uint4 &wu, const uint4 &wv, const float (&c)[8],
                                          const float (&s)[8], float (&x)[8], float (&y)[8])
{
    float u[8], w[8];
    unpack8<T>(wu, u);
    unpack8<T>(wv, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // pair i: interleaved, elements 2i and 2i + 1 of the two words
        const float a = kInterleaved ? (i < 4 ? u[(2 * i) & 7] : w[(2 * i) & 7]) : u[i];
        const float b = kInterleaved ? (i < 4 ? u[(2 * i + 1) & 7] : w[(2 * i + 1) & 7]) : w[i];
        const float r0 = a * c[i] - b * s[i];
        const float r1 = b * c[i] + a * s[i];
        if constexpr (kInterleaved) {
            (i < 4 ? x : y)[(2 * i) & 7] = r0;
            (i < 4 ? x : y)[(2 * i + 1) & 7] = r1;
        } else {
            x[i] = r0;
            y[i] = r1;
        }
    }
}

// One CTA per token.  The row's work is a list of items: first the rotary
// ones (a head's 8 pairs: two 16-byte words), heads of the query then of the
// key, then single words to pass on (elements from rot_dim on) and to cache
// (values).
template <typename T, bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kRopeMaxThreads)
    rope_and_cache_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ __align__(16) float cos_s[kRopeMaxPairs], sin_s[kRopeMaxPairs];
    const int t = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    pdl_wait_primary();
    pdl_launch_dependents();

    const int H = p.num_heads, K = p.num_kv_heads, D = p.head_dim;
    const int pairs = p.rot_dim >> 1;
    const int chunks = p.rot_dim >> 4;  // rotary items per head (8 pairs each)
    const T *q = static_cast<const T *>(p.query) + (long long)t * p.q_stride;
    const T *k = static_cast<const T *>(p.key) + (long long)t * p.k_stride;
    const T *v = static_cast<const T *>(p.value) + (long long)t * p.v_stride;
    T *qo = static_cast<T *>(p.query_out) + (long long)t * p.qo_stride;

    const int rot_items = (H + K) * chunks;
    // the two words of rotary item `it`: head h (keys after queries), chunk j
    auto locate = [&](int it, int &h, int &lo, int &hi) {
        h = it / chunks;
        const int j = it - h * chunks;
        lo = kInterleaved ? 16 * j : 8 * j;
        hi = kInterleaved ? lo + 8 : pairs + 8 * j;
        return j;
    };
    auto load2 = [&](int it, uint4 &a, uint4 &b) {
        int h, lo, hi;
        locate(it, h, lo, hi);
        const T *row = h < H ? q + h * D : k + (h - H) * D;
        a = load_word(row + lo);
        b = load_word(row + hi);
    };
    // the first items' loads go out before the angles are needed
        uint4 wa[kAhead], wb[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const int it = tid + u * threads;
        if (it < rot_items)
            load2(it, wa[u], wb[u]);
    }
    const int v_items = K * (D >> 3);
    uint4 wv0 = make_uint4(0, 0, 0, 0);
    if (tid < v_items)
        wv0 = load_word(v + 8 * tid);
    long long slot = p.slot_mapping[t];
    if (slot >= p.num_slots) {
        if (tid == 0)
            flag_error(p.error_word, PA_DEVERR_SLOT_RANGE);
        slot = -1;
    }
    if (tid < pairs) {
        const int pos = p.positions[(long long)p.axis[tid] * p.num_tokens + t];
        float s, c;
        sincospif(2.f * rope_turns(pos, p.inv_freq[tid]), &s, &c);
        cos_s[tid] = c;
        sin_s[tid] = s;
    }
    __syncthreads();

    const long long crow = slot * ((long long)K * D);  // element offset of the token's cache row
    auto put_key = [&](int h, int d, const float (&x)[8]) {
        if (slot < 0)
            return;
        const long long at = crow + (long long)h * D + d;
        if constexpr (kFp8)
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.key_cache) + at) =
                codes8(x, p.k_inv_scale);
        else
            *reinterpret_cast<uint4 *>(static_cast<T *>(p.key_cache) + at) = pack8<T>(x);
    };
    auto turn = [&](int it, const uint4 &wu, const uint4 &wv) {
        int h, lo, hi;
        const int j = locate(it, h, lo, hi);
        float c[8], s[8], x[8], y[8];
        *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(cos_s + 8 * j);
        *reinterpret_cast<float4 *>(c + 4) = *reinterpret_cast<const float4 *>(cos_s + 8 * j + 4);
        *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(sin_s + 8 * j);
        *reinterpret_cast<float4 *>(s + 4) = *reinterpret_cast<const float4 *>(sin_s + 8 * j + 4);
        rope_turn<T, kInterleaved>(wu, wv, c, s, x, y);
        if (h < H) {
            *reinterpret_cast<uint4 *>(qo + h * D + lo) = pack8<T>(x);
            *reinterpret_cast<uint4 *>(qo + h * D + hi) = pack8<T>(y);
        } else {
            put_key(h - H, lo, x);
            put_key(h - H, hi, y);
        }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const int it = tid + u * threads;
        if (it < rot_items)
            turn(it, wa[u], wb[u]);
    }
    for (int it = tid + kAhead * threads; it < rot_items; it += threads) {
        uint4 a, b;
        load2(it, a, b);
        turn(it, a, b);
    }
    // elements past the rotary ones
    const int rest = (D - p.rot_dim) >> 3;
    if (rest > 0) {
        for (int it = tid; it < (H + K) * rest; it += threads) {
            const int h = it / rest, d = p.rot_dim + 8 * (it - h * rest);
            const T *row = h < H ? q + h * D : k + (h - H) * D;
            const uint4 w = load_word(row + d);
            if (h < H) {
                *reinterpret_cast<uint4 *>(qo + h * D + d) = w;
            } else if constexpr (kFp8) {
                float x[8];
                unpack8<T>(w, x);
                put_key(h - H, d, x);
            } else if (slot >= 0) {
                *reinterpret_cast<uint4 *>(static_cast<T *>(p.key_cache) + crow +
                                           (long long)(h - H) * D + d) = w;
            }
        }
    }
    if (slot >= 0) {
        for (int it = tid; it < v_items; it += threads) {
            const uint4 w = it == tid ? wv0 : load_word(v + 8 * it);
            if constexpr (kFp8) {
                float x[8];
                unpack8<T>(w, x);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.value_cache) + crow + 8 * it) =
                    codes8(x, p.v_inv_scale);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<T *>(p.value_cache) + crow + 8 * it) = w;
            }
        }
    }
}

// ---- long batches -----------------------------------------------------------------
//
// A warp streams units (some consecutive heads of one token's query, key and
// value rows, kRingUnit bytes at most) through kRingDepth places of its own in
// shared memory: one lane asks for a unit as bulk copies, whole rows at a time,
// the warp turns and stores the unit before it.  No warp waits for another,
// and loads stay in flight while others compute and store, which a CTA a token
// lacks between its loads and its end.  A warp's units follow one another, so
// it has a token's angles once (units dealt round by round: 159 us instead of
// 111, the angles being longer than a unit).  (16 warps with 2 units of 5,120
// bytes: 123; 24 with 2 of 4,096: 117.)

// `bytes` (a multiple of 16) from 16-byte aligned global memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <typename T, bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(32 * kRingWarps, 1)
    rope_stream_kernel(const __grid_constant__ RopeParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t *own = smem + warp * (kRingDepth * kRingUnit);  // this warp's units
    float *cos_s = reinterpret_cast<float *>(smem + kRingWarps * kRingDepth * kRingUnit) +
                   warp * (2 * kRopeMaxPairs);
    float *sin_s = cos_s + kRopeMaxPairs;
    const uint32_t bars = smem_addr(smem + kRingWarps * (kRingDepth * kRingUnit +
                                                         8 * kRopeMaxPairs)) +
                          warp * (8 * kRingDepth);
    if (lane == 0) {
        for (int i = 0; i < kRingDepth; ++i)
            mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
    }
    __syncwarp();
    pdl_wait_primary();
    pdl_launch_dependents();

    const int H = p.num_heads, K = p.num_kv_heads, D = p.head_dim, R = p.rot_dim;
    const int pairs = R >> 1, chunks = R >> 4, rest = (D - R) >> 3;
    const int turned = H + K, heads = H + 2 * K;
    // this lane's place: chunk j of every head_step-th head
    const int head_step = 32 / chunks;
    const int j = lane % chunks, first_head = lane / chunks;
    const int lo = kInterleaved ? 16 * j : 8 * j;
    const int hi = kInterleaved ? lo + 8 : pairs + 8 * j;

    const long long units = (long long)p.num_tokens * p.parts;
    const long long workers = (long long)gridDim.x * kRingWarps;
    const long long w = (long long)warp * gridDim.x + blockIdx.x;
    const long long begin = units * w / workers, end = units * (w + 1) / workers;
    if (begin >= end)
        return;

    struct Cursor {  // a unit: token, and its first head
        int t, a;
    };
    auto advance = [&](Cursor &c) {
        c.a += p.part_heads;
        if (c.a >= heads) {
            c.a = 0;
            ++c.t;
        }
    };
    Cursor cur, to_fetch;
    cur.t = (int)(begin / p.parts);
    cur.a = (int)(begin - (long long)cur.t * p.parts) * p.part_heads;
    to_fetch = cur;
    const int count = (int)(end - begin);
    auto fetch = [&](const Cursor &c, int place) {  // (one lane)
        const int t = c.t, a = c.a, b = min(a + p.part_heads, heads);
        const uint32_t bar = bars + 8 * place;
        const uint32_t dst = smem_addr(own) + place * kRingUnit;
        mbar_arrive_expect_tx(bar, (uint32_t)((b - a) * D * 2));
        auto range = [&](const void *base, long long stride, int from, int to) {
            const int x = max(a, from), y = min(b, to);
            if (x < y)
                bulk_load(dst + (x - a) * D * 2,
                          static_cast<const T *>(base) + t * stride + (x - from) * D,
                          (uint32_t)((y - x) * D * 2), bar);
        };
        range(p.query, p.q_stride, 0, H);
        range(p.key, p.k_stride, H, turned);
        range(p.value, p.v_stride, turned, heads);
    };
    // what a token's angles and cache row need, loaded one unit ahead
    float freq[kRopeMaxPairs / 32];
#pragma unroll
    for (int m = 0; m < kRopeMaxPairs / 32; ++m)
        freq[m] = lane + 32 * m < pairs ? p.inv_freq[lane + 32 * m] : 0.f;
    int pos[kRopeMaxPairs / 32];
    long long slot;
    auto ahead = [&](int t) {
#pragma unroll
        for (int m = 0; m < kRopeMaxPairs / 32; ++m)
            pos[m] = lane + 32 * m < pairs
                         ? __ldg(p.positions + (long long)p.axis[lane + 32 * m] * p.num_tokens + t)
                         : 0;
        slot = __ldg(p.slot_mapping + t);
    };

    for (int i = 0; i < kRingDepth && i < count; ++i) {
        if (lane == 0 && !(p.withhold_fill != 0 && warp == 0 && i == 0))
            fetch(to_fetch, i);
        advance(to_fetch);
    }
    ahead(cur.t);
    int angles_of = -1, place = 0;
    uint32_t phase = 0;
    for (int u = 0; u < count; ++u) {
        const int t = cur.t, a = cur.a, b = min(a + p.part_heads, heads);
        advance(cur);
        if (angles_of != t) {
            __syncwarp();  // (the unit before has read the angles)
#pragma unroll
            for (int m = 0; m < kRopeMaxPairs / 32; ++m)
                if (lane + 32 * m < pairs) {
                    float s, c;
                    sincospif(2.f * rope_turns(pos[m], freq[m]), &s, &c);
                    cos_s[lane + 32 * m] = c;
                    sin_s[lane + 32 * m] = s;
                }
            __syncwarp();
            angles_of = t;
        }
        long long row = slot;
        if (row >= p.num_slots) {
            if (lane == 0)
                flag_error(p.error_word, PA_DEVERR_SLOT_RANGE);
            row = -1;
        }
        row *= (long long)K * D;  // element offset of the token's cache row (negative: none)
        if (u + 1 < count && cur.t != t)
            ahead(cur.t);
        if (!__all_sync(kFull, mbar_wait_bounded(bars + 8 * place, phase, p.wait_ns))) {
            if (lane == 0)
                flag_error(p.error_word, PA_DEVERR_TIMEOUT);
            // (no copy may land after this warp has left)
            for (int i = 0; i < kRingDepth && u + i < count; ++i) {
                mbar_wait_bounded(bars + 8 * place, phase, kDrainWaitNs);
                if (++place == kRingDepth) {
                    place = 0;
                    phase ^= 1;
                }
            }
            break;
        }
        const T *unit = reinterpret_cast<const T *>(own + place * kRingUnit);
        T *qo = static_cast<T *>(p.query_out) + (long long)t * p.qo_stride;
        auto put_cache = [&](void *cache, float inv, long long at, const uint4 &word,
                             const float (&x)[8]) {
            if (row < 0)
                return;
            if constexpr (kFp8)
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + row + at) =
                    codes8(x, inv);
            else
                *reinterpret_cast<uint4 *>(static_cast<T *>(cache) + row + at) = word;
        };
        if (first_head < head_step && a < turned) {
            float c[8], s[8];
            *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(cos_s + 8 * j);
            *reinterpret_cast<float4 *>(c + 4) =
                *reinterpret_cast<const float4 *>(cos_s + 8 * j + 4);
            *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(sin_s + 8 * j);
            *reinterpret_cast<float4 *>(s + 4) =
                *reinterpret_cast<const float4 *>(sin_s + 8 * j + 4);
            for (int h = a + first_head; h < min(b, turned); h += head_step) {
                const T *src = unit + (h - a) * D;
                float x[8], y[8];
                rope_turn<T, kInterleaved>(*reinterpret_cast<const uint4 *>(src + lo),
                                           *reinterpret_cast<const uint4 *>(src + hi), c, s, x,
                                           y);
                if (h < H) {
                    *reinterpret_cast<uint4 *>(qo + h * D + lo) = pack8<T>(x);
                    *reinterpret_cast<uint4 *>(qo + h * D + hi) = pack8<T>(y);
                } else {
                    const long long at = (long long)(h - H) * D;
                    put_cache(p.key_cache, p.k_inv_scale, at + lo, pack8<T>(x), x);
                    put_cache(p.key_cache, p.k_inv_scale, at + hi, pack8<T>(y), y);
                }
            }
        }
        // elements past the rotary ones, and values: words passed on
        const int rest_items = max(0, min(b, turned) - a) * rest;
        for (int it = lane; it < rest_items; it += 32) {
            const int h = a + it / rest, d = R + 8 * (it % rest);
            const uint4 word = *reinterpret_cast<const uint4 *>(unit + (h - a) * D + d);
            float x[8];
            unpack8<T>(word, x);
            if (h < H)
                *reinterpret_cast<uint4 *>(qo + h * D + d) = word;
            else
                put_cache(p.key_cache, p.k_inv_scale, (long long)(h - H) * D + d, word, x);
        }
        const int v0 = max(a, turned);
        const int v_words = max(0, b - v0) * (D >> 3);
        for (int it = lane; it < v_words; it += 32) {
            const uint4 word =
                *reinterpret_cast<const uint4 *>(unit + (v0 - a) * D + 8 * it);
            float x[8];
            unpack8<T>(word, x);
            put_cache(p.value_cache, p.v_inv_scale, (long long)(v0 - turned) * D + 8 * it, word,
                      x);
        }
        __syncwarp();
        if (u + kRingDepth < count) {
            if (lane == 0)
                fetch(to_fetch, place);
            advance(to_fetch);
        }
        if (++place == kRingDepth) {
            place = 0;
            phase ^= 1;
        }
    }
}

template <typename T, bool kFp8>
static pa_status launch_rope(RopeParams &p, bool interleaved, cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return record_cuda(e);
    DeviceInfo info;
    const pa_status st = device_info(dev, &info);
    if (st != PA_OK)
        return st;
    const int heads = p.num_heads + 2 * p.num_kv_heads;
    const int most = kRingUnit / (2 * p.head_dim);
    p.parts = (heads + most - 1) / most;
    p.part_heads = (heads + p.parts - 1) / p.parts;
    p.wait_ns = stage_wait_limit_ns();
    p.withhold_fill = withhold_first_fill();
    const long long row_bytes = 2ll * heads * p.head_dim;
    if (row_bytes >= kRingRowBytes && row_bytes * p.num_tokens >= kRingBytes) {
        auto kernel = interleaved ? rope_stream_kernel<T, kFp8, true>
                                  : rope_stream_kernel<T, kFp8, false>;
        constexpr size_t smem = kRingWarps * (kRingDepth * kRingUnit + 8 * kRopeMaxPairs +
                                              8 * kRingDepth);
        static bool enabled[2][kMaxDevices];
        static std::mutex mu;
        {
            std::lock_guard<std::mutex> lock(mu);
            if (!enabled[interleaved][dev]) {
                const cudaError_t err = cudaFuncSetAttribute(
                    kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
                if (err != cudaSuccess)
                    return record_cuda(err);
                enabled[interleaved][dev] = true;
            }
        }
        return launch_pdl(kernel, dim3((unsigned)info.sms), dim3(32 * kRingWarps), smem, stream,
                          p);
    }
    auto kernel = interleaved ? rope_and_cache_kernel<T, kFp8, true>
                              : rope_and_cache_kernel<T, kFp8, false>;
    // Threads that share the rotary items evenly, kAhead or fewer each for rows
    // of up to 96 heads of 128 (72 heads: 192 threads with 3 items), and one a
    // rotary pair at least.
    const int items = (p.num_heads + p.num_kv_heads) * (p.rot_dim / 16);
    const int rounds = (items + kRopeMaxThreads - 1) / kRopeMaxThreads;
    const int even = (items + rounds - 1) / rounds;
    const int threads = (std::max(even, p.rot_dim / 2) + 31) / 32 * 32;
    return launch_pdl(kernel, dim3((unsigned)p.num_tokens), dim3(threads), 0, stream, p);
}

static bool stride_ok(long long stride, int heads, int head_dim, int tokens)
{
    // rows of whole 16-byte words that do not overlap
    return stride % 8 == 0 && (tokens <= 1 || stride >= (long long)heads * head_dim) &&
           stride <= (1ll << 28);
}

// Whether the output's rows share bytes with an input's: exact for rows of
// one stride (parts of the same wider rows), by the whole ranges otherwise.
static bool rows_meet(const void *out, long long out_stride, int out_heads, const void *in,
                      long long in_stride, int in_heads, int head_dim, int tokens)
{
    const long long o = (long long)reinterpret_cast<uintptr_t>(out);
    const long long i = (long long)reinterpret_cast<uintptr_t>(in);
    const long long orow = 2ll * out_heads * head_dim, irow = 2ll * in_heads * head_dim;
    const long long oend = o + 2 * (tokens - 1) * out_stride + orow;
    const long long iend = i + 2 * (tokens - 1) * in_stride + irow;
    if (o >= iend || i >= oend)
        return false;
    if (tokens <= 1 || out_stride != in_stride)
        return true;
    const long long s = 2 * out_stride;
    const long long d = ((o - i) % s + s) % s;  // the output row's place after an input row
    return d < irow || s - d < orow;
}

static pa_status run_rope(void *query_out, long long qo_stride, const void *query,
                          long long q_stride, const void *key, long long k_stride,
                          const void *value, long long v_stride, void *key_cache,
                          void *value_cache, const int32_t *slot_mapping,
                          const int32_t *positions, int num_axes, const int32_t *axis_of_pair,
                          const float *inv_freq, int rot_dim, int interleaved, int num_tokens,
                          int num_heads, int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, bool fp8, float k_scale, float v_scale,
                          pa_dtype dtype, int32_t *error_word, void *stream)
{
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || num_axes <= 0 || rot_dim <= 0 ||
        rot_dim > head_dim || (interleaved != 0 && interleaved != 1) ||
        (dtype != PA_F16 && dtype != PA_BF16))
        return PA_ERR_INVALID_ARG;
    if (fp8 && !(std::isfinite(k_scale) && std::isfinite(v_scale) && k_scale > 0.f &&
                 v_scale > 0.f))
        return PA_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || head_dim > 2 * kRopeMaxPairs || rot_dim % 16 != 0 ||
        num_axes > 255 || num_heads > (1 << 16) || num_kv_heads > (1 << 16) ||
        (long long)num_blocks * block_size >= (1ll << 31))
        return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0)
        return PA_OK;
    if (!query_out || !query || !key || !value || !key_cache || !value_cache ||
        !slot_mapping || !positions || !inv_freq)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(query_out) || !aligned16(query) || !aligned16(key) || !aligned16(value) ||
        !aligned16(key_cache) || !aligned16(value_cache))
        return PA_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, num_heads, head_dim, num_tokens) ||
        !stride_ok(qo_stride, num_heads, head_dim, num_tokens) ||
        !stride_ok(k_stride, num_kv_heads, head_dim, num_tokens) ||
        !stride_ok(v_stride, num_kv_heads, head_dim, num_tokens))
        return PA_ERR_INVALID_ARG;
    // in place: the query's own rows, never a key's or a value's (they are read while
    // the query is written)
    const bool in_place = query_out == query && qo_stride == q_stride;
    if ((!in_place && rows_meet(query_out, qo_stride, num_heads, query, q_stride, num_heads,
                                head_dim, num_tokens)) ||
        rows_meet(query_out, qo_stride, num_heads, key, k_stride, num_kv_heads, head_dim,
                  num_tokens) ||
        rows_meet(query_out, qo_stride, num_heads, value, v_stride, num_kv_heads, head_dim,
                  num_tokens))
        return PA_ERR_INVALID_ARG;
    RopeParams p;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const int a = axis_of_pair != nullptr ? axis_of_pair[i] : 0;
        if (a < 0 || a >= num_axes)
            return PA_ERR_INVALID_ARG;
        p.axis[i] = (uint8_t)a;
    }
    p.query_out = query_out;
    p.query = query;
    p.key = key;
    p.value = value;
    p.key_cache = key_cache;
    p.value_cache = value_cache;
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.error_word = error_word;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.qo_stride = qo_stride;
    p.num_slots = (long long)num_blocks * block_size;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.k_inv_scale = 1.0f / k_scale;  // fp32, as the codes' contract states
    p.v_inv_scale = 1.0f / v_scale;
    cudaStream_t st = as_stream(stream);
    if (dtype == PA_BF16)
        return fp8 ? launch_rope<__nv_bfloat16, true>(p, interleaved, st)
                   : launch_rope<__nv_bfloat16, false>(p, interleaved, st);
    return fp8 ? launch_rope<__half, true>(p, interleaved, st)
               : launch_rope<__half, false>(p, interleaved, st);
}

} // namespace pa

using namespace pa;

extern "C" pa_status pa_rope_and_cache(
    void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
    const void *key, int64_t key_stride, const void *value, int64_t value_stride,
    void *key_cache, void *value_cache, const int32_t *slot_mapping, const int32_t *positions,
    int num_axes, const int32_t *axis_of_pair, const float *inv_freq, int rot_dim,
    int interleaved, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, pa_dtype dtype, int32_t *error_word, void *stream)
{
    return run_rope(query_out, query_out_stride, query, query_stride, key, key_stride, value,
                    value_stride, key_cache, value_cache, slot_mapping, positions, num_axes,
                    axis_of_pair, inv_freq, rot_dim, interleaved, num_tokens, num_heads,
                    num_kv_heads, head_dim, block_size, num_blocks, false, 1.f, 1.f, dtype,
                    error_word, stream);
}

extern "C" pa_status pa_rope_and_cache_fp8(
    void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
    const void *key, int64_t key_stride, const void *value, int64_t value_stride,
    void *key_cache, void *value_cache, const int32_t *slot_mapping, const int32_t *positions,
    int num_axes, const int32_t *axis_of_pair, const float *inv_freq, int rot_dim,
    int interleaved, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, pa_dtype dtype, float k_scale, float v_scale,
    int32_t *error_word, void *stream)
{
    return run_rope(query_out, query_out_stride, query, query_stride, key, key_stride, value,
                    value_stride, key_cache, value_cache, slot_mapping, positions, num_axes,
                    axis_of_pair, inv_freq, rot_dim, interleaved, num_tokens, num_heads,
                    num_kv_heads, head_dim, block_size, num_blocks, true, k_scale, v_scale,
                    dtype, error_word, stream);
}
