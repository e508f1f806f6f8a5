// pa_window_tiles.cu -- chunked prefill and mixed batches over paged pools with a
// sliding window and a few first tokens that stay visible, for sm_103a, on the
// 5th-generation tensor cores.
//
// Row of sequence s at position pos, window W, first tokens N:
//     seen = { p <= pos : p > pos - W  or  p < N }
//     out = sum_{p seen} softmax_p(scale * q . k_p) v_p
// ("PagedAttention & Continuous Batching" §2.4, §2.5 for the chunk; the window
// is an addition).
//
// What bounds it: the tensor cores (4 d flop a row and key), and beside them
// the softmax of every score.  A CTA (one an SM, all of its tensor memory) works
// through 128 query rows of one KV head at a time, in steps of 128 keys.  Times
// below: 8,192 rows of 4 sequences, 32 heads over 8, d 128, window 4,096 and 64
// first tokens of up to 32,768, blocks of 32 (0.56 TFLOP of rows and keys seen:
// 376 us by itself, 1.49 PFLOP/s; in a run of calls 417, 1.34 PFLOP/s, where the power
// limit sets the clock: 1,370 of 1,400 W at 1,725 of 2,070 MHz); and 2,048 rows of 4
// sequences, 64 heads over 8, window 512, blocks of 16 (37.6 us, 0.69 PFLOP/s).
//  * A score product reads its query rows from shared memory for every step,
//    so N = 128 keys cost what 64 do (~60 cycles an MMA for either); 64-key
//    steps pay that, and every barrier and commit, twice (505 us).
//  * Sixteen warps, each kind with a clock of its own.  0-3 and 4-7: the softmax
//    of even and odd steps, one thread a row, with a reference maximum that moves
//    only when a score passes it by 2^8 and goes from one set to the other
//    through shared memory as soon as it is known.  (A step's softmax takes
//    ~1,500 cycles of four warps, its products ~1,000 of the tensor cores: one
//    set alone 430 us.)  8-11: output rows, while the next unit is computed
//    (left to the softmax warps: 411).  12: key and query fetches, 13: value
//    fetches, 14: score products, 15: value products (both from one warp: 568,
//    since a wait for either held up the other).
//  * Tensor memory: three S buffers of 128 fp32 columns and O.  P goes over the
//    first half of its S as 16-bit pairs, in two halves of 64 keys, so the value
//    product starts on the first while the second is computed; the third S
//    lets the scores run a whole step ahead of the softmax (two: 519).
//  * The softmax step is a loop over halves, not unrolled over 128 scores: two sets
//    of warps at different places of a long body missed in the instruction cache.
//  * Keys are counted without a gap ("compact positions", at the grain of one
//    TMA box): the first tokens' boxes, then the window's, `skip` tokens further
//    on; row r sees c with c < lim_r and (c >= low_r or c < N).  Steps past the
//    window do not exist, and a last step of 64 keys or fewer is done at half
//    size.
//  * A TMA box takes ~70 cycles to issue whatever its size, so a box brings both
//    d-halves of its tokens, as atoms of 8 tokens that the descriptors step over
//    (a box a half: 403 us, and 479 instead of 400 for blocks of 16), and 32
//    tokens where a block holds them.
//  * The roles meet only at mbarriers; every wait is bounded, the first to run
//    out stops all of them, and tensor memory is released on every path.
//  * Query tiles hold floor(128 / G) whole tokens, so that any group size
//    arrives by one TMA box a d-half.
//  * Value rows that no row of a unit sees are zeroed in shared memory by the
//    value-product warp (an output warp, busy with the unit before: 382 us and
//    40.7), so that NaN or another sequence's rows never meet a zero weight; a row
//    that still comes out non-finite is computed anew from the keys it sees alone,
//    after the CTA's last unit, when no other role waits.
//  * FP8 pools: codes land where the upper half of their fp16 tile will be (d
//    128; beside it at d 64) and the output warps widen them, in whatever order
//    keys, values, query tiles and finished units come: 32 KB of codes written and
//    read and 64 KB of fp16 written a step (580 us and 58).  No unit is busy all
//    the time by its counter: tensor pipe 43 %, the shared-memory pipe of the warps'
//    loads and stores 49 % (the operands' reads come on top), issue 49 %.  The query
//    is rounded to fp16, the K scale joins the exponent's scale and the V scale the
//    output.
// P is rounded to the operands' type, relative error 2^-8 (bf16) or 2^-11: about
// that of the rounded output; the sum keeps the unrounded fp32 weights.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "pa_window.cuh"

namespace pa {

constexpr int kWtRows = 128;      // rows of a tile (M of the MMAs)
constexpr int kWtKeys = 128;      // keys of a step
constexpr int kWtHalf = 64;       // keys of a half step
constexpr int kWtOutWarp = 8;       // warps 0-3 and 4-7: softmax of even and odd steps
constexpr int kWtKeyWarp = 12;      // 8-11: output rows (FP8 pools: codes widened too)
constexpr int kWtValueWarp = 13;
constexpr int kWtScoreWarp = 14;
constexpr int kWtThreads = 512;     // (15: value products, hidden value rows)
constexpr uint32_t kWtTmemCols = 512;  // S at 0, 128 and 256 (P over each), O at 384
constexpr uint32_t kWtTmemO = 384;
constexpr int kWtOrderBuckets = 64;
constexpr int kWtOrderSegs = 512;

// A work unit: the tokens of a tile of one KV head, and their keys.
struct WtUnit {
    int row0;           // first query row (token) of the unit
    int kh;             // KV head
    int count;          // tokens
    int pos0;           // position of the first token
    int skip;           // real minus compact position, from the window on
    int kend;           // compact keys
    int hide0, hide1;   // compact keys that no row sees: [hide0, hide1)
    int seq;            // sequence (its table)
    __device__ int steps() const { return (kend + kWtKeys - 1) / kWtKeys; }
    // a last step of 64 keys or fewer
    __device__ bool half(int si) const { return half(kend, si); }
    __device__ static bool half(int kend, int si) { return kend - si * kWtKeys <= kWtHalf; }
    // a value row (compact position) that no row of the unit sees
    __device__ bool unseen(int c) const { return unseen(kend, hide0, hide1, c); }
    __device__ static bool unseen(int kend, int hide0, int hide1, int c)
    {
        return c >= kend || (c >= hide0 && c < hide1);
    }
    // whether step si has such rows
    __device__ bool hidden(int si) const
    {
        const int c0 = si * kWtKeys;
        return c0 + kWtKeys > kend || (hide1 > max(hide0, c0) && hide0 < c0 + kWtKeys);
    }
};
// units of a CTA kept in shared memory; later ones are worked out by each role
constexpr int kWtUnits = 192;

// Step g's slot g % 3 and the parity of g / 3, counted along.
struct Slot3 {
    int i = 0;
    uint32_t ph = 0;
    __device__ void next()
    {
        if (++i == 3) {
            i = 0;
            ph ^= 1;
        }
    }
    __device__ Slot3 before() const { return i > 0 ? Slot3{i - 1, ph} : Slot3{2, ph ^ 1}; }
};

template <int D, bool kFp8> struct WtLayout {
    static constexpr int kHalves = D / 64;               // 128-byte rows of 64 elements
    static constexpr int kHalfBytes = 128 * 128;         // 128 rows of one d-half
    static constexpr int kTile = kHalves * kHalfBytes;   // a query tile, or K or V of a step
    // K and V of a step are atoms of 8 tokens x 64 elements (1,024 bytes): atom
    // (token group j, d-half f) at j kGroup + f kPart.  16-bit pools: one TMA
    // box brings both halves, so they alternate
    static constexpr int kGroup = kFp8 ? 1024 : kHalves * 1024;
    static constexpr int kPart = kFp8 ? kHalfBytes : 1024;
    static constexpr int kK = 0;                         // 2 stages
    static constexpr int kV = 2 * kTile;                 // 2 stages
    static constexpr int kQ = 4 * kTile;                 // 2 query tiles
    // FP8 pools: where a step's codes land, [stage][K, V]: the upper half of
    // their own 16-bit tile at d 128, a place of their own at d 64
    static constexpr int kCodeTile = kWtKeys * D;
    static constexpr int kCodes = 6 * kTile;
    static constexpr int kRef = kCodes + (kFp8 && D == 64 ? 4 * kCodeTile : 0);
                                                         // float reference [2 steps][128]
    static constexpr int kPartL = kRef + 2 * 128 * 4;    // float l, m [2 units][2][128]
    static constexpr int kPartM = kPartL + 4 * 128 * 4;
    static constexpr int kBars = kPartM + 4 * 128 * 4;   // 34 mbarriers
    static constexpr int kTmemSlot = kBars + 34 * 8;
    static constexpr int kAbort = kTmemSlot + 8;
    static constexpr int kUnits = kTmemSlot + 16;        // the CTA's first units
    // int unit prefix[n + 1], then (ordered) order[n], units[n], key[n] and
    // the sort's buckets
    static constexpr int kSeg = kUnits + kWtUnits * (int)sizeof(WtUnit);
    static size_t bytes(int segments, bool ordered)
    {
        return 1024 + kSeg + 4 * ((size_t)segments + 1) +
               (ordered ? 4 * (3 * (size_t)segments + kWtOrderBuckets) : 0);
    }
    static_assert(1024 + kSeg + 4 * (kWindowMaxSeqs + 1) <= 227 * 1024 &&
                      kWindowMaxSeqs > 4 * kWtOrderSegs + kWtOrderBuckets,
                  "a CTA's shared memory");
};

// 16 columns of this warp's 32 lanes, without waiting for the store.
__device__ __forceinline__ void tmem_st_x16_nowait(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, "
                 "%9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                 "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint4 load_shared(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ void store_shared(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// x * 0 + acc of two 16-bit values.
template <typename T>
__device__ __forceinline__ uint32_t fma_zero_x2(uint32_t x, uint32_t acc)
{
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0), "r"(acc));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0), "r"(acc));
    return r;
}

// Whether a barrier's phase has completed (never suspends, unlike a try_wait).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t"
                 ".reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t"
                 "}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}

// The rest of a wait whose phase has not completed yet.  Out of line: it is
// called from a dozen places, and the roles' loops have to stay short enough
// for the instruction cache.
__device__ __noinline__ bool wt_wait_slow(uint32_t b, uint32_t parity, uint64_t limit_ns,
                                          volatile int *abort_flag)
{
    bool ok = *abort_flag == 0 && mbar_wait_bounded(b, parity, limit_ns);
    ok = __all_sync(kFull, ok);
    if (!ok)
        *abort_flag = 1;
    return ok;
}

// T: the query's and output's type; kFp8: the pools hold e4m3 codes (else T).
template <typename T, int D, int kBox, bool kFp8>
__global__ void __launch_bounds__(kWtThreads, 1)
    window_tiles_kernel(const __grid_constant__ WindowMqParams p,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ CUtensorMap tmap_q)
{
    using L = WtLayout<D, kFp8>;
    using OT = typename std::conditional<kFp8, __half, T>::type;  // operand type
    constexpr bool kBf16 = std::is_same<OT, __nv_bfloat16>::value;
    constexpr bool kConvQ = !std::is_same<OT, T>::value;  // queries rounded to fp16 here
    constexpr uint32_t kIdescS = idesc_f16(kBf16, kWtRows, kWtKeys, false, false);
    constexpr uint32_t kIdescSHalf = idesc_f16(kBf16, kWtRows, kWtHalf, false, false);
    constexpr uint32_t kIdescO = idesc_f16(kBf16, kWtRows, D, false, true);
    constexpr int KT = D / 16;
    constexpr int kSubs = kWtKeys / kBox;  // boxes of a step

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_addr(smem);
    int *pref = reinterpret_cast<int *>(smem + L::kSeg);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kAbort);
    // mbarriers.  [parity of the step]: K / V of a stage ready; its codes landed
    // (FP8 pools); the rows' references after the step stored.
    // [step % 3]: S computed (frees the K stage); half h of P stored by the 4
    // softmax warps; value product done (frees S, P and the V stage).  (A wait
    // for a step's phase needs the next step on the same barrier to depend on
    // the waiter: the products of step g + 2 do not depend on a wait for step
    // g's, those of step g + 3 do.)
    // [parity of the unit]: query tile ready; the unit's last value product
    // done; its sums stored by the 8 softmax warps; its O and sums read by 4.
    // Every tensor-core operation done.
    auto bar = [&](int i) { return sbase + L::kBars + 8 * i; };
    auto kfull = [&](int st) { return bar(st); };
    auto vfull = [&](int st) { return bar(2 + st); };
    auto mfull = [&](int st) { return bar(8 + st); };
    auto qfull = [&](int b) { return bar(10 + b); };
    auto ufull = [&](int b) { return bar(12 + b); };
    auto lfull = [&](int b) { return bar(14 + b); };
    auto ufree = [&](int b) { return bar(16 + b); };
    auto sfull = [&](int i) { return bar(18 + i); };
    auto pfull = [&](int h, int i) { return bar(21 + 3 * h + i); };
    auto ofull = [&](int i) { return bar(27 + i); };
    // FP8 pools: the codes of K and V landed, a bf16 query tile landed
    auto kland = [&](int st) { return bar(30 + st); };
    auto vland = [&](int st) { return bar(4 + st); };
    auto qland = [&](int b) { return bar(32 + b); };
    auto mma_drain = [&](int i) { return bar(6 + i); };
    float *ref_s = reinterpret_cast<float *>(smem + L::kRef);
    float *part_l = reinterpret_cast<float *>(smem + L::kPartL);
    float *part_m = reinterpret_cast<float *>(smem + L::kPartM);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.group, Hkv = p.num_kv_heads, H = p.num_heads;
    const int nseg = p.num_segments;
    const int tok_unit = kWtRows / G;  // whole tokens of a tile

    if (tid == 0) {
        for (int st = 0; st < 2; ++st) {
            mbar_init(kfull(st), kFp8 ? 4 : 1);  // (FP8 pools: widened by 4 warps)
            mbar_init(vfull(st), kFp8 ? 4 : 1);
            mbar_init(vland(st), 1);
            mbar_init(kland(st), 1);
            mbar_init(qfull(st), kConvQ ? 4 : 1);
            mbar_init(qland(st), 1);
            mbar_init(ufull(st), 1);
            mbar_init(lfull(st), 8);
            mbar_init(mfull(st), 4);
            mbar_init(ufree(st), 4);
        }
        for (int b = 0; b < 3; ++b) {
            mbar_init(sfull(b), 1);
            mbar_init(ofull(b), 1);
            mbar_init(pfull(0, b), 4);
            mbar_init(pfull(1, b), 4);
        }
        mbar_init(mma_drain(0), 1);
        mbar_init(mma_drain(1), 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
        prefetch_tensormap(&tmap_q);
    }
    pdl_wait_primary();
    if (warp == 0) {
        tmem_alloc(sbase + L::kTmemSlot, kWtTmemCols);
        tmem_relinquish();
    }

    // ---- work units per sequence and their prefix sums --------------------------------
    auto units_of = [&](int s) {
        return (window_rows(p, s, true) + tok_unit - 1) / tok_unit;
    };
    int *order = pref + nseg + 1;  // k-th sequence of the unit order (ordered)
    const bool ordered = p.ordered != 0;
    if (warp == 1) {
        int *seg_units = order + nseg;
        if (ordered) {
            // counting sort by the keys of the sequence's last row, most
            // first, by index within a count; every CTA computes the same order
            int *seg_key = seg_units + nseg;
            int *hist = seg_key + nseg;
            hist[lane] = 0;
            hist[lane + 32] = 0;
            __syncwarp();
            for (int sg = lane; sg < nseg; sg += 32) {
                const int key = window_order_key(p, sg, kWtOrderBuckets);
                seg_units[sg] = units_of(sg);
                seg_key[sg] = key;
                atomicAdd(&hist[key], 1);
            }
            __syncwarp();
            const int c0 = hist[2 * lane], c1 = hist[2 * lane + 1];
            int x = c0 + c1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o)
                    x += y;
            }
            __syncwarp();
            hist[2 * lane] = x - c0 - c1;  // first place of each count
            hist[2 * lane + 1] = x - c1;
            __syncwarp();
            for (int base = 0; base < nseg; base += 32) {
                const int sg = base + lane;
                const int key = sg < nseg ? seg_key[sg] : -1;
                const unsigned same = __match_any_sync(kFull, key);
                const int rank = __popc(same & ((1u << lane) - 1u));
                const int off = key >= 0 ? hist[key] : 0;
                __syncwarp();
                if (key >= 0) {
                    order[off + rank] = sg;
                    if (rank == 0)
                        hist[key] = off + __popc(same);
                }
                __syncwarp();
            }
        }
        int carry = 0;
        for (int base = 0; base < nseg; base += 32) {
            const int k = base + lane;
            const int n = k < nseg ? (ordered ? seg_units[order[k]] : units_of(k)) : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o)
                    x += y;
            }
            // (about 2^24 units a sequence at most, 2^30 in 32 of them)
            if (k < nseg)
                pref[k] = min(carry + x - n, p.max_units);
            carry += __shfl_sync(kFull, x, 31);
            if (carry > p.max_units) {
                // more rows than there are: offsets that decrease somewhere
                carry = p.max_units;
                flag_error(p.error_word, PA_DEVERR_TOKEN_RANGE);
            }
        }
        if (lane == 0)
            pref[nseg] = carry;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (a shuffle, so that the compiler knows it to be the same in every lane:
    // MMA operands live in uniform registers)
    const uint32_t tmem = __shfl_sync(
        kFull, *reinterpret_cast<volatile uint32_t *>(smem + L::kTmemSlot), 0);
    const int total_units = pref[nseg] * Hkv;
    // the number of this CTA's k-th unit in the deal: round-robin, or
    // boustrophedon over the ordered units (k is kept below 2^31 / grid)
    const int grid = gridDim.x;
    auto unit_no = [&](int k) -> int {
        return k * grid + (ordered && (k & 1) ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
    };
    const int my_units = total_units > (int)blockIdx.x ? (total_units - 1) / grid + 1 : 0;

    // ---- unit -> (sequence, KV head, tokens, keys) -------------------------------------
    // Every role walks the same units in the same order and counts the same
    // steps, so step g (over this CTA's units) names its ring stage g % 2 and
    // the phase g / 2 of every barrier of that stage.
    const int sinks = p.num_sinks, sink_tokens = p.sink_tokens;
    auto work_out = [&](int u) -> WtUnit {
        WtUnit w;
        const int q = u / Hkv;
        w.kh = u - q * Hkv;
        int lo = 0, hi = nseg - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pref[mid] <= q)
                lo = mid;
            else
                hi = mid - 1;
        }
        w.seq = ordered ? order[lo] : lo;
        const int rows = window_rows(p, w.seq);
        // ordered: the sequence's units last-first
        const int tok0 = (ordered ? pref[lo + 1] - 1 - q : q - pref[lo]) * tok_unit;
        w.row0 = window_row0(p, w.seq, false) + tok0;
        w.count = min(tok_unit, rows - tok0);
        const int ctx = window_context(p, w.seq);
        w.pos0 = ctx - rows + tok0;
        const int end = max(0, w.pos0 + w.count);        // one past the last key
        const int low = window_low(w.pos0, p.window);    // the first row's window
        w.skip = max(0, (low & ~(kBox - 1)) - sink_tokens);
        w.kend = end - w.skip;
        w.hide0 = sinks;
        w.hide1 = min(low - w.skip, w.kend);
        return w;
    };
    // the CTA's units, worked out once, a thread each (a role that did it at
    // each unit's start would add a few trips to L2 to every unit)
    WtUnit *unit_s = reinterpret_cast<WtUnit *>(smem + L::kUnits);
    if (tid < kWtUnits && tid < my_units && unit_no(tid) < total_units)
        unit_s[tid] = work_out(unit_no(tid));
    __syncthreads();
    // the CTA's k-th unit; false past its last one (in the last round of the
    // ordered deal, where the CTAs are taken backwards, it may have none)
    auto unit_at = [&](int k, WtUnit &w) -> bool {
        if (k >= my_units || unit_no(k) >= total_units)
            return false;
        w = k < kWtUnits ? unit_s[k] : work_out(unit_no(k));
        return true;
    };
    // a bounded wait, warp-uniform; the first one to run out stops every role
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        return __all_sync(kFull, mbar_try_wait(b, parity)) ||
               wt_wait_slow(b, parity, p.wait_ns, abort_flag);
    };

    // rows of a unit: row r is token r / G, head r % G of the group
    const int r = tid & (kWtRows - 1);
    const int tok = r / G, hg = r - (r / G) * G;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;

    if (warp < kWtOutWarp) {
        // ===== softmax warps: warps 0-3 the even steps, 4-7 the odd ones ====================
        const int wg = warp >> 2;
        uint32_t g = 0, nu = 0;  // steps, units with keys
        Slot3 s3;
        bool ok = true;
        WtUnit w;
        for (int ku = 0; ok && unit_at(ku, w); ++ku) {
            const int steps = w.steps();
            if (steps == 0)
                continue;  // (the output warps write its zero rows)
            const bool row = r < tok_unit * G && tok < w.count;
            // compact: one past the row's own position, its window's start
            const int lim = row ? w.pos0 + tok + 1 - w.skip : 0;
            const int low = window_low(w.pos0 + tok, p.window) - w.skip;
            const uint32_t o_at = tmem + lanes + kWtTmemO;
            float m_own = -INFINITY, l_own = 0.f;  // reference, and sum relative to it
            for (int si = 0; si < steps; ++si, ++g, s3.next()) {
                if ((int)(g & 1) != wg)
                    continue;  // the other warps' step
                const int st = g & 1;
                const uint32_t s_at = tmem + lanes + s3.i * kWtKeys;
                const int c0 = si * kWtKeys;
                const int halves = w.half(si) ? 1 : 2;
                auto load_half = [&](int h, float (&sv)[kWtHalf]) {
                    uint32_t v[kWtHalf];
                    tmem_ld_32x32b_x64(s_at + h * kWtHalf, v);
#pragma unroll
                    for (int i = 0; i < kWtHalf; ++i)
                        sv[i] = __uint_as_float(v[i]);
                };
                // Scores hidden from this row become -inf, and go back so: they
                // come in a few steps of a unit and there mostly in one place,
                // so each 32 keys are looked at by themselves.
                auto hide = [&](int h, float (&sv)[kWtHalf]) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int cb = c0 + h * kWtHalf + 32 * q;
                        const bool open = lim >= cb + 32 && (low <= cb || sinks >= cb + 32);
                        if (__all_sync(kFull, open))
                            continue;
                        auto below = [&](int c) -> uint32_t {  // bits of keys < c
                            const int k = c - cb;
                            return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
                        };
                        const uint32_t seen = below(lim) & (~below(low) | below(sinks));
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float &x = sv[32 * q + i];
                            x = (seen >> i) & 1u ? x : -INFINITY;
                            v[i] = __float_as_uint(x);
                        }
                        tmem_st_32x32b_x32(s_at + h * kWtHalf + 32 * q, v);
                    }
                };
                ok = wait(sfull(s3.i), s3.ph);
                if (!ok)
                    break;
                tc_fence_after();
                // The loops over halves stay loops: unrolled, the step's code in
                // two sets of warps passes the instruction cache (85 % of its
                // throughput measured).  Reading S twice costs less than holding it.
                float mx = -INFINITY;  // maximum raw score (the scale is positive)
#pragma unroll 1
                for (int h = 0; h < halves; ++h) {
                    float sv[kWtHalf];
                    load_half(h, sv);
                    hide(h, sv);
                    float m22[22], m8[8];
#pragma unroll
                    for (int k = 0; k < 21; ++k)
                        m22[k] = fmax3(sv[3 * k], sv[3 * k + 1], sv[3 * k + 2]);
                    m22[21] = fmaxf(sv[63], mx);
#pragma unroll
                    for (int k = 0; k < 7; ++k)
                        m8[k] = fmax3(m22[3 * k], m22[3 * k + 1], m22[3 * k + 2]);
                    m8[7] = m22[21];
                    mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                               fmaxf(m8[6], m8[7]));
                }
                mx *= p.scale_log2;
                // the reference after the step before (a unit's first: none); it
                // moves only when a score passes it by 2^kSlack
                float m_in = -INFINITY;
                if (g > 0) {
                    const uint32_t gp = g - 1;
                    ok = wait(mfull(gp & 1), (gp >> 1) & 1);
                    if (!ok)
                        break;
                    if (si > 0)
                        m_in = ref_s[(gp & 1) * kWtRows + r];
                }
                const bool moved = mx > m_in + kSlack;
                const float m_ref = moved ? mx : m_in;
                ref_s[st * kWtRows + r] = m_ref;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(mfull(st));
                if (m_ref != m_own) {
                    l_own *= exp2f(m_own - m_ref);  // 0 while m_own is -inf
                    m_own = m_ref;
                }
                // a reference moved: rescale O once the value product before is done
                if (si > 0 && __any_sync(kFull, moved)) {
                    const Slot3 sp = s3.before();
                    ok = wait(ofull(sp.i), sp.ph);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const float alpha = moved ? exp2f(m_in - m_ref) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(o_at + c * 32, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st_32x32b_x32(o_at + c * 32, o);
                    }
                }
                const float neg_mu = m_ref == -INFINITY ? 0.f : -m_ref;
                const uint64_t sl2 = pack_f32x2(p.scale_log2, p.scale_log2);
                const uint64_t nm2 = pack_f32x2(neg_mu, neg_mu);
                uint64_t acc[2] = {pack_f32x2(0.f, 0.f), pack_f32x2(0.f, 0.f)};
#pragma unroll 1
                for (int h = 0; h < halves; ++h) {
                    float sv[kWtHalf];
                    load_half(h, sv);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pw[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int k = 32 * c + 2 * i;
                            float e0, e1;
                            unpack_f32x2(ffma_f32x2(pack_f32x2(sv[k], sv[k + 1]), sl2, nm2), e0,
                                         e1);
                            const float p0 = exp2f(e0), p1 = exp2f(e1);
                            acc[i & 1] = fadd_f32x2(acc[i & 1], pack_f32x2(p0, p1));
                            pw[i] = MmaOp<OT>::pack(p0, p1);
                        }
                        // over the first half of S, which both passes have read
                        tmem_st_x16_nowait(s_at + 32 * h + 16 * c, pw);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(pfull(h, s3.i));
                }
                if (halves == 1 && lane == 0)
                    mbar_arrive(pfull(1, s3.i));  // (nobody waits for it; it keeps step)
                {
                    float a0, a1, b0, b1;
                    unpack_f32x2(acc[0], a0, a1);
                    unpack_f32x2(acc[1], b0, b1);
                    l_own += (a0 + a1) + (b0 + b1);
                }
            }
            if (!ok)
                break;
            // this unit's sums, once unit nu - 2's have been read
            const int b = nu & 1;
            if (nu >= 2) {
                ok = wait(ufree(b), ((nu - 2) >> 1) & 1);
                if (!ok)
                    break;
            }
            part_l[(2 * b + wg) * kWtRows + r] = l_own;
            part_m[(2 * b + wg) * kWtRows + r] = m_own;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(lfull(b));
            ++nu;
        }
    } else if (warp < kWtKeyWarp) {
        // ===== output warps: O / l of a unit, while the next one is computed ==============
        const bool out32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        // this thread's row of a unit
        auto row_of = [&](const WtUnit &w) -> T * {
            return r < tok_unit * G && tok < w.count
                       ? static_cast<T *>(p.out) +
                             (((long long)w.row0 + tok) * H + w.kh * G + hg) * D
                       : nullptr;
        };
        auto zero_row = [&](const WtUnit &w) {  // a unit without keys
            uint4 *dst = reinterpret_cast<uint4 *>(row_of(w));
            if (dst != nullptr)
                for (int c = 0; c < D / 8; ++c)
                    dst[c] = make_uint4(0, 0, 0, 0);
        };
        constexpr int kOutUnroll = kFp8 ? D / 32 : 1;
        unsigned mend = 0;  // the mask of unit `lane` (the last lane: all from there on)
        int units_done = 0;
        // A unit's rows (the CTA's steps up to its end: g), once its sums and last
        // value product are there: rounded and stored, O given back.
        auto write_rows = [&](const WtUnit &w, int ku, uint32_t g, int b) {
            tc_fence_after();
            // O is relative to the last step's reference, which the softmax
            // warps of that step have; the others' is not above it
            const int a0 = (2 * b + (int)((g - 1) & 1)) * kWtRows + r;
            const int a1 = (2 * b + (int)(g & 1)) * kWtRows + r;
            const float l0 = part_l[a0], l1 = part_l[a1];
            const float l = l1 == 0.f ? l0 : l0 + l1 * exp2f(part_m[a1] - part_m[a0]);
            // no weight (0 / 0): of keys that all have a score of -inf the softmax is not
            // a number; a row at a negative position, which sees no key, gets its
            // zeros below
            const float inv = p.out_scale / l;
            // (a sum that is NaN comes from scores that the row sees: it is its softmax)
            const unsigned real = __ballot_sync(kFull, l >= 0.f);
            const uint64_t inv2 = pack_f32x2(inv, inv), zero2 = pack_f32x2(0.f, 0.f);
            const uint32_t o_at = tmem + lanes + kWtTmemO;
            T *const dst = row_of(w);
            // rows that come out non-finite, perhaps for a value hidden from them:
            // x * 0 + nan is a sum that stays zero while everything is finite
            uint32_t nan = 0;
            // (16-bit pools: a loop; unrolled, it took the tensor-core warps' code
            // out of the instruction cache at the end of every unit, 38.3 us for
            // 37.6.  FP8 pools, where these warps' polling loop is the larger part:
            // unrolled, 569 us for 614 and 57 for 59)
#pragma unroll kOutUnroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32], v[16];
                tmem_ld_32x32b_x32(o_at + c * 32, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float lo, hi;
                    unpack_f32x2(ffma_f32x2(pack_f32x2(__uint_as_float(o[2 * k]),
                                                       __uint_as_float(o[2 * k + 1])),
                                            inv2, zero2),
                                 lo, hi);
                    v[k] = MmaOp<T>::pack(lo, hi);
                    nan = fma_zero_x2<T>(v[k], nan);
                }
                if (dst == nullptr)
                    continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    T *at = dst + 32 * c + 16 * i;
                    if (out32) {
                        asm volatile(
                            "st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at),
                            "r"(v[8 * i]), "r"(v[8 * i + 1]), "r"(v[8 * i + 2]),
                            "r"(v[8 * i + 3]), "r"(v[8 * i + 4]), "r"(v[8 * i + 5]),
                            "r"(v[8 * i + 6]), "r"(v[8 * i + 7])
                            : "memory");
                    } else {
                        reinterpret_cast<uint4 *>(at)[0] =
                            make_uint4(v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3]);
                        reinterpret_cast<uint4 *>(at)[1] =
                            make_uint4(v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]);
                    }
                }
            }
            // O is read: the next unit's value products may write it
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(ufree(b));
            unsigned todo =
                real & __ballot_sync(kFull, dst != nullptr && (nan & 0x7fff7fffu) != 0);
            // (looked at after the last unit, when nobody waits for this warp)
            if (lane == min(ku, 31))
                mend |= todo;
        };
        if constexpr (!kFp8) {
            uint32_t g = 0, nu = 0;
            WtUnit w;
            for (int ku = 0; unit_at(ku, w); ++ku) {
                const int steps = w.steps();
                if (steps == 0) {
                    zero_row(w);
                    continue;
                }
                g += steps;
                const int b = nu & 1;
                const uint32_t ph = (nu >> 1) & 1;
                ++nu;
                if (!wait(lfull(b), ph) || !wait(ufull(b), ph))
                    break;
                write_rows(w, ku, g, b);
                units_done = ku + 1;
            }
        } else {
            // FP8 pools: these warps also widen each step's codes to the fp16
            // operands (one thread a row; value rows that no row of the unit
            // sees become zeros) and round bf16 query tiles to fp16.  Each warp
            // takes whatever is there, its own 32 rows of it, in any order: the
            // keys of a step, its values, a query tile, a finished unit.
            struct Walk {  // steps of one kind done so far, at step si of unit ku
                int ku = -1, si = 0, steps = 0;
                uint32_t g = 0, nu = 0;
                bool more = true;
                int kend, hide0, hide1, count;  // of the unit (what is used of it)
            };
            Walk wk, wv, wq, wo;
            // the next unit with keys (zeros for one without, where asked)
            auto open = [&](Walk &x, bool zeros) {
                x.si = 0;
                x.steps = 0;
                while (x.more && x.steps == 0) {
                    WtUnit w;
                    x.more = unit_at(++x.ku, w);
                    if (x.more) {
                        x.steps = w.steps();
                        x.kend = w.kend;
                        x.hide0 = w.hide0;
                        x.hide1 = w.hide1;
                        x.count = w.count;
                        if (x.steps == 0 && zeros)
                            zero_row(w);
                    }
                }
            };
            auto half = [&](const Walk &x) { return WtUnit::half(x.kend, x.si); };
            auto step = [&](Walk &x) {
                ++x.g;
                if (++x.si == x.steps)
                    open(x, false);
            };
            // this thread's row (keys: of the tile at `tile`) from its codes
            auto widen = [&](uint32_t tile, uint32_t codes, bool zero) {
                uint4 src[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    src[c] = zero ? make_uint4(0, 0, 0, 0)
                                  : load_shared(codes + r * D + (D == 128
                                                                     ? (c ^ (r & 7)) << 4
                                                                     : (c ^ ((r >> 1) & 3)) << 4));
#pragma unroll
                for (int f = 0; f < D / 8; ++f) {  // fp16 chunk f: codes 8f .. 8f + 7
                    const uint4 s = src[f >> 1];
                    const uint32_t lo = (f & 1) ? s.z : s.x, hi = (f & 1) ? s.w : s.y;
                    store_shared(tile + (f >> 3) * L::kHalfBytes + r * 128 +
                                     (((f & 7) ^ (r & 7)) << 4),
                                 make_uint4(e4m3x2_to_f16x2((uint16_t)(lo & 0xffffu)),
                                            e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
                                            e4m3x2_to_f16x2((uint16_t)(hi & 0xffffu)),
                                            e4m3x2_to_f16x2((uint16_t)(hi >> 16))));
                }
            };
            auto announce = [&](uint32_t b) {
                fence_proxy_async_smem();  // (generic stores, read by the tensor cores)
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(b);
            };
            auto there = [&](uint32_t b, uint32_t parity) -> bool {
                return __all_sync(kFull, mbar_test(b, parity));
            };
            auto code_base = [&](int st, int vals) -> uint32_t {
                return D == 128 ? sbase + (vals ? L::kV : L::kK) + st * L::kTile + L::kHalfBytes
                                : sbase + L::kCodes + (2 * st + vals) * L::kCodeTile;
            };
            open(wk, false);
            open(wv, false);
            open(wq, false);
            open(wo, true);
            if constexpr (!kConvQ)
                wq.more = false;
            bool q_over = false;  // a query element past the fp16 range
            uint64_t idle_since = 0;
            while (wk.more || wv.more || wq.more || wo.more) {
                bool did = false;
                if (wk.more && there(kland(wk.g & 1), (wk.g >> 1) & 1)) {
                    const int st = wk.g & 1;
                    if (r < kWtHalf || !half(wk))
                        widen(sbase + L::kK + st * L::kTile, code_base(st, 0), false);
                    announce(kfull(st));
                    step(wk);
                    did = true;
                }
                if (wv.more && there(vland(wv.g & 1), (wv.g >> 1) & 1)) {
                    const int st = wv.g & 1;
                    if (r < kWtHalf || !half(wv))
                        widen(sbase + L::kV + st * L::kTile, code_base(st, 1),
                              WtUnit::unseen(wv.kend, wv.hide0, wv.hide1,
                                             wv.si * kWtKeys + r));
                    announce(vfull(st));
                    step(wv);
                    did = true;
                }
                if constexpr (kConvQ) {
                    if (wq.more && there(qland(wq.nu & 1), (wq.nu >> 1) & 1)) {
                        const uint32_t tile = sbase + L::kQ + (wq.nu & 1) * L::kTile;
                        const bool row = r < tok_unit * G && tok < wq.count;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            const uint32_t a = tile + (c >> 3) * L::kHalfBytes + r * 128 +
                                               (((c & 7) ^ (r & 7)) << 4);
                            uint4 x = load_shared(a);
                            uint32_t *xw = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float lo = __uint_as_float(xw[k] << 16);
                                const float hi = __uint_as_float(xw[k] & 0xffff0000u);
                                q_over |= row && fmaxf(fabsf(lo), fabsf(hi)) > 65504.f;
                                xw[k] = pack_f16x2(lo, hi);
                            }
                            store_shared(a, x);
                        }
                        announce(qfull(wq.nu & 1));
                        ++wq.nu;
                        open(wq, false);
                        did = true;
                    }
                }
                if (wo.more && there(lfull(wo.nu & 1), (wo.nu >> 1) & 1) &&
                    there(ufull(wo.nu & 1), (wo.nu >> 1) & 1)) {
                    wo.g += wo.steps;
                    WtUnit w;
                    unit_at(wo.ku, w);
                    write_rows(w, wo.ku, wo.g, wo.nu & 1);
                    units_done = wo.ku + 1;
                    ++wo.nu;
                    open(wo, true);
                    did = true;
                }
                if (did) {
                    idle_since = 0;
                    continue;
                }
                // nothing there: the bounded wait of this role
                const uint64_t now = global_timer_ns();
                if (idle_since == 0)
                    idle_since = now;
                const bool give_up = *abort_flag != 0 || now - idle_since > p.wait_ns;
                if (__any_sync(kFull, give_up)) {
                    *abort_flag = 1;
                    break;
                }
            }
            if (__any_sync(kFull, q_over) && lane == 0)
                flag_error(p.error_word, PA_DEVERR_QUERY_RANGE);
        }
        if (__any_sync(kFull, mend != 0)) {
            WtUnit w;
            for (int ku = 0; ku < units_done; ++ku) {
                const unsigned todo = __shfl_sync(kFull, mend, min(ku, 31));
                unit_at(ku, w);
                if (w.steps() > 0 && todo != 0)
                    window_mend_unit<T, D, kFp8>(p, w.seq, w.row0, w.kh, w.count, w.pos0, todo);
            }
        }
    } else {
        if (warp == kWtKeyWarp || warp == kWtValueWarp) {
            // ===== fetch warps: keys and query tiles (12), values (13) ==================
            // Lane j owns box j of every step: it looks up that box's physical
            // block one step ahead and issues it.
            const bool values = warp == kWtValueWarp;
            constexpr int kBoxBytes = kBox * D * (kFp8 ? 1 : 2);
            uint32_t g = 0;
            Slot3 s2;                     // of step g - 2
            int qk = 0;                   // next unit whose query tile goes out
            uint32_t nq = 0, nu = 0;      // query tiles issued, units with keys begun
            uint32_t last0 = 0, last1 = 0;      // last fill's barrier per stage (0: none)
            uint32_t last_ph0 = 0, last_ph1 = 0;  // and its phase
            bool ok = true;
            WtUnit w;
            for (int ku = 0; ok && unit_at(ku, w); ++ku) {
                const int steps = w.steps();
                const int32_t *table = p.block_tables + (size_t)w.seq * p.max_blocks_per_seq;
                auto lookup = [&](int si) -> int {
                    const int c = si * kWtKeys + lane * kBox;
                    if (lane >= kSubs || c >= w.kend)
                        return 0;
                    return __ldg(table + ((c + (c >= sink_tokens ? w.skip : 0)) >> p.block_shift));
                };
                int ent_next = steps > 0 ? lookup(0) : 0;
                for (int si = 0; si < steps; ++si, ++g) {
                    const int st = g & 1;
                    const uint32_t ph = (g >> 1) & 1;
                    int ent = ent_next;
                    if (ent < 0 || ent >= p.num_blocks) {
                        flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                        ent = 0;  // stays inside the pool; the rows' outputs are undefined
                    }
                    if (si + 1 < steps)
                        ent_next = lookup(si + 1);
                    // the stage's step g - 2 is consumed
                    if (g >= 2) {
                        ok = wait(values ? ofull(s2.i) : sfull(s2.i), s2.ph);
                        if (!ok)
                            break;
                        s2.next();
                    }
                    // test hook of the time-out path: a CTA's first key fill is
                    // never issued, so the wait for it runs out
                    if (!(p.withhold_fill != 0 && !values && g == 0)) {
                        const int c0 = si * kWtKeys;
                        const int nsub = min(kSubs, (w.kend - c0 + kBox - 1) / kBox);
                        const uint32_t fb = kFp8 ? (values ? vland(st) : kland(st))
                                                 : (values ? vfull(st) : kfull(st));
                        const uint32_t tile = sbase + (values ? L::kV : L::kK) + st * L::kTile;
                        const uint32_t dst =
                            !kFp8      ? tile
                            : D == 128 ? tile + L::kHalfBytes
                                       : sbase + L::kCodes + (2 * st + values) * L::kCodeTile;
                        if (lane == 0)
                            mbar_arrive_expect_tx(fb, (uint32_t)(nsub * kBoxBytes));
                        __syncwarp();
                        if (lane < nsub) {
                            const int c = c0 + lane * kBox;
                            const int tk = c + (c >= sink_tokens ? w.skip : 0);
                            const int row = tk & (p.block_size - 1);
                            if constexpr (kFp8)
                                tma_load_4d(dst + lane * kBoxBytes, values ? &tmap_v : &tmap_k,
                                            fb, 0, w.kh, row, ent);
                            else
                                tma_load_4d(dst + lane * kBoxBytes, values ? &tmap_v : &tmap_k,
                                            fb, 0, 0, w.kh * L::kHalves,
                                            (ent << (p.block_shift - 3)) + (row >> 3));
                        }
                        (st ? last1 : last0) = fb;
                        (st ? last_ph1 : last_ph0) = ph;
                    }
                    // Query tiles, two units deep: the tile of unit v goes into the
                    // place of unit v - 2's, whose last S is step g - 2 at the
                    // latest for this unit's own tile, and from its second step
                    // on for the next unit's.
                    if (!values) {
                        const uint32_t due = nu + (si > 0 ? 2 : 1);
                        WtUnit wq;
                        while (nq < due && unit_at(qk, wq)) {
                            if (wq.kend > 0) {
                                const uint32_t qb = kConvQ ? qland(nq & 1) : qfull(nq & 1);
                                if (lane == 0)
                                    mbar_arrive_expect_tx(qb, L::kHalves * 128 * tok_unit * G);
                                __syncwarp();
                                if (lane < L::kHalves)
                                    tma_load_3d(sbase + L::kQ + (nq & 1) * L::kTile +
                                                    lane * L::kHalfBytes,
                                                &tmap_q, qb, 64 * lane, wq.kh * G, wq.row0);
                                ++nq;
                            }
                            ++qk;
                        }
                    }
                }
                nu += steps > 0;
            }
            // fills still landing (after an abort the roles that wait for them
            // may have left)
            if (last0 != 0)
                mbar_wait_bounded(last0, last_ph0, kDrainWaitNs);
            if (last1 != 0)
                mbar_wait_bounded(last1, last_ph1, kDrainWaitNs);
            if (nq > 0)
                mbar_wait_bounded(kConvQ ? qland((nq - 1) & 1) : qfull((nq - 1) & 1),
                                  ((nq - 1) >> 1) & 1, kDrainWaitNs);
            if (nq > 1)
                mbar_wait_bounded(kConvQ ? qland((nq - 2) & 1) : qfull((nq - 2) & 1),
                                  ((nq - 2) >> 1) & 1, kDrainWaitNs);
        } else {
            // ===== tensor-core warps: scores (14), value products (15) ======================
            // One elected lane of each issues.  An MMA takes its warp ~60 cycles
            // to issue, about what it takes to run, and every wait some tens:
            // one warp for both would be what the kernel waits for.
            const bool scores = warp == kWtScoreWarp;
            const uint64_t desc_q0 = smem_desc_sw128(sbase + L::kQ, 16, 1024);
            const uint64_t desc_k0 = smem_desc_sw128(sbase + L::kK, 16, L::kGroup);
            const uint64_t desc_v0 = smem_desc_sw128(sbase + L::kV, L::kPart, L::kGroup);
            uint32_t g = 0, nu = 0;
            Slot3 s3;
            bool ok = true;
            WtUnit w;
            for (int ku = 0; ok && unit_at(ku, w); ++ku) {
                const int kend = w.kend;
                if (kend <= 0)
                    continue;
                const int b = nu & 1;
                const uint32_t bph = (nu >> 1) & 1;
                if (scores) {
                    ok = wait(qfull(b), bph);
                    const uint64_t dq = desc_q0 + (uint64_t)((b * L::kTile) >> 4);
#pragma unroll 1
                    for (int rem = kend; rem > 0 && ok; rem -= kWtKeys, ++g, s3.next()) {
                        const int st = g & 1;
                        // keys landed; the columns' last value product is done
                        ok = wait(kfull(st), (g >> 1) & 1) &&
                             (g < 3 || wait(ofull(s3.i), s3.ph ^ 1));
                        if (!ok)
                            break;
                        tc_fence_after();
                        const uint64_t dk = desc_k0 + (uint64_t)((st * L::kTile) >> 4);
                        const uint32_t at = tmem + s3.i * kWtKeys;
                        const uint32_t idesc = rem > kWtHalf ? kIdescS : kIdescSHalf;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < KT; ++kk) {
                                const uint32_t off_q = ((kk >> 2) * L::kHalfBytes + (kk & 3) * 32) >> 4;
                                const uint32_t off_k = ((kk >> 2) * L::kPart + (kk & 3) * 32) >> 4;
                                tc_mma_ss(at, dq + off_q, dk + off_k, idesc, kk > 0 ? 1u : 0u);
                            }
                            tc_commit(sfull(s3.i));
                        }
                    }
                } else {
#pragma unroll 1
                    for (int rem = kend; rem > 0 && ok; rem -= kWtKeys, ++g, s3.next()) {
                        const int st = g & 1;
                        ok = wait(vfull(st), (g >> 1) & 1);
                        // (FP8 pools: the warps that widen the codes do this)
                        if (!kFp8 && ok && w.hidden((kend - rem) / kWtKeys)) {
#pragma unroll 1
                            for (int i = lane; i < (rem > kWtHalf ? kWtKeys : kWtHalf); i += 32) {
                                if (!w.unseen(kend - rem + i))
                                    continue;
                                const uint32_t at = sbase + L::kV + st * L::kTile +
                                                    (i >> 3) * L::kGroup + (i & 7) * 128;
#pragma unroll
                                for (int hf = 0; hf < L::kHalves; ++hf)
#pragma unroll
                                    for (int k = 0; k < 8; ++k)
                                        asm volatile(
                                            "st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                at + hf * L::kPart + (((k + i) & 7) << 4)),
                                            "r"(0)
                                            : "memory");
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        // a unit's first value product waits until the O of the
                        // unit before has been read
                        if (rem == kend && nu > 0)
                            ok = ok && wait(ufree(b ^ 1), ((nu - 1) >> 1) & 1);
                        const int halves = rem > kWtHalf ? 2 : 1;
                        uint64_t dv = desc_v0 + (uint64_t)((st * L::kTile) >> 4);
                        uint32_t p_at = tmem + s3.i * kWtKeys;
#pragma unroll 1
                        for (int h = 0; h < halves && ok; ++h) {
                            ok = wait(pfull(h, s3.i), s3.ph);
                            if (!ok)
                                break;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 0; ks < kWtHalf / 16; ++ks)
                                    tc_mma_ts(tmem + kWtTmemO, p_at + ks * 8,
                                              dv + (uint64_t)((ks * 2 * L::kGroup) >> 4), kIdescO,
                                              (rem < kend || h > 0 || ks > 0) ? 1u : 0u);
                                if (h == halves - 1) {
                                    tc_commit(ofull(s3.i));
                                    if (rem <= kWtKeys)
                                        tc_commit(ufull(b));
                                }
                            }
                            dv += (kWtHalf / 8 * L::kGroup) >> 4;
                            p_at += 32;
                        }
                    }
                }
                ++nu;
            }
            // every tensor-core operation this warp issued has finished
            if (elect_one())
                tc_commit(mma_drain(scores ? 0 : 1));
            __syncwarp();
            mbar_wait_bounded(mma_drain(scores ? 0 : 1), 0, kDrainWaitNs);
        }
    }
    pdl_launch_dependents();

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag)
        flag_error(p.error_word, PA_DEVERR_TIMEOUT);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kWtTmemCols);
    }
}

// ---- host side -------------------------------------------------------------------

template <typename T, int D, int kBox, bool kFp8>
static pa_status launch_tiles_as(const WindowMqParams &prm, const CUtensorMap &mk,
                                const CUtensorMap &mv, const CUtensorMap &mq,
                                cudaStream_t stream, int grid, int optin)
{
    auto kernel = window_tiles_kernel<T, D, kBox, kFp8>;
    static size_t enabled[kMaxDevices];
    static std::mutex mu;
    const size_t smem = WtLayout<D, kFp8>::bytes(prm.num_segments, prm.ordered != 0);
    if (smem > (size_t)optin)
        return PA_ERR_UNSUPPORTED;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return record_cuda(e);
    {
        std::lock_guard<std::mutex> lock(mu);
        if (smem > enabled[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)smem);
            if (e != cudaSuccess)
                return record_cuda(e);
            enabled[dev] = smem;
        }
    }
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kWtThreads), smem, stream, prm, mk,
                      mv, mq);
}

// Tensor map of an array of `rank` dimensions (type: 16-bit or e4m3 codes as
// bytes; strides in bytes from the second dimension on), the rows of its boxes 64 or
// 128 bytes, swizzled at that grain.
static bool encode_tiles_map(CUtensorMap *map, const void *base, CUtensorMapDataType type,
                            int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                            const cuuint32_t *box)
{
    EncodeTiledFn fn = get_encode_fn();
    if (!fn)
        return false;
    const cuuint32_t row_bytes = box[0] * (type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 1 : 2);
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, type, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

pa_status launch_window_tiles(const WindowMqParams &prm_in, pa_dtype dtype, bool fp8, int head_dim,
                             cudaStream_t stream)
{
    WindowMqParams prm = prm_in;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return record_cuda(e);
    DeviceInfo info;
    const pa_status st = device_info(dev, &info);
    if (st != PA_OK)
        return st;
    // boxes of 32 tokens where a block holds them (half the TMA instructions)
    const int box_tokens = prm.block_size >= 32 ? 32 : 16;
    prm.sink_tokens = (prm.num_sinks + box_tokens - 1) & ~(box_tokens - 1);
    const int tok_tile = kWtRows / prm.group;
    const long long units = ((long long)prm.num_tokens / tok_tile + prm.num_segments) *
                            prm.num_kv_heads;
    const int grid = (int)std::max(1ll, std::min((long long)info.sms, units));
    if (units > (1ll << 31) - 1 - info.sms)
        return PA_ERR_UNSUPPORTED;  // (unit numbers stay in 32 bits)
    prm.max_units = (int)(units / prm.num_kv_heads);
    // more than a round of units: longest first
    prm.ordered = units > info.sms && prm.num_segments <= kWtOrderSegs;

    CUtensorMap mk, mv, mq;
    // 16-bit pools: [8 tokens][d-halves of all heads][64], tokens in groups of 8
    // (a whole number of them in a block); codes: [tokens][heads][d] by blocks
    using U64 = cuuint64_t;
    using U32 = cuuint32_t;
    const U64 dim = head_dim, heads = prm.num_kv_heads, tokens = prm.block_size;
    const U64 row = heads * dim * (fp8 ? 1 : 2);  // bytes of a token
    const U32 halves = head_dim / 64;
    const U64 pool16[4] = {64, 8, halves * heads, prm.num_blocks * tokens / 8};
    const U64 pool16_strides[3] = {row, 128, 8 * row};
    const U32 pool16_box[4] = {64, 8, halves, (U32)box_tokens / 8};
    const U64 pool8[4] = {dim, heads, tokens, (U64)prm.num_blocks};
    const U64 pool8_strides[3] = {dim, row, tokens * row};
    const U32 pool8_box[4] = {(U32)dim, 1, (U32)box_tokens, 1};
    const U64 rows[3] = {dim, (U64)prm.num_heads, (U64)prm.num_tokens};
    const U64 rows_strides[2] = {dim * 2, prm.num_heads * dim * 2};
    const U32 rows_box[3] = {64, (U32)prm.group, (U32)tok_tile};
    const CUtensorMapDataType type = dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    auto pool_map = [&](CUtensorMap *m, const void *base) {
        return fp8 ? encode_tiles_map(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pool8,
                                      pool8_strides, pool8_box)
                   : encode_tiles_map(m, base, type, 4, pool16, pool16_strides, pool16_box);
    };
    if (!pool_map(&mk, prm.key_cache) || !pool_map(&mv, prm.value_cache) ||
        !encode_tiles_map(&mq, prm.query, type, 3, rows, rows_strides, rows_box))
        return PA_ERR_CUDA;
    auto run = [&](auto type_tag, auto dim, auto box, auto codes) {
        return launch_tiles_as<decltype(type_tag), decltype(dim)::value, decltype(box)::value,
                               decltype(codes)::value>(prm, mk, mv, mq, stream, grid,
                                                       info.optin);
    };
    auto by_pool = [&](auto type_tag, auto dim, auto box) {
        return fp8 ? run(type_tag, dim, box, std::true_type{})
                   : run(type_tag, dim, box, std::false_type{});
    };
    auto by_box = [&](auto type_tag, auto dim) {
        return box_tokens == 32 ? by_pool(type_tag, dim, std::integral_constant<int, 32>{})
                                : by_pool(type_tag, dim, std::integral_constant<int, 16>{});
    };
    auto by_dim = [&](auto type_tag) {
        return head_dim == 128 ? by_box(type_tag, std::integral_constant<int, 128>{})
                               : by_box(type_tag, std::integral_constant<int, 64>{});
    };
    return dtype == PA_BF16 ? by_dim(__nv_bfloat16{}) : by_dim(__half{});
}

}  // namespace pa
