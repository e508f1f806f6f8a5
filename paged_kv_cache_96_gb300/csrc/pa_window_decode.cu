// pa_window_decode.cu -- paged decode attention with a sliding window and a few
// first tokens that stay visible, for sm_103a.
//
// For the one query row of sequence s with c tokens in the pool (its own at
// position c - 1), a window of W tokens and N first tokens:
//     visible = { p < c : p >= c - W  or  p < N }
//     out = sum_{p visible} softmax_p(scale * q . k_p) v_p
// read through the block table as paged decode attention is ("PagedAttention &
// Continuous Batching" §1.6, §2.4; the pages attend the whole context, the
// window is an addition).  Blocks that hold no visible token are never read,
// so an engine may have given them to other sequences.
//
// What bounds it: HBM.  Each visible K and V row is read once for the G query
// heads of its KV head; nothing else is (V rows 2 G d flop / 2 d bytes, far
// below the tensor cores' balance).  So the design is a stream of 16-token
// tiles (a tile is inside one block: blocks are multiples of 16):
//  * The visible tokens' tiles are numbered without a gap ("compact
//    positions"): the first tokens' tiles, then the window's from the tile its
//    first token is in.  A sequence's compact length is at most N + W rounded
//    up to tiles, whatever its context, and every later step -- partitions,
//    the deal of units, the tile loop -- counts in it; only the table lookup
//    and the mask of the two border tiles go back to real positions.
//  * Work unit = (sequence, KV head, partition of compact tokens), dealt
//    round-robin over a persistent grid.  Each tile warp owns a ring of
//    shared-memory stages and runs its 4-D TMA loads ahead across unit borders;
//    scores and value products are mma.sync m16n8k16 tiles with the G heads as
//    the narrow side (tcgen05 wants 64 rows or more; 16-token tiles keep every
//    warp independent); softmax is online in fp32; a merge warp combines the
//    tile warps' records while they stream the next unit.
//  * Partitions of a sequence are merged by log-sum-exp weights, in the pass
//    for up to 3 of them, else by the reduce kernel behind it, which then
//    takes the compact lengths this pass leaves in the workspace.
//  * Hidden rows of a border tile get a score of -inf by selection and a zero
//    value row, so what they hold never reaches the output.
// Weights are rounded to the pools' type (fp16 for FP8 pools) as the operand of
// the value product, relative error 2^-8 (bf16) or 2^-11: about that of the
// rounded output; their sum keeps the unrounded fp32 weights.
#include <cuda.h>

#include <type_traits>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>

#include "pa_decode_common.cuh"

namespace pa {

struct WindowParams : DecodeParams {
    int window, num_sinks;
    int sink_tokens;   // num_sinks rounded up to tiles
    int32_t *len_out;  // compact lengths for the reduce kernel (null: it will not run)
    int merge_max;     // partials of a sequence that the pass merges itself, at most
};

// Batches whose sequences have at most this many partials are merged by the
// pass, others by the reduce kernel: a merge in the pass is a trip to L2 for
// every partial or two, at the end of the last CTA or in the way of its next
// unit; the reduce kernel is ~2 us behind the pass.  1 sequence, window 2,048, 8
// heads of 8, FP8: 8 partials 14.0 us by the pass, 9.8 by the kernel, 4 partials
// 13.6 and 12.6, 2 partials 18.2 and 18.1; 128 such sequences, window 1,024: 163 and
// 96, 78 and 76, 62.5 and 65.9 (16-bit pools 183 and 117, 110 and 103, 93 and 98).
// 3 partials: 128 sequences 67.7 and 70.0 (16-bit pools 98.3 and 99.6), 8 sequences,
// window 2,048, 18.5 and 20.6, 1 sequence 18.5 and 16.5.
constexpr int kWinMergeMax = 3;

// A sequence's compact length, and how far its window's tiles lie behind
// their compact positions (a multiple of 16 tokens; 0: no tile is left out).
struct WindowSpan {
    int len, skip;
};

__device__ __forceinline__ WindowSpan window_span(const WindowParams &p, int s, bool flag)
{
    const int ctx = clamp_context(p, s, flag);
    const int first_tile = max(0, ctx - p.window) & ~(kTileTokens - 1);
    const int skip = max(0, first_tile - p.sink_tokens);
    return {ctx - skip, skip};
}

// Partitions of a sequence of `len` compact tokens: every P of them, a
// remainder of less than half a partition joining the one before (a window
// of whole partitions with a few first tokens would otherwise leave a
// partition of one tile, with a partial and a merge of its own: 97 against 89
// us for 128 sequences, window and partition 1,024).
__host__ __device__ inline int window_parts(int len, int part_tokens)
{
    const int n = (int)(((long long)len + part_tokens / 2) / part_tokens);
    return len <= 0 ? 0 : n > 0 ? n : 1;
}

// Shared-memory layout (offsets from a 1024-byte aligned base): NW warps,
// each with a private ring of NST stages.  EB = bytes per cached element.
template <int D, int NT, int NW, int NST, int EB> struct WindowLayout {
    static constexpr int kHalfBytes = kTileTokens * 128;      // 16 rows x 64 elements (EB 2)
    static constexpr int kTileBytes = kTileTokens * D * EB;   // one K (or V) tile
    static constexpr int kStageBytes = 2 * kTileBytes;        // K tile + V tile
    static constexpr int kHeads = 8 * NT;
    static constexpr int kPitch = D + 4;  // floats per merge row (bank spread)
    static constexpr int kStages = 0;
    static constexpr int kMergeO = kStages + NW * NST * kStageBytes;
    static constexpr int kMergeM = kMergeO + NW * kHeads * kPitch * 4;
    static constexpr int kMergeL = kMergeM + NW * kHeads * 4;
    static constexpr int kBars = kMergeL + NW * kHeads * 4;  // NW * NST stage barriers
    static constexpr int kFlags = kBars + NW * NST * 8;
    static constexpr int kSeq = kFlags + NW * NST * 4;  // int len[S], prefix[S + 1], skip[S]
    static size_t bytes(int num_seqs) { return 1024 + kSeq + 4 * (3 * (size_t)num_seqs + 1); }
    static_assert(kBars % 8 == 0, "mbarriers need 8-byte alignment");
    static_assert(kStageBytes % 1024 == 0, "stages must keep 1024-byte alignment");
};

// Register budget for MINB resident CTAs of NW warps: the binding limit is
// the fullest of an SM's four register files (ceil(NW * MINB / 4) warps); the
// thread count given to __launch_bounds__ is the one whose even split over
// MINB CTAs yields that per-warp budget, in whole warps.
constexpr int window_bound_threads(int NW, int MINB)
{
    return 128 * ((NW * MINB + 3) / 4) / MINB / 32 * 32;
}

// T: query/output type.  KV: cached element type -- T itself, or uint8_t for
// FP8 (e4m3) pools, whose tiles are widened to fp16 in registers (the
// tensor-core products then run in fp16).
template <typename T, typename KV, int D, int NT, int NW, int NST, int MINB>
__global__ void __launch_bounds__(window_bound_threads(NW + 1, MINB), MINB)
    window_decode_kernel(const __grid_constant__ WindowParams p,
                        const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v)
{
    constexpr bool kFp8 = sizeof(KV) == 1;
    using L = WindowLayout<D, NT, NW, NST, sizeof(KV)>;
    using MT = typename std::conditional<kFp8, __half, T>::type;  // tensor-core input type
    using Op = MmaOp<MT>;
    constexpr int KT = D / 16;  // k-steps of the score product, m-tiles of the output
    constexpr int kHeads = L::kHeads;
    constexpr int kThreads = (NW + 1) * 32;  // NW tile warps, then the merge warp
    static_assert(window_bound_threads(NW + 1, MINB) >= kThreads, "launch bound below the block size");

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_addr(smem);

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int g = lane >> 2;  // mma group (row of the accumulator fragment)
    const int t4 = lane & 3;  // thread in group (column pair)

    const int S = p.num_seqs;
    const int Hkv = p.num_kv_heads;
    const int G = p.group;
    const int P = p.part_tokens;
    // compact positions of the first tokens' tiles (a sequence that skips none
    // of its tokens has the rest of its own in place of those it lacks)
    const int sink_tokens = p.sink_tokens;
    // A sequence's tiles are counted in compact positions: its first tokens'
    // tiles, then the window's, `skip` tokens further on in the sequence.
    int *len_s = reinterpret_cast<int *>(smem + L::kSeq);  // compact length
    int *pref = len_s + S;    // pref[s] = partitions of sequences [0 .. s)
    int *skip_s = pref + S + 1;
    volatile int *flags = reinterpret_cast<volatile int *>(smem + L::kFlags);
    float *merge_o = reinterpret_cast<float *>(smem + L::kMergeO);
    float *merge_m = reinterpret_cast<float *>(smem + L::kMergeM);
    float *merge_l = reinterpret_cast<float *>(smem + L::kMergeL);
    auto bar_of = [&](int stage) { return sbase + L::kBars + (warp * NST + stage) * 8; };
    auto stage_of = [&](int stage) {
        return sbase + L::kStages + (warp * NST + stage) * L::kStageBytes;
    };
    if (lane == 0 && warp < NW) {
        for (int k = 0; k < NST; ++k)
            mbar_init(bar_of(k), 1);
        fence_barrier_init();
    }
    if (tid == 0) {
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    pdl_wait_primary();

    // ---- compact lengths and partition prefix sums ------------------------
    for (int s = tid; s < S; s += kThreads) {
        const WindowSpan w = window_span(p, s, blockIdx.x == 0);
        len_s[s] = w.len;
        skip_s[s] = w.skip;
        if (p.len_out != nullptr && blockIdx.x == 0)
            // a length of as many whole partitions, for the reduce kernel
            p.len_out[s] = (int)min((long long)window_parts(w.len, P) * P, (long long)INT32_MAX);
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        for (int base = 0; base < S; base += 32) {
            const int k = base + lane;
            const int n = k < S ? window_parts(len_s[k], P) : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o)
                    x += y;
            }
            if (k < S)
                pref[k] = carry + x - n;
            carry += __shfl_sync(kFull, x, 31);
        }
        if (lane == 0)
            pref[S] = carry;
    }
    __syncthreads();
    const int total_units = pref[S] * Hkv;

    // ---- sequences with no context get zero rows ----------------------------
    for (int s = blockIdx.x; s < S; s += gridDim.x) {
        if (len_s[s] != 0)
            continue;
        uint4 *row = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) +
                                               (size_t)s * p.num_heads * D);
        for (int i = tid; i < p.num_heads * D / 8; i += kThreads)
            row[i] = make_uint4(0, 0, 0, 0);
    }

    // unit u -> partition q = u / Hkv, kv head u % Hkv; sequence s with
    // pref[s] <= q < pref[s + 1]; tok0 is compact.
    auto decode_unit = [&](int u, int &s, int &kh, int &j, int &tok0, int &ntiles) {
        const int q = u / Hkv;
        kh = u - q * Hkv;
        int lo = 0, hi = S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pref[mid] <= q)
                lo = mid;
            else
                hi = mid - 1;
        }
        j = q - pref[lo];
        s = lo;
        tok0 = j * P;
        // (the last partition ends with the sequence)
        const int tok_end = q + 1 == pref[lo + 1] ? len_s[s] : tok0 + P;
        ntiles = (tok_end - tok0 + kTileTokens - 1) / kTileTokens;
    };

    // this CTA's units: the first, and the one after unit u
    const int u_first = (int)blockIdx.x;
    auto next_u = [&](int u) -> int { return u + (int)gridDim.x; };
    // position in the sequence of a compact position (both of a tile's start)
    auto real_tok = [&](int s, int c) -> int { return c + (c >= sink_tokens ? skip_s[s] : 0); };
    // ---- this warp's fetch cursor: its next tile, possibly in a later unit ----
    int pu = u_first, ps = 0, pkh = 0, pj = 0, ptok0 = 0, pnt = 0, ptile = warp;
    bool pdone = pu >= total_units || warp >= NW;  // the merge warp fetches nothing
    if (!pdone)
        decode_unit(pu, ps, pkh, pj, ptok0, pnt);
    auto skip_empty = [&]() {
        while (!pdone && ptile >= pnt) {
            pu = next_u(pu);
            if (pu >= total_units) {
                pdone = true;
                break;
            }
            decode_unit(pu, ps, pkh, pj, ptok0, pnt);
            ptile = warp;
        }
    };
    skip_empty();
    // Lane 0 loads the table entry of the tile at the cursor one tile ahead
    // of issuing its fetch, so the load's latency overlaps a tile of compute.
    int pphys = 0, prow = 0;
    auto prefetch_entry = [&]() {
        if (!pdone && lane == 0) {
            const int tok = real_tok(ps, ptok0 + ptile * kTileTokens);
            prow = tok & (p.block_size - 1);
            pphys = __ldg(p.block_tables + (size_t)ps * p.max_blocks_per_seq +
                          (tok >> p.block_shift));
        }
    };
    prefetch_entry();

    uint32_t issued = 0, consumed = 0;
    uint32_t inflight = 0;  // stages with a fetch not yet waited for
    bool aborted = false;
    auto produce = [&]() {
        if (pdone || aborted)
            return;
        const int stage = issued % NST;
        // test hook of the time-out path: a fill that is never issued, so
        // nothing completes the stage's phase and its wait runs out
        const bool withheld = p.withhold_fill != 0 && warp == 0 && issued == 0;
        if (lane == 0 && !withheld) {
            const bool ok = pphys >= 0 && pphys < p.num_blocks;
            flags[warp * NST + stage] = ok;
            if (ok) {
                const uint32_t dst = stage_of(stage);
                mbar_arrive_expect_tx(bar_of(stage), L::kStageBytes);
                if constexpr (kFp8) {
                    // one 128-byte row per token: a 2 KB box per tile and tensor
                    tma_load_4d(dst, &tmap_k, bar_of(stage), 0, pkh, prow, pphys);
                    tma_load_4d(dst + L::kTileBytes, &tmap_v, bar_of(stage), 0, pkh, prow,
                                pphys);
                } else {
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf) {
                        tma_load_4d(dst + hf * L::kHalfBytes, &tmap_k, bar_of(stage), hf * 64,
                                    pkh, prow, pphys);
                        tma_load_4d(dst + L::kTileBytes + hf * L::kHalfBytes, &tmap_v,
                                    bar_of(stage), hf * 64, pkh, prow, pphys);
                    }
                }
            } else {
                flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                mbar_arrive(bar_of(stage));
            }
        }
        if (!withheld)
            inflight |= 1u << stage;
        ++issued;
        ptile += NW;
        skip_empty();
        prefetch_entry();
    };
    for (int k = 0; k < NST; ++k)
        produce();

    // Per-lane ldmatrix row/chunk selectors.
    const int li = lane & 7, lj = lane >> 3;
    const int k_row = li + ((lj & 1) << 3), k_cj = lj >> 1;  // K: A operand
    const int v_row = li + ((lj >> 1) << 3), v_cj = lj & 1;  // V^T: A operand (trans)
    // Shared-memory address of 16-byte chunk `chunk` of (token, d-half) in a
    // tile at `base`: rows of 128 bytes; chunk c of row r sits at chunk
    // c ^ (r & 7) (the TMA's 128-byte swizzle).
    auto tile_addr = [&](uint32_t base, int token, int half, int chunk) -> uint32_t {
        if constexpr (kFp8) {
            const int r = token;
            if constexpr (D == 64)  // one 64-byte row per token, chunk 0..3, 64-byte swizzle
                return base + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4);
            // one 128-byte row per token, chunk 0..7
            return base + r * 128 + (((chunk + 4 * half) ^ (r & 7)) << 4);
        }
        const int r = half * kTileTokens + token;
        return base + r * 128 + ((chunk ^ (r & 7)) << 4);
    };

    // Query fragments (B operand of the score product): head 8nt+g of the
    // group.  16-bit pools: elements d = 16kk + 2t4 (+1) and +8 (+9).  FP8
    // pools: the score's sum over d is taken in a permuted order matching the
    // FP8 tile fragments -- k-steps 2t4, 2t4+1 <- d = 16kk + 4t4 (+1) and
    // k-steps 2t4+8, 2t4+9 <- d = 16kk + 4t4 + 2 (+3) -- in fp16.
    uint32_t qf[NT][KT][2];
    bool q_over = false;  // FP8 pools: a bf16 query element past the fp16 range
    auto load_query = [&](int s, int kh) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hg = nt * 8 + g;
            const T *qrow = static_cast<const T *>(p.query) +
                            ((size_t)s * p.num_heads + (size_t)kh * G + (hg < G ? hg : 0)) * D;
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                if constexpr (kFp8) {
                    uint2 w = make_uint2(0u, 0u);
                    if (hg < G)
                        w = __ldg(reinterpret_cast<const uint2 *>(qrow + kk * 16 + 4 * t4));
                    if constexpr (std::is_same<T, __half>::value) {
                        qf[nt][kk][0] = w.x;
                        qf[nt][kk][1] = w.y;
                    } else {
                        const T *e = reinterpret_cast<const T *>(&w);
                        const float x0 = __bfloat162float(e[0]), x1 = __bfloat162float(e[1]);
                        const float x2 = __bfloat162float(e[2]), x3 = __bfloat162float(e[3]);
                        // the fp16 products need |q| within the fp16 range
                        q_over |= fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3))) >
                                  65504.f;
                        qf[nt][kk][0] = pack_f16x2(x0, x1);
                        qf[nt][kk][1] = pack_f16x2(x2, x3);
                    }
                } else {
                    const uint32_t *qw = reinterpret_cast<const uint32_t *>(qrow);
                    qf[nt][kk][0] = hg < G ? __ldg(qw + kk * 8 + t4) : 0u;
                    qf[nt][kk][1] = hg < G ? __ldg(qw + kk * 8 + 4 + t4) : 0u;
                }
            }
        }
    };
    if (u_first < total_units && warp < NW) {
        int s, kh, j, tok0, ntiles;
        decode_unit(u_first, s, kh, j, tok0, ntiles);
        load_query(s, kh);
    }

    // ---- units --------------------------------------------------------------------
    // The tile warps stream a unit's tiles and hand their (m, l, O) to the
    // merge warp through shared memory; the merge warp combines them, writes the output row or the partition's
    // partial, and -- for split sequences -- arrives on the sequence's counter
    // and merges the partials when its arrival completes them.  The two sides
    // meet only at two named barriers per unit ("records written": the tile
    // warps arrive, the merge warp waits; "records read": the other way
    // round, skipped after the CTA's last unit), so tile warps never wait for
    // each other at a unit's end and the merge warp sleeps in hardware.
    constexpr int kRecFull = 1, kRecFree = 2;  // named barrier ids (0 is __syncthreads)
    if (warp < NW) {
        int k_unit = 0;          // units of this CTA so far
        for (int u = u_first; u < total_units; u = next_u(u), ++k_unit) {
            int s, kh, j, tok0, ntiles;
            decode_unit(u, s, kh, j, tok0, ntiles);
            const int ctx = len_s[s] + skip_s[s];
            const int low = max(0, ctx - p.window);  // first position of the window

            float o[KT][NT][4];
            float mrun[NT][2], lrun[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mrun[nt][0] = mrun[nt][1] = -INFINITY;
                lrun[nt][0] = lrun[nt][1] = 0.f;
#pragma unroll
                for (int mt = 0; mt < KT; ++mt)
                    o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
            }
            for (int tile = warp; tile < ntiles; tile += NW) {
                const int stage = consumed % NST;
                const uint32_t parity = (consumed / NST) & 1u;
                bool ready = false;
                if (!aborted) {
                    ready = __all_sync(kFull, mbar_wait_bounded(bar_of(stage), parity, p.wait_ns));
                    if (ready) {
                        inflight &= ~(1u << stage);
                    } else {
                        aborted = true;
                        if (lane == 0)
                            flag_error(p.error_word, PA_DEVERR_TIMEOUT);
                    }
                }
                if (ready && flags[warp * NST + stage] != 0) {
                    const uint32_t kbase = stage_of(stage);
                    const uint32_t vbase = kbase + L::kTileBytes;
                    // hidden rows: past the context, or between the first
                    // tokens and the window
                    const int t0 = real_tok(s, tok0 + tile * kTileTokens);
                    const bool partial = t0 + kTileTokens > ctx ||
                                         (t0 < low && t0 + kTileTokens > p.num_sinks);
                    auto seen = [&](int r) {
                        const int t = t0 + r;
                        return t < ctx && (t < p.num_sinks || t >= low);
                    };

                    // scores S[token][head] = K . Q^T in independent accumulator
                    // chains (k-step kk feeds chain kk % kChains), summed at the end
                    constexpr int kChains = KT >= 4 ? 4 : KT;
                    float part[kChains][NT][4];
#pragma unroll
                    for (int c = 0; c < kChains; ++c)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            part[c][nt][0] = part[c][nt][1] = part[c][nt][2] = part[c][nt][3] = 0.f;
                    if constexpr (kFp8) {
                        // one ldmatrix brings two 16-d chunks of 16 tokens as byte
                        // pairs: thread (g, t4) gets d = 16c + 4t4 .. +3 of tokens g
                        // and g + 8; widening gives the (permuted-k) A fragment
#pragma unroll
                        for (int kp = 0; kp < KT / 2; ++kp) {
                            uint32_t r[4];
                            ldmatrix_x4(tile_addr(kbase, k_row, 0, 2 * kp + k_cj), r);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int kk = 2 * kp + h;
                                const uint32_t w0 = r[2 * h], w1 = r[2 * h + 1];
                                uint32_t a[4];
                                a[0] = e4m3x2_to_f16x2((uint16_t)(w0 & 0xffffu));
                                a[1] = e4m3x2_to_f16x2((uint16_t)(w1 & 0xffffu));
                                a[2] = e4m3x2_to_f16x2((uint16_t)(w0 >> 16));
                                a[3] = e4m3x2_to_f16x2((uint16_t)(w1 >> 16));
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    Op::run(part[kk % kChains][nt], a, qf[nt][kk][0], qf[nt][kk][1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < KT; ++kk) {
                            uint32_t a[4];
                            ldmatrix_x4(tile_addr(kbase, k_row, kk >> 2, (kk & 3) * 2 + k_cj), a);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                Op::run(part[kk % kChains][nt], a, qf[nt][kk][0], qf[nt][kk][1]);
                        }
                    }
                    float sc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = part[0][nt][e];
#pragma unroll
                            for (int c = 1; c < kChains; ++c)
                                x += part[c][nt][e];
                            sc[nt][e] = x;
                        }

                    // V^T fragments (their latency overlaps the softmax); hidden
                    // rows are zeroed, so that what they hold (NaN, another
                    // sequence's rows) never meets a zero weight
                    uint32_t va[KT][4];
                    if constexpr (kFp8) {
                        // transposed byte-pair loads: thread (g, t4) gets tokens 2t4,
                        // 2t4+1 (and +8, +9) at d = 16c + 2g, 2g+1; fragment row g is
                        // d = 16c + 2g and row g + 8 is d = 16c + 2g + 1
#pragma unroll
                        for (int mp = 0; mp < KT / 2; ++mp) {
                            uint32_t r[4];
                            ldmatrix_x4_trans(tile_addr(vbase, k_row, 0, 2 * mp + k_cj), r);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t p0 = byte_perm(r[2 * h], 0u, 0x3120u);
                                const uint32_t p1 = byte_perm(r[2 * h + 1], 0u, 0x3120u);
                                va[2 * mp + h][0] = e4m3x2_to_f16x2((uint16_t)(p0 & 0xffffu));
                                va[2 * mp + h][1] = e4m3x2_to_f16x2((uint16_t)(p0 >> 16));
                                va[2 * mp + h][2] = e4m3x2_to_f16x2((uint16_t)(p1 & 0xffffu));
                                va[2 * mp + h][3] = e4m3x2_to_f16x2((uint16_t)(p1 >> 16));
                            }
                        }
                    } else {
#pragma unroll
                        for (int mt = 0; mt < KT; ++mt)
                            ldmatrix_x4_trans(tile_addr(vbase, v_row, mt >> 2, (mt & 3) * 2 + v_cj),
                                              va[mt]);
                    }
                    if (partial) {
                        const uint32_t m01 = (seen(2 * t4) ? 0x0000ffffu : 0u) |
                                             (seen(2 * t4 + 1) ? 0xffff0000u : 0u);
                        const uint32_t m89 = (seen(2 * t4 + 8) ? 0x0000ffffu : 0u) |
                                             (seen(2 * t4 + 9) ? 0xffff0000u : 0u);
#pragma unroll
                        for (int mt = 0; mt < KT; ++mt) {
                            va[mt][0] &= m01;
                            va[mt][1] &= m01;
                            va[mt][2] &= m89;
                            va[mt][3] &= m89;
                        }
                    }

                    // online softmax; P^T fragments for the value product
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float s0 = sc[nt][0] * p.scale_log2, s1 = sc[nt][1] * p.scale_log2;
                        float s2 = sc[nt][2] * p.scale_log2, s3 = sc[nt][3] * p.scale_log2;
                        if (partial) {
                            if (!seen(g))
                                s0 = s1 = -INFINITY;
                            if (!seen(g + 8))
                                s2 = s3 = -INFINITY;
                        }
                        // mrun is a reference point, not necessarily the running max:
                        // while every score of the tile stays within kSlack of it
                        // (weights <= 2^kSlack) it is kept, which skips the
                        // cross-lane max and the rescale; otherwise it moves up to
                        // the running max and l and O are rescaled.
                        const bool fits = s0 <= mrun[nt][0] + kSlack && s2 <= mrun[nt][0] + kSlack &&
                                          s1 <= mrun[nt][1] + kSlack && s3 <= mrun[nt][1] + kSlack;
                        if (!__all_sync(kFull, fits)) {
                            float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) {
                                mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, off));
                                mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, off));
                            }
                            const float mn0 = fmaxf(mrun[nt][0], mx0);
                            const float mn1 = fmaxf(mrun[nt][1], mx1);
                            const float al0 = mn0 == -INFINITY ? 1.f : exp2f(mrun[nt][0] - mn0);
                            const float al1 = mn1 == -INFINITY ? 1.f : exp2f(mrun[nt][1] - mn1);
                            lrun[nt][0] *= al0;
                            lrun[nt][1] *= al1;
#pragma unroll
                            for (int mt = 0; mt < KT; ++mt) {
                                o[mt][nt][0] *= al0;
                                o[mt][nt][1] *= al1;
                                o[mt][nt][2] *= al0;
                                o[mt][nt][3] *= al1;
                            }
                            mrun[nt][0] = mn0;
                            mrun[nt][1] = mn1;
                        }
                        const float mu0 = mrun[nt][0] == -INFINITY ? 0.f : mrun[nt][0];
                        const float mu1 = mrun[nt][1] == -INFINITY ? 0.f : mrun[nt][1];
                        const float p0 = exp2f(s0 - mu0), p2 = exp2f(s2 - mu0);
                        const float p1 = exp2f(s1 - mu1), p3 = exp2f(s3 - mu1);
                        lrun[nt][0] += p0 + p2;
                        lrun[nt][1] += p1 + p3;
                        pb[nt][0] = movmatrix_trans(Op::pack(p0, p1));
                        pb[nt][1] = movmatrix_trans(Op::pack(p2, p3));
                    }

                    // O^T[d][head] += V^T . P^T
#pragma unroll
                    for (int mt = 0; mt < KT; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            Op::run(o[mt][nt], va[mt], pb[nt][0], pb[nt][1]);
                }
                __syncwarp();
                ++consumed;
                produce();  // refill the stage just consumed
            }

            // Next unit's query: its loads land while this unit's records go out.
            if (next_u(u) < total_units) {
                int sn, khn, jn, tn, ntn;
                decode_unit(next_u(u), sn, khn, jn, tn, ntn);
                load_query(sn, khn);
            }

            // ---- end of unit: this warp's (m, l, O) to the merge warp -------------------
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        lrun[nt][k] += __shfl_xor_sync(kFull, lrun[nt][k], off);
            // the merge warp has read the previous unit's records
            if (k_unit > 0)
                named_barrier_sync(kRecFree, kThreads);
            {
                float *mo = merge_o + warp * kHeads * L::kPitch;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int h0 = nt * 8 + 2 * t4;
#pragma unroll
                    for (int mt = 0; mt < KT; ++mt) {
                        // fragment rows g, g + 8 are d = 16mt + g, + 8 (16-bit pools)
                        // or d = 16mt + 2g, + 1 (FP8 pools)
                        const int d0 = kFp8 ? mt * 16 + 2 * g : mt * 16 + g;
                        const int d1 = kFp8 ? d0 + 1 : d0 + 8;
                        mo[h0 * L::kPitch + d0] = o[mt][nt][0];
                        mo[(h0 + 1) * L::kPitch + d0] = o[mt][nt][1];
                        mo[h0 * L::kPitch + d1] = o[mt][nt][2];
                        mo[(h0 + 1) * L::kPitch + d1] = o[mt][nt][3];
                    }
                    if (g == 0) {
                        merge_m[warp * kHeads + h0] = mrun[nt][0];
                        merge_m[warp * kHeads + h0 + 1] = mrun[nt][1];
                        merge_l[warp * kHeads + h0] = lrun[nt][0];
                        merge_l[warp * kHeads + h0 + 1] = lrun[nt][1];
                    }
                }
            }
            named_barrier_arrive(kRecFull, kThreads);  // this unit's records are written
        }
    } else {
        // ===== the merge warp ======================================================
        int k_unit = 0;
        for (int u = u_first; u < total_units; u = next_u(u), ++k_unit) {
            int s, kh, j, tok0, ntiles;
            decode_unit(u, s, kh, j, tok0, ntiles);
            const int nparts = pref[s + 1] - pref[s];
            const bool split = nparts > 1;
            named_barrier_sync(kRecFull, kThreads);  // every tile warp's records are in
            const int items = G * (D / 8);
            for (int it = lane; it < items; it += 32) {
                const int jh = it / (D / 8);
                const int d0 = (it - jh * (D / 8)) * 8;
                float mmax = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    mmax = fmaxf(mmax, merge_m[w * kHeads + jh]);
                const float mu = mmax == -INFINITY ? 0.f : mmax;
                float lsum = 0.f;
                float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float wgt = exp2f(merge_m[w * kHeads + jh] - mu);
                    lsum += wgt * merge_l[w * kHeads + jh];
                    const float4 *src = reinterpret_cast<const float4 *>(
                        merge_o + (w * kHeads + jh) * L::kPitch + d0);
                    const float4 x0 = src[0], x1 = src[1];
                    acc[0] += wgt * x0.x; acc[1] += wgt * x0.y; acc[2] += wgt * x0.z; acc[3] += wgt * x0.w;
                    acc[4] += wgt * x1.x; acc[5] += wgt * x1.y; acc[6] += wgt * x1.z; acc[7] += wgt * x1.w;
                }
                // a partial of no weight (scores of -inf alone) is 0 with l = 0; a whole
                // row of none is not a number, as its softmax
                const float inv = split && lsum == 0.f ? 0.f : p.out_scale / lsum;
                const size_t h = (size_t)kh * G + jh;
                if (!split) {
                    T vals[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        vals[e] = MmaOp<T>::from_float(acc[e] * inv);
                    *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) +
                                               ((size_t)s * p.num_heads + h) * D + d0) =
                        *reinterpret_cast<const uint4 *>(vals);
                } else {
                    // partial of partition j, merged below (or by the reduce kernel)
                    const size_t idx = ((size_t)s * p.num_heads + h) * p.max_parts + j;
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + idx * D + d0);
                    dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
                    dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
                    if (d0 == 0) {
                        // (never -inf: the reduce kernel takes a finite maximum, and the
                        // merge in the pass would leave out what is not a number in a
                        // partition without one)
                        p.part_m[idx] = fmaxf(mmax * kLn2, -FLT_MAX);
                        p.part_l[idx] = lsum;
                    }
                }
            }
            // the records may be rewritten; the tile warps wait for this only
            // from their next unit on
            if (next_u(u) < total_units)
                named_barrier_arrive(kRecFree, kThreads);
            if (split && nparts <= p.merge_max)
                // records loaded per lane at once: fewer under the FP8 register cap
                arrive_and_merge<T, D, kHeads, kFp8 ? 2 : 8>(p, s, kh, nparts, lane);
        }
    }
    if (kFp8 && __any_sync(kFull, q_over) && lane == 0)
        flag_error(p.error_word, PA_DEVERR_QUERY_RANGE);
    pdl_launch_dependents();

    // ---- drain: wait (bounded) for any fetch still landing in this warp's ring ----
    if (inflight != 0) {
        for (int k = 0; k < NST; ++k) {
            if (!(inflight & (1u << k)))
                continue;
            // the most recent fetch into stage k was issue number
            // issued - 1 - ((issued - 1 - k) % NST)
            const uint32_t last = issued - 1 - ((issued - 1 - k) % NST);
            mbar_wait_bounded(bar_of(k), (last / NST) & 1u, kDrainWaitNs);
        }
    }
}


// ---- host side -------------------------------------------------------------------

// Tile warps per CTA (the merge warp comes on top), ring stages per warp and
// CTAs per SM the register budget is sized for: 16-bit pools, FP8 pools (whose
// stages are half the size and whose widening adds arithmetic per byte).
constexpr int kWinWarps = 5, kWinStages = 2, kWinMinBlocks = 2;
constexpr int kWinWarpsFp8 = 4, kWinStagesFp8 = 3, kWinMinBlocksFp8 = 3;

template <typename T, typename KV, int D, int NT, int NST>
static pa_status launch_window_pass(const WindowParams &prm, const CUtensorMap &mk,
                                    const CUtensorMap &mv, cudaStream_t stream,
                                    long long max_units)
{
    constexpr bool kFp8 = sizeof(KV) == 1;
    constexpr int NW = kFp8 ? kWinWarpsFp8 : kWinWarps;
    // the 16-head variant keeps twice the accumulators: no register cap
    constexpr int MINB = NT > 1 ? 1 : kFp8 ? kWinMinBlocksFp8 : kWinMinBlocks;
    using L = WindowLayout<D, NT, NW, NST, sizeof(KV)>;
    auto kernel = window_decode_kernel<T, KV, D, NT, NW, NST, MINB>;
    constexpr int kThreads = (NW + 1) * 32;
    static KernelSetting setting[kMaxDevices];
    static std::mutex mu;
    const size_t smem = L::bytes(prm.num_seqs);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return record_cuda(e);
    DeviceInfo info;
    const pa_status st = device_info(dev, &info);
    if (st != PA_OK)
        return st;
    if (smem > (size_t)info.optin)
        return PA_ERR_UNSUPPORTED;
    int per_sm = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        KernelSetting &ks = setting[dev];
        if (smem > ks.smem_enabled) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)smem);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         (int)cudaSharedmemCarveoutMaxShared);
            if (e != cudaSuccess)
                return record_cuda(e);
            ks.smem_enabled = smem;
        }
        if (smem != ks.smem_queried) {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ks.per_sm, kernel, kThreads, smem);
            if (e != cudaSuccess)
                return record_cuda(e);
            ks.smem_queried = smem;
        }
        per_sm = ks.per_sm;
    }
    if (per_sm < 1)
        return PA_ERR_UNSUPPORTED;
    const long long grid =
        std::max(1ll, std::min((long long)info.sms * per_sm, max_units));
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), smem, stream, prm, mk, mv);
}

template <typename T, typename KV, int D, int NT>
static pa_status launch_window(const WindowParams &prm, const CUtensorMap &mk,
                               const CUtensorMap &mv, cudaStream_t stream, int max_parts)
{
    const long long max_units = (long long)prm.num_seqs * prm.num_kv_heads * max_parts;
    constexpr int kStages = sizeof(KV) == 1 ? kWinStagesFp8 : kWinStages;
    pa_status st = launch_window_pass<T, KV, D, NT, kStages>(prm, mk, mv, stream, max_units);
    // batches whose per-sequence arrays do not fit next to the default rings
    if (st == PA_ERR_UNSUPPORTED)
        st = launch_window_pass<T, KV, D, NT, 1>(prm, mk, mv, stream, max_units);
    if (st != PA_OK || max_parts <= prm.merge_max)
        return st;
    DecodeParams reduce = prm;
    reduce.counters = nullptr;  // (nothing was merged by the pass)
    reduce.context_lens = prm.len_out;
    return launch_reduce<T, D>(reduce, stream);
}

template <typename T, typename KV>
static pa_status launch_window_as(const WindowParams &prm, const CUtensorMap &mk,
                                  const CUtensorMap &mv, cudaStream_t stream,
                                  int max_parts, int head_dim)
{
    const bool wide = prm.group > 8;
    if (head_dim == 128)
        return wide ? launch_window<T, KV, 128, 2>(prm, mk, mv, stream, max_parts)
                    : launch_window<T, KV, 128, 1>(prm, mk, mv, stream, max_parts);
    return wide ? launch_window<T, KV, 64, 2>(prm, mk, mv, stream, max_parts)
                : launch_window<T, KV, 64, 1>(prm, mk, mv, stream, max_parts);
}

// Longest compact length of any sequence: the first tokens' tiles, and the
// window's with the tile it starts inside of.
static int window_compact_max(int max_context_len, int window, int num_sinks)
{
    const long long t = kTileTokens;
    const long long n = ((long long)num_sinks + t - 1) / t * t +
                        ((long long)window + t - 1) / t * t + t;
    return (int)std::min<long long>(max_context_len, n);
}

// A length whose partitions, counted as the decode pass without a window counts
// them, are as many as this one's.
static int window_counted(int compact, int partition_size)
{
    if (partition_size <= 0)
        return compact;
    return (int)std::min<long long>(compact, (long long)window_parts(compact, partition_size) *
                                                 partition_size);
}

static WorkspaceLayout window_workspace(int S, int H, int Hkv, int D, int parts, size_t *len_off)
{
    WorkspaceLayout w = workspace_layout(S, H, Hkv, D, parts);
    *len_off = w.total;
    if (parts > kWinMergeMax)
        w.total += align256((size_t)S * 4);
    return w;
}

static pa_status run_window(void *out, const void *query, const void *key_cache,
                            const void *value_cache, const int32_t *block_tables,
                            int max_blocks_per_seq, const int32_t *context_lens,
                            int max_context_len, int window, int num_sinks, int num_seqs,
                            int num_heads, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, float scale, bool fp8, float k_scale, float v_scale,
                            int partition_size, void *workspace, size_t workspace_bytes,
                            pa_dtype dtype, int32_t *error_word, void *stream)
{
    if ((dtype != PA_F16 && dtype != PA_BF16) || window <= 0 || num_sinks < 0 ||
        max_context_len < 0)
        return PA_ERR_INVALID_ARG;
    if (fp8 && !(std::isfinite(k_scale) && std::isfinite(v_scale) && k_scale > 0.f &&
                 v_scale > 0.f))
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale * (fp8 ? k_scale : 1.f) * kLog2e))
        return PA_ERR_INVALID_ARG;
    // lengths in compact tokens here (partitions, workspace)
    const int compact = window_compact_max(max_context_len, window, num_sinks);
    WindowParams prm{};
    const pa_status ok = prepare_decode(
        &prm, out, query, key_cache, value_cache, block_tables, max_blocks_per_seq,
        context_lens, window_counted(compact, partition_size), num_seqs, num_heads, num_kv_heads, head_dim, block_size,
        num_blocks, scale, partition_size, workspace, workspace_bytes, error_word);
    if (ok != PA_OK || num_seqs == 0)
        return ok;
    // (positions of a whole tile past the last one stay in 32 bits)
    if ((long long)max_blocks_per_seq * block_size > (1ll << 31) - 256)
        return PA_ERR_UNSUPPORTED;
    size_t len_off = 0;
    if (prm.max_parts > 1 &&
        workspace_bytes < window_workspace(num_seqs, num_heads, num_kv_heads, head_dim,
                                           prm.max_parts, &len_off)
                              .total)
        return PA_ERR_WORKSPACE;
    // Partitions are there to give every CTA work.  Where the sequences and KV
    // heads by themselves give less than one unit a CTA, more partitions than
    // fill one round of CTAs only add partials and a second, nearly empty round
    // (16 sequences, 8 KV heads, window 4,096, FP8 pools: partitions of 512
    // 39.8 us, of 1,376, one round, 29.9; 16-bit pools 50.4 and 43.9).
    if (prm.max_parts > 1) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess)
            return record_cuda(e);
        DeviceInfo info;
        const pa_status di = device_info(dev, &info);
        if (di != PA_OK)
            return di;
        const long long ctas =
            (long long)info.sms * (prm.group > 8 ? 1 : fp8 ? kWinMinBlocksFp8 : kWinMinBlocks);
        const long long per = ctas / ((long long)num_seqs * num_kv_heads);
        if (per >= 1) {
            const long long t = kTileTokens;
            const long long fill = (compact + per * t - 1) / (per * t) * t;
            prm.part_tokens = (int)std::max<long long>(prm.part_tokens, fill);
        }
    }
    const int parts = window_parts(compact, prm.part_tokens) > 1
                          ? window_parts(compact, prm.part_tokens)
                          : 1;
    prm.merge_max = parts > kWinMergeMax ? 1 : kWinMergeMax;
    if (parts > prm.merge_max)
        prm.len_out = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + len_off);
    prm.max_context_len = max_context_len;
    prm.window = window;
    // (first tokens past the tables' reach hide nothing)
    prm.num_sinks = std::min(num_sinks, max_blocks_per_seq * block_size);
    prm.sink_tokens = (prm.num_sinks + kTileTokens - 1) & ~(kTileTokens - 1);
    if (fp8) {
        // scores of the K codes: the K scale in the exponent's, the V scale on
        // the outputs and partials
        prm.scale_log2 = scale * k_scale * kLog2e;
        prm.out_scale = v_scale;
    }
    CUtensorMap mk, mv;
    const pa_dtype pool = fp8 ? PA_FP8_E4M3 : dtype;
    if (!encode_pool_map(&mk, key_cache, pool, num_blocks, block_size, num_kv_heads, head_dim) ||
        !encode_pool_map(&mv, value_cache, pool, num_blocks, block_size, num_kv_heads, head_dim))
        return PA_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    using B16 = __nv_bfloat16;
    if (fp8)
        return dtype == PA_BF16
                   ? launch_window_as<B16, uint8_t>(prm, mk, mv, st, parts, head_dim)
                   : launch_window_as<__half, uint8_t>(prm, mk, mv, st, parts, head_dim);
    return dtype == PA_BF16 ? launch_window_as<B16, B16>(prm, mk, mv, st, parts, head_dim)
                            : launch_window_as<__half, __half>(prm, mk, mv, st, parts, head_dim);
}

} // namespace pa

using namespace pa;

extern "C" size_t pa_window_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                            int head_dim, int max_context_len, int window,
                                            int num_sinks, int partition_size)
{
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || partition_size < 0 || window <= 0 || num_sinks < 0)
        return 0;
    const int parts = num_parts(
        window_counted(window_compact_max(max_context_len, window, num_sinks), partition_size),
        partition_size);
    size_t len_off = 0;
    return window_workspace(num_seqs, num_heads, num_kv_heads, head_dim, parts, &len_off).total;
}

extern "C" pa_status pa_decode_attention_window(
    void *out, const void *query, const void *key_cache, const void *value_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int window, int num_sinks, int num_seqs, int num_heads,
    int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    int partition_size, void *workspace, size_t workspace_bytes, pa_dtype dtype,
    int32_t *error_word, void *stream)
{
    return run_window(out, query, key_cache, value_cache, block_tables, max_blocks_per_seq,
                      context_lens, max_context_len, window, num_sinks, num_seqs, num_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, scale, false, 1.f, 1.f,
                      partition_size, workspace, workspace_bytes, dtype, error_word, stream);
}

extern "C" pa_status pa_decode_attention_window_fp8(
    void *out, const void *query, const void *key_cache, const void *value_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int window, int num_sinks, int num_seqs, int num_heads,
    int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale, float k_scale,
    float v_scale, int partition_size, void *workspace, size_t workspace_bytes, pa_dtype dtype,
    int32_t *error_word, void *stream)
{
    return run_window(out, query, key_cache, value_cache, block_tables, max_blocks_per_seq,
                      context_lens, max_context_len, window, num_sinks, num_seqs, num_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, scale, true, k_scale,
                      v_scale, partition_size, workspace, workspace_bytes, dtype, error_word,
                      stream);
}
