// pa_list_decode.cu -- two forms of paged decode attention for long contexts, for
// sm_103a: over a list of blocks for each query row and KV head (sparse), and over the
// whole context with what each token was attended with added up (weights).  Additions
// to "PagedAttention & Continuous Batching" §1.6 and §2.4, which attend the whole
// context and keep nothing of the weights.
//
// sparse, row t at position c - 1 of its sequence, blocks L of its list:
//     out = sum_p softmax_p(scale * q . k_p) v_p over the p < c of blocks in L
// weights, the one row of a sequence with c tokens:
//     out as pa_decode_attention, and for every p < c
//     weights_out[p] = (p < weighted ? weights[p] : 0) + sum_h softmax_{h,p}
//
// What bounds both: HBM, each K and V row of a list or a context read once for the G
// query heads of its KV head.  So both are one pass over 16-token tiles, built as
// windowed decode is (pa_window_decode.cu): a persistent grid takes rows and KV heads
// or equal shares of all their tiles; every tile warp runs its own ring of
// shared-memory stages ahead by TMA, across unit borders; scores and value products are
// mma.sync m16n8k16 tiles with the G heads as the narrow side (tcgen05 wants 64 rows or
// more); softmax is online in fp32; a merge warp combines the tile warps' records while
// they stream the next unit; a row's partials are merged by log-sum-exp weights, in the
// pass for a few of them, else by the reduce kernel.
// What is different:
//  * Pool blocks of 32 of a warp's tiles are looked up at once, one a lane, and the
//    next 32 (of the same unit or the next one) before they are needed: a list's entry
//    and then its table entry are two dependent trips to memory.
//  * weights: every score goes to the workspace as it is computed (fp32, 4 bytes a
//    query head and token beside 4 d bytes of K and V a KV head), and a second kernel,
//    when the sums over the context are known, turns them into weights and adds those
//    of all heads, in one order: the same call again gives the same bits, which
//    atomics on the tokens' sums would not.  The scores are not computed anew from K,
//    which would read d times as much.
// Weights are rounded to the pools' type (fp16 for FP8 pools) as the operand of the
// value product, relative error 2^-8 (bf16) or 2^-11: about that of the rounded
// output.  Their sum, and the weights that are added up, keep fp32.
#include <cuda.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "pa_decode_common.cuh"

namespace pa {

struct ListParams : DecodeParams {
    // sparse: rows in place of sequences (num_seqs of them)
    const int32_t *selected;  // [rows][num_kv_heads][top_k]
    const int32_t *token_seq, *token_pos;
    int32_t *len_out;         // partials for the reduce kernel (null: it will not run)
    int top_k, table_rows;    // entries of a list; sequences in block_tables
    int share_min;            // split rows: least tiles of a CTA's share (0: whole rows)
    int aligned;              // shares do not go past a row's end
    int32_t *part_count;      // weights: partials of each row
    // weights
    const float *weights;     // [num_blocks][block_size]
    float *weights_out;
    const int32_t *weighted_lens;
    float *scores;            // [num_seqs][num_kv_heads][pitch][group], log2 units
    int pitch;                // positions of a sequence in scores
    int merge_max;            // partials of a row that the pass merges itself, at most
};

// Rows of at most this many partials are merged by the pass, others by the reduce
// kernel behind it (long contexts with weights, FP8: 130.5 us, up to 8 in the pass 132.5).
constexpr int kListMergeMax = 4;

// Rows whose tiles are numbered for shares, at most: 4 bytes each in every CTA's shared
// memory (as many CTAs fit an SM as without them up to about 1,600, which FP8 pools with a
// head_dim of 128 set: 4 CTAs of 51 KB in 228, less 1 KB each).
constexpr int kListShareRows = 8192;

// m of a partial without a visible token, and of one whose scores are all -inf: the
// first has no say (weight 0 beside any other partial, and an output of 0 by itself),
// the second makes a row of nothing else NaN, as its softmax.
constexpr float kNoToken = -FLT_MAX, kNoWeight = -1e38f;

// Partitions that the workspace has room for: every P tokens, a remainder of less than
// half a partition joining the one before.
static int list_partitions(int len, int part_tokens)
{
    const int n = (int)(((long long)len + part_tokens / 2) / part_tokens);
    return len <= 0 ? 0 : n > 0 ? n : 1;
}

// Shared-memory layout (offsets from a 1024-byte aligned base): NW warps, each with a
// private ring of NST stages.  EB = bytes per cached element.
template <int D, int NT, int NW, int NST, int EB> struct ListLayout {
    static constexpr int kHalfBytes = kTileTokens * 128;      // 16 rows x 64 elements (EB 2)
    static constexpr int kTileBytes = kTileTokens * D * EB;   // one K (or V) tile
    static constexpr int kStageBytes = 2 * kTileBytes;        // K tile + V tile
    static constexpr int kHeads = 8 * NT;
    static constexpr int kPitch = D + 4;  // floats per merge row (bank spread)
    static constexpr int kStages = 0;
    static constexpr int kMergeO = kStages + NW * NST * kStageBytes;
    static constexpr int kMergeM = kMergeO + NW * kHeads * kPitch * 4;
    static constexpr int kMergeL = kMergeM + NW * kHeads * 4;
    static constexpr int kMergeAny = kMergeL + NW * kHeads * 4;  // a warp saw a token
    static constexpr int kBars = (kMergeAny + NW * 4 + 7) / 8 * 8;  // NW * NST stage barriers
    static constexpr int kFirst = kBars + NW * NST * 8;  // a stage's first position, -1: none
    static constexpr int kSeq = kFirst + NW * NST * 4;   // shares: int prefix[S + 1]
    static size_t bytes(int num_seqs) { return 1024 + kSeq + 4 * ((size_t)num_seqs + 1); }
    static_assert(kStageBytes % 1024 == 0, "stages must keep 1024-byte alignment");
};

// Register budget for MINB resident CTAs of NW warps: the binding limit is the fullest
// of an SM's four register files (ceil(NW * MINB / 4) warps).
constexpr int list_bound_threads(int NW, int MINB)
{
    return 128 * ((NW * MINB + 3) / 4) / MINB / 32 * 32;
}

// T: query/output type.  KV: cached element type -- T itself, or uint8_t for FP8 (e4m3)
// pools, whose tiles are widened to fp16 in registers.  kSparse: lists, else weights.
template <typename T, typename KV, int D, int NT, int NW, int NST, int MINB, bool kSparse>
__global__ void __launch_bounds__(list_bound_threads(NW + 1, MINB), MINB)
    list_decode_kernel(const __grid_constant__ ListParams p,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v)
{
    constexpr bool kFp8 = sizeof(KV) == 1;
    using L = ListLayout<D, NT, NW, NST, sizeof(KV)>;
    using MT = typename std::conditional<kFp8, __half, T>::type;  // tensor-core input type
    using Op = MmaOp<MT>;
    constexpr int KT = D / 16;  // k-steps of the score product, m-tiles of the output
    constexpr int kHeads = L::kHeads;
    constexpr int kThreads = (NW + 1) * 32;  // NW tile warps, then the merge warp
    static_assert(list_bound_threads(NW + 1, MINB) >= kThreads, "launch bound below the block size");

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
    int *pref = reinterpret_cast<int *>(smem + L::kSeq);  // tiles of rows [0 .. r)
    volatile int *stage_pos = reinterpret_cast<volatile int *>(smem + L::kFirst);
    float *merge_o = reinterpret_cast<float *>(smem + L::kMergeO);
    float *merge_m = reinterpret_cast<float *>(smem + L::kMergeM);
    float *merge_l = reinterpret_cast<float *>(smem + L::kMergeL);
    int *merge_any = reinterpret_cast<int *>(smem + L::kMergeAny);
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
    // A row's listed blocks are read once, and need not stay in L2 (128 rows of 64 blocks 88.2
    // -> 85.3 us, 16 FP8 lists 35.3 -> 32.9).  Where rows of a sequence list the same blocks
    // they read them at about the same time, and the hint still pays (3 rows of 128 sequences
    // with a list each sequence 153.1 -> 150.8, of 16 over FP8 pools 89.1 -> 87.6).  With
    // weights it costs more than the scores that stay there bring (305 -> 324 us).
    const uint64_t once = kSparse ? policy_evict_first() : 0;
    auto load = [&](uint32_t dst, const void *map, uint32_t bar, int d, int kh, int row, int phys) {
        if constexpr (kSparse)
            tma_load_4d_hint(dst, map, bar, d, kh, row, phys, once);
        else
            tma_load_4d(dst, map, bar, d, kh, row, phys);
    };
    pdl_wait_primary();

    // A row's sequence, context and list length in tokens (sparse; a padding or bad
    // row has a context of 0).
    auto row_of = [&](int t, int &s, int &ctx, int &len, bool flag) {
        s = __ldg(p.token_seq + t);
        const int pos = __ldg(p.token_pos + t);
        ctx = 0;
        if (s < 0) {
            s = 0;
        } else if (s >= p.table_rows || pos < 0 ||
                   pos >= (long long)p.max_blocks_per_seq * p.block_size) {
            if (flag)
                flag_error(p.error_word, PA_DEVERR_TOKEN_RANGE);
            s = 0;
        } else {
            ctx = pos + 1;
        }
        const int nb = (int)(((long long)ctx + p.block_size - 1) >> p.block_shift);
        len = min(nb, p.top_k) << p.block_shift;
    };

    // tokens of a row's list or context
    auto len_of = [&](int r, bool flag) {
        int s, ctx, len;
        if constexpr (kSparse)
            row_of(r, s, ctx, len, flag);
        else
            len = clamp_context(p, r, flag);
        return len;
    };

    // ---- the CTA's work -------------------------------------------------------------
    // Whole rows in turn (a unit: a row and KV head), or, where rows are split, equal
    // shares of all tiles, numbered through the rows: as many CTAs as there are KV heads
    // take one share, a head each, so that a token's heads, which lie side by side, are
    // read at about the same time (when this came, long contexts with weights over FP8
    // pools took 138 us, now 130.5; shares numbered through the heads as well took 191).  A
    // unit is what one row has in the share.
    const bool share = p.share_min > 0;
    int W = 0;                          // tiles of a share
    int u_first = blockIdx.x, u_end = S * Hkv;
    // whether the reduce kernel merges a row of that many partials
    auto by_kernel = [&](int parts) { return p.len_out != nullptr && parts > p.merge_max; };
    auto tiles_in = [&](int len) { return (len + kTileTokens - 1) / kTileTokens; };
    // aligned: rows begin with a share of their own (share_min tiles)
    auto whole_shares = [&](int n) {
        return p.aligned ? (n + p.share_min - 1) / p.share_min * p.share_min : n;
    };
    // shares that the n tiles from tile t on are in
    auto parts_of = [&](int t, int n) { return n > 0 ? (t + n - 1) / W - t / W + 1 : 0; };
    if (share) {
        for (int r = tid; r < S; r += kThreads)
            pref[r] = whole_shares(tiles_in(len_of(r, blockIdx.x == 0)));
        __syncthreads();
        if (warp == 0) {
            int carry = 0;
            for (int base = 0; base < S; base += 32) {
                const int k = base + lane;
                const int n = k < S ? pref[k] : 0;
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
    }
    __syncthreads();
    if (share) {
        const int groups = (int)gridDim.x / Hkv, group = (int)blockIdx.x / Hkv;
        const int total = pref[S];
        // (aligned shares are taken in turn, if there are more of them than groups)
        W = p.aligned ? p.share_min : max(p.share_min, (total + groups - 1) / groups);
        u_first = group < groups ? (int)min((long long)total, (long long)group * W) : total;
        u_end = p.aligned ? total : (int)min((long long)total, (long long)u_first + W);
    }
    // rows with nothing to attend, lengths for the reduce kernel (in partials)
    for (int r = blockIdx.x; r < S; r += gridDim.x) {
        const int len = len_of(r, !share && tid == 0);
        if (tid == 0) {
            const int n = share ? parts_of(pref[r], tiles_in(len)) : len > 0;
            if (p.part_count != nullptr)
                p.part_count[r] = n;
            if (p.len_out != nullptr)
                p.len_out[r] = by_kernel(n) ? n : 0;
        }
        if (len != 0)
            continue;
        uint4 *row = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) +
                                               (size_t)r * p.num_heads * D);
        for (int i = tid; i < p.num_heads * D / 8; i += kThreads)
            row[i] = make_uint4(0, 0, 0, 0);
    }

    // A unit: partial j of nparts of row r and KV head kh, sequence s, ntiles tiles from
    // token tok0 of the list or context on; the row's context is ctx.
    struct Unit {
        int r, s, kh, j, nparts, tok0, ntiles, ctx;
    };
    auto unit_of = [&](int u) {
        Unit x;
        x.j = x.tok0 = 0;
        x.nparts = 1;
        int len = 0;
        if (share) {
            int lo = 0, hi = S - 1;  // the last row that starts at or before u
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pref[mid] <= u)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            x.r = lo;
            x.kh = (int)blockIdx.x % Hkv;
        } else {
            x.r = u / Hkv;
            x.kh = u - x.r * Hkv;
        }
        if constexpr (kSparse) {
            row_of(x.r, x.s, x.ctx, len, false);
        } else {
            x.s = x.r;
            x.ctx = len = clamp_context(p, x.r, false);
        }
        x.ntiles = tiles_in(len);
        if (share) {
            const int from = pref[x.r];
            x.j = u / W - from / W;
            x.nparts = parts_of(from, x.ntiles);
            x.tok0 = (u - from) * kTileTokens;
            x.ntiles = min(x.ntiles - (u - from), (u / W + 1) * W - u);
        }
        return x;
    };
    // this CTA's units with tiles, in turn: the one after u, which is x
    auto next_unit = [&](int u, const Unit &x) {
        if (share)
            return p.aligned ? (u / W + (int)gridDim.x / Hkv) * W : u + x.ntiles;
        for (u += (int)gridDim.x; u < u_end; u += (int)gridDim.x)
            if (unit_of(u).ntiles > 0)
                break;
        return u;
    };
    if (!share)
        u_first = next_unit(u_first - (int)gridDim.x, Unit{});

    // ---- this warp's fetch cursor -----------------------------------------------------
    // Tiles of a unit are taken in chunks of 32 a warp: lane l looks up tile
    // (32 k + l) NW + warp of chunk k.  The next chunk's list entries are loaded as a
    // chunk is entered and its table entries at the fetch after that.
    struct Chunk {
        int u, k, left;     // unit (>= u_end: none), chunk, this warp's tiles in it
        int pos, phys;      // this lane's tile: first position, pool block (-1: no fetch)
        int row, kh;        // this lane's row in the block; the unit's KV head
        const int32_t *at;  // its table entry, or null
    };
    auto tiles_of = [&](const Unit &x) {
        return x.ntiles > warp ? (x.ntiles - warp + NW - 1) / NW : 0;
    };
    // the chunk after (u, k), its positions and where its table entries are
    auto enter = [&](int u, int k) {
        Chunk c;
        c.at = nullptr;
        c.pos = c.phys = -1;
        c.row = 0;
        c.left = 0;
        c.kh = 0;
        c.k = k;
        for (; u < u_end; c.k = 0) {
            const Unit x = unit_of(u);
            const int mine = tiles_of(x) - c.k * 32;
            if (mine <= 0) {
                u = next_unit(u, x);
                continue;
            }
            c.left = min(mine, 32);
            c.kh = x.kh;
            if (lane < c.left) {
                const int tok = x.tok0 + ((c.k * 32 + lane) * NW + warp) * kTileTokens;
                c.row = tok & (p.block_size - 1);
                int blk = tok >> p.block_shift;
                if constexpr (kSparse)
                    blk = __ldg(p.selected + ((size_t)x.r * Hkv + x.kh) * p.top_k + blk);
                if (kSparse && blk >= 0 &&
                    blk >= (int)(((long long)x.ctx + p.block_size - 1) >> p.block_shift)) {
                    flag_error(p.error_word, PA_DEVERR_CONTEXT_RANGE);
                    blk = -1;
                }
                if (blk >= 0) {
                    c.pos = (blk << p.block_shift) + c.row;
                    c.at = p.block_tables + (size_t)x.s * p.max_blocks_per_seq + blk;
                }
            }
            break;
        }
        c.u = u;
        return c;
    };
    auto look_up = [&](Chunk &c) {
        if (c.at != nullptr) {
            c.phys = __ldg(c.at);
            if (c.phys < 0 || c.phys >= p.num_blocks) {
                flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                c.phys = -1;
            }
            c.at = nullptr;
        }
    };
    Chunk cur, nxt;
    int at_lane = 0;  // the chunk's tile that is fetched next
    bool pdone = warp >= NW;  // the merge warp fetches nothing
    if (!pdone) {
        cur = enter(u_first, 0);
        look_up(cur);
        pdone = cur.u >= u_end;
        if (!pdone)
            nxt = enter(cur.u, cur.k + 1);
    }

    uint32_t issued = 0, consumed = 0;
    uint32_t inflight = 0;  // stages with a fetch not yet waited for
    bool aborted = false;
    auto produce = [&]() {
        if (pdone || aborted)
            return;
        const int stage = issued % NST;
        const int phys = __shfl_sync(kFull, cur.phys, at_lane);
        const int pos = __shfl_sync(kFull, cur.pos, at_lane);
        const int row = __shfl_sync(kFull, cur.row, at_lane);
        // test hook of the time-out path: a fill that is never issued, so
        // nothing completes the stage's phase and its wait runs out
        const bool withheld = p.withhold_fill != 0 && warp == 0 && issued == 0;
        if (lane == 0 && !withheld) {
            stage_pos[warp * NST + stage] = phys >= 0 ? pos : -1;
            if (phys >= 0) {
                const uint32_t dst = stage_of(stage);
                mbar_arrive_expect_tx(bar_of(stage), L::kStageBytes);
                if constexpr (kFp8) {
                    load(dst, &tmap_k, bar_of(stage), 0, cur.kh, row, phys);
                    load(dst + L::kTileBytes, &tmap_v, bar_of(stage), 0, cur.kh, row, phys);
                } else {
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf) {
                        load(dst + hf * L::kHalfBytes, &tmap_k, bar_of(stage), hf * 64, cur.kh, row,
                             phys);
                        load(dst + L::kTileBytes + hf * L::kHalfBytes, &tmap_v, bar_of(stage),
                             hf * 64, cur.kh, row, phys);
                    }
                }
            } else {
                mbar_arrive(bar_of(stage));
            }
        }
        if (!withheld)
            inflight |= 1u << stage;
        ++issued;
        if (++at_lane == cur.left) {
            look_up(nxt);
            cur = nxt;
            at_lane = 0;
            pdone = cur.u >= u_end;
            if (!pdone)
                nxt = enter(cur.u, cur.k + 1);
        } else if (at_lane == 1) {
            look_up(nxt);
        }
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
    auto load_query = [&](int r, int kh) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hg = nt * 8 + g;
            const T *qrow = static_cast<const T *>(p.query) +
                            ((size_t)r * p.num_heads + (size_t)kh * G + (hg < G ? hg : 0)) * D;
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
    if (u_first < u_end && warp < NW) {
        const Unit x = unit_of(u_first);
        load_query(x.r, x.kh);
    }

    // ---- units --------------------------------------------------------------------
    // The tile warps stream a unit's tiles and hand their (m, l, O) to the merge warp
    // through shared memory; the merge warp combines them, writes the output row or the
    // partition's partial, and -- for split rows -- arrives on the row's counter and
    // merges the partials when its arrival completes them.  The two sides meet only at
    // two named barriers per unit ("records written", and "records read", skipped after
    // the CTA's last unit).
    constexpr int kRecFull = 1, kRecFree = 2;  // named barrier ids (0 is __syncthreads)
    if (warp < NW) {
        int k_unit = 0;          // units of this CTA so far
        for (int u = u_first; u < u_end; ++k_unit) {
            const Unit x = unit_of(u);
            const int un = next_unit(u, x);
            const int ctx = x.ctx;
            float *score_row = nullptr;  // this head group's scores of the sequence
            if constexpr (!kSparse)
                score_row = p.scores + ((size_t)x.s * Hkv + x.kh) * p.pitch * G;

            float o[KT][NT][4];
            float mrun[NT][2], lrun[NT][2];
            int any = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mrun[nt][0] = mrun[nt][1] = -INFINITY;
                lrun[nt][0] = lrun[nt][1] = 0.f;
#pragma unroll
                for (int mt = 0; mt < KT; ++mt)
                    o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
            }
            for (int tile = warp; tile < x.ntiles; tile += NW) {
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
                const int t0 = ready ? stage_pos[warp * NST + stage] : -1;
                if (t0 >= 0 && t0 < ctx) {
                    any = 1;
                    const uint32_t kbase = stage_of(stage);
                    const uint32_t vbase = kbase + L::kTileBytes;
                    // hidden rows: past the context
                    const bool partial = t0 > ctx - kTileTokens;
                    auto seen = [&](int r) { return t0 < ctx - r; };

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

                    if constexpr (!kSparse) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int t = t0 + g + 8 * e, h = nt * 8 + 2 * t4;
                                const float a = sc[nt][2 * e] * p.scale_log2;
                                const float b = sc[nt][2 * e + 1] * p.scale_log2;
                                float *to = score_row + (size_t)t * G + h;
                                if (t < ctx) {
                                    if ((G & 1) == 0) {
                                        if (h < G)
                                            *reinterpret_cast<float2 *>(to) = make_float2(a, b);
                                    } else {
                                        if (h < G)
                                            to[0] = a;
                                        if (h + 1 < G)
                                            to[1] = b;
                                    }
                                }
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
            if (un < u_end) {
                const Unit y = unit_of(un);
                load_query(y.r, y.kh);
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
            if (lane == 0)
                merge_any[warp] = any;
            named_barrier_arrive(kRecFull, kThreads);  // this unit's records are written
            u = un;
        }
    } else {
        // ===== the merge warp ======================================================
        for (int u = u_first; u < u_end;) {
            const Unit x = unit_of(u);
            const int un = next_unit(u, x);
            const bool split = x.nparts > 1;
            named_barrier_sync(kRecFull, kThreads);  // every tile warp's records are in
            int any = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                any |= merge_any[w];
            const int items = G * (D / 8);
            for (int it = lane; it < items; it += 32) {
                const int jh = it / (D / 8);
                const int d0 = (it - jh * (D / 8)) * 8;
                float mmax = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    mmax = fmaxf(mmax, merge_m[w * kHeads + jh]);
                // the partial's m in natural units, and what it stands for in log2 units:
                // l and o go by it, so that nothing is lost in its rounding
                const float m_nat = mmax == -INFINITY ? kNoWeight : mmax * kLn2;
                const float mu = mmax == -INFINITY ? 0.f : m_nat * kLog2e;
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
                // a row that sees nothing is 0, one whose scores are all -inf is not a
                // number, as its softmax; a partial of no weight is 0 either way
                const float inv = lsum == 0.f && (split || !any) ? 0.f : p.out_scale / lsum;
                const size_t h = (size_t)x.kh * G + jh;
                const size_t idx = ((size_t)x.r * p.num_heads + h) * p.max_parts + x.j;
                if (!split) {
                    T vals[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        vals[e] = MmaOp<T>::from_float(acc[e] * inv);
                    *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) +
                                               ((size_t)x.r * p.num_heads + h) * D + d0) =
                        *reinterpret_cast<const uint4 *>(vals);
                } else {
                    // partial of partition j, merged below (or by the reduce kernel)
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + idx * D + d0);
                    dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
                    dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
                }
                if ((split || !kSparse) && d0 == 0) {
                    // (never -inf: the merges take a finite maximum)
                    p.part_m[idx] = any ? m_nat : kNoToken;
                    p.part_l[idx] = any ? lsum : 1.f;
                }
            }
            // the records may be rewritten; the tile warps wait for this only
            // from their next unit on
            if (un < u_end)
                named_barrier_arrive(kRecFree, kThreads);
            if (split && !by_kernel(x.nparts))
                // (eight records loaded per lane at once: of two, long contexts with weights
                // over FP8 pools take 138.4 us for 130.5)
                arrive_and_merge<T, D, kHeads, 8>(p, x.r, x.kh, x.nparts, lane);
            u = un;
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

// ---- accumulated weights -----------------------------------------------------------
//
// One CTA per (sequence, run of kWeightThreads tokens), a thread a token: the
// scores of all heads, turned into weights with the sums over the context, are added
// up head by head, the KV heads' sums then in order.  What bounds it: the scores, 4
// bytes a query head and token, a KV head's being one run of memory for a warp's
// tokens.  The sums over the context are taken anew in each CTA from the partials'
// (m, l), which are few beside the scores.
constexpr int kWeightThreads = 256;

// V: heads loaded at once; GV: loads of a KV head (0: group / V of them, in a loop).
template <int V, int GV>
__global__ void __launch_bounds__(kWeightThreads)
    add_weights_kernel(const __grid_constant__ ListParams p)
{
    using Vec = typename std::conditional<V == 4, float4,
                typename std::conditional<V == 2, float2, float>::type>::type;
    extern __shared__ __align__(16) float sums[];  // m (log2 units) and 1 / l of each head
    const int tid = threadIdx.x;
    const int H = p.num_heads, G = p.group, Hkv = p.num_kv_heads;
    const int runs = (p.pitch + kWeightThreads - 1) / kWeightThreads;
    const int s = blockIdx.x / runs;
    const int first = (blockIdx.x - s * runs) * kWeightThreads;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int ctx = clamp_context(p, s, false);
    if (first >= ctx)
        return;
    // this thread's token: its block is on its way while the sums are taken
    const int pos = first + tid;
    const int phys = pos < ctx ? p.block_tables[(size_t)s * p.max_blocks_per_seq +
                                                (pos >> p.block_shift)] : -1;
    const int seen = p.weighted_lens[s];
    float *m = sums, *inv = sums + H;
    const int parts = p.part_count[s];  // of each head, as the pass counted them
    const float *pm = p.part_m + (size_t)s * H * p.max_parts;
    const float *pl = p.part_l + (size_t)s * H * p.max_parts;
    if (parts <= 4) {  // a thread a query head
        for (int h = tid; h < H; h += kWeightThreads) {
            float mj[4], lj[4], top = -FLT_MAX, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mj[j] = j < parts ? pm[(size_t)h * p.max_parts + j] * kLog2e : -FLT_MAX;
                lj[j] = j < parts ? pl[(size_t)h * p.max_parts + j] : 0.f;
                top = fmaxf(top, mj[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum += lj[j] * exp2f(mj[j] - top);
            m[h] = top;
            inv[h] = __fdiv_rn(1.f, sum);
        }
    } else {  // a warp four query heads at a time, a lane a partial
        constexpr int kWarps = kWeightThreads / 32;
        const int lane = tid & 31;
        for (int h0 = tid >> 5; h0 < H; h0 += 4 * kWarps) {
            float top[4], sum[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                top[u] = -FLT_MAX;
                sum[u] = 0.f;
            }
            for (int j = lane; j < parts; j += 32) {
                float mj[4], lj[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const size_t at = (size_t)min(h0 + u * kWarps, H - 1) * p.max_parts + j;
                    mj[u] = pm[at] * kLog2e;
                    lj[u] = pl[at];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float n = fmaxf(top[u], mj[u]);
                    sum[u] = sum[u] * exp2f(top[u] - n) + lj[u] * exp2f(mj[u] - n);
                    top[u] = n;
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float n = top[u];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    n = fmaxf(n, __shfl_xor_sync(kFull, n, o));
                float l = sum[u] * exp2f(top[u] - n);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    l += __shfl_xor_sync(kFull, l, o);
                if (lane == 0 && h0 + u * kWarps < H) {
                    m[h0 + u * kWarps] = n;
                    inv[h0 + u * kWarps] = __fdiv_rn(1.f, l);
                }
            }
        }
    }
    __syncthreads();
    if (phys < 0 || phys >= p.num_blocks)
        return;  // (flagged by the pass)
    const size_t slot = ((size_t)phys << p.block_shift) + (pos & (p.block_size - 1));
    const float before = pos < seen ? p.weights[slot] : 0.f;
    const float *row = p.scores + ((size_t)s * Hkv * p.pitch + pos) * G;
    float total = 0.f;
#pragma unroll 4
    for (int kh = 0; kh < Hkv; ++kh) {
        const Vec *src = reinterpret_cast<const Vec *>(row + (size_t)kh * p.pitch * G);
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < (GV ? GV : G / V); ++i) {
            const Vec x = __ldcs(src + i);
            const float *e = reinterpret_cast<const float *>(&x);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int h = kh * G + i * V + k;
                part += exp2f(e[k] - m[h]) * inv[h];
            }
        }
        total += part;
    }
    p.weights_out[slot] = before + total;
}

// ---- host side -------------------------------------------------------------------

// Tile warps per CTA (the merge warp comes on top), ring stages per warp and CTAs per
// SM the register budget is sized for: 16-bit pools, FP8 pools.  Windowed decode's 5 warps
// of 2 stages, and 3 CTAs of 4 over FP8 pools, take 319 us for 305 (128 contexts with
// weights) and 132.9 for 130.5 (long ones, FP8); 3 x 4 stages 333, 3 CTAs of 4 x 4 159.
constexpr int kListWarps = 4, kListStages = 2, kListMinBlocks = 2;
constexpr int kListWarpsFp8 = 3, kListStagesFp8 = 3, kListMinBlocksFp8 = 4;

template <typename T, typename KV, int D, int NT, int NST, bool kSparse>
static pa_status launch_list_pass(const ListParams &prm, const CUtensorMap &mk,
                                  const CUtensorMap &mv, cudaStream_t stream,
                                  long long max_units)
{
    constexpr bool kFp8 = sizeof(KV) == 1;
    constexpr int NW = kFp8 ? kListWarpsFp8 : kListWarps;
    // the 16-head variant keeps twice the accumulators: no register cap
    constexpr int MINB = NT > 1 ? 1 : kFp8 ? kListMinBlocksFp8 : kListMinBlocks;
    using L = ListLayout<D, NT, NW, NST, sizeof(KV)>;
    auto kernel = list_decode_kernel<T, KV, D, NT, NW, NST, MINB, kSparse>;
    constexpr int kThreads = (NW + 1) * 32;
    static KernelSetting setting[kMaxDevices];
    static std::mutex mu;
    const size_t smem = L::bytes(prm.share_min > 0 ? prm.num_seqs : 0);
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
    if (prm.share_min > 0 && grid < prm.num_kv_heads)
        return PA_ERR_UNSUPPORTED;  // (the caller takes whole rows)
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), smem, stream, prm, mk, mv);
}

static pa_status launch_add_weights(const ListParams &prm, cudaStream_t stream)
{
    const long long runs = ((long long)prm.pitch + kWeightThreads - 1) / kWeightThreads;
    if (runs * prm.num_seqs > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    const size_t smem = (size_t)prm.num_heads * 8;
    auto kernel = prm.group == 4    ? add_weights_kernel<4, 1>
                  : prm.group == 8  ? add_weights_kernel<4, 2>
                  : prm.group == 16 ? add_weights_kernel<4, 4>
                  : prm.group % 2   ? add_weights_kernel<1, 0>
                                    : add_weights_kernel<2, 0>;
    return launch_pdl(kernel, dim3((unsigned)(runs * prm.num_seqs)), dim3(kWeightThreads), smem,
                      stream, prm);
}

template <typename T, typename KV, int D, int NT, bool kSparse>
static pa_status launch_list(ListParams prm, const CUtensorMap &mk, const CUtensorMap &mv,
                             cudaStream_t stream, int max_parts)
{
    const long long max_units = (long long)prm.num_seqs * prm.num_kv_heads * max_parts;
    constexpr int kStages = sizeof(KV) == 1 ? kListStagesFp8 : kListStages;
    pa_status st =
        launch_list_pass<T, KV, D, NT, kStages, kSparse>(prm, mk, mv, stream, max_units);
    if (st == PA_ERR_UNSUPPORTED && prm.share_min > 0) {
        prm.share_min = 0;
        prm.len_out = nullptr;
        st = launch_list_pass<T, KV, D, NT, kStages, kSparse>(prm, mk, mv, stream, max_units);
    }
    if constexpr (!kSparse)
        if (st == PA_OK)
            st = launch_add_weights(prm, stream);
    if (st != PA_OK || prm.len_out == nullptr)
        return st;
    DecodeParams reduce = prm;
    reduce.counters = nullptr;  // (what it merges was not merged by the pass)
    reduce.context_lens = prm.len_out;  // in partials
    reduce.part_tokens = reduce.block_size = 1;
    reduce.max_blocks_per_seq = reduce.max_context_len = prm.max_parts;
    return launch_reduce<T, D>(reduce, stream);
}

template <typename T, typename KV, bool kSparse>
static pa_status launch_list_as(const ListParams &prm, const CUtensorMap &mk,
                                const CUtensorMap &mv, cudaStream_t stream,
                                int max_parts, int head_dim)
{
    const bool wide = prm.group > 8;
    if (head_dim == 128)
        return wide ? launch_list<T, KV, 128, 2, kSparse>(prm, mk, mv, stream, max_parts)
                    : launch_list<T, KV, 128, 1, kSparse>(prm, mk, mv, stream, max_parts);
    return wide ? launch_list<T, KV, 64, 2, kSparse>(prm, mk, mv, stream, max_parts)
                : launch_list<T, KV, 64, 1, kSparse>(prm, mk, mv, stream, max_parts);
}

// A length whose partitions, counted as the decode pass counts them, are as many as
// list_partitions gives for this one.
static int list_counted(long long len, int partition_size)
{
    if (partition_size <= 0)
        return (int)len;
    return (int)std::min<long long>(
        len, (long long)list_partitions((int)len, partition_size) * partition_size);
}

// Workspaces: that of a decode of as many partitions, then what these passes add.
struct ListWorkspace {
    WorkspaceLayout decode;
    size_t m_off, l_off, len_off, scores_off, total;
};

static ListWorkspace list_workspace(int rows, int H, int Hkv, int D, int parts, long long pitch)
{
    ListWorkspace w{};
    w.decode = workspace_layout(rows, H, Hkv, D, parts);
    w.m_off = w.decode.m_off;
    w.l_off = w.decode.l_off;
    w.total = w.decode.total;
    if (pitch > 0 && parts <= 1) {
        // (behind the arrival counters' place all the same: a workspace that calls with
        // partitions share keeps its zeros)
        const size_t ml = align256((size_t)rows * H * 4);
        w.m_off = align256(std::max<size_t>(kCounterWords, (size_t)rows * Hkv) * 4);
        w.l_off = w.m_off + ml;
        w.total = w.l_off + ml;
    }
    w.len_off = w.total;  // partials of each row: for the reduce kernel, and of all
    if (parts > 1 || pitch > 0)
        w.total += align256((size_t)rows * 8);
    w.scores_off = w.total;
    w.total += align256((size_t)rows * H * (size_t)pitch * 4);
    return w;
}

// Positions of a sequence in the workspace's scores: a tile at least, so that a call on
// contexts of no token has its counts' place too.
static long long score_pitch(int max_context_len)
{
    return ((long long)std::max(1, max_context_len) + kTileTokens - 1) / kTileTokens *
           kTileTokens;
}

// encode_pool_map for pools whose KV heads are read from blocks of their own: a miss brings
// the head's own elements of a token into L2 and not its neighbour's, which the shared
// map's promotion to 256 bytes does (16 lists of 4,096 tokens, FP8: 175 MB from memory for
// 133 MB of listed keys and values).
static bool encode_list_map(CUtensorMap *map, const void *pool, pa_dtype dtype, int num_blocks,
                            int block_size, int num_kv_heads, int head_dim)
{
    EncodeTiledFn fn = get_encode_fn();
    if (!fn)
        return false;
    const bool fp8 = dtype == PA_FP8_E4M3;
    const cuuint64_t e = fp8 ? 1 : 2, row = (cuuint64_t)num_kv_heads * head_dim * e;
    const CUtensorMapDataType ty = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, (cuuint64_t)num_kv_heads,
                                (cuuint64_t)block_size, (cuuint64_t)num_blocks};
    const cuuint64_t strides[3] = {(cuuint64_t)head_dim * e, row, row * block_size};
    const cuuint32_t box[4] = {fp8 ? (cuuint32_t)head_dim : 64u, 1, (cuuint32_t)kTileTokens, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapL2promotion wide = head_dim * e >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                        : head_dim * e >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                              : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    return fn(map, ty, 4, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              fp8 && head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, wide,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool scales_ok(float scale, bool fp8, float k_scale, float v_scale)
{
    if (fp8 && !(std::isfinite(k_scale) && std::isfinite(v_scale) && k_scale > 0.f &&
                 v_scale > 0.f))
        return false;
    return std::isfinite(scale * (fp8 ? k_scale : 1.f) * kLog2e);
}

// What both calls share: the sizes as the decode call checks them, for `rows` rows of
// at most `most` tokens.
template <bool kSparse>
static pa_status run_list(ListParams &prm, void *out, const void *query, const void *key_cache,
                          const void *value_cache, const int32_t *block_tables,
                          int max_blocks_per_seq, const int32_t *lens, long long most, int rows,
                          int num_heads, int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, float scale, bool fp8, float k_scale, float v_scale,
                          int partition_size, void *workspace, size_t workspace_bytes,
                          pa_dtype dtype, int32_t *error_word, void *stream)
{
    if ((dtype != PA_F16 && dtype != PA_BF16) || !scales_ok(scale, fp8, k_scale, v_scale))
        return PA_ERR_INVALID_ARG;
    if (most > INT32_MAX - 512)
        return PA_ERR_UNSUPPORTED;
    const pa_status ok = prepare_decode(
        &prm, out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, lens,
        list_counted(most, partition_size), rows, num_heads, num_kv_heads, head_dim, block_size,
        num_blocks, scale, partition_size, workspace, workspace_bytes, error_word);
    if (ok != PA_OK || rows == 0)
        return ok;
    if ((long long)max_blocks_per_seq * block_size > (1ll << 31) - 256 ||
        (long long)rows * num_kv_heads * prm.max_parts > (1ll << 30))
        return PA_ERR_UNSUPPORTED;
    prm.pitch = kSparse ? 0 : (int)score_pitch((int)most);
    const ListWorkspace w = list_workspace(rows, num_heads, num_kv_heads, head_dim,
                                           prm.max_parts, prm.pitch);
    if (w.total > 0 && (workspace == nullptr || workspace_bytes < w.total ||
                        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return PA_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (!kSparse) {
        prm.part_m = reinterpret_cast<float *>(ws + w.m_off);
        prm.part_l = reinterpret_cast<float *>(ws + w.l_off);
        prm.scores = reinterpret_cast<float *>(ws + w.scores_off);
    }
    // Split rows: shares of a partition or more, and of so many tiles that no row has more
    // partials than there is room for; whole rows where their tiles cannot be numbered in
    // 32 bits, or their numbers do not fit in shared memory.
    const long long tiles =
        (std::min<long long>(most, (long long)max_blocks_per_seq * block_size) + kTileTokens - 1) /
        kTileTokens;
    const int parts = prm.max_parts;
    int32_t *counts = reinterpret_cast<int32_t *>(ws + w.len_off);
    prm.merge_max = kListMergeMax;
    if (!kSparse)
        prm.part_count = counts + rows;
    if (parts > 1 && tiles * rows < (1ll << 29) && rows <= kListShareRows) {
        prm.share_min = (int)std::max<long long>(partition_size / kTileTokens,
                                                 (tiles - 2) / (parts - 1) + 1);
        if (kSparse) {
            // Lists are of one length, or shorter: with fewer of them than CTAs for a KV
            // head, each is cut into as many shares of its own as fill these (16 rows of
            // 4,096 tokens, FP8: 32.9 us; shares across rows have a few partials more to
            // merge, 35.8).
            DeviceInfo info;
            int dev = 0;
            const cudaError_t e = cudaGetDevice(&dev);
            const pa_status di = e != cudaSuccess ? record_cuda(e) : device_info(dev, &info);
            if (di != PA_OK)
                return di;
            const long long ctas = (long long)info.sms *
                                   (prm.group > 8 ? 1 : fp8 ? kListMinBlocksFp8 : kListMinBlocks);
            const long long per = ctas / ((long long)num_kv_heads * rows);
            if (per >= 1) {
                prm.aligned = 1;
                prm.share_min = (int)std::max<long long>(prm.share_min, (tiles + per - 1) / per);
            }
        }
        // shares that the longest row is in: its own, or (n - 2) / W + 2 that begin anywhere
        const long long longest = prm.aligned
                                      ? (tiles + prm.share_min - 1) / prm.share_min
                                      : (tiles + prm.share_min - 2) / prm.share_min + 1;
        if (longest > prm.merge_max)
            prm.len_out = counts;
    }
    prm.max_context_len = (int)most;
    if (fp8) {
        // scores of the K codes: the K scale in the exponent's, the V scale on
        // the outputs and partials
        prm.scale_log2 = scale * k_scale * kLog2e;
        prm.out_scale = v_scale;
    }
    CUtensorMap mk, mv;
    const pa_dtype pool = fp8 ? PA_FP8_E4M3 : dtype;
    const auto encode = kSparse ? encode_list_map : encode_pool_map;
    if (!encode(&mk, key_cache, pool, num_blocks, block_size, num_kv_heads, head_dim) ||
        !encode(&mv, value_cache, pool, num_blocks, block_size, num_kv_heads, head_dim))
        return PA_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    using B16 = __nv_bfloat16;
    if (fp8)
        return dtype == PA_BF16
                   ? launch_list_as<B16, uint8_t, kSparse>(prm, mk, mv, st, parts, head_dim)
                   : launch_list_as<__half, uint8_t, kSparse>(prm, mk, mv, st, parts, head_dim);
    return dtype == PA_BF16 ? launch_list_as<B16, B16, kSparse>(prm, mk, mv, st, parts, head_dim)
                            : launch_list_as<__half, __half, kSparse>(prm, mk, mv, st, parts,
                                                                      head_dim);
}

static pa_status run_sparse(void *out, const void *query, const void *key_cache,
                            const void *value_cache, const int32_t *block_tables,
                            int max_blocks_per_seq, const int32_t *token_seq,
                            const int32_t *token_pos, const int32_t *selected, int top_k,
                            int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                            int head_dim, int block_size, int num_blocks, float scale, bool fp8,
                            float k_scale, float v_scale, int partition_size, void *workspace,
                            size_t workspace_bytes, pa_dtype dtype, int32_t *error_word,
                            void *stream)
{
    if (top_k <= 0 || num_seqs < 0 || num_tokens < 0 || block_size <= 0 ||
        (num_tokens > 0 && (!token_pos || !selected)))
        return PA_ERR_INVALID_ARG;
    ListParams prm{};
    prm.selected = selected;
    prm.token_seq = token_seq;
    prm.token_pos = token_pos;
    prm.top_k = top_k;
    prm.table_rows = num_seqs;
    return run_list<true>(prm, out, query, key_cache, value_cache, block_tables,
                          max_blocks_per_seq, token_seq, (long long)top_k * block_size,
                          num_tokens, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                          scale, fp8, k_scale, v_scale, partition_size, workspace,
                          workspace_bytes, dtype, error_word, stream);
}

static pa_status run_weights(void *out, float *weights_out, const void *query,
                             const void *key_cache, const void *value_cache,
                             const float *weights, const int32_t *block_tables,
                             int max_blocks_per_seq, const int32_t *context_lens,
                             const int32_t *weighted_lens, int max_context_len, int num_seqs,
                             int num_heads, int num_kv_heads, int head_dim, int block_size,
                             int num_blocks, float scale, bool fp8, float k_scale, float v_scale,
                             int partition_size, void *workspace, size_t workspace_bytes,
                             pa_dtype dtype, int32_t *error_word, void *stream)
{
    if (num_seqs < 0 || max_context_len < 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
        (num_seqs > 0 && (!weights_out || !weights || !weighted_lens)))
        return PA_ERR_INVALID_ARG;
    if (num_heads > 4096)  // (their sums are kept in shared memory)
        return PA_ERR_UNSUPPORTED;
    ListParams prm{};
    prm.weights = weights;
    prm.weights_out = weights_out;
    prm.weighted_lens = weighted_lens;
    return run_list<false>(prm, out, query, key_cache, value_cache, block_tables,
                           max_blocks_per_seq, context_lens, max_context_len, num_seqs,
                           num_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, fp8,
                           k_scale, v_scale, partition_size, workspace, workspace_bytes, dtype,
                           error_word, stream);
}

} // namespace pa

using namespace pa;

extern "C" size_t pa_sparse_workspace_bytes(int num_tokens, int num_heads, int num_kv_heads,
                                            int head_dim, int top_k, int block_size,
                                            int partition_size)
{
    const long long most = (long long)top_k * block_size;
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || top_k <= 0 ||
        block_size <= 0 || partition_size < 0 || most > INT32_MAX - 512)
        return 0;
    const int parts = num_parts(list_counted(most, partition_size), partition_size);
    return list_workspace(num_tokens, num_heads, num_kv_heads, head_dim, parts, 0).total;
}

extern "C" size_t pa_weights_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                             int head_dim, int max_context_len,
                                             int partition_size)
{
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || partition_size < 0 || max_context_len > INT32_MAX - 512)
        return 0;
    const int parts = num_parts(list_counted(max_context_len, partition_size), partition_size);
    return list_workspace(num_seqs, num_heads, num_kv_heads, head_dim, parts,
                          score_pitch(max_context_len))
        .total;
}

extern "C" pa_status pa_decode_attention_sparse(
    void *out, const void *query, const void *key_cache, const void *value_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *token_seq,
    const int32_t *token_pos, const int32_t *selected, int top_k, int num_tokens, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    int partition_size, void *workspace, size_t workspace_bytes, pa_dtype dtype,
    int32_t *error_word, void *stream)
{
    return run_sparse(out, query, key_cache, value_cache, block_tables, max_blocks_per_seq,
                      token_seq, token_pos, selected, top_k, num_tokens, num_seqs, num_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, scale, false, 1.f, 1.f,
                      partition_size, workspace, workspace_bytes, dtype, error_word, stream);
}

extern "C" pa_status pa_decode_attention_sparse_fp8(
    void *out, const void *query, const void *key_cache, const void *value_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *token_seq,
    const int32_t *token_pos, const int32_t *selected, int top_k, int num_tokens, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    float k_scale, float v_scale, int partition_size, void *workspace, size_t workspace_bytes,
    pa_dtype dtype, int32_t *error_word, void *stream)
{
    return run_sparse(out, query, key_cache, value_cache, block_tables, max_blocks_per_seq,
                      token_seq, token_pos, selected, top_k, num_tokens, num_seqs, num_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, scale, true, k_scale,
                      v_scale, partition_size, workspace, workspace_bytes, dtype, error_word,
                      stream);
}

extern "C" pa_status pa_decode_attention_weights(
    void *out, float *weights_out, const void *query, const void *key_cache,
    const void *value_cache, const float *weights, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *context_lens, const int32_t *weighted_lens,
    int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, int partition_size, void *workspace,
    size_t workspace_bytes, pa_dtype dtype, int32_t *error_word, void *stream)
{
    return run_weights(out, weights_out, query, key_cache, value_cache, weights, block_tables,
                       max_blocks_per_seq, context_lens, weighted_lens, max_context_len,
                       num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                       scale, false, 1.f, 1.f, partition_size, workspace, workspace_bytes, dtype,
                       error_word, stream);
}

extern "C" pa_status pa_decode_attention_weights_fp8(
    void *out, float *weights_out, const void *query, const void *key_cache,
    const void *value_cache, const float *weights, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *context_lens, const int32_t *weighted_lens,
    int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, float k_scale, float v_scale,
    int partition_size, void *workspace, size_t workspace_bytes, pa_dtype dtype,
    int32_t *error_word, void *stream)
{
    return run_weights(out, weights_out, query, key_cache, value_cache, weights, block_tables,
                       max_blocks_per_seq, context_lens, weighted_lens, max_context_len,
                       num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                       scale, true, k_scale, v_scale, partition_size, workspace,
                       workspace_bytes, dtype, error_word, stream);
}
