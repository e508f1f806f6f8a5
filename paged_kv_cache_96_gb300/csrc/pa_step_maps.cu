// pa_step_maps.cu -- the index arrays of one serving step, built on the GPU
// from request lengths: block tables extended by new blocks, query offsets,
// and the sequence, position and slot of every new token ("PagedAttention &
// Continuous Batching" §1.4 block table, §1.5 slot mapping; "vLLM 架构详解",
// "Block Table 实现": a block is allocated when a token needs it).
//
// For sequence s with c cached and n new tokens (n = -1: finished) and blocks
// of b tokens:
//     have = ceil(c / b), want = ceil((c + n) / b)
//     finished: its `have` blocks are pushed on the free stack
//     running:  want - have blocks are popped from the top of the stack
//     query_start[s + 1] = sum_{r <= s} max(n_r, 0)
//     token t of s: pos = c + t - query_start[s],
//                   slot = table[s][pos / b] * b + pos % b
// Pushes come before pops; both in batch order, a sequence's blocks in logical
// order, so the result depends on nothing but the inputs.
//
// What bounds it: latency.  The arrays are a few KB to a megabyte, and the
// scan, the pops and the slots depend on one another.  So one thread-block
// cluster does the whole step in one launch -- 1 CTA for small batches, 8 for
// larger ones -- with cluster barriers where the phases meet, in place of a
// chain of scans and gathers over the device:
//   1. each thread sums its run of consecutive sequences (each sequence's
//      lengths are read by its owner alone, so the outputs may be the inputs);
//      a block scan and an exchange through distributed shared memory give the
//      totals, on which every CTA accepts or refuses the step as a whole;
//   2. blocks of finished sequences go on the stack;
//   3. offsets, lengths and new table entries are written (a warp shares the
//      entries of a sequence that takes many blocks);
//   4. tokens are dealt to the warps evenly, whatever the requests' lengths:
//      a warp finds the sequences of its first and last token by 32-way
//      searches over the offsets, its lanes theirs between those.
#include <cooperative_groups.h>

#include "pa_common.cuh"

namespace pa {

namespace cg = cooperative_groups;

constexpr int kMapThreads = 1024;
constexpr int kMapWarps = kMapThreads / 32;
constexpr int kMapMaxCluster = 8;  // largest portable cluster

struct StepMapsParams {
    int32_t *query_start, *token_seq, *token_pos, *slot_mapping;
    int32_t *context_out, *free_count_out;
    int32_t *block_tables;
    const int32_t *context_lens, *query_lens;
    int32_t *free_blocks;
    const int32_t *free_count;
    int32_t *error_word;
    int max_blocks_per_seq, num_seqs, num_tokens, block_size, num_blocks;
};

// Sums over sequences: new tokens, blocks taken, blocks given back; 64 bits,
// since lengths that are refused may be anything.
struct MapSums {
    long long tok, take, give;
};

__device__ __forceinline__ MapSums operator+(const MapSums &a, const MapSums &b)
{
    return {a.tok + b.tok, a.take + b.take, a.give + b.give};
}

// One sequence's lengths and what they ask for.
struct MapSeq {
    int c, n;          // cached tokens, new tokens (finished: 0)
    int have, want;    // blocks before and after (finished: want 0)
    bool finished, bad;
};

__device__ __forceinline__ MapSeq map_seq(const StepMapsParams &p, int s)
{
    MapSeq q;
    const int n = p.query_lens[s];
    q.c = p.context_lens[s];
    q.finished = n == PA_STEP_FINISHED;
    q.n = q.finished ? 0 : n;
    const long long cap = (long long)p.max_blocks_per_seq * p.block_size;
    q.bad = q.c < 0 || q.n < 0 || (long long)q.c + q.n > cap;
    // (only used once every sequence is known to be good)
    const unsigned b = (unsigned)p.block_size;
    q.have = q.bad ? 0 : (int)(((unsigned)q.c + b - 1) / b);
    q.want = q.bad || q.finished ? 0 : (int)(((unsigned)q.c + (unsigned)q.n + b - 1) / b);
    return q;
}

// Largest s in [0, n) with a[s] <= x, for a non-decreasing array with
// a[0] <= x: the warp probes 32 places a step.  a was written in this kernel
// by other CTAs of the cluster, so it is read through L2.
__device__ __forceinline__ int warp_search(const int32_t *a, int n, int x, int lane)
{
    int lo = 0, len = n;  // the answer is in [lo, lo + len)
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int at = lo + lane * step;
        const bool ok = lane * step < len && __ldcg(a + at) <= x;
        const int k = __popc(__ballot_sync(0xffffffffu, ok)) - 1;  // lane 0 is always ok
        lo += k * step;
        len = min(step, len - k * step);
    }
    return lo;
}

__global__ void __launch_bounds__(kMapThreads)
    step_maps_kernel(const __grid_constant__ StepMapsParams p)
{
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.num_seqs;

    __shared__ MapSums warp_sums[kMapWarps];
    __shared__ MapSums cta_sums;  // read by the other CTAs of the cluster
    __shared__ int cta_bad;
    if (tid == 0)
        cta_bad = 0;
    pdl_wait_primary();
    pdl_launch_dependents();
    __syncthreads();

    // ---- 1. this thread's run of sequences, block scan, cluster totals -------------
    const long long threads = (long long)ctas * kMapThreads;
    const int per = (int)((S + threads - 1) / threads);
    const long long s0l = ((long long)rank * kMapThreads + tid) * per;
    const int s0 = (int)min((long long)S, s0l), s1 = (int)min((long long)S, s0l + per);
    MapSums mine{0, 0, 0};
    bool bad = false;
    for (int s = s0; s < s1; ++s) {
        const MapSeq q = map_seq(p, s);
        bad |= q.bad;
        mine = mine + MapSums{q.n, q.finished ? 0 : q.want - q.have, q.finished ? q.have : 0};
    }
    const int free_in = p.free_count[0];
    MapSums scan = mine;  // inclusive, over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const MapSums y{__shfl_up_sync(0xffffffffu, scan.tok, o),
                        __shfl_up_sync(0xffffffffu, scan.take, o),
                        __shfl_up_sync(0xffffffffu, scan.give, o)};
        if (lane >= o)
            scan = scan + y;
    }
    if (lane == 31)
        warp_sums[warp] = scan;
    if (bad)
        cta_bad = 1;
    __syncthreads();
    MapSums before{0, 0, 0};  // exclusive, over the CTA
    if (warp == 0) {
        MapSums w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const MapSums y{__shfl_up_sync(0xffffffffu, w.tok, o),
                            __shfl_up_sync(0xffffffffu, w.take, o),
                            __shfl_up_sync(0xffffffffu, w.give, o)};
            if (lane >= o)
                w = w + y;
        }
        warp_sums[lane] = w;
        if (lane == 31)
            cta_sums = w;
    }
    cluster.sync();
    if (warp > 0)
        before = warp_sums[warp - 1];
    before = before + MapSums{scan.tok - mine.tok, scan.take - mine.take, scan.give - mine.give};
    MapSums total{0, 0, 0};
    int any_bad = 0;
    for (int r = 0; r < ctas; ++r) {
        const MapSums t = *cluster.map_shared_rank(&cta_sums, r);
        any_bad |= *cluster.map_shared_rank(&cta_bad, r);
        if (r < rank)
            before = before + t;
        total = total + t;
    }
    // the step is taken or refused as a whole
    int refuse = 0;
    if (any_bad)
        refuse |= PA_DEVERR_CONTEXT_RANGE;
    else if (total.tok > p.num_tokens)
        refuse |= PA_DEVERR_TOKEN_RANGE;
    else if (free_in < 0 || free_in + total.give > p.num_blocks)
        refuse |= PA_DEVERR_BLOCK_RANGE;
    else if (total.take > free_in + total.give)
        refuse |= PA_DEVERR_OUT_OF_BLOCKS;
    if (refuse != 0) {
        for (int s = s0; s < s1; ++s) {
            p.query_start[s] = 0;
            p.context_out[s] = p.context_lens[s];
        }
        for (long long t = (long long)rank * kMapThreads + tid; t < p.num_tokens; t += threads) {
            p.token_seq[t] = -1;
            p.token_pos[t] = -1;
            p.slot_mapping[t] = -1;
        }
        // every CTA has read the count and the other CTAs' totals
        cluster.sync();
        if (rank == 0 && tid == 0) {
            p.query_start[S] = 0;
            p.free_count_out[0] = free_in;
            flag_error(p.error_word, refuse);
        }
        return;
    }
    // from here on every sum fits 32 bits
    const int top = free_in + (int)total.give;

    // ---- 2. blocks of finished sequences onto the stack -----------------------------
    const int rounds = per;  // sequences of this thread, one a round (warp-uniform)
    if (total.give > 0) {
        int at = free_in + (int)before.give;
        for (int i = 0; i < rounds; ++i) {
            const int s = s0 + i;
            const bool live = s < s1;
            MapSeq q{};
            if (live)
                q = map_seq(p, s);
            const int cnt = live && q.finished ? q.have : 0;
            for (unsigned todo = __ballot_sync(0xffffffffu, cnt > 0); todo != 0; todo &= todo - 1) {
                const int src = __ffs(todo) - 1;
                const int ss = __shfl_sync(0xffffffffu, s, src);
                const int n = __shfl_sync(0xffffffffu, cnt, src);
                const int to = __shfl_sync(0xffffffffu, at, src);
                const int32_t *row = p.block_tables + (size_t)ss * p.max_blocks_per_seq;
                for (int j = lane; j < n; j += 32) {
                    const int32_t id = row[j];
                    if (id < 0 || id >= p.num_blocks)
                        flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                    p.free_blocks[to + j] = id;
                }
            }
            at += cnt;
        }
        cluster.sync();
    }

    // ---- 3. offsets, lengths, new table entries ----------------------------------------
    {
        int start = (int)before.tok, taken = (int)before.take;
        for (int i = 0; i < rounds; ++i) {
            const int s = s0 + i;
            const bool live = s < s1;
            MapSeq q{};
            if (live) {
                q = map_seq(p, s);
                p.query_start[s] = start;
                p.context_out[s] = q.finished ? 0 : q.c + q.n;
            }
            const int cnt = live && !q.finished ? q.want - q.have : 0;
            // the k-th block taken is the k-th from the top of the stack; an id
            // outside the pool is flagged and leaves -1 in the table
            auto take = [&](int ss, int lb, int k) {
                int32_t id = __ldcg(p.free_blocks + (top - 1 - k));
                if (id < 0 || id >= p.num_blocks) {
                    flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                    id = -1;
                }
                p.block_tables[(size_t)ss * p.max_blocks_per_seq + lb] = id;
            };
            if (cnt == 1)
                take(s, q.have, taken);
            for (unsigned todo = __ballot_sync(0xffffffffu, cnt > 1); todo != 0; todo &= todo - 1) {
                const int src = __ffs(todo) - 1;
                const int ss = __shfl_sync(0xffffffffu, s, src);
                const int n = __shfl_sync(0xffffffffu, cnt, src);
                const int lb = __shfl_sync(0xffffffffu, q.have, src);
                const int k = __shfl_sync(0xffffffffu, taken, src);
                for (int j = lane; j < n; j += 32)
                    take(ss, lb + j, k + j);
            }
            start += q.n;
            taken += cnt;
        }
        if (rank == 0 && tid == 0)
            p.query_start[S] = (int32_t)total.tok;
    }
    cluster.sync();
    if (rank == 0 && tid == 0)
        p.free_count_out[0] = top - (int)total.take;

    // ---- 4. every token's sequence, position and slot --------------------------------
    const int warps = ctas * kMapWarps;
    const int runs = (p.num_tokens + 31) / 32;
    const int share = (runs + warps - 1) / warps;  // 32-token runs per warp
    const int gw = rank * kMapWarps + warp;
    const long long t_first = (long long)gw * share * 32;
    const int t_end = (int)min((long long)p.num_tokens, t_first + (long long)share * 32);
    if (t_first >= t_end)
        return;
    const int used = (int)total.tok;
    int lo = 0, hi = 0;
    if (t_first < used) {
        lo = warp_search(p.query_start, S, (int)t_first, lane);
        hi = warp_search(p.query_start, S, min(t_end, used) - 1, lane);
    }
    for (int t = (int)t_first + lane; t < t_end; t += 32) {
        int seq = -1, pos = -1, slot = -1;
        if (t < used) {
            int a = lo, b = hi;  // the largest s with query_start[s] <= t
            while (a < b) {
                const int mid = (a + b + 1) >> 1;
                if (__ldcg(p.query_start + mid) <= t)
                    a = mid;
                else
                    b = mid - 1;
            }
            seq = a;
            pos = __ldcg(p.context_out + seq) - p.query_lens[seq] +
                  (t - __ldcg(p.query_start + seq));
            const int lb = (int)((unsigned)pos / (unsigned)p.block_size);
            const int32_t id =
                __ldcg(p.block_tables + (size_t)seq * p.max_blocks_per_seq + lb);
            if (id < 0 || id >= p.num_blocks)
                flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
            else
                slot = id * p.block_size + (pos - lb * p.block_size);
        }
        p.token_seq[t] = seq;
        p.token_pos[t] = pos;
        p.slot_mapping[t] = slot;
    }
}

} // namespace pa

using namespace pa;

extern "C" pa_status pa_build_step_maps(
    int32_t *query_start, int32_t *token_seq, int32_t *token_pos, int32_t *slot_mapping,
    int32_t *context_lens_out, int32_t *free_count_out, int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *context_lens, const int32_t *query_lens,
    int32_t *free_blocks, const int32_t *free_count, int num_seqs, int num_tokens,
    int block_size, int num_blocks, int32_t *error_word, void *stream)
{
    if (num_seqs < 0 || num_tokens < 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
        num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!query_start || !free_blocks || !free_count || !free_count_out)
        return PA_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!token_seq || !token_pos || !slot_mapping))
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!context_lens_out || !block_tables || !context_lens || !query_lens))
        return PA_ERR_INVALID_ARG;
    if ((long long)num_blocks * block_size > INT32_MAX ||
        (long long)max_blocks_per_seq * block_size > INT32_MAX || num_tokens > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    // An output may be the input of its own kind; query_lens is read to the end.
    if (query_lens != nullptr && (query_lens == context_lens_out || query_lens == query_start))
        return PA_ERR_INVALID_ARG;
    StepMapsParams p;
    p.query_start = query_start;
    p.token_seq = token_seq;
    p.token_pos = token_pos;
    p.slot_mapping = slot_mapping;
    p.context_out = context_lens_out;
    p.free_count_out = free_count_out;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_lens = query_lens;
    p.free_blocks = free_blocks;
    p.free_count = free_count;
    p.error_word = error_word;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.block_size = block_size;
    p.num_blocks = num_blocks;

    const int ctas = num_tokens <= 2 * kMapThreads && num_seqs <= kMapThreads ? 1 : kMapMaxCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kMapThreads);
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return record_cuda(cudaLaunchKernelEx(&cfg, step_maps_kernel, p));
}
