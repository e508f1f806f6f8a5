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
// cluster does the whole step in one launch -- 1 CTA for small batches, 16 for
// larger ones -- with barriers where the phases meet, in place of a chain of
// scans and gathers over the device.  Within a phase nothing is done in turn:
//   1. each CTA sums its sequences, one a thread (each sequence's lengths are
//      read by its owner alone, so the outputs may be the inputs); a block scan
//      and an exchange through distributed shared memory give the totals, on
//      which every CTA accepts or refuses the step as a whole;
//   2. blocks of finished sequences go on the stack,
//   3. offsets, lengths and new table entries are written -- in both, the
//      blocks of all of a CTA's sequences are one list that its threads share,
//      each finding its block's sequence by a search over the scan in shared
//      memory (a warp per sequence, one sequence after another: 12.0 us
//      against 6.1 for 61 requests with 2,048 tokens);
//   4. tokens are dealt to the CTAs evenly, whatever the requests' lengths, in
//      runs whose sequences' offsets are brought to shared memory for the same
//      search (a search through L2 per token: 35 us against 13.4 for
//      4,096 requests with 65,536 tokens).
// 128 requests of one token take 4.6 us a call in a graph: three dependent
// trips to memory (lengths, stack, table) and the launch.
#include <mutex>

#include <cooperative_groups.h>

#include "pa_common.cuh"

namespace pa {

namespace cg = cooperative_groups;

constexpr int kMapThreads = 1024;
constexpr int kMapWarps = kMapThreads / 32;
constexpr int kMapMaxCluster = 16;  // 8 is the largest portable cluster, 16 an opt-in
constexpr int kMapBatch = 4;       // blocks a thread has in flight when it gives them back
constexpr int kMapRun = 4096;      // tokens (and their sequences) a CTA takes at a time

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

// The same by one thread, in shared memory.
__device__ __forceinline__ int thread_search(const int *a, int n, int x)
{
    int lo = 0, len = n;
    while (len > 1) {
        const int half = len >> 1;
        if (a[lo + half] <= x) {
            lo += half;
            len -= half;
        } else {
            len = half;
        }
    }
    return lo;
}

__device__ __forceinline__ MapSums shfl_up(const MapSums &a, int o)
{
    return {__shfl_up_sync(0xffffffffu, a.tok, o), __shfl_up_sync(0xffffffffu, a.take, o),
            __shfl_up_sync(0xffffffffu, a.give, o)};
}

struct MapShared {
    MapSums warp_sums[kMapWarps];  // inclusive over the warps
    MapSums cta_sums;              // read by the other CTAs of the cluster
    MapSums total, upto;           // of the cluster; up to this CTA
    int cta_bad, any_bad;
    int run_lo, run_hi;
    // this CTA's chunk of sequences: blocks taken and given back before each
    int taken[kMapThreads], given[kMapThreads], have[kMapThreads];
    // offsets of a token run's sequences, and position minus token index
    int start[kMapRun], delta[kMapRun];
};

// Exclusive scan over the CTA; the CTA's total is warp_sums[kMapWarps - 1].
__device__ __forceinline__ MapSums block_scan(MapShared &sh, const MapSums &mine, int warp,
                                              int lane)
{
    MapSums x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const MapSums y = shfl_up(x, o);
        if (lane >= o)
            x = x + y;
    }
    if (lane == 31)
        sh.warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        MapSums w = sh.warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const MapSums y = shfl_up(w, o);
            if (lane >= o)
                w = w + y;
        }
        sh.warp_sums[lane] = w;
    }
    __syncthreads();
    MapSums e{x.tok - mine.tok, x.take - mine.take, x.give - mine.give};
    return warp > 0 ? sh.warp_sums[warp - 1] + e : e;
}

__global__ void __launch_bounds__(kMapThreads)
    step_maps_kernel(const __grid_constant__ StepMapsParams p)
{
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.num_seqs;
    __shared__ MapShared sh;
    auto sync_all = [&]() {
        if (ctas > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    if (tid == 0)
        sh.cta_bad = 0;
    __syncthreads();
    pdl_wait_primary();
    pdl_launch_dependents();

    // ---- 1. this CTA's sequences [c0, c1), in chunks of one a thread -------------------
    const int slice = (int)(((long long)S + ctas - 1) / ctas);
    const int c0 = (int)min((long long)S, (long long)rank * slice);
    const int c1 = (int)min((long long)S, (long long)c0 + slice);
    const int chunks = (c1 - c0 + kMapThreads - 1) / kMapThreads;
    const int free_in = p.free_count[0];
    auto lengths = [&](int chunk, MapSeq &q) -> MapSums {
        const int s = c0 + chunk * kMapThreads + tid;
        q = MapSeq{};
        if (s >= c1)
            return MapSums{0, 0, 0};
        q = map_seq(p, s);
        return MapSums{q.n, q.finished ? 0 : q.want - q.have, q.finished ? q.have : 0};
    };
    MapSeq q0;  // the first chunk's stays in registers
    const MapSums m0 = lengths(0, q0);
    MapSums mine = m0;
    bool bad = q0.bad;
    for (int c = 1; c < chunks; ++c) {
        MapSeq q;
        mine = mine + lengths(c, q);
        bad |= q.bad;
    }
    if (bad)
        sh.cta_bad = 1;
    const MapSums scan0 = block_scan(sh, mine, warp, lane);  // (of one chunk: its scan)
    if (tid == 0)
        sh.cta_sums = sh.warp_sums[kMapWarps - 1];
    sync_all();
    // lane r of one warp reads CTA r's sums (every warp doing so took 5 us: they
    // queue up at the CTAs' shared memory)
    if (warp == 0) {
        MapSums x{0, 0, 0};
        bool bad_r = false;
        if (lane < ctas) {
            x = *cluster.map_shared_rank(&sh.cta_sums, lane);
            bad_r = *cluster.map_shared_rank(&sh.cta_bad, lane) != 0;
        }
        const bool any = __any_sync(0xffffffffu, bad_r);
#pragma unroll
        for (int o = 1; o < kMapMaxCluster; o <<= 1) {
            const MapSums y = shfl_up(x, o);
            if (lane >= o)
                x = x + y;
        }
        if (lane == ctas - 1)
            sh.total = x;
        if (lane == rank)
            sh.upto = x;
        if (lane == 0)
            sh.any_bad = any;
    }
    __syncthreads();
    const MapSums total = sh.total, own = sh.cta_sums;
    const MapSums before{sh.upto.tok - own.tok, sh.upto.take - own.take,
                         sh.upto.give - own.give};
    const bool any_bad = sh.any_bad != 0;
    // the step is taken or refused as a whole
    int refuse = 0;
    if (any_bad)
        refuse = PA_DEVERR_CONTEXT_RANGE;
    else if (total.tok > p.num_tokens)
        refuse = PA_DEVERR_TOKEN_RANGE;
    else if (free_in < 0 || free_in + total.give > p.num_blocks)
        refuse = PA_DEVERR_BLOCK_RANGE;
    else if (total.take > free_in + total.give)
        refuse = PA_DEVERR_OUT_OF_BLOCKS;
    if (refuse != 0) {
        for (int s = c0 + tid; s < c1; s += kMapThreads) {
            p.query_start[s] = 0;
            p.context_out[s] = p.context_lens[s];
        }
        for (long long t = (long long)rank * kMapThreads + tid; t < p.num_tokens;
             t += ctas * kMapThreads) {
            p.token_seq[t] = -1;
            p.token_pos[t] = -1;
            p.slot_mapping[t] = -1;
        }
        // every CTA has read the count and the other CTAs' totals
        sync_all();
        if (rank == 0 && tid == 0) {
            p.query_start[S] = 0;
            p.free_count_out[0] = free_in;
            flag_error(p.error_word, refuse);
        }
        return;
    }
    // from here on every sum fits 32 bits
    const int top = free_in + (int)total.give;
    const bool one_chunk = chunks <= 1;

    // ---- 2. blocks of finished sequences onto the stack -----------------------------
    if (total.give > 0) {
        int base = (int)before.give;
        for (int c = 0; c < chunks; ++c) {
            MapSeq q = q0;
            MapSums m = m0, e = scan0;
            if (!one_chunk) {
                m = lengths(c, q);
                e = block_scan(sh, m, warp, lane);
            }
            sh.given[tid] = (int)e.give;
            const int n = (int)sh.warp_sums[kMapWarps - 1].give;
            __syncthreads();
            for (int i0 = tid; i0 < n; i0 += kMapBatch * kMapThreads) {
                int32_t id[kMapBatch];
#pragma unroll
                for (int u = 0; u < kMapBatch; ++u) {
                    const int i = i0 + u * kMapThreads;
                    if (i >= n)
                        continue;
                    const int k = thread_search(sh.given, kMapThreads, i);
                    const int s = c0 + c * kMapThreads + k;
                    id[u] = p.block_tables[(size_t)s * p.max_blocks_per_seq + (i - sh.given[k])];
                }
                bool bad_id = false;
#pragma unroll
                for (int u = 0; u < kMapBatch; ++u) {
                    const int i = i0 + u * kMapThreads;
                    if (i >= n)
                        continue;
                    bad_id |= id[u] < 0 || id[u] >= p.num_blocks;
                    p.free_blocks[free_in + base + i] = id[u];
                }
                if (bad_id)
                    flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
            }
            base += n;
            __syncthreads();
        }
        sync_all();
    }

    // ---- 3. offsets, lengths, new table entries ----------------------------------------
    {
        MapSums base = before;
        for (int c = 0; c < chunks; ++c) {
            MapSeq q = q0;
            MapSums m = m0, e = scan0;
            if (!one_chunk) {
                m = lengths(c, q);
                e = block_scan(sh, m, warp, lane);
            }
            const MapSums sum = sh.warp_sums[kMapWarps - 1];
            const int s = c0 + c * kMapThreads + tid;
            const int start = (int)(base.tok + e.tok);
            if (s < c1) {
                p.query_start[s] = start;
                p.context_out[s] = q.finished ? 0 : q.c + q.n;
            }
            sh.taken[tid] = (int)e.take;
            sh.have[tid] = q.have;
            // (a step of one chunk keeps its offsets here for the tokens)
            sh.start[tid] = start;
            sh.delta[tid] = q.c - start;
            __syncthreads();
            // the k-th block taken is the k-th from the top of the stack; an id
            // outside the pool is flagged and leaves -1 in the table
            for (int i = tid; i < (int)sum.take; i += kMapThreads) {
                const int k = thread_search(sh.taken, kMapThreads, i);
                int32_t id = __ldcg(p.free_blocks + (top - 1 - (int)base.take - i));
                if (id < 0 || id >= p.num_blocks) {
                    flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
                    id = -1;
                }
                p.block_tables[(size_t)(c0 + c * kMapThreads + k) * p.max_blocks_per_seq +
                               sh.have[k] + (i - sh.taken[k])] = id;
            }
            base = base + sum;
            __syncthreads();
        }
        if (rank == 0 && tid == 0)
            p.query_start[S] = (int32_t)total.tok;
    }
    sync_all();
    if (rank == 0 && tid == 0)
        p.free_count_out[0] = top - (int)total.take;

    // ---- 4. every token's sequence, position and slot --------------------------------
    const int used = (int)total.tok;
    const int share = (int)(((long long)p.num_tokens + ctas - 1) / ctas);
    const int t0 = (int)min((long long)p.num_tokens, (long long)rank * share);
    const int t1 = (int)min((long long)p.num_tokens, (long long)t0 + share);
    for (int r0 = t0; r0 < t1; r0 += kMapRun) {
        const int r1 = min(t1, r0 + kMapRun), live = min(r1, used);
        int lo = 0, n = S;  // the run's sequences
        if (r0 < used && (ctas > 1 || !one_chunk)) {
            if (warp < 2) {  // the sequences of the run's first and last token
                const int s = warp_search(p.query_start, S, warp == 0 ? r0 : live - 1, lane);
                if (lane == 0)
                    (warp == 0 ? sh.run_lo : sh.run_hi) = s;
            }
            __syncthreads();
            lo = sh.run_lo;
            n = sh.run_hi - lo + 1;
            for (int i = tid; i < min(n, kMapRun); i += kMapThreads) {
                const int st = __ldcg(p.query_start + lo + i);
                sh.start[i] = st;
                sh.delta[i] = __ldcg(p.context_out + lo + i) - max(p.query_lens[lo + i], 0) - st;
            }
            __syncthreads();
        }
        // all of a thread's table loads go out before one is used
        constexpr int kPer = kMapRun / kMapThreads;
        int seq[kPer], pos[kPer], id[kPer], row[kPer];  // row: place in the block
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int t = r0 + i * kMapThreads + tid;
            seq[i] = pos[i] = id[i] = -1;
            if (t >= live)
                continue;
            if (n <= kMapRun) {
                const int k = thread_search(sh.start, n, t);
                seq[i] = lo + k;
                pos[i] = t + sh.delta[k];
            } else {  // more sequences than tokens in the run: most of them idle
                int a = lo, len = n;
                while (len > 1) {
                    const int half = len >> 1;
                    if (__ldcg(p.query_start + a + half) <= t) {
                        a += half;
                        len -= half;
                    } else {
                        len = half;
                    }
                }
                seq[i] = a;
                pos[i] = __ldcg(p.context_out + a) - p.query_lens[a] +
                         (t - __ldcg(p.query_start + a));
            }
            const int lb = (int)((unsigned)pos[i] / (unsigned)p.block_size);
            row[i] = pos[i] - lb * p.block_size;
            id[i] = __ldcg(p.block_tables + (size_t)seq[i] * p.max_blocks_per_seq + lb);
        }
        bool bad_id = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int t = r0 + i * kMapThreads + tid;
            if (t >= r1)
                continue;
            int slot = -1;
            if (id[i] >= 0 && id[i] < p.num_blocks)
                slot = id[i] * p.block_size + row[i];
            else
                bad_id |= t < live;
            p.token_seq[t] = seq[i];
            p.token_pos[t] = pos[i];
            p.slot_mapping[t] = slot;
        }
        if (bad_id)
            flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
        __syncthreads();
    }
}

// CTAs of the large steps' cluster on the current device, found once: 16 where
// the device can hold such a cluster (4,096 requests with 65,536 tokens: 13.4 us
// against 22.7 with 8), else the portable 8.
static pa_status map_cluster(int *ctas)
{
    constexpr int kDevices = 64;
    static int found[kDevices];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return record_cuda(e);
    if (dev < 0 || dev >= kDevices)
        return PA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    if (found[dev] == 0) {
        e = cudaFuncSetAttribute(step_maps_kernel,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        int clusters = 0;
        if (e == cudaSuccess) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kMapMaxCluster);
            cfg.blockDim = dim3(kMapThreads);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = kMapMaxCluster;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&clusters, step_maps_kernel, &cfg);
        }
        if (e != cudaSuccess)
            return record_cuda(e);
        found[dev] = clusters > 0 ? kMapMaxCluster : 8;
    }
    *ctas = found[dev];
    return PA_OK;
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

    int ctas = 1;
    if (num_tokens > 2 * kMapThreads || num_seqs > kMapThreads) {
        const pa_status st = map_cluster(&ctas);
        if (st != PA_OK)
            return st;
    }
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
