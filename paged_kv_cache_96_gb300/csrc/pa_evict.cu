// pa_evict.cu -- sequences that have passed a limit cut down to the cached tokens that
// were attended most, for sm_103a: the plan from the weights that
// pa_decode_attention_weights accumulates, and the K and V rows that it moves.  An
// addition to the pages, whose block manager frees whole sequences ("vLLM 架构详解",
// "Block Table 实现").
//
// For a sequence of c > limit tokens, of which `budget` stay: the first num_sinks, the
// last num_recent, and of the others those with the largest weight (weights that are
// not above 0 count as 0; of equal ones the lower position stays).  Attention does not
// go by the order of cached tokens (their positions are in the rotated keys), so rows
// below `budget` that stay are not moved: the i-th row that stays at or past it takes
// the place of the i-th evicted one before it.  A sequence one step past its limit
// costs a handful of rows, not a copy of the context (step by step: the aged form).
// Blocks behind the budget go back on the free stack, sequences in batch order, blocks in
// logical order.
//
// That also takes the newest tokens to places of evicted ones, behind which older ones
// lie: by place alone the next plan's last num_recent are the newest only where at least
// as many tokens come between two evictions of a sequence (limit - budget + 1 >=
// num_recent).  The aged form keeps each token's number of arrival beside its weight and
// guards by that.
//
// What bounds it: the plan, latency (a sequence's weights are 4 bytes a token, and
// selection is a chain of passes over them); the moves, HBM: 4 rows of num_kv_heads *
// head_dim elements read or written a move.
#include <algorithm>
#include <mutex>

#include "pa_decode_common.cuh"
#include "pa_topk.cuh"

namespace pa {

struct PlanParams {
    int32_t *moves;  // [S][max_moves][2]
    int32_t *context_out, *free_count_out, *free_blocks;
    float *weights_out;
    const int32_t *block_tables, *context_lens, *free_count;
    const float *weights;
    int32_t *error_word;
    int max_moves, max_blocks_per_seq, max_context_len, limit, budget, num_sinks, num_recent;
    int num_seqs, block_shift, num_blocks;
    int apply_later;  // the outputs are the inputs: they are written behind the plan
    // aged form, or null: number of arrival of each token, of those that have one; of each
    // sequence the tokens that have one, and those evicted so far
    int32_t *arrivals, *numbered_lens, *evicted;
};

// What a sequence's length asks for.
struct PlanSeq {
    int c, end;       // tokens before and after
    int keep, have;   // blocks after and before
    bool bad;
};
__device__ __forceinline__ PlanSeq plan_seq(const PlanParams &p, int s)
{
    PlanSeq q;
    q.c = p.context_lens[s];
    const long long cap = (long long)p.max_blocks_per_seq << p.block_shift;
    q.bad = q.c < 0 || q.c > min(cap, (long long)p.max_context_len);
    q.end = !q.bad && q.c > p.limit ? p.budget : q.c;
    const unsigned round = (1u << p.block_shift) - 1;
    q.have = q.bad ? 0 : (int)(((unsigned)q.c + round) >> p.block_shift);
    q.keep = q.bad ? 0 : (int)(((unsigned)q.end + round) >> p.block_shift);
    return q;
}

// Threads of a CTA: 256 for contexts of at most kPlanShort tokens, whose passes are
// short and barriers most of the time, else 1,024.
constexpr int kPlanShort = 2048;
constexpr int kPlanBatch = 4;
// Longest context: places are counted in 32 bits, in steps of kPlanBatch tokens a thread
// past its end.
constexpr int kPlanLongest = INT32_MAX - 65536;
static_assert(kPlanBatch * 1024 <= 65536, "a step past the longest context");

struct PlanShared {
    TopkShared<11> topk;
    int above[32], ties[32], low_above[32], low_ties[32];
    long long given[32], before[32];
};

// Blocks that all sequences give back, and those of sequences below s; whether a
// length is out of range.  By the whole CTA.
struct PlanTotal {
    long long given, before;
    bool bad;
};
template <int THREADS>
__device__ __forceinline__ PlanTotal plan_total(PlanShared &sh, const PlanParams &p, int s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    PlanTotal t{0, 0, false};
    for (int k = tid; k < p.num_seqs; k += THREADS) {
        const PlanSeq q = plan_seq(p, k);
        t.given += q.have - q.keep;
        t.before += k < s ? q.have - q.keep : 0;
        t.bad |= q.bad;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        t.given += __shfl_xor_sync(kFull, t.given, o);
        t.before += __shfl_xor_sync(kFull, t.before, o);
    }
    if (lane == 0) {
        sh.given[warp] = t.given;
        sh.before[warp] = t.before;
    }
    t.bad = __syncthreads_or(t.bad);
    t.given = t.before = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        t.given += sh.given[w];
        t.before += sh.before[w];
    }
    return t;
}

// The plan is taken or refused as a whole; every CTA finds out for itself.
__device__ __forceinline__ int plan_refusal(const PlanParams &p, const PlanTotal &t)
{
    const int count = p.free_count[0];
    return t.bad ? PA_DEVERR_CONTEXT_RANGE
           : count < 0 || count + t.given > p.num_blocks ? PA_DEVERR_BLOCK_RANGE : 0;
}

// One CTA per sequence.  kKept: the keys of the whole context, and its table row, fit in
// shared memory; else each pass reads the weights again, through L2.  kAged: the last
// num_recent are those that arrived last, wherever they lie: candidates whose key is above
// any weight's.  A template of its own, so that the form by place has no test of it (plans
// of 128 sequences, those past 4,096 tokens halved: 17.6 us by place, 19.2 aged; of one
// token past 2,048 each: 12.8 and 10.5).
template <int THREADS, bool kKept, bool kAged>
__global__ void __launch_bounds__(THREADS)
    plan_eviction_kernel(const __grid_constant__ PlanParams p)
{
    __shared__ PlanShared sh;
    extern __shared__ uint32_t keys[];  // then the table row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x;
    pdl_wait_primary();

    int32_t *moves = p.moves + (size_t)s * p.max_moves * 2;
    const PlanSeq q = plan_seq(p, s);
    const int bs = 1 << p.block_shift;
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    int *row = reinterpret_cast<int *>(keys) + p.max_context_len;
    // a pool block, -1 (flagged) for one that is not in the pool
    auto block_of = [&](int b) {
        const int id = __ldg(table + b);
        if (id < 0 || id >= p.num_blocks) {
            flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
            return -1;
        }
        return id;
    };
    if (kKept)
        for (int b = tid; b < q.have; b += THREADS)
            row[b] = block_of(b);
    // the token at place i >= numbered has number i + gone
    const int gone = kAged ? p.evicted[s] : 0;
    int numbered = kAged ? p.numbered_lens[s] : 0;
    const PlanTotal sum = plan_total<THREADS>(sh, p, s);  // (with a barrier)
    const int refuse = plan_refusal(p, sum);
    const int slots = p.num_blocks << p.block_shift;
    auto slot_of = [&](int pos) {
        const int b = kKept ? row[pos >> p.block_shift] : block_of(pos >> p.block_shift);
        return b < 0 ? -1 : (b << p.block_shift) + (pos & (bs - 1));
    };
    if (!p.apply_later && tid == 0) {
        p.context_out[s] = refuse ? q.c : q.end;
        if (s == 0) {
            p.free_count_out[0] = p.free_count[0] + (refuse ? 0 : (int)sum.given);
            if (refuse)
                flag_error(p.error_word, refuse);
        }
    }
    int count = 0;  // moves
    if (refuse == 0) {
        // blocks behind the budget onto the stack
        int32_t *top = p.free_blocks + p.free_count[0] + sum.before;
        for (int i = tid; i < q.have - q.keep; i += THREADS) {
            const int id = __ldg(table + q.keep + i);
            if (id < 0 || id >= p.num_blocks)
                flag_error(p.error_word, PA_DEVERR_BLOCK_RANGE);
            top[i] = id;
        }
        // chosen from [first, tail)
        const int first = p.num_sinks, tail = kAged ? q.c : q.c - p.num_recent;
        const int n = q.end != q.c ? tail - first : 0;
        if (kAged && n > 0) {
            if (numbered < 0 || numbered > q.c) {
                if (tid == 0)
                    flag_error(p.error_word, PA_DEVERR_CONTEXT_RANGE);
                numbered = 0;
            }
            for (int i = numbered + tid; i < q.c; i += THREADS) {
                const int at = slot_of(i);
                if (at >= 0)
                    p.arrivals[at] = (int)((uint32_t)i + (uint32_t)gone);
            }
            __syncthreads();
            if (tid == 0) {
                p.numbered_lens[s] = q.end;
                p.evicted[s] = (int)((uint32_t)gone + (uint32_t)(q.c - q.end));
            }
        }
        // (by its bits: a comparison would take subnormal weights for 0)
        auto weight_key = [](float weight) {
            const int w = __float_as_int(weight);
            return w > 0 && w <= 0x7f800000 ? (uint32_t)w : 0u;
        };
        // (numbers of arrival are taken modulo 2^32: of the last num_recent a difference is
        // below it)
        const uint32_t oldest = (uint32_t)q.c + (uint32_t)gone - (uint32_t)p.num_recent;
        auto token_key = [&](float weight, int number) {
            return kAged && (uint32_t)number - oldest < (uint32_t)p.num_recent
                       ? 0xffffffffu : weight_key(weight);
        };
        // keys of the candidates, and the weights below the new length in their places;
        // kPlanBatch tokens of a thread at a time
        const bool apart = p.weights_out != p.weights;
        const int reach = kKept && n > 0 ? max(tail, q.end) : apart ? q.end : 0;
        for (int i0 = tid; i0 < reach; i0 += kPlanBatch * THREADS) {
            int at[kPlanBatch];
            float w[kPlanBatch];
            int age[kPlanBatch];
#pragma unroll
            for (int u = 0; u < kPlanBatch; ++u)
                at[u] = slot_of(min(i0 + u * THREADS, reach - 1));
#pragma unroll
            for (int u = 0; u < kPlanBatch; ++u) {
                w[u] = at[u] >= 0 ? p.weights[at[u]] : 0.f;
                age[u] = kAged && n > 0 && at[u] >= 0 ? p.arrivals[at[u]] : (int)oldest - 1;
            }
#pragma unroll
            for (int u = 0; u < kPlanBatch; ++u) {
                const int i = i0 + u * THREADS;
                if (i >= reach)
                    continue;
                if (apart && i < q.end && at[u] >= 0)
                    p.weights_out[at[u]] = w[u];
                if (kKept && i >= first && i < first + n)
                    keys[i - first] = token_key(w[u], age[u]);
            }
        }
        __syncthreads();
        if (n > 0) {
            const int want = p.budget - first - (kAged ? 0 : p.num_recent);
            auto key = [&](int i) {
                if (kKept)
                    return keys[i];
                const int at = slot_of(first + i);
                if (at < 0)
                    return 0u;
                return token_key(p.weights[at], kAged ? p.arrivals[at] : 0);
            };
            const Threshold cut = top_threshold<THREADS, 11>(sh.topk, key, n, want);
            // a warp's run of them; the tokens that stay before each run
            const int run = (n + THREADS - 1) / THREADS * 32;
            const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
            const int low = p.budget - first;  // candidates below the budget
            int above = 0, ties = 0, low_above = 0, low_ties = 0;
            for (int i = i0 + lane; i < i1; i += 32) {
                const uint32_t v = cut.level(key(i));
                above += v > cut.prefix;
                ties += v == cut.prefix;
                low_above += i < low && v > cut.prefix;
                low_ties += i < low && v == cut.prefix;
            }
            above = __reduce_add_sync(kFull, above);
            ties = __reduce_add_sync(kFull, ties);
            low_above = __reduce_add_sync(kFull, low_above);
            low_ties = __reduce_add_sync(kFull, low_ties);
            if (lane == 0) {
                sh.above[warp] = above;
                sh.ties[warp] = ties;
                sh.low_above[warp] = low_above;
                sh.low_ties[warp] = low_ties;
            }
            __syncthreads();
            above = ties = low_above = low_ties = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                above += w < warp ? sh.above[w] : 0;
                ties += w < warp ? sh.ties[w] : 0;
                low_above += sh.low_above[w];
                low_ties += sh.low_ties[w];
            }
            // candidates below the budget that stay (of equal ones the first)
            const int low_kept = low_above + min(low_ties, cut.rest);
            // visit(i, stays, how many before it do) for every candidate of the run
            auto walk = [&](auto &&visit) {
                int a = above, t = ties;
                for (int b = i0; b < i1; b += 32) {
                    const int i = b + lane;
                    const uint32_t v = i < i1 ? cut.level(key(i)) : 0u;
                    const uint32_t over = __ballot_sync(kFull, i < i1 && v > cut.prefix);
                    const uint32_t tie = __ballot_sync(kFull, i < i1 && v == cut.prefix);
                    const uint32_t below = (1u << lane) - 1;
                    const int my_ties = t + __popc(tie & below);
                    const bool stays =
                        (over >> lane & 1) || ((tie >> lane & 1) && my_ties < cut.rest);
                    if (i < i1)
                        visit(i, stays, a + __popc(over & below) + min(my_ties, cut.rest));
                    a += __popc(over);
                    t += __popc(tie);
                }
            };
            walk([&](int i, bool stays, int before) {
                if (i < low && !stays)
                    moves[2 * (i - before) + 1] = slot_of(first + i);
                if (i >= low && stays)
                    moves[2 * (before - low_kept)] = slot_of(first + i);
            });
            // the last tokens, from the budget on
            const int late = max(tail, p.budget);
            const int done = want - low_kept;  // rows before them
            for (int i = late + tid; i < q.c; i += THREADS)
                moves[2 * (done + i - late)] = slot_of(i);
            count = done + q.c - late;
            __syncthreads();
            for (int i = tid; i < count; i += THREADS) {
                const int src = moves[2 * i], dst = moves[2 * i + 1];
                if (src >= 0 && src < slots && dst >= 0 && dst < slots) {
                    p.weights_out[dst] = p.weights[src];
                    if (kAged)
                        p.arrivals[dst] = p.arrivals[src];
                }
            }
        }
    }
    for (int i = 2 * count + tid; i < 2 * p.max_moves; i += THREADS)
        moves[i] = -1;
    // (from its start, the moves' CTAs would take the SMs that later CTAs of the plan need:
    // 128 sequences and their moves 104 us, 101 from here)
    pdl_launch_dependents();
}

// Lengths and the stack's count where they replace the inputs, which every CTA of the
// plan reads: one CTA behind it.  (With arrays of their own for the outputs the plan
// writes them, and this launch, about 2 us behind it, is left out.)
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
    apply_eviction_kernel(const __grid_constant__ PlanParams p)
{
    __shared__ PlanShared sh;
    pdl_wait_primary();
    pdl_launch_dependents();
    const PlanTotal t = plan_total<THREADS>(sh, p, 0);
    const int refuse = plan_refusal(p, t);
    const int count = p.free_count[0];
    __syncthreads();  // (the count has been read)
    for (int s = threadIdx.x; s < p.num_seqs; s += THREADS) {
        const PlanSeq q = plan_seq(p, s);
        p.context_out[s] = refuse ? q.c : q.end;
    }
    if (threadIdx.x == 0) {
        p.free_count_out[0] = refuse ? count : count + (int)t.given;
        if (refuse)
            flag_error(p.error_word, refuse);
    }
}

// ---- moves --------------------------------------------------------------------------
//
// A warp takes an entry of the list at a time, with the next one on its way (a padding
// entry costs its eight bytes), and copies the K and V rows of a move together, all of a
// lane's loads before its stores, 16 bytes a lane.  60,000 moves of 4 KB among 262,000
// entries, with their plan: 100 us; runs of two or four entries a warp 102 and 112.
constexpr int kMoveThreads = 256;
constexpr int kMoveWords = 8;  // of a lane at once
constexpr int kMoveCtas = 4;   // resident on an SM, which the grid fills once

__global__ void __launch_bounds__(kMoveThreads, kMoveCtas)
    move_tokens_kernel(uint4 *__restrict__ key_cache, uint4 *__restrict__ value_cache,
                       const int2 *__restrict__ moves, long long num_moves, long long num_slots,
                       int words, int32_t *error_word)
{
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kMoveThreads / 32);
    long long at = (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    pdl_wait_primary();
    pdl_launch_dependents();
    auto entry = [&](long long i) { return i < num_moves ? __ldg(moves + i) : make_int2(-1, -1); };
    int2 next = entry(at);
    for (; at < num_moves; at += warps) {
        const int2 move = next;
        next = entry(at + warps);
        if (move.x < 0 || move.y < 0)
            continue;
        if (move.x >= num_slots || move.y >= num_slots) {
            if (lane == 0)
                flag_error(error_word, PA_DEVERR_SLOT_RANGE);
            continue;
        }
        const size_t src = (size_t)move.x * words, dst = (size_t)move.y * words;
        // words of the key row, then of the value row
        for (int i0 = lane; i0 < 2 * words; i0 += 32 * kMoveWords) {
            uint4 w[kMoveWords];
#pragma unroll
            for (int u = 0; u < kMoveWords; ++u) {
                const int i = i0 + 32 * u;
                if (i < 2 * words)
                    w[u] = __ldcs(i < words ? key_cache + src + i : value_cache + src + i - words);
            }
#pragma unroll
            for (int u = 0; u < kMoveWords; ++u) {
                const int i = i0 + 32 * u;
                if (i < words)
                    __stcs(key_cache + dst + i, w[u]);
                else if (i < 2 * words)
                    __stcs(value_cache + dst + i - words, w[u]);
            }
        }
    }
}

// ---- host side -------------------------------------------------------------------

template <bool kAged>
static pa_status launch_plan(const PlanParams &p, cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return record_cuda(e);
    DeviceInfo info;
    const pa_status st = device_info(dev, &info);
    if (st != PA_OK)
        return st;
    const size_t blocks =
        ((size_t)p.max_context_len + (((size_t)1 << p.block_shift) - 1)) >> p.block_shift;
    const size_t smem =
        ((size_t)p.max_context_len + std::min<size_t>((size_t)p.max_blocks_per_seq, blocks)) * 4;
    if (smem + sizeof(PlanShared) + 1024 > (size_t)info.optin)
        return launch_pdl(plan_eviction_kernel<1024, false, kAged>, dim3(p.num_seqs), dim3(1024), 0,
                          stream, p);
    const bool small = p.max_context_len <= kPlanShort;
    auto kernel = small ? plan_eviction_kernel<256, true, kAged>
                        : plan_eviction_kernel<1024, true, kAged>;
    static size_t enabled[2][kMaxDevices];
    static std::mutex mu;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (smem > enabled[small][dev]) {
            const cudaError_t a = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (a != cudaSuccess)
                return record_cuda(a);
            enabled[small][dev] = smem;
        }
    }
    return launch_pdl(kernel, dim3(p.num_seqs), dim3(small ? 256 : 1024), smem, stream, p);
}

static pa_status run_plan(int32_t *moves, int max_moves, int32_t *context_lens_out,
                          int32_t *free_count_out, float *weights_out,
                          const int32_t *block_tables, int max_blocks_per_seq,
                          const int32_t *context_lens, const float *weights,
                          int32_t *free_blocks, const int32_t *free_count, int max_context_len,
                          int limit, int budget, int num_sinks, int num_recent, int num_seqs,
                          int block_size, int num_blocks, int32_t *arrivals,
                          int32_t *numbered_lens, int32_t *evicted, int32_t *error_word,
                          void *stream)
{
    if (num_seqs < 0 || max_moves < 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
        num_blocks <= 0 || max_context_len < 0 || budget <= 0 || limit < budget ||
        num_sinks < 0 || num_recent < 0 || num_sinks > budget ||
        num_recent > budget - num_sinks ||
        max_moves < std::min(budget, std::max(0, max_context_len - budget)))
        return PA_ERR_INVALID_ARG;
    if (!free_blocks || !free_count || !free_count_out)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!context_lens_out || !block_tables || !context_lens || !weights ||
                         !weights_out || (max_moves > 0 && !moves)))
        return PA_ERR_INVALID_ARG;
    if ((block_size & (block_size - 1)) != 0 || (long long)num_blocks * block_size > INT32_MAX ||
        (long long)max_blocks_per_seq * block_size > INT32_MAX || max_moves > (1 << 29) ||
        std::min(max_context_len, max_blocks_per_seq * block_size) > kPlanLongest)
        return PA_ERR_UNSUPPORTED;
    PlanParams p{};
    p.moves = moves;
    p.context_out = context_lens_out;
    p.free_count_out = free_count_out;
    p.free_blocks = free_blocks;
    p.weights_out = weights_out;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.free_count = free_count;
    p.weights = weights;
    p.arrivals = arrivals;
    p.numbered_lens = numbered_lens;
    p.evicted = evicted;
    p.error_word = error_word;
    p.max_moves = max_moves;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.limit = limit;
    p.budget = budget;
    p.num_sinks = num_sinks;
    p.num_recent = num_recent;
    p.num_seqs = num_seqs;
    p.block_shift = __builtin_ctz((unsigned)block_size);
    p.num_blocks = num_blocks;
    const auto apart = [](const int32_t *a, long long n, const int32_t *b, long long m) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
        return x + 4 * n <= y || y + 4 * m <= x;
    };
    p.apply_later = num_seqs == 0 || !apart(context_lens_out, num_seqs, context_lens, num_seqs) ||
                    !apart(context_lens_out, num_seqs, free_count, 1) ||
                    !apart(free_count_out, 1, free_count, 1) ||
                    !apart(free_count_out, 1, context_lens, num_seqs);
    cudaStream_t q = as_stream(stream);
    if (num_seqs > 0) {
        const pa_status st =
            arrivals != nullptr ? launch_plan<true>(p, q) : launch_plan<false>(p, q);
        if (st != PA_OK)
            return st;
    }
    if (!p.apply_later)
        return PA_OK;
    return launch_pdl(apply_eviction_kernel<1024>, dim3(1), dim3(1024), 0, q, p);
}

} // namespace pa

using namespace pa;

extern "C" pa_status pa_plan_eviction(int32_t *moves, int max_moves, int32_t *context_lens_out,
                                      int32_t *free_count_out, float *weights_out,
                                      const int32_t *block_tables, int max_blocks_per_seq,
                                      const int32_t *context_lens, const float *weights,
                                      int32_t *free_blocks, const int32_t *free_count,
                                      int max_context_len, int limit, int budget, int num_sinks,
                                      int num_recent, int num_seqs, int block_size,
                                      int num_blocks, int32_t *error_word, void *stream)
{
    return run_plan(moves, max_moves, context_lens_out, free_count_out, weights_out, block_tables,
                    max_blocks_per_seq, context_lens, weights, free_blocks, free_count,
                    max_context_len, limit, budget, num_sinks, num_recent, num_seqs, block_size,
                    num_blocks, nullptr, nullptr, nullptr, error_word, stream);
}

extern "C" pa_status pa_plan_eviction_aged(
    int32_t *moves, int max_moves, int32_t *context_lens_out, int32_t *free_count_out,
    float *weights_out, int32_t *arrivals, int32_t *numbered_lens, int32_t *evicted,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    const float *weights, int32_t *free_blocks, const int32_t *free_count, int max_context_len,
    int limit, int budget, int num_sinks, int num_recent, int num_seqs, int block_size,
    int num_blocks, int32_t *error_word, void *stream)
{
    if (num_seqs > 0 && (!arrivals || !numbered_lens || !evicted))
        return PA_ERR_INVALID_ARG;
    return run_plan(moves, max_moves, context_lens_out, free_count_out, weights_out, block_tables,
                    max_blocks_per_seq, context_lens, weights, free_blocks, free_count,
                    max_context_len, limit, budget, num_sinks, num_recent, num_seqs, block_size,
                    num_blocks, arrivals, numbered_lens, evicted, error_word, stream);
}

extern "C" pa_status pa_move_tokens(void *key_cache, void *value_cache, const int32_t *moves,
                                    int64_t num_moves, int num_blocks, int block_size,
                                    int num_kv_heads, int head_dim, pa_dtype dtype,
                                    int32_t *error_word, void *stream)
{
    if (num_moves < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_FP8_E4M3))
        return PA_ERR_INVALID_ARG;
    if (num_moves == 0)
        return PA_OK;
    if (!key_cache || !value_cache || !moves || !aligned16(key_cache) ||
        !aligned16(value_cache) || (reinterpret_cast<uintptr_t>(moves) & 7u) != 0)
        return PA_ERR_INVALID_ARG;
    const long long row_bytes = (long long)num_kv_heads * head_dim * (dtype == PA_FP8_E4M3 ? 1 : 2);
    if (row_bytes % 16 != 0 || row_bytes > (1 << 24) || num_moves > (1ll << 40) ||
        (long long)num_blocks * block_size > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return record_cuda(e);
    DeviceInfo info;
    const pa_status st = device_info(dev, &info);
    if (st != PA_OK)
        return st;
    const long long warps = kMoveThreads / 32;
    const int grid = (int)std::min<long long>(kMoveCtas * (long long)info.sms,
                                              (num_moves + warps - 1) / warps);
    return launch_pdl(move_tokens_kernel, dim3(grid), dim3(kMoveThreads), 0, as_stream(stream),
                      static_cast<uint4 *>(key_cache), static_cast<uint4 *>(value_cache),
                      reinterpret_cast<const int2 *>(moves), (long long)num_moves,
                      (long long)num_blocks * block_size, (int)(row_bytes / 16), error_word);
}
