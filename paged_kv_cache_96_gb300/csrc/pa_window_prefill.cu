// pa_window_prefill.cu -- entry points of chunked prefill and mixed batches with
// a sliding window and a few first tokens that stay visible: checks of the
// arguments, then the tensor-core kernel.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "pa_window.cuh"

using namespace pa;

static pa_status run_window_prefill(
    void *out, const void *query, const void *key_cache, const void *value_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_start,
    const int32_t *context_lens, int max_context_len, int window, int num_sinks, int num_seqs,
    int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
    int num_blocks, float scale, bool fp8, float k_scale, float v_scale, pa_dtype dtype,
    int32_t *error_word, void *stream)
{
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 ||
        max_context_len < 0 || !std::isfinite(scale) || !(scale > 0.f) ||
        num_heads % num_kv_heads != 0 || window <= 0 || num_sinks < 0 ||
        (dtype != PA_F16 && dtype != PA_BF16))
        return PA_ERR_INVALID_ARG;
    if (fp8 && !(std::isfinite(k_scale) && std::isfinite(v_scale) && k_scale > 0.f &&
                 v_scale > 0.f))
        return PA_ERR_INVALID_ARG;
    const float scale_log2 = scale * (fp8 ? k_scale : 1.f) * kLog2e;
    if (!std::isfinite(scale_log2))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0)
        return PA_OK;
    if (!out || !query || !key_cache || !value_cache || !block_tables || !query_start ||
        !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) ||
        !aligned16(value_cache))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if ((head_dim != 64 && head_dim != 128) || block_size < kTileTokens || block_size > 256 ||
        (block_size & (block_size - 1)) != 0 || group > 16 ||
        num_seqs > kWindowMaxSeqs || (long long)num_blocks * block_size >= (1ll << 31) ||
        // (positions of a whole tile past the last one stay in 32 bits)
        (long long)max_blocks_per_seq * block_size > (1ll << 31) - 256 ||
        (long long)num_tokens * num_heads >= (1ll << 31) - 128)  // (a tile of rows past the last)
        return PA_ERR_UNSUPPORTED;
    // (a row computed anew reads its query after its output was written)
    const uintptr_t o = reinterpret_cast<uintptr_t>(out), q = reinterpret_cast<uintptr_t>(query);
    const uintptr_t row_bytes = (uintptr_t)2 * num_tokens * num_heads * head_dim;
    if (o < q + row_bytes && q < o + row_bytes)
        return PA_ERR_INVALID_ARG;

    WindowMqParams prm{};
    prm.out = out;
    prm.query = query;
    prm.block_tables = block_tables;
    prm.context_lens = context_lens;
    prm.query_start = query_start;
    prm.error_word = error_word;
    prm.wait_ns = stage_wait_limit_ns();
    prm.withhold_fill = withhold_first_fill();
    prm.num_segments = num_seqs;
    prm.num_heads = num_heads;
    prm.num_kv_heads = num_kv_heads;
    prm.group = group;
    prm.max_blocks_per_seq = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.block_size = block_size;
    prm.block_shift = __builtin_ctz((unsigned)block_size);
    prm.max_context_len = max_context_len;
    prm.window = window;
    // (first tokens past the tables' reach hide nothing)
    prm.num_sinks = std::min(num_sinks, max_blocks_per_seq * block_size);
    // The kernel flushes a subnormal factor to 0, and a hidden score of -inf times 0
    // is not a number.  The smallest normal one (2^-126) in its place moves a score
    // below 2^100 by less than 2^-26.
    prm.scale_log2 = std::max(scale_log2, FLT_MIN);
    prm.out_scale = fp8 ? v_scale : 1.f;
    prm.key_cache = key_cache;
    prm.value_cache = value_cache;
    prm.num_tokens = num_tokens;
    return launch_window_tiles(prm, dtype, fp8, head_dim, as_stream(stream));
}

extern "C" pa_status pa_prefill_attention_window(
    void *out, const void *query, const void *key_cache, const void *value_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_start,
    const int32_t *context_lens, int max_context_len, int window, int num_sinks, int num_seqs,
    int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
    int num_blocks, float scale, pa_dtype dtype, int32_t *error_word, void *stream)
{
    return run_window_prefill(out, query, key_cache, value_cache, block_tables,
                              max_blocks_per_seq, query_start, context_lens, max_context_len,
                              window, num_sinks, num_seqs, num_tokens, num_heads, num_kv_heads,
                              head_dim, block_size, num_blocks, scale, false, 1.f, 1.f, dtype,
                              error_word, stream);
}

extern "C" pa_status pa_prefill_attention_window_fp8(
    void *out, const void *query, const void *key_cache, const void *value_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_start,
    const int32_t *context_lens, int max_context_len, int window, int num_sinks, int num_seqs,
    int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
    int num_blocks, float scale, float k_scale, float v_scale, pa_dtype dtype,
    int32_t *error_word, void *stream)
{
    return run_window_prefill(out, query, key_cache, value_cache, block_tables,
                              max_blocks_per_seq, query_start, context_lens, max_context_len,
                              window, num_sinks, num_seqs, num_tokens, num_heads, num_kv_heads,
                              head_dim, block_size, num_blocks, scale, true, k_scale, v_scale,
                              dtype, error_word, stream);
}
