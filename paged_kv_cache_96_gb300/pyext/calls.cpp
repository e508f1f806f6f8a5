// calls.cpp -- the serving-step and long-context entry points of libpaged_attention
// called from Python with torch tensors: argument checks and marshalling, as binding.py does
// through ctypes for the others.
//
// One step of a small batch is a few microseconds of GPU work behind four such
// calls, each with ten tensors whose type, device, layout and address the host
// has to look at.  Attribute by attribute from Python, and through ctypes, the
// smallest calls took 9 to 13 us, host-bound; read from the tensors themselves they
// take 3.4 (4 tokens rotated) to 4.7 (4 sequences of windowed decode).
// The library is opened by the path that binding.py has loaded (bind), so that
// another build of it can stand in.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <dlfcn.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <exception>

#include "../../include/paged_attention.h"

namespace {

struct PythonError {};  // a Python exception is set

[[noreturn]] void fail(PyObject *type, const char *format, ...)
{
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw PythonError{};
}

// ---- the library's entry points -------------------------------------------------

struct Library {
    decltype(&pa_build_step_maps) step_maps;
    decltype(&pa_rope_and_cache) rope;
    decltype(&pa_rope_and_cache_fp8) rope_fp8;
    decltype(&pa_decode_attention_window) decode;
    decltype(&pa_decode_attention_window_fp8) decode_fp8;
    decltype(&pa_prefill_attention_window) prefill;
    decltype(&pa_prefill_attention_window_fp8) prefill_fp8;
    decltype(&pa_summarize_blocks) summarize;
    decltype(&pa_select_blocks) select;
    decltype(&pa_decode_attention_sparse) sparse;
    decltype(&pa_decode_attention_sparse_fp8) sparse_fp8;
    decltype(&pa_decode_attention_weights) weights;
    decltype(&pa_decode_attention_weights_fp8) weights_fp8;
    decltype(&pa_plan_eviction) plan;
    decltype(&pa_plan_eviction_aged) plan_aged;
    decltype(&pa_move_tokens) move;
};
Library lib;

template <typename F> void find(void *handle, const char *name, F &fn)
{
    fn = reinterpret_cast<F>(dlsym(handle, name));
    if (fn == nullptr)
        fail(PyExc_ImportError, "%s is missing from the library", name);
}

// ---- arguments --------------------------------------------------------------------

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, "%s: torch.Tensor expected", name);
    return THPVariable_Unpack(o);
}

// The device of a call's tensors, which has to be the current one (whose stream
// the call is queued on).
int device_of(const at::Tensor &t, const char *name)
{
    if (!t.is_cuda())
        fail(PyExc_ValueError, "%s: must be a CUDA tensor", name);
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device())
        fail(PyExc_ValueError, "%s: on device %d, which is not the current device", name, dev);
    return dev;
}

void on_device(const at::Tensor &t, const char *name, at::ScalarType type, int dev)
{
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, "%s: %s expected, got %s", name, c10::toString(type),
             c10::toString(t.scalar_type()));
    if (!t.is_cuda())
        fail(PyExc_ValueError, "%s: must be a CUDA tensor", name);
    if (t.get_device() != dev)
        fail(PyExc_ValueError, "%s: tensors of one call must be on one device", name);
}

// Address of a contiguous tensor of `type` on device `dev`.
void *address(const at::Tensor &t, const char *name, at::ScalarType type, int dev)
{
    on_device(t, name, type, dev);
    if (!t.is_contiguous())
        fail(PyExc_ValueError, "%s: must be contiguous", name);
    return t.data_ptr();
}

int32_t *ints(const at::Tensor &t, const char *name, int dev)
{
    return static_cast<int32_t *>(address(t, name, at::kInt, dev));
}

int32_t *optional_ints(PyObject *o, const char *name, int dev)
{
    return o == Py_None ? nullptr : ints(tensor(o, name), name, dev);
}

// Address and token stride of [T, heads, d] whose token rows are dense (a view
// into a wider row, as the parts of a fused QKV projection are).
struct Rows {
    void *at;
    int64_t stride;
};

Rows rows(const at::Tensor &t, const char *name, at::ScalarType type, int dev)
{
    on_device(t, name, type, dev);
    const auto size = t.sizes(), stride = t.strides();
    if ((stride[2] != 1 && size[2] > 1) || (stride[1] != size[2] && size[1] > 1))
        fail(PyExc_ValueError, "%s: heads and elements of a token must be dense", name);
    return {t.data_ptr(), size[0] > 1 ? stride[0] : size[1] * size[2]};
}

void dimensions(const at::Tensor &t, const char *name, int n)
{
    if (t.dim() != n)
        fail(PyExc_ValueError, "%s: %d dimensions expected, got %d", name, n, (int)t.dim());
}

// A size as the library's int.
int size_int(int64_t n, const char *name)
{
    if (n > INT32_MAX)
        fail(PyExc_ValueError, "%s: %lld does not fit 32 bits", name, (long long)n);
    return (int)n;
}

int64_t integer(PyObject *o, const char *name, bool saturate)
{
    // (Python's integers and what stands for one, as NumPy's; no float, no text)
    if (!PyIndex_Check(o))
        fail(PyExc_TypeError, "%s: integer expected, got %s", name, Py_TYPE(o)->tp_name);
    PyObject *n = PyNumber_Index(o);
    if (n == nullptr)
        throw PythonError{};
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(n, &over);
    Py_DECREF(n);
    if (v == -1 && over == 0 && PyErr_Occurred())
        throw PythonError{};
    const int64_t x = over > 0 ? INT64_MAX : over < 0 ? INT64_MIN : v;
    if (!saturate && (x > INT32_MAX || x < INT32_MIN))
        fail(PyExc_ValueError, "%s: does not fit 32 bits", name);
    return x;
}

int to_int(PyObject *o, const char *name)
{
    return (int)integer(o, name, false);
}

// A window or a number of first tokens: what passes the int32 range hides as
// little as its largest value, negative ones are refused by the library.
int reach(PyObject *o, const char *name)
{
    return (int)std::max<int64_t>(-1, std::min<int64_t>(integer(o, name, true), INT32_MAX));
}

float to_float(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw PythonError{};
    return (float)v;
}

pa_dtype dtype_of(const at::Tensor &t, const char *name)
{
    if (t.scalar_type() == at::kHalf)
        return PA_F16;
    if (t.scalar_type() == at::kBFloat16)
        return PA_BF16;
    fail(PyExc_TypeError, "%s: fp16 / bf16 tensor expected, got %s", name,
         c10::toString(t.scalar_type()));
}

PyObject *attribute(PyObject *o, const char *name)
{
    PyObject *v = PyObject_GetAttrString(o, name);
    if (v == nullptr)
        throw PythonError{};
    return v;
}

void *queue(PyObject *stream, int dev)
{
    if (stream == Py_None)
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    PyObject *device = attribute(stream, "device");
    PyObject *index = PyObject_GetAttrString(device, "index");
    Py_DECREF(device);
    if (index == nullptr)
        throw PythonError{};
    const long at = PyLong_AsLong(index);
    Py_DECREF(index);
    if (at == -1 && PyErr_Occurred())
        throw PythonError{};
    if (at != dev)
        fail(PyExc_ValueError, "the stream is on another device than the tensors");
    PyObject *raw = attribute(stream, "cuda_stream");
    void *s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (s == nullptr && PyErr_Occurred())
        throw PythonError{};
    return s;
}

// The interpreter is other threads' while the library queues its work.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

void need(bool ok, const char *message)
{
    if (!ok)
        fail(PyExc_ValueError, "%s", message);
}

// ---- the calls --------------------------------------------------------------------

pa_status step_maps(PyObject *const *a)
{
    const at::Tensor &tables = tensor(a[0], "block_tables"), &ctx = tensor(a[1], "context_lens"),
                     &fresh = tensor(a[2], "query_lens"), &stack = tensor(a[3], "free_blocks"),
                     &count = tensor(a[4], "free_count"), &start = tensor(a[7], "query_start"),
                     &seq = tensor(a[8], "token_seq"), &pos = tensor(a[9], "token_pos"),
                     &slots = tensor(a[10], "slot_mapping"),
                     &ctx_out = tensor(a[11], "context_lens_out"),
                     &count_out = tensor(a[12], "free_count_out");
    const int block_size = to_int(a[5], "block_size"), num_blocks = to_int(a[6], "num_blocks");
    dimensions(tables, "block_tables", 2);
    const int64_t S = tables.size(0), T = seq.numel();
    need(ctx.numel() == S && fresh.numel() == S && ctx_out.numel() == S &&
             start.numel() == S + 1,
         "one length per sequence and num_seqs + 1 offsets expected");
    need(pos.numel() == T && slots.numel() == T,
         "token_seq, token_pos and slot_mapping must have one length");
    need(stack.numel() >= num_blocks && count.numel() >= 1 && count_out.numel() >= 1,
         "a stack of num_blocks entries and its count expected");
    const int dev = device_of(tables, "block_tables");
    int32_t *p_start = ints(start, "query_start", dev), *p_seq = ints(seq, "token_seq", dev),
            *p_pos = ints(pos, "token_pos", dev), *p_slots = ints(slots, "slot_mapping", dev),
            *p_ctx_out = ints(ctx_out, "context_lens_out", dev),
            *p_count_out = ints(count_out, "free_count_out", dev),
            *p_tables = ints(tables, "block_tables", dev),
            *p_stack = ints(stack, "free_blocks", dev), *p_count = ints(count, "free_count", dev),
            *p_ctx = ints(ctx, "context_lens", dev), *p_fresh = ints(fresh, "query_lens", dev),
            *err = optional_ints(a[13], "error_word", dev);
    const int max_blocks = size_int(tables.size(1), "block_tables"),
              seqs = size_int(S, "block_tables"), tokens = size_int(T, "token_seq");
    void *stream = queue(a[14], dev);
    const Unlocked unlocked;
    return lib.step_maps(p_start, p_seq, p_pos, p_slots, p_ctx_out, p_count_out, p_tables,
                         max_blocks, p_ctx, p_fresh, p_stack, p_count, seqs, tokens, block_size,
                         num_blocks, err, stream);
}

pa_status rope(PyObject *const *a)
{
    const at::Tensor &out = tensor(a[0], "query_out"), &q = tensor(a[1], "query"),
                     &k = tensor(a[2], "key"), &v = tensor(a[3], "value"),
                     &kc = tensor(a[4], "key_cache"), &vc = tensor(a[5], "value_cache"),
                     &slots = tensor(a[6], "slot_mapping"), &pos = tensor(a[7], "positions"),
                     &freq = tensor(a[8], "inv_freq");
    dimensions(q, "query", 3);
    dimensions(kc, "key_cache", 4);
    const int64_t T = q.size(0), H = q.size(1), d = q.size(2), K = kc.size(2);
    need(d == kc.size(3) && out.sizes() == q.sizes() && k.dim() == 3 && k.size(0) == T &&
             k.size(1) == K && k.size(2) == d && v.sizes() == k.sizes() &&
             vc.sizes() == kc.sizes(),
         "shape mismatch between new tokens and pools");
    need(slots.dim() == 1 && slots.size(0) == T && (pos.dim() == 1 || pos.dim() == 2) &&
             pos.size(-1) == T && freq.dim() == 1,
         "one slot and, per axis, one position per new token expected");
    const int axes = pos.dim() == 2 ? size_int(pos.size(0), "positions") : 1;
    const int half = size_int(freq.size(0), "inv_freq");
    const int32_t *axis = nullptr;
    if (a[9] != Py_None) {
        const at::Tensor &of = tensor(a[9], "axis_of_pair");
        need(of.scalar_type() == at::kInt && of.is_cpu() && of.dim() == 1 &&
                 of.size(0) == half && of.is_contiguous(),
             "axis_of_pair: int32 CPU tensor, one axis per rotary pair");
        axis = static_cast<const int32_t *>(of.data_ptr());
    }
    const int interleaved = PyObject_IsTrue(a[10]);
    if (interleaved < 0)
        throw PythonError{};
    const int dev = device_of(q, "query");
    const pa_dtype dtype = dtype_of(q, "query");
    const at::ScalarType type = q.scalar_type();
    const bool fp8 = kc.scalar_type() == at::kByte;
    const at::ScalarType pool = fp8 ? at::kByte : type;
    const Rows ro = rows(out, "query_out", type, dev), rq = rows(q, "query", type, dev),
               rk = rows(k, "key", type, dev), rv = rows(v, "value", type, dev);
    void *pk = address(kc, "key_cache", pool, dev), *pv = address(vc, "value_cache", pool, dev);
    const int32_t *ps = ints(slots, "slot_mapping", dev), *pp = ints(pos, "positions", dev);
    const float *pf = static_cast<const float *>(address(freq, "inv_freq", at::kFloat, dev));
    const int nT = size_int(T, "query"), nH = size_int(H, "query"), nK = size_int(K, "key"),
              nd = size_int(d, "query"), bs = size_int(kc.size(1), "key_cache"),
              N = size_int(kc.size(0), "key_cache");
    const float ks = to_float(a[11]), vs = to_float(a[12]);
    int32_t *err = optional_ints(a[13], "error_word", dev);
    void *stream = queue(a[14], dev);
    need(half <= INT32_MAX / 2, "inv_freq: too many pairs");
    const Unlocked unlocked;
    if (fp8)
        return lib.rope_fp8(ro.at, ro.stride, rq.at, rq.stride, rk.at, rk.stride, rv.at,
                            rv.stride, pk, pv, ps, pp, axes, axis, pf, 2 * half, interleaved, nT,
                            nH, nK, nd, bs, N, dtype, ks, vs, err, stream);
    return lib.rope(ro.at, ro.stride, rq.at, rq.stride, rk.at, rk.stride, rv.at, rv.stride, pk,
                    pv, ps, pp, axes, axis, pf, 2 * half, interleaved, nT, nH, nK, nd, bs, N,
                    dtype, err, stream);
}

// What the two windowed calls share, in the order of their first arguments.
struct Attention {
    void *out, *query, *key_cache, *value_cache;
    int32_t *tables;
    int max_blocks, rows, heads, kv_heads, dim, block_size, num_blocks, dev;
    bool fp8;
    pa_dtype dtype;
};

Attention attention(PyObject *const *a, int64_t seqs, bool one_row)
{
    const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "query"),
                     &kc = tensor(a[2], "key_cache"), &vc = tensor(a[3], "value_cache"),
                     &tables = tensor(a[4], "block_tables");
    dimensions(q, "query", 3);
    dimensions(kc, "key_cache", 4);
    dimensions(tables, "block_tables", 2);
    need(q.size(2) == kc.size(3) && out.sizes() == q.sizes() && vc.sizes() == kc.sizes() &&
             tables.size(0) == seqs && (!one_row || q.size(0) == seqs),
         "shape mismatch");
    Attention x;
    x.dev = device_of(q, "query");
    x.dtype = dtype_of(q, "query");
    const at::ScalarType type = q.scalar_type();
    x.fp8 = kc.scalar_type() == at::kByte;
    const at::ScalarType pool = x.fp8 ? at::kByte : type;
    x.out = address(out, "out", type, x.dev);
    x.query = address(q, "query", type, x.dev);
    x.key_cache = address(kc, "key_cache", pool, x.dev);
    x.value_cache = address(vc, "value_cache", pool, x.dev);
    x.tables = ints(tables, "block_tables", x.dev);
    x.max_blocks = size_int(tables.size(1), "block_tables");
    x.rows = size_int(q.size(0), "query");
    x.heads = size_int(q.size(1), "query");
    x.dim = size_int(q.size(2), "query");
    x.num_blocks = size_int(kc.size(0), "key_cache");
    x.block_size = size_int(kc.size(1), "key_cache");
    x.kv_heads = size_int(kc.size(2), "key_cache");
    return x;
}

struct Space {
    void *at;
    size_t bytes;
};

Space workspace(PyObject *o, int dev)
{
    if (o == Py_None)
        return {nullptr, 0};
    const at::Tensor &w = tensor(o, "workspace");
    return {address(w, "workspace", w.scalar_type(), dev), w.nbytes()};
}

pa_status decode_window(PyObject *const *a)
{
    const at::Tensor &ctx = tensor(a[5], "context_lens");
    dimensions(ctx, "context_lens", 1);
    const Attention x = attention(a, ctx.size(0), true);
    const int32_t *lens = ints(ctx, "context_lens", x.dev);
    const int max_ctx = to_int(a[6], "max_context_len");
    const float scale = to_float(a[7]);
    const int window = reach(a[8], "window"), sinks = reach(a[9], "num_sinks");
    const int partition = to_int(a[10], "partition_size");
    const Space w = workspace(a[11], x.dev);
    const float ks = to_float(a[12]), vs = to_float(a[13]);
    int32_t *err = optional_ints(a[14], "error_word", x.dev);
    void *stream = queue(a[15], x.dev);
    const Unlocked unlocked;
    if (x.fp8)
        return lib.decode_fp8(x.out, x.query, x.key_cache, x.value_cache, x.tables, x.max_blocks,
                              lens, max_ctx, window, sinks, x.rows, x.heads, x.kv_heads, x.dim,
                              x.block_size, x.num_blocks, scale, ks, vs, partition, w.at, w.bytes,
                              x.dtype, err, stream);
    return lib.decode(x.out, x.query, x.key_cache, x.value_cache, x.tables, x.max_blocks, lens,
                      max_ctx, window, sinks, x.rows, x.heads, x.kv_heads, x.dim, x.block_size,
                      x.num_blocks, scale, partition, w.at, w.bytes, x.dtype, err, stream);
}

pa_status prefill_window(PyObject *const *a)
{
    const at::Tensor &start = tensor(a[5], "query_start"), &ctx = tensor(a[6], "context_lens");
    dimensions(ctx, "context_lens", 1);
    const int64_t S = ctx.size(0);
    need(start.dim() == 1 && start.size(0) == S + 1, "shape mismatch");
    const Attention x = attention(a, S, false);
    const int32_t *offsets = ints(start, "query_start", x.dev),
                  *lens = ints(ctx, "context_lens", x.dev);
    const int max_ctx = to_int(a[7], "max_context_len");
    const float scale = to_float(a[8]);
    const int window = reach(a[9], "window"), sinks = reach(a[10], "num_sinks");
    const float ks = to_float(a[11]), vs = to_float(a[12]);
    int32_t *err = optional_ints(a[13], "error_word", x.dev);
    void *stream = queue(a[14], x.dev);
    const int seqs = size_int(S, "context_lens");
    const Unlocked unlocked;
    if (x.fp8)
        return lib.prefill_fp8(x.out, x.query, x.key_cache, x.value_cache, x.tables, x.max_blocks,
                               offsets, lens, max_ctx, window, sinks, seqs, x.rows, x.heads,
                               x.kv_heads, x.dim, x.block_size, x.num_blocks, scale, ks, vs,
                               x.dtype, err, stream);
    return lib.prefill(x.out, x.query, x.key_cache, x.value_cache, x.tables, x.max_blocks,
                       offsets, lens, max_ctx, window, sinks, seqs, x.rows, x.heads, x.kv_heads,
                       x.dim, x.block_size, x.num_blocks, scale, x.dtype, err, stream);
}

// The 8-bit bounds [num_blocks, num_kv_heads, 2, head_dim] of a pool's blocks.
struct Summaries {
    int8_t *codes;
    float *scales;
    int num_blocks, kv_heads, dim;
};

Summaries summaries(PyObject *codes, PyObject *scales, int dev)
{
    const at::Tensor &c = tensor(codes, "summaries"), &s = tensor(scales, "summary_scales");
    dimensions(c, "summaries", 4);
    dimensions(s, "summary_scales", 2);
    need(c.size(2) == 2 && s.size(0) == c.size(0) && s.size(1) == c.size(1),
         "summaries [num_blocks, num_kv_heads, 2, head_dim] and one scale per block and KV head "
         "expected");
    return {static_cast<int8_t *>(address(c, "summaries", at::kChar, dev)),
            static_cast<float *>(address(s, "summary_scales", at::kFloat, dev)),
            size_int(c.size(0), "summaries"), size_int(c.size(1), "summaries"),
            size_int(c.size(3), "summaries")};
}

pa_status summarize(PyObject *const *a)
{
    const at::Tensor &kc = tensor(a[2], "key_cache"), &tables = tensor(a[3], "block_tables"),
                     &ctx = tensor(a[4], "context_lens");
    dimensions(kc, "key_cache", 4);
    dimensions(tables, "block_tables", 2);
    dimensions(ctx, "context_lens", 1);
    const int64_t S = ctx.size(0);
    const int dev = device_of(kc, "key_cache");
    const pa_dtype dtype = kc.scalar_type() == at::kByte ? PA_FP8_E4M3 : dtype_of(kc, "key_cache");
    const Summaries x = summaries(a[0], a[1], dev);
    need(tables.size(0) == S && kc.size(0) == x.num_blocks && kc.size(2) == x.kv_heads &&
             kc.size(3) == x.dim,
         "shape mismatch between summaries, pool and tables");
    const int32_t *start = nullptr;
    if (a[5] != Py_None) {
        const at::Tensor &q = tensor(a[5], "query_start");
        need(q.dim() == 1 && q.size(0) == S + 1, "query_start: num_seqs + 1 offsets expected");
        start = ints(q, "query_start", dev);
    }
    const void *pool = address(kc, "key_cache", kc.scalar_type(), dev);
    const int32_t *pt = ints(tables, "block_tables", dev), *pc = ints(ctx, "context_lens", dev);
    const int mb = size_int(tables.size(1), "block_tables"), seqs = size_int(S, "context_lens"),
              bs = size_int(kc.size(1), "key_cache");
    int32_t *err = optional_ints(a[6], "error_word", dev);
    void *stream = queue(a[7], dev);
    const Unlocked unlocked;
    return lib.summarize(x.codes, x.scales, pool, pt, mb, pc, start, seqs, x.num_blocks, bs,
                         x.kv_heads, x.dim, dtype, err, stream);
}

pa_status select_blocks(PyObject *const *a)
{
    const at::Tensor &sel = tensor(a[0], "selected"), &q = tensor(a[1], "query"),
                     &tables = tensor(a[4], "block_tables"), &seq = tensor(a[5], "token_seq"),
                     &pos = tensor(a[6], "token_pos");
    dimensions(sel, "selected", 3);
    dimensions(q, "query", 3);
    dimensions(tables, "block_tables", 2);
    const int64_t T = q.size(0);
    const int dev = device_of(q, "query");
    const pa_dtype dtype = dtype_of(q, "query");
    const Summaries x = summaries(a[2], a[3], dev);
    need(q.size(2) == x.dim && sel.size(0) == T && sel.size(1) == x.kv_heads &&
             seq.dim() == 1 && seq.size(0) == T && pos.dim() == 1 && pos.size(0) == T,
         "shape mismatch between query, selected, summaries and tokens");
    const void *pq = address(q, "query", q.scalar_type(), dev);
    int32_t *ps = ints(sel, "selected", dev);
    const int32_t *pt = ints(tables, "block_tables", dev), *pn = ints(seq, "token_seq", dev),
                  *pp = ints(pos, "token_pos", dev);
    const int max_ctx = to_int(a[7], "max_context_len"), bs = to_int(a[8], "block_size"),
              first = to_int(a[9], "num_first"), last = to_int(a[10], "num_last");
    const int top_k = size_int(sel.size(2), "selected"), mb = size_int(tables.size(1), "block_tables"),
              rows = size_int(T, "query"), seqs = size_int(tables.size(0), "block_tables"),
              heads = size_int(q.size(1), "query");
    int32_t *err = optional_ints(a[11], "error_word", dev);
    void *stream = queue(a[12], dev);
    const Unlocked unlocked;
    return lib.select(ps, top_k, pq, x.codes, x.scales, pt, mb, pn, pp, max_ctx, first, last, rows,
                      seqs, heads, x.kv_heads, x.dim, bs, x.num_blocks, dtype, err, stream);
}

pa_status decode_sparse(PyObject *const *a)
{
    const at::Tensor &tables = tensor(a[4], "block_tables"), &seq = tensor(a[5], "token_seq"),
                     &pos = tensor(a[6], "token_pos"), &sel = tensor(a[7], "selected");
    dimensions(tables, "block_tables", 2);
    dimensions(sel, "selected", 3);
    const int64_t S = tables.size(0);
    const Attention x = attention(a, S, false);
    need(seq.dim() == 1 && seq.size(0) == x.rows && pos.dim() == 1 && pos.size(0) == x.rows &&
             sel.size(0) == x.rows && sel.size(1) == x.kv_heads,
         "one sequence, position and list of blocks per KV head for every row expected");
    const int32_t *pn = ints(seq, "token_seq", x.dev), *pp = ints(pos, "token_pos", x.dev),
                  *ps = ints(sel, "selected", x.dev);
    const float scale = to_float(a[8]);
    const int partition = to_int(a[9], "partition_size");
    const Space w = workspace(a[10], x.dev);
    const float ks = to_float(a[11]), vs = to_float(a[12]);
    int32_t *err = optional_ints(a[13], "error_word", x.dev);
    void *stream = queue(a[14], x.dev);
    const int top_k = size_int(sel.size(2), "selected"), seqs = size_int(S, "block_tables");
    const Unlocked unlocked;
    if (x.fp8)
        return lib.sparse_fp8(x.out, x.query, x.key_cache, x.value_cache, x.tables, x.max_blocks,
                              pn, pp, ps, top_k, x.rows, seqs, x.heads, x.kv_heads, x.dim,
                              x.block_size, x.num_blocks, scale, ks, vs, partition, w.at, w.bytes,
                              x.dtype, err, stream);
    return lib.sparse(x.out, x.query, x.key_cache, x.value_cache, x.tables, x.max_blocks, pn, pp,
                      ps, top_k, x.rows, seqs, x.heads, x.kv_heads, x.dim, x.block_size,
                      x.num_blocks, scale, partition, w.at, w.bytes, x.dtype, err, stream);
}

// A pool of one number a slot, [num_blocks, block_size].
void *slot_pool(PyObject *o, const char *name, at::ScalarType type, int num_blocks, int block_size,
                int dev)
{
    const at::Tensor &w = tensor(o, name);
    if (w.dim() != 2 || w.size(0) != num_blocks || w.size(1) != block_size)
        fail(PyExc_ValueError, "%s: [num_blocks, block_size] expected", name);
    return address(w, name, type, dev);
}

float *weight_pool(PyObject *o, const char *name, int num_blocks, int block_size, int dev)
{
    return static_cast<float *>(slot_pool(o, name, at::kFloat, num_blocks, block_size, dev));
}

pa_status decode_weights(PyObject *const *a)
{
    const at::Tensor &ctx = tensor(a[7], "context_lens"), &old = tensor(a[8], "weighted_lens");
    dimensions(ctx, "context_lens", 1);
    const Attention x = attention(a, ctx.size(0), true);
    need(old.dim() == 1 && old.size(0) == ctx.size(0), "one weighted length per sequence expected");
    float *pw_out = weight_pool(a[5], "weights_out", x.num_blocks, x.block_size, x.dev);
    const float *pw = weight_pool(a[6], "weights", x.num_blocks, x.block_size, x.dev);
    const int32_t *pc = ints(ctx, "context_lens", x.dev), *po = ints(old, "weighted_lens", x.dev);
    const int max_ctx = to_int(a[9], "max_context_len");
    const float scale = to_float(a[10]);
    const Space w = workspace(a[11], x.dev);
    const int partition = to_int(a[12], "partition_size");
    const float ks = to_float(a[13]), vs = to_float(a[14]);
    int32_t *err = optional_ints(a[15], "error_word", x.dev);
    void *stream = queue(a[16], x.dev);
    const Unlocked unlocked;
    if (x.fp8)
        return lib.weights_fp8(x.out, pw_out, x.query, x.key_cache, x.value_cache, pw, x.tables,
                               x.max_blocks, pc, po, max_ctx, x.rows, x.heads, x.kv_heads, x.dim,
                               x.block_size, x.num_blocks, scale, ks, vs, partition, w.at, w.bytes,
                               x.dtype, err, stream);
    return lib.weights(x.out, pw_out, x.query, x.key_cache, x.value_cache, pw, x.tables,
                       x.max_blocks, pc, po, max_ctx, x.rows, x.heads, x.kv_heads, x.dim,
                       x.block_size, x.num_blocks, scale, partition, w.at, w.bytes, x.dtype, err,
                       stream);
}

pa_status plan_eviction(PyObject *const *a)
{
    const at::Tensor &moves = tensor(a[0], "moves"), &ctx_out = tensor(a[1], "context_lens_out"),
                     &count_out = tensor(a[2], "free_count_out"), &pool = tensor(a[6], "weights"),
                     &tables = tensor(a[4], "block_tables"), &ctx = tensor(a[5], "context_lens"),
                     &stack = tensor(a[7], "free_blocks"), &count = tensor(a[8], "free_count");
    dimensions(tables, "block_tables", 2);
    dimensions(pool, "weights", 2);
    dimensions(moves, "moves", 3);
    const int64_t S = tables.size(0);
    need(moves.size(0) == S && moves.size(2) == 2, "moves: [num_seqs, max_moves, 2] expected");
    need(ctx.numel() == S && ctx_out.numel() == S, "one length per sequence expected");
    const int dev = device_of(tables, "block_tables");
    const int N = size_int(pool.size(0), "weights"), bs = size_int(pool.size(1), "weights");
    need(stack.numel() >= N && count.numel() >= 1 && count_out.numel() >= 1,
         "a stack of num_blocks entries and its count expected");
    float *pw_out = weight_pool(a[3], "weights_out", N, bs, dev);
    const float *pw = weight_pool(a[6], "weights", N, bs, dev);
    int32_t *pm = ints(moves, "moves", dev), *pco = ints(ctx_out, "context_lens_out", dev),
            *pno = ints(count_out, "free_count_out", dev), *ps = ints(stack, "free_blocks", dev);
    const int32_t *pt = ints(tables, "block_tables", dev), *pc = ints(ctx, "context_lens", dev),
                  *pn = ints(count, "free_count", dev);
    const int max_ctx = to_int(a[9], "max_context_len"), limit = to_int(a[10], "limit"),
              budget = to_int(a[11], "budget"), sinks = to_int(a[12], "num_sinks"),
              recent = to_int(a[13], "num_recent");
    const int most = size_int(moves.size(1), "moves"), mb = size_int(tables.size(1), "block_tables"),
              seqs = size_int(S, "block_tables");
    int32_t *err = optional_ints(a[14], "error_word", dev);
    void *stream = queue(a[15], dev);
    int32_t *ages = nullptr, *numbered = nullptr, *gone = nullptr;
    if (a[16] != Py_None || a[17] != Py_None || a[18] != Py_None) {
        const at::Tensor &n = tensor(a[17], "numbered_lens"), &g = tensor(a[18], "evicted");
        need(n.numel() == S && g.numel() == S, "numbered_lens, evicted: one per sequence expected");
        ages = static_cast<int32_t *>(slot_pool(a[16], "arrivals", at::kInt, N, bs, dev));
        numbered = ints(n, "numbered_lens", dev);
        gone = ints(g, "evicted", dev);
    }
    const Unlocked unlocked;
    if (ages != nullptr)
        return lib.plan_aged(pm, most, pco, pno, pw_out, ages, numbered, gone, pt, mb, pc, pw, ps,
                             pn, max_ctx, limit, budget, sinks, recent, seqs, bs, N, err, stream);
    return lib.plan(pm, most, pco, pno, pw_out, pt, mb, pc, pw, ps, pn, max_ctx, limit, budget,
                    sinks, recent, seqs, bs, N, err, stream);
}

pa_status move_tokens(PyObject *const *a)
{
    const at::Tensor &kc = tensor(a[0], "key_cache"), &vc = tensor(a[1], "value_cache"),
                     &moves = tensor(a[2], "moves");
    dimensions(kc, "key_cache", 4);
    need(vc.sizes() == kc.sizes() && moves.dim() >= 1 && moves.size(-1) == 2,
         "two pools of one shape and moves [..., 2] expected");
    const int dev = device_of(kc, "key_cache");
    const pa_dtype dtype = kc.scalar_type() == at::kByte ? PA_FP8_E4M3 : dtype_of(kc, "key_cache");
    void *pk = address(kc, "key_cache", kc.scalar_type(), dev),
         *pv = address(vc, "value_cache", kc.scalar_type(), dev);
    const int32_t *pm = ints(moves, "moves", dev);
    const int N = size_int(kc.size(0), "key_cache"), bs = size_int(kc.size(1), "key_cache"),
              K = size_int(kc.size(2), "key_cache"), d = size_int(kc.size(3), "key_cache");
    const int64_t n = moves.numel() / 2;
    int32_t *err = optional_ints(a[3], "error_word", dev);
    void *stream = queue(a[4], dev);
    const Unlocked unlocked;
    return lib.move(pk, pv, pm, n, N, bs, K, d, dtype, err, stream);
}

template <pa_status (*call)(PyObject *const *), int count>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        if (lib.step_maps == nullptr)
            fail(PyExc_RuntimeError, "no library is bound");
        if (n != count)
            fail(PyExc_TypeError, "%d arguments expected, got %d", count, (int)n);
        return PyLong_FromLong(call(args));
    } catch (const PythonError &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *bind(PyObject *, PyObject *path)
{
    try {
        const char *name = PyUnicode_AsUTF8(path);
        if (name == nullptr)
            return nullptr;
        void *h = dlopen(name, RTLD_NOW | RTLD_LOCAL);
        if (h == nullptr)
            fail(PyExc_ImportError, "%s", dlerror());
        Library found;
        find(h, "pa_build_step_maps", found.step_maps);
        find(h, "pa_rope_and_cache", found.rope);
        find(h, "pa_rope_and_cache_fp8", found.rope_fp8);
        find(h, "pa_decode_attention_window", found.decode);
        find(h, "pa_decode_attention_window_fp8", found.decode_fp8);
        find(h, "pa_prefill_attention_window", found.prefill);
        find(h, "pa_prefill_attention_window_fp8", found.prefill_fp8);
        find(h, "pa_summarize_blocks", found.summarize);
        find(h, "pa_select_blocks", found.select);
        find(h, "pa_decode_attention_sparse", found.sparse);
        find(h, "pa_decode_attention_sparse_fp8", found.sparse_fp8);
        find(h, "pa_decode_attention_weights", found.weights);
        find(h, "pa_decode_attention_weights_fp8", found.weights_fp8);
        find(h, "pa_plan_eviction", found.plan);
        find(h, "pa_plan_eviction_aged", found.plan_aged);
        find(h, "pa_move_tokens", found.move);
        lib = found;
        Py_RETURN_NONE;
    } catch (const PythonError &) {
        return nullptr;
    }
}

#define PA_ENTRY(fn, count) \
    {#fn, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<fn, count>)), \
     METH_FASTCALL, nullptr}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         PA_ENTRY(step_maps, 15),
                         PA_ENTRY(rope, 15),
                         PA_ENTRY(decode_window, 16),
                         PA_ENTRY(prefill_window, 15),
                         PA_ENTRY(summarize, 8),
                         PA_ENTRY(select_blocks, 13),
                         PA_ENTRY(decode_sparse, 15),
                         PA_ENTRY(decode_weights, 17),
                         PA_ENTRY(plan_eviction, 19),
                         PA_ENTRY(move_tokens, 5),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void)
{
    return PyModule_Create(&module);
}
