// The short calls (those of the attention layers, the acceptance, and the delta
// rule's prompts and single tokens) for Python without its cost: of the 8 to 11
// us that api.py spends around a library call, most are some fifty queries of
// tensors from Python and the allocations.  Back to back on a GB300's host an
// append takes 4.8 us so and 11.9 without, an attention 8.6 and 18.2, log
// probabilities 6.3 and 15.6.
//
// Each function takes the address of the library's packed entry point and
// api.py's arguments in order.  It answers None, having done nothing, where
// anything is not plainly as it should be (api.py then finds out what, and
// says so), the library's status where that is not 0, and the outputs.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "kda.h"

namespace {

using at::Tensor;

struct NotPlain {};  // thrown where api.py has to look

void need(bool ok) {
    if (!ok) throw NotPlain{};
}

// The library launches on the current device; where the tensors are on another
// GPU, api.py switches to it.
void need_current(c10::Device device) {
    need(device.is_cuda() && device.index() == c10::cuda::current_device());
}

const Tensor &tensor(PyObject *o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

// A tensor of this type on this GPU.
const Tensor &tensor(PyObject *o, at::ScalarType type, c10::Device device) {
    const Tensor &t = tensor(o);
    need(t.scalar_type() == type && t.device() == device && t.layout() == at::kStrided);
    return t;
}

int32_t integer(PyObject *o) {
    need(PyLong_CheckExact(o));
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    need(overflow == 0 && v >= INT_MIN && v <= INT_MAX);
    return (int32_t)v;
}

int32_t narrow(int64_t v) {
    need(v >= 0 && v <= INT_MAX);
    return (int32_t)v;
}

int32_t dtype_code(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kHalf || t == at::kFloat);
    return t == at::kBFloat16 ? KDA_DTYPE_BF16 : t == at::kHalf ? KDA_DTYPE_FP16 : KDA_DTYPE_FP32;
}

// Both caches: their type, shape and strides.  The stride of a dimension of one
// element says nothing and may be anything; a head's channels stand for it.
void set_cache(kda_cache_config &c, int32_t &block_size, const Tensor &keys, const Tensor &values) {
    need(keys.dim() == 4 && keys.stride(3) == 1 && values.dim() == 4 && values.stride(3) == 1 &&
         values.sizes() == keys.sizes() && keys.scalar_type() != at::kFloat);
    int64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        const bool one = keys.size(i) == 1;
        need(one || values.stride(i) == keys.stride(i));
        strides[i] = one ? keys.size(3) : keys.stride(i);
    }
    c.dtype = dtype_code(keys.scalar_type());
    c.num_blocks = narrow(keys.size(0));
    block_size = narrow(keys.size(1));
    c.kv_heads = narrow(keys.size(2));
    c.head_dim = narrow(keys.size(3));
    c.stride_block = strides[0];
    c.stride_token = strides[1];
    c.stride_head = strides[2];
}

// A [T, heads, dim] activation, heads and channels packed: its token stride.
int64_t token_stride(const Tensor &t, int64_t dim) {
    need(t.dim() == 3 && t.size(2) == dim && t.stride(2) == 1 &&
         (t.stride(1) == dim || t.size(1) <= 1));
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * dim;
}

// The rows' side of a call.
int32_t set_rows(kda_align &a, int32_t block_size, const Tensor &cu, const Tensor &table,
                 const Tensor &computed, PyObject *requests, c10::Device device) {
    const int32_t rows = narrow(cu.numel() - 1);
    need(cu.is_contiguous() && table.dim() == 2 && (table.stride(1) == 1 || table.size(1) <= 1) &&
         computed.is_contiguous() && computed.numel() >= table.size(0));
    a = kda_align{};
    a.block_table = table.const_data_ptr<int32_t>();
    a.block_table_stride = table.size(0) > 1 ? table.stride(0) : table.size(1);
    a.block_table_width = narrow(table.size(1));
    a.block_size = block_size;
    a.num_requests = narrow(table.size(0));
    a.num_computed = computed.const_data_ptr<int32_t>();
    if (requests != Py_None) {
        const Tensor &r = tensor(requests, at::kInt, device);
        need(r.is_contiguous() && r.numel() >= rows);
        a.request_indices = r.const_data_ptr<int32_t>();
    } else {
        need(rows <= a.num_requests);
    }
    return rows;
}

int32_t *error_address(PyObject *o, c10::Device device) {
    if (o == Py_None) return nullptr;
    const Tensor &e = tensor(o, at::kInt, device);
    need(e.numel() >= 1);
    return e.data_ptr<int32_t>();
}

// Other threads run Python meanwhile: an allocation or a launch may wait for
// the GPU, and what runs there may wait for a host function in Python.
struct Unlocked {
    PyThreadState *const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

Tensor allocate(at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
    const Unlocked unlocked;
    return at::empty(shape, at::dtype(type).device(device));
}

// The output that was given, checked, or a new one.
Tensor output(PyObject *given, at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
    if (given == Py_None) return allocate(shape, type, device);
    const Tensor &t = tensor(given, type, device);
    need(t.sizes() == shape && t.is_contiguous());
    return t;
}

// A contiguous tensor in the memory of `all`, from its element `at` on, of a
// type of the same size: 0.1 us, where one of its own takes 0.6.
Tensor part(const Tensor &all, int64_t at, at::IntArrayRef shape, at::ScalarType type) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
}

template <typename Args>
int call(PyObject *address, const Args &args) {
    const auto function = reinterpret_cast<int (*)(const Args *)>(PyLong_AsVoidPtr(address));
    const Unlocked unlocked;
    return function(&args);
}

template <typename Body>
PyObject *guarded(Body body) {
    try {
        return body();
    } catch (...) {  // also what torch throws: api.py meets it again
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// The arguments from o[1] on: q, k, v, key_cache, value_cache, cu_seqlens,
// block_table, num_computed, inv_freq, interleaved, q_out, request_indices,
// error_word.  Answers the output that was allocated, if one was.
Tensor set_append(kda_append_args &a, PyObject *const *o) {
    const Tensor &keys = tensor(o[4]);
    const c10::Device device = keys.device();
    need_current(device);
    const at::ScalarType type = keys.scalar_type();
    const Tensor &k = tensor(o[2], type, device), &v = tensor(o[3], type, device);
    const Tensor &values = tensor(o[5], type, device);
    const Tensor &cu = tensor(o[6], at::kInt, device), &table = tensor(o[7], at::kInt, device);
    const Tensor &computed = tensor(o[8], at::kInt, device);
    kda_cache_config &c = a.config;
    int32_t block_size;
    set_cache(c, block_size, keys, values);
    a.B = set_rows(a.align, block_size, cu, table, computed, o[12], device);
    c.stride_k_t = token_stride(k, c.head_dim);
    c.stride_v_t = token_stride(v, c.head_dim);
    need(k.size(1) == c.kv_heads && v.size(1) == c.kv_heads && v.size(0) == k.size(0));
    a.num_tokens = narrow(k.size(0));
    c.q_heads = c.kv_heads;
    c.window = 1;
    c.scale = 1.0f;
    c.stride_q_t = 8;
    Tensor rotated;
    if (o[1] != Py_None) {
        const Tensor &q = tensor(o[1], type, device);
        c.stride_q_t = token_stride(q, c.head_dim);
        c.q_heads = narrow(q.size(1));
        need(q.size(0) == k.size(0) && c.kv_heads > 0 && c.q_heads > 0 &&
             c.q_heads % c.kv_heads == 0);
        rotated = output(o[11], q.sizes(), type, device);
        a.q = q.const_data_ptr();
        a.q_out = rotated.data_ptr();
    } else {
        need(o[11] == Py_None);
    }
    if (o[9] != Py_None) {
        const Tensor &f = tensor(o[9], at::kDouble, device);
        need(f.dim() == 1 && f.is_contiguous());
        c.rotary_dim = narrow(2 * f.numel());
        a.inv_freq = f.const_data_ptr<double>();
    }
    const int interleaved = PyObject_IsTrue(o[10]);
    need(interleaved >= 0);  // no truth value: it raises again in api.py
    c.interleaved = interleaved;
    a.k = k.const_data_ptr();
    a.v = v.const_data_ptr();
    a.key_cache = keys.data_ptr();
    a.value_cache = values.data_ptr();
    a.cu_seqlens = cu.const_data_ptr<int32_t>();
    a.error_word = error_address(o[13], device);
    a.stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    return rotated;
}

// One output: the one that was given, or the one that was allocated, or None.
PyObject *one_output(PyObject *given, const Tensor &made) {
    PyObject *result = PyTuple_New(1);
    if (result == nullptr) return nullptr;
    PyTuple_SET_ITEM(result, 0,
                     given != Py_None || !made.defined() ? Py_NewRef(given) : THPVariable_Wrap(made));
    return result;
}

// address, then set_append's
PyObject *append(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 14);
        kda_append_args a{};
        const Tensor rotated = set_append(a, o);
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        return one_output(o[11], rotated);
    });
}

// A norm's weight, and its type where it has one.
const void *weight_address(PyObject *o, int64_t dim, int32_t &dtype, c10::Device device) {
    if (o == Py_None) return nullptr;
    const Tensor &w = tensor(o);
    need(w.device() == device && w.dim() == 1 && w.numel() == dim && w.is_contiguous() &&
         w.layout() == at::kStrided);
    dtype = dtype_code(w.scalar_type());
    return w.const_data_ptr();
}

// address, set_append's, q_weight, k_weight, eps
PyObject *norm_append(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 17);
        kda_norm_append_args a{};
        const Tensor rotated = set_append(a.append, o);
        const c10::Device device = tensor(o[4]).device();
        int32_t types[2] = {-1, -1};
        a.q_weight = weight_address(o[14], a.append.config.head_dim, types[0], device);
        a.k_weight = weight_address(o[15], a.append.config.head_dim, types[1], device);
        need(types[0] < 0 || types[1] < 0 || types[0] == types[1]);
        a.weight_dtype = std::max(types[0], types[1]);
        if (a.weight_dtype < 0) a.weight_dtype = KDA_DTYPE_FP32;
        need(a.weight_dtype == KDA_DTYPE_FP32 || a.weight_dtype == a.append.config.dtype);
        need(PyFloat_CheckExact(o[16]));
        a.eps = (float)PyFloat_AS_DOUBLE(o[16]);
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        return one_output(o[11], rotated);
    });
}

// A [T, H, 128] activation, heads and channels packed: its token stride.
int64_t delta_stride(const Tensor &t, int64_t tokens, int64_t heads) {
    need(t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads);
    return token_stride(t, KDA_HEAD_DIM);
}

// address, q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool, cu_seqlens
// (None: one token a row), state_indices, lower_bound, scale,
// initial_indices, out, error_word
PyObject *delta(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 16);
        const Tensor &pool = tensor(o[8]);
        const c10::Device device = pool.device();
        need_current(device);
        need(pool.scalar_type() == at::kFloat && pool.dim() == 4 && pool.is_contiguous() &&
             pool.size(2) == KDA_HEAD_DIM && pool.size(3) == KDA_HEAD_DIM);
        const int64_t heads = pool.size(1);
        const Tensor &q = tensor(o[1], at::kBFloat16, device);
        const Tensor &k = tensor(o[2], at::kBFloat16, device);
        const Tensor &v = tensor(o[3], at::kBFloat16, device);
        const Tensor &g = tensor(o[4], at::kBFloat16, device);
        const Tensor &beta = tensor(o[5], at::kBFloat16, device);
        const Tensor &a_log = tensor(o[6], at::kFloat, device);
        const Tensor &bias = tensor(o[7], at::kFloat, device);
        const Tensor &slots = tensor(o[10], at::kInt, device);
        need(a_log.is_contiguous() && a_log.numel() >= heads && bias.is_contiguous() &&
             bias.numel() >= heads * KDA_HEAD_DIM && slots.dim() == 1 && slots.is_contiguous());
        need(q.dim() == 3 && q.size(0) > 0 && heads > 0);
        kda_delta_args a{};
        kda_config &c = a.config;
        const int64_t tokens = q.size(0);
        c.num_heads = narrow(heads);
        c.head_dim = KDA_HEAD_DIM;
        c.window = 1;
        c.num_slots = narrow(pool.size(0));
        c.stride_q_t = delta_stride(q, tokens, heads);
        c.stride_k_t = delta_stride(k, tokens, heads);
        c.stride_v_t = delta_stride(v, tokens, heads);
        c.stride_g_t = delta_stride(g, tokens, heads);
        need(beta.dim() == 2 && beta.size(0) == tokens && beta.size(1) == heads &&
             (beta.stride(1) == 1 || heads == 1));
        c.stride_beta_t = tokens > 1 ? beta.stride(0) : heads;
        a.B = narrow(slots.size(0));
        a.num_tokens = narrow(tokens);
        if (o[9] != Py_None) {
            const Tensor &cu = tensor(o[9], at::kInt, device);
            need(cu.dim() == 1 && cu.is_contiguous() && cu.numel() == (int64_t)a.B + 1);
            a.cu_seqlens = cu.const_data_ptr<int32_t>();
        } else {
            need(tokens == a.B);
        }
        if (o[11] != Py_None) {
            need(PyFloat_CheckExact(o[11]));
            c.use_lower_bound = 1;
            c.lower_bound = (float)PyFloat_AS_DOUBLE(o[11]);
        }
        need(o[12] == Py_None || PyFloat_CheckExact(o[12]));
        c.scale = (float)(o[12] == Py_None ? 1.0 / std::sqrt((double)KDA_HEAD_DIM)
                                           : PyFloat_AS_DOUBLE(o[12]));
        if (o[13] != Py_None) {
            const Tensor &from = tensor(o[13], at::kInt, device);
            need(from.dim() == 1 && from.is_contiguous() && from.numel() == a.B);
            a.initial_indices = from.const_data_ptr<int32_t>();
        }
        const Tensor out = output(o[14], q.sizes(), at::kBFloat16, device);
        a.q = q.const_data_ptr();
        a.k = k.const_data_ptr();
        a.v = v.const_data_ptr();
        a.g_raw = g.const_data_ptr();
        a.beta_raw = beta.const_data_ptr();
        a.A_log = a_log.const_data_ptr<float>();
        a.g_bias = bias.const_data_ptr<float>();
        a.state_pool = pool.data_ptr<float>();
        a.state_indices = slots.const_data_ptr<int32_t>();
        a.out = out.data_ptr();
        a.error_word = error_address(o[15], device);
        a.stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        return one_output(o[14], out);
    });
}

// address, q, key_cache, value_cache, cu_seqlens, block_table, num_computed,
// workspace, window, scale, left_window, request_indices, out, lse, error_word
PyObject *attend(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 15);
        const Tensor &keys = tensor(o[2]);
        const c10::Device device = keys.device();
        need_current(device);
        const at::ScalarType type = keys.scalar_type();
        const Tensor &q = tensor(o[1], type, device), &values = tensor(o[3], type, device);
        const Tensor &cu = tensor(o[4], at::kInt, device), &table = tensor(o[5], at::kInt, device);
        const Tensor &computed = tensor(o[6], at::kInt, device);
        const Tensor &work = tensor(o[7], at::kByte, device);
        kda_attention_args a{};
        kda_cache_config &c = a.config;
        int32_t block_size;
        set_cache(c, block_size, keys, values);
        a.B = set_rows(a.align, block_size, cu, table, computed, o[11], device);
        c.stride_q_t = token_stride(q, c.head_dim);
        c.stride_k_t = c.stride_v_t = 8;
        c.q_heads = narrow(q.size(1));
        need(c.kv_heads > 0 && c.q_heads > 0 && c.q_heads % c.kv_heads == 0 && q.size(0) > 0 &&
             work.is_contiguous());
        a.num_tokens = narrow(q.size(0));
        c.window = o[8] != Py_None
                       ? integer(o[8])
                       : std::min(KDA_MAX_WINDOW,
                                  std::max(1, KDA_MAX_QUERY_ROWS / (c.q_heads / c.kv_heads)));
        c.left_window = integer(o[10]);
        need(o[9] == Py_None || PyFloat_CheckExact(o[9]));
        c.scale = (float)(o[9] == Py_None ? 1.0 / std::sqrt((double)c.head_dim)
                                          : PyFloat_AS_DOUBLE(o[9]));
        const Tensor out = output(o[12], q.sizes(), type, device);
        const Tensor lse = output(o[13], {q.size(0), q.size(1)}, at::kFloat, device);
        a.q = q.const_data_ptr();
        a.key_cache = keys.const_data_ptr();
        a.value_cache = values.const_data_ptr();
        a.cu_seqlens = cu.const_data_ptr<int32_t>();
        a.workspace = work.data_ptr();
        a.workspace_bytes = (uint64_t)work.numel();
        a.out = out.data_ptr();
        a.lse = lse.data_ptr<float>();
        a.error_word = error_address(o[14], device);
        a.stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        PyObject *result = PyTuple_New(2);
        if (result == nullptr) return nullptr;
        PyTuple_SET_ITEM(result, 0, o[12] != Py_None ? Py_NewRef(o[12]) : THPVariable_Wrap(out));
        PyTuple_SET_ITEM(result, 1, o[13] != Py_None ? Py_NewRef(o[13]) : THPVariable_Wrap(lse));
        return result;
    });
}

// address, logits, tokens, num_top, error_word
PyObject *logprobs(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 5);
        const Tensor &x = tensor(o[1]);
        const c10::Device device = x.device();
        need_current(device);
        need(x.dim() == 2 && (x.stride(1) == 1 || x.size(1) <= 1) &&
             x.layout() == at::kStrided);
        const Tensor &tokens = tensor(o[2], at::kInt, device);
        need(tokens.dim() == 1 && tokens.numel() == x.size(0) && tokens.is_contiguous());
        kda_logprobs_args a{};
        a.dtype = dtype_code(x.scalar_type());
        a.rows = narrow(x.size(0));
        a.vocab = narrow(x.size(1));
        a.num_top = integer(o[3]);
        need(a.num_top >= 0 && a.num_top <= KDA_MAX_TOP);
        const int64_t rows = a.rows, top = a.num_top;
        const Tensor all = allocate({rows * (3 + 2 * top)}, at::kFloat, device);
        const Tensor outputs[5] = {part(all, 0, {rows}, at::kFloat),
                                   part(all, rows, {rows}, at::kFloat),
                                   part(all, 2 * rows, {rows}, at::kFloat),
                                   part(all, 3 * rows, {rows, top}, at::kFloat),
                                   part(all, (3 + top) * rows, {rows, top}, at::kInt)};
        a.logits = x.const_data_ptr();
        a.stride_row = x.stride(0);
        a.tokens = tokens.const_data_ptr<int32_t>();
        a.logprob = outputs[0].data_ptr<float>();
        a.entropy = outputs[1].data_ptr<float>();
        a.lse_out = outputs[2].data_ptr<float>();
        a.top_logprob = outputs[3].data_ptr<float>();
        a.top_index = outputs[4].data_ptr<int32_t>();
        a.error_word = error_address(o[4], device);
        a.stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        if (const int status = call(o[0], a)) return PyLong_FromLong(status);
        PyObject *result = PyTuple_New(5);
        if (result == nullptr) return nullptr;
        for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(result, i, THPVariable_Wrap(outputs[i]));
        return result;
    });
}

template <PyObject *(*kFunction)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kFunction)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<append>("append"), method<attend>("attend"),
                         method<logprobs>("logprobs"), method<norm_append>("norm_append"),
                         method<delta>("delta"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What this was built for: api.py uses it only where its own structures have the
// same sizes and PyTorch, whose tensors are laid out in here, is the same.
PyMODINIT_FUNC PyInit__binding() {
    PyObject *m = PyModule_Create(&module);
    if (m == nullptr) return nullptr;
    PyObject *sizes = Py_BuildValue("(nnn)", (Py_ssize_t)sizeof(kda_append_args),
                                    (Py_ssize_t)sizeof(kda_attention_args),
                                    (Py_ssize_t)sizeof(kda_logprobs_args));
    PyObject *more = Py_BuildValue("(nn)", (Py_ssize_t)sizeof(kda_norm_append_args),
                                   (Py_ssize_t)sizeof(kda_delta_args));
    if (sizes == nullptr || more == nullptr ||
        PyModule_AddObject(m, "argument_sizes", sizes) != 0 ||
        PyModule_AddObject(m, "more_argument_sizes", more) != 0 ||
        PyModule_AddStringConstant(m, "torch_version", KDA_TORCH_VERSION) != 0) {
        Py_XDECREF(m);
        return nullptr;
    }
    return m;
}
