// Python entries of the decoder-block operators: argument checks, output
// allocation and the call into the C ABI without an interpreter step in between.
// The operators run for a few microseconds on small batches; checked and
// marshalled in Python their calls took 12 to 18 us of host time on a Grace core.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_gb300.h"

namespace {

PyObject* g_moe_error = nullptr;  // the package's MoeError

using at::Tensor;

// Python-side failures of a call; the entry returns null.
struct Failed {};

[[noreturn]] void fail(const char* what) {
    PyErr_SetString(PyExc_ValueError, what);
    throw Failed();
}
[[noreturn]] void failf(const char* format, const char* name) {
    PyErr_Format(PyExc_ValueError, format, name);
    throw Failed();
}
void check(moe_status s, const char* what) {
    if (s == MOE_OK) return;
    PyObject* e = PyObject_CallFunction(g_moe_error, "is", (int)s, what);
    if (e) {
        PyErr_SetObject(g_moe_error, e);
        Py_DECREF(e);
    }
    throw Failed();
}

// like: a tensor of the call, whose device all share
const Tensor& tensor(PyObject* o, const char* name, const Tensor* like = nullptr) {
    if (!THPVariable_Check(o)) failf("%s must be a CUDA tensor", name);
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) failf("%s must be a CUDA tensor", name);
    if (like && t.get_device() != like->get_device()) failf("%s is on another device", name);
    return t;
}
// None: undefined
Tensor optional(PyObject* o, const char* name, const Tensor& like) {
    return o == Py_None ? Tensor() : tensor(o, name, &like);
}
long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed();
    return v;
}
int small(PyObject* o) {
    const long long v = integer(o);
    return v < INT_MIN ? INT_MIN : v > INT_MAX ? INT_MAX : (int)v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Failed();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Failed();
    return v != 0;
}
// The stream of a call: the given one, current while the entry runs so that what it
// allocates and drops stays in that stream's order, or the current one of the device.
struct OnStream {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard given;
    void* handle;
    OnStream(PyObject* o, const Tensor& t) : device(t.device()) {
        if (o == Py_None) {
            handle = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
        } else {
            handle = PyLong_AsVoidPtr(o);
            if (!handle && PyErr_Occurred()) throw Failed();
            given.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), t.get_device()));
        }
    }
};
int dtype_of(const Tensor& t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return MOE_BF16;
        case at::kHalf: return MOE_FP16;
        case at::kFloat: return MOE_FP32;
        case at::kByte: return MOE_E4M3;
        default: return -1;
    }
}
Tensor empty(at::IntArrayRef size, at::ScalarType type, const Tensor& like) {
    return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}
const void* vector_ptr(const Tensor& t, int64_t n, at::ScalarType type, const char* what) {
    if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1)) fail(what);
    return t.data_ptr();
}
uint32_t* status_ptr(PyObject* o, const Tensor& like) {
    const Tensor t = optional(o, "status", like);
    if (!t.defined()) return nullptr;
    if (t.scalar_type() != at::kByte || !t.is_contiguous() || t.numel() < 4)
        fail("status must be a device error word (new_status)");
    return static_cast<uint32_t*>(t.data_ptr());
}

// Checked cache tensors [pages, heads, page, D].
moe_kv_cache cache_of(PyObject* k_o, PyObject* v_o, PyObject* ks_o, PyObject* vs_o) {
    if (!THPVariable_Check(k_o) || !THPVariable_Check(v_o)) fail("k_cache and v_cache must be CUDA tensors");
    const Tensor &k = THPVariable_Unpack(k_o), &v = THPVariable_Unpack(v_o);
    if (!k.is_cuda() || !v.is_cuda()) fail("k_cache and v_cache must be CUDA tensors");
    if (k.get_device() != v.get_device()) fail("k_cache and v_cache are on different devices");
    moe_kv_cache c = {};
    c.dtype = dtype_of(k);
    if (c.dtype < 0 || c.dtype == MOE_FP32 || v.scalar_type() != k.scalar_type())
        fail("k_cache and v_cache must both be bf16, fp16 or uint8 (e4m3 codes)");
    if (k.dim() != 4 || v.sizes() != k.sizes()) fail("k_cache and v_cache must both be [pages, heads, page, D]");
    if (k.stride(3) != 1 || v.stride(3) != 1) fail("the last dim of k_cache and v_cache must be contiguous");
    if (k.size(0) > INT_MAX || k.size(1) > INT_MAX || k.size(2) > INT_MAX || k.size(3) > INT_MAX)
        fail("k_cache and v_cache are too large");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    const Tensor ks = optional(ks_o, "k_scale", k), vs = optional(vs_o, "v_scale", k);
    if (c.dtype == MOE_E4M3) {
        if (!ks.defined() || !vs.defined() || ks.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat)
            fail("an e4m3 cache needs k_scale and v_scale, fp32 CUDA tensors");
        if (ks.sizes() != k.sizes().slice(0, 3) || vs.sizes() != ks.sizes() || vs.strides() != ks.strides())
            fail("k_scale and v_scale must be [pages, heads, page] with equal strides");
        c.k_scale = static_cast<float*>(ks.data_ptr());
        c.v_scale = static_cast<float*>(vs.data_ptr());
        for (int i = 0; i < 3; ++i) c.scale_stride[i] = ks.stride(i);
    } else if (ks.defined() || vs.defined()) {
        fail("scales belong to an e4m3 cache (uint8)");
    }
    for (int i = 0; i < 3; ++i) c.k_stride[i] = k.stride(i), c.v_stride[i] = v.stride(i);
    c.num_pages = (int)k.size(0);
    c.kv_heads = (int)k.size(1);
    c.page_size = (int)k.size(2);
    c.head_dim = (int)k.size(3);
    return c;
}

// route_experts(logits, top_k, score, bias, groups, top_groups, group_top, renormalize, scale, stream)
PyObject* route_experts(PyObject* const* a) {
    const Tensor& logits = tensor(a[0], "logits");
    const int dt = dtype_of(logits);
    if (dt < 0 || dt == MOE_E4M3) fail("logits must be bf16, fp16 or fp32");
    if (logits.dim() != 2 || (logits.size(1) > 1 && logits.stride(1) != 1))
        fail("logits must be [T, E] with contiguous rows");
    const int64_t T = logits.size(0), E = logits.size(1);
    if (T > INT_MAX || E > INT_MAX) fail("logits are too large");
    moe_gate g;
    g.score = small(a[2]);
    if (g.score < 0) fail("score must be one of softmax, sigmoid");
    const Tensor bias = optional(a[3], "bias", logits);
    if (bias.defined() &&
        (bias.scalar_type() != at::kFloat || bias.dim() != 1 || bias.size(0) != E || !bias.is_contiguous()))
        fail("bias must be a contiguous fp32 tensor [E]");
    g.bias = bias.defined() ? static_cast<const float*>(bias.data_ptr()) : nullptr;
    g.groups = small(a[4]);
    g.top_groups = small(a[5]);
    g.group_top = small(a[6]);
    g.renormalize = truth(a[7]);
    g.scale = (float)real(a[8]);
    const int k = small(a[1]);
    if (k < 1) check(MOE_ERR_INVALID_ARG, "moe_route_experts");
    const OnStream on(a[9], logits);
    const Tensor idx = empty({T, k}, at::kInt, logits), w = empty({T, k}, at::kFloat, logits);
    if (T)
        check(moe_route_experts(&g, logits.data_ptr(), dt, T > 1 ? logits.stride(0) : E, (int)T, (int)E, k,
                                static_cast<int32_t*>(idx.data_ptr()), static_cast<float*>(w.data_ptr()),
                                on.handle),
              "moe_route_experts");
    PyObject* r = PyTuple_New(2);
    if (!r) throw Failed();
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(idx));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(w));
    return r;
}

// rotate_append(q, k, v, positions, slots, k_cache, v_cache, inv_freq, k_scale, v_scale, interleaved, rope_scale,
//               q_out, status, stream, axes)
PyObject* rotate_append(PyObject* const* a) {
    const moe_kv_cache c = cache_of(a[5], a[6], a[8], a[9]);
    const Tensor& cache = THPVariable_Unpack(a[5]);
    const Tensor &q = tensor(a[0], "q", &cache), &k = tensor(a[1], "k", &q), &v = tensor(a[2], "v", &q);
    const int dt = dtype_of(q);
    if ((dt != MOE_BF16 && dt != MOE_FP16) || k.scalar_type() != q.scalar_type() ||
        v.scalar_type() != q.scalar_type() || (c.dtype != MOE_E4M3 && c.dtype != dt))
        fail("q, k and v must be bf16 or fp16 alike, and a 16-bit cache of their type");
    if (q.dim() != 3 || q.size(2) != c.head_dim || k.dim() != 3 || k.size(0) != q.size(0) || k.size(1) != c.kv_heads ||
        k.size(2) != c.head_dim || v.sizes() != k.sizes())
        fail("q must be [N, Hq, D], k and v [N, Hkv, D] with the cache's Hkv and D");
    const int64_t N = q.size(0), Hq = q.size(1);
    if (N > INT_MAX || Hq > INT_MAX) fail("q is too large");
    const Tensor& inv_freq = tensor(a[7], "inv_freq", &q);
    if (inv_freq.scalar_type() != at::kDouble || !inv_freq.is_contiguous() || inv_freq.numel() > 4096)
        fail("inv_freq must be a contiguous fp64 CUDA tensor [R / 2]");
    const Tensor& position = tensor(a[3], "positions", &q);
    const Tensor axes = optional(a[15], "axes", q);
    const void* pos = nullptr;
    if (axes.defined()) {
        if (position.scalar_type() != at::kLong || position.dim() != 2 || position.size(0) < 1 ||
            position.size(0) > 16 || position.size(1) != N || (N > 1 && position.stride(1) != 1))
            fail("positions must be an int64 CUDA tensor [axes, N] of 1 to 16 contiguous rows");
        vector_ptr(axes, inv_freq.numel(), at::kInt, "axes must be a contiguous int32 CUDA tensor [R / 2]");
        pos = position.data_ptr();
    } else {
        pos = vector_ptr(position, N, at::kLong, "positions must be a contiguous int64 CUDA tensor [N]");
    }
    const void* slots =
        vector_ptr(tensor(a[4], "slots", &q), N, at::kLong, "slots must be a contiguous int64 CUDA tensor [N]");
    const OnStream on(a[14], q);
    Tensor out = optional(a[12], "q_out", q);
    if (!out.defined())
        out = empty(q.sizes(), q.scalar_type(), q);
    else if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
        fail("q_out must be like q");
    if (q.stride(2) != 1 || k.stride(2) != 1 || v.stride(2) != 1 || out.stride(2) != 1)
        fail("the last dim of q, k, v and q_out must be contiguous");
    const int rot = 2 * (int)inv_freq.numel(), neighbours = truth(a[10]);
    const float rope_scale = (float)real(a[11]);
    const int64_t *at = static_cast<const int64_t*>(pos), *to = static_cast<const int64_t*>(slots);
    const double* freq = static_cast<const double*>(inv_freq.data_ptr());
    uint32_t* status = status_ptr(a[13], q);
    if (N && axes.defined())
        check(moe_rotate_append_axes(&c, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, q.stride(0), q.stride(1),
                                     k.stride(0), k.stride(1), v.stride(0), v.stride(1), at, (int)position.size(0),
                                     position.stride(0), static_cast<const int32_t*>(axes.data_ptr()), to, freq, rot,
                                     neighbours, rope_scale, (int)N, (int)Hq, out.data_ptr(), out.stride(0),
                                     out.stride(1), status, on.handle),
              "moe_rotate_append_axes");
    else if (N)
        check(moe_rotate_append(&c, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, q.stride(0), q.stride(1), k.stride(0),
                                k.stride(1), v.stride(0), v.stride(1), at, to, freq, rot, neighbours, rope_scale, (int)N,
                                (int)Hq, out.data_ptr(), out.stride(0), out.stride(1), status, on.handle),
              "moe_rotate_append");
    return THPVariable_Wrap(out);
}

// paged_attention(q, k_cache, v_cache, page_table, lengths, scale, k_scale, v_scale, sinks, window, out, workspace,
//                 status, stream)
PyObject* paged_attention(PyObject* const* a) {
    const moe_kv_cache c = cache_of(a[1], a[2], a[6], a[7]);
    if (!THPVariable_Check(a[0]) || !THPVariable_Unpack(a[0]).is_cuda())
        fail("q must be a bf16 or fp16 CUDA tensor, and a 16-bit cache of its type");
    const Tensor& q = tensor(a[0], "q", &THPVariable_Unpack(a[1]));
    const int dt = dtype_of(q);
    if ((dt != MOE_BF16 && dt != MOE_FP16) || (c.dtype != MOE_E4M3 && c.dtype != dt))
        fail("q must be a bf16 or fp16 CUDA tensor, and a 16-bit cache of its type");
    if (q.dim() != 3 || q.size(2) != c.head_dim || q.stride(2) != 1)
        fail("q must be [B, Hq, D] with the cache's D and a contiguous last dim");
    const int64_t B = q.size(0), Hq = q.size(1);
    if (B > INT_MAX || Hq > INT_MAX) fail("q is too large");
    const Tensor& table = tensor(a[3], "page_table", &q);
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B || table.size(1) > INT_MAX ||
        (table.size(1) > 1 && table.stride(1) != 1))
        fail("page_table must be an int32 CUDA tensor [B, pages] with contiguous rows");
    const void* lengths =
        vector_ptr(tensor(a[4], "lengths", &q), B, at::kInt, "lengths must be a contiguous int32 CUDA tensor [B]");
    const Tensor sinks = optional(a[8], "sinks", q);
    if (sinks.defined() &&
        (sinks.scalar_type() != at::kFloat || sinks.dim() != 1 || sinks.size(0) != Hq || !sinks.is_contiguous()))
        fail("sinks must be a contiguous fp32 tensor [Hq]");
    const int window = small(a[9]);
    const OnStream on(a[13], q);
    Tensor out = optional(a[10], "out", q);
    if (!out.defined())
        out = empty(q.sizes(), q.scalar_type(), q);
    else if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type() || out.stride(2) != 1)
        fail("out must be like q, its last dim contiguous");
    if (B == 0) return THPVariable_Wrap(out);
    Tensor ws = optional(a[11], "workspace", q);
    if (ws.defined()) {
        if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) fail("workspace must be a contiguous uint8 tensor");
    } else {
        const long long most = table.size(1) * c.page_size;
        const size_t bytes = moe_attention_workspace_size(
            (int)B, (int)Hq, c.kv_heads, c.head_dim, c.dtype,
            (int)(window > 0 && window < most ? window : most < INT_MAX ? most : INT_MAX));
        if (bytes > 256) ws = empty({(int64_t)bytes}, at::kByte, q);
    }
    check(moe_paged_attention(&c, q.data_ptr(), dt, q.stride(0), q.stride(1),
                              static_cast<const int32_t*>(table.data_ptr()), table.stride(0), (int)table.size(1),
                              static_cast<const int32_t*>(lengths), (int)B, (int)Hq, (float)real(a[5]),
                              sinks.defined() ? static_cast<const float*>(sinks.data_ptr()) : nullptr, window,
                              out.data_ptr(), out.stride(0), out.stride(1), ws.defined() ? ws.data_ptr() : nullptr,
                              ws.defined() ? (size_t)ws.numel() : 0, status_ptr(a[12], q), on.handle),
          "moe_paged_attention");
    return THPVariable_Wrap(out);
}

const int32_t* ints(const Tensor& t, int64_t n, const char* what) {
    return static_cast<const int32_t*>(vector_ptr(t, n, at::kInt, what));
}
const Tensor& int_rows(PyObject* o, int64_t B, const char* name, const char* what, const Tensor& like) {
    const Tensor& t = tensor(o, name, &like);
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != B || t.size(1) > INT_MAX ||
        (t.size(1) > 1 && t.stride(1) != 1))
        fail(what);
    return t;
}

// tree_attention(q, k_cache, v_cache, page_table, lengths, starts, scale, parents, k_scale, v_scale, sinks, window,
//                out, workspace, status, stream)
PyObject* tree_attention(PyObject* const* a) {
    const moe_kv_cache c = cache_of(a[1], a[2], a[8], a[9]);
    const Tensor& q = tensor(a[0], "q", &THPVariable_Unpack(a[1]));
    const int dt = dtype_of(q);
    if ((dt != MOE_BF16 && dt != MOE_FP16) || (c.dtype != MOE_E4M3 && c.dtype != dt))
        fail("q must be a bf16 or fp16 CUDA tensor, and a 16-bit cache of its type");
    if (q.dim() != 3 || q.size(2) != c.head_dim || q.stride(2) != 1)
        fail("q must be [N, Hq, D] with the cache's D and a contiguous last dim");
    const int64_t N = q.size(0), Hq = q.size(1);
    if (N > INT_MAX || Hq > INT_MAX) fail("q is too large");
    const Tensor& lengths = tensor(a[4], "lengths", &q);
    const int64_t B = lengths.dim() == 1 ? lengths.size(0) : -1;
    if (B > INT_MAX) fail("lengths is too large");
    const int32_t* lens = ints(lengths, B, "lengths must be a contiguous int32 CUDA tensor [B]");
    const int32_t* starts = ints(tensor(a[5], "starts", &q), B + 1, "starts must be a contiguous int32 CUDA tensor [B + 1]");
    const Tensor& table =
        int_rows(a[3], B, "page_table", "page_table must be an int32 CUDA tensor [B, pages] with contiguous rows", q);
    const Tensor parents = optional(a[7], "parents", q);
    const int32_t* up = parents.defined() ? ints(parents, N, "parents must be a contiguous int32 CUDA tensor [N]") : nullptr;
    const Tensor sinks = optional(a[10], "sinks", q);
    if (sinks.defined() &&
        (sinks.scalar_type() != at::kFloat || sinks.dim() != 1 || sinks.size(0) != Hq || !sinks.is_contiguous()))
        fail("sinks must be a contiguous fp32 tensor [Hq]");
    const int window = small(a[11]);
    const float scale = (float)real(a[6]);
    const OnStream on(a[15], q);
    uint32_t* status = status_ptr(a[14], q);
    Tensor out = optional(a[12], "out", q);
    if (!out.defined())
        out = empty(q.sizes(), q.scalar_type(), q);
    else if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type() || out.stride(2) != 1)
        fail("out must be like q, its last dim contiguous");
    if (N == 0 || B == 0) return THPVariable_Wrap(out);
    Tensor ws = optional(a[13], "workspace", q);
    if (ws.defined()) {
        if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) fail("workspace must be a contiguous uint8 tensor");
    } else {
        const long long most = table.size(1) * c.page_size;
        const size_t bytes = moe_tree_attention_workspace_size(
            (int)N, (int)B, (int)Hq, c.kv_heads, c.head_dim, c.dtype,
            (int)(window > 0 && window < most ? window : most < INT_MAX ? most : INT_MAX));
        if (bytes > 256) ws = empty({(int64_t)bytes}, at::kByte, q);
    }
    check(moe_tree_attention(&c, q.data_ptr(), dt, q.stride(0), q.stride(1), static_cast<const int32_t*>(table.data_ptr()),
                             table.stride(0), (int)table.size(1), lens, starts, up, (int)N, (int)B, (int)Hq, scale,
                             sinks.defined() ? static_cast<const float*>(sinks.data_ptr()) : nullptr, window,
                             out.data_ptr(), out.stride(0), out.stride(1), ws.defined() ? ws.data_ptr() : nullptr,
                             ws.defined() ? (size_t)ws.numel() : 0, status, on.handle),
          "moe_tree_attention");
    return THPVariable_Wrap(out);
}

// Checked cache tensors of several layers, [layers, pages, heads, page, D] or without the first dim:
// layer 0 as a cache, the number of layers, the strides from layer to layer of k, v and scales.
struct Layers {
    moe_kv_cache cache;
    int layers = 1;
    int64_t stride[3] = {0, 0, 0};
};
Layers layers_of(PyObject* k_o, PyObject* v_o, PyObject* ks_o, PyObject* vs_o) {
    Layers r;
    if (!THPVariable_Check(k_o) || THPVariable_Unpack(k_o).dim() != 5) {
        r.cache = cache_of(k_o, v_o, ks_o, vs_o);
        return r;
    }
    PyObject* all[4] = {k_o, v_o, ks_o, vs_o};
    struct Owned {
        PyObject* o = nullptr;
        ~Owned() { Py_XDECREF(o); }
    } first[4];
    const int64_t n = THPVariable_Unpack(k_o).size(0);
    if (n < 1 || n > INT_MAX) fail("k_cache and v_cache need at least one layer");
    for (int i = 0; i < 4; ++i) {
        if (!THPVariable_Check(all[i])) {  // None, or what cache_of refuses
            Py_INCREF(all[i]);
            first[i].o = all[i];
            continue;
        }
        const Tensor& t = THPVariable_Unpack(all[i]);
        if (t.dim() != (i < 2 ? 5 : 4) || t.size(0) != n)
            fail("k_cache and v_cache must both be [layers, pages, heads, page, D], scales [layers, pages, heads, page]");
        if (n > 1) {
            if (i == 3 && t.stride(0) != r.stride[2]) fail("k_scale and v_scale must have equal strides");
            r.stride[i < 2 ? i : 2] = t.stride(0);
        }
        first[i].o = THPVariable_Wrap(t.select(0, 0));
        if (!first[i].o) throw Failed();
    }
    r.cache = cache_of(first[0].o, first[1].o, first[2].o, first[3].o);
    r.layers = (int)n;
    return r;
}

// copy_pages(k_cache, v_cache, src, dst, tokens, k_scale, v_scale, status, stream)
PyObject* copy_pages(PyObject* const* a) {
    const Layers c = layers_of(a[0], a[1], a[5], a[6]);
    const Tensor& k = THPVariable_Unpack(a[0]);
    const Tensor& src = tensor(a[2], "src", &k);
    const int64_t N = src.dim() == 1 ? src.size(0) : -1;
    if (N > INT_MAX) fail("src is too large");
    const int32_t* s = ints(src, N, "src must be a contiguous int32 CUDA tensor [N]");
    const int32_t* d = ints(tensor(a[3], "dst", &k), N, "dst must be a contiguous int32 CUDA tensor [N]");
    const Tensor tokens = optional(a[4], "tokens", k);
    const int32_t* t = tokens.defined() ? ints(tokens, N, "tokens must be a contiguous int32 CUDA tensor [N]") : nullptr;
    const OnStream on(a[8], k);
    uint32_t* status = status_ptr(a[7], k);
    if (N) check(moe_copy_pages(&c.cache, c.layers, c.stride, s, d, t, (int)N, status, on.handle), "moe_copy_pages");
    Py_RETURN_NONE;
}

// compact_drafts(k_cache, v_cache, page_table, lengths, starts, kept, k_scale, v_scale, out, status, stream)
PyObject* compact_drafts(PyObject* const* a) {
    const Layers c = layers_of(a[0], a[1], a[6], a[7]);
    const Tensor& k = THPVariable_Unpack(a[0]);
    const Tensor& lengths = tensor(a[3], "lengths", &k);
    const int64_t B = lengths.dim() == 1 ? lengths.size(0) : -1;
    if (B > INT_MAX) fail("lengths is too large");
    const int32_t* lens = ints(lengths, B, "lengths must be a contiguous int32 CUDA tensor [B]");
    const int32_t* starts = ints(tensor(a[4], "starts", &k), B + 1, "starts must be a contiguous int32 CUDA tensor [B + 1]");
    const Tensor& table =
        int_rows(a[2], B, "page_table", "page_table must be an int32 CUDA tensor [B, pages] with contiguous rows", k);
    const Tensor& kept = int_rows(a[5], B, "kept", "kept must be an int32 CUDA tensor [B, K] with contiguous rows", k);
    const OnStream on(a[10], k);
    Tensor out = optional(a[8], "out", k);
    if (!out.defined())
        out = empty({B}, at::kInt, k);
    else if (ints(out, B, "out must be a contiguous int32 CUDA tensor [B]") == lens && B)
        fail("out cannot be lengths itself");
    uint32_t* status = status_ptr(a[9], k);
    if (B)
        check(moe_compact_drafts(&c.cache, c.layers, c.stride, static_cast<const int32_t*>(table.data_ptr()),
                                 table.stride(0), (int)table.size(1), lens, starts,
                                 kept.size(1) ? static_cast<const int32_t*>(kept.data_ptr()) : nullptr, kept.stride(0), (int)B,
                                 (int)kept.size(1), static_cast<int32_t*>(out.data_ptr()), status, on.handle),
              "moe_compact_drafts");
    return THPVariable_Wrap(out);
}

// No C++ exception leaves an entry: failures of ours have set the Python error,
// torch's (out of memory among them) become its Python errors.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Failed&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_moe_error);
    g_moe_error = type;
    Py_RETURN_NONE;
}

PyCFunction method(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef g_methods[] = {
    {"route_experts", method(entry<route_experts, 10>), METH_FASTCALL, nullptr},
    {"rotate_append", method(entry<rotate_append, 16>), METH_FASTCALL, nullptr},
    {"paged_attention", method(entry<paged_attention, 14>), METH_FASTCALL, nullptr},
    {"tree_attention", method(entry<tree_attention, 16>), METH_FASTCALL, nullptr},
    {"copy_pages", method(entry<copy_pages, 9>), METH_FASTCALL, nullptr},
    {"compact_drafts", method(entry<compact_drafts, 11>), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
