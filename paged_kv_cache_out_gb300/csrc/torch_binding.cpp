// torch_binding.cpp -- the checks and the marshalling of the calls that a decode
// step makes for every layer, compiled: a call of a few microseconds of GPU work
// would otherwise wait for the interpreter.  Nothing is computed here.
//
// Each function checks its tensors (ValueError on a wrong one), calls the C entry
// point and returns its pkv_status; the Python wrappers allocate what the caller
// left out and raise on a status.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "pkv.h"

namespace {

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

constexpr const char *kHere = " on the current CUDA device";

// The arguments of one call, taken in order.
struct Arguments {
    PyObject *const *at;
    int64_t device;

    bool none() const { return *at == Py_None; }
    void skip() { ++at; }

    const at::Tensor &tensor(const char *name, at::ScalarType type, const char *type_name) {
        PyObject *o = *at++;
        if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != device)
            throw Refused(std::string(name) + " must be a " + type_name + " tensor" + kHere);
        return t;
    }
    const at::Tensor &dense(const char *name, at::ScalarType type, const char *type_name, int64_t dims) {
        const at::Tensor &t = tensor(name, type, type_name);
        if (t.dim() != dims || !t.is_contiguous())
            throw Refused(std::string(name) + " must be contiguous, with " + std::to_string(dims) + " dimensions");
        return t;
    }
    const at::Tensor &bf16(const char *name, int64_t dims) { return dense(name, at::kBFloat16, "bfloat16", dims); }
    const at::Tensor &f32(const char *name, int64_t dims) { return dense(name, at::kFloat, "float32", dims); }
    const at::Tensor &i32(const char *name, int64_t dims) { return dense(name, at::kInt, "int32", dims); }
    // int32 [n], nullptr for None
    const int32_t *ints(const char *name, int64_t n, bool optional) {
        if (optional && none()) return skip(), nullptr;
        const at::Tensor &t = i32(name, 1);
        if (t.size(0) != n) throw Refused(std::string(name) + " must have " + std::to_string(n) + " elements");
        return t.const_data_ptr<int32_t>();
    }
    int32_t *status() {
        if (none()) return skip(), nullptr;
        const at::Tensor &t = tensor("dev_status", at::kInt, "int32");
        if (t.numel() < 1) throw Refused("dev_status must have an element");
        return t.mutable_data_ptr<int32_t>();
    }
    long long integer() {
        const long long v = PyLong_AsLongLong(*at++);
        if (v == -1 && PyErr_Occurred()) throw Refused("");
        return v;
    }
    int small(const char *name) {
        const long long v = integer();
        if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " does not fit 32 bits");
        return static_cast<int>(v);
    }
    float real() {
        const double v = PyFloat_AsDouble(*at++);
        if (v == -1.0 && PyErr_Occurred()) throw Refused("");
        return static_cast<float>(v);
    }
    // the last argument: None for the current stream, else the raw stream
    void *stream() {
        if (none()) return skip(), c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
        return reinterpret_cast<void *>(static_cast<uintptr_t>(integer()));
    }
};

pkv_bf16 *bits(const at::Tensor &t) { return static_cast<pkv_bf16 *>(t.data_ptr()); }

void same_shape(const at::Tensor &t, const char *name, const at::Tensor &like, const char *other) {
    if (!t.sizes().equals(like.sizes())) throw Refused(std::string(name) + " must have the shape of " + other);
}

// q, k or v: [tokens, heads, head_dim] bf16 with each token's heads dense; returns
// the elements from token to token.
int64_t token_step(const at::Tensor &t, const char *name, int64_t tokens, int64_t head_dim) {
    if (t.dim() != 3 || t.size(0) != tokens || t.size(2) != head_dim)
        throw Refused(std::string(name) + " must have shape (" + std::to_string(tokens) + ", heads, " +
                      std::to_string(head_dim) + ")");
    if (t.stride(2) != 1 || (t.stride(1) != head_dim && t.size(1) > 1))
        throw Refused(std::string("the heads of each token of ") + name + " must be dense");
    return tokens > 1 ? t.stride(0) : t.size(1) * head_dim;
}

// A page table; returns its row width, every row lying inside the tensor's storage.
int64_t row_width(const at::Tensor &t, const char *name, int64_t batch) {
    if (t.dim() != 2 || t.size(0) < batch || (t.stride(1) != 1 && t.size(1) > 1))
        throw Refused(std::string(name) + " must have a row per sequence and unit column stride");
    const int64_t rows = t.size(0), width = t.stride(0);
    if (rows <= 1 || width == t.size(1)) return t.size(1);
    // columns of a wider table
    const int64_t room = static_cast<int64_t>(t.storage().nbytes()) / 4 - t.storage_offset();
    if (width < t.size(1) || rows * width > room)
        throw Refused(std::string("the last row of ") + name + " must be as wide as the others in memory");
    return width;
}

void caches(Arguments &a, const at::Tensor *&k, const at::Tensor *&v) {
    k = &a.bf16("k_cache", 4);
    v = &a.bf16("v_cache", 4);
    same_shape(*v, "v_cache", *k, "k_cache");
}

int as_int(int64_t v) {
    if (v > INT32_MAX) throw Refused("a size does not fit 32 bits");
    return static_cast<int>(v);
}

// (q, k, v, k_cache, v_cache, positions, cos_sin, out_loc, q_weight, k_weight, eps,
//  interleaved, dev_status, out, stream)
int qk_norm_rope_store(Arguments &a) {
    const at::Tensor &q = a.tensor("q", at::kBFloat16, "bfloat16");
    const at::Tensor &k = a.tensor("k", at::kBFloat16, "bfloat16");
    const at::Tensor &v = a.tensor("v", at::kBFloat16, "bfloat16");
    const at::Tensor *kc, *vc;
    caches(a, kc, vc);
    const int64_t Hkv = kc->size(2), d = kc->size(3);
    if (q.dim() != 3) throw Refused("q must have shape (tokens, heads, head size)");
    const int64_t T = q.size(0), Hq = q.size(1);
    const int64_t qs = token_step(q, "q", T, d), ks = token_step(k, "k", T, d), vs = token_step(v, "v", T, d);
    if (k.size(1) != Hkv || v.size(1) != Hkv)
        throw Refused("k, v and the caches must have the same number of heads");
    if (a.at[0] == Py_None ? a.at[1] != Py_None : a.at[1] == Py_None)
        throw Refused("positions and cos_sin come together");
    const int32_t *positions = a.ints("positions", T, true);
    const float *cos_sin = nullptr;
    int64_t rows = 0, rot = 0;
    if (a.none()) {
        a.skip();
    } else {
        const at::Tensor &t = a.f32("cos_sin", 2);
        cos_sin = t.const_data_ptr<float>(), rows = t.size(0), rot = t.size(1);
    }
    const int32_t *out_loc = a.ints("out_loc", T, false);
    const pkv_bf16 *weight[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "k_weight" : "q_weight";
        if (a.none()) {
            a.skip();
            continue;
        }
        const at::Tensor &t = a.bf16(name, 1);
        if (t.size(0) != d) throw Refused(std::string(name) + " must have an element for each of a head's");
        weight[i] = bits(t);
    }
    const float eps = a.real();
    const int interleaved = PyObject_IsTrue(*a.at++);
    int32_t *status = a.status();
    const at::Tensor &out = a.bf16("out", 3);
    same_shape(out, "out", q, "q");
    void *stream = a.stream();
    return pkv_qk_norm_rope_store(bits(q), qs, bits(k), ks, bits(v), vs, weight[0], weight[1], eps, positions, cos_sin,
                                  rows, as_int(rot), interleaved, out_loc, T, as_int(Hq), as_int(Hkv), as_int(d),
                                  bits(*kc), bits(*vc), kc->size(0), as_int(kc->size(1)), bits(out), status, stream);
}

// (q, k_cache, v_cache, page_table, seq_lens, softmax_scale, acc, max_seq_len, acc_rows,
//  workspace, dev_status, out, stream)
int paged_decode_attn_weights(Arguments &a) {
    const at::Tensor &q = a.bf16("q", 3);
    const at::Tensor *kc, *vc;
    caches(a, kc, vc);
    const int64_t B = q.size(0), Hq = q.size(1), Hkv = kc->size(2), d = kc->size(3);
    if (q.size(2) != d) throw Refused("q and the caches must have the same head size");
    const at::Tensor &table = a.tensor("page_table", at::kInt, "int32");
    const int64_t width = row_width(table, "page_table", B);
    const int32_t *seq_lens = a.ints("seq_lens", B, false);
    const float scale = a.real();
    const at::Tensor &acc = a.f32("acc", 3);
    if (acc.size(1) != Hkv) throw Refused("acc must have a row for each KV head");
    const int max_seq_len = a.small("max_seq_len");
    const int32_t *acc_rows = a.ints("acc_rows", B, true);
    const at::Tensor &workspace = a.dense("workspace", at::kByte, "uint8", 1);
    int32_t *status = a.status();
    const at::Tensor &out = a.bf16("out", 3);
    same_shape(out, "out", q, "q");
    void *stream = a.stream();
    return pkv_paged_decode_attn_weights(
        bits(q), bits(*kc), bits(*vc), table.const_data_ptr<int32_t>(), width, seq_lens, as_int(B), as_int(Hq),
        as_int(Hkv), as_int(d), as_int(kc->size(1)), kc->size(0), scale, acc.mutable_data_ptr<float>(), acc_rows,
        acc.size(0), acc.size(2), max_seq_len, workspace.data_ptr(), workspace.nbytes(), status, bits(out), stream);
}

// (k_cache, v_cache, page_table, page_table_out, seq_lens, keep_lens, num_first, num_recent, acc,
//  acc_out, acc_rows, kept, new_seq_lens, dev_status, stream)
int kv_evict(Arguments &a) {
    const at::Tensor *kc, *vc;
    caches(a, kc, vc);
    const int64_t Hkv = kc->size(2), d = kc->size(3);
    const at::Tensor &table = a.tensor("page_table", at::kInt, "int32");
    const at::Tensor &table_out = a.tensor("page_table_out", at::kInt, "int32");
    const at::Tensor &lens = a.i32("seq_lens", 1);
    const int64_t B = lens.size(0);
    const int64_t width = row_width(table, "page_table", B), width_out = row_width(table_out, "page_table_out", B);
    const int32_t *keep_lens = a.ints("keep_lens", B, false);
    const int num_first = a.small("num_first"), num_recent = a.small("num_recent");
    const at::Tensor &acc = a.f32("acc", 3);
    if (acc.size(1) != Hkv) throw Refused("acc must have a row for each KV head");
    const at::Tensor &acc_out = a.f32("acc_out", 3);
    same_shape(acc_out, "acc_out", acc, "acc");
    const int32_t *acc_rows = a.ints("acc_rows", B, true);
    const at::Tensor &kept = a.i32("kept", 3);
    if (kept.size(0) != B || kept.size(1) != Hkv) throw Refused("kept must have shape (batch, KV heads, max_keep)");
    int32_t *news = const_cast<int32_t *>(a.ints("new_seq_lens", B, false));
    int32_t *status = a.status();
    void *stream = a.stream();
    return pkv_kv_evict(bits(*kc), bits(*vc), table.const_data_ptr<int32_t>(), width,
                        table_out.const_data_ptr<int32_t>(), width_out, lens.const_data_ptr<int32_t>(), keep_lens,
                        as_int(B), as_int(Hkv), as_int(d), as_int(kc->size(1)), kc->size(0), num_first, num_recent,
                        acc.const_data_ptr<float>(), acc_out.mutable_data_ptr<float>(), acc_rows, acc.size(0),
                        acc.size(2), kept.mutable_data_ptr<int32_t>(), kept.size(2), news, status, stream);
}

template <int (*F)(Arguments &), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
        return nullptr;
    }
    try {
        c10::DeviceIndex device = -1;  // stays so without a GPU: every tensor is then refused
        if (c10::cuda::GetDevice(&device) != cudaSuccess) device = -1;
        Arguments a{args, device};
        return PyLong_FromLong(F(a));
    } catch (const Refused &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <int (*F)(Arguments &), int N>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>));
}

PyMethodDef kMethods[] = {
    {"qk_norm_rope_store", fast<qk_norm_rope_store, 15>(), METH_FASTCALL, nullptr},
    {"paged_decode_attn_weights", fast<paged_decode_attn_weights, 13>(), METH_FASTCALL, nullptr},
    {"kv_evict", fast<kv_evict, 15>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&kModule); }
