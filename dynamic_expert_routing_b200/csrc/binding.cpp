// binding.cpp -- the native side of training.py: checks the tensors of a training operator, allocates
// its outputs and scratch and calls the library.  It computes nothing.  (The calls are short: a
// launch costs about three microseconds of host time, the same steps in Python and ctypes ten.)
//
// The library is not linked: bind() opens the file that _lib.load() loaded and looks the entry
// points up, so both sides use one instance.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/extension.h>

#include <array>
#include <optional>
#include <string>

#include "../../include/beam_moe.h"

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

namespace {

constexpr int kBlock = 32;   // columns that share a scale

struct Api {
    decltype(&beam_balance_workspace) balance_workspace = nullptr;
    decltype(&beam_balance_forward) balance_forward = nullptr;
    decltype(&beam_balance_backward) balance_backward = nullptr;
    decltype(&beam_checkpoint_save) checkpoint_save = nullptr;
    decltype(&beam_checkpoint_load) checkpoint_load = nullptr;
    decltype(&beam_checkpoint_route_grad) route_grad = nullptr;
    decltype(&beam_router_weight_grad_workspace) weight_grad_workspace = nullptr;
    decltype(&beam_router_weight_grad) weight_grad = nullptr;
    decltype(&beam_router_input_grad) input_grad = nullptr;
} api;
py::object* check_fn = nullptr;   // _lib.check: raises BeamError with the library's message

template <typename F>
void find(void* lib, const char* name, F& f)
{
    f = reinterpret_cast<F>(dlsym(lib, name));
    if (!f) throw std::runtime_error(std::string(name) + " is not in the library: build it again");
}

void bind(const std::string& path, py::object check)
{
    void* lib = dlopen(path.c_str(), RTLD_NOW | RTLD_LOCAL);
    if (!lib) throw std::runtime_error(std::string("cannot open the library: ") + dlerror());
    find(lib, "beam_balance_workspace", api.balance_workspace);
    find(lib, "beam_balance_forward", api.balance_forward);
    find(lib, "beam_balance_backward", api.balance_backward);
    find(lib, "beam_checkpoint_save", api.checkpoint_save);
    find(lib, "beam_checkpoint_load", api.checkpoint_load);
    find(lib, "beam_checkpoint_route_grad", api.route_grad);
    find(lib, "beam_router_weight_grad_workspace", api.weight_grad_workspace);
    find(lib, "beam_router_weight_grad", api.weight_grad);
    find(lib, "beam_router_input_grad", api.input_grad);
    delete check_fn;
    check_fn = new py::object(std::move(check));
}

void done(int status)
{
    if (status != BEAM_OK) (*check_fn)(status);
}

// A string object made once per use in the source.
#define KEY(name)                                                       \
    ([] {                                                               \
        static PyObject* const key = PyUnicode_InternFromString(name);  \
        return py::reinterpret_borrow<py::object>(key);                 \
    }())

[[noreturn]] void bad(const std::string& msg) { throw py::value_error(msg); }

// A value of a dict that a caller hands in (borrowed).
PyObject* field(const char* what, const py::dict& d, const py::object& key)
{
    PyObject* const v = PyDict_GetItemWithError(d.ptr(), key.ptr());
    if (!v && PyErr_Occurred()) throw py::error_already_set();
    if (!v) bad(std::string(what) + " has no '" + key.cast<std::string>() + "'");
    return v;
}
Tensor field_tensor(const char* what, const py::dict& d, const py::object& key)
{
    PyObject* const v = field(what, d, key);
    if (!THPVariable_Check(v))
        throw py::type_error(std::string(what) + "['" + key.cast<std::string>() + "'] must be a tensor, got " + Py_TYPE(v)->tp_name);
    return THPVariable_Unpack(v);
}
int64_t field_int(const char* what, const py::dict& d, const py::object& key)
{
    PyObject* const v = field(what, d, key);
    if (!PyIndex_Check(v))
        throw py::type_error(std::string(what) + "['" + key.cast<std::string>() + "'] must be an integer, got " + Py_TYPE(v)->tp_name);
    const Py_ssize_t n = PyNumber_AsSsize_t(v, nullptr);   // past its range: the nearest end of it
    if (n == -1 && PyErr_Occurred()) throw py::error_already_set();
    return n;
}

// The tensors' device for the call: makes it current, gives its current stream, allocates on it.
struct On {
    c10::cuda::OptionalCUDAGuard guard;
    c10::Device device;
    void* stream;
    explicit On(const Tensor& t) : device(t.device())
    {
        if (device.index() != c10::cuda::current_device()) guard.set_index(device.index());
        stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    }
    Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const
    {
        return at::detail::empty_cuda(sizes, type, device, std::nullopt);
    }
    // Tensors that belong together in one allocation, each 256-byte aligned (balance loss 6.7 -> 5.8 us of host
    // time, slot gradients 6.4 -> 5.6).  They share a storage, so none is freed before the last.
    struct Piece {
        at::IntArrayRef sizes;
        at::ScalarType type;
    };
    template <size_t N> std::array<Tensor, N> together(const Piece (&pieces)[N]) const
    {
        int64_t at[N], bytes = 0;
        for (size_t i = 0; i < N; ++i) {
            at[i] = bytes;
            const int64_t size = c10::multiply_integers(pieces[i].sizes) * (int64_t)c10::elementSize(pieces[i].type);
            bytes += (size + 255) & ~(int64_t)255;
        }
        const Tensor all = empty({bytes}, at::kByte);
        std::array<Tensor, N> out;
        for (size_t i = 0; i < N; ++i) {
            out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                              c10::scalarTypeToTypeMeta(pieces[i].type));
            c10::TensorImpl* t = out[i].unsafeGetTensorImpl();
            t->set_storage_offset(at[i] / (int64_t)c10::elementSize(pieces[i].type));
            t->set_sizes_contiguous(pieces[i].sizes);
        }
        return out;
    }
    Tensor scratch(int64_t bytes) const { return bytes > 0 ? empty({bytes}, at::kByte) : Tensor(); }
};
void* address(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// A 2-dimensional CUDA tensor with contiguous rows.
struct Matrix {
    void* p;
    int type;
    int64_t rows, cols, ld;
};
Matrix matrix(const char* name, const Tensor& t, bool f16, const Tensor* like = nullptr)
{
    Matrix m;
    switch (t.scalar_type()) {
        case at::kFloat: m.type = BEAM_DTYPE_F32; break;
        case at::kBFloat16: m.type = BEAM_DTYPE_BF16; break;
        case at::kHalf: m.type = f16 ? BEAM_DTYPE_F16 : -1; break;
        default: m.type = -1;
    }
    if (m.type < 0 || !t.is_cuda() || t.dim() != 2)
        bad(std::string(name) + " must be a 2-dimensional CUDA tensor of dtype float32" +
            (f16 ? ", bfloat16 or float16" : " or bfloat16"));
    if (like && t.device() != like->device()) bad(std::string(name) + " must be on " + like->device().str());
    m.rows = t.size(0);
    m.cols = t.size(1);
    m.ld = m.rows > 1 ? t.stride(0) : m.cols;
    if ((m.cols > 1 && t.stride(1) != 1) || m.ld < m.cols)
        bad(std::string(name) + " must have contiguous, non-overlapping rows");
    if (m.rows > INT32_MAX || m.cols > INT32_MAX) bad(std::string(name) + " is too large");
    m.p = t.data_ptr();
    return m;
}

// A contiguous tensor of the given type and sizes on `like`'s device.
void* array(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef sizes, const Tensor& like)
{
    if (t.scalar_type() != type || t.device() != like.device() || t.sizes() != sizes || !t.is_contiguous()) {
        std::string s;
        for (int64_t n : sizes) s += (s.empty() ? "" : ", ") + std::to_string(n);
        bad(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape (" + s + ") on " +
            like.device().str());
    }
    return t.data_ptr();
}

struct Groups {
    int64_t K, n;
    const int32_t *ids, *cu;
    const uint8_t* valid;
};
Groups groups(const Tensor& logits, const Tensor& topk, const Opt& valid, const Opt& cu)
{
    if (topk.dim() != 2 || topk.size(0) != logits.size(0)) bad("topk_id must have the shape [T][K]");
    Groups g;
    g.K = topk.size(1);
    g.ids = static_cast<const int32_t*>(array("topk_id", topk, at::kInt, {logits.size(0), g.K}, logits));
    g.valid = nullptr;
    if (valid) {   // a bool is a byte of 0 or 1
        const at::ScalarType type = valid->scalar_type() == at::kBool ? at::kBool : at::kByte;
        g.valid = static_cast<const uint8_t*>(array("valid", *valid, type, {logits.size(0)}, logits));
    }
    g.cu = nullptr;
    g.n = 0;
    if (cu) {
        if (cu->dim() != 1 || cu->size(0) < 2) bad("cu_seqlens must hold the sequences' bounds: n_seq + 1 values");
        g.n = cu->size(0) - 1;
        g.cu = static_cast<const int32_t*>(array("cu_seqlens", *cu, at::kInt, {g.n + 1}, logits));
    }
    return g;
}

py::dict balance_loss(const Tensor& logits, const Tensor& topk, const Opt& valid, const Opt& cu)
{
    const Matrix m = matrix("logits", logits, false);
    const Groups g = groups(logits, topk, valid, cu);
    const On on(logits);
    const int64_t G = std::max<int64_t>(1, g.n);
    const int64_t size = api.balance_workspace((int32_t)m.rows, (int32_t)m.cols, (int32_t)g.n);
    const Tensor ws = on.scratch(size);
    // One allocation for a single group.  With sequences the loss has its own, so that a caller who keeps it does
    // not keep every sequence's rows: 0.6 us of host time, beside two launches of 8 us and more.
    const auto [prob, counts, tokens, beside] = on.together<4>(
        {{{G, m.cols}, at::kFloat}, {{G, m.cols}, at::kInt}, {{G}, at::kInt}, {{}, at::kFloat}});
    const Tensor loss = g.n > 0 ? on.empty({}, at::kFloat) : beside;
    done(api.balance_forward(m.p, m.type, (int32_t)m.rows, (int32_t)m.cols, m.ld, g.ids, (int32_t)g.K, g.valid, g.cu,
                             (int32_t)g.n, loss.data_ptr<float>(), prob.data_ptr<float>(), counts.data_ptr<int32_t>(),
                             tokens.data_ptr<int32_t>(), address(ws), size, on.stream));
    py::dict out;
    out[KEY("loss")] = loss;
    out[KEY("counts")] = counts;
    out[KEY("prob")] = prob;
    out[KEY("tokens")] = tokens;
    return out;
}

Tensor balance_loss_backward(const Tensor& logits, const Tensor& topk, const py::dict& balance, double scale,
                             const Opt& valid, const Opt& cu, const Opt& d_gate, const Opt& d_mask)
{
    const Matrix m = matrix("logits", logits, false);
    const Groups g = groups(logits, topk, valid, cu);
    const int64_t G = std::max<int64_t>(1, g.n);
    const Tensor c = field_tensor("balance", balance, KEY("counts")), t = field_tensor("balance", balance, KEY("tokens"));
    void* counts = array("balance['counts']", c, at::kInt, {G, m.cols}, logits);
    void* tokens = array("balance['tokens']", t, at::kInt, {G}, logits);
    if (d_gate.has_value() != d_mask.has_value()) bad("d_gate_logit and d_mask_logit come together");
    void *gr = nullptr, *gl = nullptr;
    if (d_gate) {
        gr = array("d_gate_logit", *d_gate, at::kFloat, {m.rows, g.K}, logits);
        gl = array("d_mask_logit", *d_mask, at::kFloat, {m.rows, g.K}, logits);
    }
    const On on(logits);
    Tensor out = on.empty({m.rows, d_gate ? 2 * m.cols : m.cols}, at::kFloat);
    done(api.balance_backward(m.p, m.type, (int32_t)m.rows, (int32_t)m.cols, m.ld, g.ids, (int32_t)g.K, g.valid, g.cu,
                              (int32_t)g.n, static_cast<int32_t*>(counts), static_cast<int32_t*>(tokens), (float)scale,
                              static_cast<float*>(gr), static_cast<float*>(gl), out.data_ptr<float>(), on.stream));
    return out;
}

py::dict checkpoint_save(const Tensor& x)
{
    const Matrix m = matrix("x", x, true);
    const On on(x);
    const int64_t nb = (m.cols + kBlock - 1) / kBlock;
    const auto [q, scale] = on.together<2>({{{m.rows, nb * kBlock}, at::kChar}, {{m.rows, nb}, at::kByte}});
    done(api.checkpoint_save(m.p, m.type, m.rows, (int32_t)m.cols, m.ld, q.data_ptr<int8_t>(), scale.data_ptr<uint8_t>(),
                             on.stream));
    py::dict out;
    out[KEY("q")] = q;
    out[KEY("scale")] = scale;
    out[KEY("d")] = m.cols;
    return out;
}

struct Ckpt {
    Tensor t;
    int8_t* q;
    uint8_t* scale;
    int64_t rows, d;
};
Ckpt checkpoint(const py::dict& c)
{
    Ckpt k;
    k.t = field_tensor("checkpoint", c, KEY("q"));
    const Tensor scale = field_tensor("checkpoint", c, KEY("scale"));
    k.d = field_int("checkpoint", c, KEY("d"));
    if (!k.t.is_cuda() || k.t.dim() != 2 || k.d < 1 || k.d > INT32_MAX - kBlock)
        bad("a checkpoint holds CUDA tensors q [rows][..] and scale and a width d >= 1");
    k.rows = k.t.size(0);
    const int64_t nb = (k.d + kBlock - 1) / kBlock;
    k.q = static_cast<int8_t*>(array("checkpoint q", k.t, at::kChar, {k.rows, nb * kBlock}, k.t));
    k.scale = static_cast<uint8_t*>(array("checkpoint scale", scale, at::kByte, {k.rows, nb}, k.t));
    return k;
}

Tensor checkpoint_load(const py::dict& ckpt, py::object dtype)
{
    const at::ScalarType type = reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
    const int dt = type == at::kFloat ? BEAM_DTYPE_F32 : type == at::kBFloat16 ? BEAM_DTYPE_BF16
                 : type == at::kHalf ? BEAM_DTYPE_F16 : -1;
    if (dt < 0) throw py::type_error(std::string("unsupported dtype ") + c10::toString(type));
    const Ckpt k = checkpoint(ckpt);
    const On on(k.t);
    Tensor y = on.empty({k.rows, k.d}, type);
    done(api.checkpoint_load(k.q, k.scale, k.rows, (int32_t)k.d, y.data_ptr(), dt, on.stream));
    return y;
}

py::dict checkpoint_route_grad(const py::dict& ckpt, const Tensor& gate, const Tensor& mask_logit, const Tensor& dy,
                               double reg_scale, int segment_len)
{
    const Ckpt k = checkpoint(ckpt);
    if (gate.dim() != 2) bad("gate must have the shape [T][K]");
    const int64_t T = gate.size(0), K = gate.size(1);
    void* g = array("gate", gate, at::kFloat, {T, K}, k.t);
    void* l = array("mask_logit", mask_logit, at::kFloat, {T, K}, k.t);
    const Matrix m = matrix("dy", dy, false, &k.t);
    if (m.rows != T || m.cols != k.d || k.rows != T * K)
        bad("dy must be [T][d] and the checkpoint hold T*K rows: got dy [" + std::to_string(m.rows) + "][" +
            std::to_string(m.cols) + "], " + std::to_string(k.rows) + " rows of " + std::to_string(k.d) +
            " values, gate [" + std::to_string(T) + "][" + std::to_string(K) + "]");
    const On on(k.t);
    const auto [s, dr, dl] = on.together<3>({{{T, K}, at::kFloat}, {{T, K}, at::kFloat}, {{T, K}, at::kFloat}});
    done(api.route_grad(k.q, k.scale, (int32_t)T, (int32_t)K, (int32_t)k.d, static_cast<float*>(g), static_cast<float*>(l),
                        m.p, m.type, m.ld, segment_len, (float)reg_scale, s.data_ptr<float>(), dr.data_ptr<float>(),
                        dl.data_ptr<float>(), on.stream));
    py::dict out;
    out[KEY("dghat")] = s;
    out[KEY("d_gate_logit")] = dr;
    out[KEY("d_mask_logit")] = dl;
    return out;
}

Tensor router_weight_grad(const py::dict& ckpt, const Tensor& dlogits, int64_t parts)
{
    const Ckpt k = checkpoint(ckpt);
    const Matrix m = matrix("dlogits", dlogits, false, &k.t);
    if (m.rows != k.rows)
        bad("dlogits has " + std::to_string(m.rows) + " rows, the checkpoint " + std::to_string(k.rows));
    if (parts < 1 || m.cols % parts)
        bad("parts=" + std::to_string(parts) + " must divide the " + std::to_string(m.cols) + " columns of dlogits");
    const On on(k.t);
    Tensor dw = parts == 1 ? on.empty({k.d, m.cols}, at::kFloat) : on.empty({parts, k.d, m.cols / parts}, at::kFloat);
    const int64_t size = api.weight_grad_workspace((int32_t)m.rows, (int32_t)k.d, (int32_t)m.cols);
    const Tensor ws = on.scratch(size);
    done(api.weight_grad(k.q, k.scale, (int32_t)m.rows, (int32_t)k.d, m.p, m.type, m.ld, (int32_t)m.cols, (int32_t)parts,
                         dw.data_ptr<float>(), address(ws), size, on.stream));
    return dw;
}

Tensor router_input_grad(const Tensor& dlogits, const Tensor& w)
{
    const Matrix g = matrix("dlogits", dlogits, false), m = matrix("w", w, false, &dlogits);
    if (m.cols != g.cols) bad("w must have dlogits' " + std::to_string(g.cols) + " columns");
    const On on(dlogits);
    Tensor dx = on.empty({g.rows, m.rows}, at::kFloat);
    done(api.input_grad(g.p, g.type, g.ld, (int32_t)g.rows, (int32_t)g.cols, m.p, m.type, m.ld, (int32_t)m.rows,
                        dx.data_ptr<float>(), m.rows, on.stream));
    return dx;
}

}  // namespace

PYBIND11_MODULE(_training, m)
{
    m.doc() = "Native side of training.py.";
    m.def("bind", &bind);
    m.def("balance_loss", &balance_loss);
    m.def("balance_loss_backward", &balance_loss_backward);
    m.def("checkpoint_save", &checkpoint_save);
    m.def("checkpoint_load", &checkpoint_load);
    m.def("checkpoint_route_grad", &checkpoint_route_grad);
    m.def("router_weight_grad", &router_weight_grad);
    m.def("router_input_grad", &router_input_grad);
}
