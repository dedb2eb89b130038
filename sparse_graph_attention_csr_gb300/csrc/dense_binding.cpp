// Python entry of the dense operators (attention over packed sequences, layer
// norm, embedding): argument checks, result and workspace allocation on the
// stream that writes them, and the call of the C ABI (include/sga.h).
//
// The smallest calls of these operators take a few microseconds on the GPU.
// Checked and allocated in Python they take 14 to 20 on the host, most of it
// interpreter time; here they take about half.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <limits>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/sga.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

PyObject *g_sga_error = nullptr;   // the package's SgaError(status, what)

void check(sga_status st, const char *what) {
    if (st == SGA_OK) return;
    py::object e = py::reinterpret_borrow<py::object>(g_sga_error)((int)st, what);
    PyErr_SetObject(g_sga_error, e.ptr());
    throw py::error_already_set();
}

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
const char *text(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        default: return c10::toString(t);
    }
}

void need_cuda(const Tensor &t, const char *name) {
    if (!t.defined() || !t.is_cuda()) throw py::value_error(std::string(name) + " must be a CUDA tensor");
}
void need_contiguous(const Tensor &t, const char *name) {
    if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
}

// A contiguous CUDA tensor of exactly this device, dtype and shape.
void need(const Tensor &t, const char *name, at::Device device, at::ScalarType dtype, at::IntArrayRef shape) {
    need_cuda(t, name);
    if (t.device() != device)
        throw py::value_error(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
    if (t.scalar_type() != dtype)
        throw py::type_error(std::string(name) + " must be " + text(dtype) + ", got " + text(t.scalar_type()));
    if (t.sizes() != shape)
        throw py::value_error(std::string(name) + " must be " + text(shape) + ", got " + text(t.sizes()));
    need_contiguous(t, name);
}

sga_dtype code(const Tensor &t) {
    if (t.scalar_type() == at::kFloat) return SGA_F32;
    if (t.scalar_type() == at::kBFloat16) return SGA_BF16;
    throw py::type_error(std::string("unsupported dtype ") + text(t.scalar_type()));
}

void *ptr(const Tensor &t) { return t.data_ptr(); }
void *ptr(const Maybe &t) { return t ? t->data_ptr() : nullptr; }

struct Named {
    const char *name;
    const Tensor *t;
};
Named named(const char *n, const Tensor &t) { return {n, &t}; }
Named named(const char *n, const Maybe &t) { return {n, t ? &*t : nullptr}; }

// Outputs must not share memory with inputs or one another.
void distinct(std::initializer_list<Named> outs, std::initializer_list<Named> ins) {
    auto clash = [](const Named &a, const Named &b) {
        if (!a.t || !b.t || a.t->numel() == 0 || b.t->numel() == 0) return;
        const char *p = static_cast<const char *>(a.t->data_ptr()), *q = static_cast<const char *>(b.t->data_ptr());
        if (p < q + b.t->nbytes() && q < p + a.t->nbytes())
            throw py::value_error(std::string(a.name) + " shares memory with " + b.name);
    };
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto u = o + 1; u != outs.end(); ++u) clash(*o, *u);
        for (const Named &i : ins) clash(*o, i);
    }
}

// A call on tensors of `device`, on `stream` (a torch.cuda.Stream) or the
// device's current stream: device and stream are current while this lives, so
// that what is allocated belongs to the stream that writes it.  With a stream
// given, the allocator is told that the inputs are used on it and the results
// on the caller's stream: memory that either frees early is not handed out
// while the other still uses it.
class Place {
  public:
    Place(at::Device device, const py::object &stream) {
        if (stream.is_none()) {
            dev_.emplace(device.index());
            raw_ = c10::cuda::getCurrentCUDAStream(device.index()).stream();
            return;
        }
        const auto s = c10::cuda::CUDAStream::unpack3(
            stream.attr("stream_id").cast<c10::StreamId>(), stream.attr("device_index").cast<c10::DeviceIndex>(),
            static_cast<c10::DeviceType>(stream.attr("device_type").cast<int>()));
        if (s.device_index() != device.index())
            throw py::value_error("stream is on cuda:" + std::to_string(s.device_index()) + ", the tensors on " + device.str());
        caller_ = c10::cuda::getCurrentCUDAStream(device.index());
        on_.emplace(s);
        raw_ = s.stream();
    }
    void *raw() const { return raw_; }
    void used(std::initializer_list<Named> ins, std::initializer_list<Named> outs) const {
        if (!caller_ || *caller_ == on_->current_stream()) return;
        auto note = [](const Named &n, c10::cuda::CUDAStream s) {
            if (n.t && n.t->numel() > 0)
                c10::cuda::CUDACachingAllocator::recordStream(n.t->storage().data_ptr(), s);
        };
        for (const Named &n : ins) note(n, on_->current_stream());
        for (const Named &n : outs) {
            note(n, on_->current_stream());   // (one given by the caller)
            note(n, *caller_);
        }
    }

  private:
    std::optional<c10::cuda::CUDAGuard> dev_;
    std::optional<c10::cuda::CUDAStreamGuard> on_;
    std::optional<c10::cuda::CUDAStream> caller_;
    void *raw_ = nullptr;
};

Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, at::Device device) {
    return at::detail::empty_cuda(shape, dtype, device, std::nullopt);   // (at::empty without the dispatcher)
}

// ---- attention over packed sequences -----------------------------------------------

struct SeqPlan {
    const sga_seq_plan *handle;
    at::Device device;
    at::ScalarType dtype;
    int64_t rows, H, Hkv, D, ws_bytes;
};

int64_t seq_inputs(const SeqPlan &p, const Tensor &Q, const Tensor &K, const Tensor &V) {
    const int64_t T = Q.dim() == 3 ? Q.size(0) : p.rows;
    if (T < p.rows)
        throw py::value_error("Q has " + std::to_string(T) + " rows, the plan's sequences cover " + std::to_string(p.rows));
    need(Q, "Q", p.device, p.dtype, {T, p.H, p.D});
    need(K, "K", p.device, p.dtype, {T, p.Hkv, p.D});
    need(V, "V", p.device, p.dtype, {T, p.Hkv, p.D});
    return T;
}

float seq_scale(const SeqPlan &p, std::optional<double> scale) {
    if (!scale) return (float)(1.0 / std::sqrt((double)p.D));
    const float f = (float)*scale;   // (a double may overflow, or round to zero)
    if (!(f > 0.f) || !std::isfinite(f * 1.4426950408889634f))   // (scores are held in units of log2)
        throw py::value_error("scale must be positive, and scale log2(e) a finite float32, got " + std::to_string(*scale));
    return f;
}

// The given result, or a new one: rows behind the last sequence, which the
// kernels leave as they are, are filled in a new one.
Tensor seq_result(const SeqPlan &p, const Maybe &given, const char *name, at::IntArrayRef shape, at::ScalarType dtype,
                  double fill) {
    if (given) {
        need(*given, name, p.device, dtype, shape);
        return *given;
    }
    Tensor t = fresh(shape, dtype, p.device);
    if (shape[0] > p.rows) t.narrow(0, p.rows, shape[0] - p.rows).fill_(fill);
    return t;
}

py::tuple seq_attn_fwd_(const SeqPlan &p, const Tensor &Q, const Tensor &K, const Tensor &V, std::optional<double> scale,
                        const Maybe &out, const Maybe &lse, const py::object &stream) {
    const int64_t T = seq_inputs(p, Q, K, V);
    const float f = seq_scale(p, scale);
    const Place on(p.device, stream);
    Tensor o = seq_result(p, out, "out", {T, p.H, p.D}, p.dtype, 0.0);
    Tensor l = seq_result(p, lse, "lse", {T, p.H}, at::kFloat, -std::numeric_limits<double>::infinity());
    if (out || lse) distinct({named("out", o), named("lse", l)}, {named("Q", Q), named("K", K), named("V", V)});
    check(seq_attn_fwd(p.handle, ptr(Q), ptr(K), ptr(V), T, f, ptr(o), static_cast<float *>(ptr(l)), on.raw()), "seq_attn_fwd");
    on.used({named("Q", Q), named("K", K), named("V", V)}, {named("out", o), named("lse", l)});
    return py::make_tuple(std::move(o), std::move(l));
}

py::tuple seq_attn_bwd_(const SeqPlan &p, const Tensor &Q, const Tensor &K, const Tensor &V, const Tensor &out,
                        const Tensor &lse, const Tensor &dOut, std::optional<double> scale, const Maybe &dQ,
                        const Maybe &dK, const Maybe &dV, const py::object &stream) {
    const int64_t T = seq_inputs(p, Q, K, V);
    need(out, "out", p.device, p.dtype, {T, p.H, p.D});
    need(dOut, "dOut", p.device, p.dtype, {T, p.H, p.D});
    need(lse, "lse", p.device, at::kFloat, {T, p.H});
    const float f = seq_scale(p, scale);
    const Place on(p.device, stream);
    Tensor q = seq_result(p, dQ, "dQ", {T, p.H, p.D}, p.dtype, 0.0);
    Tensor k = seq_result(p, dK, "dK", {T, p.Hkv, p.D}, p.dtype, 0.0);
    Tensor v = seq_result(p, dV, "dV", {T, p.Hkv, p.D}, p.dtype, 0.0);
    if (dQ || dK || dV)
        distinct({named("dQ", q), named("dK", k), named("dV", v)},
                 {named("Q", Q), named("K", K), named("V", V), named("out", out), named("lse", lse), named("dOut", dOut)});
    const Tensor ws = fresh({p.ws_bytes}, at::kByte, p.device);
    check(seq_attn_bwd(p.handle, ptr(Q), ptr(K), ptr(V), ptr(out), static_cast<const float *>(ptr(lse)), ptr(dOut), T, f,
                       ptr(q), ptr(k), ptr(v), ptr(ws), (size_t)p.ws_bytes, on.raw()),
          "seq_attn_bwd");
    on.used({named("Q", Q), named("K", K), named("V", V), named("out", out), named("lse", lse), named("dOut", dOut)},
            {named("dQ", q), named("dK", k), named("dV", v)});
    return py::make_tuple(std::move(q), std::move(k), std::move(v));
}

// ---- layer norm ---------------------------------------------------------------------

struct Norm {
    int64_t N, C;
    sga_dtype dt, wdt;
    at::IntArrayRef lead;
};

Norm norm_inputs(const Tensor &X, const Maybe &weight, const Maybe &bias) {
    need_cuda(X, "X");
    if (X.dim() < 1 || X.size(-1) < 1)
        throw py::value_error("X must be [..., C] with C >= 1, got " + text(X.sizes()));
    Norm n{};
    n.dt = n.wdt = code(X);
    need_contiguous(X, "X");
    n.C = X.size(-1);
    n.N = X.numel() / n.C;
    n.lead = X.sizes().slice(0, X.dim() - 1);
    if (!weight) {
        if (bias) throw py::value_error("a bias needs a weight");
        return n;
    }
    const at::ScalarType w = weight->scalar_type();
    if (w != at::kFloat && w != X.scalar_type())
        throw py::type_error(std::string("weight must be ") + text(X.scalar_type()) + " or torch.float32, got " + text(w));
    need(*weight, "weight", X.device(), w, {n.C});
    if (bias) need(*bias, "bias", X.device(), w, {n.C});
    n.wdt = w == at::kFloat ? SGA_F32 : SGA_BF16;
    return n;
}

py::tuple layer_norm_fwd_(const Tensor &X, const Maybe &weight, const Maybe &bias, double eps, const Maybe &out,
                          const Maybe &mean, const Maybe &rstd, const py::object &stream) {
    const Norm n = norm_inputs(X, weight, bias);
    const float feps = (float)eps;   // (a double may overflow, or round to zero)
    if (!(eps >= 0.0) || !std::isfinite(feps) || (feps == 0.f && eps != 0.0)) {
        std::ostringstream got;
        got << eps;
        throw py::value_error("eps must be zero or a positive and finite float32, got " + got.str());
    }
    const at::Device dev = X.device();
    const Place on(dev, stream);
    Tensor o = out ? *out : fresh(X.sizes(), X.scalar_type(), dev), m = mean ? *mean : fresh(n.lead, at::kFloat, dev),
           r = rstd ? *rstd : fresh(n.lead, at::kFloat, dev);
    if (out || mean || rstd) {
        need(o, "out", dev, X.scalar_type(), X.sizes());
        need(m, "mean", dev, at::kFloat, n.lead);
        need(r, "rstd", dev, at::kFloat, n.lead);
        // in place: a row is read before it is written
        const Maybe x = ptr(o) == ptr(X) ? Maybe() : Maybe(X);
        distinct({named("out", o), named("mean", m), named("rstd", r)},
                 {named("X", x), named("weight", weight), named("bias", bias)});
    }
    check(layer_norm_fwd(ptr(X), ptr(weight), ptr(bias), n.N, n.C, feps, n.dt, n.wdt, ptr(o),
                         static_cast<float *>(ptr(m)), static_cast<float *>(ptr(r)), on.raw()),
          "layer_norm_fwd");
    on.used({named("X", X), named("weight", weight), named("bias", bias)}, {named("out", o), named("mean", m), named("rstd", r)});
    return py::make_tuple(std::move(o), std::move(m), std::move(r));
}

py::tuple layer_norm_bwd_(const Tensor &X, const Maybe &weight, const Tensor &mean, const Tensor &rstd, const Tensor &dOut,
                          bool bias, const Maybe &dX, const Maybe &dweight, const Maybe &dbias, const py::object &stream) {
    const Norm n = norm_inputs(X, weight, std::nullopt);
    const at::Device dev = X.device();
    need(dOut, "dOut", dev, X.scalar_type(), X.sizes());
    need(mean, "mean", dev, at::kFloat, n.lead);
    need(rstd, "rstd", dev, at::kFloat, n.lead);
    if (!weight && (dweight || dbias)) throw py::value_error("dweight and dbias need a weight");
    if (!bias && dbias) throw py::value_error("dbias given with bias=False");
    const Place on(dev, stream);
    Tensor x = dX ? *dX : fresh(X.sizes(), X.scalar_type(), dev), ws;
    Maybe w = dweight, b = dbias;
    size_t bytes = 0;
    if (weight) {
        if (!w) w = fresh({n.C}, weight->scalar_type(), dev);
        if (bias && !b) b = fresh({n.C}, weight->scalar_type(), dev);
        bytes = sga_norm_bwd_workspace_bytes(n.N, n.C);
        ws = fresh({(int64_t)bytes}, at::kByte, dev);
    }
    if (dX || dweight || dbias) {
        need(x, "dX", dev, X.scalar_type(), X.sizes());
        if (w) need(*w, "dweight", dev, weight->scalar_type(), {n.C});
        if (b) need(*b, "dbias", dev, weight->scalar_type(), {n.C});
        distinct({named("dX", x), named("dweight", w), named("dbias", b)},
                 {named("X", X), named("weight", weight), named("mean", mean), named("rstd", rstd), named("dOut", dOut)});
    }
    check(layer_norm_bwd(ptr(X), ptr(weight), static_cast<const float *>(ptr(mean)), static_cast<const float *>(ptr(rstd)),
                         ptr(dOut), n.N, n.C, n.dt, n.wdt, ptr(x), ptr(w), ptr(b), weight ? ptr(ws) : nullptr, bytes,
                         on.raw()),
          "layer_norm_bwd");
    on.used({named("X", X), named("weight", weight), named("mean", mean), named("rstd", rstd), named("dOut", dOut)},
            {named("dX", x), named("dweight", w), named("dbias", b)});
    return py::make_tuple(std::move(x), w ? py::cast(*w) : py::none(), b ? py::cast(*b) : py::none());
}

// ---- embedding -------------------------------------------------------------------------

int id_bytes(const Tensor &ids) {
    need_cuda(ids, "ids");
    if (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong)
        throw py::type_error(std::string("ids must be torch.int32 or torch.int64, got ") + text(ids.scalar_type()));
    need_contiguous(ids, "ids");
    return (int)ids.element_size();
}
float embed_scale(double scale) {
    const float f = (float)scale;   // (a double may overflow)
    if (!std::isfinite(f)) throw py::value_error("scale must be a finite float32, got " + std::to_string(scale));
    return f;
}
at::DimVector with_width(const Tensor &ids, int64_t C) {
    at::DimVector s(ids.sizes());
    s.push_back(C);
    return s;
}

Tensor embed_fwd_(const Tensor &ids, const Tensor &table, double scale, const Maybe &out, const py::object &stream) {
    const int b = id_bytes(ids);
    if (table.dim() != 2 || table.size(1) < 1) throw py::value_error("table must be [V, C] with C >= 1");
    const sga_dtype dt = code(table);
    const at::Device dev = ids.device();
    const int64_t V = table.size(0), C = table.size(1);
    need(table, "table", dev, table.scalar_type(), {V, C});
    const float f = embed_scale(scale);
    const at::DimVector shape = with_width(ids, C);
    const Place on(dev, stream);
    Tensor o = out ? *out : fresh(shape, table.scalar_type(), dev);
    if (out) {
        need(o, "out", dev, table.scalar_type(), shape);
        distinct({named("out", o)}, {named("ids", ids), named("table", table)});
    }
    check(embed_fwd(ptr(ids), b, ptr(table), ids.numel(), V, C, f, dt, ptr(o), on.raw()), "embed_fwd");
    on.used({named("ids", ids), named("table", table)}, {named("out", o)});
    return o;
}

Tensor embed_bwd_(const Tensor &ids, const Tensor &dOut, int64_t V, double scale, std::optional<int64_t> padding_idx,
                  const Maybe &dTable, const py::object &stream) {
    const int b = id_bytes(ids);
    if (dOut.dim() < 1 || dOut.size(-1) < 1) throw py::value_error("dOut must be [*ids.shape, C] with C >= 1");
    const sga_dtype dt = code(dOut);
    const at::Device dev = ids.device();
    const int64_t C = dOut.size(-1), N = ids.numel();
    need(dOut, "dOut", dev, dOut.scalar_type(), with_width(ids, C));
    if (V < 0) throw py::value_error("num_rows must not be negative, got " + std::to_string(V));
    if (padding_idx && (*padding_idx < 0 || *padding_idx >= V))
        throw py::value_error("padding_idx must be in [0, " + std::to_string(V) + "), got " + std::to_string(*padding_idx));
    const float f = embed_scale(scale);
    const Place on(dev, stream);
    Tensor t = dTable ? *dTable : fresh({V, C}, dOut.scalar_type(), dev);
    if (dTable) {
        need(t, "dTable", dev, dOut.scalar_type(), {V, C});
        distinct({named("dTable", t)}, {named("ids", ids), named("dOut", dOut)});
    }
    const size_t bytes = sga_embed_bwd_workspace_bytes(N, V, C);
    const Tensor ws = fresh({(int64_t)bytes}, at::kByte, dev);
    check(embed_bwd(ptr(ids), b, ptr(dOut), N, V, C, f, padding_idx.value_or(-1), dt, ptr(t), ptr(ws), bytes, on.raw()),
          "embed_bwd");
    on.used({named("ids", ids), named("dOut", dOut)}, {named("dTable", t)});
    return t;
}

}  // namespace

PYBIND11_MODULE(_dense, m) {
    m.doc() = "Dense operators of sparse_graph_attention_csr_gb300 (use the package's functions).";
    m.def("set_error", [](py::object e) { g_sga_error = e.inc_ref().ptr(); });
    py::class_<SeqPlan>(m, "SeqPlan")
        .def(py::init([](uintptr_t handle, int device, bool f32, int64_t rows, int64_t H, int64_t Hkv, int64_t D, int64_t ws) {
            return SeqPlan{reinterpret_cast<const sga_seq_plan *>(handle), at::Device(at::kCUDA, (c10::DeviceIndex)device),
                           f32 ? at::kFloat : at::kBFloat16, rows, H, Hkv, D, ws};
        }));
    m.def("seq_attn_fwd", &seq_attn_fwd_);
    m.def("seq_attn_bwd", &seq_attn_bwd_);
    m.def("layer_norm_fwd", &layer_norm_fwd_);
    m.def("layer_norm_bwd", &layer_norm_bwd_);
    m.def("embed_fwd", &embed_fwd_);
    m.def("embed_bwd", &embed_bwd_);
}
