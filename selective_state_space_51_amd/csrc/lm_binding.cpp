// Python binding of libselscan_lm: checks torch tensors, allocates outputs and workspaces from torch's
// allocator on the current stream, and calls the C ABI (include/selscan_lm.h).  No arithmetic here.
//
// A token step of one sequence runs two kernels of a few microseconds each, so the time of a call is
// mostly the host's: through ctypes and checks in Python one call took 12 to 15 us, here 4 to 5.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <tuple>

#include "selscan_lm.h"

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

namespace {

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

void want_shape(const char *name, const Tensor &t, at::IntArrayRef shape) {
    if (t.sizes() != shape)
        throw py::value_error(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
}
void want_shape(const char *name, const Opt &t, at::IntArrayRef shape) {
    if (t) want_shape(name, *t, shape);
}

int io_code(const Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return SELSCAN_BF16;
    if (t.scalar_type() == at::kFloat) return SELSCAN_F32;
    throw py::type_error(std::string("unsupported io dtype ") + c10::toString(t.scalar_type()));
}

void want_device(const char *name, const Tensor &t) {
    if (!t.is_cuda()) throw py::value_error(std::string(name) + " must be a device tensor");
}
// the device of this thread's latest Launch: every operand has to be on it.  (Asking the runtime for the current device
// at each operand took 0.4 us of the two calls of a token step.)
thread_local c10::DeviceIndex launch_device = -1;
void want_here(const char *name, const Tensor &t) {
    want_device(name, t);
    if (t.get_device() != launch_device)
        throw py::value_error(std::string(name) + " is on " + t.device().str() + ", the first argument is on cuda:" +
                              std::to_string(launch_device));
}
void want_dtype(const char *name, const Tensor &t, at::ScalarType dt) {
    if (t.scalar_type() != dt) throw py::type_error(std::string(name) + " must be " + c10::toString(dt));
}

// address of a contiguous tensor of one dtype
void *ptr(const char *name, const Tensor &t, at::ScalarType dt) {
    want_here(name, t);
    if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
    want_dtype(name, t, dt);
    return t.numel() ? t.data_ptr() : nullptr;
}
template <class P = void>
P *ptr(const char *name, const Opt &t, at::ScalarType dt) {
    return t ? (P *)ptr(name, *t, dt) : nullptr;
}
const float *f32(const char *name, const Tensor &t) { return (const float *)ptr(name, t, at::kFloat); }
const float *f32(const char *name, const Opt &t) { return t ? f32(name, *t) : nullptr; }

// address and row stride of a matrix whose rows are contiguous
struct Rows {
    void *p = nullptr;
    int64_t stride = 0;
};
Rows rows_of(const char *name, const Tensor &t, at::ScalarType dt) {
    want_here(name, t);
    want_dtype(name, t, dt);
    if (t.dim() != 2) throw py::value_error(std::string(name) + " must have two dimensions");
    const int64_t rows = t.size(0), width = t.size(1);
    if (width > 1 && t.stride(1) != 1) throw py::value_error(std::string("the rows of ") + name + " must be contiguous");
    const int64_t stride = rows > 1 ? t.stride(0) : width;
    if (stride < width) throw py::value_error(std::string("the rows of ") + name + " overlap");
    return {t.numel() ? t.data_ptr() : nullptr, stride};
}
Rows rows_of(const char *name, const Opt &t, at::ScalarType dt) { return t ? rows_of(name, *t, dt) : Rows{}; }

void want_matrix(const char *name, const Tensor &t) {
    if (t.dim() != 2) throw py::value_error(std::string(name) + " must have two dimensions");
}

void check(int rc, const char *what) {
    if (rc == SELSCAN_OK) return;
    const py::object err = py::module_::import("selective_state_space_51_amd").attr("SelscanError");
    const py::object hip = py::cpp_function([] { return py::bytes(selscan_lm_last_hip_error()); });
    const py::object e = err(rc, what, hip);
    PyErr_SetObject(err.ptr(), e.ptr());
    throw py::error_already_set();
}

// the device a call runs on, made current, and the stream it is enqueued on
struct Launch {
    c10::DeviceGuard guard;
    void *stream;
    explicit Launch(const Tensor &t)
        : guard((want_device("the first argument", t), t.device())),
          stream((void *)c10::hip::getCurrentHIPStream(t.device().index()).stream()) {
        launch_device = t.device().index();
    }
};

Tensor empty(at::IntArrayRef shape, const Tensor &like, at::ScalarType dt) {
    return at::empty(shape, like.options().dtype(dt));
}

struct Workspace {
    Tensor own;
    void *p = nullptr;
    size_t bytes = 0;
};
Workspace workspace(size_t need, const Opt &given, const Tensor &like) {
    Workspace w;
    if (!need) return w;
    w.own = given ? *given : empty({(int64_t)need}, like, at::kByte);
    want_here("workspace", w.own);
    if (!w.own.is_contiguous()) throw py::value_error("workspace must be contiguous");
    w.p = w.own.data_ptr();
    w.bytes = w.own.nbytes();
    return w;
}

unsigned scan_flags(bool softplus, bool zoh) {
    return (softplus ? SELSCAN_FLAG_DELTA_SOFTPLUS : 0u) | (zoh ? SELSCAN_FLAG_ZOH : 0u);
}

struct Packed {
    int64_t nseq = 0, nslots = 0;
    const int32_t *cu = nullptr, *slots = nullptr;
    const uint8_t *carry = nullptr;
};
Packed packed(const Tensor &cu, const Opt &slots, const Opt &carry, const Opt &cache) {
    Packed p;
    p.nseq = cu.numel() - 1;
    if (cu.dim() != 1 || p.nseq < 0) throw py::value_error("cu_seqlens must be a vector of nseq + 1 offsets");
    want_shape("slots", slots, {p.nseq});
    want_shape("carry", carry, {p.nseq});
    p.nslots = cache ? cache->size(0) : 0;
    p.cu = (const int32_t *)ptr("cu_seqlens", cu, at::kInt);
    p.slots = ptr<const int32_t>("slots", slots, at::kInt);
    if (carry) p.carry = (const uint8_t *)ptr("carry", *carry, carry->scalar_type() == at::kBool ? at::kBool : at::kByte);
    return p;
}

int64_t conv_shapes(const Tensor &x, const Tensor &weight, const Opt &bias, const Opt &state) {
    want_matrix("x", x);
    want_matrix("weight", weight);
    const int64_t dim = x.size(1), width = weight.size(1);
    want_shape("weight", weight, {dim, width});
    want_shape("bias", bias, {dim});
    if (state) {
        if (state->dim() != 3) throw py::value_error("conv_state must have three dimensions");
        want_shape("conv_state", *state, {state->size(0), width - 1, dim});
    }
    return width;
}

Tensor conv_packed(const Tensor &x, const Tensor &weight, const Tensor &cu, const Opt &state, const Opt &bias,
                   const Opt &slots, const Opt &carry, bool silu, const Opt &out_) {
    const int64_t width = conv_shapes(x, weight, bias, state), tokens = x.size(0), dim = x.size(1);
    const Launch l(x);
    const int io = io_code(x);
    const at::ScalarType dt = x.scalar_type();
    const Packed p = packed(cu, slots, carry, state);
    const Tensor out = out_ ? *out_ : empty({tokens, dim}, x, dt);
    want_shape("out", out, {tokens, dim});
    const Rows xr = rows_of("x", x, dt);
    check(causal_conv1d_packed_fwd(xr.p, xr.stride, f32("weight", weight), f32("bias", bias), p.cu, p.slots, p.carry,
                                   ptr("conv_state", state, dt), silu ? SELSCAN_FLAG_SILU : 0u, ptr("out", out, dt), tokens,
                                   p.nseq, p.nslots, dim, width, io, l.stream),
          "causal_conv1d_packed_fwd");
    return out;
}

Tensor conv_step(const Tensor &x, const Tensor &weight, const Tensor &state, const Opt &bias, const Opt &slots, bool silu,
                 const Opt &out_) {
    const int64_t width = conv_shapes(x, weight, bias, state), rows = x.size(0), dim = x.size(1);
    want_shape("slots", slots, {rows});
    const Launch l(x);
    const int io = io_code(x);
    const at::ScalarType dt = x.scalar_type();
    const Tensor out = out_ ? *out_ : empty({rows, dim}, x, dt);
    want_shape("out", out, {rows, dim});
    const Rows xr = rows_of("x", x, dt);
    check(causal_conv1d_step(xr.p, xr.stride, f32("weight", weight), f32("bias", bias),
                             ptr<const int32_t>("slots", slots, at::kInt), ptr("conv_state", state, dt),
                             silu ? SELSCAN_FLAG_SILU : 0u, ptr("out", out, dt), rows, state.size(0), dim, width, io, l.stream),
          "causal_conv1d_step");
    return out;
}

int64_t scan_shapes(const Tensor &x, const Tensor &delta, const Tensor &A, const Tensor &B, const Tensor &C, const Opt &D,
                    const Opt &z, const Opt &bias, const Opt &h) {
    want_matrix("x", x);
    want_matrix("A", A);
    const int64_t rows = x.size(0), dim = x.size(1), n = A.size(1);
    want_shape("delta", delta, {rows, dim});
    want_shape("A", A, {dim, n});
    want_shape("B", B, {rows, n});
    want_shape("C", C, {rows, n});
    want_shape("D", D, {dim});
    want_shape("z", z, {rows, dim});
    want_shape("delta_bias", bias, {dim});
    if (h) {
        if (h->dim() != 3) throw py::value_error("h_state must have three dimensions");
        want_shape("h_state", *h, {h->size(0), dim, n});
    }
    return n;
}

std::tuple<Rows, Rows> bc_rows(const Tensor &B, const Tensor &C, at::ScalarType dt) {
    const Rows b = rows_of("B", B, dt), c = rows_of("C", C, dt);
    if (b.stride != c.stride) throw py::value_error("B and C must have the same row stride");
    return {b, c};
}

Tensor scan_packed(const Tensor &x, const Tensor &delta, const Tensor &A, const Tensor &B, const Tensor &C, const Tensor &cu,
                   const Opt &h, const Opt &D, const Opt &z, const Opt &bias, bool softplus, bool zoh, const Opt &slots,
                   const Opt &carry, std::optional<int64_t> max_seqlen, const Opt &y_, const Opt &ws_) {
    const int64_t n = scan_shapes(x, delta, A, B, C, D, z, bias, h), tokens = x.size(0), dim = x.size(1);
    const Launch l(x);
    const int io = io_code(x);
    const at::ScalarType dt = x.scalar_type();
    const Packed p = packed(cu, slots, carry, h);
    const int64_t longest = max_seqlen.value_or(tokens);
    const Tensor y = y_ ? *y_ : empty({tokens, dim}, x, dt);
    want_shape("y", y, {tokens, dim});
    const Workspace ws = workspace(selscan_packed_workspace_bytes(tokens, p.nseq, longest, dim, n), ws_, x);
    const auto [b, c] = bc_rows(B, C, dt);
    const Rows zr = rows_of("z", z, dt);
    check(selscan_packed_fwd(ptr("x", x, dt), ptr("delta", delta, dt), f32("A", A), b.p, c.p, b.stride, f32("D", D), zr.p,
                             zr.stride, f32("delta_bias", bias), scan_flags(softplus, zoh), p.cu, p.slots, p.carry,
                             ptr<float>("h_state", h, at::kFloat), ptr("y", y, dt), tokens, p.nseq, p.nslots, longest, dim, n,
                             io, ws.p, ws.bytes, l.stream),
          "selscan_packed_fwd");
    return y;
}

Tensor scan_step(const Tensor &x, const Tensor &delta, const Tensor &A, const Tensor &B, const Tensor &C, const Tensor &h,
                 const Opt &D, const Opt &z, const Opt &bias, bool softplus, bool zoh, const Opt &slots, const Opt &y_) {
    const int64_t n = scan_shapes(x, delta, A, B, C, D, z, bias, h), rows = x.size(0), dim = x.size(1);
    want_shape("slots", slots, {rows});
    const Launch l(x);
    const int io = io_code(x);
    const at::ScalarType dt = x.scalar_type();
    const Tensor y = y_ ? *y_ : empty({rows, dim}, x, dt);
    want_shape("y", y, {rows, dim});
    const auto [b, c] = bc_rows(B, C, dt);
    const Rows zr = rows_of("z", z, dt);
    check(selscan_step(ptr("x", x, dt), ptr("delta", delta, dt), f32("A", A), b.p, c.p, b.stride, f32("D", D), zr.p, zr.stride,
                       f32("delta_bias", bias), scan_flags(softplus, zoh), ptr<const int32_t>("slots", slots, at::kInt),
                       (float *)ptr("h_state", h, at::kFloat), ptr("y", y, dt), rows, h.size(0), dim, n, io, l.stream),
          "selscan_step");
    return y;
}

py::tuple norm_fwd(const Tensor &x, const Tensor &weight, const Opt &residual, double eps, const std::string &out,
                   std::optional<at::ScalarType> residual_dtype, bool rstd) {
    want_matrix("x", x);
    const int64_t rows = x.size(0), width = x.size(1);
    const int kind = out == "io" ? SELSCAN_LM_OUT_IO : out == "int8" ? SELSCAN_LM_OUT_INT8 : out == "fp8" ? SELSCAN_LM_OUT_FP8 : -1;
    if (kind < 0) throw py::value_error("out must be one of ['fp8', 'int8', 'io']");
    const Launch l(x);
    const int io = io_code(x);
    const at::ScalarType dt = x.scalar_type(), rdt = residual ? residual->scalar_type() : residual_dtype.value_or(dt);
    if (rdt != at::kFloat && rdt != dt) throw py::type_error("the residual must be float32 or have the io dtype");
    want_shape("weight", weight, {width});
    want_shape("residual", residual, {rows, width});
    const Tensor y = empty({rows, width}, x, kind == SELSCAN_LM_OUT_IO ? dt : kind == SELSCAN_LM_OUT_INT8 ? at::kChar : at::kFloat8_e4m3fn);
    const Tensor s = empty({rows, width}, x, rdt);
    Tensor scale, rs;
    if (kind != SELSCAN_LM_OUT_IO) scale = empty({rows}, x, at::kFloat);
    if (rstd) rs = empty({rows}, x, at::kFloat);
    const Rows xr = rows_of("x", x, dt);
    check(add_rms_norm_fwd(xr.p, xr.stride, ptr("residual", residual, rdt), f32("weight", weight), (float)eps, kind, y.data_ptr(),
                           s.data_ptr(), scale.defined() ? (float *)scale.data_ptr() : nullptr,
                           rstd ? (float *)rs.data_ptr() : nullptr, rows, width, io, io_code(s), l.stream),
          "add_rms_norm_fwd");
    py::list r;
    r.append(y);
    r.append(s);
    if (scale.defined()) r.append(scale);
    if (rstd) {
        // a sum rounded to 16 bits is not the one that was normed: the gradients form it anew from these
        if (residual && rdt != at::kFloat) r.append(py::make_tuple(rs, x, *residual));
        else r.append(rs);
    }
    return py::tuple(r);
}

std::tuple<Tensor, Tensor, Tensor> norm_bwd(const Tensor &dy, const Tensor &s, const Tensor &weight, const Tensor &rstd,
                                            const Opt &x, const Opt &dres, const Opt &ws_) {
    want_matrix("dy", dy);
    const int64_t rows = dy.size(0), width = dy.size(1);
    want_shape("s", s, {rows, width});
    want_shape("weight", weight, {width});
    want_shape("rstd", rstd, {rows});
    want_shape("x", x, {rows, width});
    want_shape("dresidual_out", dres, {rows, width});
    const Launch l(dy);
    const int io = io_code(dy);
    const at::ScalarType dt = dy.scalar_type(), rdt = s.scalar_type();
    const Tensor dx = empty({rows, width}, dy, dt), dw = empty({width}, dy, at::kFloat);
    const Tensor dr = rdt != dt ? empty({rows, width}, dy, rdt) : Tensor();
    const Workspace ws = workspace(add_rms_norm_bwd_workspace_bytes(rows, width), ws_, dy);
    const Rows xr = rows_of("x", x, dt);
    check(add_rms_norm_bwd(ptr("dy", dy, dt), ptr("s", s, rdt), xr.p, xr.stride, f32("weight", weight), f32("rstd", rstd),
                           ptr("dresidual_out", dres, rdt), dx.data_ptr(), dr.defined() ? dr.data_ptr() : nullptr,
                           (float *)dw.data_ptr(), rows, width, io, io_code(s), ws.p, ws.bytes, l.stream),
          "add_rms_norm_bwd");
    return {dx, dr.defined() ? dr : dx, dw};
}

py::tuple logprobs_fwd(const Tensor &logits, const Tensor &targets, int64_t top, double scale, const Opt &ws_) {
    want_matrix("logits", logits);
    const int64_t rows = logits.size(0), vocab = logits.size(1);
    want_shape("targets", targets, {rows});
    if (top < 0 || top > vocab) throw py::value_error("top must be in [0, vocab]");
    const Launch l(logits);
    const int io = io_code(logits);
    const Tensor lp = empty({rows}, logits, at::kFloat), ent = empty({rows}, logits, at::kFloat), st = empty({rows, 2}, logits, at::kFloat);
    Tensor val, idx;
    if (top) val = empty({rows, top}, logits, at::kFloat), idx = empty({rows, top}, logits, at::kLong);
    const int k = (int)(top > 1000 ? 1000 : top);  // (too many are refused below)
    const Workspace ws = workspace(token_logprobs_workspace_bytes(rows, vocab, k), ws_, logits);
    const Rows xr = rows_of("logits", logits, logits.scalar_type());
    check(token_logprobs_fwd(xr.p, xr.stride, (const int64_t *)ptr("targets", targets, at::kLong), (float)scale, k,
                             (float *)lp.data_ptr(), (float *)ent.data_ptr(), (float *)st.data_ptr(),
                             top ? (float *)val.data_ptr() : nullptr, top ? (int64_t *)idx.data_ptr() : nullptr, rows, vocab, io,
                             ws.p, ws.bytes, l.stream),
          "token_logprobs_fwd");
    return top ? py::make_tuple(lp, ent, st, val, idx) : py::make_tuple(lp, ent, st);
}

Tensor logprobs_bwd(const Tensor &logits, const Tensor &targets, const Tensor &stats, const Tensor &entropy, const Opt &dlogprob,
                    const Opt &dentropy, double scale) {
    want_matrix("logits", logits);
    const int64_t rows = logits.size(0), vocab = logits.size(1);
    want_shape("targets", targets, {rows});
    want_shape("stats", stats, {rows, 2});
    want_shape("entropy", entropy, {rows});
    want_shape("dlogprob", dlogprob, {rows});
    want_shape("dentropy", dentropy, {rows});
    const Launch l(logits);
    const int io = io_code(logits);
    const Tensor dx = empty({rows, vocab}, logits, logits.scalar_type());
    const Rows xr = rows_of("logits", logits, logits.scalar_type());
    check(token_logprobs_bwd(xr.p, xr.stride, (const int64_t *)ptr("targets", targets, at::kLong), f32("stats", stats),
                             f32("entropy", entropy), f32("dlogprob", dlogprob), f32("dentropy", dentropy), (float)scale,
                             dx.data_ptr(), rows, vocab, io, l.stream),
          "token_logprobs_bwd");
    return dx;
}

Tensor matvec(const Tensor &x, const Tensor &q, const Tensor &scales, const Opt &zeros, int64_t group, const Opt &bias,
              const Opt &out_) {
    want_matrix("x", x);
    want_matrix("qweight", q);
    const int64_t rows = x.size(0), k = x.size(1), n = q.size(0);
    if (group <= 0 || k % group)
        throw py::value_error("group " + std::to_string(group) + " does not divide k = " + std::to_string(k));
    want_shape("qweight", q, {n, k / 2});
    want_shape("scales", scales, {n, k / group});
    want_shape("zeros", zeros, {n, k / group});
    want_shape("bias", bias, {n});
    const Launch l(x);
    const int io = io_code(x);
    const at::ScalarType dt = x.scalar_type();
    const Tensor out = out_ ? *out_ : empty({rows, n}, x, dt);
    want_shape("out", out, {rows, n});
    const Rows xr = rows_of("x", x, dt);
    check(w4_matvec(xr.p, xr.stride, ptr("qweight", q, at::kByte), ptr("scales", scales, at::kBFloat16), ptr("zeros", zeros, at::kByte),
                    f32("bias", bias), ptr("out", out, dt), rows, n, k, group, io, l.stream),
          "w4_matvec");
    return out;
}

}  // namespace

PYBIND11_MODULE(_lm_binding, m) {
    m.def("causal_conv1d_packed_fwd", &conv_packed);
    m.def("causal_conv1d_step", &conv_step);
    m.def("selscan_packed_fwd", &scan_packed);
    m.def("selscan_step", &scan_step);
    m.def("add_rms_norm_fwd", &norm_fwd);
    m.def("add_rms_norm_bwd", &norm_bwd);
    m.def("token_logprobs_fwd", &logprobs_fwd);
    m.def("token_logprobs_bwd", &logprobs_bwd);
    m.def("w4_matvec", &matvec);
}
