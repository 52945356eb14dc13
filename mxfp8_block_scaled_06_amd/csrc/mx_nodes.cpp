// Autograd nodes of the router, the gated activation and the weighted sum over a
// token's experts, on the C ABI of include/mxmoe.h; and the calls between the
// experts' products that allocate up to six results.
//
// Host time is what a small call costs.  A forward and a backward through a node
// written in Python took 80 - 90 us where one of torch's own took 48: the backward
// runs on autograd's thread, which takes the GIL and then walks Python objects that
// the main thread has just used.  These nodes take 36 - 48 and need no GIL in the
// backward.
//
// Each call looks its operands over (contiguous GPU tensors of the right types, shapes
// and device, at addresses that wide loads take) and returns nothing where something does not fit: the Python binding then
// makes the copy that is missing or raises, check by check.  The same checks in Python
// took 1 - 2 us of a 7 us call (router of one token 7.4 -> 6.6 us, and 5.6 without a node).  The C ABI checks the rest; its refusals become MXError.
#include <torch/extension.h>

#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/functions/basic_ops.h>

#include "mxmoe.h"

namespace {

using torch::Tensor;
using Maybe = std::optional<Tensor>;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

struct Refused : std::exception {
  const char* fn;
  int status;
  std::string text;
  Refused(const char* f, int s) : fn(f), status(s), text(mx_last_error()) {}
  const char* what() const noexcept override { return text.c_str(); }
};

void check(const char* fn, mx_status st) {
  if (st != MX_OK) throw Refused(fn, (int)st);
}

// In a backward there is no caller of the C ABI to hand a status to.
void check_backward(const char* fn, mx_status st) {
  TORCH_CHECK(st == MX_OK, fn, ": ", mx_last_error());
}

void* stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }
int type_of(const Tensor& t) { return t.scalar_type() == torch::kFloat ? MX_F32 : MX_BF16; }
const uint16_t* bf16(const Tensor& t) { return (const uint16_t*)t.data_ptr(); }
template <class T>
T* ptr(const Tensor& t) {
  return t.defined() ? (T*)t.data_ptr() : nullptr;
}

// Gradients made while a graph of them is asked for (create_graph=True): they
// refuse to be differentiated, as there is no second derivative here.
variable_list first_order(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  for (auto& g : grads)
    if (g.defined()) g = g.detach().set_requires_grad(true);
  auto refuse = std::make_shared<torch::autograd::DelayedError>(
      "this gradient has no derivative of its own (the kernels compute first derivatives)", (int64_t)grads.size());
  return (*refuse)(std::move(grads));
}

bool wants_grad(const Tensor& t) { return at::GradMode::is_enabled() && t.requires_grad(); }
// Whether a call needs a node: for a gradient, or for an operand with a tangent (forward mode),
// which the nodes refuse.
bool traced(const Tensor& t) { return wants_grad(t) || t._fw_grad(0).defined(); }

// A leaf's gradient is accumulated on the stream on which the leaf first entered a
// living graph.  Where that is not the stream being captured, a captured backward
// would make a stream outside the capture wait for one inside, and the failure of
// that ends the process: refuse such a leaf while it is still an ordinary error.  To be
// called before the node is made, which takes the leaf into the new graph.
void check_capture(const Tensor& t) {
  if (!wants_grad(t) || !t.is_leaf() ||
      c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None)
    return;
  const auto node = torch::autograd::impl::try_get_grad_accumulator(t);
  if (!node) return;
  const auto stream = node->stream();
  TORCH_CHECK(!stream || stream->id() == c10::hip::getCurrentHIPStream(t.device().index()).id(),
              "captured into a graph while a graph of the same leaf from another stream lives: its backward could not "
              "be captured (drop the results of the eager calls first, or detach)");
}

// At an address that the kernels' wide loads take (views of a longer tensor may lie anywhere).
bool wide(const Tensor& t) { return (uintptr_t)t.data_ptr() % 16 == 0; }
// A gradient as the kernels read it.
Tensor dense(const Tensor& t) {
  const Tensor c = t.contiguous();
  return wide(c) ? c : c.clone();
}

bool fits(const Tensor& t, at::ScalarType type, const Tensor& with) {
  return t.is_cuda() && t.scalar_type() == type && t.is_contiguous() && t.device() == with.device();
}
bool fits(const Maybe& t, at::ScalarType type, const Tensor& with) { return !t || fits(*t, type, with); }
bool fits_either(const Tensor& t) {
  return t.is_cuda() && t.is_contiguous() && (t.scalar_type() == torch::kFloat || t.scalar_type() == torch::kBFloat16);
}
// Logits as the router reads them: four at a time, or one by one.
bool starts_a_row(const Tensor& t) {
  return (uintptr_t)t.data_ptr() % ((t.size(1) % 4 == 0 ? 4 : 1) * t.element_size()) == 0;
}
bool shaped(const Tensor& t, std::initializer_list<int64_t> shape) { return t.sizes() == at::IntArrayRef(shape); }

// Operands that stand for rows of routed items, M of them: how many items there are, or
// nothing where they do not fit (see _rows_of in the binding).
std::optional<int64_t> items_of(const Tensor& x, const Maybe& rows, const Maybe& combine, int64_t M) {
  if (!fits(rows, torch::kInt, x) || !fits(combine, torch::kFloat, x)) return std::nullopt;
  if (!rows) return combine && combine->numel() != M ? std::nullopt : std::optional<int64_t>(M);
  if (!shaped(*rows, {M})) return std::nullopt;
  return combine ? combine->numel() : ((int64_t)1 << 31) - 1;
}

// The operators without a node, for calls with no gradient to compute (a node costs a
// microsecond).
std::pair<Tensor, Tensor> run_router(const Tensor& logits, int64_t k, int64_t score, const Maybe& bias, int64_t groups,
                                     int64_t topk_groups, int64_t group_score, bool renormalize, double scale) {
  const int64_t T = logits.size(0), E = logits.size(1);
  Tensor ids = torch::empty({T, k}, logits.options().dtype(torch::kInt32));
  Tensor combine = torch::empty({T, k}, logits.options().dtype(torch::kFloat));
  check("mx_topk_router_fwd",
        mx_topk_router_fwd(logits.data_ptr(), type_of(logits), bias ? ptr<float>(*bias) : nullptr, T, E, k, (int)score,
                           groups, topk_groups, (int)group_score, renormalize, (float)scale, ptr<int32_t>(ids),
                           ptr<float>(combine), stream_of(logits)));
  return {ids, combine};
}

Tensor run_swiglu(const Tensor& gu, const Tensor& kept, const Tensor& kept_s) {
  const int64_t M = gu.size(0), N = gu.size(1) / 2;
  Tensor h = torch::empty({M, N}, gu.options());
  check("mx_swiglu_fwd", mx_swiglu_fwd(bf16(gu), M, N, ptr<uint16_t>(h), ptr<uint8_t>(kept), ptr<uint8_t>(kept_s),
                                       stream_of(gu)));
  return h;
}

Tensor run_combine(const Tensor& y, const Tensor& combine, const Maybe& pos) {
  const int64_t T = y.size(0), k = y.size(1), N = y.size(2);
  Tensor out = torch::empty({T, N}, y.options().dtype(torch::kBFloat16));
  check("mx_topk_combine_fwd", mx_topk_combine_fwd(y.data_ptr(), type_of(y), ptr<float>(combine),
                                                   pos ? ptr<int32_t>(*pos) : nullptr, T, k, N, ptr<uint16_t>(out),
                                                   stream_of(y)));
  return out;
}

struct Router : torch::autograd::Function<Router> {
  static variable_list forward(AutogradContext* ctx, const Tensor& logits, int64_t k, int64_t score, const Maybe& bias,
                               int64_t groups, int64_t topk_groups, int64_t group_score, bool renormalize,
                               double scale) {
    const auto [ids, combine] = run_router(logits, k, score, bias, groups, topk_groups, group_score, renormalize, scale);
    ctx->mark_non_differentiable({ids});
    ctx->set_materialize_grads(false);       // no zeros in the place of a gradient of the ids
    ctx->save_for_backward({logits, ids, combine});
    ctx->saved_data["score"] = score;
    ctx->saved_data["renormalize"] = renormalize;
    ctx->saved_data["scale"] = scale;
    return {ids, combine};
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    variable_list out(9);
    if (!grads[1].defined()) return out;
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &logits = saved[0], &ids = saved[1], &combine = saved[2], d = grads[1].contiguous();
    out[0] = torch::empty_like(logits);
    check_backward("mx_topk_router_bwd",
                   mx_topk_router_bwd(logits.data_ptr(), type_of(logits), ptr<int32_t>(ids), ptr<float>(combine),
                                      ptr<float>(d), logits.size(0), logits.size(1), ids.size(1),
                                      (int)ctx->saved_data["score"].toInt(), ctx->saved_data["renormalize"].toBool(),
                                      (float)ctx->saved_data["scale"].toDouble(), out[0].data_ptr(),
                                      stream_of(logits)));
    return first_order(std::move(out));
  }
};

struct Swiglu : torch::autograd::Function<Swiglu> {
  static Tensor forward(AutogradContext* ctx, const Tensor& gu) {
    const int64_t M = gu.size(0), N = gu.size(1) / 2;
    Tensor kept = torch::empty({M, 2 * N}, gu.options().dtype(torch::kByte));
    Tensor kept_s = torch::empty({M, 2 * N / 32}, gu.options().dtype(torch::kByte));
    Tensor h = run_swiglu(gu, kept, kept_s);
    ctx->save_for_backward({kept, kept_s});
    return h;
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor d = dense(grads[0]);
    const int64_t M = d.size(0), N = d.size(1);
    Tensor dgu = torch::empty({M, 2 * N}, d.options());
    check_backward("mx_swiglu_bwd", mx_swiglu_bwd(bf16(d), ptr<uint8_t>(saved[0]), ptr<uint8_t>(saved[1]), M, N,
                                                  ptr<uint16_t>(dgu), stream_of(d)));
    return first_order({dgu});
  }
};

struct Combine : torch::autograd::Function<Combine> {
  static Tensor forward(AutogradContext* ctx, const Tensor& y, const Tensor& combine, const Maybe& pos) {
    Tensor out = run_combine(y, combine, pos);
    ctx->save_for_backward({y, combine, pos ? *pos : Tensor()});
    return out;
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &y = saved[0], &combine = saved[1], &pos = saved[2], d = dense(grads[0]);
    Tensor dy, dcombine;
    if (ctx->needs_input_grad(0)) dy = torch::empty_like(y);
    if (ctx->needs_input_grad(1)) dcombine = torch::empty_like(combine);
    check_backward("mx_topk_combine_bwd",
                   mx_topk_combine_bwd(y.data_ptr(), type_of(y), ptr<float>(combine), ptr<int32_t>(pos), bf16(d),
                                       y.size(0), y.size(1), y.size(2), ptr<void>(dy), ptr<float>(dcombine),
                                       stream_of(y)));
    return first_order({dy, dcombine, Tensor()});
  }
};

Tensor bytes(const Tensor& like, std::initializer_list<int64_t> shape) {
  return torch::empty(shape, like.options().dtype(torch::kByte));
}

// layout: of the scales, as in the C ABI.
Maybe dequantize(const Tensor& q, const Tensor& s, int64_t layout) {
  if (!fits(q, torch::kByte, q) || !fits(s, torch::kByte, q) || q.dim() < 2 || q.dim() > 3 || s.dim() < 2 || layout < 0)
    return std::nullopt;
  const int64_t B = q.dim() == 3 ? q.size(0) : 1, R = q.size(-2), C = q.size(-1);
  const bool gemm = layout == MX_SCALES_GEMM;
  if (C % (gemm ? 128 : 32) != 0) return std::nullopt;
  std::vector<int64_t> shape;
  if (q.dim() == 3) shape.push_back(B);
  shape.insert(shape.end(), {gemm ? C / 128 : R, gemm ? R : C / 32});
  if (gemm) shape.push_back(4);
  if (s.sizes() != at::IntArrayRef(shape)) return std::nullopt;
  const c10::DeviceGuard on(q.device());
  Tensor out = torch::empty(q.sizes(), q.options().dtype(torch::kBFloat16));
  check("mx_dequantize", mx_dequantize(ptr<uint8_t>(q), ptr<uint8_t>(s), B, R, C, (int)layout, ptr<uint16_t>(out),
                                       stream_of(q)));
  return out;
}

bool fits_halves(const Tensor& gu) { return fits(gu, torch::kBFloat16, gu) && gu.dim() == 2 && gu.size(1) % 2 == 0; }
int64_t up_to_128(int64_t M) { return (M + 127) / 128 * 128; }

std::optional<std::pair<Tensor, Tensor>> swiglu_quantize(const Tensor& gu, const Maybe& rows) {
  if (!fits_halves(gu)) return std::nullopt;
  const int64_t M = gu.size(0), N = gu.size(1) / 2;
  const auto n = items_of(gu, rows, std::nullopt, M);
  if (!n) return std::nullopt;
  const c10::DeviceGuard on(gu.device());
  Tensor q = bytes(gu, {M, N}), s = bytes(gu, {N / 128, M, 4});
  check("mx_swiglu_quantize", mx_swiglu_quantize(bf16(gu), rows ? ptr<int32_t>(*rows) : nullptr, *n, M, N,
                                                 ptr<uint8_t>(q), ptr<uint8_t>(s), stream_of(gu)));
  return std::make_pair(q, s);
}

using Six = std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor, Tensor>;
using Five = std::tuple<Tensor, Tensor, Tensor, Tensor, Maybe>;

std::optional<Six> swiglu_quantize_fwd(const Tensor& gu, const Maybe& rows, const Maybe& combine,
                                       std::optional<int64_t> given_ldq) {
  if (!fits_halves(gu)) return std::nullopt;
  const int64_t M = gu.size(0), N = gu.size(1) / 2, ldq = given_ldq.value_or(up_to_128(M));
  const auto n = items_of(gu, rows, combine, M);
  if (!n || ldq < 0) return std::nullopt;
  const c10::DeviceGuard on(gu.device());
  Tensor q = bytes(gu, {M, N}), s = bytes(gu, {N / 128, M, 4}), q_t = bytes(gu, {N, ldq});
  Tensor s_t = bytes(gu, {ldq / 128, N, 4}), kept = bytes(gu, {M, 2 * N}), kept_s = bytes(gu, {2 * N / 128, M, 4});
  check("mx_swiglu_quantize_fwd",
        mx_swiglu_quantize_fwd(bf16(gu), rows ? ptr<int32_t>(*rows) : nullptr, combine ? ptr<float>(*combine) : nullptr,
                               *n, M, N, ldq, ptr<uint8_t>(q), ptr<uint8_t>(s), ptr<uint8_t>(q_t), ptr<uint8_t>(s_t),
                               ptr<uint8_t>(kept), ptr<uint8_t>(kept_s), stream_of(gu)));
  return Six(q, s, q_t, s_t, kept, kept_s);
}

std::optional<Five> swiglu_quantize_bwd(const Tensor& dh, const Tensor& kept, const Tensor& kept_s, const Maybe& rows,
                                        const Maybe& given_pos, const Maybe& combine, std::optional<int64_t> given_ldq) {
  if (!fits(dh, torch::kBFloat16, dh) || dh.dim() != 2 || !fits(kept, torch::kByte, dh) || !fits(kept_s, torch::kByte, dh))
    return std::nullopt;
  const int64_t M = dh.size(0), N = dh.size(1), ldq = given_ldq.value_or(up_to_128(M));
  const auto n = items_of(dh, rows, combine, M);
  if (!n || ldq < 0 || !shaped(kept, {M, 2 * N}) || !shaped(kept_s, {2 * N / 128, M, 4})) return std::nullopt;
  const Maybe pos = combine ? given_pos : std::nullopt;
  if (combine && (rows.has_value() != pos.has_value() || (pos && (!fits(pos, torch::kInt, dh) || pos->numel() != *n))))
    return std::nullopt;
  const c10::DeviceGuard on(dh.device());
  Tensor q = bytes(dh, {M, 2 * N}), s = bytes(dh, {2 * N / 128, M, 4}), q_t = bytes(dh, {2 * N, ldq});
  Tensor s_t = bytes(dh, {ldq / 128, 2 * N, 4}), dcombine, ws;
  if (combine) {
    dcombine = torch::empty_like(*combine);
    ws = bytes(dh, {(int64_t)mx_swiglu_quantize_workspace_bytes(M, N)});
  }
  check("mx_swiglu_quantize_bwd",
        mx_swiglu_quantize_bwd(bf16(dh), ptr<uint8_t>(kept), ptr<uint8_t>(kept_s),
                               rows ? ptr<int32_t>(*rows) : nullptr, pos ? ptr<int32_t>(*pos) : nullptr,
                               combine ? ptr<float>(*combine) : nullptr, *n, M, N, ldq, ptr<uint8_t>(q),
                               ptr<uint8_t>(s), ptr<uint8_t>(q_t), ptr<uint8_t>(s_t), ptr<float>(dcombine),
                               ptr<void>(ws), ws.defined() ? (size_t)ws.numel() : 0, stream_of(dh)));
  return Five(q, s, q_t, s_t, dcombine.defined() ? Maybe(dcombine) : std::nullopt);
}

std::optional<std::pair<Tensor, Tensor>> topk_router(const Tensor& logits, int64_t k, int64_t score, const Maybe& bias,
                                                     int64_t groups, int64_t topk_groups, int64_t group_score,
                                                     bool renormalize, double scale) {
  if (!fits_either(logits) || logits.dim() != 2 || !starts_a_row(logits) || k < 0 || k > MX_MOE_MAX_TOPK || score < 0 || group_score < 0)
    return std::nullopt;
  if (bias && (!fits(bias, torch::kFloat, logits) || !shaped(*bias, {logits.size(1)}) ||
               wants_grad(*bias)))
    return std::nullopt;
  const c10::DeviceGuard on(logits.device());
  if (!traced(logits) && !(bias && traced(*bias)))
    return run_router(logits, k, score, bias, groups, topk_groups, group_score, renormalize, scale);
  check_capture(logits);
  const variable_list out = Router::apply(logits, k, score, bias, groups, topk_groups, group_score, renormalize, scale);
  return std::make_pair(out[0], out[1]);
}

Maybe swiglu(const Tensor& gu) {
  if (!fits_halves(gu) || !wide(gu)) return std::nullopt;
  const c10::DeviceGuard on(gu.device());
  if (!traced(gu)) return run_swiglu(gu, Tensor(), Tensor());
  check_capture(gu);
  return Swiglu::apply(gu);
}

Maybe topk_combine(const Tensor& y, const Tensor& combine, const Maybe& pos) {
  if (!fits_either(y) || y.dim() != 3 || !wide(y) || !fits(combine, torch::kFloat, y) || !shaped(combine, {y.size(0), y.size(1)}) ||
      !fits(pos, torch::kInt, y) || (pos && pos->numel() != combine.numel()))
    return std::nullopt;
  const c10::DeviceGuard on(y.device());
  if (!traced(y) && !traced(combine)) return run_combine(y, combine, pos);
  check_capture(y);
  check_capture(combine);
  return Combine::apply(y, combine, pos);
}

}  // namespace

PYBIND11_MODULE(_nodes, m) {
  static py::object error;
  // MXError of the package
  m.def("set_error", [](py::object cls) { error = std::move(cls); });
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const Refused& r) {
      PyErr_SetObject(error.ptr(), error(r.fn, r.status, r.text).ptr());
    }
  });
  using no_gil = py::call_guard<py::gil_scoped_release>;
  m.def("topk_router", &topk_router, no_gil());
  m.def("swiglu", &swiglu, no_gil());
  m.def("topk_combine", &topk_combine, no_gil());
  m.def("check_capture", &check_capture, no_gil());
  m.def("traced", &traced, no_gil());
  m.def("dequantize", &dequantize, no_gil());
  m.def("swiglu_quantize", &swiglu_quantize, no_gil());
  m.def("swiglu_quantize_fwd", &swiglu_quantize_fwd, no_gil());
  m.def("swiglu_quantize_bwd", &swiglu_quantize_bwd, no_gil());
}
