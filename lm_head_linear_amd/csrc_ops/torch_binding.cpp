// torch_binding.cpp -- the allocating conveniences of the operators next to
// the losses, on torch tensors: check, allocate outputs and workspace, call
// the C entry point on torch's current stream.  Every step of the computation
// runs in liblce.so; this only marshals.
//
// It is compiled because the shortest calls are bound by the host: one token
// through a 1024 x 1024 layer is 5 us of GPU time, and marshalling it through
// ctypes took 8.8 us besides the launch.
//
// Each function returns (status, outputs...); a tensor that does not fit
// raises ValueError.
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/extension.h>

#include <optional>
#include <string>
#include <vector>

#include "../../include/lce.h"

namespace py = pybind11;
using at::Tensor;
typedef std::optional<Tensor> MaybeTensor;

namespace {

int32_t dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return LCE_BF16;
    case at::kHalf: return LCE_F16;
    case at::kFloat: return LCE_F32;
    case at::kDouble: return LCE_F64;
    case at::kLong: return LCE_I64;
    case at::kByte: return LCE_U8;
    case at::kBool: return LCE_U8;
    default: return 0;
  }
}

void need(bool ok, const char *what) {
  if (!ok) throw py::value_error(what);
}

// A tensor that was given has to have the shape, not only the elements: one in
// another order would be read or written wrongly.
bool fits(const MaybeTensor &t, int64_t rows, int64_t cols) {
  return !t || (t->dim() == 2 && t->size(0) == rows && t->size(1) == cols);
}
int64_t pack8_blocks(int64_t d) { return (d + LCE_PACK8_BLOCK - 1) / LCE_PACK8_BLOCK; }

// The descriptor of a contiguous tensor on the GPU of the call.
struct On {
  c10::Device device;
  explicit On(const Tensor &t) : device(t.device()) {
    need(device.is_cuda(), "tensors must be on a GPU");
  }
  lce_tensor operator()(const Tensor &t) const {
    need(t.device() == device, "tensors must be on one GPU");
    need(t.is_contiguous(), "tensors must be contiguous");
    return {t.data_ptr(), t.numel(), dtype_code(t.scalar_type())};
  }
  lce_tensor operator()(const MaybeTensor &t) const {
    return t ? (*this)(*t) : lce_tensor{nullptr, 0, 0};
  }
  Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
  }
  // Scratch of `bytes` (a query's answer) unless the caller brought some.
  // Freed on return: the allocator hands it on in stream order.
  Tensor scratch(const MaybeTensor &given, int64_t bytes) const {
    if (given) return *given;
    return bytes > 0 ? empty({bytes}, at::kByte) : Tensor();
  }
  void *stream() const { return c10::hip::getCurrentHIPStream(device.index()).stream(); }
};

lce_tensor scratch_desc(const On &on, const Tensor &t) {
  return t.defined() ? on(t) : lce_tensor{nullptr, 0, 0};
}

py::tuple pack8(const Tensor &x) {
  need(x.dim() == 2, "x must be two-dimensional");
  const On on(x);
  const c10::DeviceGuard guard(on.device);
  const int64_t n = x.size(0), d = x.size(1);
  Tensor codes = on.empty({n, d}, at::kByte);
  Tensor scales = on.empty({n, pack8_blocks(d)}, at::kByte);
  const lce_tensor tx = on(x);
  lce_tensor tc = on(codes), ts = on(scales);
  const int32_t st = lce_pack8(&tx, n, d, &tc, &ts, on.stream());
  return py::make_tuple(st, std::move(codes), std::move(scales));
}

py::tuple unpack8(const Tensor &codes, const Tensor &scales, at::ScalarType dtype) {
  need(codes.dim() == 2, "codes must be two-dimensional");
  need(fits(scales, codes.size(0), pack8_blocks(codes.size(1))), "scales do not fit their codes");
  const On on(codes);
  const c10::DeviceGuard guard(on.device);
  const int64_t n = codes.size(0), d = codes.size(1);
  Tensor out = on.empty({n, d}, dtype);
  const lce_tensor tc = on(codes), ts = on(scales);
  lce_tensor to = on(out);
  const int32_t st = lce_unpack8(&tc, &ts, n, d, &to, on.stream());
  return py::make_tuple(st, std::move(out));
}

py::tuple linear(const Tensor &x, const Tensor &weight, const MaybeTensor &bias,
                 const MaybeTensor &residual, int32_t activation, bool want_preact,
                 std::optional<at::ScalarType> out_dtype, const MaybeTensor &workspace) {
  need(x.dim() == 2 && weight.dim() == 2, "x and weight must be two-dimensional");
  const int64_t n = x.size(0), d_in = x.size(1), d_out = weight.size(0);
  need(weight.size(1) == d_in && (!bias || bias->numel() == d_out) &&
           (!residual || (residual->dim() == 2 && residual->size(0) == n &&
                          residual->size(1) == d_out)),
       "weight, bias or residual does not fit x");
  const On on(x);
  const c10::DeviceGuard guard(on.device);
  const at::ScalarType dtype = x.scalar_type();
  const lce_tensor tx = on(x), tw = on(weight), tb = on(bias), tr = on(residual);
  const int64_t bytes = lce_linear_workspace_bytes(n, d_in, d_out, dtype_code(dtype));
  if (bytes < 0) return py::make_tuple(int32_t(-bytes), py::none(), py::none());
  Tensor ws = on.scratch(workspace, bytes);
  Tensor out = on.empty({n, d_out}, out_dtype.value_or(dtype));
  MaybeTensor preact;
  if (want_preact) preact = on.empty({n, d_out}, dtype);
  lce_tensor tp = on(preact), to = on(out), tws = scratch_desc(on, ws);
  const int32_t st = lce_linear(&tx, &tw, &tb, &tr, n, d_in, d_out, activation, &tp, &to, &tws,
                                on.stream());
  return py::make_tuple(st, std::move(out), std::move(preact));
}

py::tuple linear_backward(const Tensor &d_out_grad, const MaybeTensor &x, const MaybeTensor &x_scales,
                          const MaybeTensor &weight, const MaybeTensor &preact,
                          const MaybeTensor &preact_scales, int32_t activation, bool want_x,
                          bool want_weight, bool want_bias, at::ScalarType weight_dtype,
                          const MaybeTensor &d_weight_in, const MaybeTensor &d_bias_in,
                          bool accumulate, const MaybeTensor &workspace) {
  need(d_out_grad.dim() == 2 && (!x || x->dim() == 2) && (!weight || weight->dim() == 2),
       "d_out, x and weight must be two-dimensional");
  need(x || weight, "x or weight is needed");
  const int64_t n = d_out_grad.size(0), m = d_out_grad.size(1);
  const int64_t d_in = weight ? weight->size(1) : x->size(1);
  need((!x || (x->size(0) == n && x->size(1) == d_in)) && (!weight || weight->size(0) == m),
       "x or weight does not fit d_out");
  // (what is not read or written may have any shape)
  const bool slope = activation != LCE_ACT_NONE;
  need(!slope || fits(preact, n, m), "preact does not fit d_out");
  need((!want_weight || fits(x_scales, n, pack8_blocks(d_in))) &&
           (!slope || fits(preact_scales, n, pack8_blocks(m))),
       "scales do not fit their codes");
  need(!want_weight || fits(d_weight_in, m, d_in), "d_weight does not fit weight");
  need(!want_bias || !d_bias_in || d_bias_in->numel() == m, "d_bias does not fit d_out");
  need(!accumulate || ((!want_weight || d_weight_in) && (!want_bias || d_bias_in)),
       "accumulate needs the gradients it adds to");
  const On on(d_out_grad);
  const c10::DeviceGuard guard(on.device);
  const at::ScalarType dtype = d_out_grad.scalar_type();
  const lce_tensor tg = on(d_out_grad), tx = on(x), txs = on(x_scales), tw = on(weight);
  const lce_tensor tz = on(preact), tzs = on(preact_scales);
  const int64_t bytes = lce_linear_backward_workspace_bytes(n, d_in, m, dtype_code(dtype));
  if (bytes < 0) return py::make_tuple(int32_t(-bytes), py::none(), py::none(), py::none());
  Tensor ws = on.scratch(workspace, bytes);
  MaybeTensor d_x, d_weight, d_bias;
  if (want_x) d_x = on.empty({n, d_in}, dtype);
  if (want_weight) d_weight = d_weight_in ? *d_weight_in : on.empty({m, d_in}, weight_dtype);
  if (want_bias) d_bias = d_bias_in ? *d_bias_in : on.empty({m}, at::kFloat);
  lce_tensor tdx = on(d_x), tdw = on(d_weight), tdb = on(d_bias), tws = scratch_desc(on, ws);
  const int32_t st = lce_linear_backward(&tg, &tx, &txs, &tw, &tz, &tzs, n, d_in, m, activation,
                                         &tdx, &tdw, &tdb, accumulate, &tws, on.stream());
  return py::make_tuple(st, std::move(d_x), std::move(d_weight), std::move(d_bias));
}

py::tuple beam_select(const Tensor &logits, const Tensor &scores, int64_t n_out,
                      const MaybeTensor &finished, const MaybeTensor &allowed, int64_t eos,
                      const MaybeTensor &workspace) {
  need(logits.dim() == 2 && scores.dim() == 2, "logits and scores must be two-dimensional");
  const int64_t n_seq = scores.size(0), beams = scores.size(1), vocab = logits.size(1);
  need(logits.size(0) == n_seq * beams, "logits need one row per beam");
  need(!finished || fits(finished, n_seq, beams) ||
           (finished->dim() == 1 && finished->size(0) == n_seq * beams),
       "finished does not fit scores");
  need(!allowed || fits(allowed, n_seq * beams, vocab) ||
           (allowed->dim() == 3 && allowed->size(0) == n_seq && allowed->size(1) == beams &&
            allowed->size(2) == vocab),
       "allowed does not fit logits");
  const On on(logits);
  const c10::DeviceGuard guard(on.device);
  const lce_tensor tl = on(logits), ts = on(scores), tf = on(finished), ta = on(allowed);
  const int64_t bytes = lce_beam_workspace_bytes(n_seq, beams, vocab, n_out);
  if (bytes < 0)
    return py::make_tuple(int32_t(-bytes), py::none(), py::none(), py::none(), py::none());
  Tensor ws = on.scratch(workspace, bytes);
  Tensor best = on.empty({n_seq, n_out}, at::kFloat);
  Tensor parents = on.empty({n_seq, n_out}, at::kLong), tokens = on.empty({n_seq, n_out}, at::kLong);
  Tensor done = on.empty({n_seq, n_out}, at::kBool);
  lce_tensor tb = on(best), tp = on(parents), tt = on(tokens), td = on(done);
  lce_tensor tws = scratch_desc(on, ws);
  const int32_t st = lce_beam_select(&tl, &ts, &tf, &ta, n_seq, beams, vocab, n_out, eos, &tb, &tp,
                                     &tt, &td, &tws, on.stream());
  return py::make_tuple(st, std::move(best), std::move(parents), std::move(tokens), std::move(done));
}

int32_t beam_reorder(const std::vector<Tensor> &states, const Tensor &parents, int64_t beams,
                     const std::vector<Tensor> &out, std::optional<int64_t> length, int64_t dim) {
  need(!states.empty() && states.size() == out.size(),
       "as many destinations as sources are needed, and one at least");
  need(parents.dim() == 2 && states[0].dim() >= 1, "parents must be two-dimensional");
  const int64_t n_seq = parents.size(0), n_out = parents.size(1);
  const at::IntArrayRef shape = states[0].sizes().slice(1);
  const On on(parents);
  const c10::DeviceGuard guard(on.device);
  std::vector<lce_tensor> src, dst;
  for (size_t i = 0; i < states.size(); ++i) {
    need(states[i].dim() >= 1 && out[i].dim() >= 1 && states[i].size(0) == n_seq * beams &&
             out[i].size(0) == n_seq * n_out && states[i].sizes().slice(1) == shape &&
             out[i].sizes().slice(1) == shape,
         "states need one shape and one row per beam");
    src.push_back(on(states[i]));
    dst.push_back(on(out[i]));
  }
  int64_t segs = 1, elems = 1, stride = 1;
  if (length) {
    need(dim >= 1 && dim <= int64_t(shape.size()) && *length >= 0 && *length <= shape[dim - 1],
         "length is outside the dimension");
    int64_t inner = 1;
    for (int64_t i = 0; i < int64_t(shape.size()); ++i) (i < dim - 1 ? segs : inner) *= shape[i];
    stride = inner;
    elems = shape[dim - 1] ? inner / shape[dim - 1] * *length : 0;
  } else {
    for (const int64_t s : shape) elems *= s;
    stride = elems;
  }
  const lce_tensor tp = on(parents);
  return lce_beam_reorder(src.data(), dst.data(), int32_t(src.size()), &tp, n_seq, beams, n_out,
                          segs, elems, stride, on.stream());
}

}  // namespace

PYBIND11_MODULE(_lce_torch, m) {
  m.def("pack8", &pack8);
  m.def("unpack8", &unpack8);
  m.def("linear", &linear);
  m.def("linear_backward", &linear_backward);
  m.def("beam_select", &beam_select);
  m.def("beam_reorder", &beam_reorder);
}
