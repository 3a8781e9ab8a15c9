// binding.cpp -- the Python calls of the channel-wise operators, as one native
// call each: operand checks, output allocation, the device's current stream and
// the C ABI (conv3d.h).  Through ctypes a small layer norm or product spent 10 to
// 18 us on the host, several times what the kernel takes; here it is about the
// cost of a torch operator.  Marshalling only: no arithmetic happens in torch.
//
// Wrong operands raise ValueError or TypeError; a status from the library raises
// the exception class that the package hands over (set_error_class).
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/utils/pybind.h>

#include <climits>
#include <optional>
#include <string>
#include <tuple>

#include "conv3d.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;
using OptStream = std::optional<int64_t>;

namespace {

// An uninitialised tensor from torch's caching allocator, without the
// dispatcher's round (a third of a microsecond for each output).
Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
  return Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

PyObject* g_error_class = nullptr;   // held for the life of the process

void check_status(conv3d_status_t st) {
  if (st == CONV3D_OK) return;
  const std::string text = std::string(conv3d_status_string(st)) + ": " + conv3d_last_error();
  TORCH_CHECK(g_error_class != nullptr, text);
  py::object e = py::reinterpret_borrow<py::object>(g_error_class)(static_cast<int>(st), text);
  PyErr_SetObject(g_error_class, e.ptr());
  throw py::error_already_set();
}

// A call's leading operand: a contiguous [..., C] CUDA tensor of a 16-bit type.
struct Lead {
  const Tensor& t;
  long long rows;
  int C;
  c10::Device device;
  at::ScalarType type;
  conv3d_dtype_t code;

  Lead(const char* name, const Tensor& x) : t(x), rows(0), C(0), device(x.device()), type(x.scalar_type()) {
    TORCH_CHECK_VALUE(x.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(x.dim() >= 1 && x.is_contiguous(), name, " must be a contiguous [..., C] tensor");
    code = dtype_code(type);
    C = narrow(x.size(-1));
    rows = C > 0 ? x.numel() / C : 0;
  }
  static conv3d_dtype_t dtype_code(at::ScalarType t) {
    TORCH_CHECK_TYPE(t == at::kBFloat16 || t == at::kHalf, "libconv3d computes in bf16 or fp16, got ", t);
    return t == at::kBFloat16 ? CONV3D_BF16 : CONV3D_F16;
  }
  static int narrow(int64_t n) {
    TORCH_CHECK_VALUE(n <= INT_MAX, "an extent of ", n, " is too large");
    return static_cast<int>(n);
  }
  // the leading extents with another last one
  at::DimVector with(int64_t last) const {
    at::DimVector s(t.sizes().begin(), t.sizes().end());
    s.back() = last;
    return s;
  }
  at::IntArrayRef lead() const { return t.sizes().slice(0, t.dim() - 1); }
  Tensor empty(at::IntArrayRef shape, at::ScalarType type_) const { return new_tensor(shape, type_, device); }
  Tensor empty(at::IntArrayRef shape) const { return new_tensor(shape, type, device); }
};

// One more operand on the leading one's device; returns its address.
void* operand(const char* name, const Tensor& t, const c10::Device& device, at::ScalarType type, at::IntArrayRef shape) {
  TORCH_CHECK_VALUE(t.device() == device, name, " must be a CUDA tensor on ", device, ", got ", t.device());
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " has dtype ", t.scalar_type(), ", expected ", type);
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must be ", shape, ", got ", t.sizes());
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return t.data_ptr();
}
void* operand(const char* name, const OptTensor& t, const Lead& l, at::IntArrayRef shape) {
  return t.has_value() ? operand(name, *t, l.device, l.type, shape) : nullptr;
}

// A tensor of the caller's that the call writes: autograd is told, as torch's own
// in-place operators tell it, so that a backward pass which saved it notices.
void overwritten(const OptTensor& t) {
  if (t.has_value() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

struct Act8 {
  void* codes;
  void* exponents;
};
// A checkpoint of a tensor of `shape`.
Act8 checkpoint(const char* name, const Tensor& codes, const Tensor& exponents, int64_t channels,
                const c10::Device& device, at::IntArrayRef shape) {
  TORCH_CHECK_VALUE(channels == shape.back(), name, " holds ", channels, " channels, expected ", shape.back());
  const int64_t blocks = (channels + 31) / 32;
  at::DimVector s(shape.begin(), shape.end());
  s.back() = blocks * 32;
  void* c = operand((std::string(name) + ".codes").c_str(), codes, device, at::kChar, s);
  s.back() = blocks;
  return {c, operand((std::string(name) + ".exponents").c_str(), exponents, device, at::kByte, s)};
}

// The call's device and stream, which become the current ones while it lasts, so
// that what it allocates belongs to the stream its kernels run on: a temporary
// freed at its end is not handed to other streams before they have.
//
// CUDA's own handles of the default streams: 1 is the legacy one, which torch
// knows as 0; 2 is the calling thread's, which torch's allocator cannot keep
// blocks for (one handle, another stream in every thread).  Memory comes from the
// current stream there, whose earlier work the thread's stream waits for (it may
// still use a block), and whose later work waits for the call (it may get one).
struct On {
  c10::cuda::CUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard current;
  CUstream_st* stream;
  On(const c10::Device& d, const OptStream& s) : device(d.index()) {
    if (!s.has_value()) {
      stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
      return;
    }
    stream = *s == 1 ? nullptr : reinterpret_cast<CUstream_st*>(*s);
    if (stream == cudaStreamPerThread) {
      CUstream_st* const memory = c10::cuda::getCurrentCUDAStream(d.index()).stream();
      C10_CUDA_CHECK(follow(stream, memory));
      lender = memory;
      lends = true;
    } else {
      current.reset_stream(c10::cuda::getStreamFromExternal(stream, d.index()));
    }
  }
  On(const On&) = delete;
  ~On() {
    if (lends && follow(lender, stream) != cudaSuccess) {
      // the order cannot be had on the device: have it here
      cudaGetLastError();
      cudaStreamSynchronize(stream);
    }
  }

 private:
  CUstream_st* lender = nullptr;   // the stream whose memory a call on handle 2 uses,
  bool lends = false;              // and whether there is one
  // What `later` is given from now on waits for what `earlier` was given before.
  static cudaError_t follow(cudaStream_t later, cudaStream_t earlier) {
    cudaEvent_t event;
    cudaError_t e = cudaEventCreateWithFlags(&event, cudaEventDisableTiming);
    if (e != cudaSuccess) return e;
    e = cudaEventRecord(event, earlier);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(later, event, 0);
    cudaEventDestroy(event);   // its resources go when it has completed
    return e;
  }
};

conv3d_act_t act_of(int act) { return static_cast<conv3d_act_t>(act); }

std::tuple<Tensor, Tensor> new_act8(const Lead& l, int64_t channels) {
  const int64_t blocks = (channels + 31) / 32;
  return {l.empty(l.with(blocks * 32), at::kChar), l.empty(l.with(blocks), at::kByte)};
}

std::tuple<Tensor, Tensor> act8_pack(const Tensor& x, const OptStream& stream) {
  const Lead l("x", x);
  const On on(l.device, stream);
  auto [codes, exponents] = new_act8(l, l.C);
  check_status(conv3d_act8_pack(x.data_ptr(), codes.data_ptr(), exponents.data_ptr(), l.rows, l.C, l.code, on.stream));
  return {codes, exponents};
}

Tensor act8_unpack(const Tensor& codes, const Tensor& exponents, int64_t channels, at::ScalarType type,
                   const OptTensor& gamma, const OptTensor& beta, int act, const OptTensor& y, const OptStream& stream) {
  TORCH_CHECK_VALUE(codes.is_cuda(), "a must hold CUDA tensors");
  TORCH_CHECK_VALUE(codes.dim() >= 1, "a.codes must be [..., 32 * blocks]");
  const c10::Device device = codes.device();
  const On on(device, stream);
  const conv3d_dtype_t code = Lead::dtype_code(type);
  at::DimVector shape(codes.sizes().begin(), codes.sizes().end());
  shape.back() = channels;
  const Act8 a = checkpoint("a", codes, exponents, channels, device, shape);
  Tensor out = y.has_value() ? *y : new_tensor(shape, type, device);
  if (y.has_value()) operand("y", *y, device, type, shape);
  const int C = Lead::narrow(channels);
  const void* g = gamma.has_value() ? operand("gamma", *gamma, device, type, {channels}) : nullptr;
  const void* b = beta.has_value() ? operand("beta", *beta, device, type, {channels}) : nullptr;
  check_status(conv3d_act8_unpack(a.codes, a.exponents, g, b, act_of(act), out.data_ptr(), C > 0 ? out.numel() / C : 0,
                                  C, code, on.stream));
  overwritten(y);
  return out;
}

Tensor act8_bwd(const Tensor& dy, const Tensor& codes, const Tensor& exponents, int64_t channels, int act,
                const OptTensor& dx, const OptStream& stream) {
  const Lead l("dy", dy);
  const On on(l.device, stream);
  const Act8 a = checkpoint("a", codes, exponents, channels, l.device, dy.sizes());
  operand("dx", dx, l, dy.sizes());
  Tensor out = dx.has_value() ? *dx : l.empty(dy.sizes());
  check_status(conv3d_act8_bwd(dy.data_ptr(), a.codes, a.exponents, act_of(act), out.data_ptr(), l.rows, l.C, l.code,
                               on.stream));
  overwritten(dx);
  return out;
}

// {y}, {y, mean, rstd} or {y, codes, exponents, rstd}
py::object layernorm(const Tensor& x, const OptTensor& gamma, const OptTensor& beta, double eps, bool with_stats,
                     bool checkpoint8, const OptTensor& y, const OptStream& stream) {
  TORCH_CHECK_VALUE(!(with_stats && checkpoint8), "with_stats and checkpoint8 exclude each other");
  const Lead l("x", x);
  const On on(l.device, stream);
  const void* g = operand("gamma", gamma, l, {l.C});
  const void* b = operand("beta", beta, l, {l.C});
  operand("y", y, l, x.sizes());
  Tensor out = y.has_value() ? *y : l.empty(x.sizes());
  Tensor mean, rstd, codes, exponents;
  if (with_stats || checkpoint8) rstd = l.empty(l.lead(), at::kFloat);
  if (with_stats) mean = l.empty(l.lead(), at::kFloat);
  if (checkpoint8) std::tie(codes, exponents) = new_act8(l, l.C);
  check_status(conv3d_layernorm_fwd(
      x.data_ptr(), g, b, out.data_ptr(), with_stats ? mean.data_ptr<float>() : nullptr,
      with_stats || checkpoint8 ? rstd.data_ptr<float>() : nullptr, checkpoint8 ? codes.data_ptr() : nullptr,
      checkpoint8 ? exponents.data_ptr() : nullptr, l.rows, l.C, static_cast<float>(eps), l.code, on.stream));
  overwritten(y);
  if (checkpoint8) return py::make_tuple(out, codes, exponents, rstd);
  if (with_stats) return py::make_tuple(out, mean, rstd);
  return py::cast(out);
}

// From x and mean, or from codes and exponents of `channels` channels.
std::tuple<Tensor, OptTensor, OptTensor> layernorm_bwd(const Tensor& dy, const OptTensor& x, const OptTensor& mean,
                                                       const OptTensor& codes, const OptTensor& exponents,
                                                       int64_t channels, const Tensor& rstd, const OptTensor& gamma,
                                                       const OptTensor& dres, bool with_params, const OptTensor& dx,
                                                       const OptTensor& workspace, const OptStream& stream) {
  const Lead l("dy", dy);
  Tensor ws;   // outlives `on`, which sees to it that its next owner waits
  const On on(l.device, stream);
  const void* r = operand("rstd", rstd, l.device, at::kFloat, l.lead());
  const void *xp = nullptr, *m = nullptr;
  Act8 a{nullptr, nullptr};
  if (codes.has_value()) {
    TORCH_CHECK_VALUE(!mean.has_value(), "mean belongs to x: a checkpoint holds the normalised values");
    a = checkpoint("saved", *codes, exponents.value(), channels, l.device, dy.sizes());
  } else {
    xp = operand("saved", x, l, dy.sizes());
    TORCH_CHECK_VALUE(mean.has_value(), "x needs its mean");
    m = operand("mean", *mean, l.device, at::kFloat, l.lead());
  }
  const void* g = operand("gamma", gamma, l, {l.C});
  const void* s = operand("dres", dres, l, dy.sizes());
  operand("dx", dx, l, dy.sizes());
  Tensor out = dx.has_value() ? *dx : l.empty(dy.sizes());
  Tensor dgamma, dbeta;
  size_t ws_bytes = 0;
  if (with_params) {
    dgamma = l.empty({l.C});
    dbeta = l.empty({l.C});
    if (workspace.has_value()) {
      TORCH_CHECK_VALUE(workspace->device() == l.device && workspace->is_contiguous(),
                        "workspace must be a contiguous CUDA tensor on ", l.device);
      ws = *workspace;
    } else {
      ws = l.empty({static_cast<int64_t>(conv3d_layernorm_bwd_workspace_bytes(l.rows, l.C))}, at::kByte);
    }
    ws_bytes = ws.nbytes();
  }
  check_status(conv3d_layernorm_bwd(dy.data_ptr(), xp, static_cast<const float*>(m), a.codes, a.exponents,
                                    static_cast<const float*>(r), g, s, out.data_ptr(),
                                    with_params ? dgamma.data_ptr() : nullptr, with_params ? dbeta.data_ptr() : nullptr,
                                    l.rows, l.C, l.code, with_params ? ws.data_ptr() : nullptr, ws_bytes, on.stream));
  overwritten(dx);
  if (!with_params) return {out, std::nullopt, std::nullopt};
  return {out, dgamma, dbeta};
}

// A [N, K] weight, or a 1x1x1 convolution's [N, 1, 1, 1, K]; n < 0: any N.
const void* weight(const Tensor& w, const Lead& l, int64_t K, int64_t n) {
  const auto s = w.sizes();
  const bool ok = (s.size() == 2 || (s.size() == 5 && s[1] == 1 && s[2] == 1 && s[3] == 1)) && s.back() == K &&
                  (n < 0 || s[0] == n);
  TORCH_CHECK_VALUE(ok, "w must be [", n < 0 ? std::string("N") : std::to_string(n), ", ", K, "] (or with 1, 1, 1 between), got ", s);
  return operand("w", w, l.device, l.type, s);
}

// {y} or {y, codes, exponents}
py::object linear(const Tensor& x, const Tensor& w, const OptTensor& bias, const OptTensor& residual, int act,
                  bool checkpoint8, const OptTensor& y, const OptStream& stream) {
  const Lead l("x", x);
  const On on(l.device, stream);
  const void* wp = weight(w, l, l.C, -1);
  const int N = Lead::narrow(w.size(0));
  const at::DimVector shape = l.with(N);
  const void* b = operand("bias", bias, l, {N});
  const void* r = operand("residual", residual, l, shape);
  operand("y", y, l, shape);
  Tensor out = y.has_value() ? *y : l.empty(shape);
  Tensor codes, exponents;
  if (checkpoint8) std::tie(codes, exponents) = new_act8(l, N);
  check_status(conv3d_linear_fwd(x.data_ptr(), wp, b, r, out.data_ptr(), checkpoint8 ? codes.data_ptr() : nullptr,
                                 checkpoint8 ? exponents.data_ptr() : nullptr, l.rows, l.C, N, act_of(act), l.code,
                                 on.stream));
  overwritten(y);
  if (checkpoint8) return py::make_tuple(out, codes, exponents);
  return py::cast(out);
}

// (dx, x or None)
std::tuple<Tensor, OptTensor> linear_bwd_data(const Tensor& dy, const Tensor& w, const OptTensor& codes, const OptTensor& exponents,
                       int64_t channels, int act, const OptTensor& dx, bool with_x,
                       const OptStream& stream) {
  const Lead l("dy", dy);
  const On on(l.device, stream);
  TORCH_CHECK_VALUE(w.dim() >= 1, "w must be [N, K]");
  const int K = Lead::narrow(w.size(-1));
  const void* wp = weight(w, l, K, l.C);
  const at::DimVector shape = l.with(K);
  Act8 a{nullptr, nullptr};
  if (codes.has_value()) a = checkpoint("pre", *codes, exponents.value(), channels, l.device, shape);
  TORCH_CHECK_VALUE(codes.has_value() || act == CONV3D_ACT_NONE,
                    "the derivative of an activation needs the checkpoint of its argument");
  TORCH_CHECK_VALUE(!with_x || act != CONV3D_ACT_NONE, "with_x recomputes what an activation made");
  operand("dx", dx, l, shape);
  Tensor out = dx.has_value() ? *dx : l.empty(shape);
  Tensor x;
  if (with_x) x = l.empty(shape);
  check_status(conv3d_linear_bwd_data(dy.data_ptr(), wp, a.codes, a.exponents, act_of(act), out.data_ptr(),
                                      with_x ? x.data_ptr() : nullptr, l.rows, K, l.C, l.code, on.stream));
  overwritten(dx);
  if (!with_x) return {out, std::nullopt};
  return {out, x};
}

std::tuple<Tensor, OptTensor> linear_bwd_weight(const Tensor& x, const Tensor& dy, bool with_bias,
                                                const OptTensor& workspace, const OptStream& stream) {
  const Lead l("x", x);
  Tensor ws;   // outlives `on`, which sees to it that its next owner waits
  const On on(l.device, stream);
  TORCH_CHECK_VALUE(dy.dim() >= 1, "dy must be [..., N]");
  const int N = Lead::narrow(dy.size(-1));
  const void* d = operand("dy", dy, l.device, l.type, l.with(N));
  Tensor dw = l.empty({N, l.C}), db;
  if (with_bias) db = l.empty({N});
  if (workspace.has_value()) {
    TORCH_CHECK_VALUE(workspace->device() == l.device && workspace->is_contiguous(),
                      "workspace must be a contiguous CUDA tensor on ", l.device);
    ws = *workspace;
  } else {
    const size_t need = conv3d_linear_bwd_weight_workspace_bytes(l.rows, l.C, N);
    if (need > 0) ws = l.empty({static_cast<int64_t>(need)}, at::kByte);
  }
  check_status(conv3d_linear_bwd_weight(x.data_ptr(), d, dw.data_ptr(), with_bias ? db.data_ptr() : nullptr, l.rows, l.C,
                                        N, l.code, ws.defined() ? ws.data_ptr() : nullptr,
                                        ws.defined() ? ws.nbytes() : 0, on.stream));
  if (!with_bias) return {dw, std::nullopt};
  return {dw, db};
}

// (dx, dgamma, dbeta, dw1, db1, dw2, db2) of the channel MLP block from its checkpoints.
py::tuple channel_mlp_bwd(const Tensor& dy, const Tensor& x_codes, const Tensor& x_exponents, int64_t channels,
                          const Tensor& rstd, const Tensor& pre_codes, const Tensor& pre_exponents, int64_t hidden,
                          const OptTensor& gamma, const OptTensor& beta, const Tensor& w1, const Tensor& w2, int act,
                          const OptStream& stream) {
  const at::ScalarType type = dy.scalar_type();
  const bool curved = act != CONV3D_ACT_NONE;   // then the product with act' leaves the activation h too
  auto [dpre, h] = linear_bwd_data(dy, w2, pre_codes, pre_exponents, hidden, act, std::nullopt, curved, stream);
  if (!curved)
    h = act8_unpack(pre_codes, pre_exponents, hidden, type, std::nullopt, std::nullopt, act, std::nullopt, stream);
  auto [dw2, db2] = linear_bwd_weight(*h, dy, true, std::nullopt, stream);
  h.reset();
  Tensor n = act8_unpack(x_codes, x_exponents, channels, type, gamma, beta, CONV3D_ACT_NONE, std::nullopt, stream);
  auto [dw1, db1] = linear_bwd_weight(n, dpre, true, std::nullopt, stream);
  // n has been read by the time its gradient takes its place
  Tensor dn = std::get<0>(
      linear_bwd_data(dpre, w1, std::nullopt, std::nullopt, 0, CONV3D_ACT_NONE, n, false, stream));
  auto [dx, dgamma, dbeta] = layernorm_bwd(dn, std::nullopt, std::nullopt, x_codes, x_exponents, channels, rstd, gamma,
                                           dy, true, dn, std::nullopt, stream);
  return py::make_tuple(dx, dgamma, dbeta, dw1, db1, dw2, db2);
}

}  // namespace

PYBIND11_MODULE(_channel, m) {
  m.def("set_error_class", [](py::object cls) { g_error_class = cls.release().ptr(); });
  m.def("act8_pack", &act8_pack);
  m.def("act8_unpack", &act8_unpack);
  m.def("act8_bwd", &act8_bwd);
  m.def("layernorm", &layernorm);
  m.def("layernorm_bwd", &layernorm_bwd);
  m.def("linear", &linear);
  m.def("linear_bwd_data", &linear_bwd_data);
  m.def("linear_bwd_weight", &linear_bwd_weight);
  m.def("channel_mlp_bwd", &channel_mlp_bwd);
}
