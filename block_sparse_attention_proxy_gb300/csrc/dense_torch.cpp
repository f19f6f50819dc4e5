// The torch front end of the dense attention: argument checks, output allocation and the
// autograd node around msa_dense_fwd / msa_dense_bwd.  In C++ because the calls are
// short: a forward and backward of a small batch runs about 60 us on the GPU, and the
// same front end written in Python kept the host busy for 270 us a step.  The
// computation itself is in the library's kernels.
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/saved_variable.h>
#include <torch/extension.h>

#include <limits>
#include <vector>

#include "msa.h"

namespace {

using at::Tensor;
using torch::autograd::SavedVariable;
using torch::autograd::variable_list;

// A status of the library; becomes the package's MsaError.
struct StatusError : std::runtime_error {
  int status;
  const char* where;
  StatusError(int s, const char* w)
      : std::runtime_error(std::string(w) + ": " + msa_status_string((msa_status)s)),
        status(s),
        where(w) {}
};
void raise_on(msa_status s, const char* where) {
  if (s != MSA_OK) throw StatusError(s, where);
}

void set_msa_error(const StatusError& e) {
  auto cls = py::module_::import("block_sparse_attention_proxy_gb300").attr("MsaError");
  PyErr_SetObject(cls.ptr(), cls(e.status, e.where).ptr());
}
// In the form in which the engine carries a Python exception to the thread that asked for the
// gradients; other C++ exceptions become a RuntimeError there.
[[noreturn]] void throw_to_engine(const StatusError& e) {
  py::gil_scoped_acquire gil;
  set_msa_error(e);
  python_error error;
  error.persist();
  throw std::move(error);
}

// Token stride the library takes for a [tokens, heads, d] tensor (0: packed), or -1 where
// the layout has to be copied: heads not packed, rows that overlap or are off 16 bytes.
int64_t row_stride(const Tensor& t) {
  const int64_t heads = t.size(1), d = t.size(2);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)) return -1;
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16) return -1;
  if (t.size(0) <= 1) return 0;
  return t.stride(0) < heads * d || t.stride(0) % 8 ? -1 : t.stride(0);
}
Tensor take(const Tensor& t, int64_t* stride) {
  *stride = row_stride(t);
  if (*stride >= 0) return t;
  *stride = 0;
  return t.clone(at::MemoryFormat::Contiguous);
}

// A tensor that the library takes contiguous, on 32 bytes.
Tensor whole(const Tensor& t) {
  return t.is_contiguous() && reinterpret_cast<uintptr_t>(t.data_ptr()) % 32 == 0
             ? t
             : t.clone(at::MemoryFormat::Contiguous);
}

const uint16_t* in(const Tensor& t) {
  return t.defined() ? static_cast<const uint16_t*>(t.const_data_ptr()) : nullptr;
}
uint16_t* out(const Tensor& t) {
  return t.defined() ? static_cast<uint16_t*>(t.mutable_data_ptr()) : nullptr;
}
msa_stream_t current_stream() {
  return reinterpret_cast<msa_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
}

// There is no forward-mode derivative: a tangent would be dropped, and a Jacobian-vector product
// come out as zero.
void no_tangent(const Tensor& t) {
  TORCH_CHECK_NOT_IMPLEMENTED(
      !t.defined() || !t._fw_grad(/*level=*/0).defined(),
      "dense_attention has no forward-mode derivative (an input carries a tangent)");
}

// What a forward leaves for its backward, besides the tensors.
struct Call {
  msa_dense_params prm{};
  std::vector<int32_t> starts;
  // in one buffer: lse, then o_res
  int64_t o_res_at() const { return ((int64_t)prm.total_tokens * prm.hq * 4 + 255) / 256 * 256; }
  int64_t saved() const {
    return o_res_at() + std::max<int64_t>((int64_t)prm.total_tokens * prm.hq * prm.d * 2, 256);
  }
};

// Backward of one call.  Allocates its own workspace: calls on other streams and other
// captured graphs share none.
struct DenseAttentionBackward : torch::autograd::Node {
  Call call;
  SavedVariable q, k, v, cu, bias, o, saved;

  std::string name() const override { return "DenseAttentionBackward"; }
  void release_variables() override {
    for (SavedVariable* s : {&q, &k, &v, &cu, &bias, &o, &saved}) s->reset_data();
  }
  variable_list apply(variable_list&& grads) override {
    if (!grads[0].defined()) return variable_list(4);
    no_tangent(grads[0]);
    variable_list g;
    try {
      g = compute(grads[0]);
    } catch (const StatusError& e) {
      throw_to_engine(e);
    }
    if (!at::GradMode::is_enabled()) return g;
    // asked for with create_graph: an error where somebody differentiates further
    return torch::autograd::DelayedError("dense_attention is differentiable once", 4)
        .apply(std::move(g));
  }
  // Inside a capture, a gradient that goes to a node of the default stream (a leaf that a graph
  // made outside the capture still holds) would make the engine join that stream to the
  // capture, which ends the process: an error here instead.
  void check_capture() {
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
    const c10::Stream here = c10::cuda::getCurrentCUDAStream().unwrap();
    const c10::Stream legacy = c10::cuda::getDefaultCUDAStream().unwrap();
    for (const auto& e : next_edges()) {
      const auto to = e.function ? e.function->stream() : std::nullopt;
      if (to && *to == legacy && *to != here)
        throw std::runtime_error(
            "dense_attention: a backward pass is captured while an autograd graph of the same "
            "inputs, made outside the capture on the default stream, is alive");
    }
  }
  // What a saved tensor comes back as is up to its hooks (activation offload, compression):
  // its values are those of the forward, its layout need not be.  Other sizes, types or devices
  // are refused, the rest is brought into a layout that the library takes.
  static void expect(const Tensor& t, at::IntArrayRef sizes, at::ScalarType type,
                     const at::Device& device) {
    if (!t.defined() || t.sizes() != sizes || t.scalar_type() != type || t.device() != device)
      throw StatusError(MSA_ERR_INVALID_ARG, "dense_attention: a saved tensor");
  }
  variable_list compute(Tensor d_o) {
    at::NoGradGuard no_grad;
    auto self = shared_from_this();
    Tensor q_ = q.unpack(), k_ = k.unpack(), v_ = v.unpack(), cu_ = cu.unpack();
    Tensor bias_ = bias.unpack(), o_ = o.unpack(self), saved_ = saved.unpack();
    msa_dense_params prm = call.prm;
    prm.bucket_starts = call.starts.data();
    const at::Device device = d_o.device();
    const int64_t T = prm.total_tokens;
    expect(q_, {T, prm.hq, prm.d}, at::kBFloat16, device);
    expect(k_, {T, prm.hkv, prm.d}, at::kBFloat16, device);
    expect(v_, {T, prm.hkv, prm.d}, at::kBFloat16, device);
    expect(o_, {T, prm.hq, prm.d}, at::kBFloat16, device);
    expect(cu_, {(int64_t)prm.num_docs + 1}, at::kInt, device);
    expect(saved_, {call.saved()}, at::kByte, device);
    if (prm.num_buckets > 0) expect(bias_, {prm.hq, prm.num_buckets}, at::kBFloat16, device);
    c10::cuda::CUDAGuard guard(device);
    check_capture();
    q_ = take(q_, &prm.q_stride);
    k_ = take(k_, &prm.k_stride);
    v_ = take(v_, &prm.v_stride);
    o_ = whole(o_);
    saved_ = whole(saved_);
    cu_ = cu_.contiguous();
    if (bias_.defined()) bias_ = bias_.contiguous();
    if (d_o.scalar_type() != at::kBFloat16) d_o = d_o.to(at::kBFloat16);
    d_o = take(d_o, &prm.do_stride);
    const auto opt = q_.options().requires_grad(false);
    Tensor dq = at::empty(q_.sizes(), opt), dk = at::empty(k_.sizes(), opt);
    Tensor dv = at::empty(v_.sizes(), opt), dbias;
    if (bias_.defined()) dbias = at::empty(bias_.sizes(), opt);
    const int64_t need = (int64_t)msa_dense_bwd_workspace_size(&prm);
    Tensor ws = at::empty({std::max<int64_t>(need, 256)}, opt.dtype(at::kByte));
    const uint8_t* base = saved_.const_data_ptr<uint8_t>();
    raise_on(msa_dense_bwd(&prm, cu_.const_data_ptr<int32_t>(), in(q_), in(k_), in(v_), in(bias_),
                           in(o_), reinterpret_cast<const uint16_t*>(base + call.o_res_at()),
                           reinterpret_cast<const float*>(base), in(d_o), out(dq), out(dk),
                           out(dv), out(dbias), ws.mutable_data_ptr(), (size_t)ws.numel(),
                           current_stream()),
             "msa_dense_bwd");
    return {dq, dk, dv, dbias};
  }
};

void check(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu,
           const Tensor& bias, size_t buckets) {
  for (const Tensor* t : {&q, &k, &v})
    if (t->scalar_type() != at::kBFloat16 || !t->is_cuda())
      throw py::type_error("q, k, v must be bf16 CUDA tensors");
  if (q.dim() != 3 || k.dim() != 3 || v.dim() != 3 || k.device() != q.device() ||
      v.device() != q.device())
    throw py::value_error("q, k, v must be [tokens, heads, d] on one device");
  if (k.sizes() != v.sizes() || k.size(0) != q.size(0) || k.size(2) != q.size(2))
    throw py::value_error("q [T, Hq, d] and k, v [T, Hkv, d] expected");
  if (cu.dim() != 1 || cu.numel() < 2 || cu.device() != q.device())
    throw py::value_error("cu_seqlens must be [num_docs + 1] on the device of q");
  if (cu.scalar_type() != at::kInt && cu.scalar_type() != at::kLong)
    throw py::type_error("cu_seqlens must be integers");
  if (bias.defined() != (buckets > 0))
    throw py::value_error("bias and bucket_starts go together");
  if (bias.defined()) {
    if (bias.scalar_type() != at::kBFloat16 || bias.device() != q.device())
      throw py::type_error("bias must be a bf16 tensor on the device of q");
    if (bias.dim() != 2 || bias.size(0) != q.size(1) || bias.size(1) != (int64_t)buckets)
      throw py::value_error("bias must be [Hq, number of buckets]");
  }
  constexpr int64_t kMost = std::numeric_limits<int32_t>::max();
  if (q.size(0) > kMost || q.size(1) > kMost || k.size(1) > kMost || cu.numel() > kMost)
    throw py::value_error("sizes beyond 32 bits");
}

Tensor dense_attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu_seqlens,
                       double softmax_scale, const std::optional<Tensor>& bias_table,
                       const std::optional<std::vector<int32_t>>& bucket_starts) {
  Call call;
  if (bucket_starts) call.starts = *bucket_starts;
  const Tensor bias = bias_table ? *bias_table : Tensor();
  for (const Tensor* t : {&q, &k, &v, &bias}) no_tangent(*t);
  check(q, k, v, cu_seqlens, bias, call.starts.size());
  const bool keep = at::GradMode::is_enabled() &&
                    (q.requires_grad() || k.requires_grad() || v.requires_grad() ||
                     (bias.defined() && bias.requires_grad()));
  c10::cuda::CUDAGuard guard(q.device());
  Tensor o, saved, q_, k_, v_, cu, b;
  msa_dense_params& prm = call.prm;
  {
    at::NoGradGuard no_grad;
    prm.total_tokens = (int32_t)q.size(0);
    prm.num_docs = (int32_t)(cu_seqlens.numel() - 1);
    prm.hq = (int32_t)q.size(1);
    prm.hkv = (int32_t)k.size(1);
    prm.d = (int32_t)std::min<int64_t>(q.size(2), std::numeric_limits<int32_t>::max());
    prm.num_buckets = (int32_t)call.starts.size();
    prm.bucket_starts = call.starts.data();
    prm.softmax_scale = (float)softmax_scale;
    q_ = take(q, &prm.q_stride);
    k_ = take(k, &prm.k_stride);
    v_ = take(v, &prm.v_stride);
    // out of range stays out of range in 32 bits, so that the kernels find it
    cu = cu_seqlens.scalar_type() == at::kInt
             ? cu_seqlens
             : cu_seqlens.clamp(-1, std::numeric_limits<int32_t>::max()).to(at::kInt);
    cu = cu.contiguous();
    if (bias.defined()) b = bias.contiguous();
    const auto opt = q.options().requires_grad(false);
    o = at::empty(q.sizes(), opt);
    uint8_t* base = nullptr;
    if (keep) {
      saved = at::empty({call.saved()}, opt.dtype(at::kByte));
      base = saved.mutable_data_ptr<uint8_t>();
    }
    raise_on(msa_dense_fwd(&prm, cu.const_data_ptr<int32_t>(), in(q_), in(k_), in(v_), in(b),
                           out(o),
                           keep ? reinterpret_cast<uint16_t*>(base + call.o_res_at()) : nullptr,
                           reinterpret_cast<float*>(base), current_stream()),
             "msa_dense_fwd");
  }
  if (keep) {
    std::shared_ptr<DenseAttentionBackward> node(new DenseAttentionBackward(),
                                                 torch::autograd::deleteNode);
    node->set_next_edges(torch::autograd::collect_next_edges(q, k, v, bias));
    node->call = std::move(call);
    // a saved input keeps its version counter: in-place changes before the backward are errors
    node->q = SavedVariable(q_, false);
    node->k = SavedVariable(k_, false);
    node->v = SavedVariable(v_, false);
    node->cu = SavedVariable(cu, false);
    node->bias = SavedVariable(b, false);
    node->saved = SavedVariable(saved, false);
    torch::autograd::set_history(o, node);
    node->o = SavedVariable(o, true);
  }
  return o;
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const StatusError& e) {
      set_msa_error(e);
    } catch (const c10::NotImplementedError& e) {
      PyErr_SetString(PyExc_NotImplementedError, e.what_without_backtrace());
    }
  });
  m.def("dense_attention", &dense_attention);
}
