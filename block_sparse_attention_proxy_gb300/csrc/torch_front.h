// What the torch front ends share: errors, layouts that the library takes, streams.
#pragma once
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

namespace msa_front {

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
inline void raise_on(msa_status s, const char* where) {
  if (s != MSA_OK) throw StatusError(s, where);
}

inline void set_msa_error(const StatusError& e) {
  auto cls = py::module_::import("block_sparse_attention_proxy_gb300").attr("MsaError");
  PyErr_SetObject(cls.ptr(), cls(e.status, e.where).ptr());
}
// In the form in which the engine carries a Python exception to the thread that asked for the
// gradients; other C++ exceptions become a RuntimeError there.
[[noreturn]] inline void throw_to_engine(const StatusError& e) {
  py::gil_scoped_acquire gil;
  set_msa_error(e);
  python_error error;
  error.persist();
  throw std::move(error);
}

// Token stride the library takes for a [tokens, heads, d] tensor (0: packed), or -1 where
// the layout has to be copied: heads not packed, rows that overlap or are off 16 bytes.
inline int64_t row_stride(const Tensor& t) {
  const int64_t heads = t.size(1), d = t.size(2);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)) return -1;
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16) return -1;
  if (t.size(0) <= 1) return 0;
  return t.stride(0) < heads * d || t.stride(0) * t.element_size() % 16 ? -1 : t.stride(0);
}
inline Tensor take(const Tensor& t, int64_t* stride) {
  *stride = row_stride(t);
  if (*stride >= 0) return t;
  *stride = 0;
  return t.clone(at::MemoryFormat::Contiguous);
}

// A tensor that the library takes contiguous, on 32 bytes.
inline Tensor whole(const Tensor& t) {
  return t.is_contiguous() && reinterpret_cast<uintptr_t>(t.data_ptr()) % 32 == 0
             ? t
             : t.clone(at::MemoryFormat::Contiguous);
}

inline const uint16_t* in(const Tensor& t) {
  return t.defined() ? static_cast<const uint16_t*>(t.const_data_ptr()) : nullptr;
}
inline uint16_t* out(const Tensor& t) {
  return t.defined() ? static_cast<uint16_t*>(t.mutable_data_ptr()) : nullptr;
}
inline msa_stream_t current_stream() {
  return reinterpret_cast<msa_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
}

// There is no forward-mode derivative: a tangent would be dropped, and a Jacobian-vector product
// come out as zero.
inline void no_tangent(const Tensor& t, const char* who) {
  TORCH_CHECK_NOT_IMPLEMENTED(
      !t.defined() || !t._fw_grad(/*level=*/0).defined(), who,
      " has no forward-mode derivative (an input carries a tangent)");
}

// Inside a capture, a gradient that goes to a node of the default stream (a leaf that a graph
// made outside the capture still holds) would make the engine join that stream to the
// capture, which ends the process: an error here instead.
inline void check_capture(const torch::autograd::Node& node, const char* who) {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
  const c10::Stream here = c10::cuda::getCurrentCUDAStream().unwrap();
  const c10::Stream legacy = c10::cuda::getDefaultCUDAStream().unwrap();
  for (const auto& e : node.next_edges()) {
    const auto to = e.function ? e.function->stream() : std::nullopt;
    if (to && *to == legacy && *to != here)
      throw std::runtime_error(
          std::string(who) +
          ": a backward pass is captured while an autograd graph of the same inputs, made "
          "outside the capture on the default stream, is alive");
  }
}

// A tensor of 32-bit integers; what is out of range in 64 bits stays so, so that the kernels find it.
inline Tensor ints(const Tensor& t) {
  return t.scalar_type() == at::kInt
             ? t
             : t.clamp(-1, std::numeric_limits<int32_t>::max()).to(at::kInt);
}

}  // namespace msa_front
