// C ABI of the dense attention: argument checks, workspace layout and launch
// sequencing.  See include/msa.h for the contract.
#include <cmath>

#include "dense_common.cuh"

namespace msa {

// Device status word, with the device's context made current on this thread: a
// thread's first CUDA call may be this one (autograd runs backwards on threads of its own),
// and encoding a tensor map does not do that by itself.
cudaError_t bind_device(unsigned** status) {
  static thread_local int bound = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev != bound && (e = cudaSetDevice(dev)) == cudaSuccess) bound = dev;
  return e == cudaSuccess ? status_ptr(status) : e;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }
bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1) == 0; }

// Token stride of a [T][heads][d] tensor: 0 means packed.  Rows of one token
// must not overlap the next, and every row starts on 16 bytes.
bool stride_of(int64_t given, int heads, int d, long long* out) {
  const long long packed = (long long)heads * d;
  *out = given == 0 ? packed : given;
  return *out >= packed && *out % 8 == 0 && *out < (1ll << 38);  // TMA: byte strides below 2^40
}

msa_status check_dense(const msa_dense_params* p, DenseShape* s, DenseArgs* a) {
  if (!p || p->flags != 0) return MSA_ERR_INVALID_ARG;
  if (p->total_tokens < 0 || p->num_docs < 1) return MSA_ERR_INVALID_ARG;
  if (p->hq <= 0 || p->hkv <= 0 || p->hq % p->hkv != 0) return MSA_ERR_INVALID_ARG;
  if (!(std::isfinite(p->softmax_scale * kLog2E) && p->softmax_scale > 0.f))
    return MSA_ERR_INVALID_ARG;
  if (p->num_buckets < 0 || (p->num_buckets > 0 && !p->bucket_starts)) return MSA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return MSA_ERR_UNSUPPORTED;
  if (p->hq / p->hkv > kDenseMaxGroup || p->hq > 1024) return MSA_ERR_UNSUPPORTED;
  if (p->total_tokens >= kDenseMaxTokens || p->num_docs >= kDenseMaxTokens)
    return MSA_ERR_UNSUPPORTED;
  if (p->num_buckets > kDenseMaxBuckets) return MSA_ERR_UNSUPPORTED;
  *a = DenseArgs{};
  for (int b = 0; b < p->num_buckets; ++b) {
    const int x = p->bucket_starts[b];
    if (b == 0 ? x != 0 : x <= p->bucket_starts[b - 1]) return MSA_ERR_INVALID_ARG;
    a->starts[b] = x;
  }
  s->d = p->d;
  if (!stride_of(p->q_stride, p->hq, p->d, &s->q_stride) ||
      !stride_of(p->k_stride, p->hkv, p->d, &s->k_stride) ||
      !stride_of(p->v_stride, p->hkv, p->d, &s->v_stride) ||
      !stride_of(p->do_stride, p->hq, p->d, &s->do_stride))
    return MSA_ERR_INVALID_ARG;
  a->ndoc = p->num_docs;
  a->T = p->total_tokens;
  a->hq = p->hq;
  a->hkv = p->hkv;
  a->G = p->hq / p->hkv;
  a->tpt = 128 / a->G;
  a->nb = p->num_buckets;
  dense_lut_shape(a);
  a->scale = p->softmax_scale;
  a->scale_log2 = p->softmax_scale * kLog2E;
  // CTAs of the largest grid (one per slot and KV head)
  if ((long long)dense_slots(a->T, a->ndoc, a->tpt) * a->hkv > 0x7fffffffll)
    return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

struct DenseWorkspace {
  size_t stats, refs, slots, parts, total;
};

DenseWorkspace dense_workspace(const DenseArgs& a) {
  DenseWorkspace w{};
  auto take = [&](size_t bytes) {
    const size_t o = w.total;
    w.total = (o + bytes + 255) / 256 * 256;
    return o;
  };
  w.stats = take((size_t)a.hq * a.T * sizeof(float2));
  if (a.nb > 0) {
    w.refs = take((size_t)a.hq * a.T * sizeof(float));
    w.slots = take((size_t)kDenseMaxGrid * a.nb * 256 * sizeof(float));  // one per CTA
    w.parts = take((size_t)kDenseMaxGrid * a.hq * a.nb * sizeof(float2));
  }
  return w;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_dense_bwd_workspace_size(const msa_dense_params* p) {
  DenseShape s;
  DenseArgs a;
  if (check_dense(p, &s, &a) != MSA_OK) return 0;
  return dense_workspace(a).total;
}

msa_status msa_dense_fwd(const msa_dense_params* p, const int32_t* cu_seqlens, const uint16_t* q,
                         const uint16_t* k, const uint16_t* v, const uint16_t* bias, uint16_t* o,
                         uint16_t* o_res, float* lse, msa_stream_t stream) {
  DenseShape s;
  DenseArgs a;
  const msa_status st = check_dense(p, &s, &a);
  if (st != MSA_OK) return st;
  if (a.T == 0) return MSA_OK;
  if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3)) return MSA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)q, (const void*)k, (const void*)v, (const void*)o})
    if (!ptr || !aligned16(ptr)) return MSA_ERR_INVALID_ARG;
  if (!aligned16(lse) || !aligned32(o_res) || !aligned32(o)) return MSA_ERR_INVALID_ARG;
  if (a.nb > 0 && (!bias || !aligned2(bias))) return MSA_ERR_INVALID_ARG;
  if (bind_device(&a.status) != cudaSuccess) return MSA_ERR_CUDA;
  a.cu = cu_seqlens;
  a.bias = a.nb > 0 ? bias : nullptr;
  a.o = o;
  a.o_res = o_res;
  a.lse = lse;
  if (launch_dense_fwd(s, q, k, v, a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MSA_ERR_CUDA;
  add_launches(1);
  return MSA_OK;
}

msa_status msa_dense_bwd(const msa_dense_params* p, const int32_t* cu_seqlens, const uint16_t* q,
                         const uint16_t* k, const uint16_t* v, const uint16_t* bias,
                         const uint16_t* o, const uint16_t* o_res, const float* lse,
                         const uint16_t* dO, uint16_t* dq, uint16_t* dk, uint16_t* dv,
                         uint16_t* dbias, void* ws, size_t ws_bytes, msa_stream_t stream) {
  DenseShape s;
  DenseArgs a;
  const msa_status st = check_dense(p, &s, &a);
  if (st != MSA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (a.nb > 0) {
    if (!bias || !aligned2(bias) || !dbias || !aligned2(dbias)) return MSA_ERR_INVALID_ARG;
    if (a.T == 0)
      return cudaMemsetAsync(dbias, 0, (size_t)a.hq * a.nb * 2, cs) == cudaSuccess ? MSA_OK
                                                                                  : MSA_ERR_CUDA;
  }
  if (a.T == 0) return MSA_OK;
  if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3)) return MSA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)q, (const void*)k, (const void*)v, (const void*)o,
                          (const void*)o_res, (const void*)lse, (const void*)dO, (const void*)dq,
                          (const void*)dk, (const void*)dv})
    if (!ptr || !aligned16(ptr)) return MSA_ERR_INVALID_ARG;
  if (!aligned32(dq) || !aligned32(dk) || !aligned32(dv)) return MSA_ERR_INVALID_ARG;
  const DenseWorkspace w = dense_workspace(a);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MSA_ERR_INVALID_ARG;
  if (ws_bytes < w.total) return MSA_ERR_WORKSPACE;
  if (bind_device(&a.status) != cudaSuccess) return MSA_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.cu = cu_seqlens;
  a.bias = a.nb > 0 ? bias : nullptr;
  a.o = const_cast<uint16_t*>(o);
  a.o_res = const_cast<uint16_t*>(o_res);
  a.lse = const_cast<float*>(lse);
  a.d_o = dO;
  a.do_stride = s.do_stride;
  a.stats = reinterpret_cast<float2*>(base + w.stats);
  a.refs = reinterpret_cast<float*>(base + w.refs);
  a.slots = reinterpret_cast<float*>(base + w.slots);
  a.parts = reinterpret_cast<float2*>(base + w.parts);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  if (launch_dense_bwd(s, q, k, v, dO, dbias, a, cs) != cudaSuccess) return MSA_ERR_CUDA;
  add_launches(a.nb > 0 ? 3 : 2);
  return MSA_OK;
}

}  // extern "C"
