// C ABI of rotary positions and the paged key-value cache: argument checks, workspace layout and
// launches.  See include/msa.h for the contract.
#include <algorithm>
#include <cmath>

#include "cache_common.cuh"
#include "dense_common.cuh"

namespace msa {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxTokens25 = 1 << 25;

// Token stride of a [T][heads][d] tensor: 0 means packed; rows start on 16 bytes.
bool stride_of(int64_t given, int heads, int d, int bytes, long long* out) {
  const long long packed = (long long)heads * d;
  *out = given == 0 ? packed : given;
  return *out >= packed && *out * bytes % 16 == 0 && *out < (1ll << 38);
}

msa_status check_rotary(const msa_rotary_params* p, bool cu, bool positions, RotaryArgs* a) {
  if (!p || p->flags != 0) return MSA_ERR_INVALID_ARG;
  if (p->total_tokens < 0 || p->num_docs < 0 || p->hq < 0 || p->hkv < 0 || p->hq + p->hkv < 1)
    return MSA_ERR_INVALID_ARG;
  if ((p->interleaved & ~1) || (p->inverse & ~1)) return MSA_ERR_INVALID_ARG;
  if (p->dtype < MSA_BF16 || p->dtype > MSA_FP32) return MSA_ERR_INVALID_ARG;
  if (!std::isfinite(p->amplitude)) return MSA_ERR_INVALID_ARG;
  if (cu != (p->num_docs > 0)) return MSA_ERR_INVALID_ARG;
  if (positions && p->position_bytes != 4 && p->position_bytes != 8) return MSA_ERR_INVALID_ARG;
  if (p->dims < 0 || p->dims > p->d || (p->dims > 0 && !p->freq)) return MSA_ERR_INVALID_ARG;
  if (p->d < 16 || p->d > 2 * kRotaryMaxPairs || p->d % 16 || p->dims % 16)
    return MSA_ERR_UNSUPPORTED;
  if (p->hq > 2048 || p->hkv > 2048 || p->hq + p->hkv > 2048) return MSA_ERR_UNSUPPORTED;
  if (p->total_tokens >= kMaxTokens25 || p->num_docs >= kMaxTokens25) return MSA_ERR_UNSUPPORTED;
  const int bytes = p->dtype == MSA_FP32 ? 4 : 2;
  *a = RotaryArgs{};
  if (!stride_of(p->q_stride, p->hq, p->d, bytes, &a->qs) ||
      !stride_of(p->k_stride, p->hkv, p->d, bytes, &a->ks))
    return MSA_ERR_INVALID_ARG;
  a->T = p->total_tokens;
  a->ndoc = p->num_docs;
  a->hq = p->hq;
  a->hkv = p->hkv;
  a->d = p->d;
  a->dims = p->dims;
  a->sign = p->inverse ? -1.f : 1.f;
  a->amplitude = p->amplitude;
  a->position_bytes = p->position_bytes;
  for (int i = 0; i < p->dims / 2; ++i) a->freq[i] = p->freq[i];
  return MSA_OK;
}

bool cache_stride(int64_t s, int size) {  // of a dimension of size 1 any
  return size <= 1 || (s > 0 && s % 8 == 0 && s < (1ll << 38));
}

msa_status check_cache(const msa_cache* c, const msa_table* t, CacheArgs* a) {
  if (!c || !t) return MSA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->hkv < 1 || t->num_seqs < 0 || t->max_pages < 1)
    return MSA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return MSA_ERR_UNSUPPORTED;
  int shift = 4;
  while (shift < 8 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size) return MSA_ERR_UNSUPPORTED;
  if (c->hkv > 1024 || t->num_seqs >= kCacheMaxSeqs ||
      (long long)t->max_pages << shift >= kCacheMaxEntries)
    return MSA_ERR_UNSUPPORTED;
  if (t->num_seqs > 1 && (t->stride < t->max_pages || t->stride >= (1ll << 38)))
    return MSA_ERR_INVALID_ARG;
  if (!cache_stride(c->k_page_stride, c->num_pages) ||
      !cache_stride(c->k_slot_stride, c->page_size) || !cache_stride(c->k_head_stride, c->hkv) ||
      !cache_stride(c->v_page_stride, c->num_pages) ||
      !cache_stride(c->v_slot_stride, c->page_size) || !cache_stride(c->v_head_stride, c->hkv))
    return MSA_ERR_INVALID_ARG;
  *a = CacheArgs{};
  a->k = c->k;
  a->v = c->v;
  a->weight = c->weight;
  a->position = c->position;
  a->num_pages = c->num_pages;
  a->page_shift = shift;
  a->hkv = c->hkv;
  a->d = c->d;
  a->kp = c->k_page_stride, a->ks = c->k_slot_stride, a->kh = c->k_head_stride;
  a->vp = c->v_page_stride, a->vs = c->v_slot_stride, a->vh = c->v_head_stride;
  a->table = t->pages;
  a->table_stride = t->stride;
  a->lens = t->lens;
  a->nseq = t->num_seqs;
  a->capacity = t->max_pages << shift;
  return MSA_OK;
}
msa_status check_cache_pointers(const CacheArgs& a) {
  if (!a.k || !a.v || !aligned(a.k, 16) || !aligned(a.v, 16)) return MSA_ERR_INVALID_ARG;
  if (!aligned(a.weight, 16) || !aligned(a.position, 16)) return MSA_ERR_INVALID_ARG;
  if (!a.table || !a.lens || !aligned(a.table, 4) || !aligned(a.lens, 4))
    return MSA_ERR_INVALID_ARG;
  return MSA_OK;
}

msa_status check_paged(const msa_cache* c, const msa_table* t, const msa_paged_params* p,
                       PagedArgs* a, long long* q_stride) {
  *a = PagedArgs{};
  const msa_status st = check_cache(c, t, &a->cache);
  if (st != MSA_OK) return st;
  if (!p || p->flags != 0 || (p->accumulate & ~1)) return MSA_ERR_INVALID_ARG;
  if (p->hq < 1 || p->hq % c->hkv) return MSA_ERR_INVALID_ARG;
  if (!(std::isfinite(p->softmax_scale * kLog2E) && p->softmax_scale > 0.f))
    return MSA_ERR_INVALID_ARG;
  if (p->hq > 1024 || p->hq / c->hkv > kPagedMaxGroup) return MSA_ERR_UNSUPPORTED;
  if ((((long long)a->cache.capacity + 127) >> 7) * c->hkv > 0x7fffffffll)  // tiles of a sequence
    return MSA_ERR_UNSUPPORTED;
  if (!stride_of(p->q_stride, p->hq, c->d, 2, q_stride)) return MSA_ERR_INVALID_ARG;
  if (p->accumulate) {
    if (!c->weight) return MSA_ERR_INVALID_ARG;
    // scores of every entry that the table can name: no more than memory could hold
    if ((double)t->num_seqs * p->hq * t->max_pages * c->page_size > 1e12)
      return MSA_ERR_UNSUPPORTED;
  }
  a->hq = p->hq;
  a->G = p->hq / c->hkv;
  a->scale_log2 = p->softmax_scale * kLog2E;
  paged_shape(a);
  return MSA_OK;
}

struct Carve {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t o = total;
    total = (o + bytes + 255) / 256 * 256;
    return o;
  }
};
struct PagedWorkspace {
  size_t parts, part_stats, stats, scores, total;
};
PagedWorkspace paged_workspace(const PagedArgs& a, bool accumulate) {
  PagedWorkspace w{};
  Carve c;
  if (!a.whole) {
    w.parts = c.take((size_t)kPagedMaxGrid * 2 * a.G * a.cache.d * sizeof(float));
    w.part_stats = c.take((size_t)kPagedMaxGrid * 2 * a.G * sizeof(float2));
  }
  if (accumulate) {
    w.stats = c.take((size_t)a.cache.nseq * a.hq * sizeof(float2));
    w.scores = c.take((size_t)a.cache.nseq * a.cache.hkv * ((a.cache.capacity + 127) / 128) * a.G *
                      128 * sizeof(float));
  }
  w.total = c.total;
  return w;
}

struct EvictWorkspace {
  size_t count, pairs, total;
  int most;
};
msa_status evict_workspace(const CacheArgs& a, int keep, EvictWorkspace* w) {
  if (keep < 1) return MSA_ERR_INVALID_ARG;
  const int most = std::max(0, std::min(keep, a.capacity - keep));
  Carve c;
  w->most = most;
  if (!evict_on_chip(a, most)) {
    w->count = c.take((size_t)a.nseq * a.hkv * sizeof(int32_t));
    w->pairs = c.take((size_t)a.nseq * a.hkv * 2 * most * sizeof(int64_t));
  }
  w->total = c.total;
  // blocks of the largest grid: 8 of a row, or one for 8 pairs
  return (long long)a.nseq * a.hkv * std::max((most + 7) / 8, 8) > 0x7fffffffll ? MSA_ERR_UNSUPPORTED
                                                                         : MSA_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_rotary(const msa_rotary_params* p, const int32_t* cu_seqlens, const void* positions,
                      const void* q, const void* k, void* q_out, void* k_out,
                      msa_stream_t stream) {
  RotaryArgs a;
  if (p && p->total_tokens == 0) return check_rotary(p, p->num_docs > 0, false, &a);
  if ((cu_seqlens != nullptr) == (positions != nullptr)) return MSA_ERR_INVALID_ARG;
  const msa_status st = check_rotary(p, cu_seqlens != nullptr, positions != nullptr, &a);
  if (st != MSA_OK) return st;
  const size_t bytes = p->dtype == MSA_FP32 ? 4 : 2;
  const struct { const void *in, *out; int heads; long long stride; } x[2] = {
      {q, q_out, a.hq, a.qs}, {k, k_out, a.hkv, a.ks}};
  for (const auto& y : x) {
    if (y.heads == 0) continue;
    if (!y.in || !y.out || !aligned(y.in, 16) || !aligned(y.out, 16)) return MSA_ERR_INVALID_ARG;
    for (const auto& z : x)
      if (z.heads > 0 &&
          overlap(y.out, (size_t)a.T * y.heads * a.d * bytes, z.in,
                  ((size_t)(a.T - 1) * z.stride + (size_t)z.heads * a.d) * bytes))
        return MSA_ERR_INVALID_ARG;
  }
  const size_t row = (size_t)a.T * a.d * bytes;
  if (a.hq > 0 && a.hkv > 0 && overlap(q_out, row * a.hq, k_out, row * a.hkv))
    return MSA_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4) || (positions && !aligned(positions, p->position_bytes)))
    return MSA_ERR_INVALID_ARG;
  if (status_ptr(&a.status) != cudaSuccess) return MSA_ERR_CUDA;
  a.cu = cu_seqlens;
  a.positions = positions;
  a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
  if (launch_rotary(a, p->dtype, p->interleaved != 0, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return MSA_ERR_CUDA;
  add_launches(1);
  return MSA_OK;
}

msa_status msa_cache_append(const msa_cache* cache, const msa_table* table,
                            const msa_rotary_params* p, int64_t v_stride,
                            const int32_t* cu_seqlens, const void* positions, const uint16_t* q,
                            const uint16_t* k, const uint16_t* v, uint16_t* q_out,
                            msa_stream_t stream) {
  CacheArgs c;
  RotaryArgs a;
  msa_status st = check_cache(cache, table, &c);
  if (st != MSA_OK) return st;
  if ((st = check_rotary(p, cu_seqlens != nullptr, positions != nullptr, &a)) != MSA_OK) return st;
  if (a.hkv != c.hkv || a.d != c.d || p->dtype != MSA_BF16 || p->inverse)
    return MSA_ERR_INVALID_ARG;
  if (cu_seqlens ? a.ndoc != c.nseq : a.T != c.nseq) return MSA_ERR_INVALID_ARG;
  if (!stride_of(v_stride, a.hkv, a.d, 2, &a.vs)) return MSA_ERR_INVALID_ARG;
  if (a.T == 0) return MSA_OK;
  if ((st = check_cache_pointers(c)) != MSA_OK) return st;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return MSA_ERR_INVALID_ARG;
  if (a.hq > 0) {
    if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return MSA_ERR_INVALID_ARG;
    const struct { const void* in; int heads; long long stride; } x[3] = {
        {q, a.hq, a.qs}, {k, a.hkv, a.ks}, {v, a.hkv, a.vs}};
    for (const auto& y : x)
      if (overlap(q_out, (size_t)a.T * a.hq * a.d * 2, y.in,
                  ((size_t)(a.T - 1) * y.stride + (size_t)y.heads * a.d) * 2))
        return MSA_ERR_INVALID_ARG;
  }
  if (!aligned(cu_seqlens, 4) || (positions && !aligned(positions, p->position_bytes)))
    return MSA_ERR_INVALID_ARG;
  if (status_ptr(&a.status) != cudaSuccess) return MSA_ERR_CUDA;
  c.status = a.status;
  a.cu = cu_seqlens;
  a.positions = positions;
  a.q = q, a.k = k, a.v = v, a.q_out = q_out;
  if (launch_append(a, c, p->interleaved != 0, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return MSA_ERR_CUDA;
  add_launches(1);
  return MSA_OK;
}

size_t msa_paged_attention_workspace_size(const msa_cache* cache, const msa_table* table,
                                          const msa_paged_params* p) {
  PagedArgs a;
  long long qs;
  if (check_paged(cache, table, p, &a, &qs) != MSA_OK) return 0;
  return std::max<size_t>(paged_workspace(a, p->accumulate != 0).total, 256);
}

msa_status msa_paged_attention(const msa_cache* cache, const msa_table* table,
                               const msa_paged_params* p, const uint16_t* q, uint16_t* o, void* ws,
                               size_t ws_bytes, msa_stream_t stream) {
  PagedArgs a;
  long long qs;
  msa_status st = check_paged(cache, table, p, &a, &qs);
  if (st != MSA_OK) return st;
  if (a.cache.nseq == 0) return MSA_OK;
  if ((st = check_cache_pointers(a.cache)) != MSA_OK) return st;
  if (!q || !o || !aligned(q, 16) || !aligned(o, 16)) return MSA_ERR_INVALID_ARG;
  // over itself a row is read by the CTA that writes it, or (shared rows) before the join writes
  const long long packed = (long long)a.hq * a.cache.d;
  if ((o != q || (a.cache.nseq > 1 && qs != packed)) &&
      overlap(o, (size_t)a.cache.nseq * packed * 2, q,
              ((size_t)(a.cache.nseq - 1) * qs + packed) * 2))
    return MSA_ERR_INVALID_ARG;
  const PagedWorkspace w = paged_workspace(a, p->accumulate != 0);
  if ((w.total > 0 && !ws) || !aligned(ws, 256)) return MSA_ERR_INVALID_ARG;
  if (ws_bytes < w.total) return MSA_ERR_WORKSPACE;
  if (bind_device(&a.cache.status) != cudaSuccess) return MSA_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.o = o;
  a.parts = reinterpret_cast<float*>(base + w.parts);
  a.part_stats = reinterpret_cast<float2*>(base + w.part_stats);
  if (p->accumulate) {
    a.stats = reinterpret_cast<float2*>(base + w.stats);
    a.scores = reinterpret_cast<float*>(base + w.scores);
  }
  if (launch_paged(a, q, qs, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MSA_ERR_CUDA;
  add_launches(a.whole && !p->accumulate ? 1 : 2);
  return MSA_OK;
}

size_t msa_cache_evict_workspace_size(const msa_cache* cache, const msa_table* table,
                                      int32_t keep) {
  CacheArgs c;
  EvictWorkspace w;
  if (check_cache(cache, table, &c) != MSA_OK || evict_workspace(c, keep, &w) != MSA_OK) return 0;
  return std::max<size_t>(w.total, 256);
}

msa_status msa_cache_evict(const msa_cache* cache, const msa_table* table, int32_t keep,
                           int32_t recent, int32_t* new_lens, void* ws, size_t ws_bytes,
                           msa_stream_t stream) {
  EvictArgs a{};
  msa_status st = check_cache(cache, table, &a.cache);
  if (st != MSA_OK) return st;
  EvictWorkspace w;
  if ((st = evict_workspace(a.cache, keep, &w)) != MSA_OK) return st;
  if (recent < 0 || recent > keep) return MSA_ERR_INVALID_ARG;
  if (!cache->weight || (recent > 0 && !cache->position)) return MSA_ERR_INVALID_ARG;
  if (a.cache.nseq == 0) return MSA_OK;
  if ((st = check_cache_pointers(a.cache)) != MSA_OK) return st;
  const size_t bytes = (size_t)a.cache.nseq * 4;
  if (!new_lens || !aligned(new_lens, 4) || overlap(new_lens, bytes, a.cache.lens, bytes))
    return MSA_ERR_INVALID_ARG;
  if ((w.total > 0 && !ws) || !aligned(ws, 256)) return MSA_ERR_INVALID_ARG;
  if (ws_bytes < w.total) return MSA_ERR_WORKSPACE;
  if (status_ptr(&a.cache.status) != cudaSuccess) return MSA_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.keep = keep;
  a.recent = recent;
  a.new_lens = new_lens;
  a.count = reinterpret_cast<int32_t*>(base + w.count);
  a.pairs = reinterpret_cast<long long*>(base + w.pairs);
  a.most = w.most;
  int launches = 0;
  if (launch_evict(a, reinterpret_cast<cudaStream_t>(stream), &launches) != cudaSuccess)
    return MSA_ERR_CUDA;
  add_launches(launches);
  return MSA_OK;
}

}  // extern "C"
