// Shared by the dense attention kernels: work items, document checks, the
// relative position bias.
//
// Dense attention over a packed batch: document b holds tokens
// [cu[b], cu[b + 1]), and token i attends to the tokens j <= i of its document,
//   S_ij = scale q_i . k_j + bias[h][bucket(i - j)],  P = softmax_j S,  O = P V.
// Rows behind the last document (cu[ndoc] < T: a padded batch) belong to none:
// they are treated as one more document whose outputs are zero.
#pragma once
#include <atomic>
#include <cfloat>
#include <climits>

#include "msa_internal.cuh"

namespace msa {

constexpr int kDenseMaxBuckets = 64;
constexpr int kDenseMaxGroup = 64;     // query heads per KV head
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Token strides, in elements, of the tensors a call reads.
struct DenseShape {
  int d;
  long long q_stride, k_stride, v_stride, do_stride;
};

// Kernel arguments.
struct DenseArgs {
  const int32_t* cu;
  int ndoc, T, hq, hkv;
  int G;       // query heads per KV head
  int tpt;     // tokens of a 128-row tile of packed (token, head) rows: 128 / G
  int nslots;  // work slots along the tokens (dense_slots)
  float scale, scale_log2;
  unsigned* status;
  // bias: table [hq][nb] bf16 (null: none); bucket b holds the distances
  // starts[b] <= i - j < starts[b + 1]
  const uint16_t* bias;
  int nb;
  int starts[kDenseMaxBuckets];
  // forward outputs; in the backward o and lse are inputs
  uint16_t* o;
  float* lse;
  // backward
  const uint16_t* d_o;
  long long do_stride;
  float2* stats;  // [hq][T] {lse log2(e) (+inf: no key left), D = rowsum(dO o O)}
  uint16_t *dq, *dk, *dv;
  float* slots;   // [work item][nb][2][128] per-row bucket sums of dS
  float* parts;   // [nslots][hq][nb] their sums over the rows of an item
};

// Work along the tokens is cut into slots of `bt` tokens: document b owns the
// slots from cu[b] / bt + b on.  It has at most that many tiles up to the next
// document's first slot, so a slot names at most one tile, and no prefix sum
// over the documents is needed.  ndoc + 1 documents: the last is the padding.
__host__ __device__ inline int dense_slots(int T, int ndoc, int bt) { return T / bt + ndoc + 1; }

struct DenseItem {
  int doc, start, len, tile;  // document, its first token and length, tile inside it
};

// The tile of slot `s` (all lanes of a warp; the same in every warp).  A
// document outside [0, T] or of negative length is flagged and skipped, so
// every token index derived from the item is inside the batch.
__device__ __forceinline__ bool dense_item(const DenseArgs& a, int s, int bt, DenseItem& it) {
  const int lane = threadIdx.x & 31;
  // last b in [0, ndoc] with cu[b] / bt + b <= s, 32 candidates at a time
  int lo = 0, n = a.ndoc + 1;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int off = lane * step;
    bool le = false;
    if (off < n) {
      const int c = min(max(__ldg(a.cu + lo + off), 0), a.T);
      le = c / bt + lo + off <= s;
    }
    const int last = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    const int skip = max(last, 0) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  const int b0 = __ldg(a.cu + lo);
  const int b1 = lo < a.ndoc ? __ldg(a.cu + lo + 1) : a.T;
  if (b0 < 0 || b1 < b0 || b1 > a.T) {
    if (threadIdx.x == 0) set_status(a.status, MSA_ERR_DEVICE_CHECK);
    return false;
  }
  it.doc = lo;
  it.start = b0;
  it.len = b1 - b0;
  it.tile = s - (b0 / bt + lo);
  return it.tile >= 0 && (long long)it.tile * bt < it.len;
}

// Whole check of cu_seqlens (one warp of one CTA of a launch): first entry 0,
// non-decreasing, last entry at most T.
__device__ __forceinline__ void dense_check_docs(const DenseArgs& a) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int b = lane; b <= a.ndoc; b += 32) {
    const int x = __ldg(a.cu + b);
    bad |= b == 0 ? x != 0 : x < __ldg(a.cu + b - 1);
    bad |= x < 0 || x > a.T;
  }
  if (bad) set_status(a.status, MSA_ERR_DEVICE_CHECK);
}

// A bias in log2 units.  The lowest finite values stay finite (log2(e) times
// them would not), so that rows in which only such values are left keep a
// finite maximum; -inf stays -inf and masks.
__device__ __forceinline__ float dense_bias_log2(uint16_t raw) {
  const float b = __uint_as_float((uint32_t)raw << 16);
  return b < -FLT_MAX ? b : fmaxf(b * kLog2E, -FLT_MAX);
}

// Zeroes rows [first, 128) of a 128-row bf16 tile of D columns in shared memory
// (64-column chunks of 16 KB) and makes that visible to the tensor core.  One
// warp.  The rows behind a document's end belong to the next one; as rows of
// the summed dimension of a product they are multiplied by zero
// probabilities, which would turn their infinities or NaN into NaN.
template <int D>
__device__ __forceinline__ void dense_zero_rows(uint8_t* tile, int first) {
  const int lane = threadIdx.x & 31;
  const int n16 = (128 - first) * 8;  // 16-byte pieces of one chunk
  for (int c = 0; c < D / 64; ++c)
    for (int x = lane; x < n16; x += 32)
      *reinterpret_cast<uint4*>(tile + c * 16384 + first * 128 + x * 16) = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  __syncwarp();
}

// A warp's 32 rows x 64 columns of fp32 values (one row per lane), scaled and
// rounded to bf16, through a private swizzled 32-row x 128-byte staging tile to
// global memory, four rows x 128 contiguous bytes per warp store.  `row` is
// the lane's destination (its first element; null: not stored).
__device__ __forceinline__ void dense_store_rows(const uint32_t (&va)[32], const uint32_t (&vb)[32],
                                                 float f, uint8_t* stg, uint16_t* row) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4], x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(__uint_as_float(va[8 * q + 2 * i]) * f,
                       __uint_as_float(va[8 * q + 2 * i + 1]) * f);
      x[i] = pack_bf16(__uint_as_float(vb[8 * q + 2 * i]) * f,
                       __uint_as_float(vb[8 * q + 2 * i + 1]) * f);
    }
    *reinterpret_cast<uint4*>(stg + sw128_offset(lane, q)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(stg + sw128_offset(lane, q + 4)) = make_uint4(x[0], x[1], x[2], x[3]);
  }
  __syncwarp();
  const int ch = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rr = (lane >> 3) + 4 * i;
    const uint4 x = *reinterpret_cast<const uint4*>(stg + sw128_offset(rr, ch));
    uint16_t* dst = reinterpret_cast<uint16_t*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), rr));
    if (dst) *reinterpret_cast<uint4*>(dst + ch * 8) = x;
  }
  __syncwarp();
}

// The same for a row of zeros (documents' padding), without staging: `n`
// elements (a multiple of 8) by one thread.
__device__ __forceinline__ void dense_zero_row(uint16_t* row, int n) {
  for (int i = 0; i < n; i += 8) *reinterpret_cast<uint4*>(row + i) = make_uint4(0, 0, 0, 0);
}

// Once per kernel and device: its shared-memory size, and a check that the
// registers of a launch cover the warpgroups' budgets (setmaxnreg.inc would
// otherwise wait for registers that nothing frees).
template <auto Kernel>
cudaError_t dense_prepare(int threads, int reg_budget, int smem) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, Kernel)) != cudaSuccess) return e;
  if (fa.numRegs * threads < reg_budget) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Tensor map of a [T][heads][d] bf16 tensor with token stride `stride`
// elements: boxes of 64 columns x box_heads x box_tokens, 128-byte swizzle.
cudaError_t make_tmap_rows(CUtensorMap* map, const void* base, int d, int heads, int T,
                           long long stride, int box_heads, int box_tokens);

cudaError_t launch_dense_fwd(const DenseShape& s, const uint16_t* q, const uint16_t* k,
                             const uint16_t* v, const DenseArgs& a, cudaStream_t st);
cudaError_t launch_dense_bwd(const DenseShape& s, const uint16_t* q, const uint16_t* k,
                             const uint16_t* v, const uint16_t* d_o, uint16_t* dtable,
                             const DenseArgs& a, cudaStream_t st);

}  // namespace msa
