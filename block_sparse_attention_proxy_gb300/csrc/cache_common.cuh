// Shared by the kernels around the paged key-value cache: rotary positions, append,
// attention of one new token, eviction.
#pragma once
#include <atomic>
#include <climits>

#include "msa_internal.cuh"

namespace msa {

// Waits for the kernel before this one in the stream, and for all it has written.  Every thread
// does so before its first access to memory (and to tensor memory, which the kernel before might
// still have to allocate), but for what the join of k_paged.cu says.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Allows the next kernel to be started as soon as every CTA has come this far.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// A plain load: one through the read-only path could be moved ahead of the wait, behind which alone
// its data is complete.
template <typename T>
__device__ __forceinline__ T fetch(const T* p) {
  return *p;
}

// A load of a number that the kernels before the previous one wrote, ahead of the wait: the previous
// one has waited for them before it let this kernel start, but this kernel has not, so the load goes
// past L1, which might still hold what was there before.
__device__ __forceinline__ int32_t fetch_ahead(const int32_t* p) {
  int32_t x;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}

constexpr int kRotaryMaxPairs = 128;     // head dim 256
constexpr int kCacheMaxSeqs = 1 << 20;
constexpr int kCacheMaxEntries = 1 << 30;  // of one sequence: max_pages * page_size
constexpr int kPagedMaxGroup = 64;         // query heads per KV head

// Where the cache's rows lie.  Strides in elements.
struct CacheArgs {
  uint16_t *k, *v;
  float* weight;
  int32_t* position;
  int num_pages, page_shift, hkv, d;
  long long kp, ks, kh, vp, vs, vh;  // page, slot and head strides of k and v
  const int32_t* table;
  long long table_stride;
  const int32_t* lens;
  int nseq, capacity;  // entries that a row of the table can name
  unsigned* status;
  __device__ __forceinline__ uint16_t* k_row(int page, int slot, int h) const {
    return k + page * kp + slot * ks + h * kh;
  }
  __device__ __forceinline__ uint16_t* v_row(int page, int slot, int h) const {
    return v + page * vp + slot * vs + h * vh;
  }
  // index into weight and position
  __device__ __forceinline__ long long meta(int page, int slot, int h) const {
    return (((long long)page * hkv + h) << page_shift) + slot;
  }
};

// Length of sequence b within what the table can name; others are flagged.
template <bool AHEAD = false>
__device__ __forceinline__ int cache_len(const CacheArgs& c, int b) {
  const int n = AHEAD ? fetch_ahead(c.lens + b) : fetch(c.lens + b);
  if (n >= 0 && n <= c.capacity) return n;
  set_status(c.status, MSA_ERR_DEVICE_CHECK);
  return n < 0 ? 0 : c.capacity;
}
// Page of entry i of sequence b, or -1 (flagged) where the table names none of the cache's.
template <bool AHEAD = false>
__device__ __forceinline__ int cache_page(const CacheArgs& c, int b, int i) {
  const int32_t* at = c.table + (long long)b * c.table_stride + (i >> c.page_shift);
  const int page = AHEAD ? fetch_ahead(at) : fetch(at);
  if ((unsigned)page < (unsigned)c.num_pages) return page;
  set_status(c.status, MSA_ERR_DEVICE_CHECK);
  return -1;
}

// Rows to rotate.  A row is a (token, head) pair; heads are those of q, then of k, then (append)
// of v.
struct RotaryArgs {
  int T, ndoc, hq, hkv, d, dims;
  float sign, amplitude;
  const int32_t* cu;       // null: positions
  const void* positions;   // null: cu, or (append) the entries' numbers
  int position_bytes;
  const void *q, *k, *v;
  void *q_out, *k_out;     // append writes k to the cache
  long long qs, ks, vs;    // token strides, elements
  int slots;               // threads along the heads of a token
  unsigned* status;
  uint64_t freq[kRotaryMaxPairs];
};

cudaError_t launch_rotary(RotaryArgs& a, int dtype, bool interleaved, cudaStream_t st);
cudaError_t launch_append(RotaryArgs& a, const CacheArgs& c, bool interleaved, cudaStream_t st);

// Attention of one new token (k_paged.cu).
constexpr int kPagedMaxGrid = 320;  // CTAs: bounds the workspace on every device
struct PagedArgs {
  CacheArgs cache;
  int hq, G, grid;
  int side, groups;  // CTAs of a team, each on a KV head of its own; groups of so many KV heads
  bool whole;        // rows are not shared between CTAs
  bool direct;       // and team c has row c at most
  float scale_log2;
  uint16_t* o;
  float* parts;        // [CTA][2][G][d] sums of rows that CTAs share
  float2* part_stats;  // [CTA][2][G] their references and normalisers
  float2* stats;       // [nseq][hq] reference and 1 / normaliser of whole rows (with scores)
  float* scores;       // [tile][G][128] in log2 units; null: no weights asked for
};
// a / b of numbers that are not negative; in 32 bits, a fifth of the instructions, where they fit.
__host__ __device__ inline long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// How the tiles of all rows are shared out.  Team c of the n that get any takes the tiles from
// cut(c) on: per or per + 1 of them.
struct PagedCuts {
  long long total, per;
  int more, n;  // teams with per + 1 tiles; teams with tiles
  __host__ __device__ PagedCuts(long long tiles, int teams) : total(tiles) {
    n = tiles < teams ? (int)tiles : teams;
    per = n > 0 ? quotient(tiles, n) : 0;
    more = n > 0 ? (int)(tiles - per * n) : 0;
  }
  __host__ __device__ long long cut(int c) const {
    return c >= n ? total : per * c + (c < more ? c : more);
  }
  // The team that has tile x.
  __host__ __device__ int team_of(long long x) const {
    const long long big = (per + 1) * more;
    return (int)(x < big ? quotient(x, per + 1) : more + quotient(x - big, per));
  }
};

void paged_shape(PagedArgs* a);
cudaError_t launch_paged(const PagedArgs& a, const uint16_t* q, long long q_stride,
                         cudaStream_t st);

// Eviction (k_evict.cu).
struct EvictArgs {
  CacheArgs cache;
  int keep, recent;
  int32_t* new_lens;
  int32_t* count;  // [nseq][hkv] entries that move
  long long* pairs;  // [nseq][hkv][2][most] places in the cache: from, to
  int most;        // pairs of a row at most
};
// Whether the lists of the moves need no workspace, for `most` moves of a row at most.
bool evict_on_chip(const CacheArgs& c, int most);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st, int* launches);

// Launches a kernel that may come onto the GPU while the one before it in the stream still ends
// (wait_for_previous).  Calls in a row take 2 us less each where the GPU sets the pace
// (cache_append of 32768 tokens 66.9 -> 64.0), 0.2 to 0.4 us replayed from a graph (of 64 tokens
// 3.1 -> 2.7, with the attention over one sequence of 200 9.1 -> 8.2).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, int threads, size_t smem,
                         cudaStream_t st, int cluster, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Streaming multiprocessors of the current device.
inline int sm_count() {
  static std::atomic<int> sms[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
  if (dev < 64) n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n = 1;
    if (dev < 64) sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace msa
