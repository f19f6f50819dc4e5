// Eviction from the paged cache by accumulated attention weight.
//
// A row is the entries of one sequence and KV head.  Of a row of n > keep entries stay: those whose
// position is above the newest one's less `recent`, then those with the largest weights, equal
// ones from the lowest entry on.  Weights become whole numbers of the same order, so the
// smallest one that stays is found by counting digits, 8 bits at a time from the top (a row's
// numbers are kept in shared memory where they fit).  The order of entries carries no meaning, so
// only entries that stay and lie behind `keep` move, each into the place of one that leaves; both
// are listed in ascending order by counting votes, so results do not depend on timing.
//
// Bound: HBM: weights and positions read once, the rows that move read and written once.  Few
// moves (a cache one step over its budget) are made by the block that lists them, many by a second
// kernel over all SMs.
#include "cache_common.cuh"
#include "dense_common.cuh"

namespace msa {
namespace {

constexpr int kMostKeys = 49152;  // of a row in shared memory
constexpr int kMostFused = 256;   // moves that the listing block makes itself
constexpr int kMoveThreads = 256;
constexpr uint32_t kRecent = 0xFFFFFFFFu, kNaN = 0xFFFFFFFEu;

// Order of weights as whole numbers; zeros of both signs are equal.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return kNaN;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Moves entry `from` of a row to `to`: LP lanes, 16 bytes of k or v each.
struct Move {
  const uint4* src;
  uint4* dst;
  long long from, to;  // places in weight and position
  bool ok;
};
__device__ __forceinline__ Move move_of(const CacheArgs& c, int b, int h, int from, int to,
                                        int lane) {
  Move m;
  const int p0 = cache_page(c, b, from), p1 = cache_page(c, b, to);
  const int mask = (1 << c.page_shift) - 1, half = c.d / 8;
  m.ok = p0 >= 0 && p1 >= 0;
  const int x = lane < half ? lane : lane - half;
  const uint16_t *s, *d;
  if (lane < half) {
    s = c.k_row(p0, from & mask, h);
    d = c.k_row(p1, to & mask, h);
  } else {
    s = c.v_row(p0, from & mask, h);
    d = c.v_row(p1, to & mask, h);
  }
  m.src = reinterpret_cast<const uint4*>(s) + x;
  m.dst = reinterpret_cast<uint4*>(const_cast<uint16_t*>(d)) + x;
  m.from = c.meta(p0, from & mask, h);
  m.to = c.meta(p1, to & mask, h);
  return m;
}

// Pairs i0, i0 + step, ... below n of a row, by the LP lanes of a group; N in flight.
template <int N>
__device__ __forceinline__ void move_pairs(const CacheArgs& c, int b, int h, const int* from,
                                           const int* to, int i0, int step, int n, int lane) {
  for (int i = i0; i < n; i += N * step) {
    Move m[N];
    uint4 v[N];
    float w[N];
    int p[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      m[j].ok = false;
      if (i + j * step < n) m[j] = move_of(c, b, h, from[i + j * step], to[i + j * step], lane);
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (m[j].ok) {
        v[j] = *m[j].src;
        if (lane == 0) w[j] = c.weight[m[j].from];
        if (lane == 1 && c.position) p[j] = c.position[m[j].from];
      }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (m[j].ok) {
        *m[j].dst = v[j];
        if (lane == 0) c.weight[m[j].to] = w[j];
        if (lane == 1 && c.position) c.position[m[j].to] = p[j];
      }
  }
}

// Exclusive sum over the block's warps of a value that all lanes of a warp hold, and the total.
__device__ __forceinline__ int warp_base(int x, int* sm, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) sm[warp] = x;
  __syncthreads();
  int y = lane < nw ? sm[lane] : 0, incl = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += z;
  }
  *total = __shfl_sync(0xffffffffu, incl, 31);
  return __shfl_sync(0xffffffffu, incl - y, warp);
}

template <bool KEYS, bool FUSED>
__global__ void __launch_bounds__(1024) k_evict_list(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t s_key[];
  __shared__ int s_hist[256], s_sum[32], s_pick[2];
  __shared__ int s_from[FUSED ? kMostFused : 1], s_to[FUSED ? kMostFused : 1];
  const CacheArgs& c = a.cache;
  const int b = blockIdx.x / c.hkv, h = blockIdx.x - b * c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = cache_len(c, b);
  if (h == 0 && tid == 0) a.new_lens[b] = min(n, a.keep);
  if (n <= a.keep) {
    if (!FUSED && tid == 0) a.count[blockIdx.x] = 0;
    return;
  }
  const int mask = (1 << c.page_shift) - 1;
  auto place = [&](int i) -> long long {
    const int page = cache_page(c, b, i);
    return page < 0 ? -1 : c.meta(page, i & mask, h);
  };

  long long limit = LLONG_MAX;  // positions from here on stay
  if (a.recent > 0) {
    int newest = INT_MIN;
#pragma unroll 4
    for (int i = tid; i < n; i += threads) {
      const long long m = place(i);
      if (m >= 0) newest = max(newest, c.position[m]);
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) s_sum[warp] = newest;
    __syncthreads();
    newest = __reduce_max_sync(0xffffffffu, lane < threads / 32 ? s_sum[lane] : INT_MIN);
    limit = (long long)newest - a.recent + 1;
  }
  auto load = [&](int i) -> uint32_t {
    const long long m = place(i);
    if (m < 0) return 0;
    if (a.recent > 0 && c.position[m] >= limit) return kRecent;
    return rank_of(c.weight[m]);
  };
  if (KEYS) {
#pragma unroll 4
    for (int i = tid; i < n; i += threads) s_key[i] = load(i);
  }
  auto key = [&](int i) -> uint32_t { return KEYS ? s_key[i] : load(i); };

  // the keep-th largest number `edge`, and how many of those equal to it stay
  uint32_t edge = 0;
  int left = a.keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    const uint32_t done = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = tid; i < n; i += threads) {
      const uint32_t x = key(i);
      if ((x & done) == edge) atomicAdd(&s_hist[(x >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {  // from the top: the first digit at which `left` are reached
      int x[8], mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += x[i] = s_hist[255 - 8 * lane - i];
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += z;
      }
      int before = incl - mine;
      if (before < left && left <= incl) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < left && left <= before + x[i]) {
            s_pick[0] = 255 - 8 * lane - i;
            s_pick[1] = left - before;
          }
          before += x[i];
        }
      }
    }
    __syncthreads();
    edge |= (uint32_t)s_pick[0] << shift;
    left = s_pick[1];
  }

  // Each warp has a run of entries and votes on 32 at a time.
  const int per = ((n + 31) / 32 + threads / 32 - 1) / (threads / 32) * 32;
  const int first = min(warp * per, n), last = min(first + per, n);
  const uint32_t below = (1u << lane) - 1;
  int ties = 0;
  for (int i = first; i < last; i += 32)
    ties += __popc(__ballot_sync(0xffffffffu, i + lane < last && key(i + lane) == edge));
  int total;
  const int tie0 = warp_base(ties, s_sum, &total);
  auto walk = [&](auto each) {  // each(entry, in range, stays)
    int tie = tie0;
    for (int i = first; i < last; i += 32) {
      const bool in = i + lane < last;
      const uint32_t x = in ? key(i + lane) : 0;
      const uint32_t eq = __ballot_sync(0xffffffffu, in && x == edge);
      const bool stays = in && (x > edge || (x == edge && tie + __popc(eq & below) < left));
      tie += __popc(eq);
      each(i + lane, in, stays);
    }
  };
  int outs = 0, ins = 0;
  walk([&](int i, bool in, bool stays) {
    outs += __popc(__ballot_sync(0xffffffffu, in && stays && i >= a.keep));
    ins += __popc(__ballot_sync(0xffffffffu, in && !stays && i < a.keep));
  });
  int out = warp_base(outs, s_sum, &total), into = warp_base(ins, s_sum, &total);
  int* from = FUSED ? s_from : a.pairs + (size_t)blockIdx.x * 2 * a.most;
  int* to = FUSED ? s_to : from + a.most;
  walk([&](int i, bool in, bool stays) {
    const bool o = in && stays && i >= a.keep, t = in && !stays && i < a.keep;
    const uint32_t vo = __ballot_sync(0xffffffffu, o), vt = __ballot_sync(0xffffffffu, t);
    if (o) from[out + __popc(vo & below)] = i;
    if (t) to[into + __popc(vt & below)] = i;
    out += __popc(vo);
    into += __popc(vt);
  });
  if (FUSED) {
    __syncthreads();
    const int lp = c.d / 4;  // lanes of a move
    move_pairs<4>(c, b, h, s_from, s_to, tid / lp, threads / lp, total, tid % lp);
  } else if (tid == 0) {
    a.count[blockIdx.x] = total;
  }
}

constexpr int kPairsPerBlock = 64;
__global__ void __launch_bounds__(kMoveThreads)
    k_evict_move(const __grid_constant__ EvictArgs a, int chunks) {
  const CacheArgs& c = a.cache;
  const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
  const int b = row / c.hkv, h = row - b * c.hkv, lp = c.d / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = min(__ldcg(a.count + row), (chunk + 1) * kPairsPerBlock);
  const int* from = a.pairs + (size_t)row * 2 * a.most;
  move_pairs<4>(c, b, h, from, from + a.most, chunk * kPairsPerBlock + threadIdx.x / lp,
                kMoveThreads / lp, n, threadIdx.x % lp);
}

template <bool KEYS, bool FUSED>
cudaError_t list(const EvictArgs& a, int rows, int threads, int smem, cudaStream_t st) {
  const cudaError_t e = dense_prepare<k_evict_list<KEYS, FUSED>>(0, 0, KEYS ? kMostKeys * 4 : 0);
  if (e != cudaSuccess) return e;
  k_evict_list<KEYS, FUSED><<<rows, threads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st, int* launches) {
  const CacheArgs& c = a.cache;
  const int rows = c.nseq * c.hkv;
  const bool keys = c.capacity <= kMostKeys, fused = a.most <= kMostFused;
  const int threads = c.capacity <= 8192 ? 256 : 1024, smem = keys ? c.capacity * 4 : 0;
  const cudaError_t e =
      keys ? (fused ? list<true, true>(a, rows, threads, smem, st)
                    : list<true, false>(a, rows, threads, smem, st))
           : (fused ? list<false, true>(a, rows, threads, smem, st)
                    : list<false, false>(a, rows, threads, smem, st));
  *launches = fused ? 1 : 2;
  if (e != cudaSuccess || fused) return e;
  const int chunks = (a.most + kPairsPerBlock - 1) / kPairsPerBlock;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * chunks));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_evict_move, a, chunks);
}

}  // namespace msa
