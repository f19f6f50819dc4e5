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
// A row one step or a few over its budget needs no digits: the entries that leave are found one
// after the other (48 sequences of 4097 entries, 8 heads: 24 -> 10 us), and their places are filled
// by the block itself.  Many moves are made by a second kernel over all SMs.
//
// Bound: HBM for the bytes (weights and positions read once, the rows that move read and written
// once), the chain of dependent steps for the search: four prompts of 32768 entries cut to 4096 (8
// heads, a cluster of 8 blocks a row): listing 17 us, of which loads 2.4, the newest position 1.2, each
// digit 1.7, counting and listing 4; moving 54 MB 20 us (16 at a copy's rate).
#include "cache_common.cuh"
#include "dense_common.cuh"

#include <algorithm>

namespace msa {
namespace {

constexpr int kSms = 152;          // of a GB300
constexpr int kListThreads = 512;
constexpr int kMostBlocks = 8;    // of a cluster: one row
constexpr int kMostKeys = 24576;  // entries of a block whose ranks and positions it keeps
constexpr int kMostFused = 256;   // moves that the listing blocks make themselves
constexpr int kFew = 8;           // entries that leave and are looked for one by one
constexpr int kAtOnce = 8;        // rows that a warp has on their way, of the second kernel
constexpr uint32_t kRecent = 0xFFFFFFFFu, kNaN = 0xFFFFFFFEu;

// Order of weights as whole numbers; zeros of both signs are equal.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return kNaN;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Moves between entries of a row, given by their places in the cache (page * page size + slot; -1:
// none): d / 4 lanes of a warp have 16 bytes of k or of v each, and a warp has N moves of each such
// group on their way.  They are moves i0 and up of the row's n; the lists lie in shared memory
// (`on_chip`) or in the workspace.
template <int N>
__device__ __forceinline__ void move_warp(const CacheArgs& c, int h, const long long* from,
                                          const long long* to, bool on_chip, int i0, int n) {
  const int lane = threadIdx.x & 31, lp = c.d / 4, group = lane / lp, groups = 32 / lp;
  const int x = lane % lp, half = lp / 2, mask = (1 << c.page_shift) - 1;
  // lane l has the places of move i0 + l
  const int mine = i0 + lane;
  const bool there = lane < N * groups && mine < n;
  const long long f = there ? (on_chip ? from[mine] : fetch(from + mine)) : -1;
  const long long t = there ? (on_chip ? to[mine] : fetch(to + mine)) : -1;
  uint16_t* base = (x < half ? c.k : c.v) + 8 * (x < half ? x : x - half);
  const long long ps = x < half ? c.kp : c.vp, ss = x < half ? c.ks : c.vs,
                  at = h * (x < half ? c.kh : c.vh);
  uint4 row[N];
  float w = 0.f;
  int p = 0;
  if (f >= 0 && t >= 0) {
    w = fetch(c.weight + c.meta((int)(f >> c.page_shift), (int)f & mask, h));
    if (c.position) p = fetch(c.position + c.meta((int)(f >> c.page_shift), (int)f & mask, h));
  }
  long long dst[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const long long fj = __shfl_sync(0xffffffffu, f, j * groups + group);
    const long long tj = __shfl_sync(0xffffffffu, t, j * groups + group);
    dst[j] = fj < 0 || tj < 0 ? -1 : (tj >> c.page_shift) * ps + (tj & mask) * ss + at;
    if (dst[j] >= 0)
      row[j] = fetch(reinterpret_cast<const uint4*>(base + (fj >> c.page_shift) * ps +
                                                     (fj & mask) * ss + at));
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (dst[j] >= 0) *reinterpret_cast<uint4*>(base + dst[j]) = row[j];
  if (f >= 0 && t >= 0) {
    const long long m = c.meta((int)(t >> c.page_shift), (int)t & mask, h);
    c.weight[m] = w;
    if (c.position) c.position[m] = p;
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

// A word of another block's shared memory (of the cluster).
__device__ __forceinline__ uint32_t ld_peer(const void* p, uint32_t rank) {
  uint32_t at, x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

// One cluster per row, each of its blocks with a run of `slice` entries.
template <bool KEYS, bool FUSED>
__global__ void __launch_bounds__(kListThreads, 2)
    k_evict_list(const __grid_constant__ EvictArgs a, int blocks, int slice) {
  // ranks, positions, and the pages of 16 entries each
  extern __shared__ __align__(16) uint32_t s_key[];
  __shared__ int s_hist[4][256], s_all[256], s_sum[32], s_share[4];
  int* s_pos = reinterpret_cast<int*>(s_key + (KEYS ? slice : 0));
  int* s_page = s_pos + (KEYS ? slice : 0);
  const CacheArgs& c = a.cache;
  const int row = blockIdx.x / blocks, rank = blockIdx.x - row * blocks;
  const int b = row / c.hkv, h = row - b * c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  wait_for_previous();
  let_next_start();
  // The first pages that this thread needs do not wait for the length.
  constexpr int kBatch = 4;
  const int* table = c.table + (long long)b * c.table_stride;
  int early[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int i = 4 * (tid + j * threads);
    early[j] = i < slice && i < c.capacity - rank * slice
                   ? fetch(table + ((rank * slice + i) >> c.page_shift))
                   : -1;
  }
  const int n = cache_len(c, b);
  if (h == 0 && rank == 0 && tid == 0) a.new_lens[b] = min(n, a.keep);
  if (n <= a.keep) {
    if (!FUSED && rank == 0 && tid == 0) a.count[row] = 0;
    return;  // all blocks of the cluster
  }
  const int mask = (1 << c.page_shift) - 1;
  const int begin = min(rank * slice, n), end = min(begin + slice, n);  // entries of this block
  auto place = [&](int i) -> long long {
    const int page = cache_page(c, b, i);
    return page < 0 ? -1 : c.meta(page, i & mask, h);
  };
  auto sync = [&] {
    __syncwarp();
    if (blocks > 1) cluster_sync(); else __syncthreads();
  };
  // Sum of word `p` of all blocks' shared memory, and that of the blocks before this one.
  auto gather = [&](const int* p, int* before) {
    int x[kMostBlocks], all = 0;
    *before = 0;
#pragma unroll
    for (int r = 0; r < kMostBlocks; ++r) {  // all on their way at once
      x[r] = 0;
      if (r < blocks) x[r] = blocks > 1 ? (int)ld_peer(p, r) : *p;
    }
#pragma unroll
    for (int r = 0; r < kMostBlocks; ++r) {
      if (r < rank) *before += x[r];
      all += x[r];
    }
    return all;
  };

  for (int i = tid; i < 4 * 256; i += threads) (&s_hist[0][0])[i] = 0;
  // Weights and positions, four entries at a time: pages begin at multiples of 16.
  int newest = INT_MIN;
  for (int i0 = begin + 4 * tid; i0 < end; i0 += 4 * kBatch * threads) {
    int page[kBatch];
    float4 w[kBatch];
    int4 p[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 4 * j * threads;
      page[j] = -1;
      if (i < end) page[j] = i0 == begin + 4 * tid ? early[j] : fetch(table + (i >> c.page_shift));
      if (i < end && (unsigned)page[j] >= (unsigned)c.num_pages) {
        set_status(c.status, MSA_ERR_DEVICE_CHECK);
        page[j] = -1;
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      p[j] = make_int4(INT_MIN, INT_MIN, INT_MIN, INT_MIN);
      if (page[j] < 0) continue;
      const long long m = c.meta(page[j], (i0 + 4 * j * threads) & mask, h);
      if (KEYS) w[j] = fetch(reinterpret_cast<const float4*>(c.weight + m));
      if (a.recent > 0) p[j] = fetch(reinterpret_cast<const int4*>(c.position + m));
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 4 * j * threads, k = end - i;
      if (k > 0) newest = max(newest, p[j].x);
      if (k > 1) newest = max(newest, p[j].y);
      if (k > 2) newest = max(newest, p[j].z);
      if (k > 3) newest = max(newest, p[j].w);
      if (!KEYS || k <= 0) continue;
      // a page that the table does not name ranks lowest
      *reinterpret_cast<uint4*>(s_key + i - begin) =
          page[j] < 0 ? make_uint4(0, 0, 0, 0)
                      : make_uint4(rank_of(w[j].x), rank_of(w[j].y), rank_of(w[j].z), rank_of(w[j].w));
      *reinterpret_cast<int4*>(s_pos + i - begin) = p[j];
      if (i % 16 == 0) s_page[(i - begin) / 16] = page[j];
    }
  }
  long long limit = LLONG_MAX;  // positions from here on stay
  if (a.recent > 0) {
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) s_sum[warp] = newest;
    __syncthreads();
    newest = __reduce_max_sync(0xffffffffu, lane < threads / 32 ? s_sum[lane] : INT_MIN);
    if (blocks > 1) {
      if (tid == 0) s_share[0] = newest;
      sync();
      newest = __reduce_max_sync(0xffffffffu, (int)ld_peer(&s_share[0], lane & (blocks - 1)));
    }
    limit = (long long)newest - a.recent + 1;
  } else {
    __syncthreads();
  }
  auto key = [&](int i) -> uint32_t {
    if (KEYS) return s_key[i - begin];
    const long long m = place(i);
    if (m < 0) return 0;
    if (a.recent > 0 && fetch(c.position + m) >= limit) return kRecent;
    return rank_of(fetch(c.weight + m));
  };
  if (KEYS && a.recent > 0) {  // each thread its own entries
    for (int i = 4 * tid; i < end - begin; i += 4 * threads) {
      const int4 p = *reinterpret_cast<const int4*>(s_pos + i);
      if (p.x >= limit) s_key[i] = kRecent;
      if (p.y >= limit) s_key[i + 1] = kRecent;
      if (p.z >= limit) s_key[i + 2] = kRecent;
      if (p.w >= limit) s_key[i + 3] = kRecent;
    }
    __syncthreads();
  }

  __shared__ long long s_pairs[FUSED ? 2 * kMostFused : 1];
  const bool on_chip = FUSED && blocks == 1;  // the lists; else in the workspace
  long long* from = on_chip ? s_pairs : a.pairs + (size_t)row * 2 * a.most;
  long long* to = from + (on_chip ? kMostFused : a.most);
  auto entry = [&](int i) -> long long {  // its place in the cache
    const int page = KEYS && i >= begin && i < end ? s_page[(i - begin) / 16] : cache_page(c, b, i);
    return page < 0 ? -1 : ((long long)page << c.page_shift) + (i & mask);
  };

  // A cache a step or a few over its budget: those that leave are found one after the other, by
  // (rank, the last entry first) as one number.
  if (KEYS && n - a.keep <= kFew) {
    __shared__ uint32_t s_min[2][32][2], s_best[kFew][2];
    __shared__ int s_gone[kFew];
    __shared__ long long s_from[kFew], s_to[kFew];
    const int leave = n - a.keep, warps = threads / 32;
    uint64_t mine;
    auto look = [&](uint64_t behind) {  // the least of this thread's behind that one
      mine = ~0ull;
#pragma unroll 4
      for (int i = begin + tid; i < end; i += threads) {
        const uint64_t o = (uint64_t)s_key[i - begin] << 32 | (uint32_t)~i;
        if (o >= behind && o < mine) mine = o;
      }
    };
    auto least = [](uint64_t x) {  // of the warp
      const uint32_t hi = __reduce_min_sync(0xffffffffu, (uint32_t)(x >> 32));
      const uint32_t lo =
          __reduce_min_sync(0xffffffffu, (uint32_t)(x >> 32) == hi ? (uint32_t)x : 0xFFFFFFFFu);
      return (uint64_t)hi << 32 | lo;
    };
    look(0);
    for (int j = 0; j < leave; ++j) {
      uint64_t best = least(mine);
      if (lane == 0) s_min[j & 1][warp][0] = (uint32_t)(best >> 32), s_min[j & 1][warp][1] = (uint32_t)best;
      __syncthreads();
      best = lane < warps ? (uint64_t)s_min[j & 1][lane][0] << 32 | s_min[j & 1][lane][1] : ~0ull;
      best = least(best);
      if (blocks > 1) {
        if (tid == 0) s_best[j][0] = (uint32_t)(best >> 32), s_best[j][1] = (uint32_t)best;
        sync();
        best = lane < blocks ? (uint64_t)ld_peer(&s_best[j][0], lane) << 32 | ld_peer(&s_best[j][1], lane)
                             : ~0ull;
        best = least(best);
      }
      if (tid == 0) s_gone[j] = (int)~(uint32_t)best;
      if (mine == best) look(best + 1);
    }
    if (rank == 0 && warp == 0) {
      __syncwarp();
      const int gone = lane < leave ? s_gone[lane] : INT_MAX, i = a.keep + lane;
      bool stays = lane < leave;
      int before = 0;
      for (int j = 0; j < leave; ++j) {
        stays &= s_gone[j] != i;
        before += s_gone[j] < gone;
      }
      const uint32_t vo = __ballot_sync(0xffffffffu, stays);
      const int moves = __popc(vo);
      if (stays) (FUSED ? s_from : from)[__popc(vo & ((1u << lane) - 1))] = entry(i);
      if (gone < a.keep) (FUSED ? s_to : to)[before] = entry(gone);
      __syncwarp();
      if (FUSED)
        for (int k = 0; k < moves; k += 2 * (128 / c.d)) move_warp<2>(c, h, s_from, s_to, true, k, moves);
      else if (lane == 0)
        a.count[row] = moves;
    }
    sync();  // nobody reads a block's shared memory any more
    return;
  }

  // the keep-th largest rank `edge`, and how many of those equal to it stay
  uint32_t edge = 0;
  int left = a.keep, equal = 0;
  for (int d = 0; d < 4; ++d) {
    const int shift = 24 - 8 * d;
    const uint32_t done = d == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
#pragma unroll 4
    for (int i = begin + tid; i < end; i += threads) {
      const uint32_t x = key(i);
      if ((x & done) == edge) atomicAdd(&s_hist[d][(x >> shift) & 255], 1);
    }
    sync();
    for (int i = tid; i < 256; i += threads) {
      int before;
      s_all[i] = gather(&s_hist[d][i], &before);
    }
    __syncthreads();
    // from the top: the first digit at which `left` are reached
    int x[8], mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += x[i] = s_all[255 - 8 * lane - i];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += z;
    }
    int before = incl - mine, digit = 0, of = 0, rest = 0;
    const uint32_t here = __ballot_sync(0xffffffffu, before < left && left <= incl);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (before < left && left <= before + x[i]) digit = 255 - 8 * lane - i, rest = left - before, of = x[i];
      before += x[i];
    }
    const int at = __ffs(here) - 1;
    edge |= (uint32_t)__shfl_sync(0xffffffffu, digit, at) << shift;
    left = __shfl_sync(0xffffffffu, rest, at);
    equal = __shfl_sync(0xffffffffu, of, at);
    if (equal == left) break;  // the lower digits decide nothing
  }

  // Each warp has a run of entries and votes on 32 at a time.
  const int per = ((end - begin + 31) / 32 + threads / 32 - 1) / (threads / 32) * 32;
  const int first = min(begin + warp * per, end), last = min(first + per, end);
  const uint32_t below = (1u << lane) - 1;
  int tie0 = 0, total, before;
  if (equal > left) {  // not all of them stay: those of the lowest entries
    int ties = 0;
    for (int i = first; i < last; i += 32)
      ties += __popc(__ballot_sync(0xffffffffu, i + lane < last && key(i + lane) == edge));
    tie0 = warp_base(ties, s_sum, &total);
    if (blocks > 1) {
      if (tid == 0) s_share[1] = total;
      sync();
      gather(&s_share[1], &before);
      tie0 += before;
    }
  } else {
    left = INT_MAX;
  }
  // Whether entries i + lane of this warp's run stay; `tie` counts those equal to the edge.
  const bool all_equal = left == INT_MAX;
  auto stay = [&](int i, int& tie) {
    const uint32_t x = i + lane < last ? key(i + lane) : 0;
    if (all_equal) return x >= edge;
    const uint32_t eq = __ballot_sync(0xffffffffu, i + lane < last && x == edge);
    const bool s = x > edge || (x == edge && tie + __popc(eq & below) < left);
    tie += __popc(eq);
    return s;
  };
  int outs = 0, ins = 0, tie = tie0;
#pragma unroll 4
  for (int i = first; i < last; i += 32) {
    const bool s = stay(i, tie), in = i + lane < last;
    outs += in && s && i + lane >= a.keep;
    ins += in && !s && i + lane < a.keep;
  }
  outs = __reduce_add_sync(0xffffffffu, outs);
  ins = __reduce_add_sync(0xffffffffu, ins);
  int all_in, into = warp_base(ins, s_sum, &all_in), out = warp_base(outs, s_sum, &total);
  if (blocks > 1) {
    if (tid == 0) s_share[2] = total, s_share[3] = all_in;
    sync();
    total = gather(&s_share[2], &before);
    out += before;
    gather(&s_share[3], &before);
    into += before;
  }
  tie = tie0;
#pragma unroll 4
  for (int i = first; i < last; i += 32) {
    const bool s = stay(i, tie), in = i + lane < last;
    const bool o = in && s && i + lane >= a.keep, t = in && !s && i + lane < a.keep;
    const uint32_t vo = __ballot_sync(0xffffffffu, o), vt = __ballot_sync(0xffffffffu, t);
    if (o) from[out + __popc(vo & below)] = entry(i + lane);
    if (t) to[into + __popc(vt & below)] = entry(i + lane);
    out += __popc(vo);
    into += __popc(vt);
  }
  if (!FUSED && rank == 0 && tid == 0) a.count[row] = total;
  sync();  // the lists are whole; nobody reads a block's shared memory any more
  if (FUSED) {
    const int step = 2 * (128 / c.d), warps = threads / 32;
    for (int i = (rank * warps + warp) * step; i < total; i += blocks * warps * step)
      move_warp<2>(c, h, from, to, on_chip, i, total);
  }
}

// One warp a block, so that a block's registers are free as soon as its moves are done.
__global__ void __launch_bounds__(32) k_evict_move(const __grid_constant__ EvictArgs a, int chunks) {
  const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
  wait_for_previous();
  const int n = fetch(a.count + row), i0 = chunk * kAtOnce * (128 / a.cache.d);
  if (i0 >= n) return;
  const long long* from = a.pairs + (size_t)row * 2 * a.most;
  move_warp<kAtOnce>(a.cache, row % a.cache.hkv, from, from + a.most, false,
                     i0, n);
}

template <bool KEYS, bool FUSED>
cudaError_t list(const EvictArgs& a, int rows, int blocks, int slice, int threads,
                 cudaStream_t st) {
  const cudaError_t e = dense_prepare<k_evict_list<KEYS, FUSED>>(0, 0, KEYS ? kMostKeys * 8 + kMostKeys / 4 : 0);
  if (e != cudaSuccess) return e;
  return launch_early(k_evict_list<KEYS, FUSED>, (unsigned)(rows * blocks), threads,
                      KEYS ? slice * 8 + slice / 4 : 0, st, blocks, a, blocks, slice);
}

}  // namespace

// Several blocks to a row where the rows alone leave SMs idle (and where a row's ranks do not fit
// one block), each with a few thousand entries at least.
int evict_blocks(const CacheArgs& c) {
  const long long rows = (long long)c.nseq * c.hkv;
  int blocks = 1;
  while (blocks < kMostBlocks && (rows * blocks * 2 <= 2 * kSms ? c.capacity / (2 * blocks) >= 2048
                                                               : c.capacity > blocks * kMostKeys))
    blocks *= 2;
  return blocks;
}
bool evict_on_chip(const CacheArgs& c, int most) {
  return most == 0 || (most <= kMostFused && evict_blocks(c) == 1);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st, int* launches) {
  const CacheArgs& c = a.cache;
  const int rows = c.nseq * c.hkv;
  const int blocks = evict_blocks(c);
  const int slice = (int)((((long long)c.capacity + blocks - 1) / blocks + 31) / 32 * 32);
  const bool keys = slice <= kMostKeys, fused = a.most <= kMostFused;
  const int threads = std::min(std::max((slice / 16 + 31) / 32 * 32, 128), kListThreads);
  const cudaError_t e = keys ? (fused ? list<true, true>(a, rows, blocks, slice, threads, st)
                                      : list<true, false>(a, rows, blocks, slice, threads, st))
                             : (fused ? list<false, true>(a, rows, blocks, slice, threads, st)
                                      : list<false, false>(a, rows, blocks, slice, threads, st));
  *launches = fused ? 1 : 2;
  if (e != cudaSuccess || fused) return e;
  const int step = kAtOnce * (128 / c.d), chunks = (a.most + step - 1) / step;
  return launch_early(k_evict_move, (unsigned)(rows * chunks), 32, 0, st, 1, a, chunks);
}

}  // namespace msa
