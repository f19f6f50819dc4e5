// Attention of one new token of each sequence over a paged key-value cache:
//   s_j = scale q . k_j,  p = softmax_j(s),  o = sum_j p_j v_j  over the sequence's entries.
//
// Bound: HBM, every key and value read once (4 d bytes for 4 d G operations: below the tensor
// core's rate by far, but beyond what fp32 units sustain at G = 8).  So the products run on the
// tensor core with the entries as rows, which wastes none of it on the G queries of a KV head:
//   S^T [128 entries x G] = K Q^T,   O^T [d x G] += V^T P^T,
// K and V as they lie in the cache (TMA boxes of a page, or of 128 entries of a larger one), Q and
// P as the narrow operand (G padded to 16, 32 or 64 columns).  A thread of a softmax
// warpgroup owns one entry's scores of up to 16 heads, later one row of O^T.
//
// The work is cut evenly: the tiles of 128 entries of all (sequence, KV head) rows are counted
// through, and each CTA takes as many of them, whatever rows they fall in.  A row inside one CTA's
// range is finished there; of the others each CTA leaves a partial result (fp32 sums, maximum,
// normaliser; at most two a CTA), which k_paged_join adds up in a fixed order.  No prefix sum is
// stored and nothing is read back: every CTA adds up the tiles of all sequences by itself.  Where
// rows are short, or short enough and many, they stay whole and no join is needed (paged_shape).
//
// Neighbouring KV heads of one entry lie side by side in the cache.  The CTAs of a team (`side` of
// them, the largest divisor of the KV heads up to 8) have the same range of tiles, each for its
// own head, so that neighbours in memory are read at about the same time: 64 sequences of 4096
// entries, 8 heads of d = 64: 103 us alone, 92 in twos, 91 in fours, 88 in eights; d = 128: 170 -> 165.
//
// The reference m of a head's exponentials moves only when a score exceeds it by more than 8
// (a factor of 256): one vote over a warpgroup a tile, and O is rescaled in TMEM in the
// rare tile that raises it.  P enters its product as two bf16 parts (its rounding and what that
// drops, 16 bits together) in columns of their own, of which G <= 8 leaves enough idle; with one
// part the result's error was 1.4 times that of rounding it once (64 sequences of 4096 entries:
// 2.3e-3 against 1.7e-3).  With weights asked for, the scores go out in fp32 and the join adds
// 2^(s - m) / l of the group's heads to each entry's weight.
//
// Measured: 64 sequences of 4096 entries, 32 heads on 8 of d = 128: 162 us, 6.6 TB/s, 0.97 of a
// copy's; one of 131072: 84 us, of which 4 are the join; 23 of 2047, 12 heads of d = 64: 33 us (the
// bytes take 21), with weights 38; four of 103: 6 us, most of it the way through one tile.
#include "cache_common.cuh"
#include "dense_common.cuh"

namespace msa {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kWholeTiles = 12, kMostSide = 8;
constexpr int kBarStart = 15;  // named barrier; 1 to 8: votes and sums of the softmax warpgroups
constexpr float kRaise = 8.f;
constexpr float kLowest = -FLT_MAX;  // reference of a row that has no score above it yet

// GC: query heads that are computed (G rounded up), D: head dim
template <int D, int GC>
struct PagedCfg {
  static constexpr int kN = GC < 16 ? 16 : GC;   // columns of S
  static constexpr int kGroups = GC <= 16 ? 1 : GC / 16;  // softmax warpgroups, 16 heads each
  static constexpr int kThreads = 128 * kGroups + 64;     // and a warp for loads, one for products
  // Many threads leave each of them few registers, and the tiles leave L1 too small for what
  // does not fit: there the references, the same for a whole warpgroup, are in shared memory.
  static constexpr bool kShared = kGroups > 2;
  static constexpr int kHi = GC < 8 ? 8 : GC;    // columns of O: those of P's upper parts, then
  static constexpr int kNo = 2 * kHi;            // those of its lower ones
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kQ = kN * D * 2, kP = kNo * 256;
  // Buffers of P: one where that lets two CTAs share an SM (8 sequences of 16384 entries, 16 heads on
  // each of 4: 57 us with two, 52 with one).
  static constexpr int kPs = GC == 16 && D == 128 ? 1 : 2;
  static constexpr int kCtas = GC <= 16 && 3 * kTile + 2 * kQ + kPs * kP <= 114688 ? 2 : 1;  // per SM
  static constexpr int kMisc = GC <= 16 ? 1024 : 2816;  // barriers, sums over the warps
  static constexpr int kRoom = kCtas == 2 ? 115712 : 232448;
  static constexpr int kRing = (kRoom - 2 * kQ - kPs * kP - kMisc) / kTile;  // K and V tiles in flight
  static constexpr int kSmem = kRing * kTile + 2 * kQ + kPs * kP + kMisc;
  static constexpr int kUsed = 2 * kN + 2 * kNo;  // TMEM: two S, two O
  static constexpr int kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(kRing >= 3 && kCols * kCtas <= 512, "budgets");
};

// A team's tiles [x0, x1): x0 is tile `off` of sequence b, counted over its groups of KV heads.
struct PagedSpan {
  long long x0, x1;
  int b, off;
};
template <bool AHEAD>  // whether before wait_for_previous
__device__ __forceinline__ int tiles_of(const CacheArgs& c, int b) {
  return (cache_len<AHEAD>(c, b) + 127) >> 7;
}

// Counts the tiles of all sequences (every thread of the block, n of them) and looks up the tiles
// of team c.  With `whole` its range begins and ends with rows: at the first row that begins
// at or behind the cut.  `sm`: n / 32 + 2 numbers.
template <bool AHEAD>
__device__ PagedCuts paged_span(const PagedArgs& a, int c, long long* sm, int n, PagedSpan* span) {
  if (a.direct) {  // a row for each team at most: nothing to count
    span->b = c / a.groups;
    const int tiles = span->b < a.cache.nseq ? tiles_of<AHEAD>(a.cache, span->b) : 0;
    span->off = (c - span->b * a.groups) * tiles;
    span->x0 = (long long)c * ((a.cache.capacity + 127) / 128);
    span->x1 = span->x0 + tiles;
    return PagedCuts(0, 1);
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = n / 32;
  int *s_b = reinterpret_cast<int*>(sm + nw), *s_off = s_b + 2;
  const int per = (a.cache.nseq + n - 1) / n, first = min(tid * per, a.cache.nseq),
            last = min(first + per, a.cache.nseq);
  long long mine = 0;
  for (int b = first; b < last; ++b) mine += tiles_of<AHEAD>(a.cache, b);
  mine *= a.groups;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm[warp] = incl;
  if (tid < 2) s_b[tid] = a.cache.nseq, s_off[tid] = 0;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += sm[w];
    total += sm[w];
  }
  const PagedCuts cuts(total, a.grid / a.side);
  long long x[2] = {cuts.cut(c), cuts.cut(c + 1)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && !a.whole) break;
    if (mine > 0 && x[i] >= before && x[i] < before + mine) {
      long long left = x[i] - before;
      int b = first;
      for (; b < last - 1; ++b) {
        const long long t = (long long)tiles_of<AHEAD>(a.cache, b) * a.groups;
        if (left < t) break;
        left -= t;
      }
      s_b[i] = b;
      s_off[i] = (int)left;
    }
  }
  __syncthreads();
  span->b = s_b[0];
  span->off = s_off[0];
  if (a.whole) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (s_b[i] >= a.cache.nseq) continue;
      const int tiles = tiles_of<AHEAD>(a.cache, s_b[i]), t = s_off[i] % tiles;
      if (t == 0) continue;
      x[i] += tiles - t;
      if (i == 0) span->off += tiles - t;
    }
  }
  span->x0 = x[0];
  span->x1 = x[1];
  return cuts;
}

// The rows (sequence, KV head) that a CTA's range of tiles runs through.
template <bool AHEAD>
struct PagedWalk {
  int b, h, t;      // next tile; h: group of KV heads
  long long left;   // tiles of the range that are left
  int len, tiles;   // of sequence b
  int t1;           // end of the current part of the row: tiles [t0, t1)
  int t0;
  int sb, sh;       // sequence and KV head of the current part
  int at_side;      // of the CTA
  __device__ __forceinline__ void seek(const PagedArgs& a) {
    while (b < a.cache.nseq) {
      len = cache_len<AHEAD>(a.cache, b);
      tiles = (len + 127) >> 7;
      if (tiles > 0) return;
      ++b;
    }
    left = 0;
  }
  __device__ __forceinline__ PagedWalk(const PagedArgs& a, const PagedSpan& s, int cta) {
    at_side = cta % a.side;
    b = s.b;
    left = s.x1 - s.x0;
    len = tiles = h = t = t0 = t1 = sb = sh = 0;
    if (left <= 0) return;
    seek(a);
    if (left > 0) {
      h = s.off / tiles;
      t = s.off - h * tiles;
    }
  }
  // The next part; false at the end.  len and tiles are its sequence's.
  __device__ __forceinline__ bool next(const PagedArgs& a) {
    if (t == 0 && h == a.groups) {
      h = 0;
      ++b;
      if (left > 0) seek(a);
    }
    if (left <= 0) return false;
    sb = b;
    sh = h * a.side + at_side;
    t0 = t;
    t1 = (int)min((long long)tiles, t + left);
    left -= t1 - t0;
    t = t1;
    if (t == tiles) t = 0, ++h;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// Whether `x` holds for one of a warpgroup's 128 threads; a barrier for them.
__device__ __forceinline__ bool any128(uint32_t id, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return y != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t ta, float (&f)[N]) {
  uint32_t r[N];
  if constexpr (N == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(ta)
        : "memory");
  } else if constexpr (N == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(ta)
        : "memory");
  } else {
    static_assert(N == 16, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(ta)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t ta, const float (&f)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __float_as_uint(f[i]);
  if constexpr (N == 4) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(ta),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
        : "memory");
  } else if constexpr (N == 8) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(ta),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
  } else {
    tmem_st16(ta, r);
  }
}

// Reduces N <= 16 columns over the lanes of a warp: halves of the columns are exchanged, so that
// each step works on half as many.  Afterwards lane l holds column column_of<N>(l) in x[0].
template <int N, bool MAX>
__device__ __forceinline__ void reduce_cols(float (&x)[N]) {
  const int lane = threadIdx.x & 31;
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n /= 2;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < n) {
          const bool up = lane & o;
          const float give = up ? x[i] : x[i + n], own = up ? x[i + n] : x[i];
          const float got = __shfl_xor_sync(0xffffffffu, give, o);
          x[i] = MAX ? fmaxf(own, got) : own + got;
        }
      }
    } else {
      const float got = __shfl_xor_sync(0xffffffffu, x[0], o);
      x[0] = MAX ? fmaxf(x[0], got) : x[0] + got;
    }
  }
}
template <int N>
__device__ __forceinline__ int column_of(int lane) {
  int c = 0, n = N;
#pragma unroll
  for (int o = 16; o > 0 && n > 1; o >>= 1) {
    n /= 2;
    if (lane & o) c += n;
  }
  return c;
}

template <int D, int GC, bool WEIGHTS>
__global__ void __launch_bounds__(PagedCfg<D, GC>::kThreads, PagedCfg<D, GC>::kCtas)
    k_paged(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedArgs a) {
  using C = PagedCfg<D, GC>;
  constexpr int NCH = D / 64, NR = C::kRing, N = C::kN, NO = C::kNo, HI = C::kHi, PS = C::kPs;
  constexpr int CH = GC / C::kGroups, kLoads = 4 * C::kGroups, kProducts = kLoads + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sKV = smem;
  uint8_t* sQ = sKV + NR * C::kTile;  // [2][chunk][N rows][128 bytes]
  uint8_t* sP = sQ + 2 * C::kQ;       // [PS][2][64 entries][NO rows][128 bytes]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sP + PS * C::kP);
  // ring full / empty | queries loaded / free | S complete | P stored | P V complete | O read
  constexpr int B_F = 0, B_E = B_F + NR, B_Q = B_E + NR, B_QE = B_Q + 2, B_S = B_QE + 2,
                B_P = B_S + 2, B_PV = B_P + 2, B_OE = B_PV + 2, B_END = B_OE + 2;
  constexpr int kScan = B_END + 1, kSlot = kScan + C::kThreads / 32 + 2, kMax = kSlot + 1;
  long long* scan = reinterpret_cast<long long*>(bars + kScan);  // see paged_span
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  float* sMax = reinterpret_cast<float*>(bars + kMax);  // [group][4][CH] maxima of the warps
  float* sSum = sMax + 4 * GC;                          // [group][4][CH] their sums
  // and, where they are shared, [group][CH] the references
  static_assert(8 * kMax + (C::kShared ? 36 : 32) * GC <= C::kMisc, "shared memory budget");
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (warp == kLoads && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int s = 0; s < NR; ++s) {
      mbar_init(bar(B_F + s), 1);
      mbar_init(bar(B_E + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_Q + i), 1);
      mbar_init(bar(B_QE + i), 1);
      mbar_init(bar(B_S + i), 1);
      mbar_init(bar(B_P + i), 4 * C::kGroups);
      mbar_init(bar(B_PV + i), 1);
      mbar_init(bar(B_OE + i), 4 * C::kGroups);
    }
    mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  wait_for_previous();
  // The next kernel may start only behind the allocation: it could otherwise hold tensor memory that
  // this one needs, and wait for its end.
  if (warp == kProducts) {
    tmem_alloc(smem_u32(tslot), C::kCols);
    tmem_relinquish();
    let_next_start();
  }
  __syncwarp();
  PagedSpan span;
  paged_span<false>(a, blockIdx.x / a.side, scan, C::kThreads, &span);
  // The loading warp has what it needs and starts; the others wait for its barriers.
  tc_fence_before();
  if (warp == kLoads)
    asm volatile("barrier.cta.arrive %0, %1;" ::"n"(kBarStart), "n"(C::kThreads) : "memory");
  else
    asm volatile("barrier.cta.sync %0, %1;" ::"n"(kBarStart), "n"(C::kThreads) : "memory");
  tc_fence_after();
  const uint32_t tbase = warp == kLoads ? 0 : *reinterpret_cast<volatile uint32_t*>(tslot);
  // TMEM: S of tile u at columns N (u & 1), O of part i at 2 N + NO (i & 1)
  auto wait = [&](int b, uint32_t parity, int n) {
    return wait_bar_warp(bar(b), parity, abort_flag, a.cache.status, wait_site(kKerPaged, b, n));
  };

  // The loads run in the order K0, K1, V0, K2, V1, ...: that in which the products take them, with
  // the scores of one tile ahead of the values of the one before it.
  if (warp == kLoads) {
    // ------------------------------ loads ----------------------------------------
    const int rows = min(128, 1 << a.cache.page_shift);  // of a box
    const int box = lane / NCH, ch = lane % NCH;         // one box of a tile per lane
    int s = 0, lap = 0, part = 0;
    bool ok = true;
    // The page of this lane's box of a tile.  It is looked up a tile ahead, and kept for the values.
    auto page_of = [&](int b, int len, int t) {
      const int e = t * 128 + box * rows;
      return box * rows < 128 && e < len ? max(0, cache_page(a.cache, b, e)) : 0;
    };
    auto load = [&](const CUtensorMap* tm, int h, int len, int t, int page) {
      const int valid = min(128, len - t * 128), n = (valid + rows - 1) / rows;  // entries, boxes
      if (lap > 0 && !(ok = wait(B_E + s, (lap & 1) ^ 1, t))) return;
      if (lane == 0) mbar_arrive_expect_tx(bar(B_F + s), n * rows * NCH * 128);
      __syncwarp();
      if (box < n)
        tma_load_4d(smem_u32(sKV + s * C::kTile) + ch * 16384 + box * rows * 128, tm, bar(B_F + s),
                    64 * ch, h, (t * 128 + box * rows) & ((1 << a.cache.page_shift) - 1), page);
      if (++s == NR) s = 0, ++lap;
    };
    struct { int h, len, t, page; } last{0, 0, -1, 0};
    PagedWalk<false> w(a, span, blockIdx.x);
    while (ok && w.next(a)) {
      int page = page_of(w.sb, w.len, w.t0);
      if (part >= 2 && !(ok = wait(B_QE + (part & 1), ((part >> 1) & 1) ^ 1, part))) break;
      if (lane == 0) mbar_arrive_expect_tx(bar(B_Q + (part & 1)), C::kQ);
      __syncwarp();
      if (lane < NCH)
        tma_load_4d(smem_u32(sQ + (part & 1) * C::kQ) + lane * N * 128, &tm_q,
                    bar(B_Q + (part & 1)), 64 * lane, 0, w.sh, w.sb);
      ++part;
      for (int t = w.t0; ok && t < w.t1; ++t) {
        load(&tm_k, w.sh, w.len, t, page);
        if (ok && last.t >= 0) load(&tm_v, last.h, last.len, last.t, last.page);
        last = {w.sh, w.len, t, page};
        page = page_of(w.sb, w.len, min(t + 1, w.t1 - 1));
      }
    }
    if (ok && last.t >= 0) load(&tm_v, last.h, last.len, last.t, last.page);
    // sequences without an entry: no tile names them
    for (int b = blockIdx.x; b < a.cache.nseq; b += gridDim.x)
      if (cache_len(a.cache, b) == 0)
        for (int i = lane; i < a.hq * D / 8; i += 32)
          reinterpret_cast<uint4*>(a.o + (size_t)b * a.hq * D)[i] = make_uint4(0, 0, 0, 0);
    // an aborted CTA must not leave before its copies have landed
    if (*abort_flag) {
      for (int i = max(0, part - 2); i < part; ++i) drain_bar(bar(B_Q + (i & 1)), (i >> 1) & 1);
      for (int i = 0; i < NR; ++i)
        if (i < s || lap > 0) drain_bar(bar(B_F + i), (i < s ? lap : lap - 1) & 1);
    }
  } else if (warp == kProducts) {
    // ------------------------------ products -------------------------------------
    constexpr uint32_t idS = make_idesc_bf16(128, N, false, false);
    constexpr uint32_t idO = make_idesc_bf16(128, NO, true, false);
    const uint32_t el = elect_one(), tm = uniform(tbase);
    const uint32_t k_lo = desc_lo(smem_u32(sKV), 16), q_lo = desc_lo(smem_u32(sQ), 16),
                   p_lo = desc_lo(smem_u32(sP), 16);
    // d = 64 fills half of the 128 rows of V^T: the other half repeats it and is not read
    const uint32_t v_lo = desc_lo(smem_u32(sKV), D == 128 ? 16384 : 0);
    int s = 0, lap = 0, part = 0, u = 0;  // ring position, parts, tiles
    bool ok = true, first = false, pending = false, new_part = false;
    int valid = 0;
    // O += V^T P^T of tile u - 1, which has `valid` entries; the first of part `part - 1`, or of
    // the one before where a new part's first scores have been issued since
    auto values = [&](int of) {
      if (!(ok = wait(B_F + s, lap & 1, u))) return;
      const int steps = (valid + 15) / 16;
      if (valid < 16 * steps) {  // entries behind the end: P is zero there, V must be finite
        uint8_t* tile = sKV + s * C::kTile;
        const int pieces = (16 * steps - valid) * 8;
        for (int x = lane; x < NCH * pieces; x += 32)
          *reinterpret_cast<uint4*>(tile + (x / pieces) * 16384 + valid * 128 +
                                    (x % pieces) * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
      }
      const int up = u - 1;
      if (first && of >= 2 && !(ok = wait(B_OE + (of & 1), ((of >> 1) & 1) ^ 1, of))) return;
      if (!(ok = wait(B_P + (up & 1), (up >> 1) & 1, up))) return;
      tc_fence_after();
      const uint32_t v = v_lo + s * (C::kTile >> 4), p = p_lo + up % PS * (C::kP >> 4);
      const uint32_t d = tm + 2 * N + NO * (of & 1);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        if (kk < steps)
          mma_ss(el, d, v + kk * (2048 >> 4), p + (((kk >> 2) * NO * 128 + (kk & 3) * 32) >> 4),
                 idO, !first || kk > 0);
      mma_commit(el, bar(B_PV + (up & 1)));
      mma_commit(el, bar(B_E + s));
      if (++s == NR) s = 0, ++lap;
    };
    PagedWalk<false> w(a, span, blockIdx.x);
    while (ok && w.next(a)) {
      if (!(ok = wait(B_Q + (part & 1), (part >> 1) & 1, part))) break;
      new_part = true;
      for (int t = w.t0; ok && t < w.t1; ++t) {
        if (!(ok = wait(B_F + s, lap & 1, u))) break;
        tc_fence_after();
        const uint32_t k = k_lo + s * (C::kTile >> 4), q = q_lo + (part & 1) * (C::kQ >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(el, tm + N * (u & 1), k + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                 q + (((kk >> 2) * N * 128 + (kk & 3) * 32) >> 4), idS, kk > 0);
        mma_commit(el, bar(B_S + (u & 1)));
        mma_commit(el, bar(B_E + s));
        if (t + 1 == w.t1) mma_commit(el, bar(B_QE + (part & 1)));
        if (++s == NR) s = 0, ++lap;
        if (pending) values(new_part ? part - 1 : part);
        if (!ok) break;
        pending = true;
        first = new_part;
        new_part = false;
        valid = min(128, w.len - t * 128);
        ++u;
      }
      ++part;
    }
    if (ok && pending) values(part - 1);
    if (!ok) {  // products in flight end before TMEM is freed
      mma_commit(el, bar(B_END));
      drain_bar(bar(B_END), 0);
    }
  } else {
    // ------------------------------ softmax --------------------------------------
    // A failed wait marks the warp dead: it keeps to its barriers without touching TMEM.
    const int quarter = warp & 3, group = warp >> 2;
    const int r = quarter * 32 + lane;  // entry of a tile; row of O^T
    const int h0 = group * CH;          // heads h0 .. h0 + CH are this warpgroup's
    const uint32_t lanes = tbase + ((uint32_t)(quarter * 32) << 16) + h0;
    const uint32_t id_vote = 1 + 2 * group, id_join = 2 + 2 * group;
    float *wMax = sMax + 4 * h0, *wSum = sSum + 4 * h0, *wRef = sSum + 4 * GC + h0;
    const float c = a.scale_log2;
    bool dead = false;
    int u = 0, part = 0;
    long long x = span.x0;  // tile over all rows
    PagedWalk<false> w(a, span, blockIdx.x);
    while (w.next(a)) {
      // references: of this thread, or (kShared) of the warpgroup
      float own[C::kShared ? 1 : CH], l[CH];
      float* m = C::kShared ? wRef : own;
#pragma unroll
      for (int g = 0; g < CH; ++g) {
        l[g] = 0.f;
        if (!C::kShared) m[g] = kLowest;
      }
      for (int t = w.t0; t < w.t1; ++t, ++u, ++x) {
        const int b = u & 1;
        dead = dead || !wait(B_S + b, (u >> 1) & 1, u);
        tc_fence_after();
        float y[CH];
#pragma unroll
        for (int g = 0; g < CH; ++g) y[g] = -INFINITY;
        if (!dead) tmem_ld_cols<CH>(lanes + N * b, y);
        __syncwarp();
        const bool there = r < w.len - t * 128;
        bool raise = C::kShared && t == w.t0;  // the first tile sets shared references
#pragma unroll
        for (int g = 0; g < CH; ++g) {
          y[g] = there && h0 + g < a.G ? y[g] * c : -INFINITY;
          if (!C::kShared || t > w.t0) raise |= y[g] > m[g] + kRaise;
        }
        if (WEIGHTS && there) {
          float* out = a.scores + (((size_t)x * a.side + blockIdx.x % a.side) * a.G + h0) * 128 + r;
#pragma unroll
          for (int g = 0; g < CH; ++g)
            if (h0 + g < a.G) out[g * 128] = y[g];
        }
        __syncwarp();
        if (any128(id_vote, raise)) {
          // the tile's maxima of all heads; O of the tiles before it moves to the new reference
          float z[CH];
#pragma unroll
          for (int g = 0; g < CH; ++g) z[g] = y[g];
          reduce_cols<CH, true>(z);
          wMax[quarter * CH + column_of<CH>(lane)] = z[0];
          named_bar_sync(id_join, 128);
          float f[CH];
#pragma unroll
          for (int g = 0; g < CH; ++g) {
            const float top = fmaxf(fmaxf(wMax[g], wMax[CH + g]),
                                    fmaxf(wMax[2 * CH + g], wMax[3 * CH + g]));
            const float old = C::kShared && t == w.t0 ? kLowest : m[g];
            f[g] = top > old ? ex2_approx(old - top) : 1.f;
            if (!C::kShared) m[g] = top > old ? top : old;
            l[g] *= f[g];
          }
          if (C::kShared) {
            named_bar_sync(id_join, 128);  // all have read the old ones
            if (quarter == 0 && lane < CH) {
              const float top = fmaxf(fmaxf(wMax[lane], wMax[CH + lane]),
                                      fmaxf(wMax[2 * CH + lane], wMax[3 * CH + lane]));
              const float old = t == w.t0 ? kLowest : wRef[lane];
              wRef[lane] = top > old ? top : old;
            }
            named_bar_sync(id_join, 128);
          }
          if (t > w.t0) {
            dead = dead || !wait(B_PV + (b ^ 1), ((u - 1) >> 1) & 1, u);
            tc_fence_after();
            if (!dead) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t to = lanes + 2 * N + NO * (part & 1) + HI * half;
                float o[CH];
                tmem_ld_cols<CH>(to, o);
#pragma unroll
                for (int g = 0; g < CH; ++g) o[g] *= f[g];
                tmem_st_cols<CH>(to, o);
              }
            }
          }
        }
        // the buffer of P was last read by the product of tile u - PS
        if (u >= PS) dead = dead || !wait(B_PV + ((u - PS) & 1), ((u - PS) >> 1) & 1, u);
        uint8_t* p = sP + u % PS * C::kP + (r >> 6) * NO * 128 + h0 * 128 + (r & 7) * 2;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
          if (h0 + g < a.G) {
            const float e = ex2_approx(y[g] - m[g]);
            l[g] += e;
            const __nv_bfloat16 hi = __float2bfloat16_rn(e);
            const __nv_bfloat16 lo = __float2bfloat16_rn(e - __bfloat162float(hi));
            // h0 and HI are multiples of 8 (h0 = 0 below 16 heads)
            uint8_t* to = p + g * 128 + ((((r & 63) >> 3) ^ (g & 7)) << 4);
            *reinterpret_cast<__nv_bfloat16*>(to) = hi;
            *reinterpret_cast<__nv_bfloat16*>(to + HI * 128) = lo;
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P + b));
      }
      // normalisers over the entries
      reduce_cols<CH, false>(l);
      wSum[quarter * CH + column_of<CH>(lane)] = l[0];
      named_bar_sync(id_join, 128);
      dead = dead || !wait(B_PV + ((u - 1) & 1), ((u - 1) >> 1) & 1, u);
      tc_fence_after();
      float o[CH], lo[CH];
#pragma unroll
      for (int g = 0; g < CH; ++g) o[g] = lo[g] = 0.f;
      if (!dead) {
        const uint32_t from = lanes + 2 * N + NO * (part & 1);
        tmem_ld_cols<CH>(from, o);
        tmem_ld_cols<CH>(from + HI, lo);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_OE + (part & 1)));
      const bool whole = w.whole();
      const size_t row0 = (size_t)w.sb * a.hq + w.sh * a.G + h0;
      // a part of a row: the first of this CTA's range, or the last
      const size_t at = ((size_t)blockIdx.x * 2 + (part > 0)) * a.G + h0;
#pragma unroll
      for (int g = 0; g < CH; ++g) {
        if (h0 + g >= a.G) continue;
        const float sum = (wSum[g] + wSum[CH + g]) + (wSum[2 * CH + g] + wSum[3 * CH + g]);
        // an infinite value times the lower part of its weight may be NaN
        const float v = fabsf(o[g]) == INFINITY ? o[g] : o[g] + lo[g];
        if (whole) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const __nv_bfloat16 h = __float2bfloat16_rn(sum == 0.f ? 0.f : v * inv);
          if (r < D) a.o[(row0 + g) * D + r] = *reinterpret_cast<const uint16_t*>(&h);
          if (WEIGHTS && r == 0) a.stats[row0 + g] = make_float2(m[g], inv);
        } else {
          if (r < D) a.parts[(at + g) * D + r] = v;
          if (r == 0) a.part_stats[at + g] = make_float2(m[g], sum);
        }
      }
      __syncwarp();
      ++part;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kProducts) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kCols);
  }
}

// Adds four values to four floats, on 16 bytes, without a result.
__device__ __forceinline__ void red_add_v4(float* p, float4 x) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x.x), "f"(x.y),
               "f"(x.z), "f"(x.w)
               : "memory");
}

// Adds up the rows that several CTAs share, and the weights of a CTA's tiles.
//
// The parts of a row that begins inside team i's range and ends inside team j's are i's last, and
// the first of i + 1 .. j: added in this order.  The blocks of i + 1 .. j share the row's heads
// between them.
template <int D, bool WEIGHTS>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const __grid_constant__ PagedArgs a) {
  constexpr int V = D / 4;                  // pieces of a head's row
  constexpr int R = kJoinThreads / V;       // runs over the parts
  __shared__ long long scan[kJoinThreads / 32 + 2];
  __shared__ float4 s_sum[kJoinThreads];
  __shared__ float2 s_run[R], s_ref[2][kPagedMaxGroup];
  const int c = blockIdx.x / a.side, at_side = blockIdx.x % a.side, G = a.G;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  PagedSpan span;
  const PagedCuts cuts = paged_span<true>(a, c, scan, kJoinThreads, &span);
  // Where team i keeps its part of a row whose first tile is team c0's: see k_paged.
  auto part_of = [&](int i, int c0, bool behind) {
    return (((size_t)i * a.side + at_side) * 2 + (i == c0 && behind)) * G;
  };
  // What follows from the lengths alone is worked out before k_paged's results are waited for: it
  // lets this kernel start once all before it is complete, and writes no length and no page (which
  // fetch_ahead reads here).
  // The row of this team's first tile, if it begins before that:
  int c0 = 0, c1 = 0;
  bool behind = false;
  size_t row0 = 0;
  if (!a.whole && c > 0 && c < cuts.n) {
    const int tiles = tiles_of<true>(a.cache, span.b), h = span.off / tiles, t = span.off - h * tiles;
    const long long r0 = span.x0 - t;
    if (t > 0) {
      c0 = cuts.team_of(r0);
      c1 = cuts.team_of(r0 + tiles - 1);
      behind = cuts.cut(c0) < r0;
      row0 = (size_t)span.b * a.hq + (h * a.side + at_side) * G;
    }
  }
  if constexpr (WEIGHTS) {
    // A warp has a tile, a lane four of its entries (they share a page).  Rows that are shared are
    // the first and the last of the range.
    struct { int c0, c1; bool on, behind; } shared[2] = {};
    {
      PagedWalk<true> w(a, span, blockIdx.x);
      long long x = span.x0;
      for (int parts = 0; w.next(a); ++parts, x += w.t1 - w.t0) {
        if (w.whole()) continue;
        const long long r0 = x - w.t0;
        auto& s = shared[parts > 0];
        s.on = true;
        s.c0 = cuts.team_of(r0);
        s.c1 = cuts.team_of(r0 + w.tiles - 1);
        s.behind = cuts.cut(s.c0) < r0;
      }
    }
    PagedWalk<true> w(a, span, blockIdx.x);
    int next = warp;                 // this warp's tile, counted over the range
    int part = -1, done = 0, n = 0;  // tiles before the part, of the part
    auto seek = [&] {
      while (next >= done + n) {
        done += n;
        if (!w.next(a)) return false;
        n = w.t1 - w.t0;
        ++part;
      }
      return true;
    };
    auto first_entry = [&] { return (w.t0 + next - done) * 128 + 4 * lane; };
    bool more = seek();
    int page = more && first_entry() < w.len ? cache_page<true>(a.cache, w.sb, first_entry()) : -1;
    wait_for_previous();
    for (int i = warp; i < 2 * G; i += kJoinThreads / 32) {
      const int g = i % G, which = i / G;
      const auto s = shared[which];
      if (!s.on) continue;
      float m = kLowest, l = 0.f;
      for (int k = s.c0 + lane; k <= s.c1; k += 32) {
        const float2 st = fetch(&a.part_stats[part_of(k, s.c0, s.behind) + g]);
        const float to = fmaxf(m, st.x);
        l = l * (m == to ? 1.f : ex2_approx(m - to)) + st.y * (st.x == to ? 1.f : ex2_approx(st.x - to));
        m = to;
      }
      const float top = warp_max(m);
      l = warp_sum(l * (m == top ? 1.f : ex2_approx(m - top)));
      if (lane == 0) s_ref[which][g] = make_float2(top, l == 0.f ? 0.f : 1.f / l);
    }
    __syncthreads();
    for (; more; more = seek(), page = more && first_entry() < w.len
                                           ? cache_page(a.cache, w.sb, first_entry()) : -1) {
      const int e = first_entry();
      const float2 *of_row = a.stats + (size_t)w.sb * a.hq + w.sh * G, *of_part = s_ref[part > 0];
      const bool whole = w.whole();
      const float* s =
          a.scores + ((size_t)(span.x0 + next) * a.side + at_side) * G * 128 + 4 * lane;
      next += kJoinThreads / 32;
      if (page < 0) continue;  // also behind the last entry
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int g = 0; g < G; ++g) {
        const float4 y = fetch(reinterpret_cast<const float4*>(s + g * 128));
        const float2 st = whole ? fetch(of_row + g) : of_part[g];
        sum.x += ex2_approx(y.x - st.x) * st.y;
        sum.y += ex2_approx(y.y - st.x) * st.y;
        sum.z += ex2_approx(y.z - st.x) * st.y;
        sum.w += ex2_approx(y.w - st.x) * st.y;
      }
      float* to = a.cache.weight + a.cache.meta(page, e & ((1 << a.cache.page_shift) - 1), w.sh);
      if (e + 4 <= w.len) {
        red_add_v4(to, sum);
      } else {  // the scores behind the last entry are not written
        atomicAdd(to, sum.x);
        if (e + 1 < w.len) atomicAdd(to + 1, sum.y);
        if (e + 2 < w.len) atomicAdd(to + 2, sum.z);
      }
    }
  } else {
    wait_for_previous();
  }
  if (c1 == 0) return;
  const int v = tid % V, run = tid / V;
  for (int g = c - c0 - 1; g < G; g += c1 - c0) {
    // every run with a reference of its own, so that sums need not wait for the references
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = kLowest, l = 0.f;
#pragma unroll 8
    for (int i = c0 + run; i <= c1; i += R) {
      const size_t at = part_of(i, c0, behind) + g;
      const float2 st = fetch(&a.part_stats[at]);
      const float4 p = fetch(reinterpret_cast<const float4*>(a.parts + at * D) + v);
      const float to = fmaxf(m, st.x);
      const float f = m == to ? 1.f : ex2_approx(m - to), e = st.x == to ? 1.f : ex2_approx(st.x - to);
      m = to;
      l = l * f + st.y * e;
      sum.x = sum.x * f + p.x * e, sum.y = sum.y * f + p.y * e;
      sum.z = sum.z * f + p.z * e, sum.w = sum.w * f + p.w * e;
    }
    s_sum[tid] = sum;
    if (v == 0) s_run[run] = make_float2(m, l);
    __syncthreads();
    if (run == 0) {
      float top = kLowest, all = 0.f;
#pragma unroll 8
      for (int j = 0; j < R; ++j) top = fmaxf(top, s_run[j].x);
      sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int j = 0; j < R; ++j) {
        const float2 st = s_run[j];
        const float e = st.x == top ? 1.f : ex2_approx(st.x - top);
        const float4 p = s_sum[j * V + v];
        all += st.y * e;
        sum.x += p.x * e, sum.y += p.y * e, sum.z += p.z * e, sum.w += p.w * e;
      }
      const float inv = all == 0.f ? 0.f : 1.f / all;
      const uint2 o = make_uint2(pack_bf16(sum.x * inv, sum.y * inv),
                                 pack_bf16(sum.z * inv, sum.w * inv));
      reinterpret_cast<uint2*>(a.o + (row0 + g) * D)[v] = all == 0.f ? make_uint2(0, 0) : o;
    }
    __syncthreads();
  }
}

template <int D, int GC, bool WEIGHTS>
cudaError_t launch_t(const PagedArgs& a, const CUtensorMap& mq, const CUtensorMap& mk,
                     const CUtensorMap& mv, cudaStream_t st) {
  using C = PagedCfg<D, GC>;
  cudaError_t e = dense_prepare<k_paged<D, GC, WEIGHTS>>(C::kThreads, 0, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_early(k_paged<D, GC, WEIGHTS>, a.grid, C::kThreads, C::kSmem, st, 1, mq, mk, mv, a);
  if (e != cudaSuccess || (a.whole && !WEIGHTS)) return e;
  return launch_early(k_paged_join<D, WEIGHTS>, a.grid, kJoinThreads, 0, st, 1, a);
}

template <int D, bool WEIGHTS>
cudaError_t launch_d(const PagedArgs& a, const CUtensorMap& mq, const CUtensorMap& mk,
                     const CUtensorMap& mv, cudaStream_t st) {
  if (a.G <= 4) return launch_t<D, 4, WEIGHTS>(a, mq, mk, mv, st);
  if (a.G <= 8) return launch_t<D, 8, WEIGHTS>(a, mq, mk, mv, st);
  if (a.G <= 16) return launch_t<D, 16, WEIGHTS>(a, mq, mk, mv, st);
  if (a.G <= 32) return launch_t<D, 32, WEIGHTS>(a, mq, mk, mv, st);
  return launch_t<D, 64, WEIGHTS>(a, mq, mk, mv, st);
}

template <int D>
int ctas_of(int G) {  // per SM
  return G <= 4    ? PagedCfg<D, 4>::kCtas
         : G <= 8  ? PagedCfg<D, 8>::kCtas
         : G <= 16 ? PagedCfg<D, 16>::kCtas
         : G <= 32 ? PagedCfg<D, 32>::kCtas
                   : PagedCfg<D, 64>::kCtas;
}

}  // namespace

// Teams, their size and the grid for these shapes.
void paged_shape(PagedArgs* a) {
  const CacheArgs& c = a->cache;
  a->side = kMostSide;
  while (c.hkv % a->side) --a->side;
  a->groups = c.hkv / a->side;
  const long long row = (c.capacity + 127) / 128;
  // One CTA takes a row's tiles one after the other in some 0.85 us each (d = 128); shared out, all
  // rows together take as long as their bytes, and the join 4 us more.  Measured at 8 heads of
  // d = 128 (shared, whole, in us): 1 sequence of 3 tiles 8.2, 6.7, of 5 7.9, 8.6; 16 sequences of up
  // to 7 tiles 16.9, 12.5, 14 tiles 23.4, 20.0, 26 tiles 34.9, 33.0, 51 tiles 56.7, 59.5.
  // kWholeTiles is not where full rows stop to gain but where one long row among short ones
  // starts to lose: the rule sees what the table can name, not the lengths, and then one CTA has the
  // long row to itself.  16 sequences, one of the table's width and the others of 150 entries: 12 tiles
  // 12.6, 13.6, 14 tiles 12.6, 15.4, 26 tiles 11.5, 25.6 (all of the width: 24.9, 19.5; 26.7, 21.9; 40.8,
  // 36.2); 12 heads of d = 64: 12 tiles 11.0, 11.8, 26 tiles 11.8, 21.4 (20.7, 16.0; 33.8, 28.5).
  const long long rows = (long long)c.nseq * c.hkv;
  const double tile = c.d == 128 ? 0.85 : 0.7, share = c.d == 128 ? 0.007 : 0.0035;
  a->whole = row <= kWholeTiles && row * (tile - share * rows) <= 3.5;
  int most = sm_count() * (c.d == 128 ? ctas_of<128>(a->G) : ctas_of<64>(a->G));
  if (most > kPagedMaxGrid) most = kPagedMaxGrid;
  const long long tiles = (long long)c.nseq * a->groups * (a->whole ? 1 : row);
  const int teams = most / a->side > 0 ? most / a->side : 1;
  a->grid = (int)(tiles < teams ? tiles : teams) * a->side;
  a->direct = a->whole && (long long)c.nseq * a->groups <= a->grid / a->side;
}

cudaError_t launch_paged(const PagedArgs& a, const uint16_t* q, long long q_stride,
                         cudaStream_t st) {
  const CacheArgs& c = a.cache;
  const int page = 1 << c.page_shift, rows = page < 128 ? page : 128;
  const int n = a.G <= 16 ? 16 : a.G <= 32 ? 32 : 64;
  CUtensorMap mq, mk, mv;
  cudaError_t e;
  if ((e = make_tmap_4d(&mq, q, c.d, a.G, c.hkv, c.nseq, c.d, (long long)a.G * c.d, q_stride, n,
                        1)) != cudaSuccess ||
      (e = make_tmap_4d(&mk, c.k, c.d, c.hkv, page, c.num_pages, c.kh, c.ks, c.kp, 1, rows)) !=
          cudaSuccess ||
      (e = make_tmap_4d(&mv, c.v, c.d, c.hkv, page, c.num_pages, c.vh, c.vs, c.vp, 1, rows)) !=
          cudaSuccess)
    return e;
  if (a.scores)
    return c.d == 128 ? launch_d<128, true>(a, mq, mk, mv, st) : launch_d<64, true>(a, mq, mk, mv, st);
  return c.d == 128 ? launch_d<128, false>(a, mq, mk, mv, st)
                    : launch_d<64, false>(a, mq, mk, mv, st);
}

}  // namespace msa
