// Rotary positions and the append to the paged cache.
//
// Pair (a, b) of a row at position p turns by t = p f:
//   a' = a cos t - b sin t,  b' = b cos t + a sin t.
// f is in turns a position, as a fraction of 2^64, so p f modulo a turn is one product of whole
// numbers that drops what lies above 64 bits: exact at any position, where an angle in fp32
// is off by radians from some 2^24 on.  The turn's upper 32 bits become half turns in [-1, 1)
// (see turns()).
//
// A thread has 16 elements of a row: 8 pairs (two runs of 8 elements half the rotated part apart,
// or 16 neighbours), or 16 elements that only move.  It takes 8 sines and cosines once
// and goes over several heads of its token with them, four on their way at once.  Bound: HBM, each
// row read and written once: 32768 tokens of 20 heads of d = 128 in bf16 53 us, 6.3 TB/s; 131072 of
// 10 in fp32 196 us, 6.8 TB/s (a copy: 6.8); appending 32768 tokens of 16 + 4 + 4 heads 64 us.
#include "cache_common.cuh"

#include <cuda_fp16.h>

namespace msa {
namespace {

constexpr int kThreads = 64;  // small blocks leave registers free sooner: 256 took 0 to 9 % longer
constexpr float kPi = 3.14159265358979f;

// Eight elements as fp32.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p) { w = fetch(reinterpret_cast<const uint4*>(p)); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(u[i]), x[2 * i + 1] = bf16_hi(u[i]);
  }
  __device__ void set(const float (&x)[8]) {
    w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                   pack_bf16(x[6], x[7]));
  }
  __device__ void zero() { w = make_uint4(0, 0, 0, 0); }
};
template <>
struct Eight<__half> {
  uint4 w;
  __device__ void load(const __half* p) { w = fetch(reinterpret_cast<const uint4*>(p)); }
  __device__ void store(__half* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  __device__ void set(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ void zero() { w = make_uint4(0, 0, 0, 0); }
};
template <>
struct Eight<float> {
  float4 w[2];
  __device__ void load(const float* p) {
    w[0] = fetch(reinterpret_cast<const float4*>(p));
    w[1] = fetch(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = w[0];
    reinterpret_cast<float4*>(p)[1] = w[1];
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = w[0].x, x[1] = w[0].y, x[2] = w[0].z, x[3] = w[0].w;
    x[4] = w[1].x, x[5] = w[1].y, x[6] = w[1].z, x[7] = w[1].w;
  }
  __device__ void set(const float (&x)[8]) {
    w[0] = make_float4(x[0], x[1], x[2], x[3]);
    w[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ void zero() { w[0] = w[1] = make_float4(0.f, 0.f, 0.f, 0.f); }
};

// Documents (or sequences) that do not begin at 0, fall, or end behind T.
__device__ __forceinline__ void check_docs(const RotaryArgs& a) {
  bool bad = threadIdx.x == 0 && (fetch(a.cu) != 0 || fetch(a.cu + a.ndoc) > a.T);
  for (int b = threadIdx.x; b < a.ndoc; b += kThreads)
    bad |= fetch(a.cu + b + 1) < fetch(a.cu + b);
  if (bad) set_status(a.status, MSA_ERR_DEVICE_CHECK);
}

__device__ __forceinline__ long long position_of(const RotaryArgs& a, int t) {
  return a.position_bytes == 8 ? (long long)fetch(static_cast<const long long*>(a.positions) + t)
                               : (long long)fetch(static_cast<const int*>(a.positions) + t);
}

// Cosines and sines of 8 pairs from `pair` on at position p.  The upper 32 bits of a turn do not fit a
// float; what it drops (2^-25 of half a turn at most, 9.4e-8 radians, as much as the functions' own error)
// comes back by the first term of the angle sum for fp32 results; 16-bit ones are rounded far above it.
// The hardware's sines, off by 2^-21 of a pair's length, are not taken for those either: an fp16 element
// below 2^-10 of its pair would be off by more than its rounding, and they save 1 % (32768 tokens of 20
// heads 52.9 -> 52.4 us, a step of 64 tokens 2.5 -> 2.35).
template <typename T>
__device__ __forceinline__ void turns(const RotaryArgs& a, int pair, long long p, float (&c)[8],
                                      float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t turn = a.freq[pair + i] * (uint64_t)p;
    const int32_t whole = (int32_t)(turn >> 32);  // 2^-31 half turns, in [-1, 1)
    const float half = (float)whole;
    float sn, cs;
    sincospif(half * 0x1p-31f, &sn, &cs);
    if (sizeof(T) == 4) {
      const float rest = (float)(whole - (int32_t)half) * (0x1p-31f * kPi), s0 = sn;
      sn = fmaf(cs, rest, sn);
      cs = fmaf(-s0, rest, cs);
    }
    c[i] = cs * a.amplitude;
    s[i] = sn * a.amplitude * a.sign;
  }
}

// Sixteen elements, in two runs of eight at `lo` and `hi` of the row.
template <typename T, bool INTER>
__device__ __forceinline__ void turn16(Eight<T>& x, Eight<T>& y, const float (&c)[8],
                                       const float (&s)[8]) {
  float f[8], g[8], u[8], w[8];
  x.get(f);
  y.get(g);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (INTER) {  // pairs inside each run
      if (i % 2 == 0) {
        const int h = i / 2;
        u[i] = fmaf(f[i], c[h], -f[i + 1] * s[h]);
        u[i + 1] = fmaf(f[i + 1], c[h], f[i] * s[h]);
        w[i] = fmaf(g[i], c[4 + h], -g[i + 1] * s[4 + h]);
        w[i + 1] = fmaf(g[i + 1], c[4 + h], g[i] * s[4 + h]);
      }
    } else {
      u[i] = fmaf(f[i], c[i], -g[i] * s[i]);
      w[i] = fmaf(g[i], c[i], f[i] * s[i]);
    }
  }
  x.set(u);
  y.set(w);
}

// Where a thread's elements lie.
struct Place {
  int token, slot, lo, hi, pair;
  bool turn, ok;
};
template <bool INTER>
__device__ __forceinline__ Place place_of(const RotaryArgs& a) {
  Place p;
  const int cols = a.d / 16;
  const long long x = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long y = x / cols;
  const int col = (int)(x - y * cols);
  p.ok = y < (long long)a.T * a.slots;
  p.token = (int)(y / a.slots);
  p.slot = (int)(y - (long long)p.token * a.slots);
  p.pair = 8 * col;
  p.turn = 16 * col < a.dims;
  p.lo = INTER || !p.turn ? 16 * col : 8 * col;
  p.hi = INTER || !p.turn ? p.lo + 8 : p.lo + a.dims / 2;
  return p;
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads)
    k_rotary(const __grid_constant__ RotaryArgs a) {
  wait_for_previous();
  if (a.cu && blockIdx.x == 0) check_docs(a);
  const Place p = place_of<INTER>(a);
  if (!p.ok) return;
  const T* q = static_cast<const T*>(a.q) + (long long)p.token * a.qs;
  const T* k = static_cast<const T*>(a.k) + (long long)p.token * a.ks;
  T* qo = static_cast<T*>(a.q_out) + (long long)p.token * a.hq * a.d;
  T* ko = static_cast<T*>(a.k_out) + (long long)p.token * a.hkv * a.d;
  const int H = a.hq + a.hkv;
  bool padding = false;
  long long pos;
  if (a.cu) {
    const int b = doc_of_token<false>(a.cu, a.ndoc, p.token);
    pos = p.token - fetch(a.cu + b);
    padding = p.token >= fetch(a.cu + a.ndoc);
  } else {
    pos = position_of(a, p.token);
  }
  float c[8], s[8];
  if (p.turn) turns<T>(a, p.pair, pos, c, s);
  constexpr int N = 4;  // heads in flight
  for (int h0 = p.slot; h0 < H; h0 += N * a.slots) {
    Eight<T> x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * a.slots;
      if (h < H) {
        const T* row = h < a.hq ? q + h * a.d : k + (h - a.hq) * a.d;
        x[i].load(row + p.lo);
        y[i].load(row + p.hi);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * a.slots;
      if (h < H) {
        if (padding) {
          x[i].zero();
          y[i].zero();
        } else if (p.turn) {
          turn16<T, INTER>(x[i], y[i], c, s);
        }
        T* row = h < a.hq ? qo + h * a.d : ko + (h - a.hq) * a.d;
        x[i].store(row + p.lo);
        y[i].store(row + p.hi);
      }
    }
  }
}

template <bool INTER>
__global__ void __launch_bounds__(kThreads)
    k_append(const __grid_constant__ RotaryArgs a, const __grid_constant__ CacheArgs cache) {
  using T = __nv_bfloat16;
  wait_for_previous();
  if (a.cu && blockIdx.x == 0) check_docs(a);
  const Place p = place_of<INTER>(a);
  if (!p.ok) return;
  const int t = p.token;
  // sequence, entry, and where that lies; page < 0: nowhere
  int seq = t, entry = 0, page = -1;
  bool padding = false;
  if (a.cu) {
    seq = doc_of_token<false>(a.cu, a.ndoc, t);
    entry = t - fetch(a.cu + seq);
    padding = t >= fetch(a.cu + a.ndoc);
  }
  if (!padding) {
    const int len = fetch(cache.lens + seq);
    const long long e = (long long)len + entry;
    if (len < 0 || entry < 0 || e >= cache.capacity) {
      set_status(a.status, MSA_ERR_DEVICE_CHECK);
      entry = 0;
    } else {
      entry = (int)e;
      page = cache_page(cache, seq, entry);
    }
  }
  const long long pos = a.positions ? position_of(a, t) : entry;
  const int slot = entry & ((1 << cache.page_shift) - 1);
  float c[8], s[8];
  if (p.turn) turns<T>(a, p.pair, pos, c, s);
  const T* q = static_cast<const T*>(a.q) + (long long)t * a.qs;
  const T* k = static_cast<const T*>(a.k) + (long long)t * a.ks;
  const T* v = static_cast<const T*>(a.v) + (long long)t * a.vs;
  T* qo = static_cast<T*>(a.q_out) + (long long)t * a.hq * a.d;
  const int H = a.hq + 2 * a.hkv;
  constexpr int N = 4;
  for (int h0 = p.slot; h0 < H; h0 += N * a.slots) {
    Eight<T> x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * a.slots;
      if (h < H) {
        const T* row = h < a.hq ? q + h * a.d
                       : h < a.hq + a.hkv ? k + (h - a.hq) * a.d
                                          : v + (h - a.hq - a.hkv) * a.d;
        x[i].load(row + p.lo);
        y[i].load(row + p.hi);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * a.slots;
      if (h >= H) continue;
      T* row;
      if (h < a.hq) {
        row = qo + h * a.d;
        if (padding) {
          x[i].zero();
          y[i].zero();
        }
      } else {
        if (page < 0) continue;
        const int g = h - a.hq;
        row = reinterpret_cast<T*>(g < a.hkv ? cache.k_row(page, slot, g)
                                             : cache.v_row(page, slot, g - a.hkv));
        if (g < a.hkv && p.lo == 0) {  // one thread of each key row
          const long long m = cache.meta(page, slot, g);
          if (cache.weight) cache.weight[m] = 0.f;
          if (cache.position)
            cache.position[m] = (int)(pos > INT_MAX ? INT_MAX : pos < INT_MIN ? INT_MIN : pos);
        }
      }
      if (h < a.hq + a.hkv && p.turn && !padding) turn16<T, INTER>(x[i], y[i], c, s);
      x[i].store(row + p.lo);
      y[i].store(row + p.hi);
    }
  }
}

// Threads along a token's heads: as few as give each SM 512 threads, since each of them looks its
// document up and takes the sines again (in blocks of 256, 24001 tokens of 9 heads: 19.1 us with
// 4096, 14.2 with 2048, 11.6 with 512; 2000 tokens of 40: 17.2, 11.3, 7.8, and 8.7 with 256).
unsigned grid_of(RotaryArgs& a, int heads) {
  const long long cols = a.d / 16, want = 512ll * sm_count();
  const long long rows = cols * a.T;
  long long slots = (want + rows - 1) / rows;
  if (slots > heads) slots = heads;
  if (slots < (heads + 15) / 16) slots = (heads + 15) / 16;  // at most 16 heads each
  a.slots = (int)slots;
  return (unsigned)((rows * slots + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs& a, int dtype, bool interleaved, cudaStream_t st) {
  const unsigned grid = grid_of(a, a.hq + a.hkv);
  auto go = [&](auto kernel) { return launch_early(kernel, grid, kThreads, 0, st, 1, a); };
  if (dtype == MSA_BF16)
    return interleaved ? go(k_rotary<__nv_bfloat16, true>) : go(k_rotary<__nv_bfloat16, false>);
  if (dtype == MSA_FP16)
    return interleaved ? go(k_rotary<__half, true>) : go(k_rotary<__half, false>);
  return interleaved ? go(k_rotary<float, true>) : go(k_rotary<float, false>);
}

cudaError_t launch_append(RotaryArgs& a, const CacheArgs& c, bool interleaved, cudaStream_t st) {
  const unsigned grid = grid_of(a, a.hq + 2 * a.hkv);
  return launch_early(interleaved ? k_append<true> : k_append<false>, grid, kThreads, 0, st, 1, a, c);
}

}  // namespace msa
