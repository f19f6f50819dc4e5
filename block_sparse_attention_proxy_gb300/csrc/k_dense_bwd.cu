// Dense causal attention backward: dQ (and the bias table's gradient), then dK
// and dV.  With S, P as in the forward, dP = dO V^T, D = rowsum(dO o O):
//   dS = P (dP - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
//   dtable[h][b] = sum of dS over the pairs of head h whose distance is in b.
// Two kernels, each owning its outputs: one CTA per 128 packed (token, head)
// rows sums dQ over the keys, one CTA per 128 keys of a KV head sums dK and dV
// over its group's queries.  S and dP are computed in both (7 products per
// tile pair instead of 5); in exchange there are no fp32 partial gradients in
// HBM and no atomics, and every sum has a fixed order.  Bound at d = 128 by the tensor core
// (16384 tokens, 32 heads on 8: dQ 1.90 ms, 1.74 PFLOP/s of its 3 products; dK, dV 2.64 ms,
// 1.67 of their 4); at d = 64 by the exponentials and the hand-offs between the roles, and for
// short documents by what an item costs outside its tiles.
#include "dense_common.cuh"

namespace msa {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsSoftmax = 200, kRegsCtl = 104;
constexpr int kBudget = 2 * 128 * kRegsSoftmax + 128 * kRegsCtl;
static_assert(kBudget <= 65536, "register budgets exceed the register file");

// ---------------------------------------------------------------------------
// dQ: items of 128 packed rows against their keys, tile by tile; one persistent CTA per SM.
// Warps 0-3 and 4-7 take 64 of a tile's 128 columns each (a row is one TMEM
// lane of both); warp 8 loads, warp 9 issues the MMAs.  {-lse, D = rowsum(dO o O)} of an
// item's rows (which dK, dV need too) come at d = 128 from warps 10 and 11, an item ahead,
// and at d = 64, where those two could not keep up with short items, from the softmax warps,
// which load the next item's rows before they store an item's dQ (16384 tokens, 32 heads,
// d 128, as the kernel was when that was tried: 1.96 ms from warps 10 and 11, 2.04 from the
// softmax warps; 61 documents of 24001 tokens, 8 heads, d 64: 98 and 62 us).
// S has two TMEM buffers: while the softmax warps turn S(n), dP(n) into dS(n) (bf16, over
// S(n)'s columns), S(n + 1) is computed, and dP(n + 1) as soon as dP(n) has been read.
// ---------------------------------------------------------------------------
// {-lse log2(e) (-inf: no key left), D} of packed rows of an item: rows first + u 256/D, u <
// STEPS, D/8 lanes to a row, 16 bytes each, with O = o + o_res.  `load` only starts the loads.
template <int D, int STEPS>
struct RowStats {
  static constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  uint4 xo[STEPS], xr[STEPS], xd[STEPS];
  float lse[STEPS];
  __device__ __forceinline__ void load(const DenseArgs& a, const DenseItem& it, int q0, int g,
                                       int first) {
    const int toks = min(a.tpt, it.len - q0), at = (threadIdx.x & 31) % kLanes * 8;
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      // rows behind the last one read an earlier row, so that no load is conditional
      const int rr = first + u * kRows, tok = min(rr / a.G, toks - 1), hh = g * a.G + rr % a.G;
      const size_t t = (size_t)(it.start + q0 + tok), row = t * a.hq + hh;
      xo[u] = ld_nc_v4(a.o + row * D + at);
      xr[u] = ld_nc_v4(a.o_res + row * D + at);
      xd[u] = ld_nc_v4(a.d_o + t * a.do_stride + (size_t)hh * D + at);
      lse[u] = __ldg(a.lse + row);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      xo[u] = xr[u] = xd[u] = make_uint4(0, 0, 0, 0);
      lse[u] = 0.f;
    }
  }
  // to `rows` (by packed row) and to a.stats
  __device__ __forceinline__ void store(const DenseArgs& a, const DenseItem& it, int q0, int g,
                                        int first, float2* rows) const {
    const int toks = min(a.tpt, it.len - q0);
    auto dot = [](uint32_t o, uint32_t res, uint32_t d_o) {
      return (bf16_lo(o) + bf16_lo(res)) * bf16_lo(d_o) +
             (bf16_hi(o) + bf16_hi(res)) * bf16_hi(d_o);
    };
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      float s = (dot(xo[u].x, xr[u].x, xd[u].x) + dot(xo[u].y, xr[u].y, xd[u].y)) +
                (dot(xo[u].z, xr[u].z, xd[u].z) + dot(xo[u].w, xr[u].w, xd[u].w));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const int rr = first + u * kRows, tok = rr / a.G;
      if ((threadIdx.x & 31) % kLanes == 0) {
        const bool there = tok < toks;
        const float2 v = make_float2(there && lse[u] != -INFINITY ? -lse[u] * kLog2E : -INFINITY,
                                     there ? s : 0.f);
        rows[rr] = v;
        if (there) a.stats[(size_t)(g * a.G + rr % a.G) * a.T + it.start + q0 + tok] = v;
      }
    }
  }
};

template <int D, bool BIAS>
struct DqCfg {
  static constexpr int kTile = 128 * D * 2;
  // K and V rings; with a bias its tables take the place of a tile
  static constexpr int kNK = D == 128 ? 3 : 4, kNV = D == 128 ? (BIAS ? 1 : 2) : 3;
  static constexpr int kSmem = (2 + kNK + kNV) * kTile + 256 + 2 * 1024 +
                               (BIAS ? (int)sizeof(DenseBias) : 0);
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(dense_turns(kNK) && dense_turns(kNV) && dense_turns(2), "counts are turned back");
};

template <int D, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    k_dense_dq(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ DenseArgs a) {
  using C = DqCfg<D, BIAS>;
  constexpr int NCH = D / 64, NK = C::kNK, NV = C::kNV;
  constexpr bool kRowWarps = D == 128;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sO = sQ + C::kTile;
  uint8_t* sK = sO + C::kTile;
  uint8_t* sV = sK + NK * C::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NV * C::kTile);
  // Q and dO loaded / free | rings | S buffers | dP ready, read | dS buffers | dQ complete |
  // row statistics ready, free
  constexpr int B_Q = 0, B_QE = 1, B_KF = 2, B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + NV,
                B_S = B_VE + NV, B_DP = B_S + 2, B_DPE = B_DP + 1, B_DS = B_DPE + 1,
                B_DQ = B_DS + 2, B_RF = B_DQ + 1, B_RE = B_RF + 2, B_END = B_RE + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + B_END + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((B_END + 1) * 8 + 8 <= 256, "barrier block");
  float2* sRow = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(bars) + 256);  // [2][128]
  DenseBias* sB = reinterpret_cast<DenseBias*>(sRow + 256);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (blockIdx.x == 0 && warp == 11) dense_check_docs(a);
  DenseDocs docs;
  dense_docs_load(a, docs);
  if (!dense_docs(a, a.tpt, docs)) return;

  if (threadIdx.x == 0) {
    mbar_init(bar(B_Q), 1);
    mbar_init(bar(B_QE), 1);
    for (int s = 0; s < NK; ++s) mbar_init(bar(B_KF + s), 1), mbar_init(bar(B_KE + s), 1);
    for (int s = 0; s < NV; ++s) mbar_init(bar(B_VF + s), 1), mbar_init(bar(B_VE + s), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B_S + b), 1);
      mbar_init(bar(B_DS + b), 8);
      mbar_init(bar(B_RF + b), 2);
      mbar_init(bar(B_RE + b), 8);
    }
    mbar_init(bar(B_DP), 1);
    mbar_init(bar(B_DPE), 8);
    mbar_init(bar(B_DQ), 1);
    mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tslot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(tslot);
  // TMEM: S/dS buffer b at columns [128 b, 128 b + 128), dP at 256, dQ at 384.  dS of the
  // columns of warpgroup w starts at column 64 w of its buffer.

  // The items of this CTA, in the same order for every role; ring positions and barrier
  // phases run on from item to item (X: tiles so far).
  struct Work {
    DenseItem it;
    int g, q0;
    int N;  // key tiles; 0: nothing to compute
  };
  const int rounds = dense_rounds(a);
  auto work = [&](int k, Work& w) -> bool {
    int slot;
    if (!dense_round(a, k, &slot, &w.g) || !dense_item<false>(a, docs, slot, a.tpt, w.it))
      return false;
    w.q0 = w.it.tile * a.tpt;
    w.N = w.it.doc < a.ndoc ? (min(w.q0 + a.tpt, w.it.len) + 127) >> 7 : 0;
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<kRegsCtl>();
    if (warp == 8) {
      // ------------------------------ loads --------------------------------------
      int X = 0, xk = 0, xv = 0, items = 0;  // tiles; K and V loads issued
      bool ok = true;
      auto wait = [&](int b, uint32_t par, int n) {
        return dense_wait(bar(b), par, abort_flag, a.status, wait_site(kKerDenseDq, b, n));
      };
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.N == 0) continue;
        if (items > 0 && !(ok = wait(B_QE, (items - 1) & 1, items))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_Q), 2 * NCH * (uint32_t)a.tpt * a.G * 128);
          for (int c = 0; c < NCH; ++c) {
            tma_load_3d(smem_u32(sQ + c * 16384), &tm_q, bar(B_Q), 64 * c, w.g * a.G,
                        w.it.start + w.q0);
            tma_load_3d(smem_u32(sO + c * 16384), &tm_do, bar(B_Q), 64 * c, w.g * a.G,
                        w.it.start + w.q0);
          }
        }
        ++items;
        for (int n = 0; n < w.N; ++n, ++X) {
          const int sk = X % NK, sv = X % NV, tok = w.it.start + n * 128;
          if (X >= NK && !(ok = wait(B_KE + sk, ((X / NK) & 1) ^ 1, n))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_KF + sk), C::kTile);
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(smem_u32(sK + sk * C::kTile + c * 16384), &tm_k, bar(B_KF + sk), 64 * c,
                          w.g, tok);
          }
          xk = X + 1;
          if (X >= NV && !(ok = wait(B_VE + sv, ((X / NV) & 1) ^ 1, n))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_VF + sv), C::kTile);
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(smem_u32(sV + sv * C::kTile + c * 16384), &tm_v, bar(B_VF + sv), 64 * c,
                          w.g, tok);
          }
          xv = X + 1;
        }
        __syncwarp();
        X = dense_turn(X);
      }
      if (*abort_flag) {  // copies in flight land before the CTA leaves
        if (items > 0) drain_bar(bar(B_Q), (items - 1) & 1);
        for (int y = max(0, xk - NK); y < xk; ++y) drain_bar(bar(B_KF + y % NK), (y / NK) & 1);
        for (int y = max(0, xv - NV); y < xv; ++y) drain_bar(bar(B_VF + y % NV), (y / NV) & 1);
      }
    } else if (warp == 9) {
      // ------------------------------ MMA issue ----------------------------------
      constexpr uint32_t idS = make_idesc_bf16(128, 128, false, false);
      constexpr uint32_t idQ = make_idesc_bf16(128, D, false, true);
      const uint32_t el = elect_one(), tm = uniform(tbase);
      constexpr uint32_t T16 = C::kTile >> 4;
      const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), o_lo = desc_lo(smem_u32(sO), 16),
                     k_lo = desc_lo(smem_u32(sK), 16), v_lo = desc_lo(smem_u32(sV), 16),
                     kt_lo = desc_lo(smem_u32(sK), 16384);
      auto wait = [&](int b, uint32_t par, int n) {
        return dense_wait(bar(b), par, abort_flag, a.status, wait_site(kKerDenseDq, b, n));
      };
      int X = 0, items = 0, len = 0;
      auto s_of = [&](int x, int n) -> bool {
        if (!wait(B_KF + x % NK, (x / NK) & 1, n)) return false;
        // keys behind the document's end: dS is zero there, K must be finite
        if ((n + 1) * 128 > len) dense_zero_rows<D>(sK + (x % NK) * C::kTile, len - n * 128);
        tc_fence_after();
        mma_tile_ss<D>(el, tm + 128 * (x & 1), q_lo, k_lo + (x % NK) * T16, idS);
        mma_commit(el, bar(B_S + (x & 1)));
        return true;
      };
      auto dp_of = [&](int x, int n) -> bool {
        if (!wait(B_VF + x % NV, (x / NV) & 1, n)) return false;
        if (x > 0 && !wait(B_DPE, (x - 1) & 1, n)) return false;
        tc_fence_after();
        mma_tile_ss<D>(el, tm + 256, o_lo, v_lo + (x % NV) * T16, idS);
        mma_commit(el, bar(B_DP));
        mma_commit(el, bar(B_VE + x % NV));
        return true;
      };
      bool ok = true;
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.N == 0) continue;
        const int NT = uniform(w.N);
        len = uniform(w.it.len);
        ok = wait(B_Q, items & 1, items) && s_of(X, 0) && dp_of(X, 0);
        ++items;
        if (ok && NT == 1) mma_commit(el, bar(B_QE));
        for (int n = 0; ok && n < NT; ++n, ++X) {
          if (n + 1 < NT) {
            if (!(ok = s_of(X + 1, n + 1) && dp_of(X + 1, n + 1))) break;
            if (n + 2 == NT) mma_commit(el, bar(B_QE));  // the last use of Q and dO
          }
          if (!(ok = wait(B_DS + (X & 1), (X >> 1) & 1, n))) break;
          tc_fence_after();
          const uint32_t kt = kt_lo + (X % NK) * T16, ds = tm + 128 * (X & 1);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(el, tm + 384, ds + 64 * (kk >> 2) + 8 * (kk & 3), kt + kk * (2048 >> 4), idQ,
                   n > 0 || kk > 0);
          mma_commit(el, bar(B_KE + X % NK));
        }
        mma_commit(el, bar(B_DQ));
        X = dense_turn(X);
      }
      if (!ok) {  // products in flight end before TMEM is freed
        mma_commit(el, bar(B_END));
        drain_bar(bar(B_END), 0);
      }
    } else if (kRowWarps) {
      // ------------------------------ row statistics ------------------------------
      // 64 rows per warp
      using Stats = RowStats<D, 4>;
      int items = 0;
      bool ok = true;
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.N == 0) continue;
        const int b = items & 1;
        if (items >= 2 && !(ok = dense_wait(bar(B_RE + b), ((items >> 1) & 1) ^ 1, abort_flag,
                                            a.status, wait_site(kKerDenseDq, B_RE + b, items))))
          break;
#pragma unroll 1
        for (int r0 = (warp - 10) * 64; r0 < (warp - 9) * 64; r0 += Stats::kRows * 4) {
          const int first = r0 + lane / Stats::kLanes;
          Stats x;
          x.load(a, w.it, w.q0, w.g, first);
          x.store(a, w.it, w.q0, w.g, first, sRow + b * 128);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_RF + b));
        ++items;
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------ dS ---------------------------------------------
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tl = tbase + lane_off;
    const int ti = r / a.G, hl = r % a.G;
    // this row's bucket sums: a row meets the distances in falling order, so a
    // bucket is finished when the next one begins and is stored once
    float* my = BIAS ? a.slots + (size_t)blockIdx.x * a.nb * 256 + w * 128 + r : nullptr;
    float2* sums = BIAS ? a.parts + (size_t)blockIdx.x * a.hq * a.nb : nullptr;
    if (BIAS)
      for (int x = threadIdx.x; x < a.hq * a.nb; x += 256) sums[x] = make_float2(0.f, 0.f);
    bool dead = false;
    int X = 0, items = 0, table_of = -1;  // table_of: KV head the bias tables are of
    // row statistics, 16 rows per warp
    using Stats = RowStats<D, D / 16>;
    const int dr0 = (warp & 3) * 32 + 16 * w + lane / Stats::kLanes;
    Stats rs;
    // the next item with something to compute, from round k on; what has none is written
    auto seek = [&](int& k, Work& wk) -> bool {
      for (; k < rounds; ++k) {
        if (!work(k, wk)) continue;
        if (wk.N > 0) return true;
        if (wk.it.doc == a.ndoc) {  // padding behind the last document: zero rows
          const int n = min(a.tpt, wk.it.len - wk.q0) * a.G, rr = (int)threadIdx.x;
          if (rr < n)
            dense_zero_row(a.dq + ((size_t)(wk.it.start + wk.q0 + rr / a.G) * a.hq +
                                   wk.g * a.G + rr % a.G) * D, D);
        }
      }
      return false;
    };
    int k = 0;
    Work wk;
    bool have = seek(k, wk);
    auto next_stats = [&]() {
      rs.clear();  // kept across the tile loop otherwise
      if (have) rs.load(a, wk.it, wk.q0, wk.g, dr0);
    };
    if (!kRowWarps) next_stats();
    while (have) {
      float2* part = BIAS ? sums + (size_t)wk.g * a.G * a.nb : nullptr;
      if (BIAS && table_of != wk.g) {
        dense_bias_tables<true>(a, sB, wk.g);
        table_of = wk.g;
      }
      const int qi = wk.q0 + ti;
      const bool valid = ti < a.tpt && qi < wk.it.len;
      const size_t row = (size_t)(wk.it.start + qi) * a.hq + wk.g * a.G + hl;
      const int rb = kRowWarps ? items & 1 : 0;
      if (kRowWarps) {
        dead = dead || !dense_wait(bar(B_RF + rb), (items >> 1) & 1, abort_flag, a.status,
                                   wait_site(kKerDenseDq, B_RF + rb, items));
      } else {
        rs.store(a, wk.it, wk.q0, wk.g, dr0, sRow);
        named_bar_sync(1, 256);
      }
      const float nl = sRow[rb * 128 + r].x, dsum = sRow[rb * 128 + r].y;
      if (kRowWarps) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_RE + rb));
      }
      float acc = 0.f;
      uint64_t done = 0;                 // buckets stored
      int bk = a.nb - 1, stk = INT_MAX;  // bucket of the next scores and its first distance
      float bias0 = 0.f;                 // its bias
      const uint16_t* tab = a.bias + (size_t)(wk.g * a.G + hl) * a.nb;
      float c = a.scale_log2, ref = 0.f;
      if (BIAS) {
        ref = dense_row_ref(a, sB, hl, tab, valid ? qi : -1);
        c = dense_row_scale(a, ref);
        if (w == 0 && valid) a.refs[(size_t)(wk.g * a.G + hl) * a.T + wk.it.start + qi] = ref;
      }
      for (int n = 0; n < wk.N; ++n, ++X) {
        const int b = X & 1;
        const int rel = valid ? qi - n * 128 - 64 * w : -1;  // columns 0..rel are visible
        const bool edge = __any_sync(0xffffffffu, rel < 63);
        auto wait = [&](int bb, uint32_t par) {
          dead = dead || !dense_wait(bar(bb), par, abort_flag, a.status,
                                     wait_site(kKerDenseDq, bb, n));
          tc_fence_after();
        };
        bool one = true, near = false;  // see DenseBias
        if (BIAS) {
          if (__any_sync(0xffffffffu, rel < stk)) {  // the row's first bucket here is another
            const int first = dense_bucket(sB, rel);
            if (first != bk) {
              my[bk * 256] = acc;
              done |= 1ull << bk;
              acc = 0.f;
              bk = first;
            }
            stk = bk > 0 ? sB->starts[bk] : INT_MIN;
            bias0 = dense_bias_log2(__ldg(tab + bk), ref);
          }
          one = __all_sync(0xffffffffu, bk == 0 || stk <= rel - 63);
          near = __all_sync(0xffffffffu, rel < a.lut_w && ref == 0.f);
        }
        uint32_t x[2][32];
        wait(B_S + b, (X >> 1) & 1);
        if (!dead) {
          tmem_ld32x2(tl + 128 * b + 64 * w, tl + 128 * b + 64 * w + 32, x[0], x[1]);
          // P = 2^(S scale log2(e) + bias - lse)
          if (one) {
            const float sub = nl + bias0;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              x[i >> 5][i & 31] = __float_as_uint(
                  ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), c, sub)));
          } else {
            if (near) {
              const float* lut = sB->lut + hl * a.lut_stride + dense_lut_pad(a) + rel;
#pragma unroll
              for (int i = 0; i < 64; ++i)
                x[i >> 5][i & 31] = __float_as_uint(ex2_approx(
                    fmaf(__uint_as_float(x[i >> 5][i & 31]), c, nl + lut[-i])));
            } else if (__all_sync(0xffffffffu, bk < 2 || sB->starts[bk - 1] <= rel - 63)) {
              // at most one start inside: scores before `cut` take v0, the others v1
              const int cut = bk > 0 ? rel - sB->starts[bk] + 1 : 64;
              const float v0 = nl + bias0;
              const float v1 = nl + dense_bias_log2(__ldg(tab + max(bk - 1, 0)), ref);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                if (__any_sync(0xffffffffu, cut > 16 * u && cut < 16 * u + 16)) {
#pragma unroll
                  for (int i = 16 * u; i < 16 * u + 16; ++i)
                    x[i >> 5][i & 31] = __float_as_uint(ex2_approx(fmaf(
                        __uint_as_float(x[i >> 5][i & 31]), c, i < cut ? v0 : v1)));
                } else {
                  const float sub = 16 * u < cut ? v0 : v1;
#pragma unroll
                  for (int i = 16 * u; i < 16 * u + 16; ++i)
                    x[i >> 5][i & 31] = __float_as_uint(
                        ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), c, sub)));
                }
              }
            } else {
              int q = bk;
              int st = q > 0 ? sB->starts[q] : INT_MIN;
              float sub = nl + bias0;
#pragma unroll
              for (int i = 0; i < 64; ++i) {
                if (rel - i < st) {
                  --q;
                  st = q > 0 ? sB->starts[q] : INT_MIN;
                  sub = nl + dense_bias_log2(__ldg(tab + q), ref);
                }
                x[i >> 5][i & 31] = __float_as_uint(
                    ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), c, sub)));
              }
            }
            __syncwarp();
          }
          wait(B_DP, X & 1);
          if (!dead) {
            uint32_t y[2][32];
            tmem_ld32x2(tl + 256 + 64 * w, tl + 256 + 64 * w + 32, y[0], y[1]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DPE));
#pragma unroll
            for (int i = 0; i < 64; ++i)
              x[i >> 5][i & 31] =
                  __float_as_uint(__uint_as_float(x[i >> 5][i & 31]) *
                                  (__uint_as_float(y[i >> 5][i & 31]) - dsum));
            if (edge) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (i > rel) x[i >> 5][i & 31] = 0;
            }
            if (BIAS) {
              if (one) {
                float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 64; ++i) s4[i & 3] += __uint_as_float(x[i >> 5][i & 31]);
                acc += (s4[0] + s4[1]) + (s4[2] + s4[3]);
              } else {
                // bit i of `last`: score i is the last of its bucket in this row
                uint32_t last[2];
                if (rel < kDenseBits) {
                  const int p = rel - 63 + kDenseBitsPad;
                  const uint32_t* b = sB->bits + (p >> 5);
                  last[1] = __brev(__funnelshift_r(b[0], b[1], p & 31));
                  last[0] = __brev(__funnelshift_r(b[1], b[2], p & 31));
                } else {
                  last[0] = last[1] = 0;
                  for (int q = bk; q > 0 && sB->starts[q] >= rel - 63; --q) {
                    const int i = rel - sB->starts[q];
                    last[i >> 5] |= 1u << (i & 31);
                  }
                }
                float* to = my + bk * 256;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  if (__any_sync(0xffffffffu, (last[u >> 1] >> (16 * (u & 1))) & 0xffffu)) {
#pragma unroll
                    for (int i = 16 * u; i < 16 * u + 16; ++i) {
                      acc += __uint_as_float(x[i >> 5][i & 31]);
                      if (last[u >> 1] & (1u << (i & 31))) {
                        *to = acc;
                        to -= 256;
                        acc = 0.f;
                      }
                    }
                  } else {
                    float s2[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 16 * u; i < 16 * u + 16; ++i)
                      s2[i & 1] += __uint_as_float(x[i >> 5][i & 31]);
                    acc += s2[0] + s2[1];
                  }
                }
                const int was = bk;
                bk -= __popc(last[0]) + __popc(last[1]);
                done |= (2ull << was) - (2ull << bk);  // bk + 1 .. was
                stk = INT_MAX;  // looked up again for the next tile
                __syncwarp();  // the TMEM store below is warp-collective
              }
            }
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = pack_bf16(__uint_as_float(x[i >> 4][2 * (i & 15)]),
                               __uint_as_float(x[i >> 4][2 * (i & 15) + 1]));
            tmem_st32(tl + 128 * b + 64 * w, v);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (dead) mbar_arrive(bar(B_DPE));
          // one barrier per buffer: a warpgroup may be a tile ahead of the other here
          mbar_arrive(bar(B_DS + b));
        }
      }
      ++items;
      X = dense_turn(X);
      if (BIAS) {
        my[bk * 256] = acc;
        done |= 1ull << bk;
        for (int b = 0; b < a.nb; ++b)  // buckets that the row does not reach
          if (!((done >> b) & 1)) my[b * 256] = 0.f;
        // Sums over the item's rows, head by head, in a fixed order: a warp takes every eighth
        // bucket, four at a time; P lanes to a head add up every P-th token each, and then
        // pairwise (more than 32 heads: one lane to a head, 32 heads at a time), and add that to
        // the CTA's sum: the same thread for the same entry each time.  The first barrier
        // orders the stores above before the loads, the second the loads before the next
        // item's stores.
        __threadfence_block();
        named_bar_sync(2, 256);
        const float* all = a.slots + (size_t)blockIdx.x * a.nb * 256;
        const int P = max(32 / a.G, 1), step = P * a.G, pt = lane / a.G;
        for (int b0 = warp; b0 < a.nb; b0 += 32) {
          for (int h0 = 0; h0 < a.G; h0 += 32) {
            const int h = h0 + lane;
            const int end = h < step ? a.tpt * a.G : 0;  // lanes left over have no rows
            float2 sum[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              sum[u] = part[min(h, a.G - 1) * a.nb + min(b0 + 8 * u, a.nb - 1)];
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            for (int x0 = h; __any_sync(0xffffffffu, x0 < end); x0 += 5 * step) {
              float y[4][5][2];  // all loads unconditional, so that they run together
#pragma unroll
              for (int j = 0; j < 5; ++j) {
                const float* p = all + min(x0 + j * step, 127);
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    y[u][j][e] = ld_cg_f32(p + min(b0 + 8 * u, a.nb - 1) * 256 + 128 * e);
              }
#pragma unroll
              for (int j = 0; j < 5; ++j)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  v[u] += x0 + j * step < end ? y[u][j][0] + y[u][j][1] : 0.f;
            }
            for (int o = 16; o > 0; o >>= 1) {
              if (o >= P) continue;
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float other = __shfl_down_sync(0xffffffffu, v[u], o * a.G);
                if (pt < o && pt + o < P) v[u] += other;
              }
            }
            if (h < a.G) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (b0 + 8 * u < a.nb) {
                  add_pair(sum[u], v[u]);
                  part[h * a.nb + b0 + 8 * u] = sum[u];
                }
            }
          }
        }
        named_bar_sync(2, 256);
      }
      ++k;
      have = seek(k, wk);
      if (!kRowWarps) next_stats();
      dead = dead || !dense_wait(bar(B_DQ), (items - 1) & 1, abort_flag, a.status,
                                 wait_site(kKerDenseDq, B_DQ, items));
      tc_fence_after();
      if (!dead && w < D / 64) {  // 64 columns each (d = 64: the first warpgroup)
        uint32_t v[64];
        tmem_ld_row(tl + 384 + 64 * w, v);
        dense_store_row(v, a.scale, valid ? a.dq + row * D + 64 * w : nullptr);
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------------------
// dK, dV: items of 128 keys of a KV head against the queries of its group, head by head,
// 128 queries at a time.  Transposed products, so that a key is one TMEM lane:
// S^T = K Q^T, dP^T = V dO^T, P^T and dS^T go back as bf16 over S^T and dP^T and
// are read from TMEM as the A operand of dV += P^T dO and dK += dS^T Q (no
// probability passes through shared memory).  The four accumulators fill TMEM,
// so the products are ordered dV(n), S(n + 1), dK(n), dP(n + 1): each overlaps
// the exponentials or the dS of the other half.
// Warps 0-3 and 4-7 take 64 of a tile's 128 queries each; warp 8 loads, warp 9
// issues the MMAs, warp 10 brings the rows' {-lse, D}.
// ---------------------------------------------------------------------------
template <int D, bool BIAS>
struct DkvCfg {
  static constexpr int kTile = 128 * D * 2;
  // with a bias its tables take the place of a tile
  static constexpr int kNQ = D == 128 ? (BIAS ? 2 : 3) : 4, kNO = D == 128 ? 2 : 4;  // Q, dO rings
  static constexpr int kNS = 2;  // statistics ring
  static constexpr int kSmem =
      (2 + kNQ + kNO) * kTile + kNS * 1024 + 256 +
      (BIAS ? kNS * 512 + 16 + (int)sizeof(DenseBias) : 0);
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(dense_turns(kNQ) && dense_turns(kNO) && dense_turns(kNS), "counts are turned back");
};

template <int D, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    k_dense_dkv(const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ CUtensorMap tm_do,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ DenseArgs a) {
  using C = DkvCfg<D, BIAS>;
  constexpr int NCH = D / 64, NQ = C::kNQ, NO = C::kNO, NS = C::kNS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::kTile;
  uint8_t* sQ = sV + C::kTile;
  uint8_t* sO = sQ + NQ * C::kTile;
  float2* sSt = reinterpret_cast<float2*>(sO + NO * C::kTile);  // [NS][128] {-lse log2(e), D}
  uint64_t* bars = reinterpret_cast<uint64_t*>(sSt + NS * 128);
  // K and V loaded / free | rings | S^T, P^T, dP^T, dS^T ready | dK and dV complete
  constexpr int B_KV = 0, B_KVE = 1, B_QF = 2, B_QE = B_QF + NQ, B_OF = B_QE + NQ, B_OE = B_OF + NO,
                B_TF = B_OE + NO, B_TE = B_TF + NS, B_S = B_TE + NS, B_P = B_S + 1, B_DP = B_P + 1,
                B_DS = B_DP + 1, B_G = B_DS + 1, B_END = B_G + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + B_END + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((B_END + 1) * 8 + 8 <= 256, "barrier block");
  // the rows' references, and whether one of a tile's is not zero
  float* sRef = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 256);  // [NS][128]
  int* sFar = reinterpret_cast<int*>(sRef + NS * 128);                             // [NS]
  static_assert(NS <= 4, "16 bytes");
  DenseBias* sB = reinterpret_cast<DenseBias*>(sFar + 4);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  DenseDocs docs;
  dense_docs_load(a, docs);
  if (!dense_docs(a, 128, docs)) return;

  if (threadIdx.x == 0) {
    mbar_init(bar(B_KV), 1);
    mbar_init(bar(B_KVE), 1);
    mbar_init(bar(B_G), 1);
    for (int s = 0; s < NQ; ++s) mbar_init(bar(B_QF + s), 1), mbar_init(bar(B_QE + s), 1);
    for (int s = 0; s < NO; ++s) mbar_init(bar(B_OF + s), 1), mbar_init(bar(B_OE + s), 1);
    for (int s = 0; s < NS; ++s) mbar_init(bar(B_TF + s), 1), mbar_init(bar(B_TE + s), 8);
    mbar_init(bar(B_S), 1);
    mbar_init(bar(B_P), 8);
    mbar_init(bar(B_DP), 1);
    mbar_init(bar(B_DS), 8);
    mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tslot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(tslot);
  // TMEM: S^T/P^T at column 0, dP^T/dS^T at 128, dV at 256, dK at 384.  P^T and dS^T of the
  // queries of warpgroup w start at column 64 w of theirs.

  // The items of this CTA, in the same order for every role; ring positions and barrier
  // phases run on from item to item (X: tiles so far).
  struct Work {
    DenseItem it;
    int g, j0;
    int nq, N;  // query tiles of a head, of the group (0: nothing to compute)
  };
  const int rounds = dense_rounds(a);
  auto work = [&](int k, Work& w) -> bool {
    int slot;
    if (!dense_round(a, k, &slot, &w.g) || !dense_item<true>(a, docs, slot, 128, w.it))
      return false;
    w.j0 = w.it.tile * 128;
    w.nq = w.it.doc < a.ndoc ? (w.it.len - w.j0 + 127) >> 7 : 0;
    w.N = w.nq * a.G;
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<kRegsCtl>();
    auto wait = [&](int b, uint32_t par, int n) {
      return dense_wait(bar(b), par, abort_flag, a.status, wait_site(kKerDenseDkv, b, n));
    };
    if (warp == 8) {
      // ------------------------------ loads --------------------------------------
      int X = 0, lq = 0, lo = 0, items = 0;  // tiles; Q and dO loads issued
      bool ok = true;
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.N == 0) continue;
        if (items > 0 && !(ok = wait(B_KVE, (items - 1) & 1, items))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_KV), 2 * C::kTile);
          for (int c = 0; c < NCH; ++c) {
            tma_load_3d(smem_u32(sK + c * 16384), &tm_k, bar(B_KV), 64 * c, w.g, w.it.start + w.j0);
            tma_load_3d(smem_u32(sV + c * 16384), &tm_v, bar(B_KV), 64 * c, w.g, w.it.start + w.j0);
          }
        }
        ++items;
        int h = w.g * a.G, qt = 0;
        for (int n = 0; n < w.N; ++n, ++X) {
          const int sq = X % NQ, so = X % NO, tok = w.it.start + w.j0 + qt * 128;
          if (X >= NQ && !(ok = wait(B_QE + sq, ((X / NQ) & 1) ^ 1, n))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_QF + sq), C::kTile);
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(smem_u32(sQ + sq * C::kTile + c * 16384), &tm_q, bar(B_QF + sq), 64 * c,
                          h, tok);
          }
          lq = X + 1;
          if (X >= NO && !(ok = wait(B_OE + so, ((X / NO) & 1) ^ 1, n))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_OF + so), C::kTile);
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(smem_u32(sO + so * C::kTile + c * 16384), &tm_do, bar(B_OF + so), 64 * c,
                          h, tok);
          }
          lo = X + 1;
          if (++qt == w.nq) qt = 0, ++h;
        }
        __syncwarp();
        X = dense_turn(X);
      }
      if (*abort_flag) {  // copies in flight land before the CTA leaves
        if (items > 0) drain_bar(bar(B_KV), (items - 1) & 1);
        for (int y = max(0, lq - NQ); y < lq; ++y) drain_bar(bar(B_QF + y % NQ), (y / NQ) & 1);
        for (int y = max(0, lo - NO); y < lo; ++y) drain_bar(bar(B_OF + y % NO), (y / NO) & 1);
      }
    } else if (warp == 9) {
      // ------------------------------ MMA issue ----------------------------------
      constexpr uint32_t idS = make_idesc_bf16(128, 128, false, false);
      constexpr uint32_t idG = make_idesc_bf16(128, D, false, true);
      const uint32_t el = elect_one(), tm = uniform(tbase);
      constexpr uint32_t T16 = C::kTile >> 4;
      const uint32_t k_lo = desc_lo(smem_u32(sK), 16), v_lo = desc_lo(smem_u32(sV), 16),
                     q_lo = desc_lo(smem_u32(sQ), 16), o_lo = desc_lo(smem_u32(sO), 16),
                     qt_lo = desc_lo(smem_u32(sQ), 16384), ot_lo = desc_lo(smem_u32(sO), 16384);
      int X = 0, items = 0, left = 0, nqt = 1;
      // waits for tile n (x over all items) of a ring; queries behind the document's end are
      // zeroed: their probabilities are zero, but the products sum over them
      auto arrived = [&](int bf, int depth, uint8_t* ring, int x, int n) -> bool {
        if (!wait(bf + x % depth, (x / depth) & 1, n)) return false;
        const int i0 = (n % nqt) * 128;
        if (i0 + 128 > left) dense_zero_rows<D>(ring + (x % depth) * C::kTile, left - i0);
        tc_fence_after();
        return true;
      };
      auto gradient = [&](uint32_t d, uint32_t ta, uint32_t b_lo, int n) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(el, d, ta + 64 * (kk >> 2) + 8 * (kk & 3), b_lo + kk * (2048 >> 4), idG,
                 n > 0 || kk > 0);
      };
      auto s_of = [&](int x, int n) -> bool {
        if (!arrived(B_QF, NQ, sQ, x, n)) return false;
        mma_tile_ss<D>(el, tm, k_lo, q_lo + (x % NQ) * T16, idS);
        mma_commit(el, bar(B_S));
        return true;
      };
      auto dp_of = [&](int x, int n) -> bool {
        if (!arrived(B_OF, NO, sO, x, n)) return false;
        mma_tile_ss<D>(el, tm + 128, v_lo, o_lo + (x % NO) * T16, idS);
        mma_commit(el, bar(B_DP));
        return true;
      };
      bool ok = true;
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.N == 0) continue;
        const int NT = uniform(w.N);
        left = uniform(w.it.len - w.j0);
        nqt = uniform(w.nq);
        ok = wait(B_KV, items & 1, items) && s_of(X, 0) && dp_of(X, 0);
        ++items;
        if (ok && NT == 1) mma_commit(el, bar(B_KVE));
        for (int n = 0; ok && n < NT; ++n, ++X) {
          if (!(ok = wait(B_P, X & 1, n))) break;
          tc_fence_after();
          gradient(tm + 256, tm, ot_lo + (X % NO) * T16, n);
          mma_commit(el, bar(B_OE + X % NO));
          if (n + 1 < NT && !(ok = s_of(X + 1, n + 1))) break;
          if (!(ok = wait(B_DS, X & 1, n))) break;
          tc_fence_after();
          gradient(tm + 384, tm + 128, qt_lo + (X % NQ) * T16, n);
          mma_commit(el, bar(B_QE + X % NQ));
          if (n + 1 < NT && !(ok = dp_of(X + 1, n + 1))) break;
          if (n + 2 == NT) mma_commit(el, bar(B_KVE));  // the last use of K and V
        }
        mma_commit(el, bar(B_G));
        X = dense_turn(X);
      }
      if (!ok) {  // products in flight end before TMEM is freed
        mma_commit(el, bar(B_END));
        drain_bar(bar(B_END), 0);
      }
    } else if (warp == 10) {
      // ------------------------------ statistics ---------------------------------
      int X = 0;
      bool ok = true;
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.N == 0) continue;
        int h = w.g * a.G, qt = 0;
        for (int n = 0; n < w.N; ++n, ++X) {
          const int s = X % NS;
          const float2* src = a.stats + (size_t)h * a.T + w.it.start + w.j0 + qt * 128;
          const int left = w.it.len - w.j0 - qt * 128;
          float2 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            v[u] = lane + 32 * u < left ? __ldg(src + lane + 32 * u) : make_float2(-INFINITY, 0.f);
          float f[4];
          bool far = false;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            f[u] = BIAS && lane + 32 * u < left
                       ? __ldg(a.refs + (src - a.stats) + lane + 32 * u)
                       : 0.f;
            far |= f[u] != 0.f;
          }
          if (X >= NS && !(ok = wait(B_TE + s, ((X / NS) & 1) ^ 1, n))) break;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            sSt[s * 128 + lane + 32 * u] = v[u];
            if (BIAS) sRef[s * 128 + lane + 32 * u] = f[u];
          }
          if (BIAS) {
            far = __any_sync(0xffffffffu, far);
            if (lane == 0) sFar[s] = far;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_TF + s));
          if (++qt == w.nq) qt = 0, ++h;
        }
        X = dense_turn(X);
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------ P^T and dS^T ------------------------------------
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // key of the tile
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    bool dead = false;
    int X = 0, items = 0, table_of = -1;  // table_of: KV head the bias tables are of
    for (int k = 0; k < rounds; ++k) {
      Work wk;
      if (!work(k, wk)) continue;
      if (wk.it.doc == a.ndoc) {  // padding behind the last document: zero rows
        const int rr = (int)threadIdx.x;
        if (rr < min(128, wk.it.len - wk.j0)) {
          const size_t row = (size_t)(wk.it.start + wk.j0 + rr) * a.hkv + wk.g;
          dense_zero_row(a.dk + row * D, D);
          dense_zero_row(a.dv + row * D, D);
        }
        continue;
      }
      if (BIAS && table_of != wk.g) {
        dense_bias_tables<false>(a, sB, wk.g);
        table_of = wk.g;
      }
      int qt = 0, hl = 0;
      int bk = 0, stn = 0;  // bias: bucket of the next queries, first distance of the one behind
      float bias0 = 0.f;    // its bias
      for (int n = 0; n < wk.N; ++n, ++X) {
        const int s = X % NS;
        const int rel = qt * 128 + 64 * w - r;  // distance of the first of this warpgroup's queries
        const bool diag = qt == 0;              // queries c with rel + c < 0 come before the key
        auto wait = [&](int bb, uint32_t par) {
          dead = dead || !dense_wait(bar(bb), par, abort_flag, a.status,
                                        wait_site(kKerDenseDkv, bb, n));
          tc_fence_after();
        };
        uint32_t x[2][32];
        const float4* st = reinterpret_cast<const float4*>(sSt + s * 128 + 64 * w);
        bool one = true, near = false;  // see DenseBias
        const uint16_t* tab = a.bias + (size_t)(wk.g * a.G + hl) * a.nb;
        if (BIAS) {
          if (qt == 0 || __any_sync(0xffffffffu, rel >= stn)) {  // another head, or bucket
            bk = dense_bucket(sB, rel);
            stn = bk + 1 < a.nb ? sB->starts[bk + 1] : INT_MAX;
            bias0 = dense_bias_log2(__ldg(tab + bk));
          }
          one = __all_sync(0xffffffffu, stn > rel + 63);
          near = __all_sync(0xffffffffu, rel + 63 < a.lut_w);
        }
        wait(B_TF + s, (X / NS) & 1);
        // Bucket by bucket, relative to each query's reference: where a query of the tile has
        // one, and, if the table has NaN, +inf or entries that overflow, where the tile has queries
        // behind the document's end, whose distances may reach buckets that no pair does.
        const int end = wk.it.len - wk.j0 - qt * 128 - 64 * w;
        const bool walk = BIAS && (sFar[s] || (sB->loose && end < 64));
        if (walk) one = near = false;
        wait(B_S, X & 1);
        if (!dead) {
          tmem_ld32x2(tl + 64 * w, tl + 64 * w + 32, x[0], x[1]);
          const float c = a.scale_log2;
          if (one) {
            const float bv = bias0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float4 v = st[i];
              const int e = 2 * i;
              x[e >> 5][e & 31] = __float_as_uint(ex2_approx(
                  fmaf(__uint_as_float(x[e >> 5][e & 31]), c, BIAS ? v.x + bv : v.x)));
              x[e >> 5][(e & 31) + 1] = __float_as_uint(ex2_approx(
                  fmaf(__uint_as_float(x[e >> 5][(e & 31) + 1]), c, BIAS ? v.z + bv : v.z)));
            }
          } else {
            const float2* sl = sSt + s * 128 + 64 * w;
            if (near) {
              const float* lut = sB->lut + hl * a.lut_stride + dense_lut_pad(a) + rel;
#pragma unroll
              for (int i = 0; i < 64; ++i)
                x[i >> 5][i & 31] = __float_as_uint(
                    ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), c, sl[i].x + lut[i])));
            } else if (!walk && __all_sync(0xffffffffu, bk + 2 >= a.nb ||
                                                            sB->starts[bk + 2] > rel + 63)) {
              // at most one start inside: queries before `cut` take v0, the others v1
              const int nx = min(bk + 1, a.nb - 1);
              const int cut = bk + 1 < a.nb ? sB->starts[nx] - rel : 64;
              const float v0 = bias0;
              const float v1 = dense_bias_log2(__ldg(tab + nx));
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                if (__any_sync(0xffffffffu, cut > 16 * u && cut < 16 * u + 16)) {
#pragma unroll
                  for (int i = 16 * u; i < 16 * u + 16; ++i)
                    x[i >> 5][i & 31] = __float_as_uint(ex2_approx(fmaf(
                        __uint_as_float(x[i >> 5][i & 31]), c, sl[i].x + (i < cut ? v0 : v1))));
                } else {
                  const float bv = 16 * u < cut ? v0 : v1;
#pragma unroll
                  for (int i = 16 * u; i < 16 * u + 16; ++i)
                    x[i >> 5][i & 31] = __float_as_uint(
                        ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), c, sl[i].x + bv)));
                }
              }
            } else {
              const float* rf = sRef + s * 128 + 64 * w;
              int q = bk;
              int nx = q + 1 < a.nb ? sB->starts[q + 1] : INT_MAX;
              uint16_t raw = __ldg(tab + q);
#pragma unroll
              for (int i = 0; i < 64; ++i) {
                if (rel + i >= nx) {
                  ++q;
                  nx = q + 1 < a.nb ? sB->starts[q + 1] : INT_MAX;
                  raw = __ldg(tab + q);
                }
                const float y =
                    ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), dense_row_scale(a, rf[i]),
                                    sl[i].x + dense_bias_log2(raw, rf[i])));
                x[i >> 5][i & 31] = i < end ? __float_as_uint(y) : 0;
              }
            }
            __syncwarp();  // the TMEM store below is warp-collective
          }
          if (diag) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (rel + i < 0) x[i >> 5][i & 31] = 0;
          }
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = pack_bf16(__uint_as_float(x[i >> 4][2 * (i & 15)]),
                             __uint_as_float(x[i >> 4][2 * (i & 15) + 1]));
          tmem_st32(tl + 64 * w, v);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P));
        wait(B_DP, X & 1);
        if (!dead) {
          uint32_t y[2][32];
          tmem_ld32x2(tl + 128 + 64 * w, tl + 128 + 64 * w + 32, y[0], y[1]);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float4 v = st[i];
            const int e = 2 * i;
            x[e >> 5][e & 31] =
                __float_as_uint(__uint_as_float(x[e >> 5][e & 31]) *
                                (__uint_as_float(y[e >> 5][e & 31]) - v.y));
            x[e >> 5][(e & 31) + 1] =
                __float_as_uint(__uint_as_float(x[e >> 5][(e & 31) + 1]) *
                                (__uint_as_float(y[e >> 5][(e & 31) + 1]) - v.w));
          }
          if (diag) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (rel + i < 0) x[i >> 5][i & 31] = 0;
          }
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = pack_bf16(__uint_as_float(x[i >> 4][2 * (i & 15)]),
                             __uint_as_float(x[i >> 4][2 * (i & 15) + 1]));
          tmem_st32(tl + 128 + 64 * w, v);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_TE + s));
          mbar_arrive(bar(B_DS));
        }
        if (++qt == wk.nq) qt = 0, ++hl;
      }
      ++items;
      X = dense_turn(X);
      dead = dead || !dense_wait(bar(B_G), (items - 1) & 1, abort_flag, a.status,
                                    wait_site(kKerDenseDkv, B_G, items));
      tc_fence_after();
      if (!dead) {
        // the first warpgroup stores dV, the second dK
        const size_t row = (size_t)(wk.it.start + wk.j0 + r) * a.hkv + wk.g;
        uint16_t* dst = wk.j0 + r < wk.it.len ? (w == 0 ? a.dv : a.dk) + row * D : nullptr;
#pragma unroll 1
        for (int q = 0; q < D / 64; ++q) {
          uint32_t v[64];
          tmem_ld_row(tl + 256 + 128 * w + 64 * q, v);
          dense_store_row(v, w == 0 ? 1.f : a.scale, dst ? dst + 64 * q : nullptr);
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// dtable[h][b] = sum over the CTAs of dQ, in a fixed order: one CTA per head; thread (b, c) sums
// every nc-th CTA's pair, and the nc pairs of a bucket are added pairwise.  A CTA's sum runs over
// all its items, hundreds of thousands for the largest batches, and dS cancels (a row's adds up
// to zero), so the sums carry their roundings along; the result is rounded once, to bf16.
constexpr int kTableThreads = 1024;
__global__ void __launch_bounds__(kTableThreads) k_dense_dtable(const DenseArgs a, int ctas,
                                                                uint16_t* dtable) {
  __shared__ float2 sum[kTableThreads];
  int nb2 = 1;
  while (nb2 < a.nb) nb2 <<= 1;
  const int h = blockIdx.x, b = threadIdx.x % nb2, c = threadIdx.x / nb2, nc = kTableThreads / nb2;
  float2 s = make_float2(0.f, 0.f);
  auto add = [&](float2 x) {
    add_pair(s, x.x);
    s.y += x.y;
  };
  if (b < a.nb)
    for (int x = c; x < ctas; x += nc) add(__ldg(a.parts + ((size_t)x * a.hq + h) * a.nb + b));
  sum[threadIdx.x] = s;
  for (int half = nc / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (c < half) {
      add(sum[threadIdx.x + half * nb2]);
      sum[threadIdx.x] = s;
    }
  }
  if (c == 0 && b < a.nb) {
    // what an infinite sum's roundings drop is NaN
    const __nv_bfloat16 y = __float2bfloat16(fabsf(s.x) < INFINITY ? s.x + s.y : s.x);
    dtable[(size_t)h * a.nb + b] = *reinterpret_cast<const uint16_t*>(&y);
  }
}

template <int D, bool BIAS>
cudaError_t launch_t(const CUtensorMap& mqp, const CUtensorMap& mop, const CUtensorMap& mk,
                     const CUtensorMap& mv, const CUtensorMap& mq, const CUtensorMap& mo,
                     DenseArgs a, cudaStream_t st) {
  cudaError_t e = dense_prepare<k_dense_dq<D, BIAS>>(kThreads, kBudget, DqCfg<D, BIAS>::kSmem);
  if (e != cudaSuccess) return e;
  e = dense_prepare<k_dense_dkv<D, BIAS>>(kThreads, kBudget, DkvCfg<D, BIAS>::kSmem);
  if (e != cudaSuccess) return e;
  a.nslots = dense_slots(a.T, a.ndoc, a.tpt);
  k_dense_dq<D, BIAS><<<dense_grid(a), kThreads, DqCfg<D, BIAS>::kSmem, st>>>(mqp, mop, mk, mv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  a.nslots = dense_slots(a.T, a.ndoc, 128);
  // With a bias persistent CTAs keep their tables; without one an item per CTA, started by the
  // hardware where an SM is free, balances better (packed 32768 tokens, 16 heads: 795
  // against 835 us).
  const int grid = BIAS ? dense_grid(a) : a.nslots * a.hkv;
  k_dense_dkv<D, BIAS><<<grid, kThreads, DkvCfg<D, BIAS>::kSmem, st>>>(mq, mo, mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_bwd(const DenseShape& s, const uint16_t* q, const uint16_t* k,
                             const uint16_t* v, const uint16_t* d_o, uint16_t* dtable,
                             const DenseArgs& a, cudaStream_t st) {
  CUtensorMap mqp, mop, mk, mv, mq, mo;
  cudaError_t e;
  if ((e = make_tmap_rows(&mqp, q, s.d, a.hq, a.T, s.q_stride, a.G, a.tpt)) != cudaSuccess) return e;
  if ((e = make_tmap_rows(&mop, d_o, s.d, a.hq, a.T, s.do_stride, a.G, a.tpt)) != cudaSuccess)
    return e;
  if ((e = make_tmap_rows(&mq, q, s.d, a.hq, a.T, s.q_stride, 1, 128)) != cudaSuccess) return e;
  if ((e = make_tmap_rows(&mo, d_o, s.d, a.hq, a.T, s.do_stride, 1, 128)) != cudaSuccess) return e;
  if ((e = make_tmap_rows(&mk, k, s.d, a.hkv, a.T, s.k_stride, 1, 128)) != cudaSuccess) return e;
  if ((e = make_tmap_rows(&mv, v, s.d, a.hkv, a.T, s.v_stride, 1, 128)) != cudaSuccess) return e;
  if (s.d == 128)
    e = a.bias ? launch_t<128, true>(mqp, mop, mk, mv, mq, mo, a, st)
               : launch_t<128, false>(mqp, mop, mk, mv, mq, mo, a, st);
  else
    e = a.bias ? launch_t<64, true>(mqp, mop, mk, mv, mq, mo, a, st)
               : launch_t<64, false>(mqp, mop, mk, mv, mq, mo, a, st);
  if (e != cudaSuccess || !a.bias) return e;
  DenseArgs b = a;
  b.nslots = dense_slots(a.T, a.ndoc, a.tpt);
  k_dense_dtable<<<a.hq, kTableThreads, 0, st>>>(b, dense_grid(b), dtable);
  return cudaGetLastError();
}

}  // namespace msa
