// Dense causal attention forward over a packed batch (grouped heads, optional
// relative position bias).
//
// One CTA owns 2 x 128 rows of one KV group: rows are (token, head) pairs,
// 128/G tokens x G heads to a tile (rows of a tile that a G not dividing 128
// leaves over are idle), so the group's heads share every K and V tile, and a
// token's heads sit in adjacent TMEM lanes.  K and V tiles of 128 keys stream
// through one TMA ring.  Per row tile t and key tile n:
//   S = Q K^T (tcgen05, both operands in shared memory) into TMEM, then one
//   thread per row: running maximum m and sum l of the softmax in log2 units,
//   P = 2^(S c - m) as bf16 back into the first half of S's columns, and
//   O += P V with P read from TMEM.
// m only moves when a row's maximum has grown by more than 8 (a factor of 256):
// P then stays below 2^8 and the fp32 sums of O and l keep their precision, and
// O is rescaled in TMEM a few times per row instead of once per key tile.
// P is rounded to bf16 for the product (as o itself is); l sums the fp32 values.
//
// Roles (384 threads): warps 0-3 and 4-7 are the softmax warpgroups of tile 0
// and 1, so one tile's softmax overlaps the other's products; warp 8 loads;
// warp 9 issues the MMAs: P V of a tile, then its next S, tile after tile.
// tcgen05 products of one thread run in issue order, so S(n + 1) may be issued
// right behind the product that still reads P(n) from the same columns.
#include "dense_common.cuh"

namespace msa {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsSoftmax = 200, kRegsCtl = 104;
constexpr float kRescale = 8.f;  // log2 growth of a row's maximum that moves m

template <int D, bool BIAS>
struct FwdCfg {
  static constexpr int kTile = 128 * D * 2;
  // K and V tiles in flight; with a bias its tables take the place of one
  static constexpr int kRing = D == 128 ? (BIAS ? 4 : 5) : 8;
  static constexpr int kSmem = (2 + kRing) * kTile + 256 + (BIAS ? (int)sizeof(DenseBias) : 0);
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int D, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    k_dense_fwd(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DenseArgs a) {
  using C = FwdCfg<D, BIAS>;
  constexpr int NCH = D / 64, NR = C::kRing;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;  // [2]; after the last S also the staging of O
  uint8_t* sKV = sQ + 2 * C::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + NR * C::kTile);
  constexpr int B_Q = 0, B_F = 1, B_E = 1 + NR, B_S = 1 + 2 * NR, B_P = B_S + 2, B_P2 = B_S + 4,
                B_PV = B_S + 6, B_END = B_S + 8;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + B_END + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((B_END + 1) * 8 + 8 <= 256, "barrier block");
  DenseBias* sB = reinterpret_cast<DenseBias*>(reinterpret_cast<uint8_t*>(bars) + 256);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (blockIdx.x == 0 && warp == 11) dense_check_docs(a);
  // heaviest tiles of a document first: they end last otherwise
  const int g = blockIdx.x % a.hkv;
  DenseItem it;
  const int tpc = 2 * a.tpt;  // tokens per CTA
  if (!dense_item(a, a.nslots - 1 - (int)(blockIdx.x / a.hkv), tpc, it)) return;
  const int q0 = it.tile * tpc;  // first token of the CTA inside the document
  if (it.doc == a.ndoc) {
    // padding behind the last document: zero rows
    const int n = min(tpc, it.len - q0) * a.G;
    for (int r = threadIdx.x; r < n; r += kThreads) {
      const size_t row = (size_t)(it.start + q0 + r / a.G) * a.hq + g * a.G + r % a.G;
      dense_zero_row(a.o + row * D, D);
      if (a.o_res) dense_zero_row(a.o_res + row * D, D);
      if (a.lse) a.lse[row] = -INFINITY;
    }
    return;
  }
  // key tiles of each row tile: up to its last valid token
  int nt[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = q0 + t * a.tpt;
    nt[t] = first < it.len ? (min(first + a.tpt, it.len) + 127) >> 7 : 0;
  }
  const int nmax = max(nt[0], nt[1]);

  if (threadIdx.x == 0) {
    mbar_init(bar(B_Q), 1);
    for (int s = 0; s < NR; ++s) {
      mbar_init(bar(B_F + s), 1);
      mbar_init(bar(B_E + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(B_S + t), 1);
      mbar_init(bar(B_P + t), 4);
      mbar_init(bar(B_P2 + t), 4);
      mbar_init(bar(B_PV + t), 1);
    }
    mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tslot), 512);
    tmem_relinquish();
  }
  if (BIAS) dense_bias_fill<false>(a, sB, g, min(q0 + tpc, it.len) - 1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(tslot);
  // TMEM: S/P of tile t at columns [128 t, 128 t + 128), O of tile t at 256 + D t

  if (warp >= 8) {
    setmaxnreg_dec<kRegsCtl>();
    if (warp == 8) {
      // ------------------------------ loads --------------------------------------
      if (lane == 0) {
        const uint32_t rows = (uint32_t)a.tpt * a.G * 128;  // bytes of one 64-column box
        mbar_arrive_expect_tx(bar(B_Q), (nt[1] ? 2 : 1) * NCH * rows);
        for (int t = 0; t < (nt[1] ? 2 : 1); ++t)
          for (int c = 0; c < NCH; ++c)
            tma_load_3d(smem_u32(sQ + t * C::kTile + c * 16384), &tm_q, bar(B_Q), 64 * c, g * a.G,
                        it.start + q0 + t * a.tpt);
        int x = 0;  // ring position: K0, V0, K1, V1, ...
        for (; x < 2 * nmax; ++x) {
          const int s = x % NR;
          if (x >= NR && !wait_bar(bar(B_E + s), ((x / NR) & 1) ^ 1, abort_flag, a.status,
                                   wait_site(kKerDenseFwd, B_E + s, x >> 1)))
            break;
          mbar_arrive_expect_tx(bar(B_F + s), C::kTile);
          const uint32_t dst = smem_u32(sKV + s * C::kTile);
          const int tok = it.start + (x >> 1) * 128;
          for (int c = 0; c < NCH; ++c)
            tma_load_3d(dst + c * 16384, (x & 1) ? &tm_v : &tm_k, bar(B_F + s), 64 * c, g, tok);
        }
        // an aborted CTA must not leave before its copies have landed
        if (*abort_flag) {
          drain_bar(bar(B_Q), 0);
          for (int y = max(0, x - NR); y < x; ++y) drain_bar(bar(B_F + y % NR), (y / NR) & 1);
        }
      }
    } else if (warp == 9) {
      // ------------------------------ MMA issue ----------------------------------
      constexpr uint32_t idS = make_idesc_bf16(128, 128, false, false);
      constexpr uint32_t idO = make_idesc_bf16(128, D, false, true);
      const uint32_t el = elect_one(), tm = uniform(tbase);
      const int len = uniform(it.len), nt0 = uniform(nt[0]), nt1 = uniform(nt[1]);
      const int nm = max(nt0, nt1);
      const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), k_lo = desc_lo(smem_u32(sKV), 16),
                     v_lo = desc_lo(smem_u32(sKV), 16384);
      auto wait = [&](int b, uint32_t par, int n) {
        return wait_bar_warp(bar(b), par, abort_flag, a.status, wait_site(kKerDenseFwd, b, n));
      };
      auto wait_full = [&](int x) { return wait(B_F + x % NR, (x / NR) & 1, x >> 1); };
      auto issue_s = [&](int t, int n) {
        mma_tile_ss<D>(el, tm + 128 * t, q_lo + t * (C::kTile >> 4),
                       k_lo + (2 * n % NR) * (C::kTile >> 4), idS);
        mma_commit(el, bar(B_S + t));
      };
      bool ok = wait(B_Q, 0, 0) && wait_full(0);
      if (ok) {
        tc_fence_after();
        if (nt0 > 0) issue_s(0, 0);
        if (nt1 > 0) issue_s(1, 0);
        mma_commit(el, bar(B_E + 0));
      }
      for (int n = 0; ok && n < nm; ++n) {
        const int xv = 2 * n + 1, sv = xv % NR;
        if (!(ok = wait_full(xv))) break;
        // keys behind the document's end: P is zero there, V must be finite
        if ((n + 1) * 128 > len) dense_zero_rows<D>(sKV + sv * C::kTile, len - n * 128);
        const uint32_t v = v_lo + sv * (C::kTile >> 4);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int ntt = t ? nt1 : nt0;
          if (!ok || n >= ntt) continue;
          const uint32_t po = tm + 256 + D * t, pa = tm + 128 * t;
          if (!(ok = wait(B_P + t, n & 1, n))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(el, po, pa + 8 * kk, v + kk * (2048 >> 4), idO, n > 0 || kk > 0);
          if (!(ok = wait(B_P2 + t, n & 1, n))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 4; kk < 8; ++kk)
            mma_ts(el, po, pa + 8 * kk, v + kk * (2048 >> 4), idO, 1);
          mma_commit(el, bar(B_PV + t));
          if (n + 1 < ntt) {
            if (!(ok = wait_full(xv + 1))) break;
            tc_fence_after();
            issue_s(t, n + 1);
          }
        }
        if (!ok) break;
        mma_commit(el, bar(B_E + sv));
        if (n + 1 < nm) mma_commit(el, bar(B_E + (xv + 1) % NR));
      }
      if (!ok) {  // products in flight end before TMEM is freed
        mma_commit(el, bar(B_END));
        drain_bar(bar(B_END), 0);
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------ softmax ---------------------------------------
    // A failed wait marks the warp dead: it keeps arriving on its barriers
    // without touching TMEM.
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lane_off + 128 * t, to = tbase + lane_off + 256 + D * t;
    const int ti = r / a.G, hl = r % a.G;  // hl < G also for rows behind tpt
    const int qi = q0 + t * a.tpt + ti;  // token inside the document
    const bool valid = ti < a.tpt && qi < it.len;
    const float c = a.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool dead = false;
    int bk = a.nb - 1;
    const uint16_t* tab = a.bias + (size_t)(g * a.G + hl) * a.nb;
    for (int n = 0; n < nt[t]; ++n) {
      const int rel = qi - n * 128;  // keys 0..rel of the tile are visible
      bool one = true, near = false;  // see DenseBias
      float v0 = 0.f;
      if (BIAS) {
        bk = dense_bucket(sB, bk, rel);
        one = __all_sync(0xffffffffu, bk == 0 || sB->starts[bk] <= rel - 127);
        near = __all_sync(0xffffffffu, rel < a.lut_w);
        v0 = dense_bias_log2(__ldg(tab + bk));
      }
      dead = dead || !wait_bar_warp(bar(B_S + t), n & 1, abort_flag, a.status,
                                    wait_site(kKerDenseFwd, B_S + t, n));
      tc_fence_after();
      if (!dead) {
        uint32_t x[128];
        tmem_ld128(ts, x);
        if (__any_sync(0xffffffffu, rel < 127)) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i > rel) x[i] = __float_as_uint(-INFINITY);
        }
        // P = 2^(x mul + add - m)
        float mul = c, add = 0.f;
        if (BIAS) {
          if (one) {
            add = v0;  // one bucket over the row's part of the tile
          } else {
            mul = 1.f;
            if (near) {
              const float* lut = sB->lut + hl * a.lut_stride + dense_lut_pad(a) + rel;
#pragma unroll
              for (int i = 0; i < 128; ++i)
                x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, lut[-i]));
            } else if (__all_sync(0xffffffffu, bk < 2 || sB->starts[bk - 1] <= rel - 127)) {
              // at most one start inside: scores before `cut` take v0, the others v1
              const int cut = bk > 0 ? rel - sB->starts[bk] + 1 : 128;
              const float v1 = dense_bias_log2(__ldg(tab + max(bk - 1, 0)));
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                if (__any_sync(0xffffffffu, cut > 16 * u && cut < 16 * u + 16)) {
#pragma unroll
                  for (int i = 16 * u; i < 16 * u + 16; ++i)
                    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, i < cut ? v0 : v1));
                } else {
                  const float bv = 16 * u < cut ? v0 : v1;
#pragma unroll
                  for (int i = 16 * u; i < 16 * u + 16; ++i)
                    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, bv));
                }
              }
            } else {
              int b = bk;
              int st = b > 0 ? sB->starts[b] : INT_MIN;
              float bv = v0;
#pragma unroll
              for (int i = 0; i < 128; ++i) {
                if (rel - i < st) {
                  --b;
                  st = b > 0 ? sB->starts[b] : INT_MIN;
                  bv = dense_bias_log2(__ldg(tab + b));
                }
                x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, bv));
              }
            }
            __syncwarp();
          }
        }
        float m4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          m4[u] = __uint_as_float(x[32 * u]);
#pragma unroll
          for (int i = 1; i < 31; i += 2)
            m4[u] = fmax3(m4[u], __uint_as_float(x[32 * u + i]), __uint_as_float(x[32 * u + i + 1]));
          m4[u] = fmaxf(m4[u], __uint_as_float(x[32 * u + 31]));
        }
        const float mx = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), mul, add);
        const bool grow = mx > m + kRescale || (m == -INFINITY && mx > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? mx : m;
          const float f = m_new == m ? 1.f : ex2_approx(m - m_new);
          l *= f;
          m = m_new;
          if (n > 0) {
            // O is complete up to tile n - 1 once its P V product has been read
            dead = dead || !wait_bar_warp(bar(B_PV + t), (n - 1) & 1, abort_flag, a.status,
                                          wait_site(kKerDenseFwd, B_PV + t, n));
            tc_fence_after();
            if (!dead) {
#pragma unroll 1
              for (int u = 0; u < D / 32; ++u) {
                uint32_t y[32];
                tmem_ld32(to + 32 * u, y);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                tmem_st32(to + 32 * u, y);
              }
            }
          }
        }
        const float sub = add - (m == -INFINITY ? 0.f : m);
        const f32x2 mul2_ = pack2(mul, mul), sub2 = pack2(sub, sub);
        f32x2 ls[2] = {0ull, 0ull};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int e = 64 * u + 2 * i;
            float p0, p1;
            unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), mul2_, sub2), p0,
                    p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            ls[i & 1] = add2(ls[i & 1], pack2(p0, p1));
            w[i] = pack_bf16(p0, p1);
          }
          tmem_st32_async(ts + 32 * u, w);
          tmem_wait_st();
          // the product over the first 64 keys starts while the rest is computed
          if (u == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + t));
          }
        }
        float l0, l1;
        unpack2(add2(ls[0], ls[1]), l0, l1);
        l += l0 + l1;
      } else if (lane == 0) {
        mbar_arrive(bar(B_P + t));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_P2 + t));
    }
    if (nt[t] > 0) {
      const int last = nt[t] - 1;
      dead = dead || !wait_bar_warp(bar(B_PV + t), last & 1, abort_flag, a.status,
                                    wait_site(kKerDenseFwd, B_PV + t, last));
      tc_fence_after();
      if (!dead) {
        const size_t row = (size_t)(it.start + qi) * a.hq + g * a.G + hl;
        const float inv = l > 0.f ? 1.f / l : 0.f;  // 0: no key left (bias -inf)
        uint8_t* stg = sQ + t * C::kTile + (warp & 3) * 4096;
#pragma unroll 1
        for (int u = 0; u < D / 64; ++u) {
          uint32_t va[32], vb[32];
          tmem_ld32x2(to + 64 * u, to + 64 * u + 32, va, vb);
          if (BIAS && l == 0.f) {
#pragma unroll
            for (int i = 0; i < 32; ++i) va[i] = vb[i] = 0;
          }
          dense_store_rows(va, vb, inv, stg, valid ? a.o + row * D + 64 * u : nullptr);
          if (a.o_res)
            dense_store_rows<true>(va, vb, inv, stg,
                                   valid ? a.o_res + row * D + 64 * u : nullptr);
        }
        if (valid && a.lse) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    tc_fence_before();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool BIAS>
cudaError_t launch_t(const DenseArgs& a, const CUtensorMap& mq, const CUtensorMap& mk,
                     const CUtensorMap& mv, cudaStream_t st) {
  constexpr int kBudget = 2 * 128 * kRegsSoftmax + 128 * kRegsCtl;
  static_assert(kBudget <= 65536, "register budgets exceed the register file");
  cudaError_t e = dense_prepare<k_dense_fwd<D, BIAS>>(kThreads, kBudget, FwdCfg<D, BIAS>::kSmem);
  if (e != cudaSuccess) return e;
  k_dense_fwd<D, BIAS><<<(unsigned)a.nslots * a.hkv, kThreads, FwdCfg<D, BIAS>::kSmem, st>>>(mq, mk, mv,
                                                                                       a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_fwd(const DenseShape& s, const uint16_t* q, const uint16_t* k,
                             const uint16_t* v, const DenseArgs& args, cudaStream_t st) {
  DenseArgs a = args;
  a.nslots = dense_slots(a.T, a.ndoc, 2 * a.tpt);
  CUtensorMap mq, mk, mv;
  cudaError_t e;
  if ((e = make_tmap_rows(&mq, q, s.d, a.hq, a.T, s.q_stride, a.G, a.tpt)) != cudaSuccess) return e;
  if ((e = make_tmap_rows(&mk, k, s.d, a.hkv, a.T, s.k_stride, 1, 128)) != cudaSuccess) return e;
  if ((e = make_tmap_rows(&mv, v, s.d, a.hkv, a.T, s.v_stride, 1, 128)) != cudaSuccess) return e;
  if (s.d == 128)
    return a.bias ? launch_t<128, true>(a, mq, mk, mv, st) : launch_t<128, false>(a, mq, mk, mv, st);
  return a.bias ? launch_t<64, true>(a, mq, mk, mv, st) : launch_t<64, false>(a, mq, mk, mv, st);
}

}  // namespace msa
