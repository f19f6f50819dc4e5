// Dense causal attention backward: dQ (and the bias table's gradient), then dK
// and dV.  With S, P as in the forward, dP = dO V^T, D = rowsum(dO o O):
//   dS = P (dP - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
//   dtable[h][b] = sum of dS over the pairs of head h whose distance is in b.
// Two kernels, each owning its outputs: one CTA per 128 packed (token, head)
// rows sums dQ over the keys, one CTA per 128 keys of a KV head sums dK and dV
// over its group's queries.  S and dP are computed in both (7 products per
// tile pair instead of 5); in exchange there are no fp32 partial gradients in
// HBM and no atomics, and every sum has a fixed order.
#include "dense_common.cuh"

namespace msa {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsSoftmax = 200, kRegsCtl = 104;
constexpr int kBudget = 2 * 128 * kRegsSoftmax + 128 * kRegsCtl;
static_assert(kBudget <= 65536, "register budgets exceed the register file");

// D columns of TMEM lane `row` (fp32, times f) to bf16 row `dst` (null: none).
template <int D>
__device__ __forceinline__ void store_tmem_rows(uint32_t taddr, float f, uint8_t* stg,
                                                uint16_t* dst) {
#pragma unroll 1
  for (int u = 0; u < D / 64; ++u) {
    uint32_t va[32], vb[32];
    tmem_ld32x2(taddr + 64 * u, taddr + 64 * u + 32, va, vb);
    dense_store_rows(va, vb, f, stg, dst ? dst + 64 * u : nullptr);
  }
}

// ---------------------------------------------------------------------------
// dQ: 128 packed rows against their keys, tile by tile.
// Warps 0-3 and 4-7 take 64 of a tile's 128 columns each (a row is one TMEM
// lane of both); warp 8 loads, warp 9 issues the MMAs.  S has two TMEM buffers:
// while the softmax warps turn S(n), dP(n) into dS(n) (bf16, over S(n)'s
// columns), S(n + 1) is computed, and dP(n + 1) as soon as dP(n) has been read.
// ---------------------------------------------------------------------------
template <int D, bool BIAS>
struct DqCfg {
  static constexpr int kTile = 128 * D * 2;
  // K and V rings; with a bias its tables take the place of a tile
  static constexpr int kNK = D == 128 ? 3 : 5, kNV = D == 128 ? (BIAS ? 1 : 2) : 4;
  static constexpr int kSmem =
      (2 + kNK + kNV) * kTile + 256 + 512 + (BIAS ? (int)sizeof(DenseBias) : 0);
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int D, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    k_dense_dq(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ DenseArgs a) {
  using C = DqCfg<D, BIAS>;
  constexpr int NCH = D / 64, NK = C::kNK, NV = C::kNV;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;  // after the last S also the staging of dQ
  uint8_t* sO = sQ + C::kTile;
  uint8_t* sK = sO + C::kTile;
  uint8_t* sV = sK + NK * C::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NV * C::kTile);
  constexpr int B_Q = 0, B_KF = 1, B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + NV,
                B_S = B_VE + NV, B_DP = B_S + 2, B_DPE = B_DP + 1, B_DS = B_DPE + 1,
                B_DQ = B_DS + 2, B_END = B_DQ + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + B_END + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((B_END + 1) * 8 + 8 <= 256, "barrier block");
  float* sD = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 256);  // [128] D
  DenseBias* sB = reinterpret_cast<DenseBias*>(sD + 128);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (blockIdx.x == 0 && warp == 11) dense_check_docs(a);
  const int g = blockIdx.x % a.hkv;
  const int slot = (int)(blockIdx.x / a.hkv);
  DenseItem it;
  const bool have = dense_item<false>(a, slot, a.tpt, it);
  float* part = BIAS ? a.parts + ((size_t)slot * a.hq + g * a.G) * a.nb : nullptr;
  if (!have || it.doc == a.ndoc) {
    if (BIAS)
      for (int x = threadIdx.x; x < a.G * a.nb; x += kThreads) part[x] = 0.f;
    if (have) {
      const int n = min(a.tpt, it.len - it.tile * a.tpt) * a.G;
      for (int r = threadIdx.x; r < n; r += kThreads)
        dense_zero_row(a.dq + ((size_t)(it.start + it.tile * a.tpt + r / a.G) * a.hq + g * a.G +
                               r % a.G) * D, D);
    }
    return;
  }
  const int q0 = it.tile * a.tpt;
  const int N = (min(q0 + a.tpt, it.len) + 127) >> 7;  // key tiles

  // D = rowsum(dO o O), O = o + o_res, of 16 rows per warp of the first eight: D/8 lanes to
  // a row, 16 bytes each.  Loaded here, so that the loads run under the set-up.
  constexpr int kLanes = D / 8, kSteps = 16 * kLanes / 32;
  const int dr0 = (warp & 3) * 32 + 16 * (warp >> 2);
  uint4 xo[kSteps], xr[kSteps], xd[kSteps];
  if (warp < 8) {
    const int rows = min(a.tpt, it.len - q0);  // tokens of the item
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      // rows behind the last one read an earlier row, so that no load is conditional
      const int rr = dr0 + u * (32 / kLanes) + lane / kLanes, tok = min(rr / a.G, rows - 1);
      const int hh = g * a.G + rr % a.G;
      const size_t t = (size_t)(it.start + q0 + tok);
      const size_t at = (t * a.hq + hh) * D + lane % kLanes * 8;
      xo[u] = ld_nc_v4(a.o + at);
      xr[u] = ld_nc_v4(a.o_res + at);
      xd[u] = ld_nc_v4(a.d_o + t * a.do_stride + (size_t)hh * D + lane % kLanes * 8);
    }
  }

  if (threadIdx.x == 0) {
    mbar_init(bar(B_Q), 1);
    for (int s = 0; s < NK; ++s) mbar_init(bar(B_KF + s), 1), mbar_init(bar(B_KE + s), 1);
    for (int s = 0; s < NV; ++s) mbar_init(bar(B_VF + s), 1), mbar_init(bar(B_VE + s), 1);
    mbar_init(bar(B_S), 1);
    mbar_init(bar(B_S + 1), 1);
    mbar_init(bar(B_DP), 1);
    mbar_init(bar(B_DPE), 8);
    mbar_init(bar(B_DS), 8);
    mbar_init(bar(B_DS + 1), 8);
    mbar_init(bar(B_DQ), 1);
    mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tslot), 512);
    tmem_relinquish();
  }
  if (BIAS && warp >= 10) dense_bias_starts<true>(a, sB, g);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(tslot);
  // TMEM: S/dS buffer b at columns [128 b, 128 b + 128), dP at 256, dQ at 384.  dS of the
  // columns of warpgroup w starts at column 64 w of its buffer.

  if (warp >= 8) {
    setmaxnreg_dec<kRegsCtl>();
    if (warp == 8) {
      // ------------------------------ loads --------------------------------------
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(B_Q), 2 * NCH * (uint32_t)a.tpt * a.G * 128);
        for (int c = 0; c < NCH; ++c) {
          tma_load_3d(smem_u32(sQ + c * 16384), &tm_q, bar(B_Q), 64 * c, g * a.G, it.start + q0);
          tma_load_3d(smem_u32(sO + c * 16384), &tm_do, bar(B_Q), 64 * c, g * a.G, it.start + q0);
        }
        int nk = 0, nv = 0;  // tiles whose loads were issued
        for (int n = 0; n < N; ++n) {
          const int sk = n % NK, sv = n % NV, tok = it.start + n * 128;
          if (n >= NK && !wait_bar(bar(B_KE + sk), ((n / NK) & 1) ^ 1, abort_flag, a.status,
                                   wait_site(kKerDenseDq, B_KE + sk, n)))
            break;
          mbar_arrive_expect_tx(bar(B_KF + sk), C::kTile);
          for (int c = 0; c < NCH; ++c)
            tma_load_3d(smem_u32(sK + sk * C::kTile + c * 16384), &tm_k, bar(B_KF + sk), 64 * c, g,
                        tok);
          nk = n + 1;
          if (n >= NV && !wait_bar(bar(B_VE + sv), ((n / NV) & 1) ^ 1, abort_flag, a.status,
                                   wait_site(kKerDenseDq, B_VE + sv, n)))
            break;
          mbar_arrive_expect_tx(bar(B_VF + sv), C::kTile);
          for (int c = 0; c < NCH; ++c)
            tma_load_3d(smem_u32(sV + sv * C::kTile + c * 16384), &tm_v, bar(B_VF + sv), 64 * c, g,
                        tok);
          nv = n + 1;
        }
        if (*abort_flag) {  // copies in flight land before the CTA leaves
          drain_bar(bar(B_Q), 0);
          for (int y = max(0, nk - NK); y < nk; ++y) drain_bar(bar(B_KF + y % NK), (y / NK) & 1);
          for (int y = max(0, nv - NV); y < nv; ++y) drain_bar(bar(B_VF + y % NV), (y / NV) & 1);
        }
      }
    } else if (warp == 9) {
      // ------------------------------ MMA issue ----------------------------------
      constexpr uint32_t idS = make_idesc_bf16(128, 128, false, false);
      constexpr uint32_t idQ = make_idesc_bf16(128, D, false, true);
      const uint32_t el = elect_one(), tm = uniform(tbase);
      const int len = uniform(it.len), NT = uniform(N);
      constexpr uint32_t T16 = C::kTile >> 4;
      const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), o_lo = desc_lo(smem_u32(sO), 16),
                     k_lo = desc_lo(smem_u32(sK), 16), v_lo = desc_lo(smem_u32(sV), 16),
                     kt_lo = desc_lo(smem_u32(sK), 16384);
      auto wait = [&](int b, uint32_t par, int n) {
        return wait_bar_warp(bar(b), par, abort_flag, a.status, wait_site(kKerDenseDq, b, n));
      };
      auto s_of = [&](int n) -> bool {
        if (!wait(B_KF + n % NK, (n / NK) & 1, n)) return false;
        // keys behind the document's end: dS is zero there, K must be finite
        if ((n + 1) * 128 > len) dense_zero_rows<D>(sK + (n % NK) * C::kTile, len - n * 128);
        tc_fence_after();
        mma_tile_ss<D>(el, tm + 128 * (n & 1), q_lo, k_lo + (n % NK) * T16, idS);
        mma_commit(el, bar(B_S + (n & 1)));
        return true;
      };
      auto dp_of = [&](int n) -> bool {
        if (!wait(B_VF + n % NV, (n / NV) & 1, n)) return false;
        if (n > 0 && !wait(B_DPE, (n - 1) & 1, n)) return false;
        tc_fence_after();
        mma_tile_ss<D>(el, tm + 256, o_lo, v_lo + (n % NV) * T16, idS);
        mma_commit(el, bar(B_DP));
        mma_commit(el, bar(B_VE + n % NV));
        return true;
      };
      bool ok = wait(B_Q, 0, 0) && s_of(0) && dp_of(0);
      for (int n = 0; ok && n < NT; ++n) {
        if (n + 1 < NT && !(ok = s_of(n + 1) && dp_of(n + 1))) break;
        if (!(ok = wait(B_DS + (n & 1), (n >> 1) & 1, n))) break;
        tc_fence_after();
        const uint32_t k = kt_lo + (n % NK) * T16, ds = tm + 128 * (n & 1);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(el, tm + 384, ds + 64 * (kk >> 2) + 8 * (kk & 3), k + kk * (2048 >> 4), idQ,
                 n > 0 || kk > 0);
        mma_commit(el, bar(B_KE + n % NK));
      }
      mma_commit(el, bar(B_DQ));
      if (!ok) {  // products in flight end before TMEM is freed
        mma_commit(el, bar(B_END));
        drain_bar(bar(B_END), 0);
      }
    } else if (BIAS && warp == 11) {
      // ------------------------------ bucket sums: clear --------------------------
      float4* all = reinterpret_cast<float4*>(a.slots + ((size_t)slot * a.hkv + g) * a.nb * 256);
      for (int x = lane; x < a.nb * 64; x += 32) all[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      __threadfence_block();
      named_bar_sync(1, 288);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    if (BIAS) {
      dense_bias_fill<true>(a, sB, g, min(q0 + a.tpt, it.len) - 1);
      named_bar_sync(2, 256);
    }
    // ------------------------------ dS ---------------------------------------------
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tl = tbase + lane_off;
    const int ti = r / a.G, hl = r % a.G;
    const int qi = q0 + ti;
    const bool valid = ti < a.tpt && qi < it.len;
    const size_t row = (size_t)(it.start + qi) * a.hq + g * a.G + hl;
    // D of 16 rows per warp
    {
      float s[kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        auto dot = [](uint32_t o, uint32_t res, uint32_t d_o) {
          return (bf16_lo(o) + bf16_lo(res)) * bf16_lo(d_o) +
                 (bf16_hi(o) + bf16_hi(res)) * bf16_hi(d_o);
        };
        s[u] = (dot(xo[u].x, xr[u].x, xd[u].x) + dot(xo[u].y, xr[u].y, xd[u].y)) +
               (dot(xo[u].z, xr[u].z, xd[u].z) + dot(xo[u].w, xr[u].w, xd[u].w));
      }
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
        if (lane % kLanes == 0) sD[dr0 + u * (32 / kLanes) + lane / kLanes] = s[u];
      }
      named_bar_sync(1, BIAS ? 288 : 256);  // with a bias warp 11 too: its sums are cleared
    }
    // -lse and D of the row (both warpgroups; the first also leaves them for dK, dV)
    float nl = -INFINITY, dsum = 0.f;
    if (valid) {
      dsum = sD[r];
      const float lse = __ldg(a.lse + row);
      nl = lse == -INFINITY ? -INFINITY : -lse * kLog2E;
      if (w == 0)
        a.stats[(size_t)(g * a.G + hl) * a.T + it.start + qi] = make_float2(nl, dsum);
    }
    // this row's bucket sums: a row meets the distances in falling order, so a
    // bucket is finished when the next one begins and is stored once
    float* my = nullptr;
    if (BIAS) {
      my = a.slots + ((size_t)slot * a.hkv + g) * a.nb * 256 + w * 128 + r;
    }
    float acc = 0.f;
    int bk = a.nb - 1, stk = INT_MAX;  // bucket of the next scores and its first distance
    float bias0 = 0.f;                 // its bias
    const uint16_t* tab = a.bias + (size_t)(g * a.G + hl) * a.nb;
    bool dead = false;
    for (int n = 0; n < N; ++n) {
      const int b = n & 1;
      const int rel = valid ? qi - n * 128 - 64 * w : -1;  // columns 0..rel are visible
      const bool edge = __any_sync(0xffffffffu, rel < 63);
      auto wait = [&](int bb, uint32_t par) {
        dead = dead || !wait_bar_warp(bar(bb), par, abort_flag, a.status,
                                      wait_site(kKerDenseDq, bb, n));
        tc_fence_after();
      };
      bool one = true, near = false;  // see DenseBias
      if (BIAS) {
        if (__any_sync(0xffffffffu, rel < stk)) {  // the row's first bucket here is another
          const int first = dense_bucket(sB, rel);
          if (first != bk) {
            my[bk * 256] = acc;
            acc = 0.f;
            bk = first;
          }
          stk = bk > 0 ? sB->starts[bk] : INT_MIN;
          bias0 = dense_bias_log2(__ldg(tab + bk));
        }
        one = __all_sync(0xffffffffu, bk == 0 || stk <= rel - 63);
        near = __all_sync(0xffffffffu, rel < a.lut_w);
      }
      uint32_t x[2][32];
      wait(B_S + b, (n >> 1) & 1);
      if (!dead) {
        tmem_ld32x2(tl + 128 * b + 64 * w, tl + 128 * b + 64 * w + 32, x[0], x[1]);
        // P = 2^(S scale log2(e) + bias - lse)
        if (one) {
          const float sub = nl + bias0;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            x[i >> 5][i & 31] = __float_as_uint(
                ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), a.scale_log2, sub)));
        } else {
          if (near) {
            const float* lut = sB->lut + hl * a.lut_stride + dense_lut_pad(a) + rel;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              x[i >> 5][i & 31] = __float_as_uint(ex2_approx(
                  fmaf(__uint_as_float(x[i >> 5][i & 31]), a.scale_log2, nl + lut[-i])));
          } else if (__all_sync(0xffffffffu, bk < 2 || sB->starts[bk - 1] <= rel - 63)) {
            // at most one start inside: scores before `cut` take v0, the others v1
            const int cut = bk > 0 ? rel - sB->starts[bk] + 1 : 64;
            const float v0 = nl + bias0;
            const float v1 = nl + dense_bias_log2(__ldg(tab + max(bk - 1, 0)));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (__any_sync(0xffffffffu, cut > 16 * u && cut < 16 * u + 16)) {
#pragma unroll
                for (int i = 16 * u; i < 16 * u + 16; ++i)
                  x[i >> 5][i & 31] = __float_as_uint(ex2_approx(fmaf(
                      __uint_as_float(x[i >> 5][i & 31]), a.scale_log2, i < cut ? v0 : v1)));
              } else {
                const float sub = 16 * u < cut ? v0 : v1;
#pragma unroll
                for (int i = 16 * u; i < 16 * u + 16; ++i)
                  x[i >> 5][i & 31] = __float_as_uint(
                      ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), a.scale_log2, sub)));
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
                sub = nl + dense_bias_log2(__ldg(tab + q));
              }
              x[i >> 5][i & 31] = __float_as_uint(
                  ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), a.scale_log2, sub)));
            }
          }
          __syncwarp();
        }
        wait(B_DP, n & 1);
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
              bk -= __popc(last[0]) + __popc(last[1]);
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
    if (BIAS) {
      if (valid) my[bk * 256] = acc;
      // sums over the item's rows, in a fixed order: a warp takes every eighth bucket, brings
      // its row sums (contiguous) and adds them up head by head, through shared memory where G
      // is no power of two.  The barrier orders the stores above before the loads, and the last
      // use of the bias tables before their memory is reused.
      __threadfence_block();
      named_bar_sync(2, 256);
      const float* all = a.slots + ((size_t)slot * a.hkv + g) * a.nb * 256 + lane;
      float* scr = sB->lut + warp * 128;
      float v[kDenseMaxBuckets / 8][4];
#pragma unroll
      for (int u = 0; u < kDenseMaxBuckets / 8; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* p = all + (warp + 8 * u) * 256 + 32 * i;
          v[u][i] = warp + 8 * u < a.nb ? __ldcg(p) + __ldcg(p + 128) : 0.f;
        }
#pragma unroll
      for (int u = 0; u < kDenseMaxBuckets / 8; ++u) {
        const int b = warp + 8 * u;
        if (b >= a.nb) break;
        if (a.G <= 32 && (a.G & (a.G - 1)) == 0) {  // rows 32 apart belong to one head
          float sum = (v[u][0] + v[u][1]) + (v[u][2] + v[u][3]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            if (o >= a.G) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane < a.G) part[lane * a.nb + b] = sum;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) scr[32 * i + lane] = v[u][i];
          __syncwarp();
          for (int h = lane; h < a.G; h += 32) {
            float sum[2] = {0.f, 0.f};
#pragma unroll 8
            for (int i = 0; i < a.tpt; ++i) sum[i & 1] += scr[i * a.G + h];
            part[h * a.nb + b] = sum[0] + sum[1];
          }
          __syncwarp();
        }
      }
    }
    if (w == 0) {
      dead = dead || !wait_bar_warp(bar(B_DQ), 0, abort_flag, a.status,
                                    wait_site(kKerDenseDq, B_DQ, N));
      tc_fence_after();
      if (!dead)
        store_tmem_rows<D>(tl + 384, a.scale, sQ + warp * 4096,
                           valid ? a.dq + row * D : nullptr);
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
// dK, dV: 128 keys of a KV head against the queries of its group, head by head,
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
  static constexpr int kNQ = D == 128 ? (BIAS ? 2 : 3) : 4, kNO = D == 128 ? 2 : 4;  // Q and dO rings
  static constexpr int kNS = 2;                                           // statistics ring
  static constexpr int kSmem =
      (2 + kNQ + kNO) * kTile + kNS * 1024 + 256 + (BIAS ? (int)sizeof(DenseBias) : 0);
  static_assert(kSmem <= 232448, "shared memory budget");
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
  uint8_t* sQ = sV + C::kTile;  // the rings are also the staging of dK and dV
  uint8_t* sO = sQ + NQ * C::kTile;
  float2* sSt = reinterpret_cast<float2*>(sO + NO * C::kTile);  // [NS][128] {-lse log2(e), D}
  uint64_t* bars = reinterpret_cast<uint64_t*>(sSt + NS * 128);
  constexpr int B_KV = 0, B_QF = 1, B_QE = B_QF + NQ, B_OF = B_QE + NQ, B_OE = B_OF + NO,
                B_TF = B_OE + NO, B_TE = B_TF + NS, B_S = B_TE + NS, B_P = B_S + 1, B_DP = B_P + 1,
                B_DS = B_DP + 1, B_END = B_DS + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + B_END + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((B_END + 1) * 8 + 8 <= 256, "barrier block");
  DenseBias* sB = reinterpret_cast<DenseBias*>(reinterpret_cast<uint8_t*>(bars) + 256);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  const int g = blockIdx.x % a.hkv;
  DenseItem it;
  if (!dense_item<true>(a, (int)(blockIdx.x / a.hkv), 128, it)) return;  // a tile of keys
  const int j0 = it.tile * 128;
  if (it.doc == a.ndoc) {
    const int n = min(128, it.len - j0);
    for (int r = threadIdx.x; r < n; r += kThreads) {
      const size_t row = (size_t)(it.start + j0 + r) * a.hkv + g;
      dense_zero_row(a.dk + row * D, D);
      dense_zero_row(a.dv + row * D, D);
    }
    return;
  }
  const int nq = (it.len - j0 + 127) >> 7;  // query tiles of a head
  const int N = nq * a.G;

  if (threadIdx.x == 0) {
    mbar_init(bar(B_KV), 1);
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
  if (BIAS && warp >= 10) dense_bias_starts<false>(a, sB, g);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(tslot);
  // TMEM: S^T/P^T at column 0, dP^T/dS^T at 128, dV at 256, dK at 384.  P^T and dS^T of the
  // queries of warpgroup w start at column 64 w of theirs.

  if (warp >= 8) {
    setmaxnreg_dec<kRegsCtl>();
    if (warp == 8) {
      // ------------------------------ loads --------------------------------------
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(B_KV), 2 * C::kTile);
        for (int c = 0; c < NCH; ++c) {
          tma_load_3d(smem_u32(sK + c * 16384), &tm_k, bar(B_KV), 64 * c, g, it.start + j0);
          tma_load_3d(smem_u32(sV + c * 16384), &tm_v, bar(B_KV), 64 * c, g, it.start + j0);
        }
        int lq = 0, lo = 0;  // tiles whose loads were issued
        int h = g * a.G, qt = 0;
        for (int n = 0; n < N; ++n) {
          const int sq = n % NQ, so = n % NO, tok = it.start + j0 + qt * 128;
          if (n >= NQ && !wait_bar(bar(B_QE + sq), ((n / NQ) & 1) ^ 1, abort_flag, a.status,
                                   wait_site(kKerDenseDkv, B_QE + sq, n)))
            break;
          mbar_arrive_expect_tx(bar(B_QF + sq), C::kTile);
          for (int c = 0; c < NCH; ++c)
            tma_load_3d(smem_u32(sQ + sq * C::kTile + c * 16384), &tm_q, bar(B_QF + sq), 64 * c, h,
                        tok);
          lq = n + 1;
          if (n >= NO && !wait_bar(bar(B_OE + so), ((n / NO) & 1) ^ 1, abort_flag, a.status,
                                   wait_site(kKerDenseDkv, B_OE + so, n)))
            break;
          mbar_arrive_expect_tx(bar(B_OF + so), C::kTile);
          for (int c = 0; c < NCH; ++c)
            tma_load_3d(smem_u32(sO + so * C::kTile + c * 16384), &tm_do, bar(B_OF + so), 64 * c, h,
                        tok);
          lo = n + 1;
          if (++qt == nq) qt = 0, ++h;
        }
        if (*abort_flag) {  // copies in flight land before the CTA leaves
          drain_bar(bar(B_KV), 0);
          for (int y = max(0, lq - NQ); y < lq; ++y) drain_bar(bar(B_QF + y % NQ), (y / NQ) & 1);
          for (int y = max(0, lo - NO); y < lo; ++y) drain_bar(bar(B_OF + y % NO), (y / NO) & 1);
        }
      }
    } else if (warp == 9) {
      // ------------------------------ MMA issue ----------------------------------
      constexpr uint32_t idS = make_idesc_bf16(128, 128, false, false);
      constexpr uint32_t idG = make_idesc_bf16(128, D, false, true);
      const uint32_t el = elect_one(), tm = uniform(tbase);
      const int left = uniform(it.len - j0), nqt = uniform(nq), NT = uniform(N);
      constexpr uint32_t T16 = C::kTile >> 4;
      const uint32_t k_lo = desc_lo(smem_u32(sK), 16), v_lo = desc_lo(smem_u32(sV), 16),
                     q_lo = desc_lo(smem_u32(sQ), 16), o_lo = desc_lo(smem_u32(sO), 16),
                     qt_lo = desc_lo(smem_u32(sQ), 16384), ot_lo = desc_lo(smem_u32(sO), 16384);
      auto wait = [&](int b, uint32_t par, int n) {
        return wait_bar_warp(bar(b), par, abort_flag, a.status, wait_site(kKerDenseDkv, b, n));
      };
      // waits for tile n of a ring; queries behind the document's end are zeroed: their
      // probabilities are zero, but the products sum over them
      auto arrived = [&](int bf, int depth, uint8_t* ring, int n) -> bool {
        if (!wait(bf + n % depth, (n / depth) & 1, n)) return false;
        const int i0 = (n % nqt) * 128;
        if (i0 + 128 > left) dense_zero_rows<D>(ring + (n % depth) * C::kTile, left - i0);
        tc_fence_after();
        return true;
      };
      auto gradient = [&](uint32_t d, uint32_t ta, uint32_t b_lo, int n) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(el, d, ta + 64 * (kk >> 2) + 8 * (kk & 3), b_lo + kk * (2048 >> 4), idG,
                 n > 0 || kk > 0);
      };
      auto s_of = [&](int n) -> bool {
        if (!arrived(B_QF, NQ, sQ, n)) return false;
        mma_tile_ss<D>(el, tm, k_lo, q_lo + (n % NQ) * T16, idS);
        mma_commit(el, bar(B_S));
        return true;
      };
      auto dp_of = [&](int n) -> bool {
        if (!arrived(B_OF, NO, sO, n)) return false;
        mma_tile_ss<D>(el, tm + 128, v_lo, o_lo + (n % NO) * T16, idS);
        mma_commit(el, bar(B_DP));
        return true;
      };
      bool ok = wait(B_KV, 0, 0) && s_of(0) && dp_of(0);
      for (int n = 0; ok && n < NT; ++n) {
        if (!(ok = wait(B_P, n & 1, n))) break;
        tc_fence_after();
        gradient(tm + 256, tm, ot_lo + (n % NO) * T16, n);
        mma_commit(el, bar(B_OE + n % NO));
        if (n + 1 < NT && !(ok = s_of(n + 1))) break;
        if (!(ok = wait(B_DS, n & 1, n))) break;
        tc_fence_after();
        gradient(tm + 384, tm + 128, qt_lo + (n % NQ) * T16, n);
        mma_commit(el, bar(B_QE + n % NQ));
        if (n + 1 < NT && !(ok = dp_of(n + 1))) break;
      }
      mma_commit(el, bar(B_END));
      if (!ok) drain_bar(bar(B_END), 0);  // products in flight end before TMEM is freed
    } else if (warp == 10) {
      // ------------------------------ statistics ---------------------------------
      int h = g * a.G, qt = 0;
      for (int n = 0; n < N; ++n) {
        const int s = n % NS;
        const float2* src = a.stats + (size_t)h * a.T + it.start + j0 + qt * 128;
        const int left = it.len - j0 - qt * 128;
        float2 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[u] = lane + 32 * u < left ? __ldg(src + lane + 32 * u) : make_float2(-INFINITY, 0.f);
        if (n >= NS && !wait_bar_warp(bar(B_TE + s), ((n / NS) & 1) ^ 1, abort_flag, a.status,
                                      wait_site(kKerDenseDkv, B_TE + s, n)))
          break;
#pragma unroll
        for (int u = 0; u < 4; ++u) sSt[s * 128 + lane + 32 * u] = v[u];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_TF + s));
        if (++qt == nq) qt = 0, ++h;
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    if (BIAS) {  // the padded last tile included
      dense_bias_fill<false>(a, sB, g, nq * 128 - 1);
      named_bar_sync(2, 256);
    }
    // ------------------------------ P^T and dS^T ------------------------------------
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // key of the tile
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    bool dead = false;
    int qt = 0, hl = 0;
    int bk = 0, stn = 0;  // bias: bucket of the next queries, first distance of the one behind
    float bias0 = 0.f;    // its bias
    for (int n = 0; n < N; ++n) {
      const int s = n % NS;
      const int rel = qt * 128 + 64 * w - r;  // distance of the first of this warpgroup's queries
      const bool diag = qt == 0;              // queries c with rel + c < 0 come before the key
      auto wait = [&](int bb, uint32_t par) {
        dead = dead || !wait_bar_warp(bar(bb), par, abort_flag, a.status,
                                      wait_site(kKerDenseDkv, bb, n));
        tc_fence_after();
      };
      uint32_t x[2][32];
      const float4* st = reinterpret_cast<const float4*>(sSt + s * 128 + 64 * w);
      bool one = true, near = false;  // see DenseBias
      const uint16_t* tab = a.bias + (size_t)(g * a.G + hl) * a.nb;
      if (BIAS) {
        if (qt == 0 || __any_sync(0xffffffffu, rel >= stn)) {  // another head, or bucket
          bk = dense_bucket(sB, rel);
          stn = bk + 1 < a.nb ? sB->starts[bk + 1] : INT_MAX;
          bias0 = dense_bias_log2(__ldg(tab + bk));
        }
        one = __all_sync(0xffffffffu, stn > rel + 63);
        near = __all_sync(0xffffffffu, rel + 63 < a.lut_w);
      }
      wait(B_TF + s, (n / NS) & 1);
      wait(B_S, n & 1);
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
          } else if (__all_sync(0xffffffffu,
                                bk + 2 >= a.nb || sB->starts[bk + 2] > rel + 63)) {
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
            int q = bk;
            int nx = q + 1 < a.nb ? sB->starts[q + 1] : INT_MAX;
            float bv = bias0;
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              if (rel + i >= nx) {
                ++q;
                nx = q + 1 < a.nb ? sB->starts[q + 1] : INT_MAX;
                bv = dense_bias_log2(__ldg(tab + q));
              }
              x[i >> 5][i & 31] = __float_as_uint(
                  ex2_approx(fmaf(__uint_as_float(x[i >> 5][i & 31]), c, sl[i].x + bv)));
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
      wait(B_DP, n & 1);
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
      if (++qt == nq) qt = 0, ++hl;
    }
    dead = dead || !wait_bar_warp(bar(B_END), 0, abort_flag, a.status,
                                  wait_site(kKerDenseDkv, B_END, N));
    tc_fence_after();
    if (!dead) {
      // the first warpgroup stores dV, the second dK
      const size_t row = (size_t)(it.start + j0 + r) * a.hkv + g;
      uint16_t* dst = j0 + r < it.len ? (w == 0 ? a.dv : a.dk) + row * D : nullptr;
      store_tmem_rows<D>(tl + 256 + 128 * w, w == 0 ? 1.f : a.scale, sQ + warp * 4096, dst);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// dtable[h][b] = sum over the work items, in fp64 and in a fixed order.  One CTA per head;
// thread (b, c) sums every nc-th item, then the chunks are added in order.
constexpr int kTableThreads = 1024;
__global__ void __launch_bounds__(kTableThreads) k_dense_dtable(const DenseArgs a,
                                                                uint16_t* dtable) {
  __shared__ double sum[kTableThreads];
  int nb2 = 1;
  while (nb2 < a.nb) nb2 <<= 1;
  const int h = blockIdx.x, b = threadIdx.x % nb2, c = threadIdx.x / nb2, nc = kTableThreads / nb2;
  double s = 0.0;
  if (b < a.nb) {
#pragma unroll 8
    for (int x = c; x < a.nslots; x += nc)
      s += (double)__ldg(a.parts + ((size_t)x * a.hq + h) * a.nb + b);
  }
  sum[threadIdx.x] = s;
  __syncthreads();
  if (c == 0 && b < a.nb) {
    for (int i = 1; i < nc; ++i) s += sum[i * nb2 + b];
    const __nv_bfloat16 y = __float2bfloat16((float)s);
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
  k_dense_dq<D, BIAS><<<(unsigned)a.nslots * a.hkv, kThreads, DqCfg<D, BIAS>::kSmem, st>>>(mqp, mop, mk,
                                                                                     mv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  a.nslots = dense_slots(a.T, a.ndoc, 128);
  k_dense_dkv<D, BIAS><<<(unsigned)a.nslots * a.hkv, kThreads, DkvCfg<D, BIAS>::kSmem, st>>>(mq, mo, mk, mv, a);
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
  k_dense_dtable<<<a.hq, kTableThreads, 0, st>>>(b, dtable);
  return cudaGetLastError();
}

}  // namespace msa
