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
// At d = 64 a product over 128 keys takes half as long while the exponentials take the
// same time, so the wait for the next S would show: there the softmax works on 64 keys
// at a time (S, P and their barriers in halves), and one half's products run under the
// other half's exponentials; one warp issues the products of each row tile, so that what a
// hand-off costs it (some hundred cycles) overlaps the other's (10007 tokens, 12 heads:
// 110 -> 95 us), and the exponentials start ahead of the maximum (95 -> 84 us).  At d = 128,
// where the tensor core is the bound, two issuing warps share it out between the tiles and
// finish both later (32768 tokens, 8 heads: 1.21 -> 1.74 ms with them).
//
// Bound at d = 128 by the tensor core: one document of 32768 tokens, 8 heads on 2: 1.26 ms,
// 1.74 PFLOP/s (a library product under the same power cap: 1.73); 8 ragged documents of as
// many tokens, 16 heads on 4: 0.41 ms, 1.47.
//
// Roles (384 threads): warps 0-3 and 4-7 are the softmax warpgroups of tile 0
// and 1, so one tile's softmax overlaps the other's products; warp 8 loads;
// warp 9 (and 10) issues the MMAs: P V of a tile, then its next S.
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
  static constexpr int kHalves = D == 128 ? 1 : 2;  // softmax steps per key tile
  static constexpr int kMmaWarps = D == 128 ? 1 : 2;
  // K and V tiles in flight; with a bias its tables take the place of one
  static constexpr int kRing = D == 128 ? (BIAS ? 4 : 5) : 8;
  static constexpr int kSmem = (2 + kRing) * kTile + 256 + (BIAS ? (int)sizeof(DenseBias) : 0);
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(dense_turns(kRing) && dense_turns(2 * kHalves), "counts are turned back");
};

template <int D, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    k_dense_fwd(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DenseArgs a) {
  using C = FwdCfg<D, BIAS>;
  constexpr int NCH = D / 64, NR = C::kRing, NH = C::kHalves, W = 128 / NH;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;  // [2]
  uint8_t* sKV = sQ + 2 * C::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + NR * C::kTile);
  // Q loaded / free | ring full / empty | [t][b]: S of tile t complete in buffer b; the
  // first / second 64 keys of its P stored; P V of an even / odd step complete (the
  // softmax may be a step ahead of a product)
  constexpr int B_Q = 0, B_QE = 1, B_F = 2, B_E = B_F + NR, B_S = B_E + NR, B_P = B_S + 4,
                B_PV = B_P + 4, B_END = B_PV + 4;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + B_END + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((B_END + 1) * 8 + 8 <= 256, "barrier block");
  DenseBias* sB = reinterpret_cast<DenseBias*>(reinterpret_cast<uint8_t*>(bars) + 256);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (blockIdx.x == 0 && warp == 11) dense_check_docs(a);
  const int tpc = 2 * a.tpt;  // tokens per item
  DenseDocs docs;
  dense_docs_load(a, docs);

  if (threadIdx.x == 256) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (threadIdx.x == 0) {
    mbar_init(bar(B_Q), 1);
    mbar_init(bar(B_QE), C::kMmaWarps);
    for (int s = 0; s < NR; ++s) {
      mbar_init(bar(B_F + s), 1);
      mbar_init(bar(B_E + s), C::kMmaWarps);
    }
    for (int t = 0; t < 2; ++t) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(bar(B_S + 2 * t + h), 1);
        mbar_init(bar(B_P + 2 * t + h), 4);
        mbar_init(bar(B_PV + 2 * t + h), 1);
      }
    }
    mbar_init(bar(B_END), C::kMmaWarps);
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
  // TMEM: S/P of tile t at columns [128 t, 128 t + 128), O of tile t at 256 + D t

  // The items of this CTA, in the same order for every role.  Ring positions, steps and
  // barrier phases run on from item to item: the next item's loads and first products
  // start while the softmax warps still finish the last.
  struct Work {
    DenseItem it;
    int g, q0;   // KV head; first token of the item inside the document
    int nu[2];   // steps of W keys of each row tile: up to its last valid token
    int tiles;   // key tiles
  };
  const int rounds = dense_docs(a, tpc, docs) ? dense_rounds(a) : 0;
  auto work = [&](int k, Work& w) -> bool {
    int slot;
    if (!dense_round(a, k, &slot, &w.g) || !dense_item<false>(a, docs, slot, tpc, w.it))
      return false;
    w.q0 = w.it.tile * tpc;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = w.q0 + t * a.tpt;
      w.nu[t] = first < w.it.len && w.it.doc < a.ndoc
                    ? (min(first + a.tpt, w.it.len) + W - 1) / W
                    : 0;
    }
    w.tiles = (max(w.nu[0], w.nu[1]) + NH - 1) / NH;
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<kRegsCtl>();
    if (warp == 8) {
      // ------------------------------ loads --------------------------------------
      const uint32_t rows = (uint32_t)a.tpt * a.G * 128;  // bytes of one 64-column Q box
      int x = 0, items = 0;  // ring position (K0, V0, K1, V1, ...), items begun
      bool ok = true;
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.tiles == 0) continue;
        if (items > 0 && !(ok = dense_wait(bar(B_QE), (items - 1) & 1, abort_flag, a.status,
                                           wait_site(kKerDenseFwd, B_QE, items))))
          break;
        const int nq = w.nu[1] ? 2 : 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_Q), nq * NCH * rows);
          for (int t = 0; t < nq; ++t)
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(smem_u32(sQ + t * C::kTile + c * 16384), &tm_q, bar(B_Q), 64 * c,
                          w.g * a.G, w.it.start + w.q0 + t * a.tpt);
        }
        ++items;
        for (int y = 0; y < 2 * w.tiles; ++y, ++x) {
          const int s = x % NR;
          if (x >= NR && !(ok = dense_wait(bar(B_E + s), ((x / NR) & 1) ^ 1, abort_flag,
                                           a.status, wait_site(kKerDenseFwd, B_E + s, y >> 1))))
            break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_F + s), C::kTile);
            const uint32_t dst = smem_u32(sKV + s * C::kTile);
            const int tok = w.it.start + (y >> 1) * 128;
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(dst + c * 16384, (y & 1) ? &tm_v : &tm_k, bar(B_F + s), 64 * c, w.g, tok);
          }
        }
        __syncwarp();
        x = dense_turn(x);
      }
      // an aborted CTA must not leave before its copies have landed
      if (*abort_flag) {
        if (items > 0) drain_bar(bar(B_Q), (items - 1) & 1);
        for (int y = max(0, x - NR); y < x; ++y) drain_bar(bar(B_F + y % NR), (y / NR) & 1);
      }
    } else if (warp < 9 + C::kMmaWarps) {
      // ------------------------------ MMA issue ----------------------------------
      // One warp for both row tiles (d = 128), or one for each (d = 64).
      const int t0 = warp - 9, t1 = C::kMmaWarps == 1 ? 2 : warp - 8;
      constexpr uint32_t idS = make_idesc_bf16(128, W, false, false);
      constexpr uint32_t idO = make_idesc_bf16(128, D, false, true);
      const uint32_t el = elect_one(), tm = uniform(tbase);
      const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), k_lo = desc_lo(smem_u32(sKV), 16),
                     v_lo = desc_lo(smem_u32(sKV), 16384);
      auto wait = [&](int b, uint32_t par, int n) {
        return dense_wait(bar(b), par, abort_flag, a.status, wait_site(kKerDenseFwd, b, n));
      };
      auto wait_full = [&](int x) { return wait(B_F + x % NR, (x / NR) & 1, x >> 1); };
      int x = 0, items = 0, U[2] = {0, 0};  // ring position, items, steps of each tile so far
      // S of a step of tile t into buffer b: keys h W .. of the K tile at ring position xk
      auto issue_s = [&](int t, int xk, int h, int b) {
        mma_tile_ss<D>(el, tm + 128 * t + W * b, q_lo + t * (C::kTile >> 4),
                       k_lo + (xk % NR) * (C::kTile >> 4) + h * (W * 128 >> 4), idS);
        mma_commit(el, bar(B_S + 2 * t + b));
      };
      bool ok = true;
      for (int k = 0; ok && k < rounds; ++k) {
        Work w;
        if (!work(k, w) || w.tiles == 0) continue;
        const int len = uniform(w.it.len), nu0 = uniform(w.nu[0]), nu1 = uniform(w.nu[1]);
        const int nk = uniform(w.tiles);
        if (!(ok = wait(B_Q, items & 1, items) && wait_full(x))) break;
        ++items;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if (t0 == 0 && h < nu0) issue_s(0, x, h, (U[0] + h) % NH);
          if (t1 == 2 && h < nu1) issue_s(1, x, h, (U[1] + h) % NH);
        }
        mma_commit(el, bar(B_E + x % NR));
        if (nk == 1) mma_commit(el, bar(B_QE));
        for (int n = 0; ok && n < nk; ++n) {
          const int xv = x + 2 * n + 1, sv = xv % NR;
          if (!(ok = wait_full(xv))) break;
          // keys behind the document's end: P is zero there, V must be finite
          if ((n + 1) * 128 > len) dense_zero_rows<D>(sKV + sv * C::kTile, len - n * 128);
          const uint32_t v = v_lo + sv * (C::kTile >> 4);
#pragma unroll
          for (int ht = 0; ht < 2 * NH; ++ht) {
            const int h = ht >> 1, t = ht & 1, u = n * NH + h, nut = t ? nu1 : nu0;
            if (!ok || t < t0 || t >= t1 || u >= nut) continue;
            const int Ut = U[t] + u, b = Ut % NH;
            const uint32_t po = tm + 256 + D * t, pa = tm + 128 * t + W * b;
#pragma unroll
            for (int q = 0; ok && q < 2 / NH; ++q) {  // 64 keys of O += P V
              ok = wait(B_P + 2 * t + (NH == 1 ? q : b), (Ut / NH) & 1, n);
              if (!ok) break;
              tc_fence_after();
              const int vk = NH == 1 ? 4 * q : 4 * h;  // first of the V tile's 16-key steps
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts(el, po, pa + 32 * q + 8 * kk, v + (vk + kk) * (2048 >> 4), idO,
                       u > 0 || q > 0 || kk > 0);
            }
            if (!ok) break;
            mma_commit(el, bar(B_PV + 2 * t + (Ut & 1)));
            if (u + NH < nut) {
              if (!(ok = wait_full(xv + 1))) break;
              tc_fence_after();
              issue_s(t, xv + 1, h, b);
            }
          }
          if (!ok) break;
          mma_commit(el, bar(B_E + sv));
          if (n + 1 < nk) {
            // a warp without a step left releases no tile that it has not seen arrive
            if (NH == 2 && !(ok = wait_full(xv + 1))) break;
            mma_commit(el, bar(B_E + (xv + 1) % NR));
          }
          if (n + 2 == nk) mma_commit(el, bar(B_QE));  // the last S has been issued
        }
        x = dense_turn(x + 2 * nk);
        U[0] = dense_turn(U[0] + nu0);
        U[1] = dense_turn(U[1] + nu1);
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
    float c = a.scale_log2, ref = 0.f;  // see dense_row_ref
    bool dead = false;
    int U = 0, table_of = -1;  // steps so far; KV head the bias tables are of
    for (int k = 0; k < rounds; ++k) {
      Work w;
      if (!work(k, w)) continue;
      if (w.it.doc == a.ndoc) {  // padding behind the last document: zero rows
        const int n = min(tpc, w.it.len - w.q0) * a.G;
        const int rr = (int)threadIdx.x;
        if (rr < n) {
          const size_t row =
              (size_t)(w.it.start + w.q0 + rr / a.G) * a.hq + w.g * a.G + rr % a.G;
          dense_zero_row(a.o + row * D, D);
          if (a.o_res) dense_zero_row(a.o_res + row * D, D);
          if (a.lse) a.lse[row] = -INFINITY;
        }
        continue;
      }
      if (BIAS && table_of != w.g) {
        dense_bias_tables<false>(a, sB, w.g);
        table_of = w.g;
      }
      const int qi = w.q0 + t * a.tpt + ti;  // token inside the document
      const bool valid = ti < a.tpt && qi < w.it.len;
      const int nut = t ? w.nu[1] : w.nu[0];
      float m = -INFINITY, l = 0.f;
      int bk = a.nb - 1, stk = INT_MAX;  // bucket of the next scores and its first distance
      float v0 = 0.f;                    // its bias
      const uint16_t* tab = a.bias + (size_t)(w.g * a.G + hl) * a.nb;
      if (BIAS) {
        ref = dense_row_ref(a, sB, hl, tab, qi);
        c = dense_row_scale(a, ref);
      }
      for (int u = 0; u < nut; ++u, ++U) {
        const int b = U % NH;  // buffer of this step
        const uint32_t par = (U / NH) & 1;
        const int rel = qi - u * W;  // keys 0..rel of this step are visible
        bool one = true, near = false;  // see DenseBias
        if (BIAS) {
          if (__any_sync(0xffffffffu, rel < stk)) {  // the row's first bucket here is another
            bk = dense_bucket(sB, rel);
            stk = bk > 0 ? sB->starts[bk] : INT_MIN;
            v0 = dense_bias_log2(__ldg(tab + bk), ref);
          }
          one = __all_sync(0xffffffffu, bk == 0 || stk <= rel - (W - 1));
          near = __all_sync(0xffffffffu, rel < a.lut_w && ref == 0.f);
        }
        dead = dead || !dense_wait(bar(B_S + 2 * t + b), par, abort_flag, a.status,
                                   wait_site(kKerDenseFwd, B_S + 2 * t + b, u));
        tc_fence_after();
        if (!dead) {
          uint32_t x[W];
          tmem_ld_row(ts + W * b, x);
          if (__any_sync(0xffffffffu, rel < W - 1)) {
#pragma unroll
            for (int i = 0; i < W; ++i)
              if (i > rel) x[i] = __float_as_uint(-INFINITY);
          }
          // P = 2^(x mul + add - m)
          float mul = c, add = 0.f;
          if (BIAS) {
            if (one) {
              add = v0;  // one bucket over the row's part of the tile
            } else {
              mul = 1.f;
              const float* lut = sB->lut + hl * a.lut_stride + dense_lut_pad(a) + rel;
              int kb = bk;  // the bucket of the next scores
              float bv = v0;
#pragma unroll
              for (int y = 0; y < W / 16; ++y) {
                const int lowest = rel - 16 * y - 15;  // distance of the last of these 16 scores
                const int st = kb > 0 ? sB->starts[kb] : INT_MIN;
                if (near) {
#pragma unroll
                  for (int i = 16 * y; i < 16 * y + 16; ++i)
                    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, lut[-i]));
                } else if (!__any_sync(0xffffffffu, lowest < st)) {
#pragma unroll
                  for (int i = 16 * y; i < 16 * y + 16; ++i)
                    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, bv));
                } else if (__all_sync(0xffffffffu, kb < 2 || sB->starts[kb - 1] <= lowest)) {
                  // one start inside: scores before `cut` take bv, the others v1
                  const int cut = kb > 0 ? rel - st + 1 : W;
                  const float v1 = dense_bias_log2(__ldg(tab + max(kb - 1, 0)), ref);
#pragma unroll
                  for (int i = 16 * y; i < 16 * y + 16; ++i)
                    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, i < cut ? bv : v1));
                  if (lowest < st) {
                    --kb;
                    bv = v1;
                  }
                } else {
#pragma unroll
                  for (int i = 16 * y; i < 16 * y + 16; ++i) {
                    while (kb > 0 && sB->starts[kb] > rel - i) {
                      --kb;
                      bv = dense_bias_log2(__ldg(tab + kb), ref);
                    }
                    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), c, bv));
                  }
                }
              }
              __syncwarp();
            }
          }
          float m4[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            m4[y] = __uint_as_float(x[W / 4 * y]);
#pragma unroll
            for (int i = W / 4 * y + 1; i + 1 < W / 4 * (y + 1); i += 2)
              m4[y] = fmax3(m4[y], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            m4[y] = fmaxf(m4[y], __uint_as_float(x[W / 4 * (y + 1) - 1]));
          }
          const float mx = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), mul, add);
          // At d = 64 the first half's exponentials do not wait for the maximum: they take the
          // running m, and again the new one in the rare step that moves it.
          constexpr bool kEarly = D == 64;
          const f32x2 mul2_ = pack2(mul, mul);
          f32x2 ls[2];
          uint32_t wp[W / 2];
          auto exps = [&](int part, float sub) {
            const f32x2 sub2 = pack2(sub, sub);
#pragma unroll
            for (int e = 0; e < W; e += 2) {
              const int of = e / (W / 2);
              if (of == part) {
                float p0, p1;
                unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), mul2_, sub2),
                        p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                ls[(e >> 1) & 1] = add2(ls[(e >> 1) & 1], pack2(p0, p1));
                wp[e / 2] = pack_bf16(p0, p1);
              }
            }
          };
          ls[0] = ls[1] = 0ull;
          float sub = add - (m == -INFINITY ? 0.f : m);
          if (kEarly) exps(0, sub);
          const bool grow = mx > m + kRescale || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? mx : m;
            const float f = m_new == m ? 1.f : ex2_approx(m - m_new);
            l *= f;
            m = m_new;
            if (u > 0) {
              // O is complete up to the last step once that step's P V product is
              const int pv = B_PV + 2 * t + ((U - 1) & 1);
              dead = dead || !dense_wait(bar(pv), ((U - 1) >> 1) & 1, abort_flag, a.status,
                                         wait_site(kKerDenseFwd, pv, u));
              tc_fence_after();
              if (!dead) {
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                  uint32_t y[32];
                  tmem_ld32(to + 32 * q, y);
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                  tmem_st32(to + 32 * q, y);
                }
              }
            }
            sub = add - (m == -INFINITY ? 0.f : m);
            if (kEarly) {
              ls[0] = ls[1] = 0ull;
              exps(0, sub);
            }
          }
          if (!kEarly) exps(0, sub);
          if (NH == 1) {
            // the product over the first 64 keys runs while the others are computed
            tmem_st32_async(ts, *reinterpret_cast<uint32_t(*)[32]>(wp));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + 2 * t));
          }
          exps(1, sub);
          if (NH == 1) {
            tmem_st32_async(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(wp + W / 4));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + 2 * t + 1));
          }
          if (NH == 2) {
            tmem_st32_async(ts + W * b, *reinterpret_cast<uint32_t(*)[32]>(wp));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + 2 * t + b));
          }
          float l0, l1;
          unpack2(add2(ls[0], ls[1]), l0, l1);
          l += l0 + l1;
        } else {
          if (lane == 0)
            for (int q = 0; q < 2 / NH; ++q) mbar_arrive(bar(B_P + 2 * t + (NH == 1 ? q : b)));
        }
      }
      if (nut > 0) {
        const int b = B_PV + 2 * t + ((U - 1) & 1);
        dead = dead || !dense_wait(bar(b), ((U - 1) >> 1) & 1, abort_flag, a.status,
                                   wait_site(kKerDenseFwd, b, nut));
        tc_fence_after();
        if (!dead) {
          const size_t row = (size_t)(w.it.start + qi) * a.hq + w.g * a.G + hl;
          const float inv = l == 0.f ? 0.f : 1.f / l;  // l = 0: no key left (bias -inf)
          uint16_t* dst = valid ? a.o + row * D : nullptr;
          uint16_t* res = valid && a.o_res ? a.o_res + row * D : nullptr;
#pragma unroll 1
          for (int q = 0; q < D / 64; ++q) {
            uint32_t v[64];
            tmem_ld_row(to + 64 * q, v);
            if (BIAS && l == 0.f) {
#pragma unroll
              for (int i = 0; i < 64; ++i) v[i] = 0;
            }
            dense_store_row(v, inv, dst ? dst + 64 * q : nullptr);
            if (a.o_res) dense_store_row<true>(v, inv, res ? res + 64 * q : nullptr);
          }
          if (valid && a.lse) {
            const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;  // NaN stays NaN
            a.lse[row] = a.o_res ? lse : lse + ref;
          }
        }
        tc_fence_before();
      }
      U = dense_turn(U);
    }
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
  const int grid = dense_grid(a);
  k_dense_fwd<D, BIAS><<<grid, kThreads, FwdCfg<D, BIAS>::kSmem, st>>>(mq, mk, mv, a);
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
    return a.bias ? launch_t<128, true>(a, mq, mk, mv, st)
                  : launch_t<128, false>(a, mq, mk, mv, st);
  return a.bias ? launch_t<64, true>(a, mq, mk, mv, st) : launch_t<64, false>(a, mq, mk, mv, st);
}

}  // namespace msa
