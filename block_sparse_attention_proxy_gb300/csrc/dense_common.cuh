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
// One item over all keys of a document of this length ends within the bounded waits.
constexpr int kDenseMaxTokens = 1 << 25;
constexpr int kDenseMaxGrid = 160;     // CTAs of a persistent kernel
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
  int lut_w, lut_stride;  // bias by distance in shared memory (DenseBias): distances, row length
  int starts[kDenseMaxBuckets];
  // forward outputs; in the backward o, o_res and lse are inputs
  uint16_t* o;
  uint16_t* o_res;  // bf16(O - o); null: not stored
  float* lse;       // with o_res relative to the rows' references, as the backward takes it
  // backward
  const uint16_t* d_o;
  long long do_stride;
  float2* stats;  // [hq][T] {-lse log2(e) (-inf: no key left), D = rowsum(dO o O)}
  uint16_t *dq, *dk, *dv;
  float* refs;    // [hq][T] the rows' references (dense_row_ref)
  float* slots;   // [CTA][nb][2][128] per-row bucket sums of dS
  float2* parts;  // [CTA][hq][nb] their sums over the CTA's items, each a pair (add_pair)
};

// Work along the tokens is cut into slots of `bt` tokens: document b owns the
// slots from cu[b] / bt + b on.  It has at most that many tiles up to the next
// document's first slot, so a slot names at most one tile, and no prefix sum
// over the documents is needed.  ndoc + 1 documents: the last is the padding.
__host__ __device__ inline int dense_slots(int T, int ndoc, int bt) { return T / bt + ndoc + 1; }

// Ring positions, tiles and steps are counted over all the items of a CTA, and only the place
// in a ring, the phase of its barriers and whether a ring has been filled once are taken from
// the counts.  Between items a large one is turned back by a multiple of twice every ring's
// length: long documents of many heads reach 2^31.  An item adds at most 2^24.
constexpr int kDenseTurn = 240 << 21;
__host__ __device__ constexpr int dense_turn(int x) {
  return x >= 2 * kDenseTurn ? x - kDenseTurn : x;
}
__host__ __device__ constexpr bool dense_turns(int ring) { return kDenseTurn % (2 * ring) == 0; }

// The same value in every lane (lane 0's), and known to the compiler to be: control flow on
// it does not count as divergent, which would keep operands out of uniform registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// wait_bar_warp, with a plain test first: the suspending wait costs some hundred cycles even
// where the phase has completed already, which here is the common case.
__device__ __forceinline__ bool dense_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           unsigned* status, uint32_t site) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, ok)) return true;
  return wait_bar_warp(bar, parity, abort_flag, status, site);
}

struct DenseItem {
  int doc, start, len, tile;  // document, its first token and length, tile inside it
};

// The documents as a warp holds them: up to 64, two to a lane.
struct DenseDocs {
  int first[2], len[2], n[2];  // first token, length, tiles
  int total, most;             // tiles of all documents, of the longest
};
__device__ __forceinline__ int ld_nc_s32(const int32_t* p) {
  int v;  // volatile: issued here, ahead of what follows
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// Starts loading them (all lanes; the same in every warp): `len` holds the next one's first
// token until dense_docs, so that the loads run while the CTA sets itself up.
__device__ __forceinline__ void dense_docs_load(const DenseArgs& a, DenseDocs& d) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int b = lane + 32 * u;
    d.first[u] = d.len[u] = 0;
    if (a.ndoc <= 64 && b <= a.ndoc) d.first[u] = ld_nc_s32(a.cu + b);
    if (a.ndoc <= 64 && b < a.ndoc) d.len[u] = ld_nc_s32(a.cu + b + 1);
  }
}
// False if cu_seqlens is malformed (flagged).
__device__ __forceinline__ bool dense_docs(const DenseArgs& a, int bt, DenseDocs& d) {
  if (a.ndoc > 64) return true;
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int b = lane + 32 * u;
    const int next = b < a.ndoc ? d.len[u] : d.first[u];
    d.len[u] = next - d.first[u];
    bad |= d.first[u] < 0 || d.len[u] < 0 || next > a.T || (b == 0 && d.first[u] != 0);
    d.n[u] = (d.len[u] + bt - 1) / bt;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (threadIdx.x == 0) set_status(a.status, MSA_ERR_DEVICE_CHECK);
    return false;
  }
  d.total = __reduce_add_sync(0xffffffffu, d.n[0] + d.n[1]);
  d.most = __reduce_max_sync(0xffffffffu, max(d.n[0], d.n[1]));
  return true;
}

// Work item number `x` of dense_slots(): a tile of a document (all lanes of a warp; the
// same in every warp).  A document outside [0, T] or of negative length is flagged
// and skipped, so every token index derived from the item is inside the batch.
//
// Up to 64 documents, items come by falling work, so that a long one does not start last
// and run alone.  Work grows with the tile's index i (LAST: with its distance from the
// document's end), so item x has the largest i for which
// N(i) = sum over documents of max(0, tiles - i) exceeds x, a warp sum.  More documents (many
// short ones) go document by document through the slots above, found 32 documents at a
// time.
template <bool LAST>
__device__ __forceinline__ bool dense_item(const DenseArgs& a, const DenseDocs& d, int x, int bt,
                                           DenseItem& it) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kAll = 0xffffffffu;
  int doc, b0, b1, tile;
  if (a.ndoc <= 64) {
    if (x >= d.total) {  // behind the documents: the padding
      doc = a.ndoc;
      b0 = __ldg(a.cu + a.ndoc);
      b1 = a.T;
      tile = x - d.total;
    } else {
      int lo = 0, hi = d.most - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int)__reduce_add_sync(kAll, max(0, d.n[0] - mid) + max(0, d.n[1] - mid)) > x) lo = mid;
        else hi = mid - 1;
      }
      const int above =
          __reduce_add_sync(kAll, max(0, d.n[0] - lo - 1) + max(0, d.n[1] - lo - 1));
      // the (x - above)-th document with more than lo tiles
      const uint32_t m0 = __ballot_sync(kAll, d.n[0] > lo), m1 = __ballot_sync(kAll, d.n[1] > lo);
      int r = x - above;
      const bool second = r >= __popc(m0);
      if (second) r -= __popc(m0);
      const bool in = second ? d.n[1] > lo : d.n[0] > lo;
      const uint32_t before = (second ? m1 : m0) & ((1u << lane) - 1);
      const int l = __ffs(__ballot_sync(kAll, in && __popc(before) == r)) - 1;
      doc = l + (second ? 32 : 0);
      b0 = __shfl_sync(kAll, second ? d.first[1] : d.first[0], l);
      b1 = b0 + __shfl_sync(kAll, second ? d.len[1] : d.len[0], l);
      tile = LAST ? (b1 - b0 + bt - 1) / bt - 1 - lo : lo;
    }
  } else {
    const int s = LAST ? x : a.nslots - 1 - x;  // longest tiles of a document first
    // last b in [0, ndoc] with cu[b] / bt + b <= s; the last round's lanes hold the
    // document's first token and the next one's
    int n = a.ndoc + 1;
    doc = b0 = b1 = 0;
    for (bool found = false; !found;) {
      const int step = (n + 31) >> 5;
      const int b = doc + lane * step;
      const bool in = lane * step < n;
      const int c = in ? __ldg(a.cu + b) : 0;
      const int next = step == 1 && in ? (b < a.ndoc ? __ldg(a.cu + b + 1) : a.T) : 0;
      const bool le = in && min(max(c, 0), a.T) / bt + b <= s;
      const int last = max(__popc(__ballot_sync(kAll, le)) - 1, 0);
      found = step == 1;
      if (found) {
        b0 = __shfl_sync(kAll, c, last);
        b1 = __shfl_sync(kAll, next, last);
      }
      doc += last * step;
      n = min(step, n - last * step);
    }
    if (b0 < 0 || b1 < b0 || b1 > a.T) {
      if (threadIdx.x == 0) set_status(a.status, MSA_ERR_DEVICE_CHECK);
      return false;
    }
    tile = s - (b0 / bt + doc);
  }
  it.doc = uniform(doc);
  it.start = uniform(b0);
  it.len = uniform(b1 - b0);
  it.tile = uniform(tile);
  return it.tile >= 0 && (long long)it.tile * bt < it.len;
}

// Round k of a persistent CTA over `total` = slots x KV heads items, sorted by falling work:
// even rounds run through the CTAs forwards, odd ones backwards, which evens their sums out,
// and a CTA keeps its KV head where the grid is a multiple of hkv (h runs backwards in odd rounds).
__device__ __forceinline__ bool dense_round(const DenseArgs& a, int k, int* slot, int* g) {
  const uint32_t grid = gridDim.x, hkv = a.hkv;  // items: below 2^31 (checked on the host)
  const uint32_t x = (k & 1) ? (k + 1) * grid - 1 - blockIdx.x : k * grid + blockIdx.x;
  if (x >= a.nslots * hkv) return false;
  const uint32_t h = x % hkv;
  *slot = x / hkv;
  // a slot's heads must all lie in one round for this to name each once
  *g = (k & 1) && grid % hkv == 0 ? hkv - 1 - h : h;
  return true;
}
__device__ __forceinline__ int dense_rounds(const DenseArgs& a) {
  return ((uint32_t)a.nslots * a.hkv + gridDim.x - 1) / gridDim.x;
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

// 16 bytes of read-only global memory; not moved across other volatile instructions.
__device__ __forceinline__ uint4 ld_nc_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A float of global memory from L2; not moved across other volatile instructions.
__device__ __forceinline__ float ld_cg_f32(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

// TMEM -> registers: 64 or 128 columns of this thread's lane, one wait for all of them.
__device__ __forceinline__ void tmem_ld_row(uint32_t ta, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
        "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]),
        "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(ta), "r"(ta + 32)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_row(uint32_t ta, uint32_t (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
        "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]),
        "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]),
        "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
        "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]),
        "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]),
        "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]),
        "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
        "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]),
        "=r"(r[102]), "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]),
        "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]),
        "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
        "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]),
        "=r"(r[126]), "=r"(r[127])
      : "r"(ta), "r"(ta + 32), "r"(ta + 64), "r"(ta + 96)
      : "memory");
}
// registers -> TMEM: 32 columns, completed by tmem_wait_st.
__device__ __forceinline__ void tmem_st32_async(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two fp32 values in one 64-bit register pair: one instruction does both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(f32x2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// ---------------------------------------------------------------------------
// MMA issue by a converged warp.  The tensor-core instructions take their
// descriptors from uniform registers: issued from inside `if (lane == 0)` each
// cost the issuing warp about 85-100 cycles at N = 128 (a product lasts 64), because
// every operand was moved over by itself.  Here all lanes compute the
// (warp-uniform) operands and the instruction is predicated on one elected lane.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}
// Low and high words of a shared-memory matrix descriptor (make_sdesc); moving the
// start address by `bytes` adds bytes / 16 to the low word.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (kLayoutSW128 << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t el, uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(el)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t el, uint32_t d, uint32_t a_tmem, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(el)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t el, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar),
      "r"(el)
      : "memory");
}
// 128 x N (+)= 128 x K by N x K tiles in shared memory, both K-major in 64-column
// chunks of 16 KB.
template <int K>
__device__ __forceinline__ void mma_tile_ss(uint32_t el, uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                            uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < K / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
    mma_ss(el, d, a_lo + off, b_lo + off, idesc, kk > 0);
  }
}

// A bias in log2 units, less the row's reference (dense_row_ref).
__device__ __forceinline__ float dense_bias_of(uint16_t raw) {
  return __uint_as_float((uint32_t)raw << 16);
}
__device__ __forceinline__ float dense_bias_log2(uint16_t raw, float ref = 0.f) {
  return (dense_bias_of(raw) - ref) * kLog2E;
}

// Softmax does not change when a row's scores all move by the same amount, and a score next to a
// bias of -1e9 (a mask by a large finite value) has no bits left in fp32.  So a row whose
// largest bias within reach is that far from zero takes its biases, its maximum and its
// log-sum-exp relative to that bias, its reference: equal biases cancel before a score is added,
// and what lies far below the reference has no weight whether it overflows or not.  All other
// rows have the reference 0 (a largest bias of at most 64 leaves a score 2^-17 of precision).
// From 2^56 on, the lowest value of a type among them, a sum of bias and score holds no bit of
// the score in 64 bits either: such a row weighs its keys equally, as that sum does.
constexpr float kDenseModerate = 64.f, kDenseAbsorbs = 72057594037927936.f;
__device__ __forceinline__ bool dense_extreme(float b) {
  return fabsf(b) > kDenseModerate && fabsf(b) < INFINITY;
}
// What scores of such a row are multiplied by.  Not 0: a masked score is -inf.
__device__ __forceinline__ float dense_row_scale(const DenseArgs& a, float ref) {
  return fabsf(ref) < kDenseAbsorbs ? a.scale_log2 : 1e-30f;
}

// What a CTA keeps of the bias table in shared memory.  Tiles whose rows each lie in
// one bucket (most tiles far from the diagonal) take it as one constant per row.  Near
// the diagonal a row crosses many buckets: there the bias is read by distance
// from `lut` (one conflict-free load per score, no search and no branch), which
// holds the distances below lut_w for every head of the group, preceded by zeros
// for the negative distances of masked scores.  Rows that cross a bucket farther
// out walk the bucket starts, 16 scores at a time where none begins.
constexpr int kDenseLut = 4096;       // entries over all heads of the group
constexpr int kDenseBits = 8192;      // distances whose bucket starts are kept as bits
constexpr int kDenseBitsPad = 256;    // bits before distance 0
constexpr int kDenseTable = 512;      // staged table entries over all heads of the group
struct DenseBias {
  float lut[kDenseLut];
  uint32_t bits[(kDenseBits + kDenseBitsPad) / 32 + 2];
  int starts[kDenseMaxBuckets];  // INT_MAX behind the last bucket
  float table[kDenseTable];      // [G][nb] in log2 units, if it fits
  int clear[kDenseMaxGroup];     // rows at this place of a document and later have no reference
  int loose;                     // 1: an entry is no finite number in log2 units, nor -inf
};
// Row length of the table (heads end on different banks: a warp reads 32/G tokens of G
// heads at once) and the distances that fit.
__host__ inline void dense_lut_shape(DenseArgs* a) {
  const int per = kDenseLut / a->G;
  a->lut_stride = a->G <= 32 ? (per - 32) / 32 * 32 + 32 / a->G : per;
  const int w = a->lut_stride - (127 + a->tpt), last = a->nb > 0 ? a->starts[a->nb - 1] : 0;
  a->lut_w = w < 0 ? 0 : w;
  // a warp's part of a tile spans fewer than 256 distances: beyond this it lies in one bucket
  if (a->lut_w - 256 > last) a->lut_w = last + 256;  // the last start may be INT_MAX
}
__device__ __forceinline__ int dense_lut_pad(const DenseArgs& a) { return 127 + a.tpt; }

// The bucket of distance x (0 for a negative one): the last one that begins at or before x.
__device__ __forceinline__ int dense_bucket(const DenseBias* s, int x) {
  int b = 0;
#pragma unroll
  for (int step = kDenseMaxBuckets / 2; step > 0; step >>= 1)
    if (s->starts[b + step] <= x) b += step;
  return b;
}

// The reference of a row: the largest bias over the distances 0..last of its keys, if that is
// far from zero (tab: row hl of the group's table).  All buckets up to the last one's are
// reached, so there is a key with this bias.
__device__ __forceinline__ float dense_row_ref(const DenseArgs& a, const DenseBias* s, int hl,
                                               const uint16_t* tab, int last) {
  if (last >= s->clear[hl]) return 0.f;
  float m = -INFINITY;
  for (int b = 0; b < a.nb && s->starts[b] <= last; ++b)
    m = fmaxf(m, dense_bias_of(__ldg(tab + b)));
  return dense_extreme(m) ? m : 0.f;
}

// Named barrier 2 of 256 threads, and whether `x` holds for one of them.
__device__ __forceinline__ bool dense_bar_any(bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 2, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"((uint32_t)x)
      : "memory");
  return y != 0;
}

// Fills it for KV head g (threads 0..255, all of them; none may still read the last one's).
template <bool BITS>
__device__ __forceinline__ void dense_bias_tables(const DenseArgs& a, DenseBias* s, int g) {
  const int tid = threadIdx.x, pad = dense_lut_pad(a);
  const int W = min(a.lut_w, (a.T + 127) / 128 * 128);  // distances that can occur
  const bool staged = a.G * a.nb <= kDenseTable;
  const uint16_t* tab = a.bias + (size_t)g * a.G * a.nb;
  named_bar_sync(2, 256);
  if (tid < kDenseMaxBuckets) s->starts[tid] = tid < a.nb ? a.starts[tid] : INT_MAX;
  if (tid < kDenseMaxGroup) s->clear[tid] = 0;
  if (tid == 0) s->loose = 0;
  bool extreme = false;
  for (int x = tid; x < a.G * a.nb; x += 256) {
    const uint16_t raw = __ldg(tab + x);
    if (staged) s->table[x] = dense_bias_log2(raw);
    const float b = dense_bias_of(raw);
    extreme |= !(fabsf(b) <= kDenseModerate || b == -INFINITY);
  }
  if (BITS)
    for (int x = tid; x < (kDenseBits + kDenseBitsPad) / 32 + 2; x += 256) s->bits[x] = 0;
  if (dense_bar_any(extreme) && tid < a.G) {
    // The first bucket with a moderate entry: rows that reach it have no reference, unless an
    // entry is large.  (A finite mask costs other rows no more than this comparison: a search
    // of the table by every row took 24 % of the time of 23 documents.)
    int clear = INT_MAX;
    bool high = false;
    for (int b = 0; b < a.nb; ++b) {
      const float x = dense_bias_of(__ldg(tab + tid * a.nb + b));
      high |= !(x <= kDenseModerate);
      if (x >= -kDenseModerate) clear = min(clear, s->starts[b]);
      if (!(x * kLog2E < INFINITY)) s->loose = 1;
    }
    s->clear[tid] = high ? INT_MAX : clear;
  }
  if (a.lut_w > 0) {
    for (int x = tid; x < pad; x += 256)
      for (int h = 0; h < a.G; ++h) s->lut[h * a.lut_stride + x] = 0.f;
    for (int x0 = tid; x0 < W; x0 += 1024) {
      int b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) b[u] = dense_bucket(s, x0 + 256 * u);
      for (int h = 0; h < a.G; ++h) {
        float* row = s->lut + h * a.lut_stride + pad + x0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int at = h * a.nb + b[u];
          if (x0 + 256 * u < W)
            row[256 * u] = staged ? s->table[at] : dense_bias_log2(__ldg(tab + at));
        }
      }
    }
  }
  if (BITS && tid > 0 && tid < a.nb && s->starts[tid] < kDenseBits)
    atomicOr(&s->bits[(s->starts[tid] + kDenseBitsPad) >> 5], 1u << (s->starts[tid] & 31));
  named_bar_sync(2, 256);
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

// 64 fp32 columns of a row (one row per lane), times f, rounded to bf16, to `row` (its first
// element; null: not stored): 32 bytes to a store, whole sectors, so that lanes need not
// exchange rows through shared memory first.  RES: what the rounding drops, itself as
// bf16, instead of the values.
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
template <bool RES = false>
__device__ __forceinline__ void dense_store_row(const uint32_t (&v)[64], float f, uint16_t* row) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __uint_as_float(v[16 * q + 2 * i]) * f;
      const float y = __uint_as_float(v[16 * q + 2 * i + 1]) * f;
      w[i] = pack_bf16(x, y);
      if (RES) w[i] = pack_bf16(x - bf16_lo(w[i]), y - bf16_hi(w[i]));
    }
    if (row) st_v8(row + 16 * q, w);
  }
}

// sum += x, where sum.y collects what the roundings of sum.x drop (each is exactly
// representable: Knuth's two-sum).  n terms are off by about n^2 2^-48 of the largest partial
// sum at most, whatever cancels.
__device__ __forceinline__ void add_pair(float2& sum, float x) {
  const float s = sum.x + x, b = s - sum.x;
  sum.y += (sum.x - (s - b)) + (x - b);
  sum.x = s;
}

// A row of zeros (documents' padding): `n` elements (a multiple of 8) by one thread.
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

// CTAs of a persistent kernel: one per SM, fewer if there are fewer items; with a bias a
// multiple of the KV heads where that costs few SMs, so that a CTA keeps its tables.
inline int dense_grid(const DenseArgs& a) {
  static std::atomic<int> sms[64];
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  if (dev < 64) n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n = 1;
    if (n > kDenseMaxGrid) n = kDenseMaxGrid;
    if (dev < 64) sms[dev].store(n, std::memory_order_relaxed);
  }
  if (a.bias && a.hkv * 8 <= n) n -= n % a.hkv;
  const long long items = (long long)a.nslots * a.hkv;
  return items < n ? (int)items : n;
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
