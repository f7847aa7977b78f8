// decode_device.cuh -- the decode attention kernel and its launch (see decode.cu for the
// work decomposition and the arithmetic), shared by the launches that read every packed
// group (decode.cu), those that read listed groups (groups.cu) and those that read the first
// and the last tokens, or hand out the groups' weights (stream.cu).
#pragma once

#include <algorithm>
#include <type_traits>
#include <utility>

#include "quant_device.cuh"

namespace kvc {
namespace {

constexpr int kSlotsPerWarp = kDecSlotsPerChunk;
static_assert(kSlotsPerWarp == 16, "window warps take 16 slots");
constexpr unsigned kWaitLimit = 1u << 20;   // bounded mbarrier polls (far above any copy)

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D apart from C: a chain's first product takes C as it is, or 0.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], float c0, float c1, float c2, float c3,
                                             uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------- bulk staging helpers
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n"
      :: "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// ------------------------------------------------------------ fragment helpers
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(integral_constant<int, i>) for i = 0 .. N-1, indices known at compile time
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Transpose of an 8x8 matrix of 16-bit elements held in the operand-fragment
// layout (lane = 4*row + col/2): afterwards lane 4*r + c/2 holds row r of the
// transpose.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// What a launch reads: every token; listed groups and the window; the first and the last tokens.
enum DecMode : int { kDecAll = 0, kDecList = 1, kDecRange = 2 };

// A launch over listed groups or a range of tokens (SEL) differs in four ways, for accuracy and range:
//  - The remainders ("lo" parts) are multiplied by 2^11, and their sums divided by it at the
//    end: the weights of a long list are small, their fp16 remainders would be subnormal,
//    with an error of 2^-25 whatever the weight.
//  - Codes are taken from the middle of their range (code - 2^(b-1)), so that the code sums are
//    small where the result is: the tensor cores cut an accumulator off at a step of its
//    own size. What that adds to the zero-point terms, 2^(b-1) S, goes with them.
//  - Window weights have a third part (split_rest).
//  - The queries of a unit whose products with the keys' scales may pass fp16's range, or fall below
//    it, are scaled by powers of two (scale_queries). Weights are formed from the difference to the
//    maximum, exact where logits are large.
// Over 2,048 tokens at 4 bits the output is 2e-6 off without them.
template <bool SEL>
constexpr float lo_scale() { return SEL ? 2048.f : 1.f; }

// v as a bf16 pair (hi, lo) with hi = bf16(v), lo = bf16((v - hi) lo_scale): hi in the low half.
template <bool SEL>
__device__ __forceinline__ uint32_t split_bf16(float v) {
  const float hi = __bfloat162float(__float2bfloat16_rn(v));
  const __nv_bfloat162 p = __floats2bfloat162_rn(v, SEL ? (v - hi) * lo_scale<SEL>() : v - hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// What split_bf16<true> leaves of v, for the same column as lo: (0, bf16((v - hi) lo_scale - lo)).
// (Without it a window weight is off by 2^-18 of itself, and the output by 1.5e-6 where the window
// is all there is; with it by 2^-26.)
__device__ __forceinline__ uint32_t split_rest(float v) {
  const float r = (v - __bfloat162float(__float2bfloat16_rn(v))) * lo_scale<true>();
  const __nv_bfloat162 p =
      __floats2bfloat162_rn(0.f, r - __bfloat162float(__float2bfloat16_rn(r)));
  return *reinterpret_cast<const uint32_t*>(&p);
}
// The masks of the code fields inside a byte of each 16-bit half, held in
// registers: with the mask a register operand, the field and the fp16 exponent
// bits are merged by one three-input logic instruction with the exponent as its
// immediate (a mask and an exponent both as immediates take two).
template <int BITS>
struct CodeMasks { uint32_t m[8 / BITS]; };

template <int BITS>
__device__ __forceinline__ CodeMasks<BITS> code_masks() {
  CodeMasks<BITS> cm;
  static_for<8 / BITS>([&](auto J_) {
    constexpr int J = decltype(J_)::value;
    constexpr uint32_t v = (((1u << BITS) - 1u) * 0x00010001u) << (BITS * J);
    asm volatile("mov.b32 %0, %1;" : "=r"(cm.m[J]) : "n"(v));
  });
  return cm;
}

// Exact fp16 pair of the two codes in pair slot P of word w (w8 = w >> 8). The
// field of slot P is masked in place under the fp16 exponent of 2^e, e = 10 -
// BITS*j (j = field index inside its byte), so each half reads 2^e + code; one
// subtraction leaves the code.
// MID 1: the code less 2^(BITS-1), exact too (the subtrahend 2^e + 2^(BITS-1) is an fp16 value). MID 2:
// the low half's code less one less than that: half a step to either side of the middle.
template <int BITS, int P, int MID = 0>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, uint32_t w8, const CodeMasks<BITS>& cm) {
  constexpr int CPB = 8 / BITS, SB = P / CPB, J = P % CPB;
  constexpr uint32_t mag = ((uint32_t)(25 - BITS * J) << 10) * 0x00010001u;
  constexpr uint32_t sub = mag + (MID ? ((1u << (BITS - 1)) << (BITS * J)) * 0x00010001u : 0u) -
                           (MID == 2 ? 1u << (BITS * J) : 0u);
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(SB ? w8 : w), "r"(cm.m[J]), "n"(mag));
  return h2u(__hsub2(u2h(v), u2h(sub)));
}

// A operand of key product (MT, KS) (rows = tokens, k = channels) from the lane's
// key code words.
template <int D, int BITS, int MT, int KS, int MID = 0>
__device__ __forceinline__ void key_afrag(const uint32_t* kw, const CodeMasks<BITS>& cm,
                                          uint32_t (&a)[4]) {
  if constexpr (BITS == 2) {
    constexpr int wi = MT * (D / 32) + KS / 2, b = 2 * (KS & 1);
    const uint32_t w = kw[wi], w8 = w >> 8;
    a[0] = unpack_pair<2, b, MID>(w, w8, cm);
    a[1] = unpack_pair<2, 4 + b, MID>(w, w8, cm);
    a[2] = unpack_pair<2, b + 1, MID>(w, w8, cm);
    a[3] = unpack_pair<2, 5 + b, MID>(w, w8, cm);
  } else {
    constexpr int wi = MT * (D / 16) + KS;
    const uint32_t w = kw[wi], w8 = w >> 8;
    a[0] = unpack_pair<4, 0, MID>(w, w8, cm);
    a[1] = unpack_pair<4, 2, MID>(w, w8, cm);
    a[2] = unpack_pair<4, 1, MID>(w, w8, cm);
    a[3] = unpack_pair<4, 3, MID>(w, w8, cm);
  }
}
// A operand of value product (MT, KS) (rows = channels, k = tokens).
template <int BITS, int MT, int KS, int MID = 0>
__device__ __forceinline__ void value_afrag(const uint32_t* vw, const CodeMasks<BITS>& cm,
                                            uint32_t (&a)[4]) {
  if constexpr (BITS == 2) {
    constexpr int b = 2 * KS;
    const uint32_t w = vw[MT], w8 = w >> 8;
    a[0] = unpack_pair<2, b, MID>(w, w8, cm);
    a[1] = unpack_pair<2, 4 + b, MID>(w, w8, cm);
    a[2] = unpack_pair<2, b + 1, MID>(w, w8, cm);
    a[3] = unpack_pair<2, 5 + b, MID>(w, w8, cm);
  } else {
    constexpr int wi = 2 * MT + KS;
    const uint32_t w = vw[wi], w8 = w >> 8;
    a[0] = unpack_pair<4, 0, MID>(w, w8, cm);
    a[1] = unpack_pair<4, 2, MID>(w, w8, cm);
    a[2] = unpack_pair<4, 1, MID>(w, w8, cm);
    a[3] = unpack_pair<4, 3, MID>(w, w8, cm);
  }
}

// Column layout of the B operands: column n of n-tile u belongs to query head
// 4u + n/2; even columns carry the leading ("hi") fp16/bf16 part of an operand
// product, odd columns the remainder ("lo"). A lane's C fragment (columns 2tid,
// 2tid+1) therefore holds both parts for head 4u + tid, and their sum is the
// full-precision product.
template <int GQ>
constexpr int n_tiles() { return (GQ + 3) / 4; }

template <int D, int GQ, int MODE>
struct WarpState {
  static constexpr int NH = n_tiles<GQ>();
  static constexpr bool Z = MODE == kDecList;
  // a list: value zero-point and mid-code sums per channel group (every row the same)
  float z[Z ? NH : 1][Z ? D / 32 : 1][4];
  // a range, one or two heads: lane-partial zero-point and mid-code sums of channel group tid % (D / 32)
  static constexpr bool kZp = MODE == kDecRange && GQ <= 2;
  float zp[kZp ? GQ : 1];
  float m[NH];                 // running max of the raw logits (head 4u + tid)
  float l[NH];                 // lane-partial sum of the weights
  float o[NH][D / 16][4];      // value accumulators: rows = channels, columns = (head, part)
};

template <int D, int GQ, int MODE>
__device__ __forceinline__ void state_init(WarpState<D, GQ, MODE>& st) {
  constexpr int NH = n_tiles<GQ>();
  if constexpr (WarpState<D, GQ, MODE>::kZp)
#pragma unroll
    for (int h = 0; h < GQ; ++h) st.zp[h] = 0.f;
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    st.m[u] = -INFINITY;
    st.l[u] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[u][i][e] = 0.f;
    if constexpr (MODE == kDecList)
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.z[u][i][e] = 0.f;
  }
}

// What takes logits to log2 units: one factor, or one per head 4u + tid where queries are scaled.
__device__ __forceinline__ float sl2_of(float sl2, int) { return sl2; }
template <int N>
__device__ __forceinline__ float sl2_of(const float (&sl2)[N], int u) { return sl2[u]; }
template <bool SEL, int N>
__device__ __forceinline__ const auto& sl2_pick(const float (&heads)[N], const float& all) {
  if constexpr (SEL) return heads;
  else return all;
}

// SEL: a unit's staged queries and, behind them, its marks (16 bytes) and a factor per head. Products
// of queries and key scales are formed as fp16 pairs, exact to 2^-25 at best and 65,504 at
// most. Scales are at most 512 in a unit that is not marked (kWideScale), so queries are taken as
// they are where each row's largest magnitude lies in [1/4, 64). Else this takes every row to
// [32, 64) by a power of two, in place, in a marked unit to [1/4, 1/2); the factors are then sl2
// over the rows' scales.
template <int D, int GQ>
__device__ __forceinline__ void scale_queries(__nv_bfloat16* qs, float sl2) {
  const int lane = threadIdx.x & 31;
  const bool marked = *reinterpret_cast<const unsigned*>(qs + GQ * D) & kWideScale;
  float* factors = reinterpret_cast<float*>(qs + GQ * D) + 4;
  for (int h = 0; h < GQ; ++h) {
    __nv_bfloat162* row = reinterpret_cast<__nv_bfloat162*>(qs + h * D);
    uint32_t mx = 0u;          // as bf16 bits
    for (int i = lane; i < D / 2; i += 32) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(row + i);
      mx = max(mx, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
    }
    const int ex = (int)(__reduce_max_sync(0xffffffffu, mx) >> 7);
    const int by = ex == 255 ? 0 : max(-126, (marked ? 125 : 132) - max(ex, 14));   // (not finite: as it is)
    const __nv_bfloat162 f = __float2bfloat162_rn(__int_as_float((127 + by) << 23));
    for (int i = lane; i < D / 2; i += 32) row[i] = __hmul2(row[i], f);
    if (lane == 0) factors[h] = sl2 * __int_as_float((127 - by) << 23);
  }
  __syncwarp();
}

// Query operands of the packed path: qh = fp16 query pair of this lane's B column
// (zero beyond the group's heads); qn = -qh in "lo" columns, 0 in "hi" columns.
template <int D, int GQ>
struct QRegs {
  static constexpr int NH = n_tiles<GQ>();
  uint32_t qh[NH][D / 16][2];
  uint32_t qn[NH][D / 16][2];
};

// SEL: true if some row's largest magnitude is outside [1/4, 64) or the unit is marked.
template <int D, int GQ, bool SEL>
__device__ __forceinline__ bool load_qregs(QRegs<D, GQ>& qr, const __nv_bfloat16* qs) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  bool far = SEL && (*reinterpret_cast<const unsigned*>(qs + GQ * D) & kWideScale);
#pragma unroll
  for (int u = 0; u < n_tiles<GQ>(); ++u) {
    const int h = 4 * u + (gid >> 1);
    __nv_bfloat162 most = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        const int c = 16 * ks + 2 * tid + 8 * e2;
        float2 f = make_float2(0.f, 0.f);
        if (h < GQ) {
          const __nv_bfloat162 w = *reinterpret_cast<const __nv_bfloat162*>(qs + h * D + c);
          f = __bfloat1622float2(w);
          if constexpr (SEL) most = __hmax2(most, __habs2(w));
        }
        const __half2 q2 = __float22half2_rn(f);
        qr.qh[u][ks][e2] = h2u(q2);
        qr.qn[u][ks][e2] = (gid & 1) ? h2u(__hneg2(q2)) : 0u;
      }
    if constexpr (SEL) {
      float m = fmaxf(__low2float(most), __high2float(most));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      far = far || (h < GQ && !(m >= 0.25f && m < 64.f));
    }
  }
  return SEL && __any_sync(0xffffffffu, far);
}

// Online-softmax update with the logits of 16 * NMT tokens: x[u][mt][r] is token
// 16mt + gid + 8r for head 4u + tid. The weights replace the logits.
template <int D, int GQ, int NMT, bool SEL, int MODE, typename SL2>
__device__ __forceinline__ void softmax_update(WarpState<D, GQ, MODE>& st,
                                               float (&x)[n_tiles<GQ>()][NMT][2], const SL2& sl2_) {
#pragma unroll
  for (int u = 0; u < n_tiles<GQ>(); ++u) {
    const float sl2 = sl2_of(sl2_, u);
    float gm = fmaxf(x[u][0][0], x[u][0][1]);
#pragma unroll
    for (int mt = 1; mt < NMT; ++mt) gm = fmaxf(gm, fmaxf(x[u][mt][0], x[u][mt][1]));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 4));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 8));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 16));
    const float mnew = fmaxf(st.m[u], gm);
    if (__any_sync(0xffffffffu, mnew > st.m[u])) {
      const float corr = (st.m[u] == -INFINITY) ? 0.f : fast_exp2((st.m[u] - mnew) * sl2);
      st.l[u] *= corr;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[u][i][e] *= corr;
      if constexpr (MODE == kDecList)
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.z[u][i][e] *= corr;
      if constexpr (WarpState<D, GQ, MODE>::kZp)
#pragma unroll
        for (int h = 0; h < GQ; ++h) st.zp[h] *= __shfl_sync(0xffffffffu, corr, (threadIdx.x & 28) + h);
      st.m[u] = mnew;
    }
    const float msl = (st.m[u] == -INFINITY) ? 0.f : (SEL ? st.m[u] : st.m[u] * sl2);
    float s = 0.f;
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p = SEL ? fast_exp2((x[u][mt][r] - msl) * sl2) : fast_exp2(fmaf(x[u][mt][r], sl2, -msl));
        x[u][mt][r] = p;
        s += p;
      }
    st.l[u] += s;
  }
}

// ------------------------------------------------------------ ranges of tokens
// Which of a run of tokens are seen: the first `a` and those from `b` on.
struct Seen {
  int a, b;
  __device__ __forceinline__ bool at(int t) const { return t < a || t >= b; }
  __device__ __forceinline__ bool all(int n) const { return b <= 0 || a >= n || a >= b; }
};
// A chunk of a launch over everything or over a list.
struct PlainChunk {
  static constexpr bool kRange = false;
};
// A chunk of a launch over a range: its packed groups (or, in slot[0], its window chunk), the token
// range of its unit relative to the first, and where its weights go (null: nowhere).
struct RangeChunk {
  static constexpr bool kRange = true;
  int a, b;                 // seen: the unit's tokens before a and from b on
  int t0[2];                // first token of the chunk's groups (window chunk: t0[0])
  int slot[2];              // their places in the unit's parts
  float2* part;             // the unit's parts [slots][GQ]
  __device__ __forceinline__ Seen seen(int j) const {
    const int t = j == 0 ? t0[0] : t0[1];
    return {a - t, b - t};
  }
};
// A part: per head the sum of the weights of 16 NMT tokens against the running maximum they were
// formed with, (maximum in log2 units, sum).
template <int GQ, int NMT, typename SL2>
__device__ __forceinline__ void put_part(const float (&m)[n_tiles<GQ>()],
                                         const float (&x)[n_tiles<GQ>()][NMT][2], const SL2& sl2,
                                         float2* part) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < n_tiles<GQ>(); ++u) {
    float s = 0.f;
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt) s += x[u][mt][0] + x[u][mt][1];
    s += __shfl_xor_sync(0xffffffffu, s, 4);
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (lane < 4 && 4 * u + lane < GQ)
      __stcg(part + 4 * u + lane,
             make_float2(m[u] == -INFINITY ? -INFINITY : m[u] * sl2_of(sl2, u), s));
  }
}

// ------------------------------------------------------------ packed groups
// `base` points at n_grp (<= 8) consecutive group blocks in shared
// memory. Per group: key logits (rows = tokens), one online-softmax update, the
// value products (rows = channels). The group loop stays rolled so that the hot
// code fits the instruction cache.
template <int D, int BITS, int GQ, bool SEL, typename SL2>
__device__ void packed_warp(WarpState<D, GQ, SEL ? kDecList : kDecAll>& st, const QRegs<D, GQ>& qr, const uint8_t* base,
                            int n_grp, const SL2& sl2) {
  constexpr int KS = D / 16, NGC = D / 32, BB = 8 * D * (BITS + 1), WPL = D * BITS / 32;
  constexpr int NH = n_tiles<GQ>();
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;

  const CodeMasks<BITS> cm = code_masks<BITS>();
  // key zero-point sums of every group of the chunk: C[group][n] = Z_group . q_n
  // (A rows = groups; rows past the chunk's groups repeat group 0 and are not
  // read; B = the queries, whose "hi" column is read)
  float zb[NH];
  {
    uint32_t za[KS][2];
    const int gz = gid < n_grp ? gid : 0;
    const uint4* zp = reinterpret_cast<const uint4*>(base + (size_t)gz * BB + off_kzero(D, BITS) +
                                                     tid * (D / 4) * 2);
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {
      const uint4 z = zp[i];
      za[2 * i][0] = z.x;
      za[2 * i][1] = z.y;
      za[2 * i + 1][0] = z.z;
      za[2 * i + 1][1] = z.w;
    }
#pragma unroll
    for (int u = 0; u < NH; ++u) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        mma_f16(c, za[ks][0], 0u, za[ks][1], 0u, qr.qh[u][ks][0], qr.qh[u][ks][1]);
      zb[u] = c[0];   // group gid, head 4u + tid ("hi" column)
    }
    if constexpr (SEL) {
      // and of the middle code: 2^(b-1) S_group . q_n
      const uint4* sp = reinterpret_cast<const uint4*>(base + (size_t)gz * BB + off_kscale(D, BITS) +
                                                       tid * (D / 4) * 2);
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint4 z = sp[i];
        za[2 * i][0] = z.x;
        za[2 * i][1] = z.y;
        za[2 * i + 1][0] = z.z;
        za[2 * i + 1][1] = z.w;
      }
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          mma_f16(c, za[ks][0], 0u, za[ks][1], 0u, qr.qh[u][ks][0], qr.qh[u][ks][1]);
        zb[u] = fmaf((float)(1 << (BITS - 1)), c[0], zb[u]);
      }
    }
  }

#pragma unroll 1
  for (int j = 0; j < n_grp; ++j) {
    const uint8_t* blk = base + (size_t)j * BB;
    float x[NH][2][2];
    {
      // B = hi/lo(q * S_k): one fp16 product, or its rounding remainder
      uint32_t bq[NH][KS][2];
      const uint4* sp = reinterpret_cast<const uint4*>(blk + off_kscale(D, BITS) + tid * (D / 4) * 2);
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint4 s4 = sp[i];
        const uint32_t sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int u = 0; u < NH; ++u)
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int ks = 2 * i + (h >> 1), e2 = h & 1;
            const __half2 S2 = u2h(sv[h]);
            bq[u][ks][e2] = h2u(__hfma2(u2h(qr.qh[u][ks][e2]), S2,
                                        __hmul2(u2h(qr.qn[u][ks][e2]), S2)));
          }
      }
      uint32_t kw[WPL];
      {
        const uint4* p = reinterpret_cast<const uint4*>(blk);
#pragma unroll
        for (int i = 0; i < WPL / 4; ++i) {
          const uint4 w4 = p[i * 32 + lane];
          kw[4 * i] = w4.x; kw[4 * i + 1] = w4.y; kw[4 * i + 2] = w4.z; kw[4 * i + 3] = w4.w;
        }
      }
      float acc[NH][2][2][4];   // [u][mt][chain][C]: even / odd k-steps
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        const float bias = __shfl_sync(0xffffffffu, zb[u], j * 4 + tid);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[u][mt][0][e] = (e & 1) ? 0.f : bias;
            acc[u][mt][1][e] = 0.f;
          }
      }
      static_for<2>([&](auto MT_) {
        constexpr int MT = decltype(MT_)::value;
        static_for<KS>([&](auto KS_) {
          constexpr int K = decltype(KS_)::value;
          uint32_t a[4];
          key_afrag<D, BITS, MT, K, SEL>(kw, cm, a);
#pragma unroll
          for (int u = 0; u < NH; ++u)
            mma_f16(acc[u][MT][K & 1], a[0], a[1], a[2], a[3], bq[u][K][0], bq[u][K][1]);
        });
      });
#pragma unroll
      for (int u = 0; u < NH; ++u)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          x[u][mt][0] = (acc[u][mt][0][0] + acc[u][mt][0][1]) + (acc[u][mt][1][0] + acc[u][mt][1][1]);
          x[u][mt][1] = (acc[u][mt][0][2] + acc[u][mt][0][3]) + (acc[u][mt][1][2] + acc[u][mt][1][3]);
        }
    }
    softmax_update<D, GQ, 2, SEL>(st, x, sl2);

    // values: o[channel][n] += sum_t code[channel][t] * hi/lo(p_t S_t,gc)[t][n]
    uint32_t vw[WPL];
    {
      const uint4* p = reinterpret_cast<const uint4*>(blk + off_vcodes(D, BITS));
#pragma unroll
      for (int i = 0; i < WPL / 4; ++i) {
        const uint4 w4 = p[i * 32 + lane];
        vw[4 * i] = w4.x; vw[4 * i + 1] = w4.y; vw[4 * i + 2] = w4.z; vw[4 * i + 3] = w4.w;
      }
    }
    const uint32_t* vs = reinterpret_cast<const uint32_t*>(blk + off_vscale(D, BITS));
    const uint32_t* vz = reinterpret_cast<const uint32_t*>(blk + off_vzero(D, BITS));
    static_for<2>([&](auto KS_) {
      constexpr int K = decltype(KS_)::value;
      // scales of this lane's tokens (16K + gid, 16K + gid + 8) for every channel group
      uint32_t S2[NGC];
      if constexpr (NGC == 4) {
        const uint4 v4 = *reinterpret_cast<const uint4*>(vs + (K * 8 + gid) * NGC);
        S2[0] = v4.x; S2[1] = v4.y; S2[2] = v4.z; S2[3] = v4.w;
      } else {
        const uint2 v2 = *reinterpret_cast<const uint2*>(vs + (K * 8 + gid) * NGC);
        S2[0] = v2.x; S2[1] = v2.y;
      }
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        // p of the two tokens as fp16 pairs hi (ph) + lo (pl), p = ph + pl
        const float p0 = x[u][K][0], p1 = x[u][K][1];
        const __half2 ph = __floats2half2_rn(p0, p1);
        const float2 phf = __half22float2(ph);
        const __half2 pl = SEL ? __floats2half2_rn((p0 - phf.x) * lo_scale<SEL>(),
                                                   (p1 - phf.y) * lo_scale<SEL>())
                               : __floats2half2_rn(p0 - phf.x, p1 - phf.y);
        // zero-point term operand: (hi, lo) of p per token
        const uint32_t bz0 = movm_t(__byte_perm(h2u(ph), h2u(pl), 0x5410));
        const uint32_t bz1 = movm_t(__byte_perm(h2u(ph), h2u(pl), 0x7632));
        static_for<NGC>([&](auto GC_) {
          constexpr int GC = decltype(GC_)::value;
          const uint32_t z0 = vz[(8 * K + tid) * NGC + GC];
          const uint32_t z1 = vz[(8 * K + 4 + tid) * NGC + GC];
          // (hi, lo) of p * S: hi = fp16(ph S), lo = fp16(pl S + (ph S - hi)), the
          // remainder of the fp16 product exact through the fused multiply-add
          const __half2 s2 = u2h(S2[GC]);
          __half2 hi, lo;
          if constexpr (SEL) {   // in fp32: the scaled remainder of a large product fits no fp16 step
            const float2 sf = __half22float2(s2);
            const float w0 = p0 * sf.x, w1 = p1 * sf.y;
            hi = __floats2half2_rn(w0, w1);
            const float2 hf = __half22float2(hi);
            lo = __floats2half2_rn((w0 - hf.x) * lo_scale<SEL>(), (w1 - hf.y) * lo_scale<SEL>());
          } else {
            hi = __hmul2(ph, s2);
            lo = __hfma2(pl, s2, __hfma2(ph, s2, __hneg2(hi)));
          }
          const uint32_t b0 = movm_t(__byte_perm(h2u(hi), h2u(lo), 0x5410));
          const uint32_t b1 = movm_t(__byte_perm(h2u(hi), h2u(lo), 0x7632));
          if constexpr (SEL) {
            constexpr uint32_t mid = BITS == 4 ? 0x48004800u : 0x40004000u;   // 8 or 2, twice
            mma_f16(st.z[u][GC], z0, z0, z1, z1, bz0, bz1);
            mma_f16(st.z[u][GC], mid, mid, mid, mid, b0, b1);
          }
          static_for<2>([&](auto H_) {
            constexpr int MV = 2 * GC + decltype(H_)::value;
            uint32_t a[4];
            value_afrag<BITS, MV, K, SEL>(vw, cm, a);
            if constexpr (!SEL) mma_f16(st.o[u][MV], z0, z0, z1, z1, bz0, bz1);
            mma_f16(st.o[u][MV], a[0], a[1], a[2], a[3], b0, b1);
          });
        });
      }
    });
  }
}

// Packed groups of a launch over a range: as packed_warp over a list, but for
//  - sums of their own per group: a product whose accumulator starts at 0 is cut off at a step
//    of the group's size, not of all tokens' so far; the group's zero-point and mid-code sums are
//    what its value products start from (of one or two heads: fp32 sums apart), and the outputs take
//    the whole by fp32 additions (with accumulators over all groups 3e-5 of the output was lost over
//    2,880 tokens of a warp);
//  - codes of even channels (keys) and tokens (values) are taken from half a step below the middle of
//    their range, odd ones from half a step above: codes average the middle, so that both sums
//    stay small. (The tensor cores cut off towards 0: all of one sign, 6e-8 of the values were
//    lost throughout, 2e-6 of an output over 8,000 tokens);
//  - the key zero-points and mid-codes meet the queries in fp32, four (two) channels a lane: shorter
//    than products of which one row in eight is used;
//  - hidden tokens, and the parts of the groups' weights.
// What bounds it: 160 units of 32,768 tokens at 4 bits take 217 us (3.9 TB/s): 880 warp instructions a
// group, 317 of them the unpacking (HADD2, LOP3), at 0.56 a cycle and scheduler: three warps a
// scheduler, each a chain of dependent instructions, and neither registers nor the ring leave room for more.
// Four and eight heads have two warps a scheduler, at 0.34 to 0.40 instructions a cycle; eight heads at head
// dimension 128 also spill registers (330 to 480 B): 8 units of 32,768 tokens take 50 us at 2 bits and
// 48 at 4, where their bytes take 3.7 and 6.2.
template <int D, int BITS, int GQ, typename SL2>
__device__ void range_warp(WarpState<D, GQ, kDecRange>& st, const QRegs<D, GQ>& qr, const __nv_bfloat16* qs,
                           uint8_t* base, int n_grp, const SL2& sl2, const RangeChunk& ck) {
  constexpr int KS = D / 16, NGC = D / 32, BB = 8 * D * (BITS + 1), WPL = D * BITS / 32;
  constexpr int NH = n_tiles<GQ>(), CPL = D / 32;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const CodeMasks<BITS> cm = code_masks<BITS>();

  constexpr bool ONE = dec_groups_per_chunk(D, BITS) == 1;   // groups of a chunk
#pragma unroll 1
  for (int j = 0; ONE ? j < 1 : j < n_grp; ++j) {
    uint8_t* blk = base + (size_t)j * BB;
    // q . (Z + mid S) of head 4u + tid
    float zb[NH];
    {
      float w[CPL];
      const __half2* zp = reinterpret_cast<const __half2*>(blk + off_kzero(D, BITS)) + lane * (CPL / 2);
      const __half2* sp = reinterpret_cast<const __half2*>(blk + off_kscale(D, BITS)) + lane * (CPL / 2);
#pragma unroll
      for (int i = 0; i < CPL / 2; ++i) {
        const float2 z = __half22float2(zp[i]), c = __half22float2(sp[i]);
        w[2 * i] = fmaf((float)((1 << (BITS - 1)) - 1), c.x, z.x);
        w[2 * i + 1] = fmaf((float)(1 << (BITS - 1)), c.y, z.y);
      }
      // position kperm of the lane's first channel: channels c0, c0 + 1 and (D 128) c0 + 8, c0 + 9
      const int c0 = D == 128 ? 16 * (lane & 7) + 2 * (lane >> 3)
                              : 16 * ((lane & 7) >> 1) + 2 * (lane >> 3) + 8 * (lane & 1);
      float v[4 * NH];
#pragma unroll
      for (int h = 0; h < 4 * NH; ++h) {
        v[h] = 0.f;
        if (h < GQ) {
#pragma unroll
          for (int i = 0; i < CPL / 2; ++i) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(qs + h * D + c0 + 8 * i));
            v[h] = fmaf(f.x, w[2 * i], v[h]);
            v[h] = fmaf(f.y, w[2 * i + 1], v[h]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        float r;
        if constexpr (GQ == 1) {
          r = v[0];
          r += __shfl_xor_sync(0xffffffffu, r, 1);
          r += __shfl_xor_sync(0xffffffffu, r, 2);
        } else {
          // lane tid keeps head 4u + tid: halves exchanged over lanes 2 and 1 apart
          const bool up = tid & 2, odd = tid & 1;
          float a = up ? v[4 * u + 2] : v[4 * u], b = up ? v[4 * u + 3] : v[4 * u + 1];
          a += __shfl_xor_sync(0xffffffffu, up ? v[4 * u] : v[4 * u + 2], 2);
          b += __shfl_xor_sync(0xffffffffu, up ? v[4 * u + 1] : v[4 * u + 3], 2);
          r = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
        }
        r += __shfl_xor_sync(0xffffffffu, r, 4);
        r += __shfl_xor_sync(0xffffffffu, r, 8);
        r += __shfl_xor_sync(0xffffffffu, r, 16);
        zb[u] = r;
      }
    }
    float x[NH][2][2];
    {
      // B = hi/lo(q * S_k): one fp16 product, or its rounding remainder
      uint32_t bq[NH][KS][2];
      const uint4* sp = reinterpret_cast<const uint4*>(blk + off_kscale(D, BITS) + tid * (D / 4) * 2);
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint4 s4 = sp[i];
        const uint32_t sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int u = 0; u < NH; ++u)
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int ks = 2 * i + (h >> 1), e2 = h & 1;
            const __half2 S2 = u2h(sv[h]);
            bq[u][ks][e2] = h2u(__hfma2(u2h(qr.qh[u][ks][e2]), S2,
                                        __hmul2(u2h(qr.qn[u][ks][e2]), S2)));
          }
      }
      uint32_t kw[WPL];
      {
        const uint4* p = reinterpret_cast<const uint4*>(blk);
#pragma unroll
        for (int i = 0; i < WPL / 4; ++i) {
          const uint4 w4 = p[i * 32 + lane];
          kw[4 * i] = w4.x; kw[4 * i + 1] = w4.y; kw[4 * i + 2] = w4.z; kw[4 * i + 3] = w4.w;
        }
      }
      float acc[NH][2][2][4];   // [u][mt][chain][C]: even / odd k-steps
      static_for<2>([&](auto MT_) {
        constexpr int MT = decltype(MT_)::value;
        static_for<KS>([&](auto KS_) {
          constexpr int K = decltype(KS_)::value;
          uint32_t a[4];
          key_afrag<D, BITS, MT, K, 2>(kw, cm, a);
#pragma unroll
          for (int u = 0; u < NH; ++u) {
            if constexpr (K < 2)
              mma_f16_from(acc[u][MT][K], 0.f, 0.f, 0.f, 0.f, a[0], a[1], a[2], a[3], bq[u][K][0], bq[u][K][1]);
            else
              mma_f16(acc[u][MT][K & 1], a[0], a[1], a[2], a[3], bq[u][K][0], bq[u][K][1]);
          }
        });
      });
#pragma unroll
      for (int u = 0; u < NH; ++u)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          x[u][mt][0] = ((acc[u][mt][0][0] + acc[u][mt][0][1]) + (acc[u][mt][1][0] + acc[u][mt][1][1])) + zb[u];
          x[u][mt][1] = ((acc[u][mt][0][2] + acc[u][mt][0][3]) + (acc[u][mt][1][2] + acc[u][mt][1][3])) + zb[u];
        }
    }
    const Seen seen = ck.seen(j);
    if (!seen.all(KVC_GROUP)) {
      // Hidden tokens: weight 0, and scales and zero-points of their values 0 as well (they may
      // not be finite). One token per lane.
#pragma unroll
      for (int u = 0; u < NH; ++u)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (!seen.at(16 * mt + gid + 8 * r)) x[u][mt][r] = -INFINITY;
      if (!seen.at(lane)) {
        __half* hs = reinterpret_cast<__half*>(blk + off_vscale(D, BITS));
        __half* hz = reinterpret_cast<__half*>(blk + off_vzero(D, BITS));
#pragma unroll
        for (int gc = 0; gc < NGC; ++gc) {
          hs[vs_index(lane, gc, NGC)] = __ushort_as_half(0);
          hz[vsz_index(lane, gc, NGC)] = __ushort_as_half(0);
        }
      }
      __syncwarp();
    }
    softmax_update<D, GQ, 2, true>(st, x, sl2);
    if (ck.part) put_part<GQ, 2>(st.m, x, sl2, ck.part + (size_t)(j == 0 ? ck.slot[0] : ck.slot[1]) * GQ);

    // values: sum_t Z_t p_t + sum_t (mid + (code - mid)) S_t p_t, p and S p as hi/lo pairs
    uint32_t vw[WPL];
    {
      const uint4* p = reinterpret_cast<const uint4*>(blk + off_vcodes(D, BITS));
#pragma unroll
      for (int i = 0; i < WPL / 4; ++i) {
        const uint4 w4 = p[i * 32 + lane];
        vw[4 * i] = w4.x; vw[4 * i + 1] = w4.y; vw[4 * i + 2] = w4.z; vw[4 * i + 3] = w4.w;
      }
    }
    // scales of this lane's tokens (16K + gid, 16K + gid + 8), zero-points of token pairs (8K + tid,
    // 8K + 4 + tid), for every channel group
    uint32_t S2[2][NGC];
    auto words = [&](uint32_t (&to)[NGC], int off, int row) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(blk + off) + row * NGC;
      if constexpr (NGC == 4) {
        const uint4 v4 = *reinterpret_cast<const uint4*>(p);
        to[0] = v4.x; to[1] = v4.y; to[2] = v4.z; to[3] = v4.w;
      } else {
        const uint2 v2 = *reinterpret_cast<const uint2*>(p);
        to[0] = v2.x; to[1] = v2.y;
      }
    };
#pragma unroll
    for (int K = 0; K < 2; ++K) words(S2[K], off_vscale(D, BITS), K * 8 + gid);
    constexpr int MIDC = 1 << (BITS - 1);
    if constexpr (GQ <= 2) {
      // Zero-points and mid-codes in fp32, lane (gid, tid) those of channel group tid % NGC and the
      // tokens 16K + gid + 8r (D 64: r = tid / 2 alone), whose weights lane (gid, head) holds. (By
      // products of which every row is the same, a third of all, 160 units of 32,768 tokens took 261 us,
      // and 226 this way; with more heads the exchange of weights costs what the products do.)
      const __half* vz = reinterpret_cast<const __half*>(blk + off_vzero(D, BITS));
      const int gc = tid % NGC;
#pragma unroll
      for (int K = 0; K < 2; ++K)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float p[GQ];
#pragma unroll
          for (int h = 0; h < GQ; ++h) p[h] = __shfl_sync(0xffffffffu, x[0][K][r], (lane & ~3) + h);
          if (NGC == 2 && r != tid >> 1) continue;
          const int t = 16 * K + gid + 8 * r;
          const uint32_t sw = *(reinterpret_cast<const uint32_t*>(blk + off_vscale(D, BITS)) + (K * 8 + gid) * NGC + gc);
          const float sc = r ? __high2float(u2h(sw)) : __low2float(u2h(sw));
          const float z = fmaf(sc, (float)(MIDC - 1 + (gid & 1)), __half2float(vz[vsz_index(t, gc, NGC)]));
#pragma unroll
          for (int h = 0; h < GQ; ++h) st.zp[h] = fmaf(p[h], z, st.zp[h]);
        }
    }
    const float2 big = make_float2(lo_scale<true>(), lo_scale<true>());
    const float2 neg = make_float2(-lo_scale<true>(), -lo_scale<true>());
#pragma unroll
    for (int u = 0; u < NH; ++u) {
      uint32_t bz[2][2], Z2[2][2][NGC];
      float2 pw[2];
#pragma unroll
      for (int K = 0; K < 2; ++K) {
        pw[K] = make_float2(x[u][K][0], x[u][K][1]);
        if constexpr (GQ > 2) {
          words(Z2[K][0], off_vzero(D, BITS), 8 * K + tid);
          words(Z2[K][1], off_vzero(D, BITS), 8 * K + 4 + tid);
          const __half2 ph = __float22half2_rn(pw[K]);
          const __half2 pl = __float22half2_rn(__ffma2_rn(__half22float2(ph), neg, __fmul2_rn(pw[K], big)));
          bz[K][0] = movm_t(__byte_perm(h2u(ph), h2u(pl), 0x5410));
          bz[K][1] = movm_t(__byte_perm(h2u(ph), h2u(pl), 0x7632));
        }
      }
      static_for<NGC>([&](auto GC_) {
        constexpr int GC = decltype(GC_)::value;
        uint32_t b[2][2];
        float cz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int K = 0; K < 2; ++K) {
          const float2 w = __fmul2_rn(pw[K], __half22float2(u2h(S2[K][GC])));
          const __half2 hi = __float22half2_rn(w);
          const __half2 lo = __float22half2_rn(__ffma2_rn(__half22float2(hi), neg, __fmul2_rn(w, big)));
          b[K][0] = movm_t(__byte_perm(h2u(hi), h2u(lo), 0x5410));
          b[K][1] = movm_t(__byte_perm(h2u(hi), h2u(lo), 0x7632));
          if constexpr (GQ > 2) {
            // (a product holds both terms of eight tokens: they cancel before the sum is cut off)
            constexpr uint32_t mid = BITS == 4 ? 0x48004700u : 0x40003c00u;   // 7 and 8, or 1 and 2
            if (K == 0)
              mma_f16_from(cz, 0.f, 0.f, 0.f, 0.f, Z2[K][0][GC], Z2[K][0][GC], mid, mid, bz[K][0], b[K][0]);
            else
              mma_f16(cz, Z2[K][0][GC], Z2[K][0][GC], mid, mid, bz[K][0], b[K][0]);
            mma_f16(cz, Z2[K][1][GC], Z2[K][1][GC], mid, mid, bz[K][1], b[K][1]);
          }
        }
        static_for<2>([&](auto H_) {
          constexpr int MV = 2 * GC + decltype(H_)::value;
          float c[4];
          uint32_t a[4];
          value_afrag<BITS, MV, 0, 2>(vw, cm, a);
          mma_f16_from(c, cz[0], cz[1], cz[2], cz[3], a[0], a[1], a[2], a[3], b[0][0], b[0][1]);
          value_afrag<BITS, MV, 1, 2>(vw, cm, a);
          mma_f16(c, a[0], a[1], a[2], a[3], b[1][0], b[1][1]);
          float2* o = reinterpret_cast<float2*>(st.o[u][MV]);
          o[0] = __fadd2_rn(o[0], make_float2(c[0], c[1]));
          o[1] = __fadd2_rn(o[1], make_float2(c[2], c[3]));
        });
      });
    }
  }
}

// ------------------------------------------------------------- window slots
// wk: 16 staged key rows (win_k_index layout, first slot a multiple of 16); wv: 8
// staged value pair rows (win_v_index layout); the first n_valid slots are live.
// bf16 products, exact queries, hi/lo weights.
template <int D, int GQ, bool SEL, int MODE, typename SL2, typename Chunk>
__device__ void window_warp(WarpState<D, GQ, MODE>& st, const __nv_bfloat16* qs, const __nv_bfloat16* wk,
                            const uint32_t* wv, int n_valid, const SL2& sl2, const Chunk& ck) {
  constexpr int KS = D / 16, NH = n_tiles<GQ>();
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  float x[NH][1][2];
  {
    uint32_t bq[NH][KS][2];
#pragma unroll
    for (int u = 0; u < NH; ++u) {
      const int h = 4 * u + (gid >> 1);
      const bool live = h < GQ && !(gid & 1);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2)
          bq[u][ks][e2] = live ? *reinterpret_cast<const uint32_t*>(qs + h * D + 16 * ks + 2 * tid + 8 * e2)
                               : 0u;
    }
    float acc[NH][2][4];
#pragma unroll
    for (int u = 0; u < NH; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) { acc[u][0][e] = 0.f; acc[u][1][e] = 0.f; }
    // rows gid (rl 0) and gid + 8 (rl 1); 16-byte chunks swizzled by gid
    const uint4* r0 = reinterpret_cast<const uint4*>(wk + (size_t)gid * D);
    const uint4* r1 = reinterpret_cast<const uint4*>(wk + (size_t)(gid + 8) * D);
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {
      const int ch = (tid * (KS / 2) + i) ^ gid;
      const uint4 u0 = r0[ch], u1 = r1[ch];
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        mma_bf16(acc[u][0], u0.x, u1.x, u0.y, u1.y, bq[u][2 * i][0], bq[u][2 * i][1]);
        mma_bf16(acc[u][1], u0.z, u1.z, u0.w, u1.w, bq[u][2 * i + 1][0], bq[u][2 * i + 1][1]);
      }
    }
#pragma unroll
    for (int u = 0; u < NH; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float v = (acc[u][0][2 * r] + acc[u][0][2 * r + 1]) +
                        (acc[u][1][2 * r] + acc[u][1][2 * r + 1]);
        bool live = (gid + 8 * r) < n_valid;
        if constexpr (Chunk::kRange) live = live && ck.seen(0).at(gid + 8 * r);
        x[u][0][r] = live ? v : -INFINITY;
      }
  }
  softmax_update<D, GQ, 1, SEL>(st, x, sl2);
  if constexpr (Chunk::kRange) {
    if (ck.part) put_part<GQ, 1>(st.m, x, sl2, ck.part + (size_t)ck.slot[0] * GQ);
  }
  uint32_t b0[NH], b1[NH], c0[SEL ? NH : 1], c1[SEL ? NH : 1];
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    b0[u] = movm_t(split_bf16<SEL>(x[u][0][0]));
    b1[u] = movm_t(split_bf16<SEL>(x[u][0][1]));
    if constexpr (SEL) {
      c0[u] = movm_t(split_rest(x[u][0][0]));
      c1[u] = movm_t(split_rest(x[u][0][1]));
    }
  }
  // pair rows tid (tokens 2tid, 2tid + 1) and 4 + tid (tokens 8 + 2tid, +1); chunks
  // swizzled by tid
  const uint4* p0 = reinterpret_cast<const uint4*>(wv + (size_t)tid * D);
  const uint4* p1 = reinterpret_cast<const uint4*>(wv + (size_t)(4 + tid) * D);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int ch = (gid * (D / 32) + i) ^ tid;
    const uint4 v0 = p0[ch], v1 = p1[ch];
    // words: (mt = 2i, rl 0), (2i, rl 1), (2i + 1, rl 0), (2i + 1, rl 1)
#pragma unroll
    for (int u = 0; u < NH; ++u) {
      mma_bf16(st.o[u][2 * i], v0.x, v0.y, v1.x, v1.y, b0[u], b1[u]);
      mma_bf16(st.o[u][2 * i + 1], v0.z, v0.w, v1.z, v1.w, b0[u], b1[u]);
      if constexpr (SEL) {
        mma_bf16(st.o[u][2 * i], v0.x, v0.y, v1.x, v1.y, c0[u], c1[u]);
        mma_bf16(st.o[u][2 * i + 1], v0.z, v0.w, v1.z, v1.w, c0[u], c1[u]);
      }
    }
  }
}

// ------------------------------------------------------------ launch layout
struct DecLayer {
  long long chunk_begin;  // first chunk of the layer in the launch's chunk list
  long long packed_off;   // byte offset of the layer inside the packed store
  long long win_off;      // element offset of the layer's window rings
  int n_groups;           // packed groups read (a group flushed in this step included)
  int win_start;          // ring start slot after this launch's append
  int win_len;            // window tokens after this launch's append
  int cap_groups;
  int new_slot;           // ring slot of the token appended in this launch, or -1
  int wchunks;            // window chunks (16 slots) per unit; packed chunks follow
  int pchunks;            // packed chunks per unit
  int gpc;                // packed groups per chunk
  int R;                  // ring length
  int bits;               // 2, 4 or 16 (16: no packed chunks)
};

struct DecParams {
  DecLayer L[KVC_MAX_LAUNCH_LAYERS];
  const int32_t* groups;        // [n_layers][units][n_select] packed groups to read (SEL only)
  int n_select;                 // list entries per unit (SEL only)
  const __nv_bfloat16* k_new;   // [n_layers][units][D] (fused append only)
  const __nv_bfloat16* v_new;
  const unsigned* wide;         // the cache's marks [layer][unit][4] (SEL only)
  unsigned* err;                // device error word (bit 0: a staging wait gave up)
  float* ws;                    // partial states, two per CTA: [2 * grid][dep_floats]
  unsigned* cnt;                // arrival tickets per (layer, unit) of the cache; zero between launches
  long long total;              // chunks in the launch
  int n_vwarps;                 // warps of the grid
  int n_layers;                 // layers in this launch
  int layer_begin;              // absolute index of L[0]
  int units;                    // batch * n_kv_heads
  unsigned wait_limit;          // polls of one staging wait before it gives up
  float sl2;                    // log2(e) / sqrt(head_dim)
};

// What a launch over a range reads of a layer, and where its parts begin.
struct RangeLayer {
  int a, b;               // tokens before a and from b on (in storage order: packed groups, window)
  int w_first, w_skip;    // window chunk j is chunk j, or, from w_first on, j + w_skip
  int g_first, g_skip;    // the same for packed groups
  int g_count;            // packed groups read
  int parts;              // parts of a unit: packed groups, then window chunks
  long long part_begin;   // first part of the layer, in parts
};
struct RangeParams : DecParams {
  RangeLayer R[KVC_MAX_LAUNCH_LAYERS];
  float2* part;           // [layer][unit][parts][GQ], or null
  float2* stat;           // [layer][unit][GQ]: maximum (log2 units) and sum of the unit's weights
  const float* before;    // [layer][unit][n_slots], or null: weights are formed by another launch
  float* after;
  int n_slots;
};

// G float2 (a part, or a unit's maxima and sums), all loads in flight at once.
template <int G>
__device__ __forceinline__ void load_pairs(float2 (&v)[G], const float2* p) {
  if constexpr (G == 1) {
    v[0] = __ldcg(p);
  } else {
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(p) + i);
      v[2 * i] = make_float2(q.x, q.y);
      v[2 * i + 1] = make_float2(q.z, q.w);
    }
  }
}
// What the tokens of a slot received: the packed group of that index, or two window chunks. part: the
// unit's parts, stat: its maxima and sums (a sum of 0: some parts were not written, nothing is received).
template <int G>
__device__ __forceinline__ float slot_weight(const float2* part, const float2 (&stat)[G], int slot,
                                             int n_groups, int parts) {
  int p0 = slot, p1 = slot + 1;
  if (slot >= n_groups) {
    p0 = (int)min((long long)parts, n_groups + 2LL * (slot - n_groups));
    p1 = min(p0 + 2, parts);
  }
  float2 a[2][G];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int h = 0; h < G; ++h) a[i][h] = make_float2(0.f, 0.f);
    if (p0 + i < p1) load_pairs(a[i], part + (size_t)(p0 + i) * G);
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < G; ++h)
      if (a[i][h].y != 0.f && stat[h].y != 0.f) sum += a[i][h].y * exp2f(a[i][h].x - stat[h].x) / stat[h].y;
  return sum;
}
// A unit's weights by one warp (out of line: the launch's ordinary path has no instructions to spare
// for it).
template <int G>
__device__ __noinline__ void unit_weights(const float2* part, const float2* stat, const float* before,
                                          float* after, int n_slots, int n_groups, int parts) {
  __syncwarp();
  float2 ms[G];
  load_pairs(ms, stat);
  for (int s = threadIdx.x & 31; s < n_slots; s += 32)
    after[s] = before[s] + slot_weight(part, ms, s, n_groups, parts);
}
template <int MODE>
using ParamsOf = std::conditional_t<MODE == kDecRange, RangeParams, DecParams>;

// One partial state in the workspace: o[GQ][D] (unnormalised; both column parts
// and the value zero-point sums folded in), then m[GQ] (log2 units) and l[GQ],
// padded to a whole number of 16-byte vectors so that every o starts aligned.
__host__ __device__ constexpr int dep_floats(int D, int GQ) { return GQ * D + (2 * GQ + 3) / 4 * 4; }

constexpr int kMaxGpc = 2;   // packed groups per chunk, at most
static_assert(dec_groups_per_chunk(64, 2) <= kMaxGpc && dec_groups_per_chunk(128, 2) <= kMaxGpc &&
              dec_groups_per_chunk(64, 4) <= kMaxGpc && dec_groups_per_chunk(128, 4) <= kMaxGpc,
              "a chunk's list entries");

// BMASK: bit 0 = the launch has 2-bit layers, bit 1 = 4-bit layers (the packed
// code of each present precision is instantiated; 16-bit layers need neither).
// SEL: a unit's marks and factors lie behind its queries.
template <int D, int GQ, int BMASK, bool SEL>
struct DecCfg {
  static constexpr int WB = kSlotsPerWarp * D * 4;   // one window chunk (keys + values)
  static constexpr int PB2 = (BMASK & 1) ? dec_groups_per_chunk(D, 2) * block_bytes(D, 2) : 0;
  static constexpr int PB4 = (BMASK & 2) ? dec_groups_per_chunk(D, 4) * block_bytes(D, 4) : 0;
  static constexpr int SLOT = WB > PB2 ? (WB > PB4 ? WB : PB4) : (PB2 > PB4 ? PB2 : PB4);
  static constexpr int QB = GQ * D * 2;              // one unit's queries (bf16)
  static constexpr int QS = QB + (SEL ? 48 : 0);     // their buffer
  static constexpr int DEPW = dep_floats(D, GQ);     // floats of one partial state
  static constexpr int per_warp = 2 * SLOT + 2 * QS + 2 * DEPW * 4 + 2 * 8 + 4;
  // warps per CTA: as many as shared memory holds, at most 12 (8 with four or more
  // query heads, whose state needs more registers per thread than 12 warps leave)
  static constexpr int pick(int nw) { return nw * per_warp <= 227 * 1024 ? nw : pick(nw - 1); }
  static constexpr int NW = pick(GQ > 2 ? 8 : 12);
  static constexpr int kThreads = NW * 32;
  static constexpr int oRing = 0;                    // [NW][2][SLOT]
  static constexpr int oDep = oRing + NW * 2 * SLOT; // [NW][2][DEPW] fp32 partial states
  static constexpr int oQ = oDep + NW * 2 * DEPW * 4;// [NW][2][QS]: [GQ][D] bf16 first
  static constexpr int oBars = oQ + NW * 2 * QS;     // [NW][2] mbarriers
  static constexpr int oCnt = oBars + NW * 2 * 8;    // [NW] arrival tickets
  static constexpr int total = oCnt + NW * 4;
  static_assert(SLOT % 16 == 0 && QB % 16 == 0 && oDep % 16 == 0 && oBars % 8 == 0, "alignment");
  static_assert(NW >= 4, "at least four warps per CTA");
};

// A range, one or two heads: head tid's zero-point and mid-code sums of every channel group.
template <int D, int GQ, int MODE>
__device__ __forceinline__ void zp_groups(WarpState<D, GQ, MODE>& st, float (&zg)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) zg[i] = 0.f;
  if constexpr (WarpState<D, GQ, MODE>::kZp) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < GQ; ++h) {
      float z = st.zp[h];
      z += __shfl_xor_sync(0xffffffffu, z, 4);
      z += __shfl_xor_sync(0xffffffffu, z, 8);
      z += __shfl_xor_sync(0xffffffffu, z, 16);
      if constexpr (D == 64) z += __shfl_xor_sync(0xffffffffu, z, 2);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const float v = __shfl_sync(0xffffffffu, z, (lane & 28) + i);
        if ((lane & 3) == h) zg[i] = v;
      }
    }
  }
}

// Output e of fragment mt: both column parts (and, over a list, the channel group's zero-point sums).
template <int D, int GQ, bool SEL, int MODE>
__device__ __forceinline__ float join_parts(const WarpState<D, GQ, MODE>& st, int u, int mt, int e) {
  const float hi = st.o[u][mt][e], lo = st.o[u][mt][e + 1];
  if constexpr (MODE == kDecRange)
    return fmaf(lo, 1.f / lo_scale<SEL>(), hi);
  else if constexpr (SEL)
    return fmaf(lo + st.z[u][mt / 2][e + 1], 1.f / lo_scale<SEL>(), hi + st.z[u][mt / 2][e]);
  else
    return hi + lo;
}

template <int D, int GQ, bool SEL, int MODE, typename SL2>
__device__ void write_partial(WarpState<D, GQ, MODE>& st, float* dep, const SL2& sl2) {
  constexpr int NH = n_tiles<GQ>();
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  [[maybe_unused]] float zg[D / 32];
  if constexpr (WarpState<D, GQ, MODE>::kZp) zp_groups(st, zg);
  auto join = [&](int u, int mt, int e) {
    const float v = join_parts<D, GQ, SEL>(st, u, mt, e);
    if constexpr (WarpState<D, GQ, MODE>::kZp) return v + zg[mt / 2];
    else return v;
  };
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    const int h = 4 * u + tid;
    float l = st.l[u];
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (h < GQ) {
      float* o = dep + h * D;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        o[16 * mt + gid] = join(u, mt, 0);
        o[16 * mt + gid + 8] = join(u, mt, 2);
      }
      if (gid == 0) {
        dep[GQ * D + h] = st.m[u] == -INFINITY ? -INFINITY : st.m[u] * sl2_of(sl2, u);
        dep[GQ * D + GQ + h] = l;
      }
    }
  }
}

// The warp's state normalised (o / l per head) into out[GQ][D]; STAT: its maxima (log2 units) and
// sums into stat[GQ] (if given).
template <int D, int GQ, bool SEL, bool STAT, int MODE, typename SL2>
__device__ void write_final(WarpState<D, GQ, MODE>& st, float* __restrict__ out, const SL2& sl2,
                            float2* stat) {
  constexpr int NH = n_tiles<GQ>();
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  [[maybe_unused]] float zg[D / 32];
  if constexpr (WarpState<D, GQ, MODE>::kZp) zp_groups(st, zg);
  auto join = [&](int u, int mt, int e) {
    const float v = join_parts<D, GQ, SEL>(st, u, mt, e);
    if constexpr (WarpState<D, GQ, MODE>::kZp) return v + zg[mt / 2];
    else return v;
  };
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    const int h = 4 * u + tid;
    float l = st.l[u];
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    if constexpr (STAT) {
      if (stat && h < GQ && gid == 0)
        __stcg(stat + h, make_float2(st.m[u] == -INFINITY ? -INFINITY : st.m[u] * sl2_of(sl2, u), l));
    }
    if (h < GQ) {
      float* o = out + h * D;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        o[16 * mt + gid] = join(u, mt, 0) * inv;
        o[16 * mt + gid + 8] = join(u, mt, 2) * inv;
      }
    }
  }
}

template <bool GLOBAL>
__device__ __forceinline__ float ld_dep(const float* p) {
  if constexpr (GLOBAL) return __ldcg(p);
  else return *p;
}
template <bool GLOBAL>
__device__ __forceinline__ float4 ld_dep4(const float4* p) {
  if constexpr (GLOBAL) return __ldcg(p);
  else return *p;
}

// Log-sum-exp combine of the partial states dep_of(0 .. nc-1), in that order (the
// result does not depend on which holder arrived last). GLOBAL: the partials were
// written by other SMs and are read through L2; else they are in this CTA's
// shared memory. NORMALISE: out[GQ][D] = o / l; else out is written as one
// partial state (o, m, l) of the whole set. The maxima and weights are taken with
// the lanes spread over the contributors; the outputs then loop over the
// contributors with loads that do not depend on each other.
template <int D, int GQ, bool GLOBAL, bool NORMALISE, bool STAT, typename DepOf>
__device__ void merge_partials(int nc, DepOf dep_of, float* __restrict__ out, float2* stat) {
  constexpr int N4 = GQ * D / 4;            // float4 outputs
  constexpr int E4 = (N4 + 31) / 32;        // per lane
  const int lane = threadIdx.x & 31;
  float M[GQ];
#pragma unroll
  for (int h = 0; h < GQ; ++h) M[h] = -INFINITY;
  for (int w0 = 0; w0 < nc; w0 += 32) {
    if (w0 + lane < nc) {
      const float* d = dep_of(w0 + lane) + GQ * D;
#pragma unroll
      for (int h = 0; h < GQ; ++h)
        if (ld_dep<GLOBAL>(d + GQ + h) > 0.f) M[h] = fmaxf(M[h], ld_dep<GLOBAL>(d + h));
    }
  }
#pragma unroll
  for (int h = 0; h < GQ; ++h)
#pragma unroll
    for (int o = 16; o; o >>= 1) M[h] = fmaxf(M[h], __shfl_xor_sync(0xffffffffu, M[h], o));
  float4 acc[E4];
  float L[GQ];
#pragma unroll
  for (int i = 0; i < E4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int h = 0; h < GQ; ++h) L[h] = 0.f;
  // lane element i covers outputs 4 (lane + 32 i) .. + 3 (one head)
  for (int w0 = 0; w0 < nc; w0 += 32) {
    float f[GQ];
    if (w0 + lane < nc) {
      const float* d = dep_of(w0 + lane) + GQ * D;
#pragma unroll
      for (int h = 0; h < GQ; ++h) {
        const float l = ld_dep<GLOBAL>(d + GQ + h);
        f[h] = l > 0.f ? exp2f(ld_dep<GLOBAL>(d + h) - M[h]) : 0.f;
        L[h] += f[h] * l;
      }
    } else {
#pragma unroll
      for (int h = 0; h < GQ; ++h) f[h] = 0.f;
    }
    const int cnt = min(32, nc - w0);
#pragma unroll 4
    for (int k = 0; k < cnt; ++k) {
      const float4* o4 = reinterpret_cast<const float4*>(dep_of(w0 + k));
      float fk[GQ];
#pragma unroll
      for (int h = 0; h < GQ; ++h) fk[h] = __shfl_sync(0xffffffffu, f[h], k);
#pragma unroll
      for (int i = 0; i < E4; ++i) {
        const int idx = lane + 32 * i;
        if (idx < N4) {
          const float4 v = ld_dep4<GLOBAL>(o4 + idx);
          const float fh = fk[(4 * idx) / D];
          acc[i].x += fh * v.x; acc[i].y += fh * v.y; acc[i].z += fh * v.z; acc[i].w += fh * v.w;
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < GQ; ++h)
#pragma unroll
    for (int o = 16; o; o >>= 1) L[h] += __shfl_xor_sync(0xffffffffu, L[h], o);
  float4* out4 = reinterpret_cast<float4*>(out);
#pragma unroll
  for (int i = 0; i < E4; ++i) {
    const int idx = lane + 32 * i;
    if (idx < N4) {
      float inv = 1.f;
      if constexpr (NORMALISE) {
        const int h = (4 * idx) / D;
        inv = L[h] > 0.f ? 1.f / L[h] : 0.f;
      }
      out4[idx] = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
    }
  }
  if constexpr (!NORMALISE || STAT) {
    if (lane < GQ) {
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int h = 0; h < GQ; ++h)
        if (h == lane) { m = M[h]; l = L[h]; }
      if constexpr (!NORMALISE) {
        out[GQ * D + lane] = m;
        out[GQ * D + GQ + lane] = l;
      } else if (stat) {
        __stcg(stat + lane, make_float2(m, l));
      }
    }
  }
}

__device__ __forceinline__ void mbar_init(uint64_t* bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
               :: "r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// An even split of [base, base + T) into N contiguous ranges: range i is
// [first(i), first(i+1)), and owner(c) is the range holding c. When T * N < 2^32
// (every launch of ordinary size) all products fit 32 bits: 32-bit divisions.
struct Split {
  long long T, N, base;
  __device__ long long first(long long i) const {
    if (T * N < (1LL << 32)) return base + (long long)((unsigned)i * (unsigned)T / (unsigned)N);
    return base + i * T / N;
  }
  __device__ long long owner(long long c) const {
    const long long x = c - base;
    if (T * N < (1LL << 32))
      return (long long)((((unsigned)x + 1u) * (unsigned)N - 1u) / (unsigned)T);
    return ((x + 1) * N - 1) / T;
  }
};

// kDecList: the packed chunks of a unit are the entries of its list in P.groups (an entry
// outside [0, n_groups) is skipped) in place of its first groups. kDecRange: they and the window
// chunks are those of P.R.
template <int D, int GQ, int BMASK, int MODE>
__global__ void __launch_bounds__(DecCfg<D, GQ, BMASK, MODE != kDecAll>::kThreads, 1)
decode_kernel(const ParamsOf<MODE> P, uint8_t* __restrict__ packed, __nv_bfloat16* __restrict__ win_k,
              __nv_bfloat16* __restrict__ win_v, const __nv_bfloat16* __restrict__ q,
              float* __restrict__ out) {
  constexpr bool SEL = MODE != kDecAll, LIST = MODE == kDecList, RANGE = MODE == kDecRange;
  using C = DecCfg<D, GQ, BMASK, SEL>;
  constexpr int NW = C::NW;
  extern __shared__ __align__(128) uint8_t dsm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* bar = reinterpret_cast<uint64_t*>(dsm + C::oBars) + warp * 2;
  uint8_t* ring = dsm + C::oRing + (size_t)warp * 2 * C::SLOT;
  float* sdep = reinterpret_cast<float*>(dsm + C::oDep);           // [NW][2][DEPW]
  unsigned* scnt = reinterpret_cast<unsigned*>(dsm + C::oCnt);     // [NW]
  __nv_bfloat16* qbuf = reinterpret_cast<__nv_bfloat16*>(dsm + C::oQ) + (size_t)warp * C::QS;
  if (lane == 0) {
    mbar_init(&bar[0]);
    mbar_init(&bar[1]);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    scnt[warp] = 0u;
  }
  __syncthreads();
  pdl_wait();      // the previous kernels' writes (queries, cache) are visible
  pdl_release();
  // the launch's chunk list, cut into one contiguous range per CTA, each cut into one
  // contiguous range per warp
  const Split cs{P.total, (long long)gridDim.x, 0};
  const long long C0 = cs.first(blockIdx.x), C1 = cs.first(blockIdx.x + 1);
  const int nvw = (int)(C1 - C0 < NW ? C1 - C0 : NW);   // warps with chunks (>= 1: grid <= total)
  if (warp >= nvw) return;
  const Split ws{C1 - C0, (long long)nvw, C0};
  const long long c0 = ws.first(warp), c1 = ws.first(warp + 1);
  const int n = (int)(c1 - c0);   // >= 1

  // chunk cursor: layer, unit, chunk index j inside the unit, chunks per unit
  struct Cur { int li, unit, j, cpu; };
  auto cpu_of = [&](int li) { return P.L[li].wchunks + P.L[li].pchunks; };
  auto locate = [&](long long c) {
    Cur r;
    r.li = 0;
    while (r.li + 1 < P.n_layers && c >= P.L[r.li + 1].chunk_begin) ++r.li;
    r.cpu = cpu_of(r.li);
    const long long loc = c - P.L[r.li].chunk_begin;
    r.unit = SEL && !(loc >> 32) ? (int)((unsigned)loc / (unsigned)r.cpu) : (int)(loc / r.cpu);
    r.j = (int)(loc - (long long)r.unit * r.cpu);
    return r;
  };
  auto step = [&](Cur& r) {
    if (++r.j < r.cpu) return;
    r.j = 0;
    if (++r.unit < P.units) return;
    r.unit = 0;
    do { ++r.li; } while (r.li < P.n_layers && cpu_of(r.li) == 0);
    r.cpu = r.li < P.n_layers ? cpu_of(r.li) : 1;
  };
  // LIST: the valid list entries of packed chunk r, moved to the front of id; their count
  auto listed_groups = [&](const Cur& r, int (&id)[kMaxGpc]) {
    const DecLayer& L = P.L[r.li];
    const int g0 = (r.j - L.wchunks) * L.gpc;
    const int32_t* list = P.groups + ((size_t)r.li * P.units + r.unit) * P.n_select + g0;
    int v[kMaxGpc];
#pragma unroll
    for (int k = 0; k < kMaxGpc; ++k) v[k] = k < L.gpc && g0 + k < P.n_select ? list[k] : -1;
    int ng = 0;
#pragma unroll
    for (int k = 0; k < kMaxGpc; ++k)
      if (v[k] >= 0 && v[k] < L.n_groups) {
        if (ng == 0) id[0] = v[k];
        else id[kMaxGpc - 1] = v[k];
        ++ng;
      }
    return ng;
  };
  // The list entries of the warp's first 32 chunks, chunk i's in lane i: read at once, where
  // each chunk's would wait for memory before its copy (and once more before its use).
  int first_id[kMaxGpc] = {}, first_ng = 0;
  if constexpr (LIST) {
    if (lane < n) {
      const Cur r = locate(c0 + lane);
      if (r.j >= P.L[r.li].wchunks) first_ng = listed_groups(r, first_id);
    }
    __syncwarp();
  }
  // chunk i's groups (cursor r), the same in every lane
  auto groups_of = [&](int i, const Cur& r, int (&id)[kMaxGpc]) {
    if constexpr (RANGE) {
      const DecLayer& L = P.L[r.li];
      const RangeLayer& X = P.R[r.li];
      const int g0 = (r.j - L.wchunks) * L.gpc;
#pragma unroll
      for (int k = 0; k < kMaxGpc; ++k) id[k] = g0 + k < X.g_first ? g0 + k : g0 + k + X.g_skip;
      return min(L.gpc, X.g_count - g0);
    }
    if (i >= 32) return listed_groups(r, id);
#pragma unroll
    for (int k = 0; k < kMaxGpc; ++k) id[k] = __shfl_sync(0xffffffffu, first_id[k], i);
    return __shfl_sync(0xffffffffu, first_ng, i);
  };
  // lane 0: stage chunk i (cursor r) into slot i & 1, with the unit's queries into
  // qbuf[qpar] when the chunk starts one of the warp's unit segments
  auto issue = [&](int i, const Cur& r, int qpar, bool with_q, int ngl, const int (&id)[kMaxGpc]) {
    const DecLayer& L = P.L[r.li];
    uint64_t* b = &bar[i & 1];
    uint8_t* dst = ring + (i & 1) * C::SLOT;
    const uint32_t qb = with_q ? (uint32_t)(C::QB + (SEL ? 16 : 0)) : 0u;
    if (r.j < L.wchunks) {
      const size_t rb = (size_t)L.win_off + (size_t)r.unit * L.R * D;
      int jw = r.j;
      if constexpr (RANGE) jw += r.j < P.R[r.li].w_first ? 0 : P.R[r.li].w_skip;
      const int slot0 = (L.win_start + jw * kSlotsPerWarp) % L.R;
      const uint32_t wb = (uint32_t)(kSlotsPerWarp * D * 2);
      mbar_expect(b, 2 * wb + qb);
      bulk_g2s(dst, win_k + rb + (size_t)slot0 * D, wb, b);
      bulk_g2s(dst + wb, win_v + rb + (size_t)(slot0 >> 1) * D * 2, wb, b);
    } else {
      const int bb = block_bytes(D, L.bits);
      const int g0 = (r.j - L.wchunks) * L.gpc;
      const uint8_t* src = packed + L.packed_off + (size_t)r.unit * L.cap_groups * bb;
      if constexpr (SEL) {
        mbar_expect(b, (uint32_t)(ngl * bb) + qb);
#pragma unroll
        for (int k = 0; k < kMaxGpc; ++k)
          if (k < ngl) bulk_g2s(dst + k * bb, src + (size_t)id[k] * bb, (uint32_t)bb, b);
      } else {
        const int ng = min(L.gpc, L.n_groups - g0);
        mbar_expect(b, (uint32_t)(ng * bb) + qb);
        bulk_g2s(dst, src + (size_t)g0 * bb, (uint32_t)(ng * bb), b);
      }
    }
    if (with_q) {
      __nv_bfloat16* qd = qbuf + qpar * (C::QS / 2);
      bulk_g2s(qd, q + ((size_t)r.li * P.units + r.unit) * GQ * D, (uint32_t)C::QB, b);
      if constexpr (SEL)
        bulk_g2s(qd + GQ * D, P.wide + ((size_t)(P.layer_begin + r.li) * P.units + r.unit) * kMarkWords,
                 16u, b);
    }
  };

  Cur cur = locate(c0), pre = cur;
  int pre_seg = 0;   // segment ordinal of the prefetch cursor's chunk
  auto produce = [&](int i) {   // all lanes: advance the prefetch cursor to chunk i; lane 0 issues
    if (i > 0) {
      step(pre);
      if (pre.j == 0) ++pre_seg;
    }
    int id[kMaxGpc], ngl = 0;
    if constexpr (LIST) ngl = groups_of(i, pre, id);
    if constexpr (RANGE)
      if (pre.j >= P.L[pre.li].wchunks) ngl = groups_of(i, pre, id);
    if (lane == 0) {
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      issue(i, pre, pre_seg & 1, i == 0 || pre.j == 0, ngl, id);
    }
  };
  produce(0);
  if (n > 1) produce(1);

  WarpState<D, GQ, MODE> st;
  QRegs<D, GQ> qr;
  int seg = -1;
  float head_sl2[n_tiles<GQ>()] = {};   // SEL: of the segment's heads
  const auto& sl2 = sl2_pick<SEL>(head_sl2, P.sl2);
  std::conditional_t<RANGE, RangeChunk, PlainChunk> ck;   // of the segment
  int fail = -1;   // chunk whose staging wait gave up
  // A segment = the chunks of one unit this warp holds. At its end the unit is
  // written whole; or its partial state goes to this CTA's shared memory, where the
  // last of the CTA's holders merges them; a unit that other CTAs also hold is
  // handed on as the CTA's partial state in global memory, where the last CTA
  // merges them. Tickets come from arrival counters (shared, then global); nothing
  // waits.
  auto finish = [&](const Cur& r, int seg_ord, bool failed) {
    const DecLayer& L = P.L[r.li];
    const long long ubeg = L.chunk_begin + (long long)r.unit * r.cpu, uend = ubeg + r.cpu;
    const size_t ul = (size_t)r.li * P.units + r.unit;
    float* o = out + ul * GQ * D;
    float2* stat = nullptr;
    if constexpr (RANGE) stat = P.part ? P.stat + ul * GQ : nullptr;
    auto put_weights = [&] {   // by the warp that has the unit's maxima and sums
      if constexpr (RANGE) {
        if (failed && stat && lane < GQ) __stcg(stat + lane, make_float2(-INFINITY, 0.f));
        if (!P.before) return;
        const RangeLayer& X = P.R[r.li];
        unit_weights<GQ>(P.part + ((size_t)X.part_begin + (size_t)r.unit * X.parts) * GQ, stat,
                         P.before + ul * P.n_slots, P.after + ul * P.n_slots, P.n_slots, L.n_groups,
                         X.parts);
      }
    };
    // Whether this is the last of `others` + 1 arrivals. Over a range a holder that gave up adds to the
    // high half as well: the last one then knows that the unit is not whole.
    auto arrive = [&](unsigned* counter, unsigned others) {
      unsigned last = 0;
      if constexpr (RANGE) {
        unsigned was = 0;
        if (lane == 0) was = atomicAdd(counter, failed ? 0x10001u : 1u);
        was = __shfl_sync(0xffffffffu, was, 0);
        failed = failed || was >> 16;
        last = (was & 0xffffu) == others;
      } else {
        if (lane == 0) last = atomicAdd(counter, 1u) == others;
        last = __shfl_sync(0xffffffffu, last, 0);
      }
      return last != 0;
    };
    if (ubeg >= c0 && uend <= c1) {
      if (!failed) write_final<D, GQ, SEL, RANGE>(st, o, sl2, stat);
      put_weights();
      return;
    }
    const long long lbeg = max(ubeg, C0), lend = min(uend, C1);   // the CTA's part
    const bool cta_whole = ubeg >= C0 && uend <= C1;
    const int wa = (int)ws.owner(lbeg), wb = (int)ws.owner(lend - 1);
    // this CTA's state of a unit that other CTAs also hold goes to global memory
    const int cslot = lbeg == C0 ? 0 : 1;
    float* gdep = P.ws + ((size_t)blockIdx.x * 2 + cslot) * C::DEPW;
    if (wb > wa) {
      // several holders in this CTA: partial state to shared memory, CTA ticket
      float* mine = sdep + ((size_t)warp * 2 + (seg_ord == 0 ? 0 : 1)) * C::DEPW;
      if (!failed) write_partial<D, GQ, SEL>(st, mine, sl2);
      __threadfence_block();
      __syncwarp();
      if (!arrive(&scnt[wa], (unsigned)(wb - wa))) return;
      __threadfence_block();
      const bool wa_late = ws.first(wa) < lbeg;   // its segment is its last one
      auto sdep_of = [&](int k) -> const float* {
        return sdep + ((size_t)(wa + k) * 2 + ((k == 0 && wa_late) ? 1 : 0)) * C::DEPW;
      };
      if (lane == 0) scnt[wa] = 0u;
      if (cta_whole) {
        if (!failed) merge_partials<D, GQ, false, true, RANGE>(wb - wa + 1, sdep_of, o, stat);
        put_weights();
        return;
      }
      if (!failed) merge_partials<D, GQ, false, false, false>(wb - wa + 1, sdep_of, gdep, nullptr);
    } else if (!failed) {
      write_partial<D, GQ, SEL>(st, gdep, sl2);
    }
    __threadfence();
    __syncwarp();
    const long long ca = cs.owner(ubeg), cb = cs.owner(uend - 1);
    unsigned* cnt = P.cnt + (size_t)(P.layer_begin + r.li) * P.units + r.unit;
    if (!arrive(cnt, (unsigned)(cb - ca))) return;
    __threadfence();
    const bool ca_late = cs.first(ca) < ubeg;   // the first CTA's segment is its last one
    if (!failed)
      merge_partials<D, GQ, true, true, RANGE>((int)(cb - ca + 1), [&](int k) -> const float* {
        return P.ws + ((size_t)(ca + k) * 2 + ((k == 0 && ca_late) ? 1 : 0)) * C::DEPW;
      }, o, stat);
    put_weights();
    __syncwarp();
    if (lane == 0) *cnt = 0u;   // ready for the next launch
  };

  for (int i = 0; i < n; ++i) {
    if (i > 0) step(cur);
    const bool seg_start = i == 0 || cur.j == 0;
    if (seg_start) {
      ++seg;
      state_init(st);
    }
    // wait for the chunk (and, at a segment start, the unit's queries)
    const uint32_t par = (uint32_t)((i >> 1) & 1);
    bool done = false;
    for (unsigned it = 0; it < P.wait_limit && !done; ++it) done = mbar_try_wait(&bar[i & 1], par);
    if (!__all_sync(0xffffffffu, done)) {
      if (lane == 0) atomicOr(P.err, 1u);
      fail = i;
      break;
    }
    const DecLayer& L = P.L[cur.li];
    __nv_bfloat16* qs = qbuf + (seg & 1) * (C::QS / 2);
    if constexpr (SEL) {
      if (seg_start) {
        const bool far = load_qregs<D, GQ, SEL>(qr, qs);
        if (far) {
          scale_queries<D, GQ>(qs, P.sl2);
          load_qregs<D, GQ, SEL>(qr, qs);
        }
        const float* factors = reinterpret_cast<const float*>(qs + GQ * D) + 4;
#pragma unroll
        for (int u = 0; u < n_tiles<GQ>(); ++u)
          head_sl2[u] = far ? factors[min(4 * u + (lane & 3), GQ - 1)] : P.sl2;
      }
    } else if (seg_start) {
      load_qregs<D, GQ, SEL>(qr, qs);
    }
    uint8_t* sbuf = ring + (i & 1) * C::SLOT;
    if constexpr (RANGE) {
      if (seg_start) {
        const RangeLayer& X = P.R[cur.li];
        ck.a = X.a;
        ck.b = X.b;
        ck.part = P.part ? P.part + ((size_t)X.part_begin + (size_t)cur.unit * X.parts) * GQ : nullptr;
      }
    }
    if (cur.j < L.wchunks) {
      __nv_bfloat16* sk = reinterpret_cast<__nv_bfloat16*>(sbuf);
      uint32_t* sv = reinterpret_cast<uint32_t*>(sbuf + kSlotsPerWarp * D * 2);
      int pos0 = cur.j * kSlotsPerWarp;
      if constexpr (RANGE) {
        const RangeLayer& X = P.R[cur.li];
        if (cur.j >= X.w_first) pos0 += X.w_skip * kSlotsPerWarp;
        ck.t0[0] = ck.t0[1] = L.n_groups * KVC_GROUP + pos0;
        ck.slot[0] = ck.slot[1] = L.n_groups + pos0 / kSlotsPerWarp;
      }
      const int n_valid = min(kSlotsPerWarp, L.win_len - pos0);
      if (L.new_slot >= 0 && cur.j == (L.win_len - 1) / kSlotsPerWarp) {
        // the step's new token: store it into the ring (later steps read it) and
        // patch the staged copy (the bulk copy may predate the store)
        const size_t ul = (size_t)cur.li * P.units + cur.unit;
        const size_t rb = (size_t)L.win_off + (size_t)cur.unit * L.R * D;
        const __nv_bfloat16* kn = P.k_new + ul * D;
        const __nv_bfloat16* vn = P.v_new + ul * D;
        const int r = L.new_slot - (L.win_start + pos0) % L.R;
        __nv_bfloat16* svh = reinterpret_cast<__nv_bfloat16*>(sv);
        for (int c = lane; c < D; c += 32) {
          const __nv_bfloat16 kv = kn[c], vv = vn[c];
          window_store(win_k + rb, win_v + rb, L.new_slot, c, D, kv, vv);
          sk[win_k_index(r, c, D)] = kv;
          svh[win_v_index(r, c, D)] = vv;
        }
        __syncwarp();
      }
      if (n_valid < kSlotsPerWarp) {
        // The values of slots behind the last token become 0: an older sequence may have left
        // some there that are not finite, which must not meet their weights of 0. A pair row
        // holds two slots, the earlier in the low halves.
        for (int p = n_valid >> 1; p < kSlotsPerWarp / 2; ++p) {
          const uint32_t keep = 2 * p < n_valid ? 0xffffu : 0u;
          for (int c = lane; c < D; c += 32) sv[p * D + c] &= keep;
        }
        __syncwarp();
      }
      if constexpr (RANGE) {
        const Seen seen = ck.seen(0);
        if (!seen.all(n_valid)) {   // the same for hidden slots
          for (int p = 0; p < kSlotsPerWarp / 2; ++p) {
            const uint32_t keep = (seen.at(2 * p) ? 0xffffu : 0u) | (seen.at(2 * p + 1) ? 0xffff0000u : 0u);
            if (keep != 0xffffffffu)
              for (int c = lane; c < D; c += 32) sv[p * D + c] &= keep;
          }
          __syncwarp();
        }
      }
      window_warp<D, GQ, SEL>(st, qs, sk, sv, n_valid, sl2, ck);
    } else {
      int ng;
      if constexpr (SEL) {
        int id[kMaxGpc];
        ng = groups_of(i, cur, id);
        if constexpr (RANGE)
#pragma unroll
          for (int k = 0; k < kMaxGpc; ++k) {
            ck.t0[k] = id[k] * KVC_GROUP;
            ck.slot[k] = id[k];
          }
      } else {
        ng = min(L.gpc, L.n_groups - (cur.j - L.wchunks) * L.gpc);
      }
      auto groups = [&](auto BITS_) {
        constexpr int BITS = decltype(BITS_)::value;
        if constexpr (RANGE) range_warp<D, BITS, GQ>(st, qr, qs, sbuf, ng, sl2, ck);
        else packed_warp<D, BITS, GQ, SEL>(st, qr, sbuf, ng, sl2);
      };
      if constexpr (BMASK == 1) {
        groups(std::integral_constant<int, 2>{});
      } else if constexpr (BMASK == 2) {
        groups(std::integral_constant<int, 4>{});
      } else {
        if (L.bits == 2) groups(std::integral_constant<int, 2>{});
        else groups(std::integral_constant<int, 4>{});
      }
    }
    __syncwarp();   // the slot is read: refill it with the chunk two ahead
    if (i + 2 < n) produce(i + 2);
    if (i == n - 1 || cur.j == cur.cpu - 1) finish(cur, seg, false);
  }
  if (fail >= 0) {
    // let the copies in flight land (chunk fail and the one after it), then hand
    // over the split units left open so every counter still returns to zero
    for (int i = fail; i < n && i <= fail + 1; ++i) {
      bool done = false;
      for (unsigned it = 0; it < kWaitLimit && !done; ++it)
        done = mbar_try_wait(&bar[i & 1], (uint32_t)((i >> 1) & 1));
    }
    __syncwarp();
    finish(cur, seg, true);
    if constexpr (RANGE) {   // (also the units in between, which nobody else holds: their weights)
      for (int i = fail + 1; i < n; ++i) {
        step(cur);
        if (cur.j == 0) finish(cur, ++seg, true);
      }
    } else {
      const Cur last = locate(c1 - 1);
      if (last.li != cur.li || last.unit != cur.unit) finish(last, seg + 1, true);
    }
  }
}

template <int D, int GQ, int BMASK, int MODE>
cudaError_t launch_one(ParamsOf<MODE>& P, const kvc_cache* c, const __nv_bfloat16* q, float* out,
                       cudaStream_t stream) {
  using C = DecCfg<D, GQ, BMASK, MODE != kDecAll>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(decode_kernel<D, GQ, BMASK, MODE>), C::total);
  if (e != cudaSuccess) return e;
  // one CTA per SM, each holding at least one chunk per warp where the launch has
  // that many (fewer, fuller CTAs merge less across SMs)
  const long long T = P.total;
  const int grid = (int)std::max<long long>(1, std::min<long long>(c->n_sm, T / C::NW));
  P.n_vwarps = grid * C::NW;
  if ((size_t)grid * 2 * C::DEPW > c->dec_ws_floats) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::total;
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attr()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_kernel<D, GQ, BMASK, MODE>, P, c->packed, c->win_k, c->win_v,
                            q, out);
}

template <int D, int BMASK, int MODE>
cudaError_t launch_g(ParamsOf<MODE>& P, const kvc_cache* c, const __nv_bfloat16* q, float* out,
                     cudaStream_t stream) {
  switch (c->g) {
    case 1: return launch_one<D, 1, BMASK, MODE>(P, c, q, out, stream);
    case 2: return launch_one<D, 2, BMASK, MODE>(P, c, q, out, stream);
    case 4: return launch_one<D, 4, BMASK, MODE>(P, c, q, out, stream);
    case 8: return launch_one<D, 8, BMASK, MODE>(P, c, q, out, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <int MODE>
cudaError_t launch_bits(ParamsOf<MODE>& P, const kvc_cache* c, int bmask, const __nv_bfloat16* q,
                        float* out, cudaStream_t stream) {
  const int D = c->dims.head_dim;
  if (bmask == 0) bmask = 1;   // window only: any instantiation serves
  if (D == 128 && bmask == 1) return launch_g<128, 1, MODE>(P, c, q, out, stream);
  if (D == 128 && bmask == 2) return launch_g<128, 2, MODE>(P, c, q, out, stream);
  if (D == 128) return launch_g<128, 3, MODE>(P, c, q, out, stream);
  if (bmask == 1) return launch_g<64, 1, MODE>(P, c, q, out, stream);
  if (bmask == 2) return launch_g<64, 2, MODE>(P, c, q, out, stream);
  return launch_g<64, 3, MODE>(P, c, q, out, stream);
}

}  // namespace
}  // namespace kvc
