// tree.cu -- attention of a tree of drafted tokens over the compressed cache
// (kvc_tree_attn): each node's query attends to every cached token (packed groups and
// window), to the drafted tokens on its path to the root, and to itself, in one softmax:
//     o_r = sum_t exp(q_r . k_t / sqrt d) v_t / sum_t exp(q_r . k_t / sqrt d),
// t over the tokens row r sees. The R = g n_nodes rows (query head, node) of a (layer,
// sequence, kv head) unit read the same cache, so the cache is read and unpacked once for
// up to 64 of them and multiplied on the tensor cores.
//
// Orientation. Both products are issued transposed, with the tokens' side as the A operand
// in tensor memory:
//     S^T[token][row]   = K . Q^T       A = K   (lane = token,   128 x d)
//     O^T[channel][row] += V^T . P      A = V^T (lane = channel, d x 128)
// The cost of a product then falls with the number of rows (N = 16, 32 or 64), and the
// unpacked keys and values go from registers straight into tensor memory: the operand
// fragments that the packed store's words hold are those of the 16x128b tensor-memory
// store (row = lane / 4 (+ 8), column = lane % 4), so nothing is staged or transposed in
// shared memory. Q and P are the B operands (shared memory, 128-byte swizzle; P is written
// row-contiguous per token, MN-major).
//
// Arithmetic. A packed key or value is code * S + Z in one fp16 fused multiply-add: rounded
// once, to 2^-11 of itself, an eighth of what bf16 would lose, and inside fp16's range
// because S and Z are. The queries meet them as fp16 scaled per row by a power of two to
// [1, 2) (elements below 2^-14 of the row's largest keep 2^-25 of it), the weights as fp16.
// Window and drafted tokens are bf16 as they are, against bf16 queries and weights.
// Logits, the running maximum, sums and outputs are fp32; the output is rounded to bf16.
// The reference a row's weights are taken against is raised when a logit passes it by 8
// (log2 units; the weights then stay below 2^8), each row by itself.
//
// Work. A unit's rows are cut into row tiles (of N rows); a (layer, unit, row tile) is a
// segment of tiles of 128 tokens: four packed groups each, then the window, then the
// drafted tokens. The tiles of all segments are laid end to end and cut into one
// contiguous range per CTA (one per SM). A segment that lies in several CTAs is handed
// over as partial states (o, m, l) in global memory and merged by the CTA that arrives last
// (a ticket; nothing waits), in a fixed order.
//
// Roles (18 warps): 0 bulk copies of raw tiles into a ring and the ancestor sets of the
// drafted nodes; 1 tensor memory and the products; 2-5 keys (one group of the tile each)
// and 6-9 values (one 32-channel group each) into tensor memory, and the queries; 10-17
// softmax (lane quarter = warp % 4, column half), output and merge. Every wait is bounded.
#include "decode_device.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr int kTrThreads = 18 * 32;
constexpr int kTrSoftThreads = 256;
constexpr uint32_t kTrTmemCols = 512;
constexpr int kTrTile = 128;          // tokens of a tile
constexpr float kTrSlack = 8.f;       // a row's reference is raised when passed by this
constexpr int kTrMaxNodes = KVC_MAX_TREE_NODES;
static_assert(kTrMaxNodes == 64, "ancestor sets are 64-bit, a drafted tile holds 64 tokens");
constexpr unsigned kErrTrProducer = 1u << 16, kErrTrMma = 1u << 17, kErrTrUnpack = 1u << 18,
                   kErrTrSoftmax = 1u << 19;

struct TreeLayer {
  long long tile_begin;       // first tile of the layer in the launch's list
  long long packed_off, win_off;
  int n_groups, cap_groups, bits, win_start, win_len, R;
  int pt, wt, tps;            // packed and window tiles, tiles per segment (with the drafted one)
};
struct TreeParams {
  TreeLayer L[KVC_MAX_LAUNCH_LAYERS];
  const uint8_t* packed;
  const __nv_bfloat16* win_k;
  const __nv_bfloat16* win_v;
  const int32_t* parents;         // [B][T]
  const __nv_bfloat16* q;         // [layers][units][rows][d]
  const __nv_bfloat16* k_draft;   // [layers][units][T][d]
  const __nv_bfloat16* v_draft;
  __nv_bfloat16* out;             // as q
  float* ws;                      // partial states, two per CTA
  unsigned* cnt;                  // arrival tickets [layer][unit][row tile], zero between launches
  unsigned* err;
  long long total;                // tiles of the launch
  int n_layers, layer_begin, units, H, T, rows, RT;
  float sl2;
};

template <int D, int N>
struct TrCfg {
  static constexpr int CW = N / 2;                  // columns of one softmax warp
  static constexpr int SLOT = kTrTile * D * 2;      // raw ring slot: 128 window keys or values
  static constexpr int NS = D == 128 ? 4 : 8;
  static constexpr int DP = 2 * D + 16;             // row pitch of staged drafted tokens
  static constexpr int QB = N * D * 2;
  static constexpr int PB = kTrTile * 128;          // weights: 128 tokens x 64 rows, 16 bits
  static constexpr int oRaw = 0;
  static constexpr int oQ = oRaw + NS * SLOT;       // [2]
  static constexpr int oP = oQ + 2 * QB;            // [2]
  static constexpr int oQs = oP + 2 * PB;           // [8][N] logit scale per query set and row
  static constexpr int oRef = oQs + 8 * N * 4;      // [N] minus the rows' reference
  static constexpr int oRed = oRef + N * 4;         // [4][N]
  static constexpr int oAnc = oRed + 4 * N * 4;     // [4][64] ancestor sets (0: padding)
  static constexpr int oBar = oAnc + 4 * kTrMaxNodes * 8;
  // rawfull[NS], rawempty[NS], qfull[2], kfull[2], vfull[2], qkdone[2], pvdone[2],
  // sempty[2], pfull[2], ancfull[4], drain
  static constexpr int NBAR = 2 * NS + 14 + 5;
  static constexpr int oMisc = oBar + NBAR * 8;     // tensor memory base, flags
  static constexpr int total = oMisc + 32 + 1024;   // + alignment slack
  static constexpr int STATE = N * (D + 2);         // floats of one partial state
  // tensor memory columns
  static constexpr uint32_t cK = 0, cV = D, cS = D + kTrTile, cO = cS + 2 * N;
  static_assert(cO + N <= kTrTmemCols, "tensor memory");
  static_assert(kTrMaxNodes * DP <= SLOT && 4 * block_bytes(D, 4) <= SLOT, "ring slot");
  static_assert(SLOT % 1024 == 0 && QB % 1024 == 0 && PB % 1024 == 0, "1024-byte aligned");
  static_assert(total <= 227 * 1024, "shared memory");
};

enum { kPacked = 0, kWindow = 1, kDraft = 2 };

struct TrCur {
  int li, unit, rt, j;
};
__device__ __forceinline__ TrCur tr_locate(const TreeParams& P, long long c) {
  TrCur r;
  r.li = 0;
  while (r.li + 1 < P.n_layers && c >= P.L[r.li + 1].tile_begin) ++r.li;
  const long long loc = c - P.L[r.li].tile_begin, seg = loc / P.L[r.li].tps;
  r.j = (int)(loc - seg * P.L[r.li].tps);
  r.unit = (int)(seg / P.RT);
  r.rt = (int)(seg - (long long)r.unit * P.RT);
  return r;
}
__device__ __forceinline__ void tr_step(const TreeParams& P, TrCur& r) {
  if (++r.j < P.L[r.li].tps) return;
  r.j = 0;
  if (++r.rt < P.RT) return;
  r.rt = 0;
  if (++r.unit < P.units) return;
  r.unit = 0;
  ++r.li;
}
__device__ __forceinline__ int tr_type(const TreeLayer& L, int j) {
  return j < L.pt ? kPacked : (j < L.pt + L.wt ? kWindow : kDraft);
}
// Whether tile i of a CTA's range begins a set of queries (one format, one segment).
__device__ __forceinline__ bool tr_new_set(const TreeLayer& L, int i, int j) {
  return i == 0 || j == 0 || (j == L.pt);
}

__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  return h2u(__hfma2(u2h(a), u2h(b), u2h(c)));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c,
                                      uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c,
                                       uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr));
}

// The keys of one packed group into tensor memory (32 lanes = tokens, d / 2 columns).
template <int D, int BITS>
__device__ __forceinline__ void keys_packed(const uint8_t* blk, uint32_t dst) {
  constexpr int KS = D / 16, WPL = D * BITS / 32;
  const int lane = threadIdx.x & 31, tid = lane & 3;
  const CodeMasks<BITS> cm = code_masks<BITS>();
  uint32_t kw[WPL], S[KS][2], Z[KS][2];
  const uint4* p = reinterpret_cast<const uint4*>(blk);
#pragma unroll
  for (int i = 0; i < WPL / 4; ++i) {
    const uint4 w = p[i * 32 + lane];
    kw[4 * i] = w.x; kw[4 * i + 1] = w.y; kw[4 * i + 2] = w.z; kw[4 * i + 3] = w.w;
  }
  const uint4* sp = reinterpret_cast<const uint4*>(blk + off_kscale(D, BITS) + tid * (D / 4) * 2);
  const uint4* zp = reinterpret_cast<const uint4*>(blk + off_kzero(D, BITS) + tid * (D / 4) * 2);
#pragma unroll
  for (int i = 0; i < KS / 2; ++i) {
    const uint4 s = sp[i], z = zp[i];
    S[2 * i][0] = s.x; S[2 * i][1] = s.y; S[2 * i + 1][0] = s.z; S[2 * i + 1][1] = s.w;
    Z[2 * i][0] = z.x; Z[2 * i][1] = z.y; Z[2 * i + 1][0] = z.z; Z[2 * i + 1][1] = z.w;
  }
  static_for<2>([&](auto MT_) {
    constexpr int MT = decltype(MT_)::value;
    uint32_t r[4 * KS];
    static_for<KS>([&](auto K_) {
      constexpr int k = decltype(K_)::value;
      uint32_t a[4];
      key_afrag<D, BITS, MT, k>(kw, cm, a);
      r[4 * k] = hfma2u(a[0], S[k][0], Z[k][0]);
      r[4 * k + 1] = hfma2u(a[1], S[k][0], Z[k][0]);
      r[4 * k + 2] = hfma2u(a[2], S[k][1], Z[k][1]);
      r[4 * k + 3] = hfma2u(a[3], S[k][1], Z[k][1]);
    });
    tc::tmem_st_frag(dst + ((uint32_t)(16 * MT) << 16), r);
  });
}

// The values of channels 32 w .. 32 w + 31 of one packed group (lanes = channels, 16 columns).
template <int D, int BITS>
__device__ __forceinline__ void values_packed(const uint8_t* blk, int w, uint32_t dst) {
  constexpr int NGC = D / 32;
  const int lane = threadIdx.x & 31, tid = lane & 3;
  const CodeMasks<BITS> cm = code_masks<BITS>();
  uint32_t wd[4];
  if constexpr (BITS == 4) {
    const uint4 v = reinterpret_cast<const uint4*>(blk + off_vcodes(D, BITS))[w * 32 + lane];
    wd[0] = v.x; wd[1] = v.y; wd[2] = v.z; wd[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(blk + off_vcodes(D, BITS) + (w >> 1) * 512 +
                                                    lane * 16 + (w & 1) * 8);
    wd[0] = v.x; wd[1] = v.y; wd[2] = 0u; wd[3] = 0u;
  }
  const uint32_t* vs = reinterpret_cast<const uint32_t*>(blk + off_vscale(D, BITS));
  const uint32_t* vz = reinterpret_cast<const uint32_t*>(blk + off_vzero(D, BITS));
  uint32_t S[2][2], Z[2][2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    // scales of (t, t + 8) and (t + 1, t + 9), t = 16 ks + 2 tid, regrouped by token pair
    const uint32_t a = vs[(8 * ks + 2 * tid) * NGC + w], b = vs[(8 * ks + 2 * tid + 1) * NGC + w];
    S[ks][0] = __byte_perm(a, b, 0x5410);
    S[ks][1] = __byte_perm(a, b, 0x7632);
    Z[ks][0] = vz[(8 * ks + tid) * NGC + w];
    Z[ks][1] = vz[(8 * ks + 4 + tid) * NGC + w];
  }
  static_for<2>([&](auto H_) {
    constexpr int h = decltype(H_)::value;
    uint32_t r[8];
    static_for<2>([&](auto K_) {
      constexpr int ks = decltype(K_)::value;
      uint32_t a[4];
      if constexpr (BITS == 4) {
        const uint32_t x = wd[2 * h + ks], x8 = x >> 8;
        a[0] = unpack_pair<4, 0>(x, x8, cm);
        a[1] = unpack_pair<4, 2>(x, x8, cm);
        a[2] = unpack_pair<4, 1>(x, x8, cm);
        a[3] = unpack_pair<4, 3>(x, x8, cm);
      } else {
        const uint32_t x = wd[h], x8 = x >> 8;
        a[0] = unpack_pair<2, 2 * ks>(x, x8, cm);
        a[1] = unpack_pair<2, 4 + 2 * ks>(x, x8, cm);
        a[2] = unpack_pair<2, 2 * ks + 1>(x, x8, cm);
        a[3] = unpack_pair<2, 5 + 2 * ks>(x, x8, cm);
      }
      r[4 * ks] = hfma2u(a[0], S[ks][0], Z[ks][0]);
      r[4 * ks + 1] = hfma2u(a[1], S[ks][0], Z[ks][0]);
      r[4 * ks + 2] = hfma2u(a[2], S[ks][1], Z[ks][1]);
      r[4 * ks + 3] = hfma2u(a[3], S[ks][1], Z[ks][1]);
    });
    tc::tmem_st_frag(dst + ((uint32_t)(16 * h) << 16), r);
  });
}

// 32 window keys (rows row0 .. row0 + 31 of the staged tile).
template <int D>
__device__ __forceinline__ void keys_window(const uint8_t* raw, int row0, uint32_t dst) {
  constexpr int KS = D / 16;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    const uint4* r0 = reinterpret_cast<const uint4*>(raw + (size_t)(row0 + 16 * mt + gid) * D * 2);
    const uint4* r1 = reinterpret_cast<const uint4*>(raw + (size_t)(row0 + 16 * mt + gid + 8) * D * 2);
    uint32_t r[4 * KS];
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {
      const int ch = (tid * (KS / 2) + i) ^ gid;
      const uint4 a = r0[ch], b = r1[ch];
      r[8 * i] = a.x; r[8 * i + 1] = b.x; r[8 * i + 2] = a.y; r[8 * i + 3] = b.y;
      r[8 * i + 4] = a.z; r[8 * i + 5] = b.z; r[8 * i + 6] = a.w; r[8 * i + 7] = b.w;
    }
    tc::tmem_st_frag(dst + ((uint32_t)(16 * mt) << 16), r);
  }
}

// Both halves of a token pair (t, t + 1) kept where the token is one of the first n.
__device__ __forceinline__ uint32_t keep_pair(int t, int n) {
  return t + 1 < n ? 0xffffffffu : (t < n ? 0xffffu : 0u);
}

// The window values of channels 32 w .. + 31: 128 tokens, those past the first n zero (a
// weight of zero must not meet what an old slot holds).
template <int D>
__device__ __forceinline__ void values_window(const uint8_t* raw, int w, int n, uint32_t dst) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
#pragma unroll
  for (int k4 = 0; k4 < 8; k4 += 4) {
    uint32_t r0[16], r1[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ks = k4 + k, ch = (gid * (D / 32) + w) ^ tid;
      const uint4 a = reinterpret_cast<const uint4*>(raw + (size_t)(8 * ks + tid) * D * 4)[ch];
      const uint4 b = reinterpret_cast<const uint4*>(raw + (size_t)(8 * ks + 4 + tid) * D * 4)[ch];
      const uint32_t ma = keep_pair(16 * ks + 2 * tid, n), mb = keep_pair(16 * ks + 8 + 2 * tid, n);
      r0[4 * k] = a.x & ma; r0[4 * k + 1] = a.y & ma; r0[4 * k + 2] = b.x & mb; r0[4 * k + 3] = b.y & mb;
      r1[4 * k] = a.z & ma; r1[4 * k + 1] = a.w & ma; r1[4 * k + 2] = b.z & mb; r1[4 * k + 3] = b.w & mb;
    }
    tc::tmem_st_frag(dst + 8u * k4, r0);
    tc::tmem_st_frag(dst + 8u * k4 + (16u << 16), r1);
  }
}

// 32 drafted keys (rows row0 .. of the staged tile, pitch DP).
template <int D, int DP>
__device__ __forceinline__ void keys_draft(const uint8_t* raw, int row0, uint32_t dst) {
  constexpr int KS = D / 16;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    const uint32_t a0 = tc::saddr(raw) + (uint32_t)((row0 + 16 * mt + (lane & 15)) * DP + (lane >> 4) * 16);
    uint32_t r[4 * KS];
#pragma unroll
    for (int k = 0; k < KS; ++k)
      ldsm4(a0 + 32u * k, r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
    tc::tmem_st_frag(dst + ((uint32_t)(16 * mt) << 16), r);
  }
}

// The halves of a bf16 pair that are not finite.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// The drafted values of channels 32 w .. + 31: tokens that are padding are zero; a value that is
// not finite is zero too (it must not meet the zero weights of rows that do not see it) and
// reported: the output pass adds it to the rows that do.
template <int D, int DP>
__device__ __forceinline__ bool values_draft(const uint8_t* raw, int w, unsigned long long live,
                                             uint32_t dst) {
  const int lane = threadIdx.x & 31, tid = lane & 3;
  uint32_t bad = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a0 = tc::saddr(raw) + (uint32_t)(((lane & 7) + 8 * (lane >> 4)) * DP +
                                                    (32 * w + 16 * h + 8 * ((lane >> 3) & 1)) * 2);
    uint32_t r[16];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      ldsm4t(a0 + (uint32_t)(16 * ks * DP), r[4 * ks], r[4 * ks + 1], r[4 * ks + 2], r[4 * ks + 3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned on = (unsigned)(live >> (16 * ks + 2 * tid + 8 * (e >> 1))) & 3u;
        const uint32_t x = r[4 * ks + e] & ((on & 1u ? 0xffffu : 0u) | (on & 2u ? 0xffff0000u : 0u));
        const uint32_t nf = not_finite(x);
        bad |= nf;
        r[4 * ks + e] = x & ~nf;
      }
    }
    tc::tmem_st_frag(dst + ((uint32_t)(16 * h) << 16), r);
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] = 0u;
    tc::tmem_st_frag(dst + 32u + ((uint32_t)(16 * h) << 16), r);
  }
  return __any_sync(0xffffffffu, bad != 0u);
}

__device__ __forceinline__ void soft_bar() {
  asm volatile("barrier.cta.sync 1, %0;" :: "n"(kTrSoftThreads) : "memory");
}
__device__ __forceinline__ bool soft_bar_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r) : "r"((uint32_t)p), "n"(kTrSoftThreads) : "memory");
  return r != 0u;
}

template <int D, int N>
__global__ void __launch_bounds__(kTrThreads, 1)
tree_kernel(const __grid_constant__ TreeParams P) {
  using C = TrCfg<D, N>;
  constexpr int CW = C::CW, NS = C::NS;
  extern __shared__ uint8_t dsm_raw[];
  uint8_t* dsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) &
                                            ~uintptr_t(1023));
  uint8_t* raw = dsm + C::oRaw;
  float* s_qs = reinterpret_cast<float*>(dsm + C::oQs);
  float* s_nref = reinterpret_cast<float*>(dsm + C::oRef);
  float* s_red = reinterpret_cast<float*>(dsm + C::oRed);
  unsigned long long* s_anc = reinterpret_cast<unsigned long long*>(dsm + C::oAnc);
  uint64_t* rawfull = reinterpret_cast<uint64_t*>(dsm + C::oBar);
  uint64_t* rawempty = rawfull + NS;
  uint64_t* qfull = rawempty + NS;
  uint64_t* kfull = qfull + 2;
  uint64_t* vfull = kfull + 2;
  uint64_t* qkdone = vfull + 2;
  uint64_t* pvdone = qkdone + 2;
  uint64_t* sempty = pvdone + 2;
  uint64_t* pfull = sempty + 2;
  uint64_t* ancfull = pfull + 2;
  uint64_t* drain = ancfull + 4;
  volatile uint32_t* s_misc = reinterpret_cast<volatile uint32_t*>(dsm + C::oMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) { tc::mbar_init(&rawfull[s], 1); tc::mbar_init(&rawempty[s], 8); }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&qfull[s], 8);
      tc::mbar_init(&kfull[s], 4);
      tc::mbar_init(&vfull[s], 4);
      tc::mbar_init(&qkdone[s], 1);
      tc::mbar_init(&pvdone[s], 1);
      tc::mbar_init(&sempty[s], 8);
      tc::mbar_init(&pfull[s], 8);
    }
    for (int s = 0; s < 4; ++s) tc::mbar_init(&ancfull[s], 1);
    tc::mbar_init(drain, 1);
    tc::fence_mbar_init();
    // ordinal + 1 of a drafted tile that holds a value that is not finite
    for (int k = 0; k < 4; ++k) s_misc[4 + k] = 0u;
  }
  if (warp == 1) {
    tc::tmem_alloc(const_cast<uint32_t*>(&s_misc[0]), kTrTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = s_misc[0];
  pdl_wait();      // the previous kernels' writes (inputs, cache, tickets) are visible
  pdl_release();

  const Split cs{P.total, (long long)gridDim.x, 0};
  const long long C0 = cs.first(blockIdx.x), C1 = cs.first(blockIdx.x + 1);
  const int n = (int)(C1 - C0);   // >= 1: the grid is at most the number of tiles
  TrCur cur = tr_locate(P, C0);
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------- raw tiles
    int it = 0, nd = 0;   // ring items, drafted tiles so far
    auto slot = [&]() {   // the next ring slot, free
      const int s = it % NS, round = it / NS;
      if (round > 0) ok = tc::mbar_wait(&rawempty[s], (uint32_t)((round - 1) & 1), P.err, kErrTrProducer);
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      return s;
    };
    for (int i = 0; i < n && ok; ++i) {
      const TreeLayer& L = P.L[cur.li];
      const int type = tr_type(L, cur.j);
      if (type == kPacked) {
        const int s = slot();
        if (!ok) break;
        if (lane == 0) {
          const int bb = block_bytes(D, L.bits), g0 = 4 * cur.j;
          const uint32_t bytes = (uint32_t)(min(4, L.n_groups - g0) * bb);
          tc::mbar_expect_tx(&rawfull[s], bytes);
          bulk_g2s(raw + s * C::SLOT,
                   P.packed + L.packed_off + ((size_t)cur.unit * L.cap_groups + g0) * bb, bytes,
                   &rawfull[s]);
        }
        ++it;
      } else if (type == kWindow) {
        const int w0 = (cur.j - L.pt) * kTrTile, cnt = min(kTrTile, L.win_len - w0);
        const int s0 = (L.win_start + w0) % L.R;
        const size_t rb = (size_t)L.win_off + (size_t)cur.unit * L.R * D;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int s = slot();
          if (!ok) break;
          if (lane == 0) {
            // keys: rows of d; values: rows of d token pairs. The ring may wrap inside the tile
            const int rows = kv ? (cnt + 1) / 2 : cnt, first = kv ? s0 / 2 : s0;
            const int ring = kv ? L.R / 2 : L.R, rbytes = kv ? 4 * D : 2 * D;
            const uint8_t* src = reinterpret_cast<const uint8_t*>((kv ? P.win_v : P.win_k) + rb);
            const int a = min(rows, ring - first);
            uint8_t* dst = raw + s * C::SLOT;
            tc::mbar_expect_tx(&rawfull[s], (uint32_t)(rows * rbytes));
            bulk_g2s(dst, src + (size_t)first * rbytes, (uint32_t)(a * rbytes), &rawfull[s]);
            if (rows > a)
              bulk_g2s(dst + a * rbytes, src, (uint32_t)((rows - a) * rbytes), &rawfull[s]);
          }
          ++it;
        }
      } else {
        // ancestor sets: 64 links followed by doubling; a bad link marks its node, and what
        // hangs from it, as padding (the empty set)
        const int b = cur.unit / P.H;
        unsigned long long* anc = s_anc + (nd & 3) * kTrMaxNodes;
        int up[2];
        bool dead[2];
        unsigned long long set[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i2 = lane + 32 * e;
          const int p = i2 < P.T ? P.parents[(size_t)b * P.T + i2] : -2;
          dead[e] = p < -1 || p >= i2;
          up[e] = dead[e] ? -1 : p;
          set[e] = 1ull << i2;
        }
#pragma unroll 1
        for (int step = 0; step < 6; ++step) {
          // node x's set, link and mark from lane x % 32
          unsigned long long s2[2];
          int u2[2];
          bool d2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = up[e] < 0 ? 0 : up[e];
            const unsigned long long lo = __shfl_sync(0xffffffffu, set[0], x & 31),
                                     hi = __shfl_sync(0xffffffffu, set[1], x & 31);
            const int ul = __shfl_sync(0xffffffffu, up[0], x & 31),
                      uh = __shfl_sync(0xffffffffu, up[1], x & 31);
            const int dl = __shfl_sync(0xffffffffu, (int)dead[0], x & 31),
                      dh = __shfl_sync(0xffffffffu, (int)dead[1], x & 31);
            const bool link = up[e] >= 0, high = x >= 32;
            s2[e] = set[e] | (link ? (high ? hi : lo) : 0ull);
            d2[e] = dead[e] || (link && (high ? dh : dl));
            u2[e] = link ? (high ? uh : ul) : -1;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) { set[e] = s2[e]; dead[e] = d2[e]; up[e] = u2[e]; }
        }
        anc[lane] = dead[0] ? 0ull : set[0];
        anc[lane + 32] = dead[1] ? 0ull : set[1];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ancfull[nd & 3]);
        ++nd;
        const size_t ul = ((size_t)cur.li * P.units + cur.unit) * P.T * D;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int s = slot();
          if (!ok) break;
          if (lane == 0) tc::mbar_expect_tx(&rawfull[s], (uint32_t)(P.T * D * 2));
          __syncwarp();
          for (int t = lane; t < P.T; t += 32)
            bulk_g2s(raw + s * C::SLOT + t * C::DP, (kv ? P.v_draft : P.k_draft) + ul + (size_t)t * D,
                     (uint32_t)(D * 2), &rawfull[s]);
          ++it;
        }
      }
      tr_step(P, cur);
    }
    // every copy issued here has landed before the CTA can leave
    for (int k = max(0, it - NS); k < it; ++k)
      tc::mbar_wait(&rawfull[k % NS], (uint32_t)((k / NS) & 1), P.err, kErrTrProducer);
  } else if (warp == 1) {
    // -------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t q0 = tc::saddr(dsm + C::oQ), p0 = tc::saddr(dsm + C::oP);
      TrCur qc = cur;
      int sets = 0;
      auto keys = [&](int i) {      // S^T of tile i
        const TreeLayer& L = P.L[qc.li];
        if (tr_new_set(L, i, qc.j)) {
          ok = tc::mbar_wait(&qfull[sets & 1], (uint32_t)((sets >> 1) & 1), P.err, kErrTrMma);
          ++sets;
        }
        if (ok) ok = tc::mbar_wait(&kfull[i & 1], (uint32_t)((i >> 1) & 1), P.err, kErrTrMma);
        if (ok && i >= 2)
          ok = tc::mbar_wait(&sempty[i & 1], (uint32_t)(((i >> 1) - 1) & 1), P.err, kErrTrMma);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t id = tc::idesc_ts(128, N, tr_type(L, qc.j) != kPacked, false);
        const uint32_t qa = q0 + (uint32_t)(((sets - 1) & 1) * C::QB);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ts(tbase + C::cS + (uint32_t)((i & 1) * N), tbase + C::cK + (uint32_t)((i & 1) * (D / 2) + kk * 8),
                     tc::sw128_desc(qa + (kk / 4) * N * 128 + (kk % 4) * 32), id, kk > 0 ? 1u : 0u);
        tc::mma_commit(&qkdone[i & 1]);
        tr_step(P, qc);
      };
      keys(0);
      for (int i = 0; i < n && ok; ++i) {
        if (i + 1 < n) keys(i + 1);
        if (ok) ok = tc::mbar_wait(&vfull[i & 1], (uint32_t)((i >> 1) & 1), P.err, kErrTrMma);
        if (ok) ok = tc::mbar_wait(&pfull[i & 1], (uint32_t)((i >> 1) & 1), P.err, kErrTrMma);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t id = tc::idesc_ts(128, N, tr_type(P.L[cur.li], cur.j) != kPacked, true);
        const bool fresh = i == 0 || cur.j == 0;
#pragma unroll
        for (int kk = 0; kk < kTrTile / 16; ++kk)
          tc::mma_ts(tbase + C::cO, tbase + C::cV + (uint32_t)((i & 1) * (kTrTile / 2) + kk * 8),
                     tc::sw128_mn_desc(p0 + (i & 1) * C::PB + kk * 16 * 128, C::PB, 1024), id,
                     (fresh && kk == 0) ? 0u : 1u);
        tc::mma_commit(&pvdone[i & 1]);
        tr_step(P, cur);
      }
      // every product issued here has completed before tensor memory is released
      tc::mma_commit(drain);
      tc::mbar_wait(drain, 0u, P.err, kErrTrMma);
    }
  } else if (warp < 10) {
    // ------------------------------------------- queries, keys and values
    const bool is_key = warp < 6;
    const int w = warp & 3;                       // tensor-memory lane quarter
    const uint32_t lane_base = tbase + ((uint32_t)(32 * w) << 16);
    int it = 0, sets = 0, nd = 0;
    auto take = [&]() {                           // the next ring item has landed
      ok = tc::mbar_wait(&rawfull[it % NS], (uint32_t)((it / NS) & 1), P.err, kErrTrUnpack);
      ok = __all_sync(0xffffffffu, ok);
      return raw + (it % NS) * C::SLOT;
    };
    auto give = [&]() {                           // this warp is done with it
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&rawempty[it % NS]);
      ++it;
    };
    for (int i = 0; i < n && ok; ++i) {
      const TreeLayer& L = P.L[cur.li];
      const int type = tr_type(L, cur.j);
      const bool new_set = tr_new_set(L, i, cur.j);
      // the buffers of two tiles back are free: keys (and the queries of two sets back)
      // after that tile's first product, values after its second
      if (i >= 2) {
        const uint32_t par = (uint32_t)(((i >> 1) - 1) & 1);
        if (is_key || new_set) ok = tc::mbar_wait(&qkdone[i & 1], par, P.err, kErrTrUnpack);
        if (ok && !is_key) ok = tc::mbar_wait(&pvdone[i & 1], par, P.err, kErrTrUnpack);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      tc::fence_after_sync();
      if (new_set) {
        // rows of this segment into the K-major swizzled tile: bf16 as they are, or fp16
        // scaled to [1, 2) for packed tiles
        constexpr int E = D / 32;                 // channels per lane
        uint8_t* qd = dsm + C::oQ + (sets & 1) * C::QB;
        float* qs = s_qs + (sets & 7) * N;
        const int r0 = cur.rt * N;
        const __nv_bfloat16* src =
            P.q + (((size_t)cur.li * P.units + cur.unit) * P.rows + r0) * D + lane * E;
        const int c0 = lane * E;
#pragma unroll 2
        for (int r = warp - 2; r < N; r += 8) {
          uint32_t v[E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) v[e] = 0u;
          if (r0 + r < P.rows) {
            if constexpr (E == 4) {
              const uint2 x = *reinterpret_cast<const uint2*>(src + (size_t)r * D);
              v[0] = x.x;
              v[1] = x.y;
            } else {
              v[0] = *reinterpret_cast<const uint32_t*>(src + (size_t)r * D);
            }
          }
          float scale = P.sl2;
          if (type == kPacked) {
            uint32_t mx = 0u;                     // largest magnitude, as bf16 bits
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
              mx = max(mx, max(v[e] & 0x7fffu, (v[e] >> 16) & 0x7fffu));
            mx = __reduce_max_sync(0xffffffffu, mx);
            int ex = (int)(mx >> 7);
            ex = ex == 255 ? 127 : min(max(ex, 1), 253);
            const float f = __int_as_float((254 - ex) << 23);
            scale *= __int_as_float(ex << 23);
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
              v[e] = h2u(__floats2half2_rn(__int_as_float((int)(v[e] << 16)) * f,
                                           __int_as_float((int)(v[e] & 0xffff0000u)) * f));
          }
          uint8_t* dst = qd + (c0 >> 6) * N * 128 + r * 128 + ((((c0 & 63) >> 3) ^ (r & 7)) << 4) +
                         (c0 & 7) * 2;
          if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(v[0], v[1]);
          else *reinterpret_cast<uint32_t*>(dst) = v[0];
          if (lane == 0) qs[r] = scale;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&qfull[sets & 1]);
        ++sets;
      }
      if (is_key) {
        const uint32_t dst = lane_base + C::cK + (uint32_t)((i & 1) * (D / 2));
        const uint8_t* src = take();
        if (!ok) break;
        if (type == kPacked) {
          if (4 * cur.j + w < L.n_groups) {       // rows past the last group are masked
            if (L.bits == 2) keys_packed<D, 2>(src + w * block_bytes(D, 2), dst);
            else keys_packed<D, 4>(src + w * block_bytes(D, 4), dst);
          }
          give();
        } else {
          if (type == kWindow) keys_window<D>(src, 32 * w, dst);
          else if (w < 2) keys_draft<D, C::DP>(src, 32 * w, dst);
          give();
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&kfull[i & 1]);
        if (type != kPacked) {                    // the values' item
          take();
          if (!ok) break;
          give();
        }
      } else {
        const uint32_t dst = lane_base + C::cV + (uint32_t)((i & 1) * (kTrTile / 2));
        const bool on = 32 * w < D;
        const uint8_t* src = take();
        if (!ok) break;
        if (type == kPacked) {
          const int ng = min(4, L.n_groups - 4 * cur.j);
          if (on) {
#pragma unroll 1
            for (int gr = 0; gr < 4; ++gr) {
              if (gr >= ng) {                     // zero weights must not meet old contents
                uint32_t z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = 0u;
                tc::tmem_st_frag(dst + 16u * gr, z);
                tc::tmem_st_frag(dst + 16u * gr + (16u << 16), z);
              } else if (L.bits == 2) {
                values_packed<D, 2>(src + gr * block_bytes(D, 2), w, dst + 16u * gr);
              } else {
                values_packed<D, 4>(src + gr * block_bytes(D, 4), w, dst + 16u * gr);
              }
            }
          }
          give();
        } else {
          give();                                 // the keys' item
          src = take();
          if (!ok) break;
          if (type == kWindow) {
            if (on) values_window<D>(src, w, min(kTrTile, L.win_len - (cur.j - L.pt) * kTrTile), dst);
          } else {
            ok = tc::mbar_wait(&ancfull[nd & 3], (uint32_t)((nd >> 2) & 1), P.err, kErrTrUnpack);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const unsigned long long* anc = s_anc + (nd & 3) * kTrMaxNodes;
            ++nd;
            const unsigned long long live =
                (unsigned long long)__ballot_sync(0xffffffffu, anc[lane] != 0ull) |
                (unsigned long long)__ballot_sync(0xffffffffu, anc[lane + 32] != 0ull) << 32;
            if (on && values_draft<D, C::DP>(src, w, live, dst) && lane == 0) s_misc[4 + (nd & 3)] = (uint32_t)nd;
          }
          give();
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&vfull[i & 1]);
      }
      tr_step(P, cur);
    }
  } else {
    // ------------------------------------------------- softmax and output
    const int st = threadIdx.x - 10 * 32;         // 0 .. 255
    const int w = warp & 3, half = (warp - 10) >> 2;
    const int t = 32 * w + lane;                  // token of the tile; channel of the output
    const int col0 = half * CW;
    const uint32_t lane_base = tbase + ((uint32_t)(32 * w) << 16) + (uint32_t)col0;
    float lsum[CW];
    int sets = 0, nd = 0;
    if (st < N) s_nref[st] = INFINITY;            // no reference yet
    soft_bar();
    for (int i = 0; i < n; ++i) {
      const TreeLayer& L = P.L[cur.li];
      const int type = tr_type(L, cur.j);
      const bool fresh = i == 0 || cur.j == 0;
      if (fresh) {
#pragma unroll
        for (int c = 0; c < CW; ++c) lsum[c] = 0.f;
      }
      if (tr_new_set(L, i, cur.j)) ++sets;
      const float* qs = s_qs + ((sets - 1) & 7) * N + col0;
      const float* nref = s_nref + col0;
      // columns of this thread's token that see it
      uint32_t vis = 0xffffffffu;
      const unsigned long long* anc = nullptr;
      const int r0 = cur.rt * N + col0;
      if (type == kPacked) {
        if (t >= 32 * (L.n_groups - 4 * cur.j)) vis = 0u;
      } else if (type == kWindow) {
        if (t >= L.win_len - (cur.j - L.pt) * kTrTile) vis = 0u;
      } else {
        if (ok) ok = tc::mbar_wait(&ancfull[nd & 3], (uint32_t)((nd >> 2) & 1), P.err, kErrTrSoftmax);
        anc = s_anc + (nd & 3) * kTrMaxNodes;
        ++nd;
        vis = 0u;
        if (t < P.T) {
          int node = r0 % P.T;
#pragma unroll 1
          for (int c = 0; c < CW; ++c) {
            if (r0 + c < P.rows && ((anc[node] >> t) & 1ull)) vis |= 1u << c;
            if (++node == P.T) node = 0;
          }
        }
      }
      if (ok) ok = tc::mbar_wait(&qkdone[i & 1], (uint32_t)((i >> 1) & 1), P.err, kErrTrSoftmax);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      // logits against the reference, log2 units; a token a row does not see: -inf
      const uint32_t scol = lane_base + C::cS + (uint32_t)((i & 1) * N);
      float y[CW];
      {
        uint32_t x[CW];
        tc::tmem_ld(scol, x);
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < CW; c += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(qs + c);
          const float4 n4 = *reinterpret_cast<const float4*>(nref + c);
          const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                                      make_float2(s4.x, s4.y), make_float2(n4.x, n4.y));
          const float2 b = __ffma2_rn(make_float2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])),
                                      make_float2(s4.z, s4.w), make_float2(n4.z, n4.w));
          y[c] = a.x; y[c + 1] = a.y; y[c + 2] = b.x; y[c + 3] = b.y;
        }
        if (vis != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < CW; ++c) y[c] = (vis >> c) & 1u ? y[c] : -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < CW; ++c) top = fmaxf(top, y[c]);
        // some row has no reference yet or is past it: new references for such rows
        if (soft_bar_any(top > kTrSlack)) {
          tc::tmem_ld(scol, x);
#pragma unroll
          for (int c = 0; c < CW; ++c) {
            float m = (vis >> c) & 1u ? __uint_as_float(x[c]) * qs[c] : -INFINITY;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) s_red[w * N + col0 + c] = m;
          }
          soft_bar();
          float nw = -INFINITY, corr = 1.f;       // of column col0 + lane
          if (lane < CW) {
            float m = s_red[col0 + lane];
#pragma unroll
            for (int k = 1; k < 4; ++k) m = fmaxf(m, s_red[k * N + col0 + lane]);
            const float old = -nref[lane];
            nw = (old == -INFINITY || m > old + kTrSlack) ? m : old;
            corr = nw == old ? 1.f : exp2f(old - nw);
          }
          soft_bar();
          if (w == 0 && lane < CW) s_nref[col0 + lane] = -nw;
#pragma unroll
          for (int c = 0; c < CW; ++c) {
            const float r = __shfl_sync(0xffffffffu, nw, c);
            const float v = fmaf(__uint_as_float(x[c]), qs[c], r == -INFINITY ? 0.f : -r);
            y[c] = (vis >> c) & 1u ? v : -INFINITY;
          }
          if (!fresh && __any_sync(0xffffffffu, corr != 1.f)) {
            // the output so far is at rest: rescale it (whole-warp loads and stores)
            if (ok) ok = tc::mbar_wait(&pvdone[(i - 1) & 1], (uint32_t)(((i - 1) >> 1) & 1), P.err, kErrTrSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            tc::tmem_ld(lane_base + C::cO, x);
#pragma unroll
            for (int c = 0; c < CW; ++c) {
              const float f = __shfl_sync(0xffffffffu, corr, c);
              x[c] = __float_as_uint(__uint_as_float(x[c]) * f);
              lsum[c] *= f;
            }
            tc::tmem_st(lane_base + C::cO, x);
            tc::tmem_wait_st();
          }
          soft_bar();                             // the references are in place
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sempty[i & 1]);
      uint32_t pk[CW / 2];
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        y[c] = fast_exp2(y[c]);
        lsum[c] += y[c];
      }
      if (type == kPacked) {
#pragma unroll
        for (int c = 0; c < CW; c += 2) pk[c / 2] = h2u(__floats2half2_rn(y[c], y[c + 1]));
      } else {
#pragma unroll
        for (int c = 0; c < CW; c += 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(y[c], y[c + 1]);
          pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      // the weights' buffer of two tiles back has been consumed
      if (ok && i >= 2)
        ok = tc::mbar_wait(&pvdone[i & 1], (uint32_t)(((i >> 1) - 1) & 1), P.err, kErrTrSoftmax);
      ok = __all_sync(0xffffffffu, ok);
      uint8_t* prow = dsm + C::oP + (i & 1) * C::PB + t * 128;
#pragma unroll
      for (int c8 = 0; c8 < CW / 8; ++c8)
        *reinterpret_cast<uint4*>(prow + (((col0 / 8 + c8) ^ (t & 7)) << 4)) =
            make_uint4(pk[4 * c8], pk[4 * c8 + 1], pk[4 * c8 + 2], pk[4 * c8 + 3]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&pfull[i & 1]);

      if (i == n - 1 || cur.j == L.tps - 1) {
        // ---------------------------------------- the segment's part ends here
        const long long sbeg = C0 + i - cur.j, send = sbeg + L.tps;
        const bool whole = sbeg >= C0 && send <= C1;
        const size_t ul = (size_t)cur.li * P.units + cur.unit;
        const int rbase = cur.rt * N, nrow = min(N, P.rows - rbase);
        if (ok) ok = tc::mbar_wait(&pvdone[i & 1], (uint32_t)((i >> 1) & 1), P.err, kErrTrSoftmax);
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
        uint32_t o[CW];
        tc::tmem_ld(lane_base + C::cO, o);
        tc::fence_before_sync();
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          float v = lsum[c];
#pragma unroll
          for (int k = 16; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
          if (lane == 0) s_red[w * N + col0 + c] = v;
        }
        soft_bar();
        const bool bad = type == kDraft && s_misc[4 + (nd & 3)] == (uint32_t)nd;
        const __nv_bfloat16* vd = P.v_draft + ul * P.T * D;
        float* part = P.ws + ((size_t)blockIdx.x * 2 + (max(sbeg, C0) == C0 ? 0 : 1)) * C::STATE;
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          const int col = col0 + c;
          if (col < nrow) {
            float l = s_red[col] + s_red[N + col] + s_red[2 * N + col] + s_red[3 * N + col];
            float v = __uint_as_float(o[c]);
            if (type == kDraft) {
              unsigned long long path = anc[(rbase + col) % P.T];
              if (path == 0ull) l = -1.f;         // padding
              while (bad && path) {               // values that are not finite
                const int j = __ffsll((long long)path) - 1;
                path &= path - 1;
                const float z = t < D ? __bfloat162float(vd[(size_t)j * D + t]) : 0.f;
                if (!isfinite(z)) v += z;
              }
            }
            if (whole) {
              if (ok && t < D)
                P.out[(ul * P.rows + rbase + col) * D + t] = __float2bfloat16(l == -1.f ? 0.f : v / l);
            } else {
              if (t < D) part[col * D + t] = v;
              if (t == 0) {
                part[N * D + col] = -s_nref[col];
                part[N * D + N + col] = l;
              }
            }
          }
        }
        if (!whole) {
          __threadfence();
          soft_bar();
          const long long ca = cs.owner(sbeg), cb = cs.owner(send - 1);
          const int nc = (int)(cb - ca + 1);
          unsigned* cnt = P.cnt + ((size_t)(P.layer_begin + cur.li) * P.units + cur.unit) * P.RT + cur.rt;
          if (st == 0) s_misc[1] = atomicAdd(cnt, 1u) == (unsigned)(nc - 1);
          soft_bar();
          if (s_misc[1]) {
            __threadfence();
            const bool late = cs.first(ca) < sbeg;   // the first holder's segment is its last
            auto part_of = [&](int k) -> const float* {
              return P.ws + ((size_t)(ca + k) * 2 + ((k == 0 && late) ? 1 : 0)) * C::STATE;
            };
            // maximum and 1 / sum per row (0: padding)
            if (st < nrow) {
              float M = -INFINITY, l = 0.f;
              bool pad = false;
              for (int k = 0; k < nc; ++k) {
                const float lk = __ldcg(part_of(k) + N * D + N + st);
                if (lk == -1.f) pad = true;
                else if (lk != 0.f) M = fmaxf(M, __ldcg(part_of(k) + N * D + st));
              }
              for (int k = 0; k < nc; ++k) {
                const float lk = __ldcg(part_of(k) + N * D + N + st);
                if (lk != 0.f) l += lk * exp2f(__ldcg(part_of(k) + N * D + st) - M);
              }
              s_red[st] = M;
              s_red[N + st] = pad ? 0.f : 1.f / l;
            }
            soft_bar();
            for (int idx = st; idx < nrow * (D / 4); idx += kTrSoftThreads) {
              const int row = idx / (D / 4), c4 = idx % (D / 4);
              const float M = s_red[row], inv = s_red[N + row];
              float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
              for (int k = 0; k < nc; ++k) {
                const float* pk2 = part_of(k);
                const float lk = __ldcg(pk2 + N * D + N + row), mk = __ldcg(pk2 + N * D + row);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(pk2 + row * D) + c4);
                const float f = lk != 0.f ? exp2f(mk - M) : 0.f;
                if (lk != 0.f) { a.x += f * v.x; a.y += f * v.y; a.z += f * v.z; a.w += f * v.w; }
              }
              if (inv == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);
              const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * inv, a.y * inv),
                                   hi = __floats2bfloat162_rn(a.z * inv, a.w * inv);
              if (ok)
                *reinterpret_cast<uint2*>(P.out + (ul * P.rows + rbase + row) * D + 4 * c4) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                               *reinterpret_cast<const uint32_t*>(&hi));
            }
            if (st == 0) *cnt = 0u;               // ready for the next launch
          }
        }
        soft_bar();
        if (st < N) s_nref[st] = INFINITY;
        soft_bar();
      }
      tr_step(P, cur);
    }
  }

  // teardown: every product has completed (the issuing thread drained them)
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, kTrTmemCols);
  }
}

// Rows of a row tile: 16, 32 or 64 columns of the products. Fewer columns cost less (the
// unpacking does not depend on them); beyond 64 the rows take another tile.
int tree_cols(int rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64); }

template <int D, int N>
cudaError_t launch_tree_cols(const TreeParams& P, int n_sm, cudaStream_t stream) {
  using C = TrCfg<D, N>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(tree_kernel<D, N>), C::total);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(n_sm, P.total));
  cfg.blockDim = dim3(kTrThreads);
  cfg.dynamicSmemBytes = C::total;
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attr()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_kernel<D, N>, P);
}

}  // namespace

size_t tree_workspace_floats(const kvc_cache* c) {
  return (size_t)2 * c->n_sm * 64 * (c->dims.head_dim + 2);
}
size_t tree_tickets(const kvc_cache* c) {
  return (size_t)c->dims.n_layers * c->dims.batch * c->dims.n_kv_heads *
         ((c->g * kTrMaxNodes + 63) / 64);
}

cudaError_t launch_tree(const kvc_cache* c, int layer_begin, int layer_count, int T,
                        const int32_t* parents, const __nv_bfloat16* q,
                        const __nv_bfloat16* k_draft, const __nv_bfloat16* v_draft,
                        __nv_bfloat16* out, cudaStream_t stream) {
  const kvc_dims& d = c->dims;
  const int units = d.batch * d.n_kv_heads, D = d.head_dim;
  const int rows = c->g * T, N = tree_cols(rows);
  for (int base = 0; base < layer_count; base += KVC_MAX_LAUNCH_LAYERS) {
    const int cnt = std::min(layer_count - base, KVC_MAX_LAUNCH_LAYERS);
    TreeParams P;
    P.packed = c->packed;
    P.win_k = c->win_k;
    P.win_v = c->win_v;
    P.parents = parents;
    const size_t kvn = (size_t)base * units * T * D;
    P.q = q + kvn * c->g;
    P.out = out + kvn * c->g;
    P.k_draft = k_draft + kvn;
    P.v_draft = v_draft + kvn;
    P.ws = c->tree_ws;
    P.cnt = c->tree_cnt;
    P.err = c->err;
    P.n_layers = cnt;
    P.layer_begin = layer_begin + base;
    P.units = units;
    P.H = d.n_kv_heads;
    P.T = T;
    P.rows = rows;
    P.RT = (rows + N - 1) / N;
    P.sl2 = 1.4426950408889634f / sqrtf((float)D);
    long long total = 0;
    for (int i = 0; i < cnt; ++i) {
      const LayerState& ls = c->L[layer_begin + base + i];
      TreeLayer& L = P.L[i];
      L.tile_begin = total;
      L.packed_off = (long long)ls.packed_off;
      L.win_off = (long long)ls.win_off;
      L.n_groups = ls.n_groups;
      L.cap_groups = ls.cap_groups;
      L.bits = ls.bits;
      L.win_start = ls.win_start;
      L.win_len = ls.win_len;
      L.R = ls.R;
      L.pt = (ls.n_groups + 3) / 4;
      L.wt = (ls.win_len + kTrTile - 1) / kTrTile;
      L.tps = L.pt + L.wt + 1;
      total += (long long)units * P.RT * L.tps;
    }
    P.total = total;
    cudaError_t e;
    if (D == 128)
      e = N == 16 ? launch_tree_cols<128, 16>(P, c->n_sm, stream)
                  : (N == 32 ? launch_tree_cols<128, 32>(P, c->n_sm, stream)
                             : launch_tree_cols<128, 64>(P, c->n_sm, stream));
    else
      e = N == 16 ? launch_tree_cols<64, 16>(P, c->n_sm, stream)
                  : (N == 32 ? launch_tree_cols<64, 32>(P, c->n_sm, stream)
                             : launch_tree_cols<64, 64>(P, c->n_sm, stream));
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace kvc
