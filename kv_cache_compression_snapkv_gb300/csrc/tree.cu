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
// once, to 2^-11 of itself, an eighth of what bf16 would lose. The queries meet them as fp16
// scaled per row by a power of two to [1, 2) (elements below 2^-14 of the row's largest keep
// 2^-25 of it), the weights as fp16. Z + (2^b - 1) S may pass fp16's range, by less than 16
// times (S and Z are inside). The quantizer marks the units that store such a group: their
// scales and zero-points, and the window's and the drafted values, are taken by 2^-4 as they
// arrive, their queries by 2^4 and the sums of their rows by 2^-4 (packed elements below 2^-10
// are then rounded to 2^-21, 2^-37 of the largest there is; 160 units of 32,768 tokens, all
// marked: 397 us, none: 197 us; 8 units of 131,072, 256 rows: 351 and 258 us).
// Window and drafted tokens are bf16 as they are, against bf16 queries and weights.
// Logits, the running maximum, sums and outputs are fp32; the output is rounded to bf16.
// The reference a row's weights are taken against lies 7 below the logit it comes from (log2
// units) and is raised when a logit passes that one by 8, each row by itself: weights stay below
// 2^15, inside fp16, and the smallest that fp16 holds (2^-24, to half of that) is 2^-32 of the
// largest: what many far tokens add up to beside a dominant one is kept (n tokens are off by
// n 2^-32 of the largest value at most). The row sums add the weights before their rounding.
//
// Work. A unit's rows are cut into row tiles (of N rows); a (layer, unit, row tile) is a
// segment of tiles of 128 tokens: four packed groups each, then the window, then the
// drafted tokens. The tiles of all segments are laid end to end and cut into one
// contiguous range per CTA (tree_grid says how many). A segment that lies in several CTAs is
// handed over as partial states (o, m, l) in global memory and merged by the CTA that arrives
// last (a ticket; nothing waits), in a fixed order.
//
// Roles. Warp 0: bulk copies of raw tiles into rings and the ancestor sets of the drafted nodes;
// 1 and 2: the products; then four warps of keys (one group of the tile each) and four of
// values (one 32-channel group each) into tensor memory, and the queries; then softmax (lane
// quarter = warp % 4, CW columns), output and merge. Up to 32 columns there are two sets of
// unpacking and softmax warps, for the even and the odd tiles. Every wait is bounded.
//
// What bounds it: the chain from raw tile to unpacked operand, first product, softmax and second
// product. A pipeline of 16 columns has its unpacking and softmax warps busy three quarters of
// the time, each instruction stretched by the other roles of the scheduler (issue is active 68 %
// of the time, a quarter of that in waits); the tensor pipe is active 23 % at 64 columns. Half of
// the instructions that are not waits turn codes into fp16: one logic instruction, one subtraction
// and one fused multiply-add per pair of codes. Measured: 32,768 tokens at 4 bits, 160 units of 16
// rows, 842 MB: 197 us, 4.3 TB/s (a copy of the bytes alone 124 us); 131,072 tokens at 2 bits,
// 8 units of 256 rows: 258 us, 534 TFLOP/s (the cache is unpacked once for each 64 rows); 544
// tokens, 8 units of 104 rows: 17.0 us, the latency of the launch, of one tile and of the merge.
#include "decode_device.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr uint32_t kTrTmemCols = 512;
constexpr int kTrTile = 128;          // tokens of a tile
// One poll of a wait sleeps this long at most, and a wait gives up after so many: a second or so
// at most. (Polls without the sleep, or with naps of 20 to 200 ns between them: the same time to 1 %.)
constexpr unsigned kTrPollNs = 20000, kTrPolls = 1u << 16;
constexpr float kTrLift = 7.f;        // a row's reference lies this far below the logit it comes from
constexpr float kTrSlack = kTrLift + 8.f;   // and is raised when passed by this (2^15 fits fp16)
constexpr float kTrUnset = 3e38f;     // minus the reference of a row that has none yet
constexpr float kTrBig = 0x1p16f;     // references past this are met unfused
constexpr int kTrMaxNodes = KVC_MAX_TREE_NODES;
// Ancestor sets and their barriers in flight. The producer writes the set of drafted tile k with
// the slots of tile k - 1 granted, over that of tile k - kTrAnc, whose segment must be over (its
// output reads it). The closest case is a segment of the drafted tile alone (a layer that holds
// no token) at head dimension 64 and up to 32 columns: a group's ring of four slots holds two
// tiles, so an item of tile k - 5 at least has been given back, whose values waited for the second
// product of three tiles before, k - 8; the softmax warps formed that tile's weights after they
// had all left the segment before it, k - 9. So nine sets would do (tests/test_tree_split_replay.py
// looks this up in the graph of all waits; with eight, tile k - 8's output could still read its
// own set); 16 keeps the index a mask.
constexpr int kTrAnc = 16;
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
  const unsigned* wide;           // the cache's marks [layer][unit][kMarkWords]
  long long total;                // tiles of the launch
  unsigned wait_limit;            // polls of one wait before it gives up
  int n_layers, layer_begin, units, H, T, rows, RT;
  float sl2;
};

template <int D, int N>
struct TrCfg {
  // Up to 32 columns the even and the odd tiles of a segment are two pipelines with warps,
  // references, sums and outputs of their own, joined at the segment's end: each is a chain
  // of latencies, and one runs while the other waits. At 64 columns there is one, with four
  // times the softmax warps of a 16-column one.
  static constexpr int NP = N == 64 ? 1 : 2;        // pipelines
  static constexpr int G = NP;                      // groups of unpacking warps
  // Buffers of keys and of values in tensor memory, taken in turn. With two, each pipeline has one
  // of its own and unpacks values only after the second product of its tile before.
  // (160 units of 32,768 tokens at 4 bits: 16 rows 204 us with two, 194 us with three, 32 rows
  // 229 and 218 us.) With three, keys and values have barriers of their own; with two, those of
  // the logits' and the weights' buffers serve them too (64 rows: 316 us, apart 320 us).
  static constexpr int NB = N == 64 ? 2 : 3;
  static constexpr bool kApart = NB != 2;
  static constexpr int CW = N == 32 ? 32 : 16;      // columns of one softmax warp
  static constexpr int SW = 4 * (N / CW);           // softmax warps of a pipeline
  static constexpr int kSoftAll = NP * SW * 32;     // threads of all softmax warps
  static constexpr int kThreads = (4 + 8 * G + NP * SW) * 32;
  // Registers. The block starts with R0 a thread (its warps spread evenly over the four
  // schedulers); its warpgroups share them out anew: copies and products, keys and values,
  // softmax. The sum may not pass the block's own (a warpgroup would wait for registers that
  // never come). All six forms spill (292 to 452 bytes of stores a thread), nearly all outside
  // of the loops over tiles: of the instructions executed over 131,072 tokens at 64 columns
  // 0.9 % are loads or stores of spilled registers.
  static constexpr int WG = kThreads / 128;
  static constexpr int R0 = 65536 / kThreads / 8 * 8;
  static constexpr int kRegsIssue = 48, kRegsUnpack = 64, kRegsSoft = N == 32 ? 96 : 80;
  static_assert(kRegsIssue + 2 * G * kRegsUnpack + (NP * SW / 4) * kRegsSoft <= WG * R0 &&
                R0 > kRegsUnpack && R0 < kRegsSoft, "the warpgroups' registers");
  static constexpr int SLOT = kTrTile * D * 2;      // raw ring slot: 128 window keys or values
  static constexpr int NS = D == 128 ? 4 : 8;
  static constexpr int RS = NS / G;                 // slots of a group's ring
  static constexpr int DP = 2 * D + 16;             // row pitch of staged drafted tokens
  static constexpr int QB = N * D * 2;
  static constexpr int PB = kTrTile * 128;          // weights: 128 tokens x 64 rows, 16 bits
  static constexpr int oRaw = 0;
  static constexpr int oQ = oRaw + NS * SLOT;       // [2]
  static constexpr int oP = oQ + 2 * QB;            // [2]
  static constexpr int oQs = oP + 2 * PB;           // [8][N] logit scale per query set and row
  static constexpr int oRef = oQs + 8 * N * 4;      // [NP][N] minus the rows' reference
  static constexpr int oRed = oRef + NP * N * 4;    // [NP][4][N]
  static constexpr int oCorr = oRed + NP * 4 * N * 4;   // [NP][N] factors
  static constexpr int oSum = oCorr + NP * N * 4;   // [N] sums
  static constexpr int oAnc = oSum + N * 4;         // [kTrAnc][64] ancestor sets (0: padding)
  static constexpr int oBar = oAnc + kTrAnc * kTrMaxNodes * 8;
  static constexpr int NBAR = 2 * NS + 10 + 4 * NB + kTrAnc + 2;
  static constexpr int oMisc = oBar + NBAR * 8;     // tensor memory base, flags
  static constexpr int mMark = 4 + kTrAnc;          // word of oMisc: [8] the unit's mark by query set
  static constexpr int total = oMisc + (mMark + 8) * 4 + 1024;   // + alignment slack
  static constexpr int STATE = N * (D + 2);         // floats of one partial state
  // tensor memory columns
  static constexpr uint32_t cK = 0, cV = NB * (D / 2), cS = cV + NB * (kTrTile / 2), cO = cS + 2 * N;
  static_assert(cO + NP * N <= kTrTmemCols, "tensor memory");
  static_assert(kTrMaxNodes * DP <= SLOT && 4 * block_bytes(D, 4) <= SLOT, "ring slot");
  static_assert(SLOT % 1024 == 0 && QB % 1024 == 0 && PB % 1024 == 0, "1024-byte aligned");
  static_assert(total <= 227 * 1024, "shared memory");
};

// Position in the list of tiles, with the fields of the layer that every tile needs (read
// from the kernel's parameters when the layer changes only: an indexed read of constant
// memory takes longer than some roles spend on a tile).
struct TrCur {
  int li, unit, rt, j;
  int pt, wt, tps, n_groups, win_len, bits;
  __device__ __forceinline__ void layer(const TreeParams& P) {
    const TreeLayer& L = P.L[li];
    pt = L.pt;
    wt = L.wt;
    tps = L.tps;
    n_groups = L.n_groups;
    win_len = L.win_len;
    bits = L.bits;
  }
  __device__ __forceinline__ void locate(const TreeParams& P, long long c) {
    li = 0;
    while (li + 1 < P.n_layers && c >= P.L[li + 1].tile_begin) ++li;
    layer(P);
    const long long loc = c - P.L[li].tile_begin;
    long long seg;
    if (loc >> 32) {
      seg = loc / tps;
      unit = (int)(seg / P.RT);
    } else {                                      // 32-bit divisions
      seg = (unsigned)loc / (unsigned)tps;
      unit = (int)((unsigned)seg / (unsigned)P.RT);
    }
    j = (int)(loc - seg * tps);
    rt = (int)(seg - (long long)unit * P.RT);
  }
  __device__ __forceinline__ void step(const TreeParams& P) {
    if (++j < tps) return;
    j = 0;
    if (++rt < P.RT) return;
    rt = 0;
    if (++unit < P.units) return;
    unit = 0;
    if (++li < P.n_layers) layer(P);
  }
  // to the first tile of the next segment
  __device__ __forceinline__ void next_segment(const TreeParams& P) {
    j = tps - 1;
    step(P);
  }
};

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

// The keys of one packed group into tensor memory (32 lanes = tokens, d / 2 columns). Rolled
// over 64 channels: the roles run side by side and share the instruction caches, and the
// warp has few registers.
template <int D, int BITS>
__device__ __forceinline__ void keys_packed(const uint8_t* blk, uint32_t dst,
                                            const CodeMasks<BITS>& cm) {
  constexpr int KS = D / 16, W = BITS;             // code words of a lane per 16 tokens x 64 channels
  const int lane = threadIdx.x & 31, tid = lane & 3;
  const uint4* sp = reinterpret_cast<const uint4*>(blk + off_kscale(D, BITS) + tid * (D / 4) * 2);
  const uint8_t* wp = blk + lane * 16;
#pragma unroll 1
  for (int kh = 0; kh < KS; kh += 4) {
    uint32_t S[4][2], Z[4][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 s = sp[kh / 2 + i], z = sp[kh / 2 + i + 2 * D / 16];
      S[2 * i][0] = s.x; S[2 * i][1] = s.y; S[2 * i + 1][0] = s.z; S[2 * i + 1][1] = s.w;
      Z[2 * i][0] = z.x; Z[2 * i][1] = z.y; Z[2 * i + 1][0] = z.z; Z[2 * i + 1][1] = z.w;
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t kw[W];
      const int wi = mt * (KS * BITS / 4) + kh * BITS / 4;   // first word, in the lane's order
      const uint8_t* p = wp + (wi >> 2) * 512 + (wi & 3) * 4;
      if constexpr (W == 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        kw[0] = w.x; kw[1] = w.y; kw[2] = w.z; kw[3] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        kw[0] = w.x; kw[1] = w.y;
      }
      uint32_t r[16];
      static_for<4>([&](auto K_) {
        constexpr int k = decltype(K_)::value;
        uint32_t a[4];
        key_afrag<D, BITS, 0, k>(kw, cm, a);
        r[4 * k] = hfma2u(a[0], S[k][0], Z[k][0]);
        r[4 * k + 1] = hfma2u(a[1], S[k][0], Z[k][0]);
        r[4 * k + 2] = hfma2u(a[2], S[k][1], Z[k][1]);
        r[4 * k + 3] = hfma2u(a[3], S[k][1], Z[k][1]);
      });
      tc::tmem_st_frag(dst + 8u * kh + ((uint32_t)(16 * mt) << 16), r);
    }
  }
}

// What a warp holds of the values of channels 32 w .. 32 w + 31 of one packed group.
struct ValueRegs {
  uint32_t wd[4], sa[2], sb[2], z[2][2];
};
template <int D, int BITS>
__device__ __forceinline__ void values_load(const uint8_t* blk, int w, ValueRegs& v) {
  constexpr int NGC = D / 32;
  const int lane = threadIdx.x & 31, tid = lane & 3;
  if constexpr (BITS == 4) {
    const uint4 x = reinterpret_cast<const uint4*>(blk + off_vcodes(D, BITS))[w * 32 + lane];
    v.wd[0] = x.x; v.wd[1] = x.y; v.wd[2] = x.z; v.wd[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(blk + off_vcodes(D, BITS) + (w >> 1) * 512 +
                                                    lane * 16 + (w & 1) * 8);
    v.wd[0] = x.x; v.wd[1] = x.y; v.wd[2] = 0u; v.wd[3] = 0u;
  }
  const uint32_t* vs = reinterpret_cast<const uint32_t*>(blk + off_vscale(D, BITS));
  const uint32_t* vz = reinterpret_cast<const uint32_t*>(blk + off_vzero(D, BITS));
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    v.sa[ks] = vs[(8 * ks + 2 * tid) * NGC + w];
    v.sb[ks] = vs[(8 * ks + 2 * tid + 1) * NGC + w];
    v.z[ks][0] = vz[(8 * ks + tid) * NGC + w];
    v.z[ks][1] = vz[(8 * ks + 4 + tid) * NGC + w];
  }
}
template <int BITS>
__device__ __forceinline__ void values_store(const ValueRegs& v, uint32_t dst,
                                             const CodeMasks<BITS>& cm) {
  static_for<2>([&](auto H_) {
    constexpr int h = decltype(H_)::value;
    uint32_t r[8];
    static_for<2>([&](auto K_) {
      constexpr int ks = decltype(K_)::value;
      // scales of (t, t + 8) and (t + 1, t + 9), t = 16 ks + 2 tid, regrouped by token pair
      const uint32_t s0 = __byte_perm(v.sa[ks], v.sb[ks], 0x5410);
      const uint32_t s1 = __byte_perm(v.sa[ks], v.sb[ks], 0x7632);
      uint32_t a[4];
      if constexpr (BITS == 4) {
        const uint32_t x = v.wd[2 * h + ks], x8 = x >> 8;
        a[0] = unpack_pair<4, 0>(x, x8, cm);
        a[1] = unpack_pair<4, 2>(x, x8, cm);
        a[2] = unpack_pair<4, 1>(x, x8, cm);
        a[3] = unpack_pair<4, 3>(x, x8, cm);
      } else {
        const uint32_t x = v.wd[h], x8 = x >> 8;
        a[0] = unpack_pair<2, 2 * ks>(x, x8, cm);
        a[1] = unpack_pair<2, 4 + 2 * ks>(x, x8, cm);
        a[2] = unpack_pair<2, 2 * ks + 1>(x, x8, cm);
        a[3] = unpack_pair<2, 5 + 2 * ks>(x, x8, cm);
      }
      r[4 * ks] = hfma2u(a[0], s0, v.z[ks][0]);
      r[4 * ks + 1] = hfma2u(a[1], s0, v.z[ks][0]);
      r[4 * ks + 2] = hfma2u(a[2], s1, v.z[ks][1]);
      r[4 * ks + 3] = hfma2u(a[3], s1, v.z[ks][1]);
    });
    tc::tmem_st_frag(dst + ((uint32_t)(16 * h) << 16), r);
  });
}
// The values of channels 32 w .. + 31 of a packed tile's ng groups (lanes = channels, 16
// columns a group), two groups at a time.
template <int D, int BITS>
__device__ __forceinline__ void values_packed(const uint8_t* raw, int w, int ng, uint32_t dst,
                                              const CodeMasks<BITS>& cm) {
  constexpr int BB = block_bytes(D, BITS);
  ValueRegs a, b;
  if (ng == 4) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h, raw += 2 * BB, dst += 32u) {
      values_load<D, BITS>(raw, w, a);
      values_load<D, BITS>(raw + BB, w, b);
      values_store<BITS>(a, dst, cm);
      values_store<BITS>(b, dst + 16u, cm);
    }
    return;
  }
#pragma unroll 1
  for (int gr = 0; gr < 4; ++gr, dst += 16u) {    // the last tile
    if (gr < ng) {
      values_load<D, BITS>(raw + gr * BB, w, a);
      values_store<BITS>(a, dst, cm);
    } else {                                      // zero weights must not meet old contents
      const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      tc::tmem_st_frag(dst, z);
      tc::tmem_st_frag(dst + (16u << 16), z);
    }
  }
}

// 32 window keys (rows row0 .. row0 + 31 of the staged tile).
template <int D>
__device__ __forceinline__ void keys_window(const uint8_t* raw, int row0, uint32_t dst) {
  constexpr int KS = D / 16;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
#pragma unroll 1
  for (int mt = 0; mt < 2; ++mt) {
    const uint4* r0 = reinterpret_cast<const uint4*>(raw + (size_t)(row0 + 16 * mt + gid) * D * 2);
    const uint4* r1 = reinterpret_cast<const uint4*>(raw + (size_t)(row0 + 16 * mt + gid + 8) * D * 2);
#pragma unroll 1
    for (int kh = 0; kh < KS; kh += 4) {
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ch = (tid * (KS / 2) + kh / 2 + i) ^ gid;
        const uint4 a = r0[ch], b = r1[ch];
        r[8 * i] = a.x; r[8 * i + 1] = b.x; r[8 * i + 2] = a.y; r[8 * i + 3] = b.y;
        r[8 * i + 4] = a.z; r[8 * i + 5] = b.z; r[8 * i + 6] = a.w; r[8 * i + 7] = b.w;
      }
      tc::tmem_st_frag(dst + 8u * kh + ((uint32_t)(16 * mt) << 16), r);
    }
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
#pragma unroll 1
  for (int k2 = 0; k2 < 8; k2 += 2) {
    uint32_t r0[8], r1[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int ks = k2 + k, ch = (gid * (D / 32) + w) ^ tid;
      const uint4 a = reinterpret_cast<const uint4*>(raw + (size_t)(8 * ks + tid) * D * 4)[ch];
      const uint4 b = reinterpret_cast<const uint4*>(raw + (size_t)(8 * ks + 4 + tid) * D * 4)[ch];
      const uint32_t ma = keep_pair(16 * ks + 2 * tid, n), mb = keep_pair(16 * ks + 8 + 2 * tid, n);
      r0[4 * k] = a.x & ma; r0[4 * k + 1] = a.y & ma; r0[4 * k + 2] = b.x & mb; r0[4 * k + 3] = b.y & mb;
      r1[4 * k] = a.z & ma; r1[4 * k + 1] = a.w & ma; r1[4 * k + 2] = b.z & mb; r1[4 * k + 3] = b.w & mb;
    }
    tc::tmem_st_frag(dst + 8u * k2, r0);
    tc::tmem_st_frag(dst + 8u * k2 + (16u << 16), r1);
  }
}

// 32 drafted keys (rows row0 .. of the staged tile, pitch DP).
template <int D, int DP>
__device__ __forceinline__ void keys_draft(const uint8_t* raw, int row0, uint32_t dst) {
  constexpr int KS = D / 16;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int mt = 0; mt < 2; ++mt) {
    const uint32_t a0 = tc::saddr(raw) + (uint32_t)((row0 + 16 * mt + (lane & 15)) * DP + (lane >> 4) * 16);
#pragma unroll 1
    for (int kh = 0; kh < KS; kh += 4) {
      uint32_t r[16];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ldsm4(a0 + 32u * (kh + k), r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
      tc::tmem_st_frag(dst + 8u * kh + ((uint32_t)(16 * mt) << 16), r);
    }
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
#pragma unroll 1
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

template <int R>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(R));
}
template <int R>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(R));
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// v[c] of every lane combined over the warp's lanes: lane l gets column l * W / 32's value
// (W columns, a power of two up to 32; W / 2 + W / 4 + ... exchanges instead of 5 W).
template <int W, typename Op>
__device__ __forceinline__ float reduce_columns(float (&v)[W], Op op) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int half = W / 2; half >= 1; half >>= 1, o >>= 1) {
    const bool high = (lane & o) != 0;
#pragma unroll
    for (int c = 0; c < half; ++c) {
      const float give = high ? v[c] : v[c + half], keep = high ? v[c + half] : v[c];
      v[c] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  float r = v[0];
#pragma unroll
  for (; o; o >>= 1) r = op(r, __shfl_xor_sync(0xffffffffu, r, o));
  return r;
}

// Bounded wait for the phase of parity `parity`; false (and `errbit` in the error word) after
// `limit` polls.
__device__ __noinline__ bool tr_gave_up(unsigned* err, unsigned errbit) {
  atomicOr(err, errbit);
  return false;
}
__device__ __forceinline__ bool tr_wait(uint32_t bar, uint32_t parity, unsigned limit, unsigned* err,
                                        unsigned errbit) {
#pragma unroll 1
  for (unsigned it = 0; it < limit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(bar), "r"(parity), "r"(kTrPollNs) : "memory");
    if (done) return true;
  }
  return tr_gave_up(err, errbit);
}
__device__ __forceinline__ void tr_init(uint32_t bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void tr_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void tr_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
               :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tr_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void tr_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :: "r"(bar) : "memory");
}

// Named barrier of W threads; `any`: whether p holds in one of them.
template <int W>
__device__ __forceinline__ void soft_sync(int id) {
  asm volatile("barrier.cta.sync %0, %1;" :: "r"(id), "n"(W) : "memory");
}
template <int W>
__device__ __forceinline__ bool soft_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r) : "r"((uint32_t)p), "r"(id), "n"(W) : "memory");
  return r != 0u;
}

// A logit against its row's reference.
__device__ __forceinline__ float less_ref(float x, float scale, float nref) {
  return fabsf(nref) > kTrBig ? __fadd_rn(__fmul_rn(x, scale), nref) : __fmaf_rn(x, scale, nref);
}

template <int D, int N>
__global__ void __launch_bounds__(TrCfg<D, N>::kThreads, 1)
tree_kernel(const __grid_constant__ TreeParams P) {
  using C = TrCfg<D, N>;
  constexpr int CW = C::CW, NS = C::NS, NP = C::NP;
  extern __shared__ uint8_t dsm_raw[];
  // (an offset, not a rounded pointer: the accesses stay shared-memory ones)
  uint8_t* const dsm = dsm_raw + ((1024u - (tc::saddr(dsm_raw) & 1023u)) & 1023u);
  uint8_t* raw = dsm + C::oRaw;
  float* s_qs = reinterpret_cast<float*>(dsm + C::oQs);
  float* s_nref = reinterpret_cast<float*>(dsm + C::oRef);
  float* s_red = reinterpret_cast<float*>(dsm + C::oRed);
  float* s_corr = reinterpret_cast<float*>(dsm + C::oCorr);
  float* s_sum = reinterpret_cast<float*>(dsm + C::oSum);
  unsigned long long* s_anc = reinterpret_cast<unsigned long long*>(dsm + C::oAnc);
  // barriers, as shared-memory addresses (barrier k of an array: + 8 k)
  const uint32_t rawfull = tc::saddr(dsm + C::oBar), rawempty = rawfull + 8 * NS;
  const uint32_t qfull = rawempty + 8 * NS;     // [2] a query set is in place
  const uint32_t sfree = qfull + 16;            // [2] the logits' buffer is free
  const uint32_t pready = sfree + 16;           // [2] weights in place
  const uint32_t qkdone = pready + 16, pvdone = qkdone + 16;   // [2] products complete
  const uint32_t own = pvdone + 16;             // [4][NB], where they are apart:
  const uint32_t kready = C::kApart ? own : sfree;                    // keys in place,
  const uint32_t vready = C::kApart ? own + 8 * C::NB : pready;       // values in place,
  const uint32_t kfree = C::kApart ? own + 16 * C::NB : qkdone;       // keys multiplied,
  const uint32_t vfree = C::kApart ? own + 24 * C::NB : pvdone;       // values multiplied
  const uint32_t ancfull = own + 32 * C::NB;    // [kTrAnc] ancestor sets in place
  const uint32_t drain = ancfull + 8 * kTrAnc;
  const uint32_t landed_bar = drain + 8;        // a marked unit's item has landed
  volatile uint32_t* s_misc = reinterpret_cast<volatile uint32_t*>(dsm + C::oMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) { tr_init(rawfull + 8 * s, 1); tr_init(rawempty + 8 * s, 8); }
    for (int s = 0; s < 2; ++s) {
      tr_init(qfull + 8 * s, 8);
      tr_init(sfree + 8 * s, C::SW + (C::kApart ? 0 : 4));
      tr_init(pready + 8 * s, C::SW + (C::kApart ? 0 : 4));
      tr_init(qkdone + 8 * s, 1);
      tr_init(pvdone + 8 * s, 1);
    }
    for (int s = 0; C::kApart && s < C::NB; ++s) {
      tr_init(kready + 8 * s, 4);
      tr_init(vready + 8 * s, 4);
      tr_init(kfree + 8 * s, 1);
      tr_init(vfree + 8 * s, 1);
    }
    for (int s = 0; s < kTrAnc; ++s) tr_init(ancfull + 8 * s, 1);
    tr_init(drain, NP);
    tr_init(landed_bar, 1);
    tc::fence_mbar_init();
    // ordinal + 1 of a drafted tile that holds a value that is not finite
    for (int k = 0; k < kTrAnc; ++k) s_misc[4 + k] = 0u;
  }
  if (warp == 1) {
    tc::tmem_alloc(const_cast<uint32_t*>(&s_misc[0]), kTrTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = s_misc[0];
  const Split cs{P.total, (long long)gridDim.x, 0};
  const long long C0 = cs.first(blockIdx.x), C1 = cs.first(blockIdx.x + 1);
  const int n = (int)(C1 - C0);   // >= 1: the grid is at most the number of tiles
  TrCur cur;
  cur.locate(P, C0);
  // Each role waits for the previous kernels (their writes: inputs, cache, tickets) where it would
  // first wait or read: taking its registers and setting up then overlap their ends.
  pdl_release();
  bool ok = true;

  if (warp < 4) {
  fewer_registers<C::kRegsIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------- raw tiles
    // Each group of unpacking warps has a ring of its own: a warp then sees every phase of
    // its slots in turn.
    const uint32_t raw0 = tc::saddr(raw);
    int it0 = 0, it1 = 0, nd = 0;   // ring items of the groups, drafted tiles so far
    // A marked unit's items land on a barrier of their own; this warp then takes what is in them by
    // 2^-4 (n 16-byte vectors from byte `first` on, `run` of them together, one run every `pitch`
    // bytes) and hands them on, one item at a time.
    int marked_items = 0;
    auto take = [&](int s, auto sixteenth, int n, int run, int pitch, int first) {
      const uint32_t phase = (uint32_t)(marked_items++ & 1);
      ok = tr_wait(landed_bar, phase, P.wait_limit, P.err, kErrTrProducer);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) tr_wait(landed_bar, phase, kTrPolls, P.err, kErrTrProducer);   // (before the CTA leaves)
#pragma unroll 1
      for (int i = lane; ok && i < n; i += 32) {
        auto* x = reinterpret_cast<decltype(sixteenth)*>(raw + s * C::SLOT + first + i / run * pitch + i % run * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __hmul2(x[e], sixteenth);
      }
      __syncwarp();
      if (lane == 0) tr_arrive(rawfull + 8 * s);
      __syncwarp();
    };
    const __half2 h16 = __float2half2_rn(0.0625f);
    const __nv_bfloat162 b16 = __float2bfloat162_rn(0.0625f);
    auto mark_of = [&](const TrCur& c) {
      return c.bits == 16 ? 0u : __ldcg(P.wide + ((size_t)(P.layer_begin + c.li) * P.units + c.unit) *
                                                     kMarkWords) & kWideValue;
    };
    auto slot = [&](int i) {      // the next ring slot of tile i's group, free
      const int gr = C::G == 2 ? i & 1 : 0;
      int& it = gr ? it1 : it0;
      const int s = gr * C::RS + it % C::RS, round = it / C::RS;
      ok = tr_wait(rawempty + 8 * (s), (uint32_t)(round & 1) ^ 1u, P.wait_limit, P.err, kErrTrProducer);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) ++it;
      if (lane == 0) asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      return s;
    };
    pdl_wait();
    // (known before the first copy: 0.3 us of a short call, 544 tokens 17.0 us, without it 16.7)
    unsigned marked = mark_of(cur);
    for (int i = 0; i < n && ok;) {
      const TreeLayer& L = P.L[cur.li];
      if (cur.j == 0 && i > 0) marked = mark_of(cur);
      // the segment's packed tiles of this CTA, in a tight loop: the layer's fields are read once
      const int np = min(cur.pt - cur.j, n - i);
      if (np > 0) {
        const int bb = block_bytes(D, cur.bits);
        int groups = cur.n_groups - 4 * cur.j;    // from the tile's first on
        const uint8_t* src =
            P.packed + L.packed_off + ((size_t)cur.unit * L.cap_groups + 4 * cur.j) * bb;
#pragma unroll 1
        for (int k = 0; marked && k < np; ++k, groups -= 4, src += 4 * bb) {
          const int s = slot(i + k), ng = min(4, groups);
          if (!ok) break;
          if (lane == 0) {
            tr_expect(landed_bar, (uint32_t)(ng * bb));
            tr_copy(raw0 + s * C::SLOT, src, (uint32_t)(ng * bb), landed_bar);
          }
          take(s, h16, ng * D / 2, D / 2, bb, off_kscale(D, cur.bits));   // scales, zero-points
          if (!ok) break;
        }
#pragma unroll 1
        for (int k = marked ? np : 0; k < np; ++k, groups -= 4, src += 4 * bb) {
          const int s = slot(i + k);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t bytes = (uint32_t)(min(4, groups) * bb);
            tr_expect(rawfull + 8 * s, bytes);
            tr_copy(raw0 + s * C::SLOT, src, bytes, rawfull + 8 * s);
          }
        }
        if (!ok) break;
        i += np;
        cur.j += np - 1;
        cur.step(P);                              // (the drafted tile is the segment's last)
        continue;
      }
      if (cur.j < cur.pt + cur.wt) {
        const int w0 = (cur.j - L.pt) * kTrTile, cnt = min(kTrTile, L.win_len - w0);
        const int s0 = (L.win_start + w0) % L.R;
        const size_t rb = (size_t)L.win_off + (size_t)cur.unit * L.R * D;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int s = slot(i);
          if (!ok) break;
          if (lane == 0) {
            // keys: rows of d; values: rows of d token pairs. The ring may wrap inside the tile
            const int rows = kv ? (cnt + 1) / 2 : cnt, first = kv ? s0 / 2 : s0;
            const int ring = kv ? L.R / 2 : L.R, rbytes = kv ? 4 * D : 2 * D;
            const uint8_t* src = reinterpret_cast<const uint8_t*>((kv ? P.win_v : P.win_k) + rb);
            const int a = min(rows, ring - first);
            const uint32_t dst = raw0 + s * C::SLOT;
            const uint32_t bar = kv && marked ? landed_bar : rawfull + 8 * s;
            tr_expect(bar, (uint32_t)(rows * rbytes));
            tr_copy(dst, src + (size_t)first * rbytes, (uint32_t)(a * rbytes), bar);
            if (rows > a) tr_copy(dst + a * rbytes, src, (uint32_t)((rows - a) * rbytes), bar);
          }
          if (kv && marked) take(s, b16, (cnt + 1) / 2 * (D / 4), 1, 16, 0);
        }
      } else {
        // ancestor sets: 64 links followed by doubling; a bad link marks its node, and what
        // hangs from it, as padding (the empty set)
        const int b = cur.unit / P.H;
        unsigned long long* anc = s_anc + nd % kTrAnc * kTrMaxNodes;
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
        if (lane == 0) tr_arrive(ancfull + 8 * (nd % kTrAnc));
        ++nd;
        const size_t ul = ((size_t)cur.li * P.units + cur.unit) * P.T * D;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int s = slot(i);
          if (!ok) break;
          const uint32_t bar = kv && marked ? landed_bar : rawfull + 8 * s;
          if (lane == 0) tr_expect(bar, (uint32_t)(P.T * D * 2));
          __syncwarp();
          for (int t = lane; t < P.T; t += 32)
            tr_copy(raw0 + s * C::SLOT + t * C::DP, (kv ? P.v_draft : P.k_draft) + ul + (size_t)t * D,
                     (uint32_t)(D * 2), bar);
          if (kv && marked) take(s, b16, P.T * (D / 8), D / 8, C::DP, 0);
        }
      }
      cur.step(P);
      ++i;
    }
    // every copy issued here has landed before the CTA can leave
    for (int k = max(0, it0 - C::RS); k < it0; ++k)
      tr_wait(rawfull + 8 * (k % C::RS), (uint32_t)((k / C::RS) & 1), kTrPolls, P.err, kErrTrProducer);
    for (int k = max(0, it1 - C::RS); k < it1; ++k)
      tr_wait(rawfull + 8 * (C::RS + k % C::RS), (uint32_t)((k / C::RS) & 1), kTrPolls, P.err, kErrTrProducer);
  } else if (warp == 1 || (NP == 2 && warp == 2)) {
    // -------------------------------------------------------------- products
    // (the warps run this converged, so that addresses and descriptors stay in uniform
    // registers; one lane issues). Up to 32 columns a tile is so short that one warp issuing
    // both products was what bounded it: warp 1 issues the first products, warp 2 the second.
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    int left = 0, done = 0, sets = 0;             // tiles left of the query set, of the sets so far
    bool packed = false;
    int vleft = 0, vdone = 0, vk = 0;             // the same of the second products; tiles of the segment
    bool vpacked = false;
    TrCur vc = cur;
    // the next set's tiles: the segment's packed ones, else its others
    auto set_of = [&](TrCur& c, int before, bool& packed) {
      if (c.j >= c.tps) c.next_segment(P);
      packed = c.j < c.pt;
      const int end = min(packed ? c.pt : c.tps, c.j + n - before), m = end - c.j;
      c.j = end;
      return m;
    };
    const uint64_t q0 = tc::sw128_desc(tc::saddr(dsm + C::oQ));
    auto keys = [&](int i) {        // S^T of tile i
      const uint32_t b = (uint32_t)(i & 1), ph = (uint32_t)((i >> 1) & 1);
      if (left == 0) {
        left = set_of(cur, done, packed);
        done += left;
        ok = tr_wait(qfull + 8 * (sets & 1), (uint32_t)((sets >> 1) & 1), P.wait_limit, P.err, kErrTrMma);
        ++sets;
      }
      --left;
      const uint32_t kb = (uint32_t)(i % C::NB);
      if (ok && C::kApart) ok = tr_wait(kready + 8 * kb, (uint32_t)(i / C::NB & 1), P.wait_limit, P.err, kErrTrMma);
      if (ok) ok = tr_wait(sfree + 8 * b, ph, P.wait_limit, P.err, kErrTrMma);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      tc::fence_after_sync();
      const uint32_t id = tc::idesc_ts(128, N, !packed, false);
      const uint64_t qd = q0 + (uint64_t)(((sets - 1) & 1) * (C::QB >> 4));
      const uint32_t st = tb + C::cS + b * N, kt = tb + C::cK + kb * (D / 2);
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ts(st, kt + kk * 8, qd + (uint64_t)(((kk / 4) * N * 128 + (kk % 4) * 32) >> 4),
                     id, kk > 0 ? 1u : 0u);
        tr_commit(qkdone + 8 * b);
        if constexpr (C::kApart) tr_commit(kfree + 8 * kb);
      }
      __syncwarp();
    };
    const uint64_t p0 = tc::sw128_mn_desc(tc::saddr(dsm + C::oP), C::PB, 1024);
    auto values = [&](int i) {      // O^T of tile i
      const uint32_t b = (uint32_t)(i & 1), ph = (uint32_t)((i >> 1) & 1);
      if (vleft == 0) {
        if (vc.j >= vc.tps) vk = 0;               // a segment begins
        vleft = set_of(vc, vdone, vpacked);
        vdone += vleft;
      }
      --vleft;
      const uint32_t vb = (uint32_t)(i % C::NB);
      if (ok && C::kApart) ok = tr_wait(vready + 8 * vb, (uint32_t)(i / C::NB & 1), P.wait_limit, P.err, kErrTrMma);
      if (ok) ok = tr_wait(pready + 8 * b, ph, P.wait_limit, P.err, kErrTrMma);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      tc::fence_after_sync();
      const uint32_t id = tc::idesc_ts(128, N, !vpacked, true);
      const uint32_t more = vk < NP ? 0u : 1u;    // 0: the pipeline's first tile of the segment
      ++vk;
      const uint32_t vt = tb + C::cV + vb * (kTrTile / 2);
      const uint32_t ot = tb + C::cO + (NP == 2 ? b * N : 0u);
      const uint64_t pd = p0 + (uint64_t)(b * (C::PB >> 4));
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTrTile / 16; ++kk)
          tc::mma_ts(ot, vt + kk * 8, pd + (uint64_t)((kk * 16 * 128) >> 4), id, kk > 0 ? 1u : more);
        tr_commit(pvdone + 8 * b);
        if constexpr (C::kApart) tr_commit(vfree + 8 * vb);
      }
      __syncwarp();
    };
    pdl_wait();
    if constexpr (NP == 2) {
      if (warp == 1)
        for (int i = 0; i < n && ok; ++i) keys(i);
      else
        for (int i = 0; i < n && ok; ++i) values(i);
    } else {
      keys(0);
      for (int i = 0; i < n && ok; ++i) {
        if (i + 1 < n) keys(i + 1);
        if (ok) values(i);
      }
    }
    // every product issued has completed before tensor memory is released
    if (tc::elect_one()) tr_commit(drain);
    __syncwarp();
    tr_wait(drain, 0u, kTrPolls, P.err, kErrTrMma);
  }   // the first warpgroup's other warps are idle
  } else if (warp < 4 + 8 * C::G) {
    // ------------------------------------------- queries, keys and values
    fewer_registers<C::kRegsUnpack>();
    constexpr int G = C::G;
    const bool is_key = warp < 4 + 4 * G;
    const int group = G == 2 ? ((warp >> 2) & 1) ^ 1 : 0;   // G = 2: the even or the odd tiles
    const int member = (warp & 3) + (is_key ? 0 : 4);
    const int w = warp & 3;                       // tensor-memory lane quarter
    const uint32_t dst0 = tbase + ((uint32_t)(32 * w) << 16) + (is_key ? C::cK : C::cV);
    const uint32_t dstep = is_key ? D / 2 : kTrTile / 2;   // columns of a buffer
    const uint32_t freed = is_key ? kfree : vfree, filled = is_key ? kready : vready;
    const CodeMasks<2> cm2 = code_masks<2>();
    const CodeMasks<4> cm4 = code_masks<4>();
    // tile i's buffer is free: its product of NB tiles back is complete (a fresh barrier's phase
    // before its first counts as complete)
    auto free_buffer = [&](int i) {
      ok = tr_wait(freed + 8 * (i % C::NB), (uint32_t)(i / C::NB & 1) ^ 1u, P.wait_limit, P.err, kErrTrUnpack);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
    };
    int it = 0;                                   // items of the group's ring so far
    const int slot0 = group * C::RS;
    auto landed = [&]() {                         // the ring's next item has landed
      ok = tr_wait(rawfull + 8 * (slot0 + it % C::RS), (uint32_t)((it / C::RS) & 1), P.wait_limit, P.err, kErrTrUnpack);
      ok = __all_sync(0xffffffffu, ok);
      return raw + (slot0 + it % C::RS) * C::SLOT;
    };
    auto give = [&]() {                           // this warp is done with it
      __syncwarp();
      if (lane == 0) tr_arrive(rawempty + 8 * (slot0 + it % C::RS));
      ++it;
    };
    auto finish = [&](int i) {                    // tile i's operand is in place
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tr_arrive(filled + 8 * (i % C::NB));
    };
    // Rows of the segment into the K-major swizzled tile of query set `set`: bf16 as they
    // are, or fp16 scaled to [1, 2) for packed tiles. A set two back is done with when the first
    // product of two tiles back is complete (one thread issues them in order). That of four
    // tiles back is, since a buffer of NB tiles back was free: the phase is not mistaken.
    auto queries = [&](int i, int set, bool packed) {
      if (C::kApart || !is_key) ok = tr_wait(qkdone + 8 * (i & 1), (uint32_t)((i >> 1) & 1) ^ 1u, P.wait_limit, P.err, kErrTrUnpack);
      ok = __all_sync(0xffffffffu, ok);
      constexpr int E = D / 32;                   // channels per lane
      uint8_t* qd = dsm + C::oQ + (set & 1) * C::QB;
      float* qs = s_qs + (set & 7) * N;
      const int r0 = cur.rt * N;
      const __nv_bfloat16* src =
          P.q + (((size_t)cur.li * P.units + cur.unit) * P.rows + r0) * D + lane * E;
      const int c0 = lane * E;
      const unsigned marked = cur.bits == 16 ? 0u :
          __ldcg(P.wide + ((size_t)(P.layer_begin + cur.li) * P.units + cur.unit) * kMarkWords) & kWideValue;
      uint32_t rows[N / 8][E / 2];                // all loads of the warp's rows in flight
#pragma unroll
      for (int k = 0; k < N / 8; ++k) {
        const int r = member + 8 * k;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) rows[k][e] = 0u;
        if (r0 + r < P.rows) {
          if constexpr (E == 4) {
            const uint2 x = *reinterpret_cast<const uint2*>(src + (size_t)r * D);
            rows[k][0] = x.x;
            rows[k][1] = x.y;
          } else {
            rows[k][0] = *reinterpret_cast<const uint32_t*>(src + (size_t)r * D);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < N / 8; ++k) {
        const int r = member + 8 * k;
        uint32_t (&v)[E / 2] = rows[k];
        float scale = P.sl2;
        if (packed) {
          uint32_t mx = 0u;                       // largest magnitude, as bf16 bits
#pragma unroll
          for (int e = 0; e < E / 2; ++e)
            mx = max(mx, max(v[e] & 0x7fffu, (v[e] >> 16) & 0x7fffu));
          mx = __reduce_max_sync(0xffffffffu, mx);
          int ex = (int)(mx >> 7);
          ex = ex == 255 ? 127 : min(max(ex, 5), 253);
          const float f = __int_as_float((254 - ex + (marked ? 4 : 0)) << 23);
          scale *= __int_as_float(ex << 23);
#pragma unroll
          for (int e = 0; e < E / 2; ++e)
            v[e] = h2u(__floats2half2_rn(__int_as_float((int)(v[e] << 16)) * f,
                                         __int_as_float((int)(v[e] & 0xffff0000u)) * f));
        }
        uint8_t* qrow = qd + (c0 >> 6) * N * 128 + r * 128 + ((((c0 & 63) >> 3) ^ (r & 7)) << 4) +
                        (c0 & 7) * 2;
        if constexpr (E == 4) *reinterpret_cast<uint2*>(qrow) = make_uint2(v[0], v[1]);
        else *reinterpret_cast<uint32_t*>(qrow) = v[0];
        if (lane == 0) qs[r] = scale;
      }
      if (member == 0 && lane == 0) s_misc[C::mMark + (set & 7)] = marked;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tr_arrive(qfull + 8 * (set & 1));
    };
    int sets = 0, nd = 0;                         // query sets, drafted tiles
    pdl_wait();
    for (int i = 0; i < n && ok; cur.next_segment(P)) {
      // the segment's tiles of this CTA: [cur.j, end), packed ones first
      const int end = min(cur.tps, cur.j + n - i), np = max(0, min(end, cur.pt) - cur.j);
      if (np > 0) {
        const int off = G == 2 ? (i ^ group) & 1 : 0;   // this warp's first tile among them
        if (off == 0) {
          free_buffer(i);
          if (!ok) break;
          queries(i, sets, true);
        }
        ++sets;
        auto tiles = [&](auto BITS_, const auto& cm) {
          constexpr int BITS = decltype(BITS_)::value, BB = block_bytes(D, BITS);
#pragma unroll 1
          for (int k = off; k < np && ok; k += G) {
            const int ng = min(4, cur.n_groups - 4 * (cur.j + k));
            const uint32_t dst = dst0 + (uint32_t)((i + k) % C::NB) * dstep;
            free_buffer(i + k);
            if (!ok) break;
            const uint8_t* src = landed();
            if (!ok) break;
            if (is_key) {
              if (w < ng) keys_packed<D, BITS>(src + w * BB, dst, cm);   // others are masked
            } else if (32 * w < D) {
              values_packed<D, BITS>(src, w, ng, dst, cm);
            }
            give();
            finish(i + k);
          }
        };
        if (cur.bits == 2) tiles(std::integral_constant<int, 2>{}, cm2);
        else tiles(std::integral_constant<int, 4>{}, cm4);
        if (!ok) break;
        i += np;
      }
      // window and drafted tiles: an item of keys, then one of values
      for (int j = cur.j + np; j < end; ++j, ++i) {
        const bool draft = j == cur.pt + cur.wt;
        if (G == 1 || ((i ^ group) & 1) == 0) {
          const uint32_t dst = dst0 + (uint32_t)(i % C::NB) * dstep;
          free_buffer(i);
          if (!ok) break;
          if (j == cur.j + np) queries(i, sets, false);
          if (!ok) break;
          const uint8_t* src = landed();
          if (!ok) break;
          if (is_key) {
            if (!draft) keys_window<D>(src, 32 * w, dst);
            else if (w < 2) keys_draft<D, C::DP>(src, 32 * w, dst);
            give();
            finish(i);
            landed();
            if (!ok) break;
          } else {
            give();
            src = landed();
            if (!ok) break;
            const bool on = 32 * w < D;
            if (!draft) {
              if (on) values_window<D>(src, w, min(kTrTile, cur.win_len - (j - cur.pt) * kTrTile), dst);
            } else {
              ok = tr_wait(ancfull + 8 * (nd % kTrAnc), (uint32_t)(nd / kTrAnc & 1), P.wait_limit, P.err, kErrTrUnpack);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              const unsigned long long* anc = s_anc + nd % kTrAnc * kTrMaxNodes;
              const unsigned long long live =
                  (unsigned long long)__ballot_sync(0xffffffffu, anc[lane] != 0ull) |
                  (unsigned long long)__ballot_sync(0xffffffffu, anc[lane + 32] != 0ull) << 32;
              if (on && values_draft<D, C::DP>(src, w, live, dst) && lane == 0)
                s_misc[4 + nd % kTrAnc] = (uint32_t)(nd + 1);
            }
            finish(i);
          }
          give();
        }
        if (j == cur.j + np) ++sets;
        nd += draft;
      }
    }
  } else {
    // ------------------------------------------------- softmax and output
    more_registers<C::kRegsSoft>();
    constexpr int kWarp0 = 4 + 8 * C::G;          // first softmax warp
    const int pipe = (warp - kWarp0) / C::SW;     // pipeline; NP = 2: the even or the odd tiles
    const int sa = threadIdx.x - kWarp0 * 32;     // thread of the softmax warps
    const int w = warp & 3, col0 = (((warp - kWarp0) % C::SW) >> 2) * CW;
    // The four warps of a column group agree on new references by themselves.
    const int group_bar = 1 + (warp - kWarp0) / 4;
    auto group_sync = [&] { soft_sync<128>(group_bar); };
    auto all_bar = [] { soft_sync<C::kSoftAll>(1 + C::kSoftAll / 128); };
    float* const all_nref = s_nref;
    float* const all_red = s_red;
    float* const all_corr = s_corr;
    s_nref += pipe * N;                           // this pipeline's
    s_red += pipe * 4 * N;
    s_corr += pipe * N;
    const int t = 32 * w + lane;                  // token of the tile; channel of the output
    const uint32_t lane_base = tbase + ((uint32_t)(32 * w) << 16) + (uint32_t)col0;
    const uint32_t ocol = lane_base + C::cO + (uint32_t)(pipe * N);
    const int my_col = col0 + (lane * CW) / 32;   // column whose reductions end in this lane
    const bool owner = (lane * CW) % 32 == 0;
    uint8_t* const prow = dsm + C::oP + t * 128;
    const int sw = t & 7;
    float2 lsum[CW / 2];
    float* const nref = s_nref + col0;
    int sets = 0, nd = 0;
    bool big = false;                             // some row's reference is past 2^16
    // One tile: logits of S^T against the rows' references, weights, their sums. PACKED: fp16
    // weights (else bf16); vis: the columns that see this thread's token; fresh: nothing of
    // the segment has been summed yet.
    auto tile = [&](auto PACKED_, int i, const float* qs, uint32_t vis, bool fresh) {
      constexpr bool PACKED = decltype(PACKED_)::value;
      const uint32_t b = (uint32_t)(i & 1), ph = (uint32_t)((i >> 1) & 1);
      if (ok) ok = tr_wait(qkdone + 8 * (b), ph, P.wait_limit, P.err, kErrTrSoftmax);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      const uint32_t scol = lane_base + C::cS + b * N;
      float y[CW];
      bool known = !fresh;                        // the rows have references (first tile: none)
      for (int pass = 0;; ++pass) {
        if (known) {
          if (big) {
            // The reference comes from a rounded logit: fused, the difference would keep the
            // logit's own rounding, which is anything where logits are large. Rounded first, it is
            // off by the rounding of the reference only, the same for all of the row's tokens (the
            // lift of 7 may round to 0 or 8).
            // (Row by row: a row's value does not depend on the others'.)
            uint32_t x[CW];
            tc::tmem_ld(scol, x);
#pragma unroll
            for (int c = 0; c < CW; ++c)
              y[c] = less_ref(__uint_as_float(x[c]), qs[c], nref[c]);
          } else {
            uint32_t x[CW];
            tc::tmem_ld(scol, x);
#pragma unroll
            for (int c = 0; c < CW; c += 4) {
              const float4 s4 = *reinterpret_cast<const float4*>(qs + c);
              const float4 n4 = *reinterpret_cast<const float4*>(nref + c);
              const float2 u = __ffma2_rn(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                                          make_float2(s4.x, s4.y), make_float2(n4.x, n4.y));
              const float2 v = __ffma2_rn(make_float2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])),
                                          make_float2(s4.z, s4.w), make_float2(n4.z, n4.w));
              y[c] = u.x; y[c + 1] = u.y; y[c + 2] = v.x; y[c + 3] = v.y;
            }
          }
          if (vis != 0xffffffffu) {                 // a token that a row does not see: -inf
#pragma unroll
            for (int c = 0; c < CW; ++c) y[c] = (vis >> c) & 1u ? y[c] : -INFINITY;
          }
          float top = y[0];
#pragma unroll
          for (int c = 1; c < CW - 1; c += 2) top = max3f(top, y[c], y[c + 1]);
          top = fmaxf(top, y[CW - 1]);
          if (pass || !soft_any<128>(group_bar, top > kTrSlack)) break;
        }
        known = true;
        // some row has no reference yet or is past it: new references for such rows (each
        // by its own logits alone), and the weights so far rescaled
        {
          uint32_t x[CW];
          tc::tmem_ld(scol, x);
#pragma unroll
          for (int c = 0; c < CW; ++c)
            y[c] = (vis >> c) & 1u ? __uint_as_float(x[c]) : -INFINITY;
        }
        const float m1 = reduce_columns<CW>(y, [](float u, float v) { return fmaxf(u, v); });
        if (owner) s_red[w * N + my_col] = m1;
        group_sync();
        if (w == 0 && owner) {
          const float m = fmaxf(fmaxf(s_red[my_col], s_red[N + my_col]),
                                fmaxf(s_red[2 * N + my_col], s_red[3 * N + my_col]));
          const float old = s_nref[my_col], scale = qs[my_col - col0];   // (positive)
          float nw = old, corr = 1.f;             // minus the row's reference, the factor
          if (m != -INFINITY && (old == kTrUnset || less_ref(m, scale, old) > kTrSlack)) {
            nw = __fsub_rn(kTrLift, __fmul_rn(m, scale));
            corr = old == kTrUnset ? 0.f : exp2f(nw - old);
          }
          s_nref[my_col] = nw;
          s_corr[my_col] = corr;
        }
        group_sync();
        {
          const float r = lane < CW ? nref[lane] : 0.f;
          big = soft_any<128>(group_bar, fabsf(r) > kTrBig && r != kTrUnset);
        }
#pragma unroll
        for (int c = 0; c < CW; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_corr + col0 + c);
          lsum[c / 2].x *= f.x; lsum[c / 2].y *= f.y;
          lsum[c / 2 + 1].x *= f.z; lsum[c / 2 + 1].y *= f.w;
        }
        if (!fresh) {
          // the output so far is at rest: rescale it (whole-warp loads and stores)
          const int before = i - NP;              // the pipeline's tile before this one
          if (ok) ok = tr_wait(pvdone + 8 * (before & 1), (uint32_t)((before >> 1) & 1), P.wait_limit, P.err, kErrTrSoftmax);
          ok = __all_sync(0xffffffffu, ok);
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < CW; c += 8) {
            uint32_t o[8];
            tc::tmem_ld(ocol + (uint32_t)c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * s_corr[col0 + c + e]);
            tc::tmem_st(ocol + (uint32_t)c, o);
            tc::tmem_wait_st();
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tr_arrive(sfree + 8 * b);
      uint32_t pk[CW / 2];
#pragma unroll
      for (int c = 0; c < CW; ++c) y[c] = fast_exp2(y[c]);
#pragma unroll
      for (int c = 0; c < CW; c += 2) {
        lsum[c / 2] = __fadd2_rn(lsum[c / 2], make_float2(y[c], y[c + 1]));
        if constexpr (PACKED) {
          pk[c / 2] = h2u(__floats2half2_rn(y[c], y[c + 1]));
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(y[c], y[c + 1]);
          pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      // The weights' buffer of two tiles back has been consumed. (With one issuing warp this
      // tile's first product came after that tile's second, and its barrier covers both.)
      if constexpr (NP == 2) {
        if (ok) ok = tr_wait(pvdone + 8 * (b), ph ^ 1u, P.wait_limit, P.err, kErrTrSoftmax);
        ok = __all_sync(0xffffffffu, ok);
      }
#pragma unroll
      for (int c8 = 0; c8 < CW / 8; ++c8)
        *reinterpret_cast<uint4*>(prow + b * C::PB + (((col0 / 8 + c8) ^ sw) << 4)) =
            make_uint4(pk[4 * c8], pk[4 * c8 + 1], pk[4 * c8 + 2], pk[4 * c8 + 3]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tr_arrive(pready + 8 * b);
    };
    if (sa < NP * N) all_nref[sa] = kTrUnset;
    if (lane == 0) {                              // the logits' buffers are free at first
      if (NP == 1 || pipe == 0) tr_arrive(sfree);
      if (NP == 1 || pipe == 1) tr_arrive(sfree + 8);
    }
    all_bar();
    pdl_wait();
    for (int i = 0; i < n; cur.next_segment(P)) {
      const int j0 = cur.j, end = min(cur.tps, j0 + n - i);
      const int np = max(0, min(end, cur.pt) - j0);
      const unsigned long long* anc = nullptr;
      const bool drafted = end == cur.tps;        // the last tile is the drafted one
      auto ancestors = [&]() {                    // not before: the copies of the tile bring them
        if (anc) return;
        if (ok) ok = tr_wait(ancfull + 8 * (nd % kTrAnc), (uint32_t)(nd / kTrAnc & 1), P.wait_limit, P.err, kErrTrSoftmax);
        anc = s_anc + nd % kTrAnc * kTrMaxNodes;
        ++nd;
      };
#pragma unroll
      for (int c = 0; c < CW / 2; ++c) lsum[c] = make_float2(0.f, 0.f);
      big = false;
      const int i0 = i, off = NP == 2 ? (i0 ^ pipe) & 1 : 0;   // the pipeline's first tile: i0 + off
      if (np > 0) {
        const float* qs = s_qs + (sets++ & 7) * N + col0;
#pragma unroll 1
        for (int k = off; k < np; k += NP)
          tile(std::true_type{}, i0 + k, qs, t < 32 * (cur.n_groups - 4 * (j0 + k)) ? 0xffffffffu : 0u, k < NP);
      }
      if (j0 + np < end) {
        const float* qs = s_qs + (sets++ & 7) * N + col0;
#pragma unroll 1
        for (int k = np + (NP == 2 ? (np ^ off) & 1 : 0); j0 + k < end; k += NP) {
          const int j = j0 + k;
          uint32_t vis = t < cur.win_len - (j - cur.pt) * kTrTile ? 0xffffffffu : 0u;
          if (j == cur.tps - 1) {
            ancestors();
            vis = 0u;
            const int r0 = cur.rt * N + col0;
            if (t < P.T) {
              int node = r0 % P.T;
#pragma unroll 1
              for (int c = 0; c < CW; ++c) {
                if (r0 + c < P.rows && ((anc[node] >> t) & 1ull)) vis |= 1u << c;
                if (++node == P.T) node = 0;
              }
            }
          }
          tile(std::false_type{}, i0 + k, qs, vis, k < NP);
        }
      }
      if (drafted) ancestors();
      i += end - j0;
      {
        // ---------------------------------------- the segment's part ends here
        const long long sbeg = C0 + i - end, send = sbeg + cur.tps;
        const bool whole = sbeg >= C0 && send <= C1;
        const size_t ul = (size_t)cur.li * P.units + cur.unit;
        const int rbase = cur.rt * N, nrow = min(N, P.rows - rbase);
        float* part = P.ws + ((size_t)blockIdx.x * 2 + (max(sbeg, C0) == C0 ? 0 : 1)) * C::STATE;
        float y[CW];
#pragma unroll
        for (int c = 0; c < CW; c += 2) { y[c] = lsum[c / 2].x; y[c + 1] = lsum[c / 2].y; }
        const float l1 = reduce_columns<CW>(y, [](float a, float b) { return a + b; });
        if (owner) s_red[w * N + my_col] = l1;
        all_bar();
        if (sa < nrow) {
          // the row's reference over the pipelines, their factors, its sum (-1: padding)
          float m = -INFINITY, l = 0.f;
#pragma unroll
          for (int p = 0; p < NP; ++p)
            if (all_nref[p * N + sa] != kTrUnset) m = fmaxf(m, -all_nref[p * N + sa]);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const float* r = all_red + p * 4 * N + sa;
            const float nr = all_nref[p * N + sa];
            const float f = nr == kTrUnset ? 0.f : (nr == -m ? 1.f : exp2f(-nr - m));
            all_corr[p * N + sa] = f;
            l += f * ((r[0] + r[N]) + (r[2 * N] + r[3 * N]));
          }
          if (s_misc[C::mMark + ((sets - 1) & 7)]) l *= 0.0625f;   // (as its values were)
          if (drafted && anc[(rbase + sa) % P.T] == 0ull) l = -1.f;
          s_sum[sa] = l;
          if (!whole) {
            part[N * D + sa] = m;
            part[N * D + N + sa] = l;
          }
        }
        const int tiles = end - j0;
#pragma unroll
        for (int p = 0; p < 2; ++p) {             // both buffers' last products
          const int last = i - 1 - p;
          if (ok && (p == 0 || tiles > 1))
            ok = tr_wait(pvdone + 8 * (last & 1), (uint32_t)((last >> 1) & 1), P.wait_limit, P.err, kErrTrSoftmax);
        }
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
        all_bar();
        const bool bad = drafted && s_misc[4 + (nd - 1) % kTrAnc] == (uint32_t)nd;
        // eight columns at a time, half of a warp's by each pipeline's; both outputs joined
        const uint32_t pfirst = NP == 2 ? (uint32_t)((i - 1) & 1) : 0u;   // pipeline of the last tile
#pragma unroll 1
        for (int c8 = NP == 2 ? pipe * (CW / 2) : 0;
             c8 < (NP == 2 ? (pipe + 1) * (CW / 2) : CW) && col0 + c8 < nrow; c8 += 8) {
          float o[8];
          uint32_t x[8];
          tc::tmem_ld(lane_base + C::cO + pfirst * N + (uint32_t)c8, x);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            o[e] = NP == 1 ? __uint_as_float(x[e])
                           : all_corr[pfirst * N + col0 + c8 + e] * __uint_as_float(x[e]);
          if (NP == 2 && tiles > 1) {
            tc::tmem_ld(lane_base + C::cO + (pfirst ^ 1u) * N + (uint32_t)c8, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e] = fmaf(all_corr[(pfirst ^ 1u) * N + col0 + c8 + e], __uint_as_float(x[e]), o[e]);
          }
          if (bad && t < D) {                     // values that are not finite, to the rows that see them
            const __nv_bfloat16* vd = P.v_draft + ul * P.T * D + t;
#pragma unroll 1
            for (int j = 0; j < P.T; ++j) {
              const float z = __bfloat162float(vd[(size_t)j * D]);
              if (isfinite(z)) continue;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int col = col0 + c8 + e;
                if (col < nrow && ((anc[(rbase + col) % P.T] >> j) & 1ull)) o[e] += z;
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int col = col0 + c8 + e;
            if (col < nrow && t < D) {
              const float l = s_sum[col];
              if (!whole) part[col * D + t] = o[e];
              else if (ok)
                P.out[(ul * P.rows + rbase + col) * D + t] = __float2bfloat16(l == -1.f ? 0.f : o[e] / l);
            }
          }
          __syncwarp();
        }
        tc::fence_before_sync();
        if (!whole) {
          all_bar();
          const long long ca = cs.owner(sbeg), cb = cs.owner(send - 1);
          const int nc = (int)(cb - ca + 1);
          unsigned* cnt = P.cnt + ((size_t)(P.layer_begin + cur.li) * P.units + cur.unit) * P.RT + cur.rt;
          if (sa == 0) {
            __threadfence();                      // (after the barrier: releases all warps' partial state)
            s_misc[1] = atomicAdd(cnt, 1u) == (unsigned)(nc - 1);
            __threadfence();
          }
          all_bar();
          if (s_misc[1]) {
            const bool late = cs.first(ca) < sbeg;   // the first holder's segment is its last
            auto part_of = [&](int k) -> const float* {
              return P.ws + ((size_t)(ca + k) * 2 + ((k == 0 && late) ? 1 : 0)) * C::STATE;
            };
            // The holders' maxima and sums go to a table in the weights' buffers (at rest
            // here), KB holders at a time; then every thread sums its four channels of
            // its rows, all rows' loads of a holder in flight at once.
            constexpr int KB = C::PB / (4 * N);      // holders in a table of [KB][N] floats
            constexpr int RS = C::kSoftAll / (D / 4), NR = N / RS;
            float* tm = reinterpret_cast<float*>(dsm + C::oP);
            float* tl = tm + KB * N;
            auto table = [&](int k0) {
              const int nb = min(KB, nc - k0);
#pragma unroll 4
              for (int p = sa; p < nb * N; p += C::kSoftAll) {
                const int r = p % N;
                const float* pp = part_of(k0 + p / N) + N * D;
                tm[p] = r < nrow ? __ldcg(pp + r) : -INFINITY;
                tl[p] = r < nrow ? __ldcg(pp + N + r) : 0.f;
              }
              all_bar();
              return nb;
            };
            float M = -INFINITY, sum = 0.f;
            bool pad = false;
            for (int k0 = 0; k0 < nc; k0 += KB) {
              if (k0) all_bar();
              const int nb = table(k0);
              if (sa < nrow)
                for (int k = 0; k < nb; ++k) {
                  const float lk = tl[k * N + sa];
                  if (lk == -1.f) pad = true;
                  else if (lk != 0.f) M = fmaxf(M, tm[k * N + sa]);
                }
            }
            float4 acc[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int c4 = sa % (D / 4), row0 = sa / (D / 4);
            for (int k0 = 0; k0 < nc; k0 += KB) {
              if (nc > KB) all_bar();
              const int nb = nc > KB ? table(k0) : nc;
              if (sa < nrow)                         // the holders' factors
                for (int k = 0; k < nb; ++k) {
                  const float lk = tl[k * N + sa];
                  const float f = lk != 0.f ? exp2f(tm[k * N + sa] - M) : 0.f;
                  sum += f * lk;
                  tm[k * N + sa] = f;
                }
              all_bar();
              // eight loads in flight: RU rows of HU holders (past the last: factor 0)
              constexpr int RU = NR < 4 ? NR : 4, HU = NR < 4 ? 4 : 2;
#pragma unroll
              for (int rc = 0; rc < NR; rc += RU)
#pragma unroll 1
                for (int k = 0; k < nb; k += HU) {
                  float4 v[HU][RU];
#pragma unroll
                  for (int u = 0; u < HU; ++u)
#pragma unroll
                    for (int r = 0; r < RU; ++r)
                      v[u][r] = __ldcg(reinterpret_cast<const float4*>(part_of(k0 + min(k + u, nb - 1))) +
                                       c4 + min(row0 + (rc + r) * RS, nrow - 1) * (D / 4));
#pragma unroll
                  for (int u = 0; u < HU; ++u)
#pragma unroll
                    for (int r = 0; r < RU; ++r)
                      if (k + u < nb) {
                        const float f = tm[(k + u) * N + min(row0 + (rc + r) * RS, nrow - 1)];
                        float4& a = acc[rc + r];
                        a.x = fmaf(f, v[u][r].x, a.x); a.y = fmaf(f, v[u][r].y, a.y);
                        a.z = fmaf(f, v[u][r].z, a.z); a.w = fmaf(f, v[u][r].w, a.w);
                      }
                }
            }
            if (sa < nrow) all_red[sa] = pad ? 0.f : 1.f / sum;
            all_bar();
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const int row = row0 + r * RS;
              if (ok && row < nrow) {
                const float inv = all_red[row];
                float4 a = acc[r];
                if (inv == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);   // padding
                const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * inv, a.y * inv),
                                     hi = __floats2bfloat162_rn(a.z * inv, a.w * inv);
                *reinterpret_cast<uint2*>(P.out + (ul * P.rows + rbase + row) * D + 4 * c4) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                               *reinterpret_cast<const uint32_t*>(&hi));
              }
            }
            if (sa == 0) *cnt = 0u;               // ready for the next launch
          }
        }
        all_bar();
        if (sa < NP * N) all_nref[sa] = kTrUnset;
        all_bar();
      }
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

// CTAs of the launch, which cut the list of tiles evenly. A part of a segment that ends inside a
// CTA costs about as much as six tiles (its output written and merged), so where the segments
// are no more than the SMs, each is cut into whole parts, one a CTA, unless the idle SMs cost
// more (32 segments of 66 tiles: 36 us, cut evenly over the SMs 46 us; 32 of 257: 91 and 88 us);
// a part then has two tiles at least where the segment has more than eight (18 tiles: 12.8 us,
// with single tiles 14.7 us; 6 tiles: 11.5 and 10.9 us), and up to three tiles are one part (9.0
// us, three parts 10.7 us).
long long tree_grid(const TreeParams& P, int n_sm) {
  const long long segs = (long long)P.n_layers * P.units * P.RT, tps = P.L[0].tps;
  bool even = segs <= n_sm;
  for (int i = 1; i < P.n_layers; ++i) even = even && P.L[i].tps == tps;
  if (even) {
    const long long s = std::min<long long>(n_sm / segs, tps > 8 ? (tps + 1) / 2 : (tps > 3 ? tps : 1));
    if ((tps + s - 1) / s <= (P.total + n_sm - 1) / n_sm + 6) return segs * s;
  }
  return std::min<long long>(n_sm, P.total);
}

template <int D, int N>
cudaError_t launch_tree_cols(const TreeParams& P, int n_sm, cudaStream_t stream) {
  using C = TrCfg<D, N>;
  const void* fn = reinterpret_cast<const void*>(tree_kernel<D, N>);
  cudaError_t e = ensure_smem(fn, C::total);
  if (e != cudaSuccess) return e;
  // the warpgroups' shares add up to the registers the block is launched with
  static const bool regs_ok = [&] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, fn) == cudaSuccess && a.numRegs >= C::R0;
  }();
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tree_grid(P, n_sm));
  cfg.blockDim = dim3(C::kThreads);
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
    P.wide = c->wide;
    P.wait_limit = c->wait_limit_set ? c->wait_limit : kTrPolls;
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
