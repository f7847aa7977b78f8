// window_tc.cu -- prompt attention over a sliding window and the first tokens (sinks) on the
// 5th-generation tensor cores (kvc_prefill_window).
//
//   o_i = sum_j p_ij v_j,  p_i = softmax_j(q_i . k_j / sqrt(d)),  j <= i and (j < s or i - j < W).
//
// Work: an item is (unit = (sequence, kv head), 2 P consecutive positions), P = 128 / g positions for
// each of the g query heads making a tile of 128 rows, two tiles an item, so that every key read
// serves 256 rows. An item visits the keys [0, s) in front of its first row's window in tiles of
// 64, then the keys from that window's first on; a tile that one of the two row tiles does not see
// is left out for it. Keys and values stream through a ring of 64-row stages by TMA from maps
// of [unit][position][channel], whose rows past the prompt read as 0.
//
// Row tile x has buffers of S = Q_x . K^T in tensor memory (64 columns each; three at head dimension
// 64, two at 128, where outputs take 256 of the 512 columns), used in turn, and two groups of four
// warps, one for the even and one for the odd tiles that it takes part in, a row per thread:
// maximum, P = exp2 into the same columns as bf16, sums in fp32. Warps of their own issue, per row tile,
// S_x(t) = Q_x K(t) as soon as a buffer's last weights are used, and O_x += P_x(t) V(t), P read from
// tensor memory, as soon as they are there: the groups of both row tiles and all four kinds of
// product run at the same time.
//
// What bounds it: at head dimension 64 the groups (3 x 20,011 tokens, 16/2 heads, window 1,000: 458 us,
// 543 TFLOP/s; issue slots 64 % busy, of 570 warp instructions per 64 keys of 32 rows 62 are exp2, 32
// conversions, 30 scaling, 29 maxima and 28 sums); at 128 the products: with 64 columns of S one takes 75
// cycles per 16 channels where its operands' 6 KB of shared memory allow 48 (131,072 tokens, 32/8 heads,
// window 4,096: 6.9 to 7.3 ms as the card's clock goes, 1.2 PFLOP/s of the pairs seen). Tried, when these
// two took 7.6 ms and 484 us: one buffer of 128 columns a row tile with one warp issuing everything (7.6
// ms and 535 us) or with four (9.6 ms: products wait for the weights' product to end and the ring holds
// two tiles); one warp issuing products of 64 columns (11.6 to 12.8 ms: it issues one in 80 cycles and
// takes 200 for a wait that is over).
//
// A row's weights are taken against a reference that follows its running maximum only when that
// has grown by more than 2^8 (then O_x is rescaled): P stays below 2^8 and its sums in fp32. The
// reference goes from tile to tile, and so from group to group, through shared memory. Sums
// are of the fp32 weights; P itself is rounded to bf16 (2^-8 of each weight): the product takes both
// operands in one 16-bit type, V is bf16, and the remainders would be a second product as long as the
// first. Outputs are 2.2e-3 from 64 bits with it, of which their own rounding is 1.6e-3.
//
// Values that are not finite reach, through a weight of 0, rows that do not see them. A group
// that has written such a row goes over its items once more at the end. What a row that is not finite
// should hold follows from the values it sees, channel by channel: NaN with a NaN or infinities of both
// signs, an infinity with infinities of one (mend_rows reads them once for a warp's 32 rows). A row is
// formed again, from the keys that it sees and no others, only where a channel sees finite values
// alone (a hidden value spoiled it, or its sum passed fp32's range), or where an infinite value may stand
// beside an infinite key: one hidden value reaches the rows of an item or two, in front of it and behind
// its window. Rows whose sum of weights is not finite, or 0, are NaN by the formula (a key that they see
// did that); they are written as kRowNaN, which tells them from the others. 16,384 tokens, 8/2 heads of
// 128, window 1,024: 0.11 ms; with one NaN that every row sees 0.40 (25.4 with every such row formed
// again), with an infinity in the middle, which 224 rows must not see, 3.8; 65,536 tokens that see all
// before them, with one NaN 14.7 ms, without 6.4.
//
// Roles: warps 0..15 the groups, four warps each (row tile 0 even, odd, row tile 1 even, odd), warp 16 the
// copies, warps 17 and 18 the scores of the two row tiles, 19 and 20 their outputs, the rest idle
// (registers are handed out by four warps). Every wait is bounded; one that gives up sets a bit of
// the error word, and its warp goes on without further waits (the pairs of warps that share rows
// meet at barriers all the same).
#include <algorithm>
#include <type_traits>
#include <cudaTypedefs.h>

#include "ask_once.h"
#include "kvc_internal.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr int kWnThreads = 32 * 24;
// registers a thread: at launch (65,536 over the threads), of the groups' warps, of the others
constexpr int kWnRegs = 65536 / kWnThreads / 8 * 8, kWnRegsGroup = 96, kWnRegsIssue = 48;
static_assert(4 * kWnRegsGroup + 2 * kWnRegsIssue <= 6 * kWnRegs, "the warpgroups' registers");
constexpr int kWnKeys = 64;            // keys of a tile
constexpr int kWnTmemCols = 512;
constexpr int kWnSmemLimit = 232448;   // opt-in shared memory per CTA
constexpr float kWnSlack = 8.f;        // log2 units a maximum may pass its reference by
constexpr unsigned kWnPolls = 1u << 20;   // polls of one wait before it gives up
constexpr unsigned kWnSpins = 16u;        // looks at a reference for one such poll

constexpr uint32_t kRowNaN = 0x7fc07fc0u; // two outputs of a row without a sum (conversions give NaN as 0x7fff)

enum : unsigned { kErrWnCopy = 1u << 16, kErrWnMma = 1u << 17, kErrWnGroup = 1u << 18 };

template <int D>
struct WnCfg {
  static constexpr int KB = D / 64;                // 64-element blocks of a row
  static constexpr int TQ = 128 * D * 2;           // one row tile's queries
  static constexpr int TB = kWnKeys * D * 2;       // one tile of keys or values
  static constexpr int SB = D == 64 ? 3 : 2;       // buffers of scores per row tile (tensor memory)
  static constexpr int NB = D == 64 ? 2 : 1;       // of queries (shared memory)
  static constexpr uint32_t cO = 2 * SB * kWnKeys; // first column of the outputs
  static_assert(cO + 2 * D <= kWnTmemCols, "scores and outputs fit tensor memory");
  static constexpr int FIT = (kWnSmemLimit - 2 * NB * TQ - 9216) / TB;
  static constexpr int KS = FIT > 16 ? 8 : FIT / 2;          // stages of keys,
  static constexpr int VS = FIT > 16 ? 8 : FIT - FIT / 2;    // of values
  static constexpr int STAGES = KS + VS;
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * NB * TQ;
  static constexpr int oBar = oKV + STAGES * TB;
  // full[S], empty[S] (keys, then values), qfull[2][2], qempty[2][2], sfull[2][3], pfull[2][3],
  // pvdone[2][3], oread[2], ofull[2], drain[4]
  static constexpr int NBAR = 2 * STAGES + 34;
  static constexpr int oTmem = oBar + NBAR * 8;
  static constexpr int oRef = (oTmem + 16 + 15) / 16 * 16;   // [2 items in turn][2][128] references, their tiles
  static constexpr int oSum = oRef + 2 * 2 * 128 * 8;        // [2 items in turn][2][2][128] sums
  static constexpr int total = oSum + 2 * 2 * 2 * 128 * 4 + 1024;   // + alignment slack
  static_assert(KS >= 3, "keys two tiles ahead of values");
  static_assert(total <= kWnSmemLimit, "fits the shared memory of one CTA");
};

struct WnArgs {
  int n, s, W;     // prompt length, sinks, window (neither above n)
  int g, P;        // query heads per kv head, positions per row tile (128 / g)
  int step;        // positions per item: 2 P, or P (its second row tile then has no rows)
  int Hq, Hk;
  int blocks;      // items per unit
  long long items;
  float sl2;       // log2(e) / sqrt(d)
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* x_out;   // [B][Hq][n][d]
  unsigned* err;
  unsigned wait_limit;    // polls of one wait before it gives up
};

// An item's place: its rows, its key tiles [0, ts) of sinks and [ts, T) from key j0 on, and the
// tiles that row tile x takes part in: all of the sinks', and [lo, hi).
struct Item {
  int unit, p0, j0, s0, ts, T;
  int lo0, lo1, hi0, hi1;
  __device__ __forceinline__ int lo(int x) const { return x ? lo1 : lo0; }
  __device__ __forceinline__ int hi(int x) const { return x ? hi1 : hi0; }
  __device__ __forceinline__ bool live(int x) const { return hi(x) > 0; }
  __device__ __forceinline__ int first(int x) const { return ts > 0 ? 0 : lo(x); }
  __device__ __forceinline__ int key0(int t) const { return t < ts ? t * kWnKeys : j0 + (t - ts) * kWnKeys; }
};
__device__ __forceinline__ Item item_of(long long i, const WnArgs& a) {
  Item it;
  it.unit = i >> 32 ? (int)(i / a.blocks) : (int)((unsigned)i / (unsigned)a.blocks);
  it.p0 = (int)(i - (long long)it.unit * a.blocks) * a.step;
  const int end = min(it.p0 + a.step, a.n);       // of its positions
  it.j0 = max(0, it.p0 - (a.W - 1));
  it.s0 = min(a.s, it.j0);
  it.ts = (it.s0 + kWnKeys - 1) / kWnKeys;
  it.T = it.ts + (end - 1 - it.j0) / kWnKeys + 1;
  auto tiles = [&](int q0, int& lo, int& hi) {
    const int from = a.s > it.j0 ? it.j0 : max(it.j0, q0 - (a.W - 1));
    lo = it.ts + (from - it.j0) / kWnKeys;
    hi = q0 < end ? it.ts + (min(q0 + a.P, end) - 1 - it.j0) / kWnKeys + 1 : 0;   // 0: no row of the prompt
  };
  tiles(it.p0, it.lo0, it.hi0);
  tiles(it.p0 + a.P, it.lo1, it.hi1);
  return it;
}

__device__ __noinline__ bool gave_up(unsigned* err, unsigned errbit) {
  if (err) atomicOr(err, errbit);
  return false;
}
// Bounded wait for the phase of parity `phase` & 1; false (and `errbit` in the error word) after
// `limit` polls.
__device__ __forceinline__ bool wn_wait(uint64_t* bar, int phase, unsigned limit, unsigned* err,
                                        unsigned errbit) {
  const uint32_t b = tc::saddr(bar);
#pragma unroll 1
  for (unsigned it = 0; it < limit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(b), "r"((uint32_t)(phase & 1)) : "memory");
    if (done) return true;
  }
  return gave_up(err, errbit);
}
template <int R>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(R));
}
template <int R>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(R));
}
__device__ __forceinline__ void pair_bar(int id) {
  asm volatile("bar.sync %0, 64;" :: "r"(id) : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(tc::saddr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z),
         "r"(tc::saddr(bar))
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Ones in the lowest k bits.
__device__ __forceinline__ uint32_t below(int k) { return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u; }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Rows of one unit again, by one warp, from the keys that each sees alone: the lowest kWnAgain of `rows`
// (bits as in mend_rows; the last one taken again where there are fewer), so that a key is read once for
// them. Where a sum of values is not finite they are taken once more with weights that add up to 1: sums of
// finite values cannot pass fp32's range then. (Three rows: with four the compiler shares out the registers of
// the kernel's ordinary path worse, 131,072 tokens took 7.5 ms for 6.9.)
constexpr int kWnAgain = 3;
template <int D>
__device__ __noinline__ void rows_again(const WnArgs& a, int unit, int q0, int quarter, unsigned rows) {
  constexpr int R = kWnAgain, C = D / 32;
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* k = a.k + (size_t)unit * a.n * D;
  const __nv_bfloat16* v = a.v + (size_t)unit * a.n * D;
  int pos[R], lo = INT_MAX, hi = 0;
  size_t at[R];
  float m[R], l[R], o[R][C];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = quarter * 32 + __ffs(rows) - 1;
    if (rows & (rows - 1)) rows &= rows - 1;
    pos[r] = q0 + i % a.P;
    at[r] = (((size_t)(unit / a.Hk) * a.Hq + (size_t)(unit % a.Hk) * a.g + i / a.P) * a.n + pos[r]) * D;
    lo = min(lo, pos[r]);
    hi = max(hi, pos[r]);
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) o[r][c] = 0.f;
  }
  auto sees = [&](int r, int j) { return j <= pos[r] && (j < a.s || pos[r] - j < a.W); };
  const int s1 = min(a.s, hi + 1), w0 = max(s1, lo - (a.W - 1));
  bool whole = false;                           // m is the row's maximum, and l 1 over its sum
  for (int part = 0; part < 4; ++part) {
    if (part == 2) {
      bool bad = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 16; i; i >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], i);
#pragma unroll
        for (int c = 0; c < C; ++c) bad = bad || !(fabsf(o[r][c]) < INFINITY);
      }
      whole = __any_sync(0xffffffffu, bad);
      if (!whole) break;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        l[r] = 1.f / l[r];
#pragma unroll
        for (int c = 0; c < C; ++c) o[r][c] = 0.f;
      }
    }
    const int end = part & 1 ? hi + 1 : s1;
    for (int j0 = part & 1 ? w0 : 0; j0 < end; j0 += 32) {
      const int j = min(j0 + lane, end - 1);
      float x[R] = {};
#pragma unroll 2
      for (int c = 0; c < D / 8; ++c) {
        const uint4 kw = reinterpret_cast<const uint4*>(k + (size_t)j * D)[c];
        const uint32_t ks[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint4 qw = reinterpret_cast<const uint4*>(a.q + at[r])[c];
          const uint32_t qs[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 qf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(qs + e));
            const float2 kf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(ks + e));
            x[r] = fmaf(qf.x, kf.x, x[r]);
            x[r] = fmaf(qf.y, kf.y, x[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool in = j0 + lane < end && sees(r, j);
        float top = in ? x[r] : -INFINITY;
#pragma unroll
        for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        top = fmaxf(top, m[r]);
        const float f = m[r] == -INFINITY ? 0.f : ex2((m[r] - top) * a.sl2);
        m[r] = top;
        x[r] = in ? ex2((x[r] - (top == -INFINITY ? 0.f : top)) * a.sl2) : 0.f;
        if (whole) {
          x[r] *= l[r];
          continue;
        }
        l[r] = l[r] * f + x[r];
#pragma unroll
        for (int c = 0; c < C; ++c) o[r][c] *= f;
      }
      for (int i0 = 0; i0 < min(32, end - j0); i0 += 8) {   // eight values in flight
        __nv_bfloat162 w[8][C / 2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int c = 0; c < C / 2; ++c)
            w[i][c] = reinterpret_cast<const __nv_bfloat162*>(v + (size_t)min(j0 + i0 + i, end - 1) * D + lane * C)[c];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float p = __shfl_sync(0xffffffffu, x[r], i0 + i);
            if (j0 + i0 + i >= end || !sees(r, j0 + i0 + i)) continue;
#pragma unroll
            for (int c = 0; c < C / 2; ++c) {
              const float2 z = __bfloat1622float2(w[i][c]);
              o[r][2 * c] = fmaf(p, z.x, o[r][2 * c]);
              o[r][2 * c + 1] = fmaf(p, z.y, o[r][2 * c + 1]);
            }
          }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    for (int c = 0; c < C; ++c)
      a.x_out[at[r] + lane * C + c] = __float2bfloat16_rn(whole ? o[r][c] : o[r][c] / l[r]);
  }
}

// Largest and smallest of what a row sees of two channels of a word, NaN where one is.
template <int N>
struct Extent {
  __nv_bfloat162 hi[N], lo[N];
};
// Outputs that are not finite of some of a warp's 32 rows (those in `rows`), put right: see above. q0: first
// position of the row tile.
template <int D>
__device__ __noinline__ void mend_rows(const WnArgs& a, int unit, int q0, int quarter, unsigned rows) {
  const int lane = threadIdx.x & 31;
  constexpr int N = D / 64;                     // words of a lane: channels 2 N lane .. 2 N lane + 2 N - 1
  const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k + (size_t)unit * a.n * D) + lane * N;
  const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v + (size_t)unit * a.n * D) + lane * N;
  auto load = [](uint32_t (&w)[N], const uint32_t* p) {
    if constexpr (N == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x; w[1] = u.y;
    } else {
      w[0] = *p;
    }
  };
  auto pair = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  // rows [from, to) of x, eight at a time (the last one again past the end)
  auto visit = [&](const uint32_t* x, int from, int to, auto use) {
    for (int j = from; j < to; j += 8) {
      uint32_t w[8][N];
#pragma unroll
      for (int i = 0; i < 8; ++i) load(w[i], x + (size_t)min(j + i, to - 1) * (D / 2));
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c) use(c, pair(w[i][c]));
    }
  };
  auto see = [&](Extent<N>& e, int from, int to) {
    visit(v, from, to, [&](int c, __nv_bfloat162 z) {
      e.hi[c] = __hmax2_nan(e.hi[c], z);
      e.lo[c] = __hmin2_nan(e.lo[c], z);
    });
  };
  // what all of the rows see: [0, s1) and [w0, first]
  const int mine = q0 + (quarter * 32 + lane) % a.P, back = a.W - 1;
  const bool in = rows >> lane & 1u;
  const int first = __reduce_min_sync(0xffffffffu, in ? mine : INT_MAX);
  const int last = __reduce_max_sync(0xffffffffu, in ? mine : -1);
  const int s1 = min(a.s, first + 1), w0 = max(s1, last - back);
  Extent<N> all;
#pragma unroll
  for (int c = 0; c < N; ++c) all.hi[c] = all.lo[c] = pair(0u);
  see(all, 0, s1);
  see(all, w0, first + 1);
  int keys = -1;                                // whether the keys are finite, where it was asked
  auto finite_keys = [&] {                      // (of all that some of the rows see)
    if (keys >= 0) return keys != 0;
    __nv_bfloat162 top = pair(0u);
    auto use = [&](int, __nv_bfloat162 z) { top = __hmax2_nan(top, __habs2(z)); };
    visit(k, 0, min(a.s, last + 1), use);
    visit(k, max(0, first - back), last + 1, use);
    keys = __all_sync(0xffffffffu, __low2float(top) < INFINITY && __high2float(top) < INFINITY);
    return keys != 0;
  };
  unsigned todo = 0u;                           // rows to form again
  for (; rows; rows &= rows - 1) {
    const int r = quarter * 32 + __ffs(rows) - 1, pos = q0 + r % a.P, head = r / a.P;
    Extent<N> e = all;                          // and what this one sees besides
    see(e, max(s1, pos - back), min(w0, pos + 1));
    see(e, max(first + 1, pos - back), pos + 1);
    see(e, s1, min(a.s, pos + 1));
    const size_t row = ((size_t)(unit / a.Hk) * a.Hq + (size_t)(unit % a.Hk) * a.g + head) * a.n + pos;
    uint32_t* x = reinterpret_cast<uint32_t*>(a.x_out + row * D) + lane * N;
    uint32_t w[N];
    bool form = false, infinite = false;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      w[c] = __ldcg(x + c);
      const float2 hi = __bfloat1622float2(e.hi[c]), lo = __bfloat1622float2(e.lo[c]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t z = w[c] >> (16 * h) & 0xffffu;
        if ((z & 0x7f80u) != 0x7f80u) continue;
        const float top = h ? hi.y : hi.x, low = h ? lo.y : lo.x;
        const bool up = top == INFINITY, down = low == -INFINITY;
        if (top != top || (up && down)) {
          form = form || (z & 0x7fu) == 0u;     // (an infinity: not of the values seen)
        } else if (!up && !down) {
          form = true;
        } else {
          const uint32_t want = up ? 0x7f80u : 0xff80u;
          if (z == want) continue;
          form = form || (z & 0x7fu) == 0u;
          infinite = true;
          w[c] = (w[c] & ~(0xffffu << (16 * h))) | want << (16 * h);
        }
      }
    }
    form = __any_sync(0xffffffffu, form);
    if (!form && __any_sync(0xffffffffu, infinite)) {
      if (!finite_keys()) form = true;          // (an infinite value may have a weight of 0: NaN)
      else if (infinite)
#pragma unroll
        for (int c = 0; c < N; ++c) x[c] = w[c];
    }
    if (form) todo |= rows & (0u - rows);
  }
  while (todo) {
    rows_again<D>(a, unit, q0, quarter, todo);
    for (int i = 0; i < kWnAgain; ++i) todo &= todo - 1;
  }
}
// The rows of row tile x that came out not finite in some output, of every item of the CTA, by the warps of
// one of its groups.
template <int D>
__device__ __noinline__ void mend_items(const WnArgs& a, int x, int quarter) {
  const int r = quarter * 32 + (threadIdx.x & 31);
  for (long long i = blockIdx.x; i < a.items; i += gridDim.x) {
    const Item it = item_of(i, a);
    if (!it.live(x)) continue;
    const int pos = it.p0 + x * a.P + r % a.P;
    bool mine = false;
    if (pos < a.n) {
      const size_t row = ((size_t)(it.unit / a.Hk) * a.Hq + (size_t)(it.unit % a.Hk) * a.g + r / a.P) * a.n + pos;
      const uint4* w = reinterpret_cast<const uint4*>(a.x_out + row * D);
      for (int c = 0; c < D / 8; ++c) {
        const uint4 u = __ldcg(w + c);
        for (uint32_t z : {u.x, u.y, u.z, u.w})
          mine = mine || (z != kRowNaN && ((z & 0x7f80u) == 0x7f80u || (z & 0x7f800000u) == 0x7f800000u));
      }
    }
    if (const unsigned rows = __ballot_sync(0xffffffffu, mine))
      mend_rows<D>(a, it.unit, it.p0 + x * a.P, quarter, rows);
  }
}

template <int D>
__global__ void __launch_bounds__(kWnThreads, 1)
window_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const WnArgs a) {
  using C = WnCfg<D>;
  extern __shared__ uint8_t dsm_raw[];
  uint8_t* dsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) &
                                            ~uintptr_t(1023));
  uint8_t* sQ = dsm + C::oQ;
  uint8_t* sKV = dsm + C::oKV;
  uint64_t* full = reinterpret_cast<uint64_t*>(dsm + C::oBar);
  uint64_t* empty = full + C::STAGES;
  uint64_t* qfull = full + 2 * C::STAGES;
  uint64_t* qempty = qfull + 4;    // [row tile][buffer]
  uint64_t* sfull = qfull + 8;     // [row tile][buffer], as the next two
  uint64_t* pfull = qfull + 14;
  uint64_t* pvdone = qfull + 20;
  uint64_t* oread = qfull + 26;    // [row tile]
  uint64_t* ofull = qfull + 28;
  uint64_t* drain = qfull + 30;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(dsm + C::oTmem);
  unsigned long long* sref = reinterpret_cast<unsigned long long*>(dsm + C::oRef);
  float* ssum = reinterpret_cast<float*>(dsm + C::oSum);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) { tc::mbar_init(&full[s], 1); tc::mbar_init(&empty[s], 2); }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(&ofull[x], 1);
      tc::mbar_init(&oread[x], 8);
      for (int b = 0; b < 2; ++b) {
        tc::mbar_init(&qfull[2 * x + b], 1);
        tc::mbar_init(&qempty[2 * x + b], 1);
      }
      for (int b = 0; b < 3; ++b) {
        tc::mbar_init(&sfull[3 * x + b], 1);
        tc::mbar_init(&pfull[3 * x + b], 4);
        tc::mbar_init(&pvdone[3 * x + b], 1);
      }
    }
    for (int w = 0; w < 4; ++w) tc::mbar_init(&drain[w], 1);
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmQ);
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  if (threadIdx.x < 512) sref[threadIdx.x] = ~0ull;   // of no tile
  if (warp == 17) {
    tc::tmem_alloc(tmem_holder, kWnTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_holder;
  pdl_wait();
  pdl_release();
  bool ok = true;

  if (warp >= 16) {
  fewer_registers<kWnRegsIssue>();
  if (warp == 16) {
    // --------------------------------------------------------------- copies
    if (lane == 0) {
      int nk = 0, nv = 0, nq[2] = {0, 0};
      struct Cur { long long i; Item it; int t; };
      // tile `tile` of keys (first stage 0) or values (first stage KS)
      auto stage = [&](const CUtensorMap* map, int first, int stages, int& tile, int row, int unit) {
        const int s = first + tile % stages, round = tile / stages;
        if (ok && round > 0) ok = wn_wait(&empty[s], round - 1, a.wait_limit, a.err, kErrWnCopy);
        if (!ok) return;
        tc::mbar_expect_tx(&full[s], (uint32_t)C::TB);
        for (int kb = 0; kb < C::KB; ++kb)
          tma_load_3d(sKV + s * C::TB + kb * kWnKeys * 128, map, kb * 64, row, unit, &full[s]);
        ++tile;
      };
      auto next = [&](Cur& c) {
        if (++c.t < c.it.T) return;
        c.t = 0;
        c.i += gridDim.x;
        if (c.i < a.items) c.it = item_of(c.i, a);
      };
      auto keys = [&](Cur& c) {   // the item's queries with its first keys
        if (c.i >= a.items) return;
        if (c.t == 0) {
          const int b = c.it.unit / a.Hk, hk = c.it.unit % a.Hk;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!c.it.live(x)) continue;
            const int qb = nq[x] % C::NB, round = nq[x] / C::NB;
            if (ok && round > 0) ok = wn_wait(&qempty[2 * x + qb], round - 1, a.wait_limit, a.err, kErrWnCopy);
            if (!ok) return;
            tc::mbar_expect_tx(&qfull[2 * x + qb], (uint32_t)C::TQ);
            for (int hh = 0; hh < a.g; ++hh)
              for (int kb = 0; kb < C::KB; ++kb)
                tma_load_3d(sQ + (x * C::NB + qb) * C::TQ + kb * 128 * 128 + hh * a.P * 128, &tmQ, kb * 64,
                            c.it.p0 + x * a.P, b * a.Hq + hk * a.g + hh, &qfull[2 * x + qb]);
            ++nq[x];
          }
        }
        stage(&tmK, 0, C::KS, nk, c.it.key0(c.t), c.it.unit);
        next(c);
      };
      Cur ck{blockIdx.x, item_of(blockIdx.x, a), 0}, cv = ck;
      keys(ck);
      if (ok) keys(ck);
      while (ok && cv.i < a.items) {
        stage(&tmV, C::KS, C::VS, nv, cv.it.key0(cv.t), cv.it.unit);
        next(cv);
        if (ok) keys(ck);
      }
      // every copy issued here has landed before the CTA can leave
      for (int j = max(0, nk - C::KS); j < nk; ++j)
        wn_wait(&full[j % C::KS], j / C::KS, kWnPolls, a.err, kErrWnCopy);
      for (int j = max(0, nv - C::VS); j < nv; ++j)
        wn_wait(&full[C::KS + j % C::VS], j / C::VS, kWnPolls, a.err, kErrWnCopy);
      for (int x = 0; x < 2; ++x)
        for (int j = max(0, nq[x] - C::NB); j < nq[x]; ++j)
          wn_wait(&qfull[2 * x + j % C::NB], j / C::NB, kWnPolls, a.err, kErrWnCopy);
    }
  } else if (warp <= 20) {
    // ------------------------------------------------------------- products
    // Warps 17 and 18 issue the scores of row tiles 0 and 1, warps 19 and 20 their outputs. (The
    // warps run this converged, so that addresses and descriptors stay in uniform registers; one
    // lane issues.)
    const int x = (warp - 17) & 1;
    const bool keys = warp < 19;
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, tc::saddr(dsm), 0);
    auto wait = [&](uint64_t* b, int phase) {
      if (ok) ok = wn_wait(b, phase, a.wait_limit, a.err, kErrWnMma);
      ok = __all_sync(0xffffffffu, ok);
    };
    int no = 0;                      // the row tile's items so far
    int nb = 0, nr = 0;              // its tile's buffer of scores, the buffers' round
    int s = 0, round = 0;            // the stage, the stages' round
    auto tiles = [&](int first, int stages, auto product) {
      for (long long i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
        const Item it = item_of(i, a);
        const int begin = it.first(x), end = it.hi(x), lo = it.lo(x);
        for (int t = 0; t < it.T && ok; ++t) {
          wait(&full[first + s], round);          // (also where this row tile leaves it out)
          if (t < end && (t < it.ts || t >= lo)) {
            product(first + s, t == begin, t == end - 1);
          } else if (tc::elect_one()) {
            tc::mbar_arrive(&empty[first + s]);   // (not this row tile's)
          }
          __syncwarp();
          if (++s == stages) { s = 0; ++round; }
        }
      }
    };
    if (keys) {
      constexpr uint32_t idesc = tc::idesc_bf16_f32(128, kWnKeys);
      const uint64_t q0 = tc::sw128_desc(base + C::oQ + x * C::NB * C::TQ), k0 = tc::sw128_desc(base + C::oKV);
      int qb = 0;                                 // the item's queries
      tiles(0, C::KS, [&](int st, bool begin, bool end) {
        if (begin) {
          qb = no % C::NB;
          wait(&qfull[2 * x + qb], no++ / C::NB);
        }
        if (nr > 0) wait(&pvdone[3 * x + nb], nr - 1);   // the buffer's last weights are used
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t d = tb + (x * C::SB + nb) * (uint32_t)kWnKeys;
        const uint64_t kd = k0 + (uint64_t)(st * (C::TB >> 4)), qd = q0 + (uint64_t)(qb * (C::TQ >> 4));
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_bf16(d, qd + (uint64_t)(((kk / 4) * 128 * 128 + (kk % 4) * 32) >> 4),
                         kd + (uint64_t)(((kk / 4) * kWnKeys * 128 + (kk % 4) * 32) >> 4), idesc,
                         kk > 0 ? 1u : 0u);
          tc::mma_commit(&sfull[3 * x + nb]);
          tc::mma_commit(&empty[st]);
          if (end) tc::mma_commit(&qempty[2 * x + qb]);
        }
        if (++nb == C::SB) { nb = 0; ++nr; }
      });
    } else {
      constexpr uint32_t idesc = tc::idesc_ts(128, D, true, true);
      const uint64_t v0 = tc::sw128_mn_desc(base + C::oKV, kWnKeys * 128, 1024);
      const uint32_t d = tb + C::cO + x * (uint32_t)D;
      tiles(C::KS, C::VS, [&](int st, bool begin, bool end) {
        if (begin && no++ > 0) wait(&oread[x], no - 2);   // the item before is read
        wait(&pfull[3 * x + nb], nr);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t p = tb + (x * C::SB + nb) * (uint32_t)kWnKeys, acc = begin ? 0u : 1u;
        const uint64_t vd = v0 + (uint64_t)(st * (C::TB >> 4));
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kWnKeys / 16; ++kk)   // A = P (keys along K); B = V, its rows the keys
            tc::mma_ts(d, p + kk * 8u, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc, kk > 0 ? 1u : acc);
          tc::mma_commit(&pvdone[3 * x + nb]);
          tc::mma_commit(&empty[st]);
          if (end) tc::mma_commit(&ofull[x]);
        }
        if (++nb == C::SB) { nb = 0; ++nr; }
      });
    }
    // every product issued here has completed before tensor memory is released
    if (tc::elect_one()) tc::mma_commit(&drain[warp - 17]);
    __syncwarp();
    wn_wait(&drain[warp - 17], 0, kWnPolls, a.err, kErrWnMma);
  }   // the others are idle
  } else {
    // --------------------------------------------------------------- groups
    more_registers<kWnRegsGroup>();
    const int x = warp >> 3, buf = (warp >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;              // row of the tile: head * P + position
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t st0 = tbase + lane_addr + x * (uint32_t)(C::SB * kWnKeys);
    const uint32_t ot = tbase + lane_addr + C::cO + x * (uint32_t)D;
    const int hh = r / a.P, dp = x * a.P + r % a.P;
    const int bar_id = 1 + x * 4 + quarter;         // the two warps that share rows
    // the row's reference (log2 units) and, above, the tile that left it: handed on from group to group
    // (two items in turn: a group that is still with the one reads it while the other begins)
    volatile unsigned long long* my_ref = sref + x * 128 + r;
    int n = 0, no = 0;                              // the row tile's tiles and items so far
    int nb = C::SB == 2 ? buf : -1, nr = 0;         // tile n's buffer of scores, the buffers' round
    bool again = false;                             // some row came out not finite
    auto wait = [&](uint64_t* b, int phase) {
      if (ok) ok = wn_wait(b, phase, a.wait_limit, a.err, kErrWnGroup);
      ok = __all_sync(0xffffffffu, ok);
    };
    auto reference = [&](int tile) {
      const volatile unsigned long long* p = my_ref + (no & 1) * 256;
      unsigned long long u = *p;
      if (!__all_sync(0xffffffffu, (int)(u >> 32) == tile)) {
        for (unsigned long long left = (unsigned long long)a.wait_limit * kWnSpins;
             ok && (int)(u >> 32) != tile; u = *p) {
          if (left-- == 0) ok = gave_up(a.err, kErrWnGroup);
          __nanosleep(20);                          // (the other warps need the issue slots)
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      return __uint_as_float((uint32_t)u);
    };
    const bool wide = reinterpret_cast<uintptr_t>(a.x_out) % 32 == 0;   // whole sectors
    for (long long i = blockIdx.x; i < a.items; i += gridDim.x) {
      const Item it = item_of(i, a);
      if (!it.live(x)) continue;
      const int pos = it.p0 + dp;
      const int q0 = it.p0 + x * a.P, q1 = q0 + a.P - 1;   // the tile's positions
      const int t0 = it.first(x), t1 = it.hi(x), t_lo = it.lo(x);
      float ref = -INFINITY, lsum = 0.f;            // reference of the sum so far (log2 units), the sum
      for (int t = t0; t < t1; t = t + 1 == it.ts ? t_lo : t + 1, ++n) {
        // (three buffers: counted; two: the group's own)
        if constexpr (C::SB == 3) {
          if (++nb == C::SB) { nb = 0; ++nr; }
        }
        if ((n & 1) != buf) continue;
        if constexpr (C::SB == 2) nr = n >> 1;
        const uint32_t st = st0 + (uint32_t)(nb * kWnKeys);
        wait(&sfull[3 * x + nb], nr);
        tc::fence_after_sync();
        float v[64];
        {
          uint32_t w[2][32];
          tc::tmem_ld32_async(st, w[0]);
          tc::tmem_ld32_async(st + 32u, w[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tc::tmem_wait_ld32(w[c]);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[32 * c + e] = __uint_as_float(w[c][e]);
          }
        }
        const int key0 = it.key0(t);
        const bool sinks = t < it.ts;
        if (sinks ? key0 + kWnKeys > it.s0 : key0 + kWnKeys - 1 > q0 || key0 < q1 - (a.W - 1)) {
          // seen: sinks, or up to the row's own key, from its window's first on or a sink
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = key0 + 32 * h;
            const uint32_t bits = sinks ? below(it.s0 - k)
                                        : below(pos + 1 - k) & (~below(pos - (a.W - 1) - k) | below(a.s - k));
#pragma unroll
            for (int c = 0; c < 32; ++c) v[32 * h + c] = bits >> c & 1u ? v[32 * h + c] : -INFINITY;
          }
        }
        float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
        for (int c = 4; c < 60; c += 8) {
          m0 = max3(m0, v[c], v[c + 1]);
          m1 = max3(m1, v[c + 2], v[c + 3]);
          m2 = max3(m2, v[c + 4], v[c + 5]);
          m3 = max3(m3, v[c + 6], v[c + 7]);
        }
        const float mx = max3(max3(m0, v[60], v[61]), max3(m1, v[62], v[63]), fmaxf(m2, m3));
        const float m = mx == -INFINITY ? -INFINITY : mx * a.sl2;
        // the reference after the tile before (the other group's)
        const float before = t == t0 ? -INFINITY : reference(n - 1);
        const bool raise = m > before + kWnSlack || (before == -INFINITY && m != -INFINITY);
        const float now = raise ? m : before;
        // (tensor-memory accesses are whole-warp: the other lanes rescale by 1)
        const bool resc = raise && before != -INFINITY;
        if (__any_sync(0xffffffffu, resc)) {
          wait(&pvdone[3 * x + (nb ? nb - 1 : C::SB - 1)], nb ? nr : nr - 1);   // of tile n - 1
          tc::fence_after_sync();
          const float f = resc ? ex2(before - m) : 1.f;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t o[16];
            tc::tmem_ld(ot + (uint32_t)c0, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::tmem_st(ot + (uint32_t)c0, o);
          }
          tc::tmem_wait_st();
        }
        my_ref[(no & 1) * 256] = (unsigned long long)__float_as_uint(now) | (unsigned long long)(unsigned)n << 32;
        const float nref = now == -INFINITY ? 0.f : -now;
        if (__any_sync(0xffffffffu, fabsf(nref) > 65536.f)) {
          // far references: the product is rounded as theirs was, so that the difference is exact
#pragma unroll
          for (int c = 0; c < 64; ++c) v[c] = __fadd_rn(__fmul_rn(v[c], a.sl2), nref);
        } else {
          const float2 s2 = make_float2(a.sl2, a.sl2), n2 = make_float2(nref, nref);
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            const float2 e = __ffma2_rn(make_float2(v[c], v[c + 1]), s2, n2);
            v[c] = e.x;
            v[c + 1] = e.y;
          }
        }
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c0 + c] = ex2(v[c0 + c]);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[c0 + c], v[c0 + c + 1]);
            pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tc::tmem_st(st + (uint32_t)(c0 / 2), pk);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&pfull[3 * x + nb]);
        __syncwarp();
        // (the sum after P is handed over)
        float2 l0 = make_float2(v[0], v[1]), l1 = make_float2(v[2], v[3]);
#pragma unroll
        for (int c = 4; c < 64; c += 4) {
          l0 = __fadd2_rn(l0, make_float2(v[c], v[c + 1]));
          l1 = __fadd2_rn(l1, make_float2(v[c + 2], v[c + 3]));
        }
        lsum = (ref == now || ref == -INFINITY ? lsum : lsum * ex2(ref - now)) + ((l0.x + l0.y) + (l1.x + l1.y));
        ref = now;
      }
      // this group's sum against the last reference
      const float last = reference(n - 1);
      if (ref != last && ref != -INFINITY) lsum *= ex2(ref - last);
      ssum[((no & 1) * 2 + x) * 256 + buf * 128 + r] = lsum;
      pair_bar(bar_id);
      const float inv = 1.f / (lsum + ssum[((no & 1) * 2 + x) * 256 + (buf ^ 1) * 128 + r]);
      // the outputs, half of the columns each group
      wait(&ofull[x], no);
      tc::fence_after_sync();
      const size_t row = ((size_t)(it.unit / a.Hk) * a.Hq + (size_t)(it.unit % a.Hk) * a.g + hh) * a.n +
                         min(pos, a.n - 1);
      __nv_bfloat16* dst = a.x_out + row * D + buf * (D / 2);
      float bad = 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < D / 2; c0 += 16) {
        uint32_t o[16];
        tc::tmem_ld(ot + (uint32_t)(buf * (D / 2) + c0), o);
        if (pos < a.n && ok) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float o0 = __uint_as_float(o[2 * e]) * inv, o1 = __uint_as_float(o[2 * e + 1]) * inv;
            bad += (o0 - o0) + (o1 - o1);           // NaN where one is not finite
            const __nv_bfloat162 h = __floats2bfloat162_rn(o0, o1);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" :: "l"(dst + c0),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                         "r"(w[7]) : "memory");
          } else {
            reinterpret_cast<uint4*>(dst + c0)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst + c0)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        __syncwarp();
      }
      if (inv > 0.f && inv < INFINITY) {
        again = again || bad != 0.f;
      } else if (pos < a.n && ok) {                 // the row is NaN whatever the values
        for (int c = 0; c < D / 2; c += 2) *reinterpret_cast<uint32_t*>(dst + c) = kRowNaN;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&oread[x]);
      __syncwarp();
      ++no;
    }
    // (the two warps of a row meet: what one has written the other reads)
    again = __any_sync(0xffffffffu, again);
    float* flags = ssum + ((no & 1) * 2 + x) * 256 + r;
    flags[buf * 128] = again ? 1.f : 0.f;
    __threadfence();
    pair_bar(bar_id);
    again = again || flags[(buf ^ 1) * 128] != 0.f;
    if (again && ok && buf == 0) mend_items<D>(a, x, quarter);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 17) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, kWnTmemCols);
  }
}

// ------------------------------------------------------------------ host side
cudaError_t encode_fn(PFN_cuTensorMapEncodeTiled_v12000* fn) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known;
  return ask_once(known, fn, [](PFN_cuTensorMapEncodeTiled_v12000* answer) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    *answer = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return cudaSuccess;
  });
}

// bf16 map over [units][n][d]: boxes of 64 elements x box_rows positions, 128-byte swizzle, rows
// outside [0, n) read as 0.
cudaError_t make_map(CUtensorMap* m, const void* base, long long units, int n, int d, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (const cudaError_t e = encode_fn(&fn)) return e;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)n, (cuuint64_t)units};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)n * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t run(const kvc_dims& d, int n_sm, const WnArgs& a, cudaStream_t stream) {
  using C = WnCfg<D>;
  const long long units = (long long)d.batch * a.Hk;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_map(&mq, a.q, (long long)d.batch * a.Hq, a.n, D, a.P);
  if (e == cudaSuccess) e = make_map(&mk, a.k, units, a.n, D, kWnKeys);
  if (e == cudaSuccess) e = make_map(&mv, a.v, units, a.n, D, kWnKeys);
  if (e == cudaSuccess) e = ensure_smem(reinterpret_cast<const void*>(window_attn_kernel<D>), C::total);
  if (e != cudaSuccess) return e;
  // the warpgroups' shares add up to the registers the block is launched with
  static std::atomic<int> known;
  int regs = 0;
  e = ask_once(known, &regs, [](int* answer) {
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, reinterpret_cast<const void*>(window_attn_kernel<D>));
    if (e == cudaSuccess) *answer = f.numRegs;
    return e;
  });
  if (e != cudaSuccess) return e;
  if (regs < kWnRegs) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(n_sm, a.items));
  cfg.blockDim = dim3(kWnThreads);
  cfg.dynamicSmemBytes = C::total;
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attr()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, window_attn_kernel<D>, mq, mk, mv, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_window_attn(const kvc_dims& d, int n_sm, int n_sinks, int window,
                               const __nv_bfloat16* q, const __nv_bfloat16* k,
                               const __nv_bfloat16* v, __nv_bfloat16* x_out, unsigned* err,
                               const unsigned* wait_limit, cudaStream_t stream) {
  WnArgs a{};
  a.n = d.prompt_len;
  a.s = std::min(n_sinks, a.n);
  a.W = std::min(window, a.n);
  a.g = d.n_q_heads / d.n_kv_heads;
  a.P = 128 / a.g;
  a.Hq = d.n_q_heads;
  a.Hk = d.n_kv_heads;
  // Items of two row tiles share every key read; of one where that leaves half of the SMs without
  // any, which then have fewer keys to visit (528 tokens of 4 heads, window 128: 8.9 us, was 11.9).
  const long long units = (long long)d.batch * a.Hk;
  a.step = 2 * a.P;
  a.blocks = (a.n + a.step - 1) / a.step;
  if (2 * units * a.blocks <= n_sm) {
    a.step = a.P;
    a.blocks = (a.n + a.step - 1) / a.step;
  }
  a.items = units * a.blocks;
  a.sl2 = 1.4426950408889634f / sqrtf((float)d.head_dim);
  a.q = q;
  a.k = k;
  a.v = v;
  a.x_out = x_out;
  a.err = err;
  a.wait_limit = wait_limit ? *wait_limit : kWnPolls;
  if (d.head_dim == 128) return run<128>(d, n_sm, a, stream);
  return run<64>(d, n_sm, a, stream);
}

}  // namespace kvc
