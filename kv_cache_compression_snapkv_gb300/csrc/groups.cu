// groups.cu -- attention over the packed groups a cheap score selects for each query:
// the score and selection (kvc_select_groups) and the decode attention over listed
// groups (kvc_decode_groups).
//
// Score. A packed group of 32 keys stores, per channel c, its minimum as the zero-point
// Z_c and its range as the scale S_c: every stored key k has lo_c <= k_c <= hi_c with
// lo = Z and hi = Z + (2^b - 1) S. So for a query q
//     max over the group's keys of q . k  <=  sum_c max(q_c lo_c, q_c hi_c),
// and the group's score is the sum of these bounds over the g query heads that share the
// kv head. With D_c = sum_h q_hc and P_c = sum_h max(q_hc, 0) that is
//     sum_c Z_c D_c + S_c (2^b - 1) P_c,
// two products per channel whatever g is, from 4 d of a group's 8 d (b + 1) bytes (1/10 at 4 bits,
// 1/6 at 2).
//
// The list has to be the true one, whatever the order of summation, and scores next to the
// border decide it. So every score is formed in fp32 (one pass over the scales and
// zero-points, two fused multiply-adds a channel), with a bound on the error of all of a
// unit's scores from its largest scale and zero-point; the border is found among the fp32 scores;
// and the few groups that the bound cannot place on either side of it are scored again in
// double-float (products and sums with their rounding errors, by the two-sum of T. J. Dekker
// and D. E. Knuth, good to about 2^-45 of the terms) and ranked by that, ties to the lower
// index. The kernel of one launch does both: the CTA of a unit that finishes last selects.
//
// What bounds it. Long caches: the scattered read (4 d bytes of each 8 d (b + 1)); 160 units of
// 32,768 tokens at 4 bits, 84 MB: 29 us, 2.9 TB/s, where a kernel that only reads 512 of every 5,120
// bytes comes to 6.0 TB/s. The read takes 24 us of it from a cold cache (a CTA of eight warps has 32
// KB in flight, and an SM holds one); 4.4 us are the last unit's selection. Few units: latency; 8
// units of 131,072 tokens, 17 MB: 13.0 us, of which 3.4 us are the read and 4.4 us the selection
// (4,096 scores in registers). Longer units are selected from shared memory (8 units of 6,100 groups:
// 21 us) and, behind 6,144 scores, from global memory as well (8,192 groups 35 us, 16,384 66 us,
// 32,768 139 us: about 1 TB/s of what is read). The smallest call takes 5.4 us in a graph of such
// calls, where a launch with nothing to score takes 0.7 us.
//
// Decode over listed groups (launch_decode_groups) is the decode kernel with a list in place of
// the range: 64 of 1,024 groups of 160 units at 4 bits, 52 MB: 25 us (all groups 215 us); 64 of
// 4,096 groups of 8 units at 2 bits: 12 us (all 51 us). The latter is bound as that kernel is on
// small caches: by the chain of a warp's first copy (here behind the read of its list entries), a
// chunk's unpacking and the merge of the unit's partial states. The former adds five or six
// chunks of one group for each warp, about 1,000 instructions each; three warps a scheduler, each
// waiting for its own results most of the time, use 46 % of the issue slots.
#include "decode_device.cuh"

namespace kvc {
namespace {

constexpr int kSelThreads = 256;       // d / 8 lanes per group, eight channels each
constexpr int kSelFlight = 4;          // groups in flight per lane
constexpr int kSelResident = 2;        // CTAs of an SM
constexpr int kSelHeld = 16;           // scores per thread that the selecting CTA holds in registers
constexpr int kSelBins = 2048;         // of a histogram of the scores' range
constexpr int kSelStaged = 6144;       // scores kept in shared memory by the selecting CTA
constexpr int kSelBorder = 384;        // groups at the border that are ranked in shared memory

struct SelLayer {
  long long packed_off;   // byte offset of the layer in the packed store
  long long key_off;      // element offset of the layer in the scratch
  int n_groups;
  int cap_groups;
  int bits;
};

struct SelParams {
  SelLayer L[KVC_MAX_LAUNCH_LAYERS];
  const uint8_t* packed;
  const __nv_bfloat16* q;        // [layers][units][g][d]
  unsigned long long* keys;      // per unit n words: fp32 scores [n], then each CTA's error scale; or exact keys
  unsigned* cnt;                 // finished CTAs per (layer, unit), zero between launches
  int32_t* out;                  // [layers][units][n_select]
  int units;
  int g;
  int n_select;
  int blocks;                    // CTAs per unit
  int per;                       // groups of one CTA
};

// s + e = a + b exactly.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}
// (s, e) += x (dh + dl)
__device__ __forceinline__ void acc_prod(float& s, float& e, float x, float dh, float dl) {
  const float p = __fmul_rn(x, dh);
  const float r = __fmaf_rn(x, dh, -p);
  float t;
  two_sum(s, p, s, t);
  e = __fadd_rn(e, __fadd_rn(t, __fmaf_rn(x, dl, r)));
}

// Order-preserving integers of scores; a score that is not finite gets 0, below all others.
__device__ __forceinline__ unsigned long long score_key(double v) {
  const long long b = __double_as_longlong(v);
  if ((b & 0x7ff0000000000000ll) == 0x7ff0000000000000ll) return 0ull;
  if (v == 0.0) return 0x8000000000000000ull;   // -0 and +0 are equal
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}
// Order-preserving integer of a float (for maxima and minima by atomics).
__device__ __forceinline__ unsigned ordered(float v) {
  const unsigned b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The exact key of a group, in lane 0 of its d / 8 lanes; scales: the lane's eight key scales
// (the zero-points 2 d bytes further). sq: the query terms by stored position (sum of the heads'
// queries and scaled sum of their positive parts, two floats each).
template <int D>
__device__ __forceinline__ unsigned long long exact_key(const uint8_t* scales, const float4* sq,
                                                        int li) {
  float s = 0.f, e = 0.f;
  const uint4 sv = *reinterpret_cast<const uint4*>(scales);
  const uint4 zv = *reinterpret_cast<const uint4*>(scales + 2 * D);
  const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w}, zw[4] = {zv.x, zv.y, zv.z, zv.w};
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float2 S = __half22float2(u2h(sw[c >> 1])), Z = __half22float2(u2h(zw[c >> 1]));
    const float4 t = sq[li * 8 + c];
    acc_prod(s, e, c & 1 ? Z.y : Z.x, t.x, t.y);
    acc_prod(s, e, c & 1 ? S.y : S.x, t.z, t.w);
  }
#pragma unroll
  for (int o = D / 16; o; o >>= 1) {
    const float s1 = __shfl_xor_sync(0xffffffffu, s, o), e1 = __shfl_xor_sync(0xffffffffu, e, o);
    float t;
    two_sum(s, s1, s, t);
    e = __fadd_rn(__fadd_rn(e, e1), t);
  }
  return score_key((double)s + (double)e);
}

// Shared memory of the selecting CTA.
struct SelShared {
  unsigned hist[kSelBins];
  unsigned wsum[kSelThreads / 32], wtie[kSelThreads / 32];
  unsigned need;          // still to be taken of the digit's groups
  unsigned digit;
  unsigned n_border;
  unsigned long long thr; // exact path: the border's key
  unsigned lo, hi, amax;  // ordered(): smallest and largest score considered, largest error scale
  int last;
};

// The digit (bin of `hist`) that the need-th largest key falls into, counted from the top;
// need becomes its rank among the keys of that digit. All threads; hist is complete.
template <int BINS>
__device__ __forceinline__ void find_digit(SelShared& sh) {
  constexpr int PT = BINS / kSelThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned need = sh.need;
  unsigned c[PT], sum = 0;
#pragma unroll
  for (int k = 0; k < PT; ++k) {      // thread t owns bins BINS - 1 - t PT - k: larger ones first
    c[k] = sh.hist[BINS - 1 - tid * PT - k];
    sum += c[k];
  }
  unsigned incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh.wsum[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl += sh.wsum[w];
  unsigned before = incl - sum;
#pragma unroll
  for (int k = 0; k < PT; ++k) {
    if (before < need && before + c[k] >= need) {
      sh.digit = BINS - 1 - tid * PT - k;
      sh.need = need - before;
    }
    before += c[k];
  }
  __syncthreads();
}

// The scores of a unit with the CTA's threads: in registers (score tid + 256 u in v[u]) where
// they fit, else read again for every pass, from shared memory and from global behind that.
// each(f): f(score, index) for all of them; keep(above): the indices whose score is above
// `above` or marked as taken, ascending, to out.
struct HeldScores {
  float v[kSelHeld];
  unsigned* taken;                    // [kSelThreads] bits u, shared memory, zero at first
  unsigned* counts;                   // [kSelHeld][warps]
  int n;
  __device__ __forceinline__ void range(const float* fkeys, unsigned& lo, unsigned& hi) {
#pragma unroll
    for (int u = 0; u < kSelHeld; ++u) {
      const int i = (int)threadIdx.x + u * kSelThreads;
      v[u] = i < n ? __ldcg(fkeys + i) : -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < kSelHeld; ++u)
      if (v[u] != -INFINITY) {
        lo = min(lo, ordered(v[u]));
        hi = max(hi, ordered(v[u]));
      }
    taken[threadIdx.x] = 0u;
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) {
#pragma unroll
    for (int u = 0; u < kSelHeld; ++u) {
      const int i = (int)threadIdx.x + u * kSelThreads;
      if (i < n) f(v[u], i);
    }
  }
  __device__ __forceinline__ void take(int i) { atomicOr(&taken[i % kSelThreads], 1u << (i / kSelThreads)); }
  __device__ __forceinline__ void drop(int) {}
  // border scores lie in [below, above]
  __device__ __forceinline__ void keep(SelShared& sh, float above, int32_t* out) {
    constexpr int W = kSelThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned mine = taken[threadIdx.x];
    unsigned b[kSelHeld];
#pragma unroll
    for (int u = 0; u < kSelHeld; ++u) {
      b[u] = __ballot_sync(0xffffffffu, v[u] > above || (mine >> u & 1u));
      if (lane == 0) counts[u * W + warp] = __popc(b[u]);
    }
    __syncthreads();
    if (warp == 0) {                  // exclusive sums of the 128 counts
      static_assert(kSelHeld * W == 128, "four counts a lane");
      unsigned c[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) { c[e] = counts[4 * lane + e]; sum += c[e]; }
      unsigned incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      unsigned at = incl - sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) { counts[4 * lane + e] = at; at += c[e]; }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSelHeld; ++u)
      if (b[u] >> lane & 1u)
        out[counts[u * W + warp] + __popc(b[u] & ((1u << lane) - 1u))] = (int)threadIdx.x + u * kSelThreads;
  }
};

struct StagedScores {
  float* staged;                      // [kSelStaged], shared memory
  float* fkeys;
  int n;
  __device__ __forceinline__ float at(int i) const { return i < kSelStaged ? staged[i] : __ldcg(fkeys + i); }
  __device__ __forceinline__ void range(const float*, unsigned& lo, unsigned& hi) {
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      const float x = __ldcg(fkeys + i);
      if (i < kSelStaged) staged[i] = x;
      if (x != -INFINITY) {
        lo = min(lo, ordered(x));
        hi = max(hi, ordered(x));
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) {
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kSelThreads) f(at(i), i);
  }
  __device__ __forceinline__ void mark(int i, float x) {
    if (i < kSelStaged) staged[i] = x;
    else __stcg(fkeys + i, x);
  }
  __device__ __forceinline__ void take(int i) { mark(i, INFINITY); }
  __device__ __forceinline__ void drop(int i) { mark(i, -INFINITY); }
  // each warp takes one contiguous piece: it counts, and writes behind the pieces before
  __device__ __forceinline__ void keep(SelShared& sh, float above, int32_t* out) {
    constexpr int W = kSelThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = (n + kSelThreads - 1) / kSelThreads * 32;
    const int i0 = warp * piece, i1 = min(n, i0 + piece);
    unsigned cnt = 0;
#pragma unroll 4
    for (int i = i0 + lane; i - lane < i1; i += 32)
      cnt += __popc(__ballot_sync(0xffffffffu, i < i1 && at(i) > above));
    if (lane == 0) sh.wsum[warp] = cnt;
    __syncthreads();
    unsigned p = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) p += w < warp ? sh.wsum[w] : 0u;
    for (int i = i0 + lane; i - lane < i1; i += 32) {
      const bool on = i < i1 && at(i) > above;
      const unsigned b = __ballot_sync(0xffffffffu, on);
      if (on) out[p + __popc(b & ((1u << lane) - 1u))] = i;
      p += __popc(b);
    }
  }
};

// Every score exactly, and a radix select of eight 8-bit digits: the path of a unit with more
// groups at the border than shared memory ranks (as a rule equal ones). All threads.
template <int D>
__device__ __noinline__ void select_exact(SelShared& sh, const uint8_t* scales, int bb, const float4* sq,
                                          unsigned long long* keys, int n, int k, int32_t* out) {
  constexpr int LPG = D / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, li = lane % LPG;
  for (int g0 = 0; g0 < n; g0 += kSelThreads / LPG) {
    const int grp = g0 + tid / LPG;
    const unsigned long long x = exact_key<D>(scales + (size_t)min(grp, n - 1) * bb + li * 16, sq, li);
    if (li == 0 && grp < n) __stcg(keys + grp, x);
  }
  if (tid == 0) {
    sh.thr = 0ull;
    sh.need = (unsigned)k;
  }
  __syncthreads();   // (a block's own global writes are visible to it past the barrier)
  for (int shift = 56; shift >= 0; shift -= 8) {
    sh.hist[tid] = 0u;
    __syncthreads();
    const unsigned long long thr = sh.thr;
    for (int i = tid; i < n; i += kSelThreads) {
      const unsigned long long x = __ldcg(keys + i);
      if (shift == 56 || (x >> (shift + 8)) == (thr >> (shift + 8)))
        atomicAdd(&sh.hist[(unsigned)(x >> shift) & 255u], 1u);
    }
    __syncthreads();
    find_digit<256>(sh);
    if (tid == 0) sh.thr = thr | (unsigned long long)sh.digit << shift;
    __syncthreads();
  }
  const unsigned long long thr = sh.thr;
  const unsigned ties = sh.need;    // of the keys equal to thr, the first `ties` are kept
  unsigned tied = 0, done = 0;      // equal / kept keys before this block of indices
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const unsigned long long x = i < n ? __ldcg(keys + i) : 0ull;
    const bool eq = i < n && x == thr;
    const unsigned be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) sh.wtie[warp] = __popc(be);
    __syncthreads();
    unsigned t0 = tied;
    for (int w = 0; w < warp; ++w) t0 += sh.wtie[w];
    const bool on = (i < n && x > thr) || (eq && t0 + __popc(be & ((1u << lane) - 1u)) < ties);
    const unsigned b = __ballot_sync(0xffffffffu, on);
    if (lane == 0) sh.wsum[warp] = __popc(b);
    __syncthreads();
    unsigned p0 = done;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) p0 += sh.wsum[w];
      done += sh.wsum[w];
      tied += sh.wtie[w];
    }
    if (on) out[p0 + __popc(b & ((1u << lane) - 1u))] = i;
    __syncthreads();
  }
}

struct SelWork {          // shared memory of the selection proper
  SelShared sh;
  union {
    float staged[kSelStaged];
    struct {
      unsigned taken[kSelThreads], counts[kSelHeld * kSelThreads / 32];
    } held;
  } u;
  int32_t border[kSelBorder];
  unsigned long long bkey[kSelBorder];
};

// The list of one unit from its n fp32 scores (fkeys; nblk error scales behind them). All threads
// of the CTA.
template <int D, typename Scores>
__device__ __forceinline__ void select_unit(Scores& sc, SelWork& wk, const uint8_t* scales, int bb,
                                            const float4* sq, float* fkeys, int nblk, int n, int k,
                                            int32_t* out) {
  constexpr int LPG = D / 8, STEP = kSelThreads / LPG;
  SelShared& sh = wk.sh;
  const int tid = threadIdx.x, lane = tid & 31, li = lane % LPG, warp = tid >> 5;
  // The scores' range (of those that are finite) and the largest error scale.
  auto join_range = [&](unsigned lo_o, unsigned hi_o) {
    lo_o = __reduce_min_sync(0xffffffffu, lo_o);
    hi_o = __reduce_max_sync(0xffffffffu, hi_o);
    if (lane == 0) {
      atomicMin(&sh.lo, lo_o);
      atomicMax(&sh.hi, hi_o);
    }
  };
  {
    unsigned lo_o = 0xffffffffu, hi_o = 0u;
    float am = 0.f;
    for (int i = tid; i < nblk; i += kSelThreads) am = fmaxf(am, __ldcg(fkeys + n + i));
    sc.range(fkeys, lo_o, hi_o);
    const unsigned am_o = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
    if (lane == 0) atomicMax(&sh.amax, am_o);
    join_range(lo_o, hi_o);
  }
  __syncthreads();
  // The k-th largest score's bin among kSelBins of the range, then of that bin's own range while
  // it holds more groups than the border may (a few far scores can leave the others in one bin).
  // A bin is a monotone function of the score, so bins are in the scores' order.
  const float eps = __uint_as_float(sh.amax) * 0x1p-18f;
  float lo = unordered(sh.lo), hi = unordered(sh.hi);
  bool open = sh.hi == 0u;            // no score is finite
#pragma unroll 1
  for (int round = 0; round < 4 && !open; ++round) {
    __syncthreads();
#pragma unroll
    for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[i] = 0u;
    if (tid == 0) {
      sh.lo = 0xffffffffu;
      sh.hi = 0u;
      sh.digit = 0xffffffffu;
    }
    __syncthreads();
    const float scale = hi > lo ? (float)kSelBins / (hi - lo) : 0.f;
    auto bin_of = [&](float v) { return min(kSelBins - 1, (int)((v - lo) * scale)); };
    sc.each([&](float v, int) {
      if (v >= lo && v <= hi) atomicAdd(&sh.hist[bin_of(v)], 1u);
    });
    __syncthreads();
    find_digit<kSelBins>(sh);
    const int bin = (int)sh.digit;
    if (bin < 0) {                    // fewer finite scores than k: the border is at those that are not
      open = true;
      break;
    }
    const int in_bin = (int)sh.hist[bin];
    if (in_bin <= kSelBorder / 2 && scale < INFINITY) {
      // Few enough: the bin's edges stand for its scores' range (a pass over them less: 0.4 us). A
      // score's place among the bins is off by 2^-21 of the range at most (three roundings of
      // it, one of the scale's two), the edges by 2^-24 of their size and 2^-23 of the range.
      const float w = (hi - lo) * (1.f / kSelBins);
      const float room = fmaf(hi - lo, 0x1p-20f, fmaxf(fabsf(lo), fabsf(hi)) * 0x1p-22f);
      const float e0 = fmaf((float)bin, w, lo) - room, e1 = fmaf((float)(bin + 1), w, lo) + room;
      lo = fmaxf(lo, e0);
      if (bin < kSelBins - 1) hi = fminf(hi, e1);
      break;
    }
    unsigned lo_o = 0xffffffffu, hi_o = 0u;
    sc.each([&](float v, int) {
      if (v >= lo && v <= hi && bin_of(v) == bin) {
        lo_o = min(lo_o, ordered(v));
        hi_o = max(hi_o, ordered(v));
      }
    });
    join_range(lo_o, hi_o);
    __syncthreads();
    lo = unordered(sh.lo);
    hi = unordered(sh.hi);
    if (!(hi - lo > eps)) break;
  }
  // The k-th largest fp32 score lies in [lo, hi]. A score is off by at most 12 roundings of the
  // sum of its terms' magnitudes (four fused multiply-adds a lane and sum, two joins, four
  // exchanges, two of the query term itself), 3/4 of 2^-20 of it; that sum is at most max |Z| sum |D|
  // + max S sum P over the groups of its warp, whose maximum over the unit is the error scale. Two
  // scores can so change places if they are within 3/4 of 2^-19. eps is 2^-18 of the scale: a group
  // above hi + eps belongs to the list, one below lo - eps does not, and the others are at the
  // border. (A score that is not finite is stored as -inf; only a border at -inf holds it.)
  const float above = open ? -INFINITY : hi + eps, below = open ? -INFINITY : lo - eps;
  unsigned sure = 0;
  sc.each([&](float v, int i) {
    if (v > above) {
      ++sure;
    } else if (v >= below) {
      const unsigned at = atomicAdd(&sh.n_border, 1u);
      if (at < kSelBorder) wk.border[at] = i;
    }
  });
  sure = __reduce_add_sync(0xffffffffu, sure);
  if (lane == 0) sh.wtie[warp] = sure;
  __syncthreads();
  unsigned all = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) all += sh.wtie[w];
  const int nb = (int)sh.n_border, take = k - (int)all;   // 0 < take <= nb
  if (nb > kSelBorder) {
    select_exact<D>(sh, scales - li * 16, bb, sq, reinterpret_cast<unsigned long long*>(fkeys), n, k, out);
    return;
  }
  if (take < nb) {                    // (else all of the border belongs to the list)
    for (int c0 = 0; c0 < nb; c0 += STEP) {
      const int c = c0 + tid / LPG;
      const unsigned long long x = exact_key<D>(scales + (size_t)wk.border[min(c, nb - 1)] * bb, sq, li);
      if (li == 0 && c < nb) wk.bkey[c] = x;
    }
    __syncthreads();
  }
  for (int c = tid; c < nb; c += kSelThreads) {
    const int i = wk.border[c];
    int rank = 0;
    if (take < nb) {
      const unsigned long long x = wk.bkey[c];
      for (int j = 0; j < nb; ++j) rank += wk.bkey[j] > x || (wk.bkey[j] == x && wk.border[j] < i);
    }
    if (rank < take) sc.take(i);
    else sc.drop(i);
  }
  __syncthreads();
  sc.keep(sh, above, out);
}

// One CTA: P.per groups of one (layer, unit); the unit's last one selects.
template <int D>
__global__ void __launch_bounds__(kSelThreads, kSelResident)
select_groups_kernel(const __grid_constant__ SelParams P) {
  constexpr int LPG = D / 8, STEP = kSelThreads / LPG, U = kSelFlight;
  __shared__ float4 sq[D];
  __shared__ SelWork wk;
  SelShared& sh = wk.sh;
  const SelLayer& L = P.L[blockIdx.y];
  const int unit = blockIdx.x / P.blocks, blk = blockIdx.x % P.blocks;
  const int tid = threadIdx.x, lane = tid & 31, li = lane % LPG;
  const int n = L.n_groups, k = P.n_select;
  int32_t* out = P.out + ((size_t)blockIdx.y * P.units + unit) * k;
  if (tid == 0) sh.hi = sh.amax = 0u;
  __syncthreads();
  pdl_wait();
  pdl_release();
  if (n <= k) {                       // every group
    if (blk == 0)
      for (int i = tid; i < k; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int nblk = (n + P.per - 1) / P.per;
  if (blk >= nblk) return;
  const int bb = block_bytes(D, L.bits);
  const uint8_t* scales =
      P.packed + L.packed_off + (size_t)unit * L.cap_groups * bb + off_kscale(D, L.bits) + li * 16;
  // The queries first, then the first groups' scales, which are on their way while the query
  // terms are formed.
  float x[8];
  if (tid < D) {
    const __nv_bfloat16* q = P.q + ((size_t)blockIdx.y * P.units + unit) * P.g * D + tid;
#pragma unroll
    for (int h = 0; h < 8; ++h) x[h] = h < P.g ? __bfloat162float(q[(size_t)h * D]) : 0.f;
  }
  const int g_end = min(n, (blk + 1) * P.per), first = blk * P.per + tid / LPG;
  uint4 sv[U] = {}, zv[U] = {};
  auto fetch = [&](int grp, uint4& s, uint4& z) {
    if (grp < g_end) {
      const uint8_t* p = scales + (size_t)grp * bb;
      s = *reinterpret_cast<const uint4*>(p);
      z = *reinterpret_cast<const uint4*>(p + 2 * D);
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(first + u * STEP, sv[u], zv[u]);
  // Query terms per stored position, each as two floats: the sum of the heads' queries (two-sum:
  // exact) and (2^b - 1) times the sum of their positive parts; scaled by a power of two so that
  // the largest magnitude is below 4 (no product can then overflow).
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (tid < D) {
    float mx = 0.f;
#pragma unroll
    for (int h = 0; h < 8; ++h) mx = fmaxf(mx, fabsf(x[h]));
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    if (lane == 0) atomicMax(&sh.hi, __float_as_uint(mx));
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      float e;
      two_sum(t.x, x[h], t.x, e);
      t.y += e;
      two_sum(t.z, fmaxf(x[h], 0.f), t.z, e);
      t.w += e;
      if (x[h] != x[h]) t.z = x[h];    // (fmaxf drops it)
    }
    // (heads that cancel may have left the sum in the second float: the fp32 scores read the first)
    two_sum(t.x, t.y, t.x, t.y);
    two_sum(t.z, t.w, t.z, t.w);
  }
  __syncthreads();
  if (tid < D) {
    // |x| < 2^(ex - 126), sums of eight below 2^(ex - 123), positive ones times 15 below 2^(ex - 119):
    // scaled by 2^(121 - ex) in two steps, each inside the exponent range
    const int ex = min(max((int)(sh.hi >> 23), 1), 254);
    const int sc = 121 - ex, h = sc / 2;   // from -133 to 120
    const float f0 = __int_as_float((127 + h) << 23), f1 = __int_as_float((127 + sc - h) << 23);
    const float m = (float)((1 << L.bits) - 1);
    t.x = t.x * f0 * f1;
    t.y = t.y * f0 * f1;
    const float hi = t.z * f0 * f1, lo = t.w * f0 * f1;
    t.z = hi * m;
    t.w = fmaf(lo, m, fmaf(hi, m, -t.z));
    sq[kperm(tid, D)] = t;
  }
  __syncthreads();
  float2 dq[4], pq[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 a = sq[li * 8 + 2 * c], b = sq[li * 8 + 2 * c + 1];
    dq[c] = make_float2(a.x, b.x);
    pq[c] = make_float2(a.z, b.z);
  }
  float* fkeys = reinterpret_cast<float*>(P.keys + L.key_off + (size_t)unit * n);
  __half2 mz = __float2half2_rn(0.f), ms = mz;   // largest magnitudes
#pragma unroll 1
  for (int g0 = first; g0 - tid / LPG < g_end; g0 += U * STEP) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int grp = g0 + u * STEP;
      float2 v2 = make_float2(0.f, 0.f), w2 = v2;   // sums of Z D and S P
      const uint32_t sw[4] = {sv[u].x, sv[u].y, sv[u].z, sv[u].w};
      const uint32_t zw[4] = {zv[u].x, zv[u].y, zv[u].z, zv[u].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v2 = __ffma2_rn(__half22float2(u2h(zw[c])), dq[c], v2);
        w2 = __ffma2_rn(__half22float2(u2h(sw[c])), pq[c], w2);
        mz = __hmax2(mz, __habs2(u2h(zw[c])));
        ms = __hmax2(ms, u2h(sw[c]));
      }
      fetch(grp + U * STEP, sv[u], zv[u]);
      float v = (v2.x + v2.y) + (w2.x + w2.y);
#pragma unroll
      for (int o = LPG / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (li == 0 && grp < g_end) __stcg(fkeys + grp, isfinite(v) ? v : -INFINITY);
    }
  }
  {
    // the error scale of the warp's groups: max |Z| sum |D| + max S sum P, the CTA's is the largest
    // (infinite maxima belong to groups that rank last anyway: the largest finite value stands in)
    float d1 = 0.f, p1 = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      d1 += fabsf(dq[c].x) + fabsf(dq[c].y);
      p1 += pq[c].x + pq[c].y;
    }
#pragma unroll
    for (int o = LPG / 2; o; o >>= 1) {
      d1 += __shfl_xor_sync(0xffffffffu, d1, o);
      p1 += __shfl_xor_sync(0xffffffffu, p1, o);
    }
    auto warp_max = [](__half2 v) {   // (magnitudes: their bits are in their order)
      const float m = fminf(fmaxf(__low2float(v), __high2float(v)), 65504.f);
      return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    };
    const float z1 = warp_max(mz), s1 = warp_max(ms);
    if (lane == 0) atomicMax(&sh.amax, __float_as_uint(fmaxf(z1 * d1 + s1 * p1, 0.f)));
  }
  __syncthreads();
  if (tid == 0) {
    sh.last = 1;
    __stcg(fkeys + n + blk, __uint_as_float(sh.amax));
    if (nblk > 1) {
      unsigned* cnt = P.cnt + (size_t)blockIdx.y * P.units + unit;
      __threadfence();                // (after the barrier: releases the whole CTA's scores)
      sh.last = atomicAdd(cnt, 1u) == (unsigned)(nblk - 1);
      if (sh.last) *cnt = 0u;         // ready for the next launch
      __threadfence();
    }
    sh.need = (unsigned)k;
    sh.n_border = 0u;
    sh.lo = 0xffffffffu;
    sh.hi = 0u;
    sh.amax = 0u;
  }
  __syncthreads();
  if (!sh.last) return;
  if (n <= kSelHeld * kSelThreads) {
    HeldScores sc;
    sc.taken = wk.u.held.taken;
    sc.counts = wk.u.held.counts;
    sc.n = n;
    select_unit<D>(sc, wk, scales, bb, sq, fkeys, nblk, n, k, out);
  } else {
    StagedScores sc{wk.u.staged, fkeys, n};
    select_unit<D>(sc, wk, scales, bb, sq, fkeys, nblk, n, k, out);
  }
}

cudaError_t launch_pdl(const void* kernel, dim3 grid, int threads, void** args,
                       cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attr()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace

size_t select_keys(const kvc_cache* c) {
  size_t n = 0;
  for (const LayerState& ls : c->L)
    n += (size_t)c->dims.batch * c->dims.n_kv_heads * ls.cap_groups;
  return n;
}

cudaError_t launch_select_groups(const kvc_cache* c, int layer_begin, int layer_count,
                                 const __nv_bfloat16* q, int n_select, int32_t* groups,
                                 cudaStream_t stream) {
  const kvc_dims& d = c->dims;
  const int units = d.batch * d.n_kv_heads;
  for (int base = 0; base < layer_count; base += KVC_MAX_LAUNCH_LAYERS) {
    const int cnt = std::min(layer_count - base, KVC_MAX_LAUNCH_LAYERS);
    SelParams P;
    P.packed = c->packed;
    P.q = q + (size_t)base * units * c->g * d.head_dim;
    P.keys = c->sel_keys;
    P.cnt = c->dec_cnt;
    P.out = groups + (size_t)base * units * n_select;
    P.units = units;
    P.g = c->g;
    P.n_select = n_select;
    long long off = 0;
    int most = 0;
    for (int i = 0; i < cnt; ++i) {
      const LayerState& ls = c->L[layer_begin + base + i];
      P.L[i] = {(long long)ls.packed_off, off, ls.n_groups, ls.cap_groups, ls.bits};
      off += (long long)units * ls.n_groups;
      if (ls.n_groups > n_select) most = std::max(most, ls.n_groups);
    }
    // Groups of a CTA: what its threads have in flight at once, or, where that makes more CTAs
    // than the device holds at once, the fewest times as much that does not: each CTA forms
    // the query terms anew (160 units of 1,024 groups: 160 CTAs 29 us, 320 or 640 CTAs 32 us; 8
    // units of 4,094: 256 CTAs).
    const int step = kSelFlight * kSelThreads / (d.head_dim / 8);
    auto ctas = [&](long long per) {
      long long n = 0;
      for (int i = 0; i < cnt; ++i)
        if (P.L[i].n_groups > n_select) n += units * ((P.L[i].n_groups + per - 1) / per);
      return n;
    };
    // (bisected: the CTAs fall as `per` grows, and a launch has many layers and lengths)
    int least = 1, enough = std::max(1, (most + step - 1) / step);
    while (least < enough) {
      const int m = least + (enough - least) / 2;
      if (ctas((long long)step * m) <= (long long)kSelResident * c->n_sm) enough = m;
      else least = m + 1;
    }
    P.per = step * enough;
    P.blocks = std::max(1, (most + P.per - 1) / P.per);
    void* args[1] = {&P};
    const void* fn = d.head_dim == 128 ? reinterpret_cast<const void*>(select_groups_kernel<128>)
                                       : reinterpret_cast<const void*>(select_groups_kernel<64>);
    cudaError_t e = launch_pdl(fn, dim3((unsigned)units * P.blocks, cnt), kSelThreads, args, stream);
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaGetLastError();
}

cudaError_t launch_decode_groups(const kvc_cache* c, int layer_begin, int layer_count,
                                 const __nv_bfloat16* q, int n_select, const int32_t* groups,
                                 float* out, cudaStream_t stream) {
  const kvc_dims& d = c->dims;
  const int units = d.batch * d.n_kv_heads;
  const size_t gq = (size_t)c->g * d.head_dim;
  for (int base = 0; base < layer_count; base += KVC_MAX_LAUNCH_LAYERS) {
    const int cnt = std::min(layer_count - base, KVC_MAX_LAUNCH_LAYERS);
    DecParams P;
    P.n_layers = cnt;
    P.layer_begin = layer_begin + base;
    P.units = units;
    P.sl2 = 1.4426950408889634f / sqrtf((float)d.head_dim);
    P.err = c->err;
    P.ws = c->dec_ws;
    P.cnt = c->dec_cnt;
    P.wait_limit = c->wait_limit_set ? c->wait_limit : kWaitLimit;
    P.k_new = nullptr;
    P.v_new = nullptr;
    P.groups = groups + (size_t)base * units * n_select;
    P.n_select = n_select;
    P.wide = c->wide;
    long long total = 0;
    int bmask = 0;
    float* ob = out + (size_t)base * units * gq;
    for (int i = 0; i < cnt; ++i) {
      const LayerState& ls = c->L[layer_begin + base + i];
      DecLayer& L = P.L[i];
      L.cap_groups = ls.cap_groups;
      L.packed_off = (long long)ls.packed_off;
      L.win_off = (long long)ls.win_off;
      L.R = ls.R;
      L.bits = ls.bits;
      L.gpc = dec_groups_per_chunk(d.head_dim, ls.bits == 16 ? 2 : ls.bits);
      L.new_slot = -1;
      L.n_groups = ls.n_groups;
      L.win_start = ls.win_start;
      L.win_len = ls.win_len;
      L.wchunks = (L.win_len + kSlotsPerWarp - 1) / kSlotsPerWarp;
      L.pchunks = ls.n_groups > 0 ? (n_select + L.gpc - 1) / L.gpc : 0;
      L.chunk_begin = total;
      total += (long long)units * (L.wchunks + L.pchunks);
      if (L.pchunks > 0) bmask |= ls.bits == 2 ? 1 : 2;
      if (L.wchunks + L.pchunks == 0) {   // a layer that holds no token: the output is zero
        cudaError_t e = cudaMemsetAsync(ob + (size_t)i * units * gq, 0, units * gq * 4, stream);
        if (e != cudaSuccess) return e;
      }
    }
    P.total = total;
    if (total == 0) continue;
    cudaError_t e = launch_bits<true>(P, c, bmask, q + (size_t)base * units * gq, ob, stream);
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace kvc
