// window_tc.cu -- prompt attention over a sliding window and the first tokens (sinks) on the
// 5th-generation tensor cores (kvc_prefill_window).
//
//   o_i = sum_j p_ij v_j,  p_i = softmax_j(q_i . k_j / sqrt(d)),  j <= i and (j < s or i - j < W).
//
// Work: an item is (unit = (sequence, kv head), 2 P consecutive positions), P = 128 / g positions for
// each of the g query heads making a tile of 128 rows, two tiles an item, so that every key read
// serves 256 rows. An item visits the keys [0, s) in front of its first row's window in tiles of
// 128, then the keys from that window's first on; a tile that one of the two row tiles does not see
// is left out for it. Keys and values stream through a ring of 128-row stages by TMA from maps
// of [unit][position][channel], whose rows past the prompt read as 0.
//
// Per key tile and row tile x: S_x = Q_x . K^T in tensor memory (128 columns); the eight warps of
// group x take a row in two halves of 64 columns, a thread each: maximum (of both, exchanged in
// shared memory), P = exp2 into the same columns as bf16, sums in fp32; then
// O_x += P_x . V with P read from tensor memory. The product warp issues, tile x in turn,
// O_x += P_x(t) V(t) and S_x(t + 1) = Q_x K(t + 1): while group 0 forms its weights, the products of
// group 1 run, and the other way round. S_x(t + 1) is published by a commit that follows O_x's product
// of tile t, so a group that has S_x(t + 1) may change O_x and write P_x(t + 1).
//
// A row's weights are taken against a reference that follows its running maximum only when that
// has grown by more than 2^8 (then O_x is rescaled): P stays below 2^8 and its sums in fp32. Sums
// are of the fp32 weights; P itself is rounded to bf16 (2^-8 of each weight).
//
// Values that are not finite reach, through a weight of 0, rows that do not see them. A group
// that has written such a row goes over its items once more at the end, and forms the rows
// that hold something not finite again, from the keys that they see and no others.
//
// Roles: warps 0..7 and 8..15 the two groups, warp 16 the copies, warp 17 tensor memory and products.
// Every wait is bounded; one that gives up sets a bit of the error word, and its warp goes on without
// further waits (the pairs of warps that share rows meet at barriers all the same).
#include <algorithm>
#include <cudaTypedefs.h>

#include "kvc_internal.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr int kWnGroupWarps = 8;
constexpr int kWnThreads = 32 * (2 * kWnGroupWarps + 2);
constexpr int kWnTmemCols = 512;
constexpr int kWnSmemLimit = 232448;   // opt-in shared memory per CTA
constexpr float kWnSlack = 8.f;        // log2 units a maximum may pass its reference by
constexpr unsigned kWnPolls = 1u << 14;   // polls of one wait before it gives up
constexpr unsigned kWnPollNs = 20000u;    // a poll waits up to this long

enum : unsigned { kErrWnCopy = 1u << 16, kErrWnMma = 1u << 17, kErrWnGroup = 1u << 18 };

template <int D>
struct WnCfg {
  static constexpr int KB = D / 64;                // 64-element blocks of a row
  static constexpr int TB = 128 * D * 2;           // one 128-row bf16 tile
  static constexpr int FIT = (kWnSmemLimit - 2 * TB - 6144) / TB;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * TB;
  static constexpr int oBar = oKV + STAGES * TB;
  // full[S], empty[S], qfull[2], qempty[2], sfull[2], pfull[2], ofull[2], drain
  static constexpr int NBAR = 2 * STAGES + 11;
  static constexpr int oTmem = oBar + NBAR * 8;
  // [2 tiles in turn][2 groups][2 halves][128 rows] maxima; sums use the first
  static constexpr int oMax = (oTmem + 16 + 15) / 16 * 16;
  static constexpr int total = oMax + 2 * 2 * 2 * 128 * 4 + 1024;   // + alignment slack
  static_assert(STAGES >= 4, "two tiles of keys and values");
  static_assert(total <= kWnSmemLimit, "fits the shared memory of one CTA");
};

struct WnArgs {
  int n, s, W;     // prompt length, sinks, window (neither above n)
  int g, P;        // query heads per kv head, positions per row tile (128 / g)
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
  __device__ __forceinline__ bool active(int x, int t) const {
    return t < hi(x) && (t < ts || t >= lo(x));
  }
  __device__ __forceinline__ int first(int x) const { return ts > 0 ? 0 : lo(x); }
  __device__ __forceinline__ int last(int x) const { return hi(x) - 1; }
  __device__ __forceinline__ int key0(int t) const { return t < ts ? t * 128 : j0 + (t - ts) * 128; }
};
__device__ __forceinline__ Item item_of(long long i, const WnArgs& a) {
  Item it;
  it.unit = i >> 32 ? (int)(i / a.blocks) : (int)((unsigned)i / (unsigned)a.blocks);
  it.p0 = (int)(i - (long long)it.unit * a.blocks) * 2 * a.P;
  it.j0 = max(0, it.p0 - (a.W - 1));
  it.s0 = min(a.s, it.j0);
  it.ts = (it.s0 + 127) / 128;
  it.T = it.ts + (min(it.p0 + 2 * a.P, a.n) - 1 - it.j0) / 128 + 1;
  auto tiles = [&](int q0, int& lo, int& hi) {
    const int from = a.s > it.j0 ? it.j0 : max(it.j0, q0 - (a.W - 1));
    lo = it.ts + (from - it.j0) / 128;
    hi = q0 < a.n ? it.ts + (min(q0 + a.P, a.n) - 1 - it.j0) / 128 + 1 : 0;   // 0: no row of the prompt
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
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(b), "r"((uint32_t)(phase & 1)), "r"(kWnPollNs) : "memory");
    if (done) return true;
  }
  return gave_up(err, errbit);
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One row again, by one warp, from the keys that it sees alone (for a row that came out not finite).
template <int D>
__device__ __noinline__ void row_again(const WnArgs& a, int unit, int head, int pos) {
  const int lane = threadIdx.x & 31;
  const size_t b = unit / a.Hk;
  const size_t qrow = (b * a.Hq + (size_t)(unit % a.Hk) * a.g + head) * a.n + pos;
  const __nv_bfloat16* q = a.q + qrow * D;
  const __nv_bfloat16* k = a.k + (size_t)unit * a.n * D;
  const __nv_bfloat16* v = a.v + (size_t)unit * a.n * D;
  constexpr int C = D / 32;
  float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  const int w0 = max(0, pos - (a.W - 1)), s1 = min(a.s, w0);
  for (int part = 0; part < 2; ++part) {
    const int e = part ? pos + 1 : s1;
    for (int j0 = part ? w0 : 0; j0 < e; j0 += 32) {
      const int j = j0 + lane;
      float x = -INFINITY;
      if (j < e) {
        x = 0.f;
        for (int c = 0; c < D; ++c)
          x = fmaf(__bfloat162float(q[c]), __bfloat162float(k[(size_t)j * D + c]), x);
      }
      float top = x;
#pragma unroll
      for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      top = fmaxf(top, m);
      const float f = m == -INFINITY ? 0.f : ex2((m - top) * a.sl2);
      m = top;
      const float p = j >= e ? 0.f : ex2((x - (m == -INFINITY ? 0.f : m)) * a.sl2);
      l = l * f + p;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] *= f;
      for (int i = 0; i < min(32, e - j0); ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i);
#pragma unroll
        for (int c = 0; c < C; ++c)
          o[c] = fmaf(pi, __bfloat162float(v[(size_t)(j0 + i) * D + lane * C + c]), o[c]);
      }
    }
  }
#pragma unroll
  for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
#pragma unroll
  for (int c = 0; c < C; ++c) a.x_out[qrow * D + lane * C + c] = __float2bfloat16_rn(o[c] / l);
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
  uint64_t* qempty = qfull + 2;
  uint64_t* sfull = qfull + 4;
  uint64_t* pfull = qfull + 6;
  uint64_t* ofull = qfull + 8;
  uint64_t* drain = qfull + 10;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(dsm + C::oTmem);
  float* smax = reinterpret_cast<float*>(dsm + C::oMax);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) { tc::mbar_init(&full[s], 1); tc::mbar_init(&empty[s], 1); }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(&qfull[x], 1);
      tc::mbar_init(&qempty[x], 1);
      tc::mbar_init(&sfull[x], 1);
      tc::mbar_init(&pfull[x], kWnGroupWarps);
      tc::mbar_init(&ofull[x], 1);
    }
    tc::mbar_init(drain, 1);
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmQ);
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
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

  if (warp == 16) {
    // --------------------------------------------------------------- copies
    if (lane == 0) {
      int k = 0, nq[2] = {0, 0};
      auto stage = [&](const CUtensorMap* map, int row, int unit) {
        const int s = k % C::STAGES, round = k / C::STAGES;
        if (round > 0) ok = wn_wait(&empty[s], round - 1, a.wait_limit, a.err, kErrWnCopy);
        if (!ok) return;
        tc::mbar_expect_tx(&full[s], (uint32_t)C::TB);
        for (int kb = 0; kb < C::KB; ++kb)
          tma_load_3d(sKV + s * C::TB + kb * 128 * 128, map, kb * 64, row, unit, &full[s]);
        ++k;
      };
      for (long long i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
        const Item it = item_of(i, a);
        const int b = it.unit / a.Hk, hk = it.unit % a.Hk;
        for (int t = 0; t < it.T && ok; ++t) {
          if (t == 0) {
            for (int x = 0; x < 2 && ok; ++x) {
              if (!it.live(x)) continue;
              if (nq[x] > 0) ok = wn_wait(&qempty[x], nq[x] - 1, a.wait_limit, a.err, kErrWnCopy);
              if (!ok) break;
              tc::mbar_expect_tx(&qfull[x], (uint32_t)C::TB);
              for (int hh = 0; hh < a.g; ++hh)
                for (int kb = 0; kb < C::KB; ++kb)
                  tma_load_3d(sQ + x * C::TB + kb * 128 * 128 + hh * a.P * 128, &tmQ, kb * 64,
                              it.p0 + x * a.P, b * a.Hq + hk * a.g + hh, &qfull[x]);
              ++nq[x];
            }
          }
          if (ok) stage(&tmK, it.key0(t), it.unit);
          if (ok) stage(&tmV, it.key0(t), it.unit);
        }
      }
      // every copy issued here has landed before the CTA can leave
      for (int kk = max(0, k - C::STAGES); kk < k; ++kk)
        wn_wait(&full[kk % C::STAGES], kk / C::STAGES, kWnPolls, a.err, kErrWnCopy);
      for (int x = 0; x < 2; ++x)
        if (nq[x] > 0) wn_wait(&qfull[x], nq[x] - 1, kWnPolls, a.err, kErrWnCopy);
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------- products
    constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128);
    constexpr uint32_t idesc_o = tc::idesc_ts(128, D, true, true);
    const uint32_t sQa = tc::saddr(sQ), sKVa = tc::saddr(sKV);
    int nq[2] = {0, 0}, np[2] = {0, 0};
    int k = 0;                       // stages waited for: keys of the next tile, values of this one
    struct Cur { long long i; Item it; int t; };
    auto wait = [&](uint64_t* b, int phase) {
      if (ok) ok = wn_wait(b, phase, a.wait_limit, a.err, kErrWnMma);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
    };
    // S_x of tile c, whose keys lie in stage s
    auto scores = [&](const Cur& c, int x, int s) {
      if (!c.it.active(x, c.t)) return;
      if (c.t == c.it.first(x)) wait(&qfull[x], nq[x]++);
      if (!ok) return;
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int at = (kk / 4) * 128 * 128 + (kk % 4) * 32;
          tc::mma_bf16(tbase + x * 128u, tc::sw128_desc(sQa + x * C::TB + at),
                       tc::sw128_desc(sKVa + s * C::TB + at), idesc_s, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit(&sfull[x]);
        if (c.t == c.it.last(x)) tc::mma_commit(&qempty[x]);
      }
      __syncwarp();
    };
    Cur nxt{blockIdx.x, item_of(blockIdx.x, a), 0};
    wait(&full[0], 0);
    for (int x = 0; x < 2 && ok; ++x) scores(nxt, x, 0);
    if (ok && tc::elect_one()) tc::mma_commit(&empty[0]);
    __syncwarp();
    ++k;
    while (ok) {
      const Cur cur = nxt;
      if (++nxt.t == cur.it.T) {
        nxt.t = 0;
        nxt.i += gridDim.x;
        if (nxt.i < a.items) nxt.it = item_of(nxt.i, a);
      }
      const bool more = nxt.i < a.items;
      const int sv = k % C::STAGES, sk = (k + 1) % C::STAGES;
      wait(&full[sv], k / C::STAGES);
      for (int x = 0; x < 2 && ok; ++x) {
        if (cur.it.active(x, cur.t)) {
          wait(&pfull[x], np[x]++);
          if (!ok) break;
          if (tc::elect_one()) {
            const uint32_t acc = cur.t > cur.it.first(x) ? 1u : 0u;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)   // A = P (keys along K); B = V, its rows the keys
              tc::mma_ts(tbase + 256u + x * (uint32_t)D, tbase + x * 128u + kk * 8u,
                         tc::sw128_mn_desc(sKVa + sv * C::TB + kk * 16 * 128, 128 * 128, 1024),
                         idesc_o, kk > 0 ? 1u : acc);
            if (cur.t == cur.it.last(x)) tc::mma_commit(&ofull[x]);
          }
          __syncwarp();
        }
        if (x == 1) {
          if (tc::elect_one()) tc::mma_commit(&empty[sv]);
          __syncwarp();
        }
        if (more) {
          if (x == 0) wait(&full[sk], (k + 1) / C::STAGES);
          if (ok) scores(nxt, x, sk);
        }
      }
      if (!ok || !more) break;
      if (tc::elect_one()) tc::mma_commit(&empty[sk]);
      __syncwarp();
      k += 2;
    }
    // every product issued here has completed before tensor memory is released
    if (tc::elect_one()) tc::mma_commit(drain);
    __syncwarp();
    wn_wait(drain, 0, kWnPolls, a.err, kErrWnMma);
  } else {
    // --------------------------------------------------------------- groups
    const int x = warp >> 3, quarter = warp & 3, half = (warp >> 2) & 1;
    const int r = quarter * 32 + lane;              // row of the tile: head * P + position
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t st = tbase + lane_addr + x * 128u + half * 64u;
    const uint32_t pt = tbase + lane_addr + x * 128u + half * 32u;
    const uint32_t ot = tbase + lane_addr + 256u + x * (uint32_t)D + half * (uint32_t)(D / 2);
    const int hh = r / a.P, dp = x * a.P + r % a.P;
    const int bar_id = 1 + x * 4 + quarter;         // the two warps that share rows
    float* mx_own = smax + x * 256 + half * 128 + r;          // [2][2 groups][2 halves][128]
    const float* mx_other = smax + x * 256 + (half ^ 1) * 128 + r;
    int ns = 0, no = 0;                             // S tiles and outputs so far
    bool again = false;                             // some row came out not finite
    auto wait = [&](uint64_t* b, int phase) {
      if (ok) ok = wn_wait(b, phase, a.wait_limit, a.err, kErrWnGroup);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
    };
    for (long long i = blockIdx.x; i < a.items; i += gridDim.x) {
      const Item it = item_of(i, a);
      if (!it.live(x)) continue;
      const int pos = it.p0 + dp;
      const int q0 = it.p0 + x * a.P, q1 = q0 + a.P - 1;   // the tile's positions
      const int t1 = it.hi(x), t_lo = it.lo(x);
      float ref = -INFINITY, lsum = 0.f;            // reference of the weights (log2 units), their sum
      for (int t = it.first(x); t < t1; t = t + 1 == it.ts ? t_lo : t + 1) {
        wait(&sfull[x], ns);
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
        const int key0 = it.key0(t) + half * 64;
        if (t < it.ts) {
          if (key0 + 64 > it.s0) {
            const int lim = it.s0 - key0;
#pragma unroll
            for (int c = 0; c < 64; ++c) v[c] = c < lim ? v[c] : -INFINITY;
          }
        } else if (key0 + 63 > q0 || key0 < q1 - (a.W - 1)) {
          // seen: up to the row's own key, from its window's first on or a sink
          const int hi = pos - key0, lo = pos - (a.W - 1) - key0, sk = a.s - key0;
#pragma unroll
          for (int c = 0; c < 64; ++c) v[c] = c <= hi && (c >= lo || c < sk) ? v[c] : -INFINITY;
        }
        float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
        for (int c = 4; c < 60; c += 8) {
          m0 = max3(m0, v[c], v[c + 1]);
          m1 = max3(m1, v[c + 2], v[c + 3]);
          m2 = max3(m2, v[c + 4], v[c + 5]);
          m3 = max3(m3, v[c + 6], v[c + 7]);
        }
        float mx = max3(max3(m0, v[60], v[61]), max3(m1, v[62], v[63]), fmaxf(m2, m3));
        const int buf = (ns & 1) * 512;
        mx_own[buf] = mx;
        pair_bar(bar_id);                           // (both halves of S are in registers, too)
        mx = fmaxf(mx, mx_other[buf]);
        ++ns;
        const float m = mx == -INFINITY ? -INFINITY : mx * a.sl2;
        const bool raise = m > ref + kWnSlack || (ref == -INFINITY && m != -INFINITY);
        // (tensor-memory accesses are whole-warp: the other lanes rescale by 1)
        const bool resc = raise && ref != -INFINITY;
        if (__any_sync(0xffffffffu, resc)) {
          const float f = resc ? ex2(ref - m) : 1.f;
          lsum *= f;
#pragma unroll 1
          for (int c0 = 0; c0 < D / 2; c0 += 16) {
            uint32_t o[16];
            tc::tmem_ld(ot + (uint32_t)c0, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::tmem_st(ot + (uint32_t)c0, o);
          }
          tc::tmem_wait_st();
        }
        if (raise) ref = m;
        const float nref = ref == -INFINITY ? 0.f : -ref;
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
        float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float p0 = ex2(v[c0 + c]), p1 = ex2(v[c0 + c + 1]);
            const float p2 = ex2(v[c0 + c + 2]), p3 = ex2(v[c0 + c + 3]);
            l0 = __fadd2_rn(l0, make_float2(p0, p1));
            l1 = __fadd2_rn(l1, make_float2(p2, p3));
            const __nv_bfloat162 h0 = __floats2bfloat162_rn(p0, p1), h1 = __floats2bfloat162_rn(p2, p3);
            pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h0);
            pk[c / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
          }
          tc::tmem_st(pt + (uint32_t)(c0 / 2), pk);
        }
        lsum += (l0.x + l0.y) + (l1.x + l1.y);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&pfull[x]);
        __syncwarp();
      }
      const int buf = (ns & 1) * 512;               // (the maxima's next buffer)
      mx_own[buf] = lsum;
      pair_bar(bar_id);
      lsum += mx_other[buf];
      pair_bar(bar_id);                             // the buffer is read
      wait(&ofull[x], no++);
      const float inv = 1.f / lsum;
      const size_t row = ((size_t)(it.unit / a.Hk) * a.Hq + (size_t)(it.unit % a.Hk) * a.g + hh) * a.n +
                         min(pos, a.n - 1);
      __nv_bfloat16* dst = a.x_out + row * D + half * (D / 2);
      float bad = 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < D / 2; c0 += 32) {
        float o[32];
        tc::tmem_ld32(ot + (uint32_t)c0, o);
        if (pos < a.n && ok) {
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float o0 = o[c + 2 * e] * inv, o1 = o[c + 2 * e + 1] * inv;
              bad += (o0 - o0) + (o1 - o1);         // NaN where one is not finite
              const __nv_bfloat162 h = __floats2bfloat162_rn(o0, o1);
              w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(dst + c0 + c) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
      }
      again = again || bad != 0.f;
      tc::fence_before_sync();   // O is read before this group's next P is published
    }
    // (the two warps of a row meet: what one has written the other reads)
    again = __any_sync(0xffffffffu, again);
    mx_own[0] = again ? 1.f : 0.f;
    __threadfence();
    pair_bar(bar_id);
    again = again || *mx_other != 0.f;
    if (again && ok && half == 0) {
      for (long long i = blockIdx.x; i < a.items; i += gridDim.x) {
        const Item it = item_of(i, a);
        const int pos = it.p0 + dp;
        bool mine = false;
        if (pos < a.n) {
          const size_t row = ((size_t)(it.unit / a.Hk) * a.Hq + (size_t)(it.unit % a.Hk) * a.g + hh) * a.n + pos;
          const uint4* w = reinterpret_cast<const uint4*>(a.x_out + row * D);
          for (int c = 0; c < D / 8; ++c) {
            const uint4 u = __ldcg(w + c);
            for (uint32_t z : {u.x, u.y, u.z, u.w})
              mine = mine || (z & 0x7f80u) == 0x7f80u || (z & 0x7f800000u) == 0x7f800000u;
          }
        }
        for (unsigned rows = __ballot_sync(0xffffffffu, mine); rows; rows &= rows - 1) {
          const int rr = quarter * 32 + __ffs(rows) - 1;
          row_again<D>(a, it.unit, rr / a.P, it.p0 + x * a.P + rr % a.P);
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 17) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, kWnTmemCols);
  }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// bf16 map over [units][n][d]: boxes of 64 elements x box_rows positions, 128-byte swizzle, rows
// outside [0, n) read as 0.
cudaError_t make_map(CUtensorMap* m, const void* base, long long units, int n, int d, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
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
  if (e == cudaSuccess) e = make_map(&mk, a.k, units, a.n, D, 128);
  if (e == cudaSuccess) e = make_map(&mv, a.v, units, a.n, D, 128);
  if (e == cudaSuccess) e = ensure_smem(reinterpret_cast<const void*>(window_attn_kernel<D>), C::total);
  if (e != cudaSuccess) return e;
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
  a.blocks = (a.n + 2 * a.P - 1) / (2 * a.P);
  a.items = (long long)d.batch * a.Hk * a.blocks;
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
