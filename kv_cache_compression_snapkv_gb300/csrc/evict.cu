// evict.cu -- groups of 32 tokens that received the least attention leave a cache: those that stay
// go, in order and with the window, to another (smaller) cache (kvc_evict_groups).
//
// Per (layer, unit): of E groups the n_recent newest stay; of the others the ones of the largest
// weights, ties to the lower index. Weights are compared as 32-bit keys in their order (-0 as 0, a
// NaN below everything). The border is found digit by digit (11, 11 and 10 bits) from counts of the
// digits, which are exact, so the list does not depend on the order of anything.
//
// What bounds it: the copies. 512 of 1,024 groups of 160 units at 4 bits 131 us (841 MB: 6.4 TB/s, 0.95
// of a plain copy's rate), 1,024 of 4,095 groups of 8 units at 2 bits 11.1 us (50 MB; where there are only
// the 1,024 5.7: the choice is 5.4), 8 of 16 groups of 4 units 2.7 us (launch and latency); 64 of 128 groups
// of 256 16-bit units 91 us (537 MB, 5.9 TB/s).
//
// One launch. A unit's blocks are shared out over several CTAs, each of which finds the border by
// itself (it reads 4 bytes of weight per group of 1,536 to 5,120 bytes), keeps the ids of its own part
// of the list and copies that part: nothing waits on another CTA.
#include <algorithm>

#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvItems = 8;                          // weights of a thread in one tile
constexpr int kEvTile = kEvThreads * kEvItems;
constexpr int kEvMost = 2048;                        // list entries of a CTA, at most
static_assert(kEvMost == 4 * kEvThreads && kEvMost == 1 << 11, "a digit's counts, four per thread");
// Groups ranked by comparison with all others, at most (half of 64, 128 and 256 groups of 8 units stay:
// 3.2, 3.6 and 5.2 us, by digits 5.7, 5.8 and 5.8; 160 units: 6.8, 11.3 and 31.9, by digits 9.6, 13.8 and 34.0).
constexpr int kEvFew = 256;
static_assert(kEvFew <= kEvThreads && kEvThreads <= 1024, "a group per thread, a count per lane");

struct EvLayer {
  long long src_off, dst_off;   // bytes of the layer inside the packed stores (16 bits: unused)
  long long src_win, dst_win;   // elements of the layer inside the rings
  int src_cap, dst_cap;         // packed capacity of a unit in groups
  int src_R, dst_R;
  int E;                        // groups that may leave
  int m;                        // groups that stay
  int recent;                   // the newest of them, in any case
  int slots;                    // weights of a unit that move: E and the window's
  int win_first, win_blocks;    // first ring block of 32 slots that stays as it is, and their number
  int ring_blocks;              // ring blocks in storage order start here (win_start / 32)
  int bits;
};
struct EvParams {
  EvLayer L[KVC_MAX_LAUNCH_LAYERS];
  const uint8_t* src;
  uint8_t* dst;
  const __nv_bfloat16 *src_k, *src_v;
  __nv_bfloat16 *dst_k, *dst_v;
  const unsigned* src_wide;     // marks [layer][unit][kMarkWords]
  unsigned* dst_wide;
  unsigned* dst_seen;
  const float* weights;         // [layer][unit][n_slots]
  float* stay;
  int32_t* groups;              // [layer][unit][n_keep]
  int n_slots, n_keep, units, layer_begin;
  int per;                      // list entries of a CTA
  int ctas;                     // CTAs of a unit
};

// A weight's place in the order of weights.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Copy of VECS 16-byte words per lane by one warp, at most ten in flight.
template <int VECS>
__device__ __forceinline__ void warp_copy(uint8_t* dst, const uint8_t* src) {
  if constexpr (VECS > 10) {
    warp_copy<VECS / 2>(dst, src);
    warp_copy<VECS / 2>(dst + VECS / 2 * 512, src + VECS / 2 * 512);
    return;
  }
  const int lane = threadIdx.x & 31;
  uint4 v[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(src) + i * 32 + lane);
#pragma unroll
  for (int i = 0; i < VECS; ++i) reinterpret_cast<uint4*>(dst)[i * 32 + lane] = v[i];
}

template <int D>
__global__ void __launch_bounds__(kEvThreads, 2)
evict_kernel(const EvParams P) {
  __shared__ int sh_warp[kEvWarps];
  __shared__ __align__(16) uint32_t sh_tab[kEvItems * kEvWarps];   // a tile's counts in index order
  __shared__ int sh_tot[2];
  __shared__ __align__(16) uint32_t sh_few[kEvFew];
  __shared__ __align__(16) int ids[kEvMost];         // before the list is there: counts of digits
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // CTAs: (layer, unit, part)
  const unsigned ulu = blockIdx.x / (unsigned)P.ctas, layer = ulu / (unsigned)P.units;
  const int part = (int)(blockIdx.x - ulu * (unsigned)P.ctas), unit = (int)(ulu - layer * (unsigned)P.units);
  const EvLayer& L = P.L[layer];
  const int E1 = L.E - L.recent, need = L.m - L.recent;
  // this CTA's entries of the list: the groups that stay, then the window's blocks
  const int all = L.m + L.win_blocks;
  const int k0 = part * P.per, k1 = min(all, k0 + P.per);
  const bool first = part == 0;
  if (k0 >= all && !first) return;
  pdl_wait();
  pdl_release();
  const size_t ul = ulu;
  const float* w = P.weights + ul * P.n_slots;
  float* stay = P.stay + ul * P.n_slots;
  int32_t* out = P.groups + ul * P.n_keep;

  // Item i of a thread is weight tile + i * kEvThreads + tid: index order is item, warp, lane.
  const bool held = E1 <= kEvTile;
  uint32_t key[kEvItems];
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < kEvItems; ++i) {
      const int at = tile + i * kEvThreads + tid;
      key[i] = at < E1 ? weight_key(__ldg(w + at)) : 0u;
    }
  };
  const bool choose = need > 0 && need < E1;
  if (choose && E1 <= kEvFew) {
    // Few: every group's rank by comparison with all the others, then its place among those that stay.
    const uint32_t mine = tid < E1 ? weight_key(__ldg(w + tid)) : 0u;
    if (tid < kEvFew) sh_few[tid] = mine;
    __syncthreads();
    int rank = 0;
    if (warp * 32 < E1)
      for (int j = 0; j < E1; j += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(sh_few + j);   // (past the last: 0, after all)
        rank += (o.x > mine || (o.x == mine && j < tid)) + (o.y > mine || (o.y == mine && j + 1 < tid)) +
                (o.z > mine || (o.z == mine && j + 2 < tid)) + (o.w > mine || (o.w == mine && j + 3 < tid));
      }
    const unsigned in = __ballot_sync(0xffffffffu, tid < E1 && rank < need);
    if (lane == 0) sh_tab[warp] = __popc(in);
    __syncthreads();
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? (int)sh_tab[lane] : 0);
    const int at = before + __popc(in & ((1u << lane) - 1u));
    if ((in >> lane & 1u) && at >= k0 && at < k1) ids[at - k0] = tid;
  } else if (choose) {
    // the border: the largest key that at least `need` of the first E1 groups reach; ties: how many
    // of those at it stay
    uint32_t border = 0u;
    int ties = need;
    fetch(0);
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
      reinterpret_cast<int4*>(ids)[tid] = make_int4(0, 0, 0, 0);
      __syncthreads();
      for (int tile = 0; tile < E1; tile += kEvTile) {
        if (!held) fetch(tile);
#pragma unroll
        for (int i = 0; i < kEvItems; ++i)
          if (tile + i * kEvThreads + tid < E1 && (pass == 0 || key[i] >> (shift + bits) == border))
            atomicAdd(&ids[key[i] >> shift & ((1u << bits) - 1u)], 1);
      }
      __syncthreads();
      const int4 h = reinterpret_cast<const int4*>(ids)[tid];   // digits 4 tid .. 4 tid + 3
      const int sum = h.x + h.y + h.z + h.w;
      int x = sum;                                  // of this thread's digits and the warp's later ones
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, x, o);
        if (lane + o < 32) x += y;
      }
      if (lane == 0) sh_warp[warp] = x;
      __syncthreads();
      int above = __reduce_add_sync(0xffffffffu, lane > warp && lane < kEvWarps ? sh_warp[lane] : 0) + x - sum;
      if (above < ties && above + sum >= ties) {    // (one thread's)
        const int c[4] = {h.x, h.y, h.z, h.w};
        int q = 3;
        for (; above + c[q] < ties; --q) above += c[q];
        sh_tot[0] = 4 * tid + q;
        sh_tot[1] = ties - above;
      }
      __syncthreads();
      border = border << bits | (uint32_t)sh_tot[0];
      ties = sh_tot[1];
    }
    // The list in order, of which this CTA keeps its part: rank = groups past the border before this
    // one, and of those at it as many as stay.
    int past = 0, at_border = 0;       // of the tiles before
    for (int tile = 0; tile < E1; tile += kEvTile) {
      if (!held) fetch(tile);
      unsigned gt[kEvItems], eq[kEvItems];
      __syncthreads();                 // (the table and the totals of the tile before are read)
#pragma unroll
      for (int i = 0; i < kEvItems; ++i) {
        const bool in = tile + i * kEvThreads + tid < E1;
        gt[i] = __ballot_sync(0xffffffffu, in && key[i] > border);
        eq[i] = __ballot_sync(0xffffffffu, in && key[i] == border);
        if (lane == 0) sh_tab[i * kEvWarps + warp] = __popc(gt[i]) | __popc(eq[i]) << 16;
      }
      __syncthreads();
      if (warp == 0) {                 // exclusive prefixes of the table, and its total
        uint32_t v[kEvItems * kEvWarps / 32], sum = 0u;
#pragma unroll
        for (int j = 0; j < kEvItems * kEvWarps / 32; ++j) {
          v[j] = sh_tab[lane * (kEvItems * kEvWarps / 32) + j];
          sum += v[j];
        }
        uint32_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (lane == 31) {
          sh_tot[0] = (int)(x & 0xffff);
          sh_tot[1] = (int)(x >> 16);
        }
        x -= sum;
#pragma unroll
        for (int j = 0; j < kEvItems * kEvWarps / 32; ++j) {
          sh_tab[lane * (kEvItems * kEvWarps / 32) + j] = x;
          x += v[j];
        }
      }
      __syncthreads();
      const unsigned below = (1u << lane) - 1u;
#pragma unroll
      for (int i = 0; i < kEvItems; ++i) {
        const uint32_t t = sh_tab[i * kEvWarps + warp];
        const int g = past + (int)(t & 0xffff) + __popc(gt[i] & below);
        const int e = at_border + (int)(t >> 16) + __popc(eq[i] & below);
        const int rank = g + min(e, ties);
        if ((gt[i] >> lane & 1u) || ((eq[i] >> lane & 1u) && e < ties))
          if (rank >= k0 && rank < k1) ids[rank - k0] = tile + i * kEvThreads + tid;
      }
      past += sh_tot[0];
      at_border += sh_tot[1];
    }
  } else {
    for (int k = k0 + tid; k < min(k1, need); k += kEvThreads) ids[k - k0] = k;   // (all, or none)
  }
  for (int k = max(k0, need) + tid; k < min(k1, L.m); k += kEvThreads) ids[k - k0] = E1 + k - need;
  __syncthreads();

  // the list and the weights that stay
  for (int k = k0 + tid; k < min(k1, L.m); k += kEvThreads) {
    out[k] = ids[k - k0];
    stay[k] = w[ids[k - k0]];
  }
  if (first) {
    for (int k = L.m + tid; k < P.n_keep; k += kEvThreads) out[k] = -1;
    for (int k = L.m + tid; k < P.n_slots; k += kEvThreads)
      stay[k] = k - L.m < L.slots - L.E ? w[k - L.m + L.E] : 0.f;
    if (tid == 0) {
      const size_t at = ((size_t)(P.layer_begin + layer) * P.units + unit) * kMarkWords;
      const unsigned mark = P.src_wide[at];
      P.dst_wide[at] = mark;
      if (mark) *reinterpret_cast<volatile unsigned*>(P.dst_seen) = 1u;
    }
  }
  // the blocks: one per warp at a time
  const int bb = L.bits == 16 ? 0 : block_bytes(D, L.bits);
  constexpr int RB = KVC_GROUP * D * 2;   // 32 slots of a ring
  const size_t sring = (size_t)L.src_win + (size_t)unit * L.src_R * D;
  const size_t dring = (size_t)L.dst_win + (size_t)unit * L.dst_R * D;
  for (int k = k0 + warp; k < k1; k += kEvWarps) {
    if (k < L.m && L.bits != 16) {
      const uint8_t* s = P.src + L.src_off + ((size_t)unit * L.src_cap + ids[k - k0]) * bb;
      uint8_t* t = P.dst + L.dst_off + ((size_t)unit * L.dst_cap + k) * bb;
      if (L.bits == 2) warp_copy<8 * D * 3 / 512>(t, s);
      else warp_copy<8 * D * 5 / 512>(t, s);
    } else {
      // ring blocks in storage order; 32 slots keep their places inside the swizzle
      const int from = k < L.m ? ids[k - k0] : L.win_first + k - L.m;
      const int to = L.bits == 16 ? k : k - L.m;
      const size_t so = sring + (size_t)((L.ring_blocks + from) % (L.src_R / KVC_GROUP)) * KVC_GROUP * D;
      const size_t to_ = dring + (size_t)to * KVC_GROUP * D;
      warp_copy<RB / 512>(reinterpret_cast<uint8_t*>(P.dst_k + to_), reinterpret_cast<const uint8_t*>(P.src_k + so));
      warp_copy<RB / 512>(reinterpret_cast<uint8_t*>(P.dst_v + to_), reinterpret_cast<const uint8_t*>(P.src_v + so));
    }
  }
}

}  // namespace

cudaError_t launch_evict(const kvc_cache* src, const kvc_cache* dst, int layer_begin,
                         int layer_count, int n_keep, int n_recent, int n_slots,
                         const float* weights, float* stay, int32_t* groups, cudaStream_t stream) {
  const kvc_dims& d = src->dims;
  const int units = d.batch * d.n_kv_heads;
  for (int base = 0; base < layer_count; base += KVC_MAX_LAUNCH_LAYERS) {
    const int cnt = std::min(layer_count - base, KVC_MAX_LAUNCH_LAYERS);
    EvParams P;
    P.src = src->packed;
    P.dst = dst->packed;
    P.src_k = src->win_k;
    P.src_v = src->win_v;
    P.dst_k = dst->win_k;
    P.dst_v = dst->win_v;
    P.src_wide = src->wide;
    P.dst_wide = dst->wide;
    P.dst_seen = dst->wide_seen;
    P.weights = weights + (size_t)base * units * n_slots;
    P.stay = stay + (size_t)base * units * n_slots;
    P.groups = groups + (size_t)base * units * n_keep;
    P.n_slots = n_slots;
    P.n_keep = n_keep;
    P.units = units;
    P.layer_begin = layer_begin + base;
    int most = 1;
    for (int i = 0; i < cnt; ++i) {
      const LayerState& a = src->L[layer_begin + base + i];
      const LayerState& b = dst->L[layer_begin + base + i];
      EvLayer& L = P.L[i];
      L.src_off = (long long)a.packed_off;
      L.dst_off = (long long)b.packed_off;
      L.src_win = (long long)a.win_off;
      L.dst_win = (long long)b.win_off;
      L.src_cap = a.cap_groups;
      L.dst_cap = b.cap_groups;
      L.src_R = a.R;
      L.dst_R = b.R;
      L.bits = a.bits;
      L.E = evictable_groups(a);
      L.m = std::min(n_keep, L.E);
      L.recent = std::min(n_recent, L.E);
      const int wb = (a.win_len + KVC_GROUP - 1) / KVC_GROUP;
      L.slots = a.n_groups + wb;
      L.win_first = a.bits == 16 ? L.E : 0;
      L.win_blocks = wb - L.win_first;
      L.ring_blocks = a.win_start / KVC_GROUP;
      most = std::max(most, L.m + L.win_blocks);
    }
    // A CTA's part of a unit's list: what makes one wave of two CTAs an SM, or, where that is more
    // than 64 blocks, of eight (each CTA chooses anew: 8 units, 1,024 of 4,064 groups 11.4 us in one
    // wave of 28 blocks, 17.6 us in two; 160 units, 512 of 1,024 groups 154 us with one CTA a unit, 131
    // with seven).
    auto part_of = [&](long long per_sm) {
      const long long ctas = std::max<long long>(1, per_sm * src->n_sm / ((long long)units * cnt));
      return std::min<long long>(kEvMost, std::max<long long>(kEvWarps, (most + ctas - 1) / ctas));
    };
    P.per = (int)(part_of(2) <= 64 ? part_of(2) : part_of(8));
    P.ctas = (most + P.per - 1) / P.per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)P.ctas * (unsigned)units * (unsigned)cnt);
    cfg.blockDim = dim3(kEvThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1] = {pdl_attr()};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = d.head_dim == 128 ? cudaLaunchKernelEx(&cfg, evict_kernel<128>, P)
                                            : cudaLaunchKernelEx(&cfg, evict_kernel<64>, P);
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace kvc
