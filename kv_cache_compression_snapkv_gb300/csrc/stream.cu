// stream.cu -- decode attention that a long generation bounds: over the first and the last cached
// tokens (kvc_decode_window), and over the whole cache with what attention every 32 tokens receive
// (kvc_decode_weights).
//
// Both are the decode kernel (decode_device.cuh) over a range. A layer's tokens in storage order,
// its packed groups and then its window, are seen before token a and from token b on. Only the
// groups and window chunks that hold a seen token are read; inside the two at the edges the hidden
// tokens' logits become -inf and what they would multiply becomes 0, whatever is stored there.
//
// The split of the work, the copies and the merges are the decode kernel's (decode.cu), the arithmetic of
// packed groups is range_warp's. 4,100 of 131,072 tokens (8 units, 2 bits) 12.5 us, 8,050 of
// 32,768 (160 units, 4 bits) 61 us (3.4 TB/s): what bounds the first is latency (launch 2 us, start
// 1, copy 1.1, a warp's chunk of two groups 4 to 5, the first with a cold instruction cache, merges 3).
// 16-bit caches: 2,004 of 4,096 tokens of 256 units 53 us, all of them with weights 101 us (5.3 TB/s).
//
// Weights. With x_ht the logit of token t for query head h, M_h and L_h the maximum and the sum
// of exp2 over all tokens, a group G receives sum_h sum_{t in G} exp2(x_ht - M_h) / L_h. M and L are
// known only when a unit's last warp has merged its parts, so every chunk leaves its parts, per head
// the sum of its exp2 and the running maximum they were taken against, and
// sum_h s_h exp2(m_h - M_h) / L_h is formed in a fixed order afterwards: 8 bytes per head for 32
// packed or 16 window tokens, a few hundredths of what those are stored in at most. Where a unit has
// few parts its last warp forms the weights, else a second launch does.
#include "decode_device.cuh"

namespace kvc {
namespace {

constexpr int kWeightThreads = 256;
// Slots of a unit that its last warp still forms the weights of: one look at memory, against a launch.
// 16 and 32 slots against the launch: 4 units of 1 head 10.6 and 11.5 us (11.1, 12.0), 8 of 4 heads 10.7 and
// 11.1 (11.1, 11.5), 16 of 8 heads 12.2 and 12.5 (12.9, 13.2), 8 of 8 heads the same either way, 128 of 1
// head 14.3 and 16.6 (14.4, 16.0); 64 slots 12.6, 12.5, 14.9, 20.4 and 21.4 (12.1, 12.3, 13.9, 19.3, 20.9).
constexpr int kWarpSlots = 32;

struct WeightLayer {
  int n_groups;           // packed groups; the window's parts follow, two for 32 tokens
  int parts;              // parts of a unit
  long long part_begin;
};
struct WeightParams {
  WeightLayer L[KVC_MAX_LAUNCH_LAYERS];
  const float2* part;     // as RangeParams
  const float2* stat;
  const float* before;    // [layer][unit][n_slots]
  float* after;
  int n_slots, units;
};

// One thread per slot of 32 tokens.
template <int G>
__global__ void __launch_bounds__(kWeightThreads)
group_weights_kernel(const WeightParams P, unsigned blocks) {
  pdl_wait();
  pdl_release();
  const unsigned ul = blockIdx.x / blocks;   // (layer, unit)
  const int slot = (int)((blockIdx.x - ul * blocks) * kWeightThreads + threadIdx.x);
  if (slot >= P.n_slots) return;
  const WeightLayer& L = P.L[ul / (unsigned)P.units];
  const float2* part = P.part + ((size_t)L.part_begin + (size_t)(ul % (unsigned)P.units) * L.parts) * G;
  const size_t at = (size_t)ul * P.n_slots + slot;
  const float was = P.before[at];
  float2 stat[G];
  load_pairs(stat, P.stat + (size_t)ul * G);
  P.after[at] = was + slot_weight(part, stat, slot, L.n_groups, L.parts);
}

// What of layer ls is seen: the first n_sinks tokens and the last `window`.
RangeLayer range_of(const LayerState& ls, long long n_sinks, long long window, int wchunks) {
  const long long packed = (long long)ls.n_groups * KVC_GROUP, T = packed + ls.win_len;
  const long long a = std::min(n_sinks, T), b = std::max(0LL, T - window);
  RangeLayer r{};
  r.g_first = r.g_count = ls.n_groups;
  r.w_first = wchunks;
  if (a >= b) return r;   // every token (a = b = 0)
  r.a = (int)a;
  r.b = (int)b;
  const int ga = (int)std::min<long long>(ls.n_groups, (a + KVC_GROUP - 1) / KVC_GROUP);
  const int gb = (int)std::min<long long>(ls.n_groups, b / KVC_GROUP);
  if (ga < gb) {
    r.g_first = ga;
    r.g_skip = gb - ga;
    r.g_count = ls.n_groups - r.g_skip;
  }
  const int wa = (int)((std::max(0LL, a - packed) + kSlotsPerWarp - 1) / kSlotsPerWarp);
  const int wb = (int)(std::max(0LL, b - packed) / kSlotsPerWarp);
  if (wa < wb) {
    r.w_first = wa;
    r.w_skip = wb - wa;
  }
  return r;
}

cudaError_t launch_weights(const WeightParams& W, int layers, int g, cudaStream_t stream) {
  const unsigned blocks = ((unsigned)W.n_slots + kWeightThreads - 1) / kWeightThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks * (unsigned)W.units * (unsigned)layers);
  cfg.blockDim = dim3(kWeightThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attr()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = g == 1   ? cudaLaunchKernelEx(&cfg, group_weights_kernel<1>, W, blocks)
                        : g == 2 ? cudaLaunchKernelEx(&cfg, group_weights_kernel<2>, W, blocks)
                        : g == 4 ? cudaLaunchKernelEx(&cfg, group_weights_kernel<4>, W, blocks)
                                 : cudaLaunchKernelEx(&cfg, group_weights_kernel<8>, W, blocks);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

size_t weight_parts(const kvc_cache* c) {
  size_t n = 0;
  for (const LayerState& ls : c->L) n += ls.cap_groups + (size_t)ls.R / kSlotsPerWarp + 1;
  return n * c->dims.batch * c->dims.n_q_heads;
}

cudaError_t launch_decode_range(const kvc_cache* c, int layer_begin, int layer_count,
                                const __nv_bfloat16* q, int n_sinks, int window, int n_slots,
                                const float* before, float* after, float* out,
                                cudaStream_t stream) {
  const kvc_dims& d = c->dims;
  const int units = d.batch * d.n_kv_heads;
  const size_t gq = (size_t)c->g * d.head_dim;
  for (int base = 0; base < layer_count; base += KVC_MAX_LAUNCH_LAYERS) {
    const int cnt = std::min(layer_count - base, KVC_MAX_LAUNCH_LAYERS);
    RangeParams P;
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
    P.groups = nullptr;
    P.n_select = 0;
    P.wide = c->wide;
    P.part = after ? c->part : nullptr;
    P.stat = after ? c->part_stat : nullptr;
    long long total = 0, parts = 0;
    int most = 0;
    bool empty = false;
    int bmask = 0;
    float* ob = out + (size_t)base * units * gq;
    for (int i = 0; i < cnt; ++i) {
      const LayerState& ls = c->L[layer_begin + base + i];
      DecLayer& L = P.L[i];
      RangeLayer& X = P.R[i];
      const int wchunks = (ls.win_len + kSlotsPerWarp - 1) / kSlotsPerWarp;
      X = range_of(ls, n_sinks, window, wchunks);
      X.parts = ls.n_groups + wchunks;
      X.part_begin = parts;
      parts += (long long)units * X.parts;
      most = std::max(most, std::max(X.parts, n_slots));
      empty = empty || X.parts == 0;
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
      L.wchunks = wchunks - X.w_skip;
      L.pchunks = (X.g_count + L.gpc - 1) / L.gpc;
      L.chunk_begin = total;
      total += (long long)units * (L.wchunks + L.pchunks);
      if (L.pchunks > 0) bmask |= ls.bits == 2 ? 1 : 2;
      if (L.wchunks + L.pchunks == 0) {   // a layer that holds no token: the output is zero
        cudaError_t e = cudaMemsetAsync(ob + (size_t)i * units * gq, 0, units * gq * 4, stream);
        if (e != cudaSuccess) return e;
      }
    }
    const bool by_warp = after && !empty && most <= kWarpSlots;
    P.before = by_warp ? before + (size_t)base * units * n_slots : nullptr;
    P.after = by_warp ? after + (size_t)base * units * n_slots : nullptr;
    P.n_slots = n_slots;
    P.total = total;
    if (total > 0) {
      cudaError_t e = launch_bits<kDecRange>(P, c, bmask, q + (size_t)base * units * gq, ob, stream);
      if (e != cudaSuccess) return e;
      count_launches(1);
    }
    if (after && !by_warp) {
      WeightParams W;
      for (int i = 0; i < cnt; ++i)
        W.L[i] = {P.L[i].n_groups, P.R[i].parts, P.R[i].part_begin};
      W.part = P.part;
      W.stat = P.stat;
      W.before = before + (size_t)base * units * n_slots;
      W.after = after + (size_t)base * units * n_slots;
      W.n_slots = n_slots;
      W.units = units;
      cudaError_t e = launch_weights(W, cnt, c->g, stream);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaGetLastError();
}

}  // namespace kvc
