// decode.cu -- decode attention over the packed cache plus the bf16 window,
// optionally fused with the append of the step's new token.
//
// MiniKV: Pushing the Limits of LLM Inference via 2-Bit Layer-Discriminative KV
// Cache, §2 eq. (1) and Algorithm 1 (decoding): append the new key/value to the
// 16-bit buffer, quantize when it fills, then one softmax over the dequantized
// packed keys and the buffer's keys; output = A_quant . dequant(Q_V) +
// A_unquant . R_V. Blog "KV Cache Compression: Eviction and Quantization",
// "Measured on a real model": exact recent window, rounded rest, one softmax.
//
// Work decomposition (one launch for a range of layers): a unit = (layer,
//   sequence b, kv head h); its work is cut into chunks of 16 window slots or
//   GPC packed group blocks (GPC = groups that fill one window chunk's bytes: 2 at
//   2 bits, 1 at 4 bits). The chunks of every unit of the launch are laid end to
//   end (layer by layer, unit by unit) and the list is cut into equal contiguous
//   ranges, one per warp of the grid (one CTA per SM): a split-K over the whole
//   launch, so a large unit is spread over many warps of many SMs and small units
//   share a warp, and every warp gets the same number of chunks. Each warp
//   double-buffers its chunks in shared memory with bulk asynchronous copies
//   (cp.async.bulk on per-slot mbarriers, bounded waits); the copy of a unit's
//   first chunk also brings the unit's g queries. A warp keeps an online softmax
//   of the g query heads over the part of a unit it holds. A unit held whole by
//   one warp is normalised and written by it; otherwise each holder writes its
//   partial state (m, l, o) to a workspace in global memory and takes a ticket
//   from the unit's arrival counter, and the holder that arrives last merges
//   the partial states with a log-sum-exp combine in a fixed order (the result
//   does not depend on arrival order), writes the fp32 output and resets the
//   counter. Nothing waits on another warp or CTA.
//   The new token of a fused step is stored into the ring by the warp whose
//   window chunk holds its slot (which also patches its staged copy). A step in
//   which some layer's window reaches R runs the append kernel first (it stores
//   the new tokens and quantizes the oldest group of each full window) and then
//   this kernel over the updated cache. Layers of one launch may differ in
//   precision (2 or 4 bits, or 16: window only) and in ring length.
//
// Arithmetic. Per 32-token group block the key logits are
//     q . k_t = sum_c (q_c S_c) code_tc + sum_c q_c Z_c
// and the value output is
//     o_c = sum_t (p_t S_t,gc) code_tc + sum_t p_t Z_t,gc.
// Both code sums run on the tensor cores (mma m16n8k16, fp16 operands, fp32
// accumulate): codes are unpacked in registers to exact fp16 integers, and the
// fp16 operand products (q_c S_c, p_t S_t) are split into hi + lo fp16 parts in
// adjacent columns of the 8-column operand (column 2h hi, 2h + 1 lo for head h),
// so the rounding of the operand does not limit accuracy. The key zero-point sums
// are one small extra product per chunk (q against the chunk's groups' key zeros).
// The value zero-point sums are products of the zero-points (every row of a channel
// group carrying Z_t) against hi/lo(p), accumulated into the same registers as the
// code sums of the same 16 tokens: the two terms nearly cancel (the code term is
// about +range/2 times the weight, the zero term about -range/2 times it), so
// keeping them apart would leave a small result as the difference of two large
// fp32 sums over all tokens. The window runs the same flow on bf16 operands.
#include "decode_device.cuh"

namespace kvc {
namespace {

// Shared host path: a non-null k_new appends the step's token first. Without a
// group flush in the step the decode launch stores the new token itself; when
// some layer's window reaches R, the append kernel (which also quantizes the
// flushed groups) runs first and the decode launch reads the updated cache.
cudaError_t launch_common(const kvc_cache* c, int layer_begin, int layer_count,
                          const __nv_bfloat16* q, const __nv_bfloat16* k_new,
                          const __nv_bfloat16* v_new, const int* flush_flags, float* out,
                          cudaStream_t stream) {
  const kvc_dims& d = c->dims;
  const int units = d.batch * d.n_kv_heads;
  const int D = d.head_dim;
  bool appending = k_new != nullptr;
  bool any_flush = false;
  if (appending)
    for (int i = 0; i < layer_count; ++i) any_flush = any_flush || flush_flags[i] != 0;
  if (any_flush) {
    cudaError_t e = launch_append(c, layer_begin, layer_count, k_new, v_new, flush_flags, stream);
    if (e != cudaSuccess) return e;
  }
  for (int base = 0; base < layer_count; base += KVC_MAX_LAUNCH_LAYERS) {
    const int cnt = layer_count - base < KVC_MAX_LAUNCH_LAYERS ? layer_count - base
                                                               : KVC_MAX_LAUNCH_LAYERS;
    DecParams P;
    P.n_layers = cnt;
    P.layer_begin = layer_begin + base;
    P.units = units;
    P.sl2 = 1.4426950408889634f / sqrtf((float)D);
    P.err = c->err;
    P.ws = c->dec_ws;
    P.cnt = c->dec_cnt;
    P.groups = nullptr;
    P.wide = nullptr;
    P.n_select = 0;
    P.wait_limit = c->wait_limit_set ? c->wait_limit : kWaitLimit;
    const bool fused = appending && !any_flush;
    P.k_new = fused ? k_new + (size_t)base * units * D : nullptr;
    P.v_new = fused ? v_new + (size_t)base * units * D : nullptr;
    long long total = 0;
    int bmask = 0;
    const size_t gq = (size_t)c->g * D;
    float* ob = out + (size_t)base * units * gq;
    for (int i = 0; i < cnt; ++i) {
      const LayerState& ls = c->L[layer_begin + base + i];
      DecLayer& L = P.L[i];
      const int R = ls.R;
      L.cap_groups = ls.cap_groups;
      L.packed_off = (long long)ls.packed_off;
      L.win_off = (long long)ls.win_off;
      L.R = R;
      L.bits = ls.bits;
      L.gpc = dec_groups_per_chunk(D, ls.bits == 16 ? 2 : ls.bits);
      if (appending) {
        const bool flush = flush_flags[base + i] != 0;
        L.new_slot = fused ? (ls.win_start + ls.win_len) % R : -1;
        L.n_groups = ls.n_groups + (flush ? 1 : 0);
        L.win_start = flush ? (ls.win_start + KVC_GROUP) % R : ls.win_start;
        L.win_len = ls.win_len + 1 - (flush ? KVC_GROUP : 0);
      } else {
        L.new_slot = -1;
        L.n_groups = ls.n_groups;
        L.win_start = ls.win_start;
        L.win_len = ls.win_len;
      }
      L.wchunks = (L.win_len + kSlotsPerWarp - 1) / kSlotsPerWarp;
      L.pchunks = (L.n_groups + L.gpc - 1) / L.gpc;
      L.chunk_begin = total;
      total += (long long)units * (L.wchunks + L.pchunks);
      if (L.pchunks > 0) bmask |= ls.bits == 2 ? 1 : (ls.bits == 4 ? 2 : 0);
      if (L.wchunks + L.pchunks == 0) {   // nothing stored: the output is zero
        cudaError_t e = cudaMemsetAsync(ob + (size_t)i * units * gq, 0, units * gq * 4, stream);
        if (e != cudaSuccess) return e;
      }
    }
    P.total = total;
    if (total == 0) continue;
    const __nv_bfloat16* qb = q + (size_t)base * units * gq;
    cudaError_t e = launch_bits<false>(P, c, bmask, qb, ob, stream);
    if (e != cudaSuccess) return e;
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_decode(const kvc_cache* c, int layer_begin, int layer_count,
                          const __nv_bfloat16* q, float* out, cudaStream_t stream) {
  return launch_common(c, layer_begin, layer_count, q, nullptr, nullptr, nullptr, out, stream);
}

cudaError_t launch_decode_step(const kvc_cache* c, int layer_begin, int layer_count,
                               const __nv_bfloat16* q, const __nv_bfloat16* k_new,
                               const __nv_bfloat16* v_new, const int* flush_flags, float* out,
                               cudaStream_t stream) {
  return launch_common(c, layer_begin, layer_count, q, k_new, v_new, flush_flags, out, stream);
}

size_t decode_workspace_floats(int n_sm, int g, int D) {
  return (size_t)2 * n_sm * 16 * dep_floats(D, g);
}

}  // namespace kvc
