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
// two products per channel whatever g is, from 4 d bytes per group (1/5 of a 4-bit
// group at d = 128, 1/3 of a 2-bit one).
//
// The selection has to be the same on every machine and in every order of summation, so
// the sums carry a 32-bit error term (double-float): D and P as the sum of two floats,
// each product exact as a product and its rounding error, sums by the two-sum of
// T. J. Dekker and D. E. Knuth. What is left is about 2^-45 of the largest term, below any
// gap between scores that are not equal.
#include "decode_device.cuh"

namespace kvc {
namespace {

constexpr int kScoreThreads = 128;     // four warps of four groups each
constexpr int kScoreGroups = 64;       // groups of one CTA
constexpr int kTopkThreads = 256;

struct SelLayer {
  long long packed_off;   // byte offset of the layer in the packed store
  long long key_off;      // element offset of the layer in the score keys
  int n_groups;
  int cap_groups;
  int bits;
};

struct SelParams {
  SelLayer L[KVC_MAX_LAUNCH_LAYERS];
  const uint8_t* packed;
  const __nv_bfloat16* q;        // [layers][units][g][d]
  unsigned long long* keys;      // order-preserving score keys [layer][unit][n_groups]
  int32_t* out;                  // [layers][units][n_select]
  int units;
  int g;
  int n_select;
  int blocks;                    // CTAs per unit of the scoring launch
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

// Order-preserving integer of a score; a score that is not finite gets 0, below all others.
__device__ __forceinline__ unsigned long long score_key(double v) {
  const long long b = __double_as_longlong(v);
  if ((b & 0x7ff0000000000000ll) == 0x7ff0000000000000ll) return 0ull;
  if (v == 0.0) return 0x8000000000000000ull;   // -0 and +0 are equal
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

// One CTA: kScoreGroups groups of one (layer, unit). Eight lanes share a group: lane i of
// the eight holds channel positions 8 i .. 8 i + 7 of each 64 (the key scales' stored
// order) and their query terms in registers.
template <int D>
__global__ void __launch_bounds__(kScoreThreads)
score_groups_kernel(const __grid_constant__ SelParams P) {
  constexpr int NB = D / 64;
  __shared__ float sq[D][4];
  __shared__ int s_exp;
  const SelLayer& L = P.L[blockIdx.y];
  const int unit = blockIdx.x / P.blocks, blk = blockIdx.x % P.blocks;
  if (threadIdx.x == 0) s_exp = 0;
  __syncthreads();
  pdl_wait();
  pdl_release();
  if (blk * kScoreGroups >= L.n_groups || L.n_groups <= P.n_select) return;
  // query terms per stored position, scaled by a power of two so that the largest
  // magnitude is below 2 (no product can then overflow)
  const float m = (float)((1 << L.bits) - 1);
  double dsum = 0.0, psum = 0.0;
  if (threadIdx.x < D) {
    const __nv_bfloat16* q = P.q + ((size_t)blockIdx.y * P.units + unit) * P.g * D + threadIdx.x;
    for (int h = 0; h < P.g; ++h) {
      const double x = (double)__bfloat162float(q[(size_t)h * D]);
      dsum += x;
      psum += x > 0.0 ? x : 0.0;
    }
    psum = isfinite(psum) ? psum * m : psum;
    const int e = (int)((__double_as_longlong(fmax(fabs(dsum), psum)) >> 52) & 0x7ff);
    atomicMax(&s_exp, e);   // 0x7ff: not finite
  }
  __syncthreads();
  if (threadIdx.x < D) {
    const int e = s_exp;
    const double f = e > 0 && e < 0x7ff ? __longlong_as_double((long long)(2046 - e) << 52) : 1.0;
    dsum *= f;
    psum *= f;
    float* t = sq[kperm(threadIdx.x, D)];
    t[0] = (float)dsum;
    t[1] = (float)(dsum - (double)t[0]);
    t[2] = (float)psum;
    t[3] = (float)(psum - (double)t[2]);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, li = lane & 7, sub = lane >> 3, warp = threadIdx.x >> 5;
  float4 qt[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int c = 0; c < 8; ++c)
      qt[b][c] = *reinterpret_cast<const float4*>(sq[b * 64 + li * 8 + c]);
  const int bb = block_bytes(D, L.bits), so = off_kscale(D, L.bits);
  const uint8_t* base = P.packed + L.packed_off + (size_t)unit * L.cap_groups * bb + so;
  unsigned long long* keys = P.keys + L.key_off + (size_t)unit * L.n_groups;
  const int g_end = min(L.n_groups, (blk + 1) * kScoreGroups);
  for (int g0 = blk * kScoreGroups + warp * 4; g0 < g_end; g0 += kScoreThreads / 8) {
    const int grp = g0 + sub;
    float s = 0.f, e = 0.f;
    if (grp < g_end) {
      const uint8_t* p = base + (size_t)grp * bb + li * 16;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 sv = *reinterpret_cast<const uint4*>(p + b * 128);
        const uint4 zv = *reinterpret_cast<const uint4*>(p + 2 * D + b * 128);
        const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w}, zw[4] = {zv.x, zv.y, zv.z, zv.w};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const __half2 s2 = u2h(sw[c >> 1]), z2 = u2h(zw[c >> 1]);
          const float S = (c & 1) ? __high2float(s2) : __low2float(s2);
          const float Z = (c & 1) ? __high2float(z2) : __low2float(z2);
          acc_prod(s, e, Z, qt[b][c].x, qt[b][c].y);
          acc_prod(s, e, S, qt[b][c].z, qt[b][c].w);
        }
      }
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) {
      const float s1 = __shfl_xor_sync(0xffffffffu, s, o), e1 = __shfl_xor_sync(0xffffffffu, e, o);
      float t;
      two_sum(s, s1, s, t);
      e = __fadd_rn(__fadd_rn(e, e1), t);
    }
    if (grp < g_end && li == 0) keys[grp] = score_key((double)s + (double)e);
  }
}

// The n_select largest keys of one unit (ties to the lower index), ascending: a radix
// select of eight 8-bit digits from the top, then an ordered compaction.
__global__ void __launch_bounds__(kTopkThreads)
select_groups_kernel(const __grid_constant__ SelParams P) {
  __shared__ unsigned hist[256];
  __shared__ unsigned wsum[kTopkThreads / 32], wtie[kTopkThreads / 32];
  __shared__ unsigned long long s_thr;
  __shared__ unsigned s_need;
  pdl_wait();
  pdl_release();
  const SelLayer& L = P.L[blockIdx.y];
  const int unit = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = L.n_groups, k = P.n_select;
  int32_t* out = P.out + ((size_t)blockIdx.y * P.units + unit) * k;
  if (n <= k) {
    for (int i = tid; i < k; i += kTopkThreads) out[i] = i < n ? i : -1;
    return;
  }
  const unsigned long long* keys = P.keys + L.key_off + (size_t)unit * n;
  if (tid == 0) {
    s_thr = 0ull;
    s_need = (unsigned)k;
  }
  // s_thr collects the digits of the k-th largest key; s_need: keys still to be taken
  // among those that share the digits found so far
  for (int shift = 56; shift >= 0; shift -= 8) {
    hist[tid] = 0u;
    __syncthreads();
    const unsigned long long thr = s_thr;
    const unsigned need = s_need;
    for (int i = tid; i < n; i += kTopkThreads) {
      const unsigned long long x = keys[i];
      if (shift == 56 || (x >> (shift + 8)) == (thr >> (shift + 8)))
        atomicAdd(&hist[(unsigned)(x >> shift) & 255u], 1u);
    }
    __syncthreads();
    // thread t owns digit 255 - t: keys of larger digits come first
    const unsigned c = hist[255 - tid];
    unsigned incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += wsum[w];
    if (incl >= need && incl - c < need) {
      s_thr = thr | (unsigned long long)(255 - tid) << shift;
      s_need = need - (incl - c);
    }
    __syncthreads();
  }
  const unsigned long long thr = s_thr;
  const unsigned ties = s_need;    // of the keys equal to thr, the first `ties` are kept
  unsigned done = 0, tied = 0;     // kept / equal keys before this block of indices
  for (int i0 = 0; i0 < n; i0 += kTopkThreads) {
    const int i = i0 + tid;
    const unsigned long long x = i < n ? keys[i] : 0ull;
    const bool gt = i < n && x > thr, eq = i < n && x == thr;
    const unsigned beq = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) wtie[warp] = __popc(beq);
    __syncthreads();
    unsigned t0 = tied;
    for (int w = 0; w < warp; ++w) t0 += wtie[w];
    const bool keep = gt || (eq && t0 + __popc(beq & ((1u << lane) - 1u)) < ties);
    const unsigned bk = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) wsum[warp] = __popc(bk);
    __syncthreads();
    unsigned p0 = done, all = 0, allt = 0;
    for (int w = 0; w < kTopkThreads / 32; ++w) {
      if (w < warp) p0 += wsum[w];
      all += wsum[w];
      allt += wtie[w];
    }
    if (keep) out[p0 + __popc(bk & ((1u << lane) - 1u))] = i;
    done += all;
    tied += allt;
    __syncthreads();
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
    P.blocks = std::max(1, (most + kScoreGroups - 1) / kScoreGroups);
    cudaError_t e;
    void* args[1] = {&P};
    if (most > 0) {   // some layer has more groups than are asked for
      const void* fn = d.head_dim == 128 ? reinterpret_cast<const void*>(score_groups_kernel<128>)
                                         : reinterpret_cast<const void*>(score_groups_kernel<64>);
      e = launch_pdl(fn, dim3((unsigned)units * P.blocks, cnt), kScoreThreads, args, stream);
      if (e != cudaSuccess) return e;
      count_launches(1);
    }
    e = launch_pdl(reinterpret_cast<const void*>(select_groups_kernel), dim3(units, cnt),
                   kTopkThreads, args, stream);
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
      if (L.wchunks + L.pchunks == 0) {   // nothing stored: the output is zero
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
