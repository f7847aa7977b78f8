// tree.cu -- attention of a tree of drafted tokens over the compressed cache
// (kvc_tree_attn): each node's query attends to every cached token (packed groups and
// window), to the drafted tokens on its path to the root, and to itself, in one softmax.
//
// One warp per query row (node and query head): the lanes take 32 tokens at a time for
// the logits and the channels for the output, with a running maximum and sum.
#include "decode_device.cuh"

namespace kvc {
namespace {

constexpr int kTreeWarps = 4;

struct TreeLayer {
  long long packed_off, win_off;
  int n_groups, cap_groups, bits, win_start, win_len, R;
};
struct TreeParams {
  TreeLayer L[KVC_MAX_LAUNCH_LAYERS];
  const uint8_t* packed;
  const __nv_bfloat16* win_k;
  const __nv_bfloat16* win_v;
  const int32_t* parents;         // [B][T]
  const __nv_bfloat16* q;         // [layers][B][Hq][T][d]
  const __nv_bfloat16* k_draft;   // [layers][B][H][T][d]
  const __nv_bfloat16* v_draft;
  __nv_bfloat16* out;             // as q
  int units, H, g, T;
  float sl2;
};

template <int D>
__global__ void __launch_bounds__(kTreeWarps * 32)
tree_simple_kernel(const __grid_constant__ TreeParams P) {
  constexpr int C = D / 32;
  __shared__ float sq[kTreeWarps][D];
  const TreeLayer& L = P.L[blockIdx.z];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x, row = blockIdx.y * kTreeWarps + warp, T = P.T;
  if (row >= P.g * T) return;
  const int node = row % T, b = unit / P.H;
  const size_t ul = (size_t)blockIdx.z * P.units + unit;
  const __nv_bfloat16* q = P.q + (ul * P.g * T + row) * D;
  __nv_bfloat16* out = P.out + (ul * P.g * T + row) * D;
  // the path to the root; a node whose path does not end at -1 is padding
  unsigned long long path = 0ull;
  int p = node;
  while (p >= 0) {
    path |= 1ull << p;
    const int up = P.parents[(size_t)b * T + p];
    p = up >= p ? -2 : up;
  }
  if (p != -1) {
    for (int c = lane; c < D; c += 32) out[c] = __float2bfloat16(0.f);
    return;
  }
  for (int c = lane; c < D; c += 32) sq[warp][c] = __bfloat162float(q[c]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.f;
  // 32 tokens: key(c) of this lane's token, value(t, c) of token t
  auto block = [&](bool live, auto key, auto value) {
    float x = 0.f;
    if (live)
      for (int c = 0; c < D; ++c) x = fmaf(sq[warp][c], key(c), x);
    x = live ? x * P.sl2 : -INFINITY;
    float mx = x;
    for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float mn = fmaxf(m, mx);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float w = live ? exp2f(x - mn) : 0.f;
    m = mn;
    float sum = w;
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    l = l * f + sum;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] *= f;
    unsigned act = __ballot_sync(0xffffffffu, live);
    while (act) {
      const int t = __ffs(act) - 1;
      act &= act - 1;
      const float wt = __shfl_sync(0xffffffffu, w, t);
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = fmaf(wt, value(t, lane + 32 * i), o[i]);
    }
  };
  for (int gr = 0; gr < L.n_groups; ++gr) {
    const int bits = L.bits;
    const uint8_t* blk = P.packed + L.packed_off +
                         ((size_t)unit * L.cap_groups + gr) * block_bytes(D, bits);
    const uint32_t* kw = reinterpret_cast<const uint32_t*>(blk);
    const uint32_t* vw = reinterpret_cast<const uint32_t*>(blk + off_vcodes(D, bits));
    const __half* ks = reinterpret_cast<const __half*>(blk + off_kscale(D, bits));
    const __half* kz = reinterpret_cast<const __half*>(blk + off_kzero(D, bits));
    const __half* vs = reinterpret_cast<const __half*>(blk + off_vscale(D, bits));
    const __half* vz = reinterpret_cast<const __half*>(blk + off_vzero(D, bits));
    const uint32_t msk = (1u << bits) - 1u;
    block(true,
          [&](int c) {
            const CodePos cp = kcode_pos(lane, c, D, bits);
            const int i = kperm(c, D);
            return fmaf((float)((kw[cp.word] >> cp.bit) & msk), __half2float(ks[i]),
                        __half2float(kz[i]));
          },
          [&](int t, int c) {
            const CodePos cp = vcode_pos(t, c, D, bits);
            return fmaf((float)((vw[cp.word] >> cp.bit) & msk),
                        __half2float(vs[vs_index(t, c >> 5, D / 32)]),
                        __half2float(vz[vsz_index(t, c >> 5, D / 32)]));
          });
  }
  const size_t rb = (size_t)L.win_off + (size_t)unit * L.R * D;
  for (int w0 = 0; w0 < L.win_len; w0 += 32)
    block(w0 + lane < L.win_len,
          [&](int c) {
            return __bfloat162float(
                P.win_k[rb + win_k_index((L.win_start + w0 + lane) % L.R, c, D)]);
          },
          [&](int t, int c) {
            return __bfloat162float(P.win_v[rb + win_v_index((L.win_start + w0 + t) % L.R, c, D)]);
          });
  const __nv_bfloat16* kd = P.k_draft + ul * T * D;
  const __nv_bfloat16* vd = P.v_draft + ul * T * D;
  for (int t0 = 0; t0 < T; t0 += 32)
    block((path >> (t0 + lane)) & 1ull,
          [&](int c) { return __bfloat162float(kd[(size_t)(t0 + lane) * D + c]); },
          [&](int t, int c) { return __bfloat162float(vd[(size_t)(t0 + t) * D + c]); });
  for (int i = 0; i < C; ++i) out[lane + 32 * i] = __float2bfloat16(o[i] / l);
}

}  // namespace

cudaError_t launch_tree(const kvc_cache* c, int layer_begin, int layer_count, int T,
                        const int32_t* parents, const __nv_bfloat16* q,
                        const __nv_bfloat16* k_draft, const __nv_bfloat16* v_draft,
                        __nv_bfloat16* out, cudaStream_t stream) {
  const kvc_dims& d = c->dims;
  const int units = d.batch * d.n_kv_heads;
  for (int base = 0; base < layer_count; base += KVC_MAX_LAUNCH_LAYERS) {
    const int cnt = std::min(layer_count - base, KVC_MAX_LAUNCH_LAYERS);
    TreeParams P;
    P.packed = c->packed;
    P.win_k = c->win_k;
    P.win_v = c->win_v;
    P.parents = parents;
    const size_t kvn = (size_t)base * units * T * d.head_dim;
    P.q = q + kvn * c->g;
    P.out = out + kvn * c->g;
    P.k_draft = k_draft + kvn;
    P.v_draft = v_draft + kvn;
    P.units = units;
    P.H = d.n_kv_heads;
    P.g = c->g;
    P.T = T;
    P.sl2 = 1.4426950408889634f / sqrtf((float)d.head_dim);
    for (int i = 0; i < cnt; ++i) {
      const LayerState& ls = c->L[layer_begin + base + i];
      P.L[i] = {(long long)ls.packed_off, (long long)ls.win_off, ls.n_groups, ls.cap_groups,
                ls.bits, ls.win_start, ls.win_len, ls.R};
    }
    const dim3 grid(units, (c->g * T + kTreeWarps - 1) / kTreeWarps, cnt);
    if (d.head_dim == 128) tree_simple_kernel<128><<<grid, kTreeWarps * 32, 0, stream>>>(P);
    else tree_simple_kernel<64><<<grid, kTreeWarps * 32, 0, stream>>>(P);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaSuccess;
}

}  // namespace kvc
