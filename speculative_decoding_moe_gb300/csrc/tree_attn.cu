// tree_attn.cu -- attention of drafted tree nodes over the paged cache.
#include "tree_common.cuh"

namespace dfv {
namespace {

constexpr int kWarps = 4;

// One CTA per (sequence, node, query head): each warp takes every fourth key,
// lanes hold D / 32 elements, with the running maximum and sum of a softmax;
// the warps' states are joined at the end.
template <bool F16, int D>
__global__ void __launch_bounds__(32 * kWarps) tree_attn_simple_kernel(const TreeAttnParams p) {
  constexpr int E = D / 64;  // 32-bit words per lane
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const SeqView v = seq_view(p.c, p.t, b);
  if (i >= v.n) return;
  const int row = v.row0 + i, hk = h / p.G;
  const uint64_t mask = row_mask(p.t, v.row0, i);
  const int total = v.s < 0 ? 0 : v.len + v.n;
  float2 q[E], o[E];
  const uint32_t *qp = reinterpret_cast<const uint32_t *>(p.q + 2 * (row * p.q_row + h * p.q_head));
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = unpack2<F16>(qp[lane + 32 * e]);
    o[e] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  for (int pos = warp; pos < total; pos += kWarps) {
    if (pos >= v.len && !((mask >> (pos - v.len)) & 1)) continue;
    const int pg = page_of(p.c, v.s, pos);
    const long long off = kv_off(p.c, p.layer, pg < 0 ? 0 : pg, hk, pos & ((1 << p.c.page_shift) - 1));
    const uint32_t *kp = reinterpret_cast<const uint32_t *>(p.c.k + 2 * off);
    const uint32_t *vp = reinterpret_cast<const uint32_t *>(p.c.v + 2 * off);
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 kk = unpack2<F16>(kp[lane + 32 * e]);
      x += q[e].x * kk.x + q[e].y * kk.y;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= p.scale_log2;
    const float mn = fmaxf(m, x);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), pr = x == -INFINITY ? 0.f : exp2f(x - mn);
    l = l * a + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 vv = unpack2<F16>(vp[lane + 32 * e]);
      o[e].x = o[e].x * a + pr * vv.x;
      o[e].y = o[e].y * a + pr * vv.y;
    }
    m = mn;
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int e = 0; e < E; ++e) reinterpret_cast<float2 *>(s_o[warp])[lane + 32 * e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f, f[kWarps];
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  for (int w = 0; w < kWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
    L += f[w] * s_l[w];
  }
  for (int e = threadIdx.x; e < D / 2; e += 32 * kWarps) {
    float x = 0.f, y = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      x += f[w] * s_o[w][2 * e];
      y += f[w] * s_o[w][2 * e + 1];
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // NaN stays NaN
    reinterpret_cast<uint32_t *>(p.o + 2 * (row * p.o_row + h * p.o_head))[e] = pack2<F16>(x * inv, y * inv);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(size_t)row * p.H + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_tree_attn(const TreeAttnParams &p, cudaStream_t s) {
  const dim3 grid(p.H, p.t.max_nodes, p.t.n_seqs), block(32 * kWarps);
  if (p.c.D == 128)
    return p.c.f16 ? launch_chained(tree_attn_simple_kernel<true, 128>, grid, block, 0, s, p)
                   : launch_chained(tree_attn_simple_kernel<false, 128>, grid, block, 0, s, p);
  return p.c.f16 ? launch_chained(tree_attn_simple_kernel<true, 64>, grid, block, 0, s, p)
                 : launch_chained(tree_attn_simple_kernel<false, 64>, grid, block, 0, s, p);
}

}  // namespace dfv
