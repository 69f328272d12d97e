// rope.cu -- rotary positions of the drafted rows and their keys and values
// stored into the paged cache, in one launch.
//
// Mathematics: the angle of pair i at position p is p * f_i.  Its sine and
// cosine only need the fraction of a turn, p * f_i / (2 pi) mod 1.  The table
// holds F_i = round(f_i / (2 pi) * 2^64); p * F_i in wrapping 64-bit integers is
// then that fraction as a 0.64 fixed-point number, exact up to p * 2^-65 turns,
// at any position.  Its upper 32 bits, read as signed, are an angle in
// [-1/2, 1/2) turns that sincospi takes without further reduction (an fp32
// product p * f_i would be off by 4e-3 rad at p = 65536).
//
// Bound by latency: a row is a few KB, read and written once.  One CTA per row
// finds its sines and cosines once for all heads.  Measured on the device: 2.9 us
// for one row of 40 heads of 128, 9.0 us for 1549 such rows (31.7 MB, 3.5 TB/s).
#include <cmath>

#include "tree_common.cuh"

namespace dfv {
namespace {

constexpr int kRopeThreads = 256;

template <bool F16>
__device__ __forceinline__ void rot8(uint4 &a, uint4 &b, const float2 *cs) {
  uint32_t *x = &a.x, *y = &b.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<F16>(x[i]), w = unpack2<F16>(y[i]);
    const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
    x[i] = pack2<F16>(u.x * c0.x - w.x * c0.y, u.y * c1.x - w.y * c1.y);
    y[i] = pack2<F16>(w.x * c0.x + u.x * c0.y, w.y * c1.x + u.y * c1.y);
  }
}
template <bool F16>
__device__ __forceinline__ void rot4i(uint4 &a, const float2 *cs) {
  uint32_t *x = &a.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<F16>(x[i]);
    x[i] = pack2<F16>(u.x * cs[i].x - u.y * cs[i].y, u.y * cs[i].x + u.x * cs[i].y);
  }
}

// One CTA per (sequence, node): the row's cos / sin once, then its heads in
// 16-byte pieces (half layout: two pieces half a rotation apart).
template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p) {
  __shared__ float2 s_cs[128];
  const int b = blockIdx.x, i = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const SeqView v = seq_view(p.c, p.t, b);
  if (i >= v.n) return;
  const int row = v.row0 + i;
  const long long pos = p.positions[row];
  for (int j = tid; j < p.rot / 2; j += kRopeThreads) {
    const uint64_t turn = (uint64_t)pos * p.turns[j];
    float sn, cs;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
    s_cs[j] = make_float2(cs * p.scale, sn * p.scale);
  }
  int pg = -1;
  long long dst = 0;
  if (v.s >= 0) {
    const int at = v.len + i;
    pg = page_of(p.c, v.s, at);
    dst = kv_off(p.c, p.layer, pg, 0, at & ((1 << p.c.page_shift) - 1));
  }
  __syncthreads();
  const int D8 = p.c.D / 8, r8 = p.rot / 8;
  // pieces of a turned head: pairs of pieces (half) or single pieces (interleaved), then the tail
  const int nrot = p.inter ? r8 : r8 / 2, per = nrot + D8 - r8;
  const int nq = p.H * per, nk = p.c.Hkv * per, nv = p.c.Hkv * D8;
  for (int u = tid; u < nq + nk + nv; u += kRopeThreads) {
    const char *src;
    char *to;
    int e;
    bool turned = true;
    if (u < nq + nk) {
      const bool isq = u < nq;
      const int w = isq ? u : u - nq, h = w / per;
      e = w - h * per;
      src = isq ? p.q + 2 * (row * p.q_row + h * p.q_head) : p.k + 2 * (row * p.k_row + h * p.k_head);
      to = isq ? p.o + 2 * (row * p.o_row + h * p.o_head) : p.c.k + 2 * (dst + h * p.c.sh);
      if (!isq && pg < 0) continue;
      if (e >= nrot) {
        turned = false;
        e += r8 - nrot;
      }
    } else {
      if (pg < 0) continue;
      const int w = u - nq - nk, h = w / D8;
      e = w - h * D8;
      src = p.v + 2 * (row * p.v_row + h * p.v_head);
      to = p.c.v + 2 * (dst + h * p.c.sh);
      turned = false;
    }
    const uint4 *s4 = reinterpret_cast<const uint4 *>(src);
    uint4 *t4 = reinterpret_cast<uint4 *>(to);
    uint4 x = s4[e];
    if (!turned) {
      t4[e] = x;
    } else if (p.inter) {
      rot4i<F16>(x, s_cs + 4 * e);
      t4[e] = x;
    } else {
      uint4 y = s4[e + nrot];
      rot8<F16>(x, y, s_cs + 8 * e);
      t4[e] = x;
      t4[e + nrot] = y;
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams &p, cudaStream_t s) {
  const dim3 grid(p.t.n_seqs, p.t.max_nodes);
  return p.c.f16 ? launch_chained(rope_append_kernel<true>, grid, dim3(kRopeThreads), 0, s, p)
                 : launch_chained(rope_append_kernel<false>, grid, dim3(kRopeThreads), 0, s, p);
}

}  // namespace dfv
