// logits.cu -- penalties for repeated tokens, biases and grammar masks on the
// logits of drafted nodes, with the argmax of each row in the same pass.
//
// A row's counts are those of its sequence's history plus the drafted tokens on
// the row's own path.  A CTA owns one vocabulary slice of one sequence: it
// counts the history's tokens of that slice in shared memory once (integer
// atomics: the order does not matter), and then takes rows of the sequence one
// after the other, adding the row's path tokens before and removing them after.
#include "tree_common.cuh"

namespace dfv {
namespace {

constexpr int kLogitThreads = 512;
constexpr uint32_t kSeenBit = 0x80000000u;  // the token is in the prompt; low bits count generated ones

struct RowRules {
  float rep, freq, pres;
  bool pen;
};

// Steps 1-5 of dfv_logits_process, every product, quotient and difference
// rounded on its own (no contraction).
__device__ __forceinline__ float rule(float x, uint32_t cnt, const RowRules &r, const LogitsParams &p, float bias,
                                      bool allowed) {
  if (r.pen) {
    const uint32_t c = cnt & ~kSeenBit;
    if (p.r.repetition && cnt) x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
    if (p.r.frequency) x = __fsub_rn(x, __fmul_rn(r.freq, (float)c));
    if (p.r.presence && c) x = __fsub_rn(x, r.pres);
  }
  if (p.r.bias) x = __fadd_rn(x, bias);
  return allowed ? x : -INFINITY;
}

template <bool F32>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(const LogitsParams p) {
  extern __shared__ uint32_t s_cnt[];
  __shared__ unsigned long long s_w[kLogitThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, b = blockIdx.y;
  const int v0 = blockIdx.x * p.slice, v1 = min(p.V, v0 + p.slice);
  int r0 = p.t.row_off[b], r1 = p.t.row_off[b + 1];
  if (r0 < 0 || r1 > p.t.n_rows || r1 - r0 > p.t.max_nodes) return;
  const int n = r1 - r0;
  if (n <= 0) return;
  RowRules rr = {};
  rr.pen = p.r.repetition || p.r.frequency || p.r.presence;
  if (rr.pen) {
    if (p.r.repetition) rr.rep = p.r.repetition[b];
    if (p.r.frequency) rr.freq = p.r.frequency[b];
    if (p.r.presence) rr.pres = p.r.presence[b];
    for (int i = tid; i < v1 - v0; i += kLogitThreads) s_cnt[i] = 0u;
    __syncthreads();
    if (p.r.hist) {
      const int32_t *h = p.r.hist + b * p.r.hist_row;
      const int L = (int)min((long long)p.r.hist_len[b], (long long)p.r.hist_row), P = p.r.prompt_len ? p.r.prompt_len[b] : 0;
      for (int i = tid; i < L; i += kLogitThreads) {
        const unsigned c = (unsigned)h[i] - (unsigned)v0;
        if (c < (unsigned)(v1 - v0)) {
          if (i < P)
            atomicOr(&s_cnt[c], kSeenBit);
          else
            atomicAdd(&s_cnt[c], 1u);
        }
      }
    }
    __syncthreads();
  }
  for (int i = blockIdx.z; i < n; i += gridDim.z) {
    const int row = r0 + i;
    unsigned mine = 0xffffffffu;  // slice column of the path token this thread adds
    if (rr.pen && p.tokens) {
      if (tid < n && ((row_mask(p.t, r0, i) >> tid) & 1)) mine = (unsigned)p.tokens[r0 + tid] - (unsigned)v0;
      if (mine < (unsigned)(v1 - v0))
        atomicAdd(&s_cnt[mine], 1u);
      else
        mine = 0xffffffffu;
      __syncthreads();
    }
    const float *bias = p.r.bias ? p.r.bias + b * p.r.bias_row : nullptr;
    const uint32_t *ok = p.r.allowed ? p.r.allowed + row * p.r.allowed_row : nullptr;
    unsigned long long best = 0ull;
    for (int v = v0 + tid; v < v1; v += kLogitThreads) {
      float x = F32 ? reinterpret_cast<const float *>(p.x)[row * p.row + v]
                    : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p.x)[row * p.row + v] << 16);
      x = rule(x, rr.pen ? s_cnt[v - v0] : 0u, rr, p, bias ? bias[v] : 0.f,
               !ok || ((ok[v >> 5] >> (v & 31)) & 1u));
      if (!F32) {
        const uint16_t y = f32_to_bf16_bits(x);
        x = __uint_as_float((uint32_t)y << 16);
        if (p.out) reinterpret_cast<uint16_t *>(p.out)[row * p.out_row + v] = y;
      } else if (p.out) {
        reinterpret_cast<float *>(p.out)[row * p.out_row + v] = x;
      }
      const unsigned long long key =
          ((unsigned long long)float_key(x) << 32) | (unsigned long long)(0xffffffffu - (unsigned)v);
      best = key > best ? key : best;
    }
    if (p.argmax) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long w = __shfl_xor_sync(0xffffffffu, best, o);
        best = w > best ? w : best;
      }
      if ((tid & 31) == 0) s_w[tid >> 5] = best;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kLogitThreads / 32; ++w) best = s_w[w] > best ? s_w[w] : best;
        atomicMax(&p.key[row], best);
        __threadfence();
        if (atomicAdd(&p.ticket[row], 1u) == gridDim.x - 1) {
          __threadfence();
          const unsigned long long k = atomicExch(&p.key[row], 0ull);
          p.argmax[row] = (int32_t)(0xffffffffu - (unsigned)(k & 0xffffffffull));
          p.ticket[row] = 0u;
        }
      }
    }
    __syncthreads();  // the counts and s_w are read
    if (mine != 0xffffffffu) atomicSub(&s_cnt[mine], 1u);
  }
}

}  // namespace

cudaError_t launch_logits(const LogitsParams &p0, cudaStream_t s) {
  LogitsParams p = p0;
  p.slice = 4096;
  const dim3 grid((p.V + p.slice - 1) / p.slice, p.t.n_seqs, 1);
  const size_t smem = (size_t)p.slice * 4;
  return p.f32 ? launch_chained(logits_kernel<true>, grid, dim3(kLogitThreads), smem, s, p)
               : launch_chained(logits_kernel<false>, grid, dim3(kLogitThreads), smem, s, p);
}

}  // namespace dfv
