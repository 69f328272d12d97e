// cache.cu -- the greedy walk of drafted trees and the pages of the cache:
// committing an accepted path, copying, reserving, forking and freeing pages.
//
// All bookkeeping lives on the device (page table, lengths, reference counts),
// so that a verify step needs no host round trip and can be captured.  A free
// page is one with reference count 0 and pages are given out lowest index
// first: what a call does depends on no order of atomics.
//
// Bound by latency: a few launches over little data.  Measured on the device:
// walk and commit 4.8 us for one 16-node tree in 8 layers and 8.5 us for 32
// 64-node trees in 40 layers (20 MB moved); 12 sequences dropped and forked again
// in 40 layers 10.3 us (three launches).
#include "tree_common.cuh"

namespace dfv {
namespace {

// ---------------------------------------------------------------- greedy walk
// One warp per sequence, two nodes per lane: (parent, token) of every node in
// registers, the target tokens in shared memory; each step of the walk is one
// ballot over the children of the current node.
__global__ void __launch_bounds__(32) accept_tree_kernel(const AcceptTreeParams p) {
  __shared__ int s_target[DFV_MAX_TREE];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, lane = threadIdx.x;
  const int r0 = p.t.row_off[b], r1 = p.t.row_off[b + 1];
  int n = r1 - r0;
  if (r0 < 0 || r1 > p.t.n_rows || n < 0 || n > p.t.max_nodes) n = 0;
  int up[2], tok[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = lane + 32 * q;
    up[q] = -1;
    tok[q] = 0;
    if (i < n) {
      const uint64_t below = row_mask(p.t, r0, i) & ((1ull << i) - 1ull);
      up[q] = below ? 63 - __clzll((long long)below) : -1;
      tok[q] = p.tokens[r0 + i];
      s_target[i] = p.target[r0 + i];
    }
  }
  __syncwarp();
  int32_t *path = p.path + b * p.path_row;
  int cur = 0, tau = 0;
  int mine[2] = {-1, -1};  // path entries lane and lane + 32
  while (tau < n) {
    if (tau < 32) { if (lane == tau) mine[0] = cur; } else { if (lane == tau - 32) mine[1] = cur; }
    ++tau;
    const int want = s_target[cur];
    const unsigned lo = __ballot_sync(0xffffffffu, lane < n && up[0] == cur && tok[0] == want);
    const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < n && up[1] == cur && tok[1] == want);
    if (!(lo | hi)) break;
    cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (lane + 32 * q < p.t.max_nodes) path[lane + 32 * q] = mine[q];
  if (lane == 0) p.tau[b] = tau;
}

// ---------------------------------------------------------------- commit
constexpr int kCommitThreads = 128;

// One CTA per (sequence, layer): thread = one 16-byte piece of (k or v, head);
// it moves the piece of every accepted row, in batches that are read before
// they are written.  Row j is read from path[j] >= j, and a later batch reads
// only rows at or above every row written so far: no row is lost.
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const CommitParams p) {
  __shared__ int s_path[DFV_MAX_TREE];
  __shared__ long long s_from[DFV_MAX_TREE], s_to[DFV_MAX_TREE];
  __shared__ int s_bad;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const CacheParams &c = p.c;
  const SeqView v = seq_view(c, p.t, b);
  int tau = p.tau[b];
  if (tid == 0) s_bad = 0;
  __syncthreads();
  if (tau < 0 || tau > v.n) {
    if (tid == 0) flag_err(c.err, DFV_KVERR_PATH);
    tau = 0;
  }
  if (v.s < 0) tau = 0;
  if (tid < tau) s_path[tid] = p.path[b * p.path_row + tid];
  __syncthreads();
  if (tid < tau) {
    const int x = s_path[tid], y = tid ? s_path[tid - 1] : -1;
    if (x <= y || x >= v.n) {
      s_bad = DFV_KVERR_PATH;
    } else {
      const int pm = (1 << c.page_shift) - 1, from = v.len + x, to = v.len + tid;
      const int pf = page_of(c, v.s, from), pt = page_of(c, v.s, to);
      if (pf < 0 || pt < 0)
        s_bad = DFV_KVERR_PAGE;
      else {
        s_from[tid] = kv_off(c, layer, pf, 0, from & pm);
        s_to[tid] = kv_off(c, layer, pt, 0, to & pm);
      }
    }
  }
  __syncthreads();
  if (s_bad) {
    if (tid == 0) flag_err(c.err, (uint32_t)s_bad);
    tau = 0;
  }
  const int D8 = c.D / 8, pieces = 2 * c.Hkv * D8;
  // accepted rows that are already in place
  int first = 0;
  while (first < tau && s_path[first] == first) ++first;
  for (int u = tid; u < pieces; u += kCommitThreads) {
    const int kv = u / (c.Hkv * D8), w = u - kv * c.Hkv * D8, h = w / D8, e = w - h * D8;
    char *base = (kv ? c.v : c.k) + 2 * (h * c.sh + e * 8);
    for (int j0 = first; j0 < tau; j0 += 8) {
      uint4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < tau) x[j] = *reinterpret_cast<const uint4 *>(base + 2 * s_from[j0 + j]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < tau) *reinterpret_cast<uint4 *>(base + 2 * s_to[j0 + j]) = x[j];
    }
  }
  // the last layer's CTA of the sequence to finish sets the new length: by then
  // every CTA has read the old one
  __syncthreads();
  if (tid == 0 && v.s >= 0) {
    __threadfence();
    if (atomicAdd(&p.ticket[b], 1u) == gridDim.y - 1) {
      p.new_lens[v.s] = v.len + tau;
      p.ticket[b] = 0u;
    }
  }
}

// ---------------------------------------------------------------- pages
constexpr int kCopyThreads = 256;

// rows [0, rows) of page `from` to page `to`, in one layer
__device__ __forceinline__ void copy_rows(const CacheParams &c, int layer, int from, int to, int rows, int part,
                                          int parts) {
  const int D8 = c.D / 8, per = c.Hkv * rows * D8;
  const long long f = kv_off(c, layer, from, 0, 0), t = kv_off(c, layer, to, 0, 0);
  for (int u = part; u < 2 * per; u += parts) {
    const int kv = u >= per, w = kv ? u - per : u;
    const int e = w % D8, hr = w / D8, r = hr % rows, h = hr / rows;
    const long long off = h * c.sh + r * c.st + e * 8;
    char *base = kv ? c.v : c.k;
    *reinterpret_cast<uint4 *>(base + 2 * (t + off)) = *reinterpret_cast<const uint4 *>(base + 2 * (f + off));
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const PagesParams p) {
  pdl_trigger();
  pdl_wait();
  const int from = p.a[blockIdx.x], to = p.b[blockIdx.x];
  if ((unsigned)from >= (unsigned)p.c.n_pages || (unsigned)to >= (unsigned)p.c.n_pages) {
    if (threadIdx.x == 0) flag_err(p.c.err, DFV_KVERR_PAGE);
    return;
  }
  if (from != to) copy_rows(p.c, blockIdx.y, from, to, 1 << p.c.page_shift, threadIdx.x, kCopyThreads);
}

constexpr int kPageThreads = 1024;

// exclusive scan over the CTA; returns the total in *sum.  s: 33 ints.
__device__ __forceinline__ int block_scan(int x, int *s, int *sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += a;
  }
  __syncthreads();  // s is free again
  if (lane == 31) s[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = s[lane], z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += a;
    }
    s[lane] = z - w;
    if (lane == 31) s[32] = z;
  }
  __syncthreads();
  *sum = s[32];
  return s[warp] + v - x;
}

// got[0 .. min(m, free)) = the lowest free pages; returns how many were found.
// Threads take 16 consecutive pages each.
__device__ int find_free(const CacheParams &c, int m, int32_t *got, int *s) {
  int found = 0;
  for (int base = 0; base < c.n_pages && found < m; base += 16 * kPageThreads) {
    const int p0 = base + 16 * threadIdx.x;
    unsigned free16 = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (p0 + j < c.n_pages && c.refs[p0 + j] == 0) free16 |= 1u << j;
    int sum;
    int rank = found + block_scan(__popc(free16), s, &sum);
    while (free16 && rank < m) {
      const int j = __ffs(free16) - 1;
      free16 &= free16 - 1;
      got[rank++] = p0 + j;
    }
    found += sum;
  }
  __syncthreads();
  return found < m ? found : m;
}

// One CTA.  Sequences are counted one per thread, free pages found, and handed
// out by the prefix sums of the counts.
__global__ void __launch_bounds__(kPageThreads) reserve_kernel(const PagesParams p) {
  __shared__ int s_scan[33], s_seq[DFV_MAX_TREE_SEQS], s_first[DFV_MAX_TREE_SEQS], s_need[DFV_MAX_TREE_SEQS],
      s_end[DFV_MAX_TREE_SEQS];
  pdl_trigger();
  pdl_wait();
  const CacheParams &c = p.c;
  const int tid = threadIdx.x;
  int s = -1;
  if (tid < p.n) {
    s = p.a[tid];
    if (s < 0 || s >= c.max_seqs) {
      flag_err(c.err, DFV_KVERR_SEQ);
      s = -1;
    }
    s_seq[tid] = s;
  }
  __syncthreads();
  int p0 = 0, p1 = 0, need = 0;
  if (s >= 0) {
    for (int j = 0; j < tid; ++j)
      if (s_seq[j] == s) {
        flag_err(c.err, DFV_KVERR_SEQ);
        s = -1;
        break;
      }
  }
  if (s >= 0) {
    const long long len = c.lens[s], want = len + p.b[tid];
    if (len < 0 || p.b[tid] < 0 || want > ((long long)c.max_pages << c.page_shift)) {
      flag_err(c.err, DFV_KVERR_LEN);
      s = -1;
    } else {
      p1 = (int)((want + (1 << c.page_shift) - 1) >> c.page_shift);
      for (int j = p0; j < p1; ++j) need += c.table[(size_t)s * c.max_pages + j] < 0;
    }
  }
  int m;
  const int first = block_scan(need, s_scan, &m);
  const int found = find_free(c, m, p.got, s_scan);
  if (tid < p.n) {
    if (first + need > found) {
      flag_err(c.err, DFV_KVERR_NO_PAGE);
      need = 0;
    }
    s_first[tid] = first;
    s_need[tid] = s < 0 ? 0 : need;
    s_end[tid] = p1;
  }
  __syncthreads();
  // a warp per sequence: missing entries in order
  const int lane = tid & 31;
  for (int b = tid >> 5; b < p.n; b += kPageThreads / 32) {
    int left = s_need[b], at = s_first[b];
    int32_t *row = c.table + (size_t)s_seq[b] * c.max_pages;
    for (int j0 = 0; j0 < s_end[b] && left > 0; j0 += 32) {
      const bool miss = j0 + lane < s_end[b] && row[j0 + lane] < 0;
      const unsigned bal = __ballot_sync(0xffffffffu, miss);
      if (miss) {
        const int pg = p.got[at + __popc(bal & ((1u << lane) - 1u))];
        row[j0 + lane] = pg;
        c.refs[pg] = 1;
      }
      at += __popc(bal);
      left -= __popc(bal);
    }
  }
}

// One CTA: which forks go ahead, and the pages for their copied last pages.
// plan[f] = {source length or -1, last source page or -1, its copy, 0}
__global__ void __launch_bounds__(kPageThreads) fork_plan_kernel(const PagesParams p) {
  __shared__ int s_scan[33], s_dst[DFV_MAX_TREE_SEQS];
  pdl_trigger();
  pdl_wait();
  const CacheParams &c = p.c;
  const int tid = threadIdx.x;
  int src = -1, dst = -1, len = -1, last = -1, need = 0;
  if (tid < p.n) {
    src = p.a[tid];
    dst = p.b[tid];
    s_dst[tid] = dst;
  }
  __syncthreads();
  if (tid < p.n) {
    bool ok = src >= 0 && src < c.max_seqs && dst >= 0 && dst < c.max_seqs && src != dst;
    for (int j = 0; ok && j < tid; ++j) ok = s_dst[j] != dst;
    if (ok) ok = c.lens[dst] == 0 && c.table[(size_t)dst * c.max_pages] < 0;
    if (!ok) {
      flag_err(c.err, DFV_KVERR_SEQ);
    } else {
      len = c.lens[src];
      if (len < 0 || len > ((long long)c.max_pages << c.page_shift)) {
        flag_err(c.err, DFV_KVERR_LEN);
        len = -1;
      } else if (len & ((1 << c.page_shift) - 1)) {
        last = page_of(c, src, len);
        if (last < 0)
          len = -1;
        else
          need = 1;
      }
    }
  }
  int m;
  const int rank = block_scan(need, s_scan, &m);
  const int found = find_free(c, m, p.got, s_scan);
  if (tid < p.n) {
    int got = -1;
    if (need && rank >= found) {
      flag_err(c.err, DFV_KVERR_NO_PAGE);
      len = -1;
    } else if (need) {
      got = p.got[rank];
      c.refs[got] = 1;
    }
    reinterpret_cast<int4 *>(p.plan)[tid] = make_int4(len, last, got, 0);
  }
}

// One CTA per (fork, layer): the used rows of the last page; layer 0 also
// shares the whole pages and writes the new table row.
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(const PagesParams p) {
  pdl_trigger();
  pdl_wait();
  const CacheParams &c = p.c;
  const int4 pl = reinterpret_cast<const int4 *>(p.plan)[blockIdx.x];
  const int len = pl.x;
  if (len < 0) return;
  const int full = len >> c.page_shift, rest = len & ((1 << c.page_shift) - 1);
  if (blockIdx.y == 0) {
    const int src = p.a[blockIdx.x], dst = p.b[blockIdx.x];
    const int32_t *from = c.table + (size_t)src * c.max_pages;
    int32_t *to = c.table + (size_t)dst * c.max_pages;
    for (int j = threadIdx.x; j < full; j += kCopyThreads) {
      const int pg = from[j];
      if ((unsigned)pg < (unsigned)c.n_pages)
        atomicAdd(&c.refs[pg], 1);
      else
        flag_err(c.err, DFV_KVERR_PAGE);
      to[j] = pg;
    }
    if (threadIdx.x == 0) {
      if (rest) to[full] = pl.z;
      c.lens[dst] = len;
    }
  }
  if (rest) copy_rows(c, blockIdx.y, pl.y, pl.z, rest, threadIdx.x, kCopyThreads);
}

// One CTA per sequence.  Entries are taken with an exchange, so a sequence
// given twice is dropped once.
__global__ void __launch_bounds__(kCopyThreads) free_kernel(const PagesParams p) {
  pdl_trigger();
  pdl_wait();
  const CacheParams &c = p.c;
  const int s = p.a[blockIdx.x];
  if (s < 0 || s >= c.max_seqs) {
    if (threadIdx.x == 0) flag_err(c.err, DFV_KVERR_SEQ);
    return;
  }
  int32_t *row = c.table + (size_t)s * c.max_pages;
  for (int j = threadIdx.x; j < c.max_pages; j += kCopyThreads) {
    if (row[j] == -1) continue;
    const int pg = atomicExch(&row[j], -1);
    if (pg == -1) continue;
    if ((unsigned)pg >= (unsigned)c.n_pages)
      flag_err(c.err, DFV_KVERR_PAGE);
    else if (atomicSub(&c.refs[pg], 1) <= 0) {
      atomicAdd(&c.refs[pg], 1);  // it was free already
      flag_err(c.err, DFV_KVERR_PAGE);
    }
  }
  if (threadIdx.x == 0) c.lens[s] = 0;
}

}  // namespace

cudaError_t launch_accept_tree(const AcceptTreeParams &p, cudaStream_t s) {
  return launch_chained(accept_tree_kernel, dim3(p.t.n_seqs), dim3(32), 0, s, p);
}

cudaError_t launch_commit(const CommitParams &p, cudaStream_t s) {
  return launch_chained(commit_kernel, dim3(p.t.n_seqs, p.c.n_layers), dim3(kCommitThreads), 0, s, p);
}

cudaError_t launch_copy_pages(const PagesParams &p, cudaStream_t s) {
  return launch_chained(copy_pages_kernel, dim3(p.n, p.c.n_layers), dim3(kCopyThreads), 0, s, p);
}

cudaError_t launch_reserve(const PagesParams &p, cudaStream_t s) {
  return launch_chained(reserve_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
}

cudaError_t launch_fork(const PagesParams &p, cudaStream_t s) {
  const cudaError_t e = launch_chained(fork_plan_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_chained(fork_copy_kernel, dim3(p.n, p.c.n_layers), dim3(kCopyThreads), 0, s, p);
}

cudaError_t launch_free(const PagesParams &p, cudaStream_t s) {
  return launch_chained(free_kernel, dim3(p.n), dim3(kCopyThreads), 0, s, p);
}

}  // namespace dfv
