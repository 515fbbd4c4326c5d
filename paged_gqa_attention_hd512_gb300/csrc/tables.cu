// tables.cu -- page tables on the GPU: requests that grow or shrink take pages from a free
// list or give them back (the block table's rows follow), and a batch's block-table rows and
// lengths become the CSR page lists, slots and positions that the other calls take.
//
// Pages of a length: ceil(len / page_size).  Both kernels turn the batch's page (and token)
// counts into offsets by block-wide scans over rounds of 1024 sequences, then hand out the
// moved or listed entries evenly over the threads, each finding its sequence by a binary
// search among the round's ends in shared memory.  What bounds them is latency: the launch
// and the chain length -> scan -> entry (a decode step moves a few hundred bytes, the tables
// of 128 sequences of 32768 tokens at 16 tokens a page are 2 MB).  Both are launched as
// programmatic dependents and let their own dependents launch at once, so that the kernels of a
// step (resize, build, append, decode) overlap their launches.
#include <algorithm>

#include "launch.h"
#include "common.cuh"

namespace pa {

namespace {

constexpr int kT = 1024;  // threads, and sequences per round
constexpr int kU = 4;     // pages of a resize's thread whose loads are in flight together

// Inclusive block-wide sums of a and of b (kT threads); w holds the totals in w[.][32].
struct ScanWords {
  long long w[2][33];
};
__device__ __forceinline__ void block_scan(long long& a, long long& b, ScanWords& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ta = __shfl_up_sync(0xffffffffu, a, o), tb = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += ta, b += tb;
  }
  if (lane == 31) s.w[0][warp] = a, s.w[1][warp] = b;
  __syncthreads();
  if (warp < 2) {  // a warp for each of the sums
    long long v = s.w[warp][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    s.w[warp][lane] = v;
    if (lane == 31) s.w[warp][32] = v;
  }
  __syncthreads();
  if (warp > 0) a += s.w[0][warp - 1], b += s.w[1][warp - 1];
}

__device__ __forceinline__ long long block_sum(long long v, long long* s_w) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) v += s_w[w];
  __syncthreads();
  return v;
}

// The first of the round's kT inclusive ends that lies above x (there is one): ten steps.
__device__ __forceinline__ int find_end(const int* ends, int x) {
  int lo = 0;
#pragma unroll
  for (int step = kT / 2; step > 0; step >>= 1)
    if (ends[lo + step - 1] <= x) lo += step;
  return lo;
}

struct Change {
  int row, p_old, p_new, len_new;
  bool bad;
};

// Sequence b's row and page counts before and after (row -1: nothing to do).
__device__ __forceinline__ Change change_of(const ResizeParams& p, int b) {
  Change c = {-1, 0, 0, 0, false};
  if (b >= p.batch) return c;
  const int row = p.row_ids ? p.row_ids[b] : b;
  if (row < 0) return c;
  c.bad = true;
  if (row >= p.rows) return c;
  const long long len = p.kv_lens[row], to = len + p.deltas[b], most = (long long)p.max_pages << p.log2_page;
  if (len < 0 || to < 0 || len > most || to > most) return c;
  c.bad = false;
  c.row = row;
  c.p_old = (int)((len + (1 << p.log2_page) - 1) >> p.log2_page);
  c.p_new = (int)((to + (1 << p.log2_page) - 1) >> p.log2_page);
  c.len_new = (int)to;
  return c;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster: every CTA reads lengths and count and forms the same offsets, each moves its
// share of the pages, and the barriers order what one CTA moves against what another reads
// (a page given back may be taken again) and the updates of lengths and count against their
// readers.
__global__ void __launch_bounds__(kT, 1) resize_kernel(const ResizeParams p) {
  __shared__ int s_end[kT], s_row[kT], s_first[kT];
  __shared__ ScanWords s_w;
  __shared__ long long s_l[32];
  const int tid = threadIdx.x, part = blockIdx.x, parts = gridDim.x;
  grid_dep_wait();
  grid_dep_launch();  // the next call's kernel may start its set-up (it waits for this grid)
  const long long count = *p.free_count;
  const Change c0 = change_of(p, tid);
  const bool one_round = p.batch <= kT;
  long long back = max(c0.p_old - c0.p_new, 0), take = max(c0.p_new - c0.p_old, 0);
  int bad = c0.bad;
  for (int b = tid + kT; b < p.batch; b += kT) {
    const Change c = change_of(p, b);
    bad |= c.bad;
    back += max(c.p_old - c.p_new, 0);
    take += max(c.p_new - c.p_old, 0);
  }
  bad = __syncthreads_or(bad);
  // ends of this thread's sequence among the pages given back and among those taken
  long long end_back = back, end_take = take;
  if (one_round) {
    block_scan(end_back, end_take, s_w);
    back = s_w.w[0][32];
    take = s_w.w[1][32];
  } else {
    back = block_sum(back, s_l);
    take = block_sum(take, s_l);
  }
  if (bad || count < 0 || count + back > p.free_size || take > count + back) {
    if (part == 0 && tid == 0) record_error(p.data_err, SITE_RESIZE);  // nothing is changed
    return;  // every CTA of the cluster
  }
  // pages given back go behind the free list's end, in batch and table order; then pages
  // are taken from its end
  for (int phase = 0; phase < 2; ++phase) {
    if (phase == 0 ? back == 0 : take == 0) continue;
    if (phase == 1 && back > 0) cluster_barrier();
    long long done = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kT) {
      const Change c = one_round ? c0 : change_of(p, b0 + tid);
      const int n = phase == 0 ? max(c.p_old - c.p_new, 0) : max(c.p_new - c.p_old, 0);
      if (!one_round) {
        end_back = end_take = n;
        block_scan(end_back, end_take, s_w);
      }
      const int end = (int)(phase == 0 ? end_back : end_take);
      s_end[tid] = end;
      s_row[tid] = c.row;
      s_first[tid] = min(c.p_old, c.p_new) + n - end;  // + item: the page's place in its row
      const int total = (int)s_w.w[phase][32];
      __syncthreads();
      for (unsigned i0 = part * kT + tid; i0 < (unsigned)total; i0 += kU * parts * kT) {
        int* dst[kU];
        int page[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = (int)min(i0 + u * parts * kT, (unsigned)total - 1);
          const int k = find_end(s_end, i);
          int* entry = p.block_table + (size_t)s_row[k] * p.table_stride + s_first[k] + i;
          int* listed = p.free_pages + (phase == 0 ? count + done + i : count + back - 1 - done - i);
          dst[u] = phase == 0 ? listed : entry;
          page[u] = __ldcg(phase == 0 ? entry : listed);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (i0 + u * parts * kT < (unsigned)total) *dst[u] = page[u];
      }
      done += total;
      __syncthreads();
    }
  }
  cluster_barrier();  // every CTA has read lengths and count
  if (part == 0) {
    if (c0.row >= 0) p.kv_lens[c0.row] = c0.len_new;
    for (int b = tid + kT; b < p.batch; b += kT) {
      const Change c = change_of(p, b);
      if (c.row >= 0) p.kv_lens[c.row] = c.len_new;
    }
  }
  if (part == 0 && tid == 0) *p.free_count = (int)(count + back - take);
}

struct Listed {
  int row, len, pages, fresh;
  bool bad;
};

// Sequence b's row, length, pages and new tokens (all 0 for padding and for bad entries).
__device__ __forceinline__ Listed listed_of(const BuildParams& p, int b) {
  Listed l = {0, 0, 0, 0, false};
  if (b >= p.batch) return l;
  const int row = p.row_ids ? p.row_ids[b] : b;
  if (row < 0) return l;
  l.bad = true;
  if (row >= p.rows) return l;
  const int len = p.kv_lens[row], fresh = max(0, p.new_counts[b]);
  if (len < 0 || len > ((long long)p.max_pages << p.log2_page) || fresh > len) return l;
  return {row, len, (int)(((long long)len + (1 << p.log2_page) - 1) >> p.log2_page), fresh, false};
}

// Every CTA scans the whole batch (a few loads per thread) and writes its share of the
// entries, so that one launch does without a grid-wide exchange.
__global__ void __launch_bounds__(kT, 1) build_kernel(const BuildParams p) {
  __shared__ int s_page_end[kT], s_page_first[kT], s_tok_end[kT], s_tok_first[kT], s_row[kT];
  __shared__ ScanWords s_w;
  __shared__ long long s_l[32];
  const int tid = threadIdx.x, ps = 1 << p.log2_page;
  grid_dep_wait();
  grid_dep_launch();
  const Listed l0 = listed_of(p, tid);
  const bool one_round = p.batch <= kT;
  long long pages = l0.pages, tokens = l0.fresh;
  int bad = l0.bad;
  for (int b = tid + kT; b < p.batch; b += kT) {
    const Listed l = listed_of(p, b);
    bad |= l.bad;
    pages += l.pages;
    tokens += l.fresh;
  }
  bad = __syncthreads_or(bad);
  long long end_pages = pages, end_tokens = tokens;  // of this thread's sequence
  if (one_round) {
    block_scan(end_pages, end_tokens, s_w);
    pages = s_w.w[0][32];
    tokens = s_w.w[1][32];
  } else {
    pages = block_sum(pages, s_l);
    tokens = block_sum(tokens, s_l);
  }
  // more than the outputs hold: the tables of an empty batch
  const bool none = pages > p.max_indices || tokens > p.num_tokens;
  if ((bad || none) && blockIdx.x == 0 && tid == 0) record_error(p.data_err, SITE_BUILD);
  const unsigned first = blockIdx.x * kT + tid, step = gridDim.x * kT;
  if (blockIdx.x == 0 && tid == 0) p.kv_indptr[0] = p.new_indptr[0] = 0;
  int page0 = 0, tok0 = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kT) {
    const int b = b0 + tid;
    Listed l = one_round ? l0 : listed_of(p, b);
    if (none) l = {0, 0, 0, 0, false};
    if (!one_round) {
      end_pages = l.pages;
      end_tokens = l.fresh;
      block_scan(end_pages, end_tokens, s_w);
    }
    const int page_end = none ? 0 : (int)end_pages, tok_end = none ? 0 : (int)end_tokens;
    const int n_pages = none ? 0 : (int)s_w.w[0][32], n_toks = none ? 0 : (int)s_w.w[1][32];
    s_page_end[tid] = page_end;
    s_page_first[tid] = page_end - l.pages;
    s_tok_end[tid] = tok_end;
    s_tok_first[tid] = l.len - tok_end;  // + token: its position
    s_row[tid] = l.row;
    if (blockIdx.x == 0 && b < p.batch) {
      p.kv_indptr[b + 1] = page0 + page_end;
      p.new_indptr[b + 1] = tok0 + tok_end;
      p.kv_last_page_len[b] = l.len > 0 ? ((l.len - 1) & (ps - 1)) + 1 : 0;
    }
    __syncthreads();
    auto page_of = [&](int k, int i) {
      const int page = p.block_table[(size_t)s_row[k] * p.table_stride + i];
      if (page >= 0 && page < p.num_pages) return page;
      record_error(p.data_err, SITE_BUILD);
      return -1;
    };
    for (unsigned i = first; i < (unsigned)n_pages; i += step) {
      const int k = find_end(s_page_end, (int)i);
      p.kv_indices[page0 + i] = max(0, page_of(k, (int)i - s_page_first[k]));
    }
    if (p.slot_map || p.positions) {
      for (unsigned i = first; i < (unsigned)n_toks; i += step) {
        const int k = find_end(s_tok_end, (int)i);
        const int pos = s_tok_first[k] + (int)i;
        if (p.positions) p.positions[tok0 + i] = pos;
        if (p.slot_map) {
          const long long page = page_of(k, pos >> p.log2_page);
          p.slot_map[tok0 + i] = page < 0 ? -1 : (page << p.log2_page) + (pos & (ps - 1));
        }
      }
    }
    page0 += n_pages;
    tok0 += n_toks;
    __syncthreads();
  }
  for (unsigned i = tok0 + first; i < (unsigned)p.num_tokens; i += step) {  // rows behind the last sequence
    if (p.slot_map) p.slot_map[i] = -1;
    if (p.positions) p.positions[i] = -1;
  }
}

}  // namespace

// The cluster of a resize on the current device: 16 CTAs (beyond the portable 8, so asked for
// once a device) where such a cluster fits.  205k pages in and out: 300 us with one CTA, 29
// with 8, 18 with 16.
static unsigned resize_parts() {
  static std::atomic<int> known[64];  // 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8;
  int parts = known[dev].load();
  if (parts == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kT);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool fits = cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                          cudaSuccess &&
                      cudaOccupancyMaxActiveClusters(&n, resize_kernel, &cfg) == cudaSuccess && n > 0;
    if (!fits) cudaGetLastError();  // the failed query's error is dealt with
    known[dev] = parts = fits ? 16 : 8;
  }
  return (unsigned)parts;
}

cudaError_t launch_resize_tables(const ResizeParams& p, cudaStream_t s) {
  // one CTA where no more pages could move than its threads read at once (a call that moves
  // 1024 or 4096 pages: 4.1 and 4.2 us, with the cluster 4.3 and 4.4)
  const unsigned parts = (long long)p.batch * p.max_pages <= kU * kT ? 1 : resize_parts();
  return launch_pdl(resize_kernel, dim3(parts), dim3(kT), 0, s, parts, p);
}

cudaError_t launch_build_tables(const BuildParams& p, int sms, cudaStream_t s) {
  // one entry per thread, up to one CTA per SM
  const long long most = std::max<long long>(std::max(p.max_indices, p.num_tokens), 1);
  return launch_pdl(build_kernel, dim3((unsigned)std::min<long long>((most + kT - 1) / kT, sms)), dim3(kT), 0, s, 1, p);
}

}  // namespace pa
