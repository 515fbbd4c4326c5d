// append_block.cu -- write new tokens' K and V into a paged cache of 8-bit codes (int8 or
// e4m3) with one fp32 scale per block of tokens and kv head.
//
// A block is 2^log2_tokens consecutive slots of a page; K and V of a kv head have a scale
// each per block, and a value is code * scale.  Per touched block, kv head and side:
//   s = max(s_old, amax * c)   amax = the largest finite |x| of the block's new rows, c =
//                              RN(1/127) (int8) or RN(1/448) (e4m3), s_old = 0 when the
//                              block holds no earlier token of the sequence
//   r = min(RN(1/s), FLT_MAX)
//   code(x) = round-to-nearest-even of RN(x * r) to an integer in [-127, 127] or to e4m3
//             (saturating); 0 when s = 0; NaN gives 0 (int8) or NaN (e4m3)
// and where s > s_old the earlier tokens' codes become the code of RN(code * RN(s_old * r)).
// Every product is one correctly rounded fp32 operation, so codes and scales are a function
// of the inputs alone.
//
// Bytes: 2 read and 1 written per element, plus a scale per block.  A group of threads takes
// one (block, kv head, side): it finds its new rows' largest magnitude, then writes the codes.
// Short appends take a warp per row and head (append_step_kernel); long ones stream the rows
// through shared memory (append_stream_kernel), or, in blocks of two or four tokens, load them
// into registers (append_block_kernel).
#include <algorithm>

#include "launch.h"
#include "common.cuh"

namespace pa {

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Per half of m = two bf16 values: the magnitude bits, 0 where the value is not finite.
__device__ __forceinline__ uint32_t finite_abs2(uint32_t w) {
  const uint32_t m = w & 0x7FFF7FFFu;
  return m & __vcmpltu2(m, 0x7F807F80u);
}

// Four scaled values as four codes (the first in the low byte).  ANY: they may be infinite or
// NaN, or (int8) beyond the range; otherwise |y| is at most 127 (1 + 2^-21).
template <int KVT, bool ANY>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (KVT == KV_INT8B) {
    // 1.5 * 2^23 + y: the sum's low byte is y rounded to nearest even, in two's complement
    auto one = [](float y) {
      if (ANY) y = y == y ? fminf(fmaxf(y, -127.f), 127.f) : 0.f;
      return __float_as_uint(__fadd_rn(y, 12582912.f));
    };
    return prmt(prmt(one(a), one(b), 0x0040), prmt(one(c), one(d), 0x0040), 0x5410);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return lo | ((uint32_t)hi << 16);
  }
}

// Four bf16 values (two words) times r, as codes.
template <int KVT, bool ANY>
__device__ __forceinline__ uint32_t codes4w(uint32_t w0, uint32_t w1, float r) {
  return codes4<KVT, ANY>(__fmul_rn(bf16_lo(w0), r), __fmul_rn(bf16_hi(w0), r), __fmul_rn(bf16_lo(w1), r),
                          __fmul_rn(bf16_hi(w1), r));
}

// Sixteen bf16 values times r, as codes.
template <int KVT, bool ANY>
__device__ __forceinline__ uint4 codes16(const uint32_t* w, float r) {
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = codes4w<KVT, ANY>(w[2 * k], w[2 * k + 1], r);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Four codes times `ratio`, as codes again.
template <int KVT>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  float x[4];
  if constexpr (KVT == KV_INT8B) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = (float)(int8_t)(w >> (8 * k));
  } else {
    const uint32_t h0 = e4m3x2_to_f16x2(w & 0xFFFFu), h1 = e4m3x2_to_f16x2(w >> 16);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
    x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
  }
  return codes4<KVT, true>(__fmul_rn(x[0], ratio), __fmul_rn(x[1], ratio), __fmul_rn(x[2], ratio),
                           __fmul_rn(x[3], ratio));
}

constexpr int kStepWarps = 8;  // warps per CTA of append_step_kernel
constexpr int kRegs = 4;       // 16-element pieces of a block's new rows that a thread keeps

// Long appends in blocks of two or four tokens, fewer than a TMA box.  A group of G threads (a
// power of two, at least a warp) takes the blocks whose first new row lies among a block's
// worth of consecutive new rows, for one kv head and side; blockDim.x / G groups per CTA.
template <int KVT>
__global__ void __launch_bounds__(512, 2) append_block_kernel(const AppendBlockParams p, const int G) {
  __shared__ uint32_t s_max[2][32];  // per warp, in turn: the largest magnitude
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x & (G - 1);
  grid_dep_wait();
  grid_dep_launch();  // the next call's kernel may start its set-up (it waits for this grid)
  const long long unit = (long long)blockIdx.x * (blockDim.x / G) + group;
  const bool is_v = unit & 1;
  const int h = (int)((unit >> 1) % p.Hkv);
  const int lbt = p.log2_tokens, bt = 1 << lbt, ps = p.page_size;
  const long long i_first = (unit >> 1) / p.Hkv << lbt;
  if (i_first >= p.total_new) return;  // the whole group
  const int i_end = (int)min((long long)p.total_new, i_first + bt);
  const int d = is_v ? p.d_vo : p.d_qk;
  const int lrow = d == 512 ? 5 : 4;  // log2 of a row's 16-element pieces
  const size_t row_elems = (size_t)p.Hkv * d;
  const uint16_t* x0 = (is_v ? p.v_new : p.k_new) + (size_t)h * d;
  const size_t side_bytes = (size_t)p.Hkv * ps * p.d_qk, page_bytes = side_bytes + (size_t)p.Hkv * ps * p.d_vo;
  uint32_t turn = 0;
  int b = -1, a0 = 0, a_end = 0, n_new = 0, ip0 = 0, kv_len = 0;
  auto enter = [&](int seq, int lo, int hi, int k0, int k1, int last) {
    b = seq;
    a0 = lo;
    n_new = hi - lo;
    a_end = min(hi, p.total_new);
    ip0 = k0;
    kv_len = k1 > k0 ? (k1 - k0 - 1) * ps + last : 0;
  };
  for (int i = (int)i_first; i < i_end;) {
    if (b < 0 || i >= a_end) {
      // the last sequence b with append_indptr[b] <= i, 32 candidates per round
      int lo = max(b, 0), hi = p.batch;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int c = lo + step * lane;
        const bool le = lane > 0 && c < hi && p.append_indptr[c] <= i;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        if (m) lo += step * (31 - __clz(m));
        hi = min(hi, lo + step);
      }
      enter(lo, p.append_indptr[lo], p.append_indptr[lo + 1], p.kv_indptr[lo], p.kv_indptr[lo + 1],
            p.kv_last_page_len[lo]);
      if (i < a0 || i >= a_end) return;  // rows past the last sequence
    }
    const int t = kv_len - n_new + (i - a0);  // position in the sequence
    if (t < 0) {  // more new rows than the sequence holds
      if (tid == 0) record_error(p.data_err, SITE_APPEND_POS);
      i += min(-t, a_end - i);
      continue;
    }
    const int in_blk = t & (bt - 1);
    const int n = min(bt - in_blk, a_end - i);  // rows from i on that share its block
    if (i > a0 && in_blk > 0) {  // not the block's first new row
      i += n;
      continue;
    }
    const int page = p.kv_indices[ip0 + t / ps];
    const uint16_t* src = x0 + (size_t)i * row_elems;
    const int pieces = n << lrow;
    auto load = [&](int u, uint32_t* w) {
      const uint4* q = reinterpret_cast<const uint4*>(src + (size_t)(u >> lrow) * row_elems) + 2 * (u & ((1 << lrow) - 1));
      const uint4 a = q[0], c = q[1];
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      w[4] = c.x, w[5] = c.y, w[6] = c.z, w[7] = c.w;
    };
    uint32_t w[kRegs][8];
#pragma unroll
    for (int k = 0; k < kRegs; ++k)
      if (tid + k * G < pieces) load(tid + k * G, w[k]);
    if (page < 0 || page >= p.num_pages) {
      if (tid == 0) record_error(p.data_err, SITE_APPEND_POS);
      i += n;
      continue;
    }
    const int slot = t & (ps - 1);
    uint8_t* blk_rows = p.cache + (size_t)page * page_bytes + (is_v ? side_bytes : 0) +
                        ((size_t)h * ps + (slot - in_blk)) * d;  // the block's first slot
    float* sp = p.scales + (((size_t)page * 2 + (is_v ? 1 : 0)) * p.Hkv + h) * p.per_head + (slot >> lbt);
    const float s_old = in_blk > 0 ? *sp : 0.f;
    // the largest magnitude (bf16 bits; infinities and NaN are above every finite one)
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < kRegs; ++k)
      if (tid + k * G < pieces) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, w[k][j] & 0x7FFF7FFFu);
      }
    for (int u = tid + kRegs * G; u < pieces; u += G) {
      uint32_t v[8];
      load(u, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, v[j] & 0x7FFF7FFFu);
    }
    auto group_max = [&](uint32_t m) -> uint32_t {
      m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
      if (G == 32) return m;
      // (the slots of two turns ago: every warp has passed the barrier in between)
      uint32_t* slots = s_max[turn++ & 1] + group * (G / 32);
      if (lane == 0) slots[warp & (G / 32 - 1)] = m;
      named_bar_sync(1 + group, G);
      for (int k = 0; k < G / 32; ++k) m = max(m, slots[k]);
      return m;
    };
    uint32_t mb = group_max(m2);
    const bool any = mb >= 0x7F80u;  // infinities or NaN among the values: the finite ones' maximum
    if (any) {
      m2 = 0;
      for (int u = tid; u < pieces; u += G) {
        uint32_t v[8];
        load(u, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, finite_abs2(v[j]));
      }
      mb = group_max(m2);
    }
    const float amax = __uint_as_float(mb << 16);
    const float s = fmaxf(s_old, __fmul_rn(amax, KVT == KV_INT8B ? 1.f / 127.f : 1.f / 448.f));
    const float r = s > 0.f ? fminf(__frcp_rn(s), 3.402823466e38f) : 0.f;
    if (in_blk > 0 && s > s_old) {
      const float ratio = __fmul_rn(s_old, r);
      for (int u = tid; u < in_blk << lrow; u += G) {
        uint4* q = reinterpret_cast<uint4*>(blk_rows) + u;
        const uint4 c = *q;
        *q = make_uint4(recode4<KVT>(c.x, ratio), recode4<KVT>(c.y, ratio), recode4<KVT>(c.z, ratio),
                        recode4<KVT>(c.w, ratio));
      }
    }
    // (written after every thread of the group has read s_old: the maximum's exchange)
    if (tid == 0) *sp = s;
    uint4* dst = reinterpret_cast<uint4*>(blk_rows + (size_t)in_blk * d);
    if (any || s == 0.f) {
      for (int u = tid; u < pieces; u += G) {
        uint32_t v[8];
        load(u, v);
        dst[u] = s == 0.f ? make_uint4(0, 0, 0, 0) : codes16<KVT, true>(v, r);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kRegs; ++k)
        if (tid + k * G < pieces) dst[tid + k * G] = codes16<KVT, false>(w[k], r);
      for (int u = tid + kRegs * G; u < pieces; u += G) {
        uint32_t v[8];
        load(u, v);
        dst[u] = codes16<KVT, false>(v, r);
      }
    }
    i += n;
  }
}

// ---------------------------------------------------------------------------------------
// Short appends (a decode step's, few new rows a sequence) and blocks of one token: a warp per
// (new row, kv head), K and V together.  What takes time is the chain of dependent loads, so
// the row's values are loaded at once, beside the guess that row i belongs to sequence i; then
// the page id, then the old scales.  A warp whose row is not its block's first new one leaves;
// one whose block has more new rows reads those too.
template <int KVT>
__global__ void __launch_bounds__(32 * kStepWarps, 4) append_step_kernel(const AppendBlockParams p) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kStepWarps + (threadIdx.x >> 5);
  grid_dep_wait();
  grid_dep_launch();  // the next call's kernel may start its set-up (it waits for this grid)
  const int h = (int)(unit % p.Hkv);
  if (unit / p.Hkv >= p.total_new) return;
  const int i = (int)(unit / p.Hkv);
  const int lbt = p.log2_tokens, bt = 1 << lbt, ps = p.page_size;
  // 8-element pieces lane and lane + 32 (512 elements) of row r of a side
  auto load_row = [&](int side, int r, uint4* w) {
    const int d = side ? p.d_vo : p.d_qk;
    const uint4* src = reinterpret_cast<const uint4*>((side ? p.v_new : p.k_new) + ((size_t)r * p.Hkv + h) * d);
    w[0] = src[lane];
    w[1] = d == 512 ? src[lane + 32] : make_uint4(0, 0, 0, 0);
  };
  uint4 w[2][2];
  load_row(0, i, w[0]);
  load_row(1, i, w[1]);
  int b = min(i, p.batch - 1);
  int a0 = p.append_indptr[b], a_end = p.append_indptr[b + 1];
  int ip0 = p.kv_indptr[b], ip1 = p.kv_indptr[b + 1], last = p.kv_last_page_len[b];
  if (i < a0 || i >= a_end) {
    // the last sequence b with append_indptr[b] <= i, 32 candidates per round
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int c = lo + step * lane;
      const bool le = lane > 0 && c < hi && p.append_indptr[c] <= i;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      if (m) lo += step * (31 - __clz(m));
      hi = min(hi, lo + step);
    }
    b = lo;
    a0 = p.append_indptr[b];
    a_end = p.append_indptr[b + 1];
    ip0 = p.kv_indptr[b];
    ip1 = p.kv_indptr[b + 1];
    last = p.kv_last_page_len[b];
    if (i < a0 || i >= a_end) return;  // rows past the last sequence
  }
  const int kv_len = ip1 > ip0 ? (ip1 - ip0 - 1) * ps + last : 0;
  const int t = kv_len - (a_end - a0) + (i - a0);  // position in the sequence
  if (t < 0) {                                     // more new rows than the sequence holds
    if (lane == 0) record_error(p.data_err, SITE_APPEND_POS);
    return;
  }
  const int in_blk = t & (bt - 1), slot = t & (ps - 1);
  if (i > a0 && in_blk > 0) return;  // not the block's first new row
  const int n = min(bt - in_blk, min(a_end, p.total_new) - i);
  const int page = p.kv_indices[ip0 + t / ps];
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_error(p.data_err, SITE_APPEND_POS);
    return;
  }
  float* sp = p.scales + ((size_t)page * 2 * p.Hkv + h) * p.per_head + (slot >> lbt);
  const size_t v_scales = (size_t)p.Hkv * p.per_head;
  float s_old[2] = {0.f, 0.f};
  if (in_blk > 0) {
    s_old[0] = sp[0];
    s_old[1] = sp[v_scales];
  }
  auto max8 = [](uint4 v) {
    return __vmaxu2(__vmaxu2(finite_abs2(v.x), finite_abs2(v.y)), __vmaxu2(finite_abs2(v.z), finite_abs2(v.w)));
  };
  const size_t side_bytes = (size_t)p.Hkv * ps * p.d_qk, page_bytes = side_bytes + (size_t)p.Hkv * ps * p.d_vo;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int d = side ? p.d_vo : p.d_qk;
    uint32_t m2 = __vmaxu2(max8(w[side][0]), max8(w[side][1]));
    for (int r = 1; r < n; ++r) {
      uint4 x[2];
      load_row(side, i + r, x);
      m2 = __vmaxu2(m2, __vmaxu2(max8(x[0]), max8(x[1])));
    }
    const uint32_t mb = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
    const float s = fmaxf(s_old[side], __fmul_rn(__uint_as_float(mb << 16), KVT == KV_INT8B ? 1.f / 127.f : 1.f / 448.f));
    const float r0 = s > 0.f ? fminf(__frcp_rn(s), 3.402823466e38f) : 0.f;
    uint8_t* rows = p.cache + (size_t)page * page_bytes + (side ? side_bytes : 0) + ((size_t)h * ps + (slot - in_blk)) * d;
    if (in_blk > 0 && s > s_old[side]) {
      const float ratio = __fmul_rn(s_old[side], r0);
      for (int u = lane; u < in_blk * (d / 16); u += 32) {
        uint4* q = reinterpret_cast<uint4*>(rows) + u;
        const uint4 c = *q;
        *q = make_uint4(recode4<KVT>(c.x, ratio), recode4<KVT>(c.y, ratio), recode4<KVT>(c.z, ratio),
                        recode4<KVT>(c.w, ratio));
      }
    }
    if (lane == 0) sp[side * v_scales] = s;  // (every lane has read s_old: the maximum's exchange)
    for (int r = 0; r < n; ++r) {
      uint4 x[2] = {w[side][0], w[side][1]};
      if (r > 0) load_row(side, i + r, x);
      uint2* dst = reinterpret_cast<uint2*>(rows + (size_t)(in_blk + r) * d) + lane;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (k == 0 || d == 512)
          dst[32 * k] = s > 0.f ? make_uint2(codes4w<KVT, true>(x[k].x, x[k].y, r0), codes4w<KVT, true>(x[k].z, x[k].w, r0))
                                : make_uint2(0, 0);
    }
  }
}

// ---------------------------------------------------------------------------------------
// Long appends: persistent CTAs; producer warps stream the blocks' new rows into a ring of
// shared-memory stages (one TMA box a block; a copy per row took the producer 84 cycles each,
// 5400 for a block of 64), and kConsumers consumers in groups of G take a stage each, one
// (block, kv head, side): a pass over it for the largest magnitude, one for the codes.  Several
// groups work on different stages while the others load, which the register kernel above, two
// CTAs an SM, does not reach: 33 thousand rows of 4 x (512 + 512) int8 91 -> 73 us (5.5 TB/s),
// 64 thousand rows of 2 x (512 + 256) e4m3 in blocks of 16 69 -> 51 us (5.8 TB/s).  Groups that
// keep their rows in registers between the passes, and so are fewer, took 83 us.
constexpr int kConsumers = 768;
constexpr int kBoxRows = 8;
constexpr int kStreamElems = 128;  // of a consumer thread: G threads take a whole block
// Stage n belongs to group n % groups, and the ring's length is the number of groups, so that a
// slot always serves the same group, which is at most one phase away from its barriers (a
// parity wait cannot tell more apart).  For the same reason a slot is always filled by the same
// producer warp: every producer walks the blocks, and fills those of its slots.  (One producer
// took about 1100 cycles a stage, more than a small block's bytes take.)
constexpr int kMaxStages = kConsumers / 32;
constexpr int kProducers = 4;  // warps

struct StreamBlock {
  int page, slot, rows, hs;  // rows 0: the end; hs: 2 * kv head + side
};

template <int KVT>
__global__ void __launch_bounds__(kConsumers + 32 * kProducers, 1)
    append_stream_kernel(const __grid_constant__ AppendBlockMaps tm, const AppendBlockParams p, const int G,
                         const int stages, const int stage_bytes, const long long units) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint32_t s_max[2][kConsumers / 32];
  __shared__ StreamBlock s_blk[kMaxStages];
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = kConsumers / G;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], G / 32);
    }
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  const int lbt = p.log2_tokens, bt = 1 << lbt, ps = p.page_size, HS = 2 * p.Hkv;
  const size_t side_bytes = (size_t)p.Hkv * ps * p.d_qk, page_bytes = side_bytes + (size_t)p.Hkv * ps * p.d_vo;

  if (warp >= kConsumers / 32) {
    // ------------------------------------------------------------------ producers
    const int me = warp - kConsumers / 32;
    // unit u: the blocks whose first new row lies in rows [u / HS * bt, (u / HS + 1) * bt), for
    // head and side u % HS; this CTA has a run of consecutive units
    const long long u_begin = units * blockIdx.x / gridDim.x, u_end = units * (blockIdx.x + 1) / gridDim.x;
    int s = 0;           // the next stage, and the phase of its slot
    uint32_t phase = 0;
    int b = -1, a0 = 0, a_end = 0, n_new = 0, ip0 = 0, kv_len = 0;
    auto put = [&](int page, int slot, int rows, int hs, int i) -> bool {
      const int slot_s = s;
      const uint32_t parity = phase ^ 1;
      if (++s == stages) {
        s = 0;
        phase ^= 1;
      }
      if (slot_s % kProducers != me) return true;
      if (!__all_sync(0xffffffffu, mbar_wait(&s_empty[slot_s], parity, p.err, SITE_APPEND_RING))) {
        // (not in the first phase, whose slots are empty) no copy of this warp may still be on
        // its way when the CTA ends: those of this phase before slot_s, of the last from it on
        for (int k = me; k < stages; k += kProducers) mbar_wait(&s_full[k], k < slot_s ? parity ^ 1 : parity, nullptr, 0);
        return false;
      }
      const bool is_v = hs & 1;
      uint64_t* full = &s_full[slot_s];
      const uint32_t dst = smem_u32(ring) + slot_s * stage_bytes;
      // a whole block in one box; others in boxes of kBoxRows rows, up to kBoxRows - 1 of them
      // not the block's (0 past the last row)
      const bool whole = rows == bt;
      const uint32_t row_bytes = 2u * (is_v ? p.d_vo : p.d_qk), boxes = (rows + kBoxRows - 1) / kBoxRows;
      if (lane == 0) {
        s_blk[slot_s] = {page, slot, rows, hs};
        if (rows > 0) mbar_arrive_expect_tx(full, boxes * kBoxRows * row_bytes);
        else mbar_arrive(full);
        if (whole) tma_load_4d(dst, &tm.block[is_v], 0, 0, hs >> 1, i, full);
      }
      if (!whole) {
        __syncwarp();
        if (lane < boxes)
          tma_load_4d(dst + lane * kBoxRows * row_bytes, &tm.rows[is_v], 0, 0, hs >> 1, i + lane * kBoxRows, full);
      }
      return true;
    };
    int q0 = 0, my_page = -1;  // pages of the sequence's blocks q0 + lane
    bool more = true;
    for (long long c = u_begin / HS; more && c * HS < u_end; ++c) {
      const int hs0 = (int)max(0ll, u_begin - c * HS), hs1 = (int)min((long long)HS, u_end - c * HS);
      const int i_end = (int)min((long long)p.total_new, (c + 1) * bt);
      for (int i = (int)(c * bt); i < i_end;) {
        if (b < 0 || i >= a_end) {
          // the last sequence b with append_indptr[b] <= i, 32 candidates per round
          int lo = max(b, 0), hi = p.batch;
          while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int k = lo + step * lane;
            const bool le = lane > 0 && k < hi && p.append_indptr[k] <= i;
            const unsigned m = __ballot_sync(0xffffffffu, le);
            if (m) lo += step * (31 - __clz(m));
            hi = min(hi, lo + step);
          }
          b = lo;
          a0 = p.append_indptr[b];
          a_end = p.append_indptr[b + 1];
          n_new = a_end - a0;
          a_end = min(a_end, p.total_new);
          if (i < a0 || i >= a_end) {  // rows past the last sequence
            more = false;
            break;
          }
          ip0 = p.kv_indptr[b];
          const int np = p.kv_indptr[b + 1] - ip0;
          kv_len = np > 0 ? (np - 1) * ps + p.kv_last_page_len[b] : 0;
          q0 = -32;
        }
        const int t = kv_len - n_new + (i - a0);  // position in the sequence
        if (t < 0) {  // more new rows than the sequence holds
          if (lane == 0) record_error(p.data_err, SITE_APPEND_POS);
          i += min(-t, a_end - i);
          continue;
        }
        const int in_blk = t & (bt - 1);
        const int rows = min(bt - in_blk, a_end - i);  // rows from i on that share its block
        if (i == a0 || in_blk == 0) {                  // the block's first new row
          const int q = t >> lbt;
          if (q - q0 >= 32) {
            q0 = q;
            const long long first = (long long)(q + lane) << lbt;
            my_page = first < kv_len ? p.kv_indices[ip0 + (int)first / ps] : -1;
          }
          const int page = __shfl_sync(0xffffffffu, my_page, q - q0);
          if (page < 0 || page >= p.num_pages) {
            if (lane == 0) record_error(p.data_err, SITE_APPEND_POS);
          } else {
            for (int hs = hs0; hs < hs1; ++hs)
              if (!put(page, t & (ps - 1), rows, hs, i)) return;
          }
        }
        i += rows;
      }
    }
    for (int k = 0; k < groups; ++k)  // the end, once for each group
      if (!put(0, 0, 0, 0, 0)) return;
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int group = threadIdx.x / G, tid = threadIdx.x & (G - 1);
  uint32_t turn = 0;
  for (uint32_t n = group;; n += groups) {
    const int s = n % stages;
    // (a wait that gives up leaves the error word set, and every other wait gives up at once)
    if (!mbar_wait(&s_full[s], (n / stages) & 1, p.err, SITE_APPEND_RING)) return;
    const StreamBlock blk = s_blk[s];
    if (blk.rows == 0) return;
    const bool is_v = blk.hs & 1;
    const int h = blk.hs >> 1, d = is_v ? p.d_vo : p.d_qk;
    const int pieces = blk.rows * (d / 8), in_blk = blk.slot & (bt - 1);
    float* sp = p.scales + (((size_t)blk.page * 2 + (is_v ? 1 : 0)) * p.Hkv + h) * p.per_head + (blk.slot >> lbt);
    const float s_old = in_blk > 0 ? *sp : 0.f;
    const uint4* src = reinterpret_cast<const uint4*>(ring + (size_t)s * stage_bytes);
    // f(u, piece u) for this thread's 8-element pieces, eight reads in flight
    auto each = [&](auto f) {
#pragma unroll 1
      for (int u0 = tid; u0 < pieces; u0 += 8 * G) {
        uint4 v[8];
        if (u0 + 7 * G < pieces) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = src[u0 + k * G];
#pragma unroll
          for (int k = 0; k < 8; ++k) f(u0 + k * G, v[k]);
        } else {
#pragma unroll 1
          for (int u = u0; u < pieces; u += G) f(u, src[u]);
        }
      }
    };
    // the largest magnitude (bf16 bits; infinities and NaN are above every finite one)
    uint32_t m2 = 0;
    each([&](int, uint4 v) {
      m2 = __vmaxu2(__vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                             __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)), m2);
    });
    auto group_max = [&](uint32_t m) -> uint32_t {
      m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
      if (G == 32) return m;
      // (the slots of two turns ago: every warp has passed the barrier in between)
      uint32_t* slots = s_max[turn++ & 1] + group * (G / 32);
      if (lane == 0) slots[warp & (G / 32 - 1)] = m;
      named_bar_sync(1 + group, G);
      for (int k = 0; k < G / 32; ++k) m = max(m, slots[k]);
      return m;
    };
    uint32_t mb = group_max(m2);
    const bool any = mb >= 0x7F80u;
    if (any) {  // infinities or NaN: the finite values' maximum
      m2 = 0;
      for (int u = tid; u < pieces; u += G) {
        const uint4 v = src[u];
        m2 = __vmaxu2(__vmaxu2(__vmaxu2(finite_abs2(v.x), finite_abs2(v.y)),
                               __vmaxu2(finite_abs2(v.z), finite_abs2(v.w))), m2);
      }
      mb = group_max(m2);
    }
    const float sc = fmaxf(s_old, __fmul_rn(__uint_as_float(mb << 16), KVT == KV_INT8B ? 1.f / 127.f : 1.f / 448.f));
    const float r = sc > 0.f ? fminf(__frcp_rn(sc), 3.402823466e38f) : 0.f;
    uint8_t* blk_rows = p.cache + (size_t)blk.page * page_bytes + (is_v ? side_bytes : 0) +
                        ((size_t)h * ps + (blk.slot - in_blk)) * d;  // the block's first slot
    if (in_blk > 0 && sc > s_old) {
      const float ratio = __fmul_rn(s_old, r);
      for (int u = tid; u < in_blk * (d / 16); u += G) {
        uint4* q = reinterpret_cast<uint4*>(blk_rows) + u;
        const uint4 c = *q;
        *q = make_uint4(recode4<KVT>(c.x, ratio), recode4<KVT>(c.y, ratio), recode4<KVT>(c.z, ratio),
                        recode4<KVT>(c.w, ratio));
      }
    }
    // (with G = 32 every lane has read s_old at the maximum's reduction, else at its barrier)
    if (tid == 0) *sp = sc;
    uint2* dst = reinterpret_cast<uint2*>(blk_rows + (size_t)in_blk * d);
    if (any || sc == 0.f) {
      for (int u = tid; u < pieces; u += G) {
        const uint4 v = src[u];
        dst[u] = sc > 0.f ? make_uint2(codes4w<KVT, true>(v.x, v.y, r), codes4w<KVT, true>(v.z, v.w, r))
                          : make_uint2(0, 0);
      }
    } else {
      each([&](int u, uint4 v) { dst[u] = make_uint2(codes4w<KVT, false>(v.x, v.y, r), codes4w<KVT, false>(v.z, v.w, r)); });
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s_empty[s]);
  }
}

// Few new rows a sequence (a decode step's append).  In microseconds, a warp per row and head /
// the long forms, new rows a sequence 1, 4, 8, 16: 64 sequences of 4 x (512 + 512) in blocks of
// 16 2.9 / 18.1, 5.8 / 7.4, 10.6 / 7.8, 14.3 / 7.2; 256 of 1 x (256 + 256) in blocks of 64
// 2.7 / 63.7, 6.0 / 18.7, 7.8 / 11.3, 13.3 / 7.8; 64 of 4 x (512 + 512) in blocks of 4
// 2.9 / 8.7, 6.0 / 3.9, 6.6 / 3.9 (1 and 2 rows, which leave a block unfinished: 4.1 / 5.8).
bool append_block_steps(int total_new, int batch) { return total_new <= 4ll * batch; }

}  // namespace

bool append_block_streams(int total_new, int batch, int block_tokens) {
  return !append_block_steps(total_new, batch) && block_tokens >= kBoxRows;
}
int append_block_box_rows() { return kBoxRows; }

template <int KVT>
static cudaError_t run_append(const AppendBlockMaps& tm, const AppendBlockParams& p, int sms, cudaStream_t s) {
  const int bt = 1 << p.log2_tokens, d = std::max(p.d_qk, p.d_vo);
  // (Blocks of one token too: 19 thousand rows of 4 x (256 + 256) 47 us in groups, 27 us in
  // warps; blocks of four, 84 rows for each of 88 sequences, 18 and 30 us.)
  if (append_block_steps(p.total_new, p.batch) || bt == 1) {
    const long long grid = ((long long)p.total_new * p.Hkv + kStepWarps - 1) / kStepWarps;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_pdl(append_step_kernel<KVT>, dim3((unsigned)grid), dim3(32 * kStepWarps), 0, s, 1, p);
  }
  // A block's worth of rows per group of threads, among which about one block starts.
  int G = 32;
  const long long units = ((long long)p.total_new + bt - 1) / bt * p.Hkv * 2;
  // Streamed where a block is at least a box (8 tokens): G from 32 (8 x 256) to 256
  // threads (64 x 512)
  if (append_block_streams(p.total_new, p.batch, bt)) {
    while (G * kStreamElems < d * bt) G *= 2;
    const int stage = bt * d * 2, stages = kConsumers / G;
    auto kern = append_stream_kernel<KVT>;
    static std::atomic<uint64_t> smem_set;
    const cudaError_t e = set_smem_limit_once(kern, kConsumers * kStreamElems * 2, smem_set);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)std::min<long long>(units, sms)), dim3(kConsumers + 32 * kProducers),
                      stages * stage, s, 1, tm, p, G, stages, stage, units);
  }
  while (G * 16 * kRegs < d * bt) G *= 2;  // the whole block in registers
  const int threads = G > 256 ? G : 256;
  const long long grid = (units + threads / G - 1) / (threads / G);
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_pdl(append_block_kernel<KVT>, dim3((unsigned)grid), dim3(threads), 0, s, 1, p, G);
}

cudaError_t launch_append_block(int kvt, const AppendBlockMaps& tm, const AppendBlockParams& p, int sms,
                                cudaStream_t s) {
  if (kvt == KV_INT8B) return run_append<KV_INT8B>(tm, p, sms, s);
  if (kvt == KV_FP8B) return run_append<KV_FP8B>(tm, p, sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace pa
