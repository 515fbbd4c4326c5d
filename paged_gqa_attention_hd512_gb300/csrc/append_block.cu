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
// one (block, kv head, side), loads its new rows once into registers (64 elements a thread),
// finds their largest magnitude across the group and writes the codes.
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

// Sixteen bf16 values times r, as codes.
template <int KVT, bool ANY>
__device__ __forceinline__ uint4 codes16(const uint32_t* w, float r) {
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k] = codes4<KVT, ANY>(__fmul_rn(bf16_lo(w[2 * k]), r), __fmul_rn(bf16_hi(w[2 * k]), r),
                            __fmul_rn(bf16_lo(w[2 * k + 1]), r), __fmul_rn(bf16_hi(w[2 * k + 1]), r));
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

constexpr int kRegs = 4;  // 16-element pieces of a block's new rows that a thread keeps

// A group of G threads (a power of two, at least a warp) takes the blocks whose first new row
// lies among `tokens` consecutive new rows, for one kv head and side; blockDim.x / G groups
// per CTA.  New rows beyond what the group's registers hold are read a second time.
template <int KVT>
__global__ void __launch_bounds__(512, 2) append_block_kernel(const AppendBlockParams p, const int tokens, const int G) {
  __shared__ uint32_t s_max[2][32];  // per warp, in turn: the largest magnitude
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x & (G - 1);
  const long long unit = (long long)blockIdx.x * (blockDim.x / G) + group;
  const bool is_v = unit & 1;
  const int h = (int)((unit >> 1) % p.Hkv);
  const long long i_first = (unit >> 1) / p.Hkv * tokens;
  if (i_first >= p.total_new) return;  // the whole group
  const int i_end = (int)min((long long)p.total_new, i_first + tokens);
  const int lbt = p.log2_tokens, bt = 1 << lbt, ps = p.page_size;
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
    if (b < 0) {
      // a batch of single tokens has row i in sequence i: look there first, with every load
      // that the sequence needs in flight at once
      const int g = min(i, p.batch - 1);
      const int lo = __ldg(p.append_indptr + g), hi = __ldg(p.append_indptr + g + 1);
      const int k0 = __ldg(p.kv_indptr + g), k1 = __ldg(p.kv_indptr + g + 1), last = __ldg(p.kv_last_page_len + g);
      if (lo <= i && i < hi) enter(g, lo, hi, k0, k1, last);
    }
    if (b < 0 || i >= a_end) {
      // the last sequence b with append_indptr[b] <= i, 32 candidates per round
      int lo = max(b, 0), hi = p.batch;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int c = lo + step * lane;
        const bool le = lane > 0 && c < hi && __ldg(p.append_indptr + c) <= i;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        if (m) lo += step * (31 - __clz(m));
        hi = min(hi, lo + step);
      }
      enter(lo, __ldg(p.append_indptr + lo), __ldg(p.append_indptr + lo + 1), __ldg(p.kv_indptr + lo),
            __ldg(p.kv_indptr + lo + 1), __ldg(p.kv_last_page_len + lo));
      if (i < a0 || i >= a_end) return;  // rows past the last sequence
    }
    const int t = kv_len - n_new + (i - a0);  // position in the sequence
    if (t < 0) {  // more new rows than the sequence holds
      if (tid == 0) record_error(p.err, SITE_APPEND_POS);
      i += min(-t, a_end - i);
      continue;
    }
    const int in_blk = t & (bt - 1);
    const int n = min(bt - in_blk, a_end - i);  // rows from i on that share its block
    if (i > a0 && in_blk > 0) {  // not the block's first new row
      i += n;
      continue;
    }
    const int page = __ldg(p.kv_indices + ip0 + t / ps);
    const uint16_t* src = x0 + (size_t)i * row_elems;
    const int pieces = n << lrow;
    auto load = [&](int u, uint32_t* w) {
      const uint4* q = reinterpret_cast<const uint4*>(src + (size_t)(u >> lrow) * row_elems) + 2 * (u & ((1 << lrow) - 1));
      const uint4 a = __ldg(q), c = __ldg(q + 1);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      w[4] = c.x, w[5] = c.y, w[6] = c.z, w[7] = c.w;
    };
    uint32_t w[kRegs][8];
#pragma unroll
    for (int k = 0; k < kRegs; ++k)
      if (tid + k * G < pieces) load(tid + k * G, w[k]);
    if (page < 0 || page >= p.num_pages) {
      if (tid == 0) record_error(p.err, SITE_APPEND_POS);
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

}  // namespace

cudaError_t launch_append_block(int kvt, const AppendBlockParams& p, cudaStream_t s) {
  // Short appends (a decode step's: few new rows a sequence): a warp per row, so that every row
  // starts at once.  Otherwise a block's worth of rows per group, among which about one block
  // starts, and as many threads as keep the whole block in registers.
  const bool steps = p.total_new <= 4ll * p.batch;
  const int tokens = steps ? 1 : 1 << p.log2_tokens;
  int G = 32;
  const int d = p.d_qk > p.d_vo ? p.d_qk : p.d_vo;
  while (!steps && G < 512 && G * kRegs * 16 < d << p.log2_tokens) G *= 2;
  const int threads = G > 256 ? G : 256;
  const long long units = ((long long)p.total_new + tokens - 1) / tokens * p.Hkv * 2;
  const long long grid = (units + threads / G - 1) / (threads / G);
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  if (kvt == KV_INT8B) append_block_kernel<KV_INT8B><<<(unsigned)grid, threads, 0, s>>>(p, tokens, G);
  else if (kvt == KV_FP8B) append_block_kernel<KV_FP8B><<<(unsigned)grid, threads, 0, s>>>(p, tokens, G);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace pa
