// Definitions shared by the kernels of windowed attention over packed caches
// (tq_attend_window.cu: few query rows per kv head, on mma.sync;
// tq_attend_window_tc.cu: many, on tcgen05) and their merge kernel: the launch
// arguments, the rules for query rows and visible positions, and small helpers.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "tq_attend.cuh"

namespace tq {

struct AwArgs {
  uint32_t k_sign_h2[TQ_MAX_D / 2];
  uint32_t v_sign_h2[TQ_MAX_D / 2];
  uint16_t k_lev[TQ_MAX_L];  // fp16 bits of lev_scale * level (tq_ctx::lev_f16)
  uint16_t v_lev[TQ_MAX_L];
  float q_scale;             // log2(e) / (d sqrt(d) K lev_scale)
  float o_scale;             // 1 / (d V lev_scale)
  const __half* q;           // [n_tok, hq, d]
  __half* out;
  const int32_t* q_offsets;  // [B + 1], or null: one token per sequence
  const uint8_t* k_packed;
  const float* k_norms;
  const uint8_t* v_packed;
  const float* v_norms;
  const int32_t* block_tables;  // null: contiguous caches of s_max rows
  const int32_t* ctx_lens;
  int64_t s_max, num_blocks;
  int64_t n_tok;
  int max_blocks;
  int B, max_q, hq, hkv, g;
  int window, sinks;  // window: INT_MAX for none
  int n_split;
  int halves;     // tcgen05 kernel: a CTA's two row tiles hold the same rows, two splits
  float* ws_m;    // [n_tok * hq, n_split] running max (log2 domain)
  float* ws_l;    // [n_tok * hq, n_split] sum of weights
  float* ws_acc;  // [n_tok * hq, n_split, D] rotated accumulator
  uint32_t* err;
};

// The sequence's first query token, its number of query tokens (0: nothing to
// do) and its context length. Offsets that leave [0, n_tok], decrease or
// exceed max_q are flagged and the sequence is left out.
struct AwSeq {
  int64_t q0;
  int n, ctx;
};
TQ_DEV AwSeq aw_sequence(const AwArgs& a, int b, bool report) {
  AwSeq s;
  if (a.q_offsets) {
    const int64_t lo = a.q_offsets[b], hi = a.q_offsets[b + 1];
    s.q0 = lo;
    s.n = (int)(hi - lo);
    if (lo < 0 || hi < lo || hi > a.n_tok || hi - lo > a.max_q) {
      if (report) record_error(a.err, TQ_DEVERR_ROW_RANGE);
      s.n = 0;
    }
  } else {
    s.q0 = b;
    s.n = 1;
  }
  int64_t ctx = a.ctx_lens[b];
  if (ctx > a.s_max) {
    if (report) record_error(a.err, TQ_DEVERR_POS_RANGE);
    ctx = a.s_max;
  }
  s.ctx = (int)(ctx < 0 ? 0 : ctx);
  return s;
}

// Query token i of a sequence stands at position ctx - n + i (below 0: the row
// sees nothing) and sees position t when t <= p and (t < sinks or
// t > p - window).
TQ_DEV int aw_position(const AwSeq& s, int i) { return max(s.ctx - s.n + i, -1); }
TQ_DEV bool aw_visible(int t, int p, int window, int sinks) { return t <= p && (t < sinks || t > p - window); }
// Whether one of the queries at positions p_lo..p_hi sees position t.
TQ_DEV bool aw_seen(int t, int p_lo, int p_hi, int window, int sinks) {
  return t <= p_hi && (t < sinks || t > p_lo - window);
}

// The 16-position blocks that queries at positions p_lo..p_hi see together:
// the sinks' blocks [0, n_sink), then the window's from w0 on; n in all.
struct AwBlocks {
  int n_sink, w0, n;
};
TQ_DEV AwBlocks aw_blocks(int p_lo, int p_hi, int window, int sinks) {
  AwBlocks r;
  if (p_hi < 0) {
    r.n_sink = r.w0 = r.n = 0;
    return r;
  }
  const int lo = max(max(p_lo, 0) - window + 1, 0);  // first position of the window
  const int last = p_hi / ATT_BLOCK;
  r.w0 = lo / ATT_BLOCK;
  r.n_sink = sinks > 0 ? min(min((sinks - 1) / ATT_BLOCK, last) + 1, r.w0) : 0;
  r.n = r.n_sink + (last - r.w0 + 1);
  return r;
}
TQ_DEV int aw_block(const AwBlocks& r, int m) { return m < r.n_sink ? m : r.w0 + (m - r.n_sink); }

// Cache row (all kv heads) of the first position of block j of sequence b, in
// two steps so that the table entry can be loaded ahead of its use: the entry
// (j itself in contiguous caches) and its row.
TQ_DEV int aw_block_entry(const AwArgs& a, int b, int j) {
  return a.block_tables == nullptr ? j : __ldg(a.block_tables + (int64_t)b * a.max_blocks + j);
}
TQ_DEV int64_t aw_entry_row(const AwArgs& a, int b, int entry) {
  if (a.block_tables == nullptr) return (int64_t)b * a.s_max + (int64_t)entry * ATT_BLOCK;
  int64_t page = entry;
  if (page < 0 || page >= a.num_blocks) {
    record_error(a.err, TQ_DEVERR_BLOCK_RANGE);
    page = page < 0 ? 0 : a.num_blocks - 1;
  }
  return page * ATT_BLOCK;
}

TQ_DEV float aw_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Power of two that brings a positive magnitude into [2^TO, 2^(TO + 1)) and
// its inverse (1 for 0, infinities and NaN).
template <int TO>
TQ_DEV float aw_pow2_for(float mag, float& inv) {
  const int e = (int)((__float_as_uint(mag) >> 23) & 255u);  // biased exponent
  if (e == 0 || e == 255) {
    inv = 1.f;
    return 1.f;
  }
  const int up = min(max(TO - (e - 127), -126), 126);
  inv = __uint_as_float((uint32_t)(127 - up) << 23);
  return __uint_as_float((uint32_t)(127 + up) << 23);
}

// The reference that a row's weights w_t = 2^(s_t - ref) refer to is free: the
// row's sum and accumulator share it. It is the row's largest score, unless the
// largest weight x value norm (times the tile's power of two, below 64) would
// then lie below AW_SMALL, where its fp16 remainder (a multiple of 2^-24) runs
// out of bits: norms that this row does not see, or positions that it gives no
// weight, may be larger by any factor. Then the reference is lowered until that
// product lies in [2^2, 2^3), or the row's sum of weights near 2^AW_SUM (so that
// norms 2^90 apart are covered over 2^24 positions of one weight). (With 2
// for AW_SMALL and [2^5, 2^6), 2 x 2048 tokens whose norms spread by e^1 took
// 1018 us, with these 734, both before tw_largest took logarithms.)
constexpr float AW_SMALL = 0.25f;
constexpr int AW_SUM = 110;
// Reference for a row whose scores have reached `top`, at which its sum is `sum`
// and its largest weight x norm `most`, which becomes the one at the result.
TQ_DEV float aw_reference(float top, float sum, float& most) {
  if (most >= AW_SMALL || !(most > 0.f)) return top;
  const int e = (int)(__float_as_uint(most) >> 23) - 127, e_sum = (int)(__float_as_uint(sum) >> 23) - 127;
  const int low = max(min(2 - e, AW_SUM - max(e_sum, 0)), 0);
  most *= __uint_as_float((uint32_t)(127 + low) << 23);
  return top - (float)low;
}

// NBYTES bytes from byte `off` of a cache row as a little-endian word stream;
// reads stay inside the row (rows are 8-byte aligned multiples of 8 bytes).
template <int NBYTES, int NW>
TQ_DEV void aw_load(uint32_t (&w)[NW], const uint8_t* row, int off, int row_bytes) {
  static_assert(NW == (NBYTES + 3) / 4, "words of the stream");
  if constexpr (NBYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < NBYTES / 16; ++i) {
      const uint4 r = __ldg(reinterpret_cast<const uint4*>(row + off) + i);
      w[4 * i] = r.x, w[4 * i + 1] = r.y, w[4 * i + 2] = r.z, w[4 * i + 3] = r.w;
    }
  } else if constexpr (NBYTES % 8 == 0) {
#pragma unroll
    for (int i = 0; i < NBYTES / 8; ++i) {
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(row + off) + i);
      w[2 * i] = r.x, w[2 * i + 1] = r.y;
    }
  } else if constexpr (NBYTES % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NBYTES / 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + off) + i);
  } else if constexpr (NBYTES == 2) {
    w[0] = __ldg(reinterpret_cast<const uint16_t*>(row + off));
  } else {  // 3 or 6 bytes: two aligned words
    const int base = off & ~3;
    const uint32_t r0 = __ldg(reinterpret_cast<const uint32_t*>(row + base));
    const uint32_t r1 = __ldg(reinterpret_cast<const uint32_t*>(row + min(base + 4, row_bytes - 4)));
    const uint32_t sh = (uint32_t)(off & 3) * 8u;
    w[0] = __funnelshift_r(r0, r1, sh);
    if constexpr (NW > 1) w[1] = r1 >> sh;
  }
}

// `NB` bits at bit `off` of a word stream (compile-time offsets).
template <int NB, int N>
TQ_DEV uint32_t aw_bits(const uint32_t (&w)[N], int off) {
  uint32_t f = w[off >> 5] >> (off & 31);
  if ((off & 31) + NB > 32 && (off >> 5) + 1 < N) f |= w[(off >> 5) + 1] << (32 - (off & 31));
  return f & ((1u << NB) - 1u);
}

// Let `kernel` use `bytes` of dynamic shared memory, once per device (`done`:
// a bit per device, one word per kernel instance).
inline cudaError_t aw_allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace tq

// The kernel for many query rows per kv head (tq_attend_window_tc.cu): rows of
// a CTA, and its launch.
int tq_window_tc_rows(int d);
cudaError_t tq_launch_window_tc(const tq::AwArgs& a, int d, int k_bits, int v_bits, cudaStream_t st);

// Merge of the splits (tq_attend_window.cu).
cudaError_t tq_launch_window_combine(const tq::AwArgs& a, int d, cudaStream_t st);
