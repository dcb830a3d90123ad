// Norm of every query and key head and rotation by position, in one pass over
// the strided output of a projection: the step before tq_encode_slots (keys)
// and the attention calls (queries).
//
// Mathematics, per token at position p and head row x of length d:
//   y = x * (1 / sqrt(mean(x^2) + eps)) * w            (if weights are given)
//   theta_i = p f_i, i < rot / 2
//   (y_a, y_b) -> s (y_a cos theta_i - y_b sin theta_i, y_b cos theta_i + y_a sin theta_i)
// with (a, b) = (2i, 2i + 1) (interleaved) or (i, i + rot / 2) (half layout),
// s = rope_scale, coordinates from rot on unchanged. Everything is f32 from
// the load to one rounding to fp16 at the store; the angle is reduced to a
// fraction of a turn in f64 (p f_i / 2 pi needs more than f32's 24 bits from
// positions of a few thousand on; in f64 a position of 2^31 leaves 4e-8
// turns), and sincospif takes the fraction.
//
// Bound: 2 B read and 2 B written per coordinate; a token's d / 2 angles cost
// as much as a few of its rows and are shared by all its heads through shared
// memory. A lane holds 8 neighbouring coordinates (one 16-byte load and
// store), so a row is d / 8 lanes and a warp works on 256 / d rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tq_common.cuh"

namespace tq {

constexpr int NR_THREADS = 256;
constexpr int NR_MAX_TOKENS = 8;  // tokens of one CTA (their angles share 8 KB at d = 256)

struct NrArgs {
  const uint16_t* x[2];  // queries, keys
  uint16_t* out[2];
  const void* w[2];
  int64_t tok_stride[2], head_stride[2];  // in elements
  const int32_t* positions;
  const double* inv_freq;
  int64_t n_tok;
  int h[2];     // rows of a token: queries, keys
  int rows;     // h[0] + h[1]
  int rot, half;
  int tokens;   // tokens per CTA
  int row_step; // rows of a token handled by one CTA (gridDim.y CTAs share a token)
  int w_f32;
  float eps, scale, inv_d;
};

// Two 16-bit inputs of a word as f32.
template <bool BF>
TQ_DEV float2 nr_unpack(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF>
TQ_DEV void nr_weights(const NrArgs& a, int t, int e0, float (&w)[8]) {
  if (a.w_f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.w[t]) + e0);
    const float4 u = __ldg(p), v = __ldg(p + 1);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
  } else {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w[t]) + e0));
    const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = nr_unpack<BF>(q[i]);
      w[2 * i] = f.x, w[2 * i + 1] = f.y;
    }
  }
}

// LAYOUT 0: interleaved pairs (both in the lane); 1: half layout with rot / 2
// a multiple of 8 (the partner coordinates are another lane's 8, taken by
// shuffles of the raw 16-bit pairs and normalised again: 4 shuffles instead
// of 8); 2: half layout with any rot / 2 (through a shared f32 row).
template <int D, bool BF, int LAYOUT>
__global__ void __launch_bounds__(NR_THREADS) norm_rope_kernel(const __grid_constant__ NrArgs a) {
  constexpr int LPR = D / 8;       // lanes of a row
  constexpr int RPC = NR_THREADS / LPR;
  __shared__ __align__(16) float2 cs[NR_MAX_TOKENS * D / 2];  // (s cos, s sin) of (token, i)
  __shared__ __align__(16) float rowbuf[LAYOUT == 2 ? NR_THREADS * 8 : 4];
  const int tid = threadIdx.x, lane = tid & 31;
  const int l = lane % LPR, e0 = 8 * l;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min64(a.tokens, a.n_tok - t0);
  const int r_lo = blockIdx.y * a.row_step, r_hi = min(a.rows, r_lo + a.row_step);
  const int nr = r_hi - r_lo;      // rows of each token here
  const int items = nt * nr;

  // item -> token and row; the first item's load is issued before the angles
  auto source = [&](int item, int& tok, int& which, int& head) {
    tok = item / nr;
    const int r = r_lo + item - tok * nr;
    which = r >= a.h[0];
    head = which ? r - a.h[0] : r;
    return reinterpret_cast<const uint4*>(a.x[which] + (t0 + tok) * a.tok_stride[which] +
                                          head * a.head_stride[which] + e0);
  };
  int item = tid / LPR;
  uint4 raw = make_uint4(0, 0, 0, 0);
  int tok = 0, which = 0, head = 0;
  if (item < items) raw = *source(item, tok, which, head);

  for (int i = tid; i < nt * a.half; i += NR_THREADS) {
    const int t = i / a.half, k = i - t * a.half;
    const double turns = (double)a.positions[t0 + t] * a.inv_freq[k] * 0.15915494309189533577;
    const float frac = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * frac, &s, &c);
    cs[t * (D / 2) + k] = make_float2(c * a.scale, s * a.scale);
  }
  __syncthreads();

  // every lane of a warp runs the same number of passes (shuffles inside)
  for (int base = 0; base < items; base += RPC) {
    const bool live = item < items;
    const uint4 cur = raw;
    const int c_tok = tok, c_which = which, c_head = head;
    const int next = item + RPC;
    if (next < items) raw = *source(next, tok, which, head);

    const uint32_t in[4] = {cur.x, cur.y, cur.z, cur.w};
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = nr_unpack<BF>(in[i]);
      y[2 * i] = f.x, y[2 * i + 1] = f.y;
    }
    float rs = 1.f;
    const bool norm = a.w[c_which] != nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (norm) {
      rs = 1.0f / sqrtf(fmaf(ss, a.inv_d, a.eps));
      float w[8];
      nr_weights<BF>(a, c_which, e0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= rs * w[i];
    }
    const float2* tc = cs + c_tok * (D / 2);
    if (LAYOUT == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e0 + 2 * i < a.rot) {
          const float2 t = tc[(e0 >> 1) + i];
          const float u = y[2 * i], v = y[2 * i + 1];
          y[2 * i] = u * t.x - v * t.y;
          y[2 * i + 1] = v * t.x + u * t.y;
        }
      }
    } else if (LAYOUT == 1) {
      const bool low = e0 < a.half, in_rot = e0 < a.rot;
      const int po = in_rot ? (low ? a.half : -a.half) : 0;  // partner's offset
      const int src = (lane - l) + ((e0 + po) >> 3);
      uint32_t pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = __shfl_sync(0xffffffffu, in[i], src);
      if (in_rot) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = nr_unpack<BF>(pr[i]);
          p[2 * i] = f.x, p[2 * i + 1] = f.y;
        }
        if (norm) {
          float w[8];
          nr_weights<BF>(a, c_which, e0 + po, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] *= rs * w[i];
        }
        const float4* tq4 = reinterpret_cast<const float4*>(tc + (low ? e0 : e0 - a.half));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 t = tq4[i];  // two angles
          const float s0 = low ? -t.y : t.y, s1 = low ? -t.w : t.w;
          y[2 * i] = y[2 * i] * t.x + p[2 * i] * s0;
          y[2 * i + 1] = y[2 * i + 1] * t.z + p[2 * i + 1] * s1;
        }
      }
    } else {
      float* row = rowbuf + (tid / LPR) * D;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) row[e0 + i] = y[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        if (e < a.rot) {
          const bool low = e < a.half;
          const float2 t = tc[low ? e : e - a.half];
          const float p = row[low ? e + a.half : e - a.half];
          y[i] = y[i] * t.x + (low ? -p : p) * t.y;
        }
      }
    }
    if (live) {
      __half2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
      uint16_t* dst = a.out[c_which] + ((t0 + c_tok) * a.h[c_which] + c_head) * D + e0;
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
    }
    item = next;
  }
}

template <int D, bool BF>
static cudaError_t launch_d(const NrArgs& a, int layout, dim3 grid, cudaStream_t st) {
  if (layout == 0) norm_rope_kernel<D, BF, 0><<<grid, NR_THREADS, 0, st>>>(a);
  else if (layout == 1) norm_rope_kernel<D, BF, 1><<<grid, NR_THREADS, 0, st>>>(a);
  else norm_rope_kernel<D, BF, 2><<<grid, NR_THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace tq

using namespace tq;

tq_status tq_launch_norm_rope(const void* q, const void* k, int dtype, int64_t n_tok, int hq, int hkv, int d,
                              int64_t q_tok_stride, int64_t q_head_stride, int64_t k_tok_stride,
                              int64_t k_head_stride, const int32_t* positions, const double* inv_freq, int rot_dim,
                              int interleaved, float rope_scale, const void* q_weight, const void* k_weight,
                              int weight_f32, float eps, void* q_out, void* k_out, void* stream) {
  NrArgs a{};
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.out[0] = static_cast<uint16_t*>(q_out);
  a.out[1] = static_cast<uint16_t*>(k_out);
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.tok_stride[0] = q_tok_stride;
  a.tok_stride[1] = k_tok_stride;
  a.head_stride[0] = q_head_stride;
  a.head_stride[1] = k_head_stride;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.n_tok = n_tok;
  a.h[0] = hq;
  a.h[1] = hkv;
  a.rows = hq + hkv;
  a.rot = rot_dim;
  a.half = rot_dim / 2;
  a.w_f32 = weight_f32;
  a.eps = eps;
  a.scale = rope_scale;
  a.inv_d = 1.0f / (float)d;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
  // Tokens of few rows share a CTA until its threads hold two passes of rows;
  // while the tokens alone do not fill the SMs twice, a token's rows are
  // divided among CTAs of one pass each (every CTA redoes the token's angles).
  const int rpc = NR_THREADS / (d / 8);
  const int64_t fill = 2 * (int64_t)tq_sm_count(dev);
  a.tokens = 1;
  while (a.tokens < NR_MAX_TOKENS && a.tokens * a.rows < 2 * rpc && n_tok / (2 * a.tokens) >= fill) a.tokens *= 2;
  a.row_step = n_tok >= fill ? a.rows : rpc;
  const int64_t gx = (n_tok + a.tokens - 1) / a.tokens;
  const int64_t gy = (a.rows + a.row_step - 1) / a.row_step;
  if (gx > 0x7fffffff || gy > 65535) return TQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  const int layout = interleaved || rot_dim == 0 ? 0 : (a.half % 8 == 0 ? 1 : 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define TQ_NR_CASE(D_) \
  if (d == D_) e = dtype == TQ_BF16 ? launch_d<D_, true>(a, layout, grid, st) : launch_d<D_, false>(a, layout, grid, st);
  TQ_NR_CASE(64) TQ_NR_CASE(128) TQ_NR_CASE(256)
#undef TQ_NR_CASE
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
