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
// Bound: 2 B read and 2 B written per coordinate. Measured, 8191 tokens of 40
// heads of 128 bf16 coordinates with norm and 64 of them rotated (168 MB):
// 36.7 us, 4.6 TB/s (25.5 us at a plain copy's rate); the schedulers issue 78 %
// of their slots, about 154 warp instructions per pass (two rows of 128), so
// instructions are the bound there. 16 tokens take 4.2 us, a launch's latency
// and the chain position -> angle -> row.
//
// A CTA takes the rows of
// up to 8 tokens, all queries or all keys: its threads first make the tokens'
// angles (one or two each, (s cos, s sin) in shared memory), then pass over the
// rows together, each stepping its own pointers. A lane holds 8 neighbouring
// coordinates (one 16-byte load and store), so a row is d / 8 lanes. Weights
// stay in registers; the angles of a lane lie in planes of 16 bytes per lane
// (no bank conflicts).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

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
  int h[2];      // rows of a token: queries, keys
  int rot, half;
  int tokens;    // tokens per CTA
  int row_step;  // rows of a token handled by one CTA
  int q_ctas;    // CTAs (in y) that share a token's queries; the others its keys
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

// Place of angle i of a token: lanes read PER consecutive angles each, two at
// a time (16 bytes), from planes in which neighbouring lanes are neighbours.
template <int D, int PER>
TQ_DEV int nr_place(int i) {
  if (PER == 1) return i;
  constexpr int LANES = D / 2 / PER;
  return ((i % PER) / 2) * (2 * LANES) + (i / PER) * 2 + (i & 1);
}

// LAYOUT 0: interleaved pairs (both in the lane); 1: half layout with rot / 2
// a multiple of 8 (the partner coordinates are another lane's 8, taken by
// shuffles of the raw 16-bit pairs and normalised again: 4 shuffles instead
// of 8); 2: half layout with any rot / 2 (through a shared f32 row).
template <int D, bool BF, int LAYOUT>
__global__ void __launch_bounds__(NR_THREADS) norm_rope_kernel(const __grid_constant__ NrArgs a) {
  constexpr int LPR = D / 8;       // lanes of a row
  constexpr int RPC = NR_THREADS / LPR;
  constexpr int PER = LAYOUT == 0 ? 4 : LAYOUT == 1 ? 8 : 1;  // angles of a lane
  __shared__ __align__(16) float2 cs[NR_MAX_TOKENS * D / 2];  // (s cos, s sin) of (token, i)
  __shared__ __align__(16) float rowbuf[LAYOUT == 2 ? NR_THREADS * 8 : 4];
  const int tid = threadIdx.x, lane = tid & 31;
  const int l = lane % LPR, e0 = 8 * l;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min64(a.tokens, a.n_tok - t0);
  const int which = (int)blockIdx.y >= a.q_ctas;
  const int h0 = ((int)blockIdx.y - (which ? a.q_ctas : 0)) * a.row_step;  // first head here
  const int nr = min(a.h[which], h0 + a.row_step) - h0;                      // rows of a token here
  const int passes = (nt * nr + RPC - 1) / RPC;
  const int64_t ts = a.tok_stride[which], hs = a.head_stride[which];

  // this thread's row: token `tok`, row `r` of its rows here; a pass moves it
  // RPC rows on
  const int first = tid / LPR, step_tok = RPC / nr, step_r = RPC - step_tok * nr;
  int tok = first / nr, r = first - tok * nr;
  const uint16_t* x = a.x[which] + (t0 + tok) * ts + (h0 + r) * hs + e0;
  uint16_t* out = a.out[which] + ((t0 + tok) * a.h[which] + h0 + r) * D + e0;
  const int64_t x_step = step_tok * ts + step_r * hs, x_wrap = ts - nr * hs;
  const int out_step = (step_tok * a.h[which] + step_r) * D, out_wrap = (a.h[which] - nr) * D;
  uint4 raw = make_uint4(0, 0, 0, 0);  // the first row is loaded before the angles are made
  if (tok < nt) raw = *reinterpret_cast<const uint4*>(x);
  const bool norm = a.w[which] != nullptr;
  const bool low = e0 < a.half, in_rot = e0 < a.rot;
  const int po = LAYOUT == 1 && in_rot ? (low ? a.half : -a.half) : 0;  // partner's offset
  const int src = (lane - l) + ((e0 + po) >> 3);
  f2 w[4], wp[LAYOUT == 1 ? 4 : 1];
  if (norm) {
    float f[8];
    nr_weights<BF>(a, which, e0, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_float2(f[2 * i], f[2 * i + 1]);
    if (LAYOUT == 1) {
      nr_weights<BF>(a, which, e0 + po, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) wp[i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
  }

  for (int i = tid; i < nt * a.half; i += NR_THREADS) {
    const int t = i / a.half, k = i - t * a.half;
    const double turns = (double)a.positions[t0 + t] * a.inv_freq[k] * 0.15915494309189533577;
    const float frac = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * frac, &s, &c);
    cs[t * (D / 2) + nr_place<D, PER>(k)] = make_float2(c * a.scale, s * a.scale);
  }
  __syncthreads();

  // every lane of a warp runs the same number of passes (shuffles inside)
#pragma unroll 1
  for (int pass = 0; pass < passes; ++pass) {
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    const bool live = tok < nt;
    const float2* tc = cs + (live ? tok : 0) * (D / 2);
    uint16_t* const to = out;
    r += step_r;
    tok += step_tok;
    x += x_step;
    out += out_step;
    if (r >= nr) {
      r -= nr;
      ++tok;
      x += x_wrap;
      out += out_wrap;
    }
    if (tok < nt) raw = *reinterpret_cast<const uint4*>(x);  // the next row, in flight during this one
    f2 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = nr_unpack<BF>(in[i]);
    f2 s2 = mul2(y[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s2 = fma2(y[i], y[i], s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    // rsqrtf is good to 2 ulp; a zero row with eps 0 gives 0 * inf = NaN
    const float rs = norm ? rsqrtf(fmaf(ss, a.inv_d, a.eps)) : 1.f;
    if (norm) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], mul2(w[i], make_float2(rs, rs)));
    }
    if (LAYOUT == 0) {
      if (in_rot) {
        const float4* plane = reinterpret_cast<const float4*>(tc) + l;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float4 t = plane[(i / 2) * (D / 8)];  // two angles
          const f2 u = y[i], v = y[i + 1];
          y[i] = make_float2(u.x * t.x - u.y * t.y, u.y * t.x + u.x * t.y);
          y[i + 1] = make_float2(v.x * t.z - v.y * t.w, v.y * t.z + v.x * t.w);
          if (a.rot & 7) {  // the rotated part ends inside a lane's coordinates
            if (e0 + 2 * i >= a.rot) y[i] = u;
            if (e0 + 2 * i + 2 >= a.rot) y[i + 1] = v;
          }
        }
      }
    } else if (LAYOUT == 1) {
      uint32_t pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = __shfl_sync(0xffffffffu, in[i], src);
      if (in_rot) {
        const float4* plane = reinterpret_cast<const float4*>(tc) + ((low ? e0 : e0 - a.half) >> 3);
        const float sg = low ? -rs : rs;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f2 p = nr_unpack<BF>(pr[i]);
          if (norm) p = mul2(p, wp[i]);
          const float4 t = plane[i * (D / 16)];  // two angles
          y[i] = fma2(y[i], make_float2(t.x, t.z), mul2(p, mul2(make_float2(t.y, t.w), make_float2(sg, sg))));
        }
      }
    } else {
      float* buf = rowbuf + (tid / LPR) * D;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(buf + e0 + 2 * i) = y[i];
      __syncwarp();
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        f[i] = i & 1 ? y[i / 2].y : y[i / 2].x;
        if (e < a.rot) {
          const bool lo = e < a.half;
          const float2 t = tc[lo ? e : e - a.half];
          const float p = buf[lo ? e + a.half : e - a.half];
          f[i] = f[i] * t.x + (lo ? -p : p) * t.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
    if (live) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(y[i].x, y[i].y);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
    }
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
  a.rot = rot_dim;
  a.half = rot_dim / 2;
  a.w_f32 = weight_f32;
  a.eps = eps;
  a.scale = rope_scale;
  a.inv_d = 1.0f / (float)d;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
  // As many tokens per CTA (up to 8) as leave enough CTAs for the SMs to hold
  // four each; while the tokens alone do not fill the SMs twice, a token's rows
  // are divided among CTAs of one pass each (every CTA redoes the token's
  // angles).
  const int rpc = NR_THREADS / (d / 8);
  const int64_t sms = tq_sm_count(dev);
  a.tokens = 1;
  while (a.tokens < NR_MAX_TOKENS && n_tok / (2 * a.tokens) >= 4 * sms) a.tokens *= 2;
  a.row_step = n_tok >= 2 * sms ? std::max(hq, hkv) : rpc;
  a.q_ctas = (hq + a.row_step - 1) / a.row_step;
  const int64_t gx = (n_tok + a.tokens - 1) / a.tokens;
  const int64_t gy = a.q_ctas + (hkv + a.row_step - 1) / a.row_step;
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
