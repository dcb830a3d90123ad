// Attention of one or more query tokens per sequence over packed caches,
// causal, within a sliding window plus the first `sinks` positions.
//
// Mathematics, for the query at position p of a sequence and the kv head it
// reads: o = sum_t w_t v_hat_t / sum_t w_t over the visible t (t <= p and
// (t < sinks or t > p - window)), w_t = exp(q . k_hat_t / sqrt(d)). As in the
// decode-step attention (tq_attend.cu) nothing is decoded:
//   q . k_hat_t / sqrt(d) = n_t (H_pm D_K q) . c_K[idx_t] / (d sqrt(d)),
//   o = D_V H_pm (sum_t w_t n^V_t c_V[idx^V_t]) / (d sum_t w_t),
// so a query row is rotated once, scored against codebook levels, and its
// accumulator rotated back once. One pass over the cache with a running
// maximum and sum.
//
// This kernel is for few query rows per kv head (decode steps, drafted
// tokens). A warp takes RT = 4 NT query rows of one kv head and one share of
// the 16-position blocks that they see; warps of a CTA take neighbouring kv
// heads of the same share, so their loads are neighbours in a cache row. Codes
// go from global memory to registers (the next 32 positions' words are loaded
// while the current ones are worked on), become fp16 pairs through
// lane-replicated tables in shared memory (one conflict-free lookup per two
// codes, four at 2-bit values) and are used NT times:
//  * scores: mma m16n8k16 with A = 16 positions x 16 dims of levels, B = 16
//    dims x (4 rows x (hi, lo)) of the rotated query, whose fp16 value and
//    remainder are added up in f32;
//  * values: A = 16 dims x 16 positions of levels, B = 16 positions x (4 rows
//    x (hi, lo)) of the weights, turned from the score layout by movmatrix.
//
// Precision: sums, maxima and scores are f32. The fp16 operands are the levels
// times a common factor that puts them within 2^-14 of fp16 values (host,
// lev_f16), the rotated query as value + remainder (22 bits) scaled by a power
// of two per row, and weight x norm as value + remainder, scaled by a power of
// two that follows the largest value norm seen, so norms of any size neither
// overflow nor vanish.
//
// Bound: (P_K + P_V + 8) bytes per visible position and kv head against about
// 30 warp instructions per block and kv head for each of lookups, MMAs and
// softmax: like the decode-step kernel it issues at about half the rate that
// HBM would allow.
#include <climits>
#include <cmath>

#include "tq_attend_window.cuh"

namespace tq {

constexpr int AW_WARPS = 8;
constexpr int AW_TILE = 32;  // positions per step: two blocks

// Shared tables: pairs of codes -> two fp16 levels, one copy per lane; at
// 2-bit values, four codes -> four levels, eight copies.
template <int KB, int VB>
struct AwTables {
  static constexpr int K_BYTES = (1 << (2 * KB)) * 128;
  static constexpr bool V_QUAD = VB == 2;
  static constexpr int V_BYTES = V_QUAD ? 256 * 64 : (1 << (2 * VB)) * 128;
  static constexpr int BYTES = K_BYTES + V_BYTES;
};

template <int KB, int VB>
TQ_DEV void aw_build_tables(uint8_t* smem, const AwArgs& a) {
  using T = AwTables<KB, VB>;
  uint32_t* lk = reinterpret_cast<uint32_t*>(smem);
  for (int e = threadIdx.x; e < T::K_BYTES / 4; e += blockDim.x) {
    const int f = e >> 5;
    lk[e] = a.k_lev[f & ((1 << KB) - 1)] | (uint32_t)a.k_lev[f >> KB] << 16;
  }
  if (T::V_QUAD) {
    uint2* lv = reinterpret_cast<uint2*>(smem + T::K_BYTES);
    for (int e = threadIdx.x; e < 256 * 8; e += blockDim.x) {
      const int f = e >> 3;
      lv[e] = make_uint2(a.v_lev[f & 3] | (uint32_t)a.v_lev[(f >> 2) & 3] << 16,
                         a.v_lev[(f >> 4) & 3] | (uint32_t)a.v_lev[f >> 6] << 16);
    }
  } else {
    uint32_t* lv = reinterpret_cast<uint32_t*>(smem + T::K_BYTES);
    for (int e = threadIdx.x; e < T::V_BYTES / 4; e += blockDim.x) {
      const int f = e >> 5;
      lv[e] = a.v_lev[f & ((1 << VB) - 1)] | (uint32_t)a.v_lev[f >> VB] << 16;
    }
  }
}

TQ_DEV uint32_t aw_transpose(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int KB, int VB, int NT>
__global__ void __launch_bounds__(AW_WARPS * 32, D == 256 || NT > 1 ? 1 : 2)
    window_partial_kernel(const __grid_constant__ AwArgs a) {
  constexpr int PK = D * KB / 8, PV = D * VB / 8;
  constexpr int KT = PK / 4, VT = PV / 8;  // bytes of a thread: a quarter of a K row, an eighth of a V row
  constexpr int KW = (KT + 3) / 4, VW = (VT + 3) / 4;
  constexpr int NB = D / 16;
  constexpr int KF = 2 * KB, VF = 2 * VB;
  constexpr int RT = 4 * NT;
  using Tab = AwTables<KB, VB>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const int b = blockIdx.z;
  const int unit = blockIdx.x * AW_WARPS + warp;  // (split, kv head), heads fastest
  const int split = unit / a.hkv, hk = unit - split * a.hkv;
  const bool live = split < a.n_split;

  const AwSeq sq = aw_sequence(a, b, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  const int rows = sq.n * a.g, r0 = blockIdx.y * RT;
  if (r0 >= rows) return;  // the whole CTA
  aw_build_tables<KB, VB>(smem, a);
  __syncthreads();
  if (!live) return;
  const uint32_t lutk = smem_u32(smem) + lane * 4u;
  const uint32_t lutv = smem_u32(smem) + Tab::K_BYTES + (Tab::V_QUAD ? (lane & 7) * 8u : lane * 4u);

  // ---- rotated queries: this lane's quarter of the row of its B column
  uint32_t bq[NT][NB][2];
  float row_inv[NT];  // undoes the row's power of two, for this thread's score row
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = r0 + 4 * j + (gq >> 1);
    const bool ok = r < rows;
    const int i = ok ? r / a.g : 0, hj = ok ? r - i * a.g : 0;
    const __half* src = a.q + ((sq.q0 + i) * a.hq + hk * a.g + hj) * D + tq * (D / 4);
    float x[D / 4];
#pragma unroll
    for (int e = 0; e < D / 4; e += 8) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (ok) w = __ldg(reinterpret_cast<const uint4*>(src + e));
      const uint32_t hw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t s = hw[c] ^ a.k_sign_h2[(tq * (D / 4) + e) / 2 + c];
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&s));
        x[e + 2 * c] = f.x, x[e + 2 * c + 1] = f.y;
      }
    }
#pragma unroll
    for (int h = 1; h < D / 4; h <<= 1)
#pragma unroll
      for (int e = 0; e < D / 4; ++e)
        if ((e & h) == 0) {
          const float u = x[e], v = x[e + h];
          x[e] = u + v;
          x[e + h] = u - v;
        }
#pragma unroll
    for (int m = 1; m < 4; m <<= 1)
#pragma unroll
      for (int e = 0; e < D / 4; ++e) {
        const float o = __shfl_xor_sync(0xffffffffu, x[e], m);
        x[e] = (tq & m) ? o - x[e] : x[e] + o;
      }
    float mag = 0.f;
#pragma unroll
    for (int e = 0; e < D / 4; ++e) {
      x[e] *= a.q_scale;
      mag = fmaxf(mag, fabsf(x[e]));
    }
    mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
    mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
    float inv;
    const float up = aw_pow2_for<10>(mag, inv);
    row_inv[j] = __shfl_sync(0xffffffffu, inv, 8 * tq);  // the lane whose column holds row tq
    const bool lo = gq & 1;
#pragma unroll
    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        float v0 = x[4 * kb + 2 * e2] * up, v1 = x[4 * kb + 2 * e2 + 1] * up;
        if (lo) {
          v0 -= __half2float(__float2half_rn(v0));
          v1 -= __half2float(__float2half_rn(v1));
        }
        bq[j][kb][e2] = pack_half2(v0, v1);
      }
  }

  // ---- positions of this thread's score rows, and the blocks of the tile
  int p_row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = r0 + 4 * j + tq;
    p_row[j] = r < rows ? aw_position(sq, r / a.g) : -1;
  }
  const int p_lo = aw_position(sq, r0 / a.g), p_hi = aw_position(sq, min(r0 + RT - 1, rows - 1) / a.g);
  const AwBlocks bl = aw_blocks(p_lo, p_hi, a.window, a.sinks);
  const int share = 2 * ((bl.n + 2 * a.n_split - 1) / (2 * a.n_split));
  const int m0 = split * share, m1 = min(m0 + share, bl.n);

  float m_run[NT], l_run[NT], acc[NT][NB][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    m_run[j] = -INFINITY;
    l_run[j] = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][i][c] = 0.f;
  }
  // weights are held times 2^10 / (a power of two near the largest value norm)
  float v_up = 1.f, v_inv = 1.f, v_most = 0.f;

  // one step's codes and norms; rows behind the context are read from its last row
  uint32_t kw[2][2][KW], vw[2][4][VW];
  float nk[2][2], nv[2][2];
  int t_blk[2];
  auto fetch = [&](int m) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = aw_block(bl, min(m + h, m1 - 1));
      t_blk[h] = m + h < m1 ? j * ATT_BLOCK : INT_MAX - 64;  // behind every query
      const int64_t base = aw_block_row(a, b, j);
      const int most = sq.ctx - 1 - j * ATT_BLOCK;  // last row of the block inside the context
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = (base + min(gq + 8 * r, most)) * a.hkv + hk;
        aw_load<KT, KW>(kw[h][r], a.k_packed + row * PK, tq * KT, PK);
        nk[h][r] = __ldg(a.k_norms + row);
        nv[h][r] = __ldg(a.v_norms + row);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t row = (base + min(2 * tq + (r & 1) + 8 * (r >> 1), most)) * a.hkv + hk;
        aw_load<VT, VW>(vw[h][r], a.v_packed + row * PV, gq * VT, PV);
      }
    }
  };
  if (m0 < m1) fetch(m0);

  for (int m = m0; m < m1; m += 2) {
    uint32_t ck[2][2][KW], cv[2][4][VW];
    float cnk[2][2], cnv[2][2];
    int ct[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ct[h] = t_blk[h];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        cnk[h][r] = nk[h][r];
        cnv[h][r] = nv[h][r];
#pragma unroll
        for (int i = 0; i < KW; ++i) ck[h][r][i] = kw[h][r][i];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < VW; ++i) cv[h][r][i] = vw[h][r][i];
    }
    if (m + 2 < m1) fetch(m + 2);

    // ---- scores
    float sc[NT][2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float c[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[j][i] = 0.f;
#pragma unroll
      for (int kb = 0; kb < NB; ++kb) {
        const uint32_t a0 = lds32(aw_bits<KF>(ck[h][0], 2 * kb * KF) * 128u + lutk);
        const uint32_t a1 = lds32(aw_bits<KF>(ck[h][1], 2 * kb * KF) * 128u + lutk);
        const uint32_t a2 = lds32(aw_bits<KF>(ck[h][0], (2 * kb + 1) * KF) * 128u + lutk);
        const uint32_t a3 = lds32(aw_bits<KF>(ck[h][1], (2 * kb + 1) * KF) * 128u + lutk);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816(c[j], a0, a1, a2, a3, bq[j][kb][0], bq[j][kb][1]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bool see = aw_visible(ct[h] + gq + 8 * r, p_row[j], a.window, a.sinks);
          sc[j][h][r] = see ? (c[j][2 * r] + c[j][2 * r + 1]) * (cnk[h][r] * row_inv[j]) : -INFINITY;
        }
    }
    // ---- the power of two of the weights: follows the largest value norm
    float nmax = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float v = fabsf(cnv[h][r]);
        if (ct[h] + gq + 8 * r <= p_hi && v < INFINITY) nmax = fmaxf(nmax, v);
      }
    nmax = warp_max8(nmax);
    float v_fix = 1.f;
    if (nmax > v_most) {
      v_most = nmax;
      float inv;
      const float up = aw_pow2_for<10>(nmax, inv);
      v_fix = up * v_inv;  // <= 1 from the second time on
      v_up = up;
      v_inv = inv;
    }
    // ---- running maximum and sum; weights times norms as value + remainder
    uint32_t bp[NT][2][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float mx = warp_max8(fmaxf(fmaxf(sc[j][0][0], sc[j][0][1]), fmaxf(sc[j][1][0], sc[j][1][1])));
      const float mn = fmaxf(m_run[j], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every weight is exp2(-inf) = 0
      const float alpha = aw_exp2(m_run[j] - ref);
      float p[2][2], sum = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          p[h][r] = aw_exp2(sc[j][h][r] - ref);
          sum += p[h][r];
        }
      l_run[j] = l_run[j] * alpha + sum;  // of this lane's positions
      m_run[j] = mn;
      // the accumulator's columns 2 tq, 2 tq + 1 belong to this same row
      const float fix = alpha * v_fix;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[j][i][c] *= fix;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float w = sc[j][h][r] == -INFINITY ? 0.f : p[h][r] * (cnv[h][r] * v_up);
          const float hi = __half2float(__float2half_rn(w));
          bp[j][h][r] = aw_transpose(pack_half2(hi, w - hi));
        }
    }
    // ---- values
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (Tab::V_QUAD) {
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
          uint2 lv[4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(lv[r].x), "=r"(lv[r].y)
                         : "r"(aw_bits<8>(cv[h][r], 8 * i) * 64u + lutv));
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t l0 = s ? lv[0].y : lv[0].x, l1 = s ? lv[1].y : lv[1].x;
            const uint32_t l2 = s ? lv[2].y : lv[2].x, l3 = s ? lv[3].y : lv[3].x;
            const uint32_t a0 = __byte_perm(l0, l1, 0x5410), a1 = __byte_perm(l0, l1, 0x7632);
            const uint32_t a2 = __byte_perm(l2, l3, 0x5410), a3 = __byte_perm(l2, l3, 0x7632);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16816(acc[j][2 * i + s], a0, a1, a2, a3, bp[j][h][0], bp[j][h][1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const uint32_t l0 = lds32(aw_bits<VF>(cv[h][0], i * VF) * 128u + lutv);
          const uint32_t l1 = lds32(aw_bits<VF>(cv[h][1], i * VF) * 128u + lutv);
          const uint32_t l2 = lds32(aw_bits<VF>(cv[h][2], i * VF) * 128u + lutv);
          const uint32_t l3 = lds32(aw_bits<VF>(cv[h][3], i * VF) * 128u + lutv);
          const uint32_t a0 = __byte_perm(l0, l1, 0x5410), a1 = __byte_perm(l0, l1, 0x7632);
          const uint32_t a2 = __byte_perm(l2, l3, 0x5410), a3 = __byte_perm(l2, l3, 0x7632);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma16816(acc[j][i], a0, a1, a2, a3, bp[j][h][0], bp[j][h][1]);
        }
      }
    }
  }

  // ---- results: this thread's row of each tile, dims [gq D/8, + D/8)
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = r0 + 4 * j + tq;
    const bool ok = r < rows;
    const int i = ok ? r / a.g : 0, hj = ok ? r - i * a.g : 0;
    const int64_t out_row = (sq.q0 + i) * a.hq + hk * a.g + hj;
    const float l = warp_sum8(l_run[j]);
    float x[D / 8];
#pragma unroll
    for (int e = 0; e < NB; ++e) {
      x[2 * e] = acc[j][e][0] + acc[j][e][1];
      x[2 * e + 1] = acc[j][e][2] + acc[j][e][3];
    }
    if (a.n_split > 1) {
      if (ok) {
        const int64_t idx = out_row * a.n_split + split;
        if (gq == 0) {
          a.ws_m[idx] = m_run[j];
          a.ws_l[idx] = l;
        }
        if (m_run[j] != -INFINITY) {
          float4* dst = reinterpret_cast<float4*>(a.ws_acc + idx * D + gq * (D / 8));
#pragma unroll
          for (int e = 0; e < D / 8; e += 4)
            dst[e / 4] = make_float4(x[e] * v_inv, x[e + 1] * v_inv, x[e + 2] * v_inv, x[e + 3] * v_inv);
        }
      }
      continue;
    }
    const float inv = l > 0.f ? v_inv * a.o_scale / l : 0.f;
#pragma unroll
    for (int h = 1; h < D / 8; h <<= 1)
#pragma unroll
      for (int e = 0; e < D / 8; ++e)
        if ((e & h) == 0) {
          const float u = x[e], v = x[e + h];
          x[e] = u + v;
          x[e + h] = u - v;
        }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1)
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {
        const float o = __shfl_xor_sync(0xffffffffu, x[e], 4 * m);
        x[e] = (gq & m) ? o - x[e] : x[e] + o;
      }
    if (ok) {
      uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + gq * (D / 8));
#pragma unroll
      for (int e = 0; e < D / 8; e += 8) {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c] = pack_half2(x[e + 2 * c] * inv, x[e + 2 * c + 1] * inv) ^ a.v_sign_h2[(gq * (D / 8) + e) / 2 + c];
        dst[e / 8] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// Merge of the splits of a row, one warp per row: M = max m_s, weights
// 2^(m_s - M), o = D_V H_pm (sum_s weight acc_s / sum_s weight l_s) / d.
template <int D>
__global__ void __launch_bounds__(256) window_combine_kernel(const __grid_constant__ AwArgs a) {
  constexpr int E = D / 32;  // elements of a lane: dims [E lane, + E)
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const AwSeq sq = aw_sequence(a, blockIdx.y, false);
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= (int64_t)sq.n * a.hq) return;
  const int64_t row = sq.q0 * a.hq + r;
  const float* ms = a.ws_m + row * a.n_split;
  const float* ls = a.ws_l + row * a.n_split;
  float M = -INFINITY;
  bool bad = false;  // a NaN score leaves a NaN sum, whatever its split's maximum
  for (int s = lane; s < a.n_split; s += 32) {
    M = fmaxf(M, ms[s]);
    bad = bad || ls[s] != ls[s];
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
  float x[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.f;
  if (M != -INFINITY) {
    for (int s0 = 0; s0 < a.n_split; s0 += 32) {
      float w = 0.f;
      if (s0 + lane < a.n_split) {
        w = aw_exp2(ms[s0 + lane] - M);
        l = fmaf(w, ls[s0 + lane], l);
      }
      const int n = min(32, a.n_split - s0);
      const float* acc = a.ws_acc + (row * a.n_split + s0) * D + lane * E;
#pragma unroll 4
      for (int s = 0; s < n; ++s) {
        const float ws = __shfl_sync(0xffffffffu, w, s);
        if (ws == 0.f) continue;  // an empty split has written no accumulator
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = *reinterpret_cast<const float2*>(acc + (int64_t)s * D + e);
          x[e] = fmaf(ws, v.x, x[e]);
          x[e + 1] = fmaf(ws, v.y, x[e + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) l += __shfl_xor_sync(0xffffffffu, l, m);
  float inv = l > 0.f ? a.o_scale / l : 0.f;
  if (__any_sync(0xffffffffu, bad)) inv = __int_as_float(0x7fc00000);
#pragma unroll
  for (int h = 1; h < E; h <<= 1)
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((e & h) == 0) {
        const float u = x[e], v = x[e + h];
        x[e] = u + v;
        x[e + h] = u - v;
      }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float o = __shfl_xor_sync(0xffffffffu, x[e], m);
      x[e] = (lane & m) ? o - x[e] : x[e] + o;
    }
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    dst[e / 2] = pack_half2(x[e] * inv, x[e + 1] * inv) ^ a.v_sign_h2[(lane * E + e) / 2];
}

// Query rows per kv head from which the tensor-memory kernel takes a call.
constexpr int64_t AW_TC_ROWS = 32;

static bool window_tc(int hq, int hkv, int max_q) { return (int64_t)max_q * (hq / hkv) >= AW_TC_ROWS; }

// Splits of a call, from the sizes alone, so that the workspace is too: this
// kernel, enough warps to fill the SMs twice over, at least one step of 32
// positions each; the tensor-memory kernel, one CTA per SM, at least four
// tiles of 64 each.
static int window_splits(int B, int hq, int hkv, int max_q, int d, int64_t s_max, int64_t window, int64_t sinks) {
  const bool tc = window_tc(hq, hkv, max_q);
  const int64_t rt = tc ? tq_window_tc_rows(d) : 4;
  const int64_t tiles = ((int64_t)max_q * (hq / hkv) + rt - 1) / rt;
  const int64_t units = (int64_t)B * hkv * tiles;
  int64_t seen = s_max;
  if (window > 0) seen = std::min(seen, window + sinks + max_q + 2 * ATT_BLOCK);
  const int64_t steps = tc ? (seen + 255) / 256 : (seen + AW_TILE - 1) / AW_TILE;
  const int64_t slots = tc ? 148 : (d == 256 ? 1 : 2) * 148 * AW_WARPS;
  return (int)std::max<int64_t>(1, std::min<int64_t>(slots / units, steps));
}

template <int D, int KB, int VB, int NT>
static cudaError_t launch_window_t(const AwArgs& a, cudaStream_t st) {
  constexpr int smem = AwTables<KB, VB>::BYTES;
  cudaError_t e = cudaFuncSetAttribute(window_partial_kernel<D, KB, VB, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t gx = ((int64_t)a.n_split * a.hkv + AW_WARPS - 1) / AW_WARPS;
  const int64_t gy = ((int64_t)a.max_q * a.g + 4 * NT - 1) / (4 * NT);
  if (gx > 0x7fffffff || gy > 65535) return cudaErrorNotSupported;
  window_partial_kernel<D, KB, VB, NT><<<dim3((unsigned)gx, (unsigned)gy, a.B), AW_WARPS * 32, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.n_split == 1) return e;
  return tq_launch_window_combine(a, D, st);
}

template <int D, int KB, int VB>
static cudaError_t launch_window(const AwArgs& a, cudaStream_t st) {
  // two column tiles share every lookup where a kv head has more than 4 query rows
  if (D <= 128 && (int64_t)a.max_q * a.g > 4) return launch_window_t<D, KB, VB, D <= 128 ? 2 : 1>(a, st);
  return launch_window_t<D, KB, VB, 1>(a, st);
}

template <int D>
static cudaError_t launch_window_d(const AwArgs& a, int kb, int vb, cudaStream_t st) {
#define TQ_AW_CASE(KB_, VB_) \
  if (kb == KB_ && vb == VB_) return launch_window<D, KB_, VB_>(a, st);
  TQ_AW_CASE(2, 2) TQ_AW_CASE(2, 3) TQ_AW_CASE(2, 4) TQ_AW_CASE(3, 2) TQ_AW_CASE(3, 3) TQ_AW_CASE(3, 4)
  TQ_AW_CASE(4, 2) TQ_AW_CASE(4, 3) TQ_AW_CASE(4, 4)
#undef TQ_AW_CASE
  return cudaErrorInvalidValue;
}

}  // namespace tq

using namespace tq;

cudaError_t tq_launch_window_combine(const AwArgs& a, int d, cudaStream_t st) {
  const int64_t gx = ((int64_t)a.max_q * a.hq + 7) / 8;
  if (gx > 0x7fffffff) return cudaErrorNotSupported;
  const dim3 grid((unsigned)gx, a.B);
  if (d == 64) return tq_launch_pdl(window_combine_kernel<64>, grid, dim3(256), 0, st, a);
  if (d == 128) return tq_launch_pdl(window_combine_kernel<128>, grid, dim3(256), 0, st, a);
  return tq_launch_pdl(window_combine_kernel<256>, grid, dim3(256), 0, st, a);
}

size_t tq_attend_window_workspace_impl(int64_t n_tok, int B, int max_q, int hq, int hkv, int head_dim, int64_t s_max,
                                       int64_t window, int64_t sinks) {
  const int ns = window_splits(B, hq, hkv, max_q, head_dim, s_max, window, sinks);
  if (ns == 1) return 0;
  const size_t rows = (size_t)n_tok * hq * ns;
  return 2 * align16(rows * 4) + rows * (size_t)head_dim * 4;
}

tq_status tq_launch_attend_window(const tq_ctx* k, const tq_ctx* v, const void* q, int64_t n_tok, int B,
                                  const int32_t* q_offsets, int max_q, int hq, int hkv, const void* k_cache,
                                  const float* k_norms, const void* v_cache, const float* v_norms, int64_t s_max,
                                  int64_t num_blocks, const int32_t* block_tables, int max_blocks,
                                  const int32_t* ctx_lens, int64_t window, int64_t sinks, void* out, void* workspace,
                                  void* stream) {
  const int d = k->d;
  AwArgs a{};
  for (int i = 0; i < TQ_MAX_D / 2; ++i) {
    a.k_sign_h2[i] = k->t.sign_h2[i];
    a.v_sign_h2[i] = v->t.sign_h2[i];
  }
  for (int i = 0; i < TQ_MAX_L; ++i) {
    a.k_lev[i] = k->lev_f16[i];
    a.v_lev[i] = v->lev_f16[i];
  }
  a.q_scale = (float)(1.4426950408889634 / ((double)d * std::sqrt((double)d) * k->lev_scale));
  a.o_scale = (float)(1.0 / ((double)d * v->lev_scale));
  a.q = static_cast<const __half*>(q);
  a.out = static_cast<__half*>(out);
  a.q_offsets = q_offsets;
  a.k_packed = static_cast<const uint8_t*>(k_cache);
  a.k_norms = k_norms;
  a.v_packed = static_cast<const uint8_t*>(v_cache);
  a.v_norms = v_norms;
  a.block_tables = block_tables;
  a.ctx_lens = ctx_lens;
  a.s_max = s_max;
  a.num_blocks = num_blocks;
  a.n_tok = n_tok;
  a.max_blocks = max_blocks;
  a.B = B;
  a.max_q = max_q;
  a.hq = hq;
  a.hkv = hkv;
  a.g = hq / hkv;
  a.window = window <= 0 || window > INT_MAX ? INT_MAX : (int)window;
  a.sinks = (int)std::min<int64_t>(sinks, INT_MAX);
  a.n_split = window_splits(B, hq, hkv, max_q, d, s_max, window, sinks);
  const size_t rows = (size_t)n_tok * hq * a.n_split;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_m = reinterpret_cast<float*>(ws);
  a.ws_l = reinterpret_cast<float*>(ws + align16(rows * 4));
  a.ws_acc = reinterpret_cast<float*>(ws + 2 * align16(rows * 4));
  a.err = tq_error_word();
  if (!a.err) return TQ_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.wait_limit = TQ_WAIT_LIMIT_CYCLES;
  cudaError_t e = cudaErrorInvalidValue;
  if (window_tc(hq, hkv, max_q)) {
    e = tq_launch_window_tc(a, d, k->bits, v->bits, st);
    if (e == cudaSuccess && a.n_split > 1) e = tq_launch_window_combine(a, d, st);
    if (e == cudaErrorNotSupported) return TQ_ERR_UNSUPPORTED;
    return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
  }
  if (d == 64) e = launch_window_d<64>(a, k->bits, v->bits, st);
  if (d == 128) e = launch_window_d<128>(a, k->bits, v->bits, st);
  if (d == 256) e = launch_window_d<256>(a, k->bits, v->bits, st);
  if (e == cudaErrorNotSupported) return TQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
