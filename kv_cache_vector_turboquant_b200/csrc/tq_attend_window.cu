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
// the 16-position blocks that they see; neighbouring warps take neighbouring
// kv heads of the same share, whose cache rows are neighbours in memory. Each
// warp copies its own tiles of 32 positions (codes and norms) into a private
// ring in shared memory with asynchronous 4- to 16-byte copies and waits for
// nobody. Codes become fp16 pairs through lane-replicated tables and are used
// NT times:
//  * scores: mma m16n8k16 with A = 16 positions x 16 dims of levels, B = 16
//    dims x (4 rows x (hi, lo)) of the rotated query, whose fp16 value and
//    remainder are added up in f32;
//  * values: A = 16 dims x 16 positions of levels, B = 16 positions x (4 rows
//    x (hi, lo)) of the weights, turned from the score layout by movmatrix.
// Table entries are 256 bytes apart at a shared address that is a multiple of
// 64 KB: the lookup's address is one byte permute that puts the index byte
// over the lane's constant (128 bytes of key entries, then 128 of value
// entries per index). An index byte is two 4-bit or four 2-bit key codes, one
// 4-bit value code of two positions, or two 2-bit value codes of two
// positions, so that a lookup returns whole operand registers; 3-bit codes
// are looked up in pairs.
//
// Precision: sums, maxima and scores are f32. The fp16 operands are the levels
// times a common factor that puts them within 2^-14 of fp16 values (host,
// lev_f16), the rotated query as value + remainder (22 bits) scaled by a power
// of two per row, and weight x norm as value + remainder, scaled by a power of
// two that follows the largest value norm that a row of the warp sees (up to
// 2^14: nothing overflows). A row whose own products are much smaller takes a
// lower reference for its weights (aw_reference), so each product is off by
// 2^-22 of itself or 2^-23 of the row's largest, whatever other rows see, for
// norms within 2^90 of the largest. The reference moves only when a score
// exceeds it by more than 2^8 or the row's products are small (exact: sum and
// accumulator share it).
//
// Bound: (P_K + P_V + 8) bytes per visible position and kv head, against about
// 680 warp instructions and 200 shared-memory wavefronts per 32 positions and
// kv head. Measured, 16 sequences with 8192 visible positions, 32 query and 8 kv
// heads of 128, keys 4 and values 2 bits (109 MB): 48.2 us a call (2.3 TB/s;
// each kernel by itself 45 and its merge 7, which overlap); issue slots 55 %,
// shared-memory pipe 59 %, ALU 47 %. The instances at 128 registers spill a few words
// (head_dim 128, up to 4 query rows). More warps of fewer registers (24 of 80) take 55 us: the pipes are
// what is shared, not latency that is left open.
#include <climits>
#include <cmath>

#include "tq_attend_window.cuh"

namespace tq {

constexpr int AW_TILE = 32;             // positions per step: two blocks
constexpr uint32_t AW_TABLE = 65536;    // bytes of the table, and its alignment
constexpr int AW_SMEM = 232448;

template <int D, int KB, int VB, int NT>
struct AwCfg {
  static constexpr int PK = D * KB / 8, PV = D * VB / 8;
  static constexpr int WARPS = D * NT <= 128 ? 16 : 8;  // by registers: 128 or 255 of a thread
  static constexpr int CK = PK % 16 ? 8 : 16, CV = PV % 16 ? 8 : 16;  // bytes of a copy
  static constexpr int K0 = 0, V0 = AW_TILE * PK, N0 = V0 + AW_TILE * PV;
  static constexpr int STAGE = N0 + AW_TILE * 8;
  // rings lie below and above the table; the dynamic region starts within 2 KB
  // of shared address 0 (checked at run time)
  static constexpr int BELOW = (int)AW_TABLE - 2048, ABOVE = AW_SMEM - 2 * (int)AW_TABLE;
  static constexpr bool fits(int stages) {
    return BELOW / (stages * STAGE) + ABOVE / (stages * STAGE) >= WARPS;
  }
  static constexpr int STAGES = fits(4) ? 4 : fits(3) ? 3 : 2;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int LOW = BELOW / RING < WARPS ? BELOW / RING : WARPS;  // rings below the table
  static_assert(fits(STAGES), "shared memory of the rings");
};

// Table entry of index f: operand words of the key half and of the value half.
template <int KB>
TQ_DEV uint2 aw_k_entry(const uint16_t* lev, int f) {
  if (KB == 2)
    return make_uint2(lev[f & 3] | (uint32_t)lev[(f >> 2) & 3] << 16,
                      lev[(f >> 4) & 3] | (uint32_t)lev[(f >> 6) & 3] << 16);
  const int m = (1 << KB) - 1;
  return make_uint2(lev[f & m] | (uint32_t)lev[(f >> KB) & m] << 16, 0u);
}
template <int VB>
TQ_DEV uint2 aw_v_entry(const uint16_t* lev, int f) {
  if (VB == 2)  // two dims of one position (low nibble) and of the next (high)
    return make_uint2(lev[f & 3] | (uint32_t)lev[(f >> 4) & 3] << 16,
                      lev[(f >> 2) & 3] | (uint32_t)lev[(f >> 6) & 3] << 16);
  const int m = (1 << VB) - 1;  // 4 bits: one dim of two positions; 3 bits: two dims
  return make_uint2(lev[f & m] | (uint32_t)lev[(f >> VB) & m] << 16, 0u);
}

template <int BYTES>
TQ_DEV void aw_copy(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
TQ_DEV void aw_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
TQ_DEV void aw_copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

TQ_DEV uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
  return r;
}

// NBYTES bytes at shared address `addr` (a multiple of the largest power of
// two up to 16 that divides NBYTES, at least 2; 3 bytes: any) as words; `end`
// = first address behind the row, not read.
template <int NBYTES, int NW>
TQ_DEV void aw_lds(uint32_t (&w)[NW], uint32_t addr, uint32_t end) {
  static_assert(NW == (NBYTES + 3) / 4, "words of the stream");
  if constexpr (NBYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < NBYTES / 16; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(addr + 16 * i));
  } else if constexpr (NBYTES % 8 == 0) {
#pragma unroll
    for (int i = 0; i < NBYTES / 8; ++i) {
      const uint2 r = lds64(addr + 8 * i);
      w[2 * i] = r.x, w[2 * i + 1] = r.y;
    }
  } else if constexpr (NBYTES % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NBYTES / 4; ++i) w[i] = lds32(addr + 4 * i);
  } else if constexpr (NBYTES == 2) {
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else {  // 3 or 6 bytes: two aligned words
    const uint32_t at = addr & ~3u, sh = (addr & 3u) * 8u;
    const uint32_t r0 = lds32(at), r1 = lds32(min(at + 4u, end - 4u));
    w[0] = __funnelshift_r(r0, r1, sh);
    if constexpr (NW > 1) w[1] = r1 >> sh;
  }
}

// 16-byte chunk of a row in its ring slot: rows of 64 and 128 bytes are
// swizzled so that the fragment loads of a warp fall in distinct banks. Value
// rows go to slot (r % 2) 16 + r / 2 (a load's four rows are then neighbours).
template <int P>
TQ_DEV int aw_k_chunk(int row, int c) {
  return P == 128 ? c ^ (row & 1) : c;
}
template <int P>
TQ_DEV int aw_v_chunk(int slot, int c) {
  return P == 64 ? c ^ (((slot >> 1) & 1) << 1) : P == 128 ? c ^ ((slot & 3) << 1) : c;
}

TQ_DEV uint32_t aw_transpose(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Address of the entry whose index is byte `i` of w.
TQ_DEV uint32_t aw_at(uint32_t w, uint32_t lane_base, int i) { return __byte_perm(w, lane_base, 0x7604u | (i << 4)); }

template <int D, int KB, int VB, int NT>
__global__ void __launch_bounds__(AwCfg<D, KB, VB, NT>::WARPS * 32, 1)
    window_partial_kernel(const __grid_constant__ AwArgs a) {
  using C = AwCfg<D, KB, VB, NT>;
  constexpr int PK = C::PK, PV = C::PV, STAGES = C::STAGES, WARPS = C::WARPS;
  constexpr int KT = PK / 4, VT = PV / 8;  // bytes of a thread: a quarter of a K row, an eighth of a V row
  constexpr int KW = (KT + 3) / 4, VW = (VT + 3) / 4;
  constexpr int NB = D / 16;
  constexpr int RT = 4 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  // what is the same for a warp is broadcast from its first lane, so that what
  // follows from it (blocks, addresses) is known to be the same for the warp
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const int b = blockIdx.z;
  const int unit = blockIdx.x * WARPS + warp;  // (split, kv head), heads fastest
  const int split = unit / a.hkv, hk = unit - split * a.hkv;

  AwSeq sq = aw_sequence(a, b, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  sq.n = __shfl_sync(0xffffffffu, sq.n, 0);
  sq.ctx = __shfl_sync(0xffffffffu, sq.ctx, 0);
  const int rows = sq.n * a.g, r0 = blockIdx.y * RT;
  if (r0 >= rows) return;  // the whole CTA
  const uint32_t raw = smem_u32(smem);
  if (raw > 2048u) {  // the rings would not lie where they were planned
    if (threadIdx.x == 0) record_error(a.err, TQ_DEVERR_SMEM_LAYOUT);
    return;
  }
  const uint32_t table = AW_TABLE;
  const uint32_t ring = warp < C::LOW ? ((raw + 127u) & ~127u) + (uint32_t)(warp * C::RING)
                                      : 2 * AW_TABLE + (uint32_t)((warp - C::LOW) * C::RING);

  // ---- positions of this thread's score rows, the blocks of the tile, this split's share
  int p_row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = r0 + 4 * j + tq;
    p_row[j] = r < rows ? aw_position(sq, r / a.g) : -1;
  }
  const int p_lo = aw_position(sq, r0 / a.g), p_hi = aw_position(sq, min(r0 + RT - 1, rows - 1) / a.g);
  const AwBlocks bl = aw_blocks(p_lo, p_hi, a.window, a.sinks);
  const int share = 2 * ((bl.n + 2 * a.n_split - 1) / (2 * a.n_split));
  const int m0 = min(split * share, bl.n), m1 = split < a.n_split ? min(m0 + share, bl.n) : m0;
  const int tiles = (m1 - m0 + 1) / 2;

  // ---- copies of tile i into stage i % STAGES; rows behind the context are
  // read from its last one. Table entries are loaded one tile ahead.
  int ent[2];
  auto entries = [&](int i) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      ent[h] = __shfl_sync(0xffffffffu, aw_block_entry(a, b, aw_block(bl, min(m0 + 2 * i + h, m1 - 1))), 0);
  };
  constexpr int NK = PK / C::CK, NV = PV / C::CV;  // copies per row; as many per lane
  const int k_step = a.hkv * PK, v_step = a.hkv * PV;
  // offsets of this lane's copies within a block that is whole
  int k_off[NK], v_off[NV];
#pragma unroll
  for (int it = 0; it < NK; ++it) {
    const int e = it * 32 + lane, row = e / NK;
    k_off[it] = (row & 15) * k_step + (e - row * NK) * C::CK;
  }
#pragma unroll
  for (int it = 0; it < NV; ++it) {
    const int e = it * 32 + lane, row = e / NV;
    v_off[it] = (row & 15) * v_step + (e - row * NV) * C::CV;
  }
  auto copy = [&](int i) {
    const uint32_t st = ring + (uint32_t)((i % STAGES) * C::STAGE);
    const uint8_t *kb[2], *vb[2];
    int64_t row0[2];
    int over = 0;  // rows of the last block behind the context
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row0[h] = aw_entry_row(a, b, ent[h]) * a.hkv + hk;
      kb[h] = a.k_packed + row0[h] * PK;
      vb[h] = a.v_packed + row0[h] * PV;
      over = max(over, (aw_block(bl, min(m0 + 2 * i + h, m1 - 1)) + 1) * ATT_BLOCK - sq.ctx);
    }
    const int n_row = lane & 15;
    int64_t n = row0[0] + (int64_t)n_row * a.hkv;
    if (lane >= 16) n = row0[1] + (int64_t)n_row * a.hkv;
    if (over <= 0) {
#pragma unroll
      for (int it = 0; it < NK; ++it) {
        const int e = it * 32 + lane, row = e / NK, c = e - row * NK;
        aw_copy<C::CK>(st + C::K0 + row * PK + (C::CK == 16 ? aw_k_chunk<PK>(row, c) : c) * C::CK,
                       (row < 16 ? kb[0] : kb[1]) + k_off[it]);
      }
#pragma unroll
      for (int it = 0; it < NV; ++it) {
        const int e = it * 32 + lane, row = e / NV, c = e - row * NV, slot = (row & 1) * 16 + (row >> 1);
        aw_copy<C::CV>(st + C::V0 + slot * PV + (C::CV == 16 ? aw_v_chunk<PV>(slot, c) : c) * C::CV,
                       (row < 16 ? vb[0] : vb[1]) + v_off[it]);
      }
    } else {
      int most[2];  // last row of each block inside the context
#pragma unroll
      for (int h = 0; h < 2; ++h)
        most[h] = min(15, sq.ctx - 1 - aw_block(bl, min(m0 + 2 * i + h, m1 - 1)) * ATT_BLOCK);
#pragma unroll 1
      for (int e = lane; e < 32 * NK; e += 32) {
        const int row = e / NK, c = e - row * NK, h = row >> 4;
        aw_copy<C::CK>(st + C::K0 + row * PK + (C::CK == 16 ? aw_k_chunk<PK>(row, c) : c) * C::CK,
                       (h ? kb[1] : kb[0]) + min(row & 15, h ? most[1] : most[0]) * k_step + c * C::CK);
      }
#pragma unroll 1
      for (int e = lane; e < 32 * NV; e += 32) {
        const int row = e / NV, c = e - row * NV, h = row >> 4, slot = (row & 1) * 16 + (row >> 1);
        aw_copy<C::CV>(st + C::V0 + slot * PV + (C::CV == 16 ? aw_v_chunk<PV>(slot, c) : c) * C::CV,
                       (h ? vb[1] : vb[0]) + min(row & 15, h ? most[1] : most[0]) * v_step + c * C::CV);
      }
      const int h = lane >> 4;
      n = (h ? row0[1] : row0[0]) + (int64_t)min(n_row, h ? most[1] : most[0]) * a.hkv;
    }
    aw_copy<4>(st + C::N0 + lane * 4, a.k_norms + n);
    aw_copy<4>(st + C::N0 + 128 + lane * 4, a.v_norms + n);
  };
  if (tiles > 0) entries(0);
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    if (i < tiles) {
      copy(i);
      if (i + 1 < tiles) entries(i + 1);
    }
    aw_copy_commit();
  }

  // ---- the table: 8 threads per index, each 32 bytes of its two halves' copies
  for (int e = threadIdx.x; e < 256 * 16; e += WARPS * 32) {
    const int f = e >> 4, part = e & 15;  // 16 bytes each: 8 of keys, 8 of values
    const uint2 w = part < 8 ? aw_k_entry<KB>(a.k_lev, f) : aw_v_entry<VB>(a.v_lev, f);
    const bool two = part < 8 ? KB == 2 : VB == 2;
    const uint4 v = two ? make_uint4(w.x, w.y, w.x, w.y) : make_uint4(w.x, w.x, w.x, w.x);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(table + (uint32_t)(f * 256 + part * 16)), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
  }

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
  __syncthreads();  // the table is complete
  if (split >= a.n_split) return;

  const uint32_t lut_k = table + (KB == 2 ? (lane & 15) * 8u : lane * 4u);
  const uint32_t lut_v = table + 128u + (VB == 2 ? (lane & 15) * 8u : lane * 4u);
  // w_low: a lower bound of the largest |weight x norm| of the row so far
  // (infinite before the row's first position: no reason to move)
  float m_ref[NT], w_low[NT], l_run[NT], acc[NT][NB][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    m_ref[j] = -INFINITY;
    w_low[j] = INFINITY;
    l_run[j] = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][i][c] = 0.f;
  }
  // value norms times v_up lie below 64; v_up is 2^5 over a power of two near
  // the largest one seen
  float v_up = 0.f, v_inv = 1.f;

  for (int i = 0; i < tiles; ++i) {
    aw_copy_wait<STAGES - 2>();
    __syncwarp();  // every lane's copies of this tile are there, and the stage before it is free
    if (i + STAGES - 1 < tiles) {
      copy(i + STAGES - 1);
      if (i + STAGES < tiles) entries(i + STAGES);
    }
    aw_copy_commit();
    const uint32_t st = ring + (uint32_t)((i % STAGES) * C::STAGE);
    int t_blk[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      t_blk[h] = m0 + 2 * i + h < m1 ? aw_block(bl, m0 + 2 * i + h) * ATT_BLOCK : INT_MAX - 64;  // behind every query
    // whether some position may be masked for some row (also in the sinks' blocks)
    const bool hidden = t_blk[0] <= p_hi - a.window || t_blk[1] + (ATT_BLOCK - 1) > p_lo;

    // ---- scores
    float sc[NT][2][2], nv[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float c[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) c[j][q] = 0.f;
      uint32_t w0[KW], w1[KW];
      const int ra = 16 * h + gq;
      if constexpr (PK == 128) {  // two swizzled chunks of 16 bytes
#pragma unroll
        for (int q = 0; q < KT / 16; ++q) {
          uint32_t u[4];
          const uint32_t at = st + C::K0 + ra * PK + aw_k_chunk<PK>(ra, tq * (KT / 16) + q) * 16;
          aw_lds<16>(u, at, 0);
#pragma unroll
          for (int z = 0; z < 4; ++z) w0[4 * q + z] = u[z];
          aw_lds<16>(u, at + 8 * PK, 0);
#pragma unroll
          for (int z = 0; z < 4; ++z) w1[4 * q + z] = u[z];
        }
      } else {
        const uint32_t row = st + C::K0 + ra * PK;
        aw_lds<KT>(w0, row + tq * KT, row + PK);
        aw_lds<KT>(w1, row + 8 * PK + tq * KT, row + 9 * PK);
      }
#pragma unroll
      for (int kb = 0; kb < NB; ++kb) {
        uint32_t a0, a1, a2, a3;
        if constexpr (KB == 4) {
          a0 = lds32(aw_at(w0[kb / 2], lut_k, 2 * (kb & 1)));
          a1 = lds32(aw_at(w1[kb / 2], lut_k, 2 * (kb & 1)));
          a2 = lds32(aw_at(w0[kb / 2], lut_k, 2 * (kb & 1) + 1));
          a3 = lds32(aw_at(w1[kb / 2], lut_k, 2 * (kb & 1) + 1));
        } else if constexpr (KB == 2) {
          const uint2 u = lds64(aw_at(w0[kb / 4], lut_k, kb & 3)), v = lds64(aw_at(w1[kb / 4], lut_k, kb & 3));
          a0 = u.x, a2 = u.y, a1 = v.x, a3 = v.y;
        } else {
          a0 = lds32(aw_bits<6>(w0, 12 * kb) * 256u + lut_k);
          a1 = lds32(aw_bits<6>(w1, 12 * kb) * 256u + lut_k);
          a2 = lds32(aw_bits<6>(w0, 12 * kb + 6) * 256u + lut_k);
          a3 = lds32(aw_bits<6>(w1, 12 * kb + 6) * 256u + lut_k);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816(c[j], a0, a1, a2, a3, bq[j][kb][0], bq[j][kb][1]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float nk = __uint_as_float(lds32(st + C::N0 + (ra + 8 * r) * 4));
        nv[h][r] = __uint_as_float(lds32(st + C::N0 + 128 + (ra + 8 * r) * 4));
#pragma unroll
        for (int j = 0; j < NT; ++j) sc[j][h][r] = (c[j][2 * r] + c[j][2 * r + 1]) * (nk * row_inv[j]);
      }
    }
    if (hidden) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (!aw_visible(t_blk[h] + gq + 8 * r, p_row[j], a.window, a.sinks)) sc[j][h][r] = -INFINITY;
          // a norm that no row sees takes no part in the power of two, whatever it is
          if (!aw_seen(t_blk[h] + gq + 8 * r, p_lo, p_hi, a.window, a.sinks)) nv[h][r] = 0.f;
        }
    }
    // ---- a larger value norm than any before moves their power of two
    float fix_all = 1.f;
    {
      float most = fmaxf(fmaxf(fabsf(nv[0][0]), fabsf(nv[0][1])), fmaxf(fabsf(nv[1][0]), fabsf(nv[1][1])));
      if (__any_sync(0xffffffffu, v_up == 0.f ? most > 0.f : most * v_up >= 64.f)) {
        most = 0.f;  // the largest finite one
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float v = fabsf(nv[h][r]);
            if (v < INFINITY) most = fmaxf(most, v);
          }
        most = fmaxf(warp_max8(most), v_up == 0.f ? 0.f : 32.f * v_inv);  // at least the power of two so far
        if (most > 0.f) {
          float inv;
          const float up = aw_pow2_for<5>(most, inv);
          fix_all = v_up == 0.f ? 1.f : up * v_inv;
          v_up = up;
          v_inv = inv;
        }
      }
    }
    // ---- reference maxima and sums; weights times norms as value + remainder
    uint32_t bp[NT][2][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float mx = warp_max8(fmaxf(fmaxf(sc[j][0][0], sc[j][0][1]), fmaxf(sc[j][1][0], sc[j][1][1])));
      w_low[j] *= fix_all;
      const bool move = mx > m_ref[j] + 8.0f || w_low[j] < AW_SMALL;  // from -inf by any score
      if (__any_sync(0xffffffffu, move || fix_all != 1.f)) {
        float fix = fix_all;
        const float top = fmaxf(m_ref[j], mx);
        float most = 0.f;  // of this tile, at `top` (NaN, from masked norms, left out)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) most = fmaxf(most, aw_exp2(sc[j][h][r] - top) * fabsf(nv[h][r] * v_up));
        most = warp_max8(most);
        const float sum = warp_max8(l_run[j]);  // within a factor of 8
        if (move) {
          const float old = aw_exp2(m_ref[j] - top);
          most = fmaxf(most, w_low[j] * old);  // (inf * 0 = NaN is left out)
          const float ref = aw_reference(top, sum * old, most), f = aw_exp2(m_ref[j] - ref);
          l_run[j] *= f;
          fix *= f;
          m_ref[j] = ref;
          w_low[j] = most;
        }
        // (the accumulator's columns 2 tq, 2 tq + 1 belong to this same row)
#pragma unroll
        for (int q = 0; q < NB; ++q)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][q][c] *= fix;
      }
      const float ref = m_ref[j] == -INFINITY ? 0.f : m_ref[j];  // nothing seen yet: weights exp2(-inf) = 0
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p = aw_exp2(sc[j][h][r] - ref);
          l_run[j] += p;  // of this lane's positions
          float w = p * (nv[h][r] * v_up);
          if (hidden && sc[j][h][r] == -INFINITY) w = 0.f;  // whatever the norm is
          const float hi = __half2float(__float2half_rn(w));
          bp[j][h][r] = aw_transpose(pack_half2(hi, w - hi));
        }
    }
    // ---- values
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4][VW];
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // positions 2 tq, 2 tq + 1, + 8, + 9 of the block
        const int row = 16 * h + 2 * tq + (q & 1) + 8 * (q >> 1), slot = (row & 1) * 16 + (row >> 1);
        const uint32_t at = st + C::V0 + slot * PV;
        if constexpr (PV == 64 || PV == 128) {
          constexpr int PER = PV == 64 ? 2 : 1;  // threads sharing a 16-byte chunk
          aw_lds<VT>(w[q], at + aw_v_chunk<PV>(slot, gq / PER) * 16 + (gq % PER) * VT, 0);
        } else {
          aw_lds<VT>(w[q], at + gq * VT, at + PV);
        }
      }
      auto product = [&](int mb, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816(acc[j][mb], a0, a1, a2, a3, bp[j][h][0], bp[j][h][1]);
      };
      if constexpr (VB == 3) {
#pragma unroll
        for (int mb = 0; mb < NB; ++mb) {
          const uint32_t l0 = lds32(aw_bits<6>(w[0], 6 * mb) * 256u + lut_v);
          const uint32_t l1 = lds32(aw_bits<6>(w[1], 6 * mb) * 256u + lut_v);
          const uint32_t l2 = lds32(aw_bits<6>(w[2], 6 * mb) * 256u + lut_v);
          const uint32_t l3 = lds32(aw_bits<6>(w[3], 6 * mb) * 256u + lut_v);
          product(mb, __byte_perm(l0, l1, 0x5410), __byte_perm(l0, l1, 0x7632), __byte_perm(l2, l3, 0x5410),
                  __byte_perm(l2, l3, 0x7632));
        }
      } else {
        // index bytes: a nibble of one position with the same nibble of the
        // next (low nibbles of every byte, then high ones)
        constexpr uint32_t LOWS = 0x0f0f0f0fu;
#pragma unroll
        for (int z = 0; z < VW; ++z) {
          const uint32_t e0 = (w[0][z] & LOWS) | ((w[1][z] << 4) & ~LOWS);
          const uint32_t o0 = ((w[0][z] >> 4) & LOWS) | (w[1][z] & ~LOWS);
          const uint32_t e1 = (w[2][z] & LOWS) | ((w[3][z] << 4) & ~LOWS);
          const uint32_t o1 = ((w[2][z] >> 4) & LOWS) | (w[3][z] & ~LOWS);
          constexpr int BY = VT < 4 ? VT : 4;  // bytes of a word
#pragma unroll
          for (int y = 0; y < BY; ++y) {
            if constexpr (VB == 2) {  // nibble = two dims: an M-block per nibble
              const uint2 u = lds64(aw_at(e0, lut_v, y)), v = lds64(aw_at(e1, lut_v, y));
              product(8 * z + 2 * y, u.x, u.y, v.x, v.y);
              const uint2 s = lds64(aw_at(o0, lut_v, y)), t = lds64(aw_at(o1, lut_v, y));
              product(8 * z + 2 * y + 1, s.x, s.y, t.x, t.y);
            } else {  // nibble = one dim: an M-block per byte
              product(4 * z + y, lds32(aw_at(e0, lut_v, y)), lds32(aw_at(o0, lut_v, y)), lds32(aw_at(e1, lut_v, y)),
                      lds32(aw_at(o1, lut_v, y)));
            }
          }
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
          a.ws_m[idx] = m_ref[j];
          a.ws_l[idx] = l;
        }
        if (m_ref[j] != -INFINITY) {
          float4* dst = reinterpret_cast<float4*>(a.ws_acc + idx * D + gq * (D / 8));
#pragma unroll
          for (int e = 0; e < D / 8; e += 4)
            dst[e / 4] = make_float4(x[e] * v_inv, x[e + 1] * v_inv, x[e + 2] * v_inv, x[e + 3] * v_inv);
        }
      }
      continue;
    }
    const float inv = l > 0.f ? v_inv * a.o_scale / l : (l == l ? 0.f : l);  // NaN where the sum is
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
// (Starting it while the partial kernel's last CTAs still run, by an early
// griddepcontrol.launch_dependents there, cost when it was tried: 16 x 8192
// positions 49.0 -> 51.3 us, 8 x 5 tokens 61.5 -> 63.0.)
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
      for (int s1 = 0; s1 < n; s1 += 8) {  // eight splits' loads in flight
        float v[8][E];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 u = s1 + k < n ? *reinterpret_cast<const float2*>(acc + (int64_t)(s1 + k) * D + e)
                                        : make_float2(0.f, 0.f);
            v[k][e] = u.x, v[k][e + 1] = u.y;
          }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float ws = __shfl_sync(0xffffffffu, w, (s1 + k) & 31);
          const bool some = s1 + k < n && ws != 0.f;  // an empty split has written no accumulator
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = some ? fmaf(ws, v[k][e], x[e]) : x[e];
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

// Which kernel takes a call. This one costs in proportion to the query rows per
// kv head, the tensor-memory kernel the same up to 128 (d = 256) or 256 rows,
// but more to start; so that one takes 64 rows and more, this one fewer than 40
// (32 at d = 256), and between them the estimates below decide (us; `seen`
// positions at most). They were fitted to, and checked at, sizes in that range
// only, so they stop at 64 rows, although one short sequence loses there: 64 rows over
// 300 positions take about 15 us on this kernel and 22.7 on that one. `rows` is
// that of the longest sequence: one kernel and one number of splits serve all of
// a call (32 sequences over 8192 positions, a chunk of 2048 tokens in one and a
// token in each other: 965 us, the chunk alone 491, the 31 tokens alone 111).
// Measured, this kernel / that one, keys 4 and values 2 bits:
//   d = 128, 8 sequences x 4 kv heads x 8000: 32 rows 56 / 62, 40 rows 68 / 63, 64 rows 105 / 63
//            32 x 8 x 1000: 40 rows 60 / 81, 48 rows 97 / 81;  32 x 8 x 2000: 106 / 122, 169 / 123
//            8 x 8 x 2000: 40 rows 46 / 39;  1 x 8 x 300: 48 rows 15 / 23;  1 x 8 x 1000: 48 rows 18 / 25
//   d = 64 (3 / 3 bits), 32 x 8 x 1000: 40 rows 60 / 64, 48 rows 97 / 64;  8 x 8 x 4000: 40 rows 58 / 56
//   d = 256, 8 x 4 x 4000: 24 rows 53 / 66, 32 rows 72 / 65;  2 x 4 x 4000: 32 rows 33 / 37, 48 rows 41 / 39
static bool window_takes_tc(int64_t rows, int64_t units, int d, int64_t seen) {
  if (rows < (d == 256 ? 32 : 40)) return false;
  if (rows >= 64) return true;
  const double here = 12.0 + (d == 64 ? 3.7e-5 : d == 128 ? 4.6e-5 : 1.2e-4) * (double)(units * ((rows + 7) / 8)) * seen;
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(148 / units, (seen + 255) / 256));
  const int64_t waves = (units * splits + 147) / 148;
  const double there = 6.0 + waves * (12.0 + (d == 64 ? 0.019 : d == 128 ? 0.023 : 0.05) * seen / splits);
  return there < here;
}

// With at most 128 query rows per kv head, so one row tile of head_dim 64 or 128
// in use, the tensor-memory kernel's two row tiles hold the same rows and take
// alternate tiles of positions, each as a split of its own, from this many
// positions on. Measured when this was built, d = 128 (one row tile / halves): 8 sequences of 8000
// positions 78 / 68 us, 32 sequences of 2048 135 / 130, of 1024 86 / 86, of
// 512 63 / 68 (twice the partial results to merge).
constexpr int64_t AW_HALVES = 1024;

// Splits of a call, from the sizes alone, so that the workspace is too: this
// kernel, enough warps to fill the SMs twice over, at least one step of 32
// positions each; the tensor-memory kernel, one CTA per SM, at least four
// tiles of 64 each.
struct WindowPlan {
  int n_split;
  bool tc, halves;
};
static WindowPlan window_plan(int B, int hq, int hkv, int max_q, int d, int64_t s_max, int64_t window, int64_t sinks) {
  WindowPlan p{};
  const int64_t rows = (int64_t)max_q * (hq / hkv);
  int64_t seen = s_max;
  if (window > 0)  // (s_max is below 2^31; larger limits are none)
    seen = std::min(seen, std::min<int64_t>(window, INT_MAX) + std::min<int64_t>(sinks, INT_MAX) + max_q + 2 * ATT_BLOCK);
  p.tc = window_takes_tc(rows, (int64_t)B * hkv, d, seen);
  const bool tc = p.tc;
  const int64_t rt = tc ? tq_window_tc_rows(d) : rows > 4 && d <= 128 ? 8 : 4;
  const int64_t tiles = (rows + rt - 1) / rt;
  const int64_t units = (int64_t)B * hkv * tiles;
  const int64_t steps = tc ? (seen + 255) / 256 : (seen + AW_TILE - 1) / AW_TILE;
  const int64_t slots = tc ? 148 : 148 * (d * rt <= 512 ? 16 : 8);
  p.n_split = (int)std::max<int64_t>(1, std::min<int64_t>(slots / units, steps));
  p.halves = tc && d <= 128 && rows <= 128 && seen >= AW_HALVES;
  if (p.halves) p.n_split *= 2;
  return p;
}

template <int D, int KB, int VB, int NT>
static cudaError_t launch_window_t(const AwArgs& a, cudaStream_t st) {
  using C = AwCfg<D, KB, VB, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = aw_allow_smem(reinterpret_cast<const void*>(window_partial_kernel<D, KB, VB, NT>), AW_SMEM, done);
  if (e != cudaSuccess) return e;
  const int64_t gx = ((int64_t)a.n_split * a.hkv + C::WARPS - 1) / C::WARPS;
  const int64_t gy = ((int64_t)a.max_q * a.g + 4 * NT - 1) / (4 * NT);
  if (gx > 0x7fffffff || gy > 65535) return cudaErrorNotSupported;
  window_partial_kernel<D, KB, VB, NT><<<dim3((unsigned)gx, (unsigned)gy, a.B), C::WARPS * 32, AW_SMEM, st>>>(a);
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
  const int ns = window_plan(B, hq, hkv, max_q, head_dim, s_max, window, sinks).n_split;
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
  const WindowPlan plan = window_plan(B, hq, hkv, max_q, d, s_max, window, sinks);
  a.n_split = plan.n_split;
  a.halves = plan.halves;
  const size_t rows = (size_t)n_tok * hq * a.n_split;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_m = reinterpret_cast<float*>(ws);
  a.ws_l = reinterpret_cast<float*>(ws + align16(rows * 4));
  a.ws_acc = reinterpret_cast<float*>(ws + 2 * align16(rows * 4));
  a.err = tq_error_word();
  if (!a.err) return TQ_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  if (plan.tc) {
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
