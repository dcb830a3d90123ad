// Windowed attention over packed caches for many query rows per kv head
// (prompt chunks, drafted tokens of wide head groups) on the fifth-generation
// tensor cores. The mathematics, the rotation of queries and output and the
// precision are those of tq_attend_window.cu; here the codes become fp16
// tiles in shared memory once and serve MT x 128 query rows.
//
// A CTA takes MT tiles of 128 query rows (row = token x query head of the
// group) of one kv head and walks over the 64-position tiles that they see
// (four 16-position blocks of the list sinks, window). Roles:
//  * 4 warps turn key codes into fp16 levels and write them as a K-major,
//    128-byte-swizzled operand [64 positions x d]. Codes of 2 and 4 bits are
//    looked up by byte permutes (no shared memory, whose ports the products
//    need: 8 x 5 tokens at 4 bits 67.5 -> 65.9 us against tables), 3-bit codes
//    in pairs from a table of 16 lane copies;
//  * 4 warps do the same for the values, transposed, [d x 64 positions]: a
//    thread takes 8 positions x 8 neighbouring dims, whose codes are one word
//    per position, and writes dim 8 dg + j to row j d/8 + dg (then the 8
//    lanes of a store phase hit 8 different bank groups). The accumulator's
//    columns come out in that order; a Hadamard transform commutes with such
//    a permutation of index bits, so the final rotation is done in it;
//  * a spare warp puts the tiles' norms and positions into a ring of slots;
//  * one warp per row tile issues tcgen05.mma: S = (Q_hi + Q_lo) K^T into
//    tensor memory, and O += (P_hi + P_lo) V with P read from tensor memory;
//  * 4 warps per row tile, one row per thread: scores from tensor memory,
//    times the key norm, running maximum, weights times value norms as fp16
//    value + remainder back to tensor memory, over the scores. The reference
//    of the weights moves only when a weight times the tile's norms could
//    pass 2^14 (a score 2^8 above it where the tile holds the largest norm) or the
//    row's products with the norms are small (aw_reference; exact: sum and
//    accumulator share it), so the accumulator is rescaled rarely.
// Scores are double-buffered: the next tile's S is computed while the
// softmax works on the current one. Calls whose rows fit one row tile may have
// it twice (`halves`): both hold the same rows, and each walks over every
// other tile of positions as a split of its own, so that two softmax groups
// work on one set of rows.
//
// Bound: per row tile and 64 positions 4 x 64 x 128 x d multiply-adds (scores
// and values, each with its remainder). At d = 128 the 16 score products take
// 763 cycles when nothing else runs (48 each: reading 128 + 64 operand rows
// from shared memory, not the 32 of the arithmetic) and the 8 value products
// 502, so two row tiles need 2540 cycles; beside them an exponential and about
// 9 other instructions per score and the codes' conversion (about 1000 warp
// instructions, shared by the row tiles). Measured, 2 x 2048 tokens of 32 query
// and 8 kv heads of 128 within 4096 + 64 positions, keys 4 and values 2 bits:
// 614 to 635 us a call on different GPUs (945 k cycles), 0.89 PFLOP/s with the
// remainders counted. A CTA's loop takes
// about 3700 cycles per 64 positions, of which a softmax warp works 3300 (some
// 550 instructions at 6 cycles each: 20 warps, a fifth of the wait for
// instructions; issue slots 54 %, tensor pipe 50 %), so the softmax of a row
// tile is the bound, not the products; its start took 12 000 to 16 000 cycles
// (8 000 to 12 000 of them the rotation of the query rows, before it ran in
// packed additions: 626 -> 616 us then, and 66 -> 61.5 below) and its end 9 000; 512
// CTAs leave 148 SMs 3.46 waves. 8 x 5 tokens of 8 query heads per kv head over
// 8000 positions, 4 bits: 63.5 us (two softmax groups and the value conversion,
// 2000 cycles a tile, both take about 4000 cycles per two tiles). Loading codes
// one more tile ahead changes nothing.
#include <climits>
#include <cmath>
#include <type_traits>

#include "tq_attend_window.cuh"
#include "tq_umma.cuh"

namespace tq {

constexpr int TW_TP = 64;       // positions of a tile
constexpr int TW_SLOTS = 8;     // norm slots in flight
constexpr int TW_TMEM = 512;

// Norms and positions of one tile.
struct TwSlot {
  float nk[TW_TP];
  float nv[TW_TP];   // times the power of two of the tile
  float lg[TW_TP];   // log2 |nv|
  int blk_t[4];      // first position of each 16-position block (INT_MAX - 64: none)
  int t_min, t_max;  // first and last position
  float v_up, v_inv; // this tile's power of two and its inverse
  uint32_t odd[2];   // positions whose value norm is infinite or NaN (0 in nv)
  float nv_min;      // smallest finite |nv| that a row sees
  float head;        // weights up to 2^head times the tile's norms stay below 2^14
};

template <int D, int KB, int VB>
struct TwCfg {
  static constexpr int MT = D == 256 ? 1 : 2;    // row tiles of 128
  static constexpr int NBUF = D == 256 ? 1 : 2;  // key operands, value operands in shared memory
  static constexpr int SM_WARPS = 4 * MT;
  // softmax, conversion and issuing warpgroups (of the last, MT warps work)
  static constexpr int WARPS = SM_WARPS + 8 + 4;
  // registers of a thread by role: a softmax row (64 scores and their packed
  // weights) needs more than the launch's share of the register file. Per
  // scheduler MT R_SM + 2 R_CV + R_MMA is the MT + 3 launched warps' share
  // (96 at MT = 2, 128 at MT = 1) or less.
  static constexpr int R_SM = MT == 2 ? 144 : 160, R_CV = MT == 2 ? 64 : 120, R_MMA = MT == 2 ? 64 : 96;
  static_assert(MT * R_SM + 2 * R_CV + R_MMA <= (MT + 3) * (MT == 2 ? 96 : 128), "register shares");
  static constexpr int Q_PART = D * 256;         // [128 rows x d] fp16
  static constexpr int KV = D * TW_TP * 2;       // [64 x d] fp16
  // tables of the 3-bit codes (one serves both); 2 and 4 bits go by byte permutes
  static constexpr int K_TAB = KB == 3 ? 64 * 64 : 0;
  static constexpr int V_TAB = VB == 3 && KB != 3 ? 64 * 64 : 0;
  static constexpr int Q0 = 0;
  static constexpr int K0 = Q0 + 2 * MT * Q_PART;
  static constexpr int V0 = K0 + NBUF * KV;
  static constexpr int T0 = V0 + NBUF * KV;
  static constexpr int N0 = T0 + K_TAB + V_TAB;
  static constexpr int BAR = N0 + TW_SLOTS * (int)sizeof(TwSlot);
  static constexpr int BARS = 4 * NBUF + TW_SLOTS + MT * 8;
  static constexpr int SLOT = BAR + BARS * 8;
  static constexpr int NEED = SLOT + 16 + 1024;
  // one CTA per SM also where less shared memory would do: each takes all of
  // the SM's tensor memory
  static constexpr int BYTES = NEED < 120 * 1024 ? 120 * 1024 : NEED;
  static_assert(BYTES <= 232448, "shared memory of a CTA");
};

// In-register Hadamard transform of 64 values (natural order, no scaling), two
// in a register pair: all stages but the first are packed additions.
TQ_DEV void wht64(f2 (&x)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = make_float2(x[e].x + x[e].y, x[e].x - x[e].y);
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if ((e & h) == 0) {
        const f2 u = x[e], v = x[e + h];
        x[e] = add2(u, v);
        x[e + h] = sub2(u, v);
      }
}

// fp16 levels of the two 2-bit codes at bits 0 and 8 of x (other bits ignored):
// a byte permute of the four levels in two words, code c taking bytes 2c, 2c + 1.
TQ_DEV uint32_t tw_levels2(uint32_t x, uint32_t lo, uint32_t hi) {
  return __byte_perm(lo, hi, (x & 0x0303u) * 0x22u + 0x1010u);
}

// The same for 4-bit codes, eight in a word. The codebook is symmetric (level
// 15 - c is minus level c), so the byte permutes look up the bytes of the eight
// positive levels by c - 8 or 7 - c, and the sign is put into the high bytes.
struct TwLevels16 {
  uint32_t l0, l1, h0, h1;  // low and high bytes of levels 8 ... 15
};
TQ_DEV TwLevels16 tw_table16(const uint16_t* lev) {
  TwLevels16 t;
  const uint32_t a = lev[8] | (uint32_t)lev[9] << 16, b = lev[10] | (uint32_t)lev[11] << 16;
  const uint32_t c = lev[12] | (uint32_t)lev[13] << 16, d = lev[14] | (uint32_t)lev[15] << 16;
  t.l0 = __byte_perm(a, b, 0x6420);
  t.h0 = __byte_perm(a, b, 0x7531);
  t.l1 = __byte_perm(c, d, 0x6420);
  t.h1 = __byte_perm(c, d, 0x7531);
  return t;
}
TQ_DEV void tw_levels8(uint32_t x, const TwLevels16& t, uint32_t (&w)[4]) {
  const uint32_t neg = ~x & 0x88888888u;                          // bit 3 of the negative levels' codes
  const uint32_t m = (x ^ (neg - (neg >> 3))) & 0x77777777u;      // c - 8 or 7 - c
  const uint32_t se = (neg << 4) & 0x80808080u, so = neg & 0x80808080u;  // signs of the even, the odd codes
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t sel = k ? m >> 16 : m;
    const uint32_t lo = __byte_perm(t.l0, t.l1, sel);
    const uint32_t hi = __byte_perm(t.h0, t.h1, sel) | __byte_perm(se, so, k ? 0x7362 : 0x5140);
    w[2 * k] = __byte_perm(lo, hi, 0x5140);
    w[2 * k + 1] = __byte_perm(lo, hi, 0x7362);
  }
}

// Bounded wait for phase `parity` of a barrier. Twenty warps polling as
// mbar_wait_bounded does (a clock read and a 64-bit comparison each time) took
// half of the SM's issue slots, so this one counts its tries, and with NS > 0
// sleeps between them (roles that run ahead of the others). False after
// `tries` of them (a second or more).
constexpr uint32_t TW_TRIES = 30000000u;
constexpr int TW_NAP = 64;
template <int NS = 0>
TQ_DEV bool tw_wait(uint32_t bar, uint32_t parity, uint32_t tries) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (uint32_t n = 0; n < tries; ++n) {
    if (NS > 0) __nanosleep(NS);
    if (mbar_try_wait(bar, parity)) return true;
  }
  return false;
}

TQ_DEV float tw_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Weights 2^(x row_inv - ref) of a row's 64 scores; returns their sum and
// stores weight x value norm as fp16 value (columns 0-31 from `col`) and
// remainder (32-63). (A masked score's weight is 0 times a finite norm.)
TQ_DEV float tw_weights(const float (&x)[64], const float* nv, float row_inv, float ref, uint32_t col) {
  f2 sum = make_float2(0.f, 0.f);
  const f2 scale = make_float2(row_inv, row_inv), shift = make_float2(-ref, -ref);
#pragma unroll
  for (int c0 = 0; c0 < 64; c0 += 32) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      const float4 n4 = *reinterpret_cast<const float4*>(nv + c0 + c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = c0 + c + 2 * k;
        const f2 z = fma2(make_float2(x[e], x[e + 1]), scale, shift);
        const f2 p = make_float2(aw_exp2(z.x), aw_exp2(z.y));
        sum = add2(sum, p);
        const f2 w = mul2(p, k ? make_float2(n4.z, n4.w) : make_float2(n4.x, n4.y));
        const uint32_t h2 = pack_half2(w.x, w.y);
        const f2 r = sub2(w, __half22float2(*reinterpret_cast<const __half2*>(&h2)));
        hi[c / 2 + k] = h2;
        lo[c / 2 + k] = pack_half2(r.x, r.y);
      }
    }
    tmem_st16(col + (uint32_t)(c0 / 2), hi);
    tmem_st16(col + 32u + (uint32_t)(c0 / 2), lo);
  }
  return sum.x + sum.y;
}

// The visible ones (aw_visible) of the 16 positions from t0 on, as bits.
TQ_DEV uint32_t tw_visible16(int t0, int p, int window, int sinks) {
  const int seen = min(max(p - t0 + 1, 0), 16), before = min(max(max(p - window + 1, 0) - t0, 0), 16),
            first = min(max(sinks - t0, 0), 16);
  return ((1u << seen) - 1u) & (~((1u << before) - 1u) | ((1u << first) - 1u));
}

// log2 of the largest |weight x value norm| of a row in a tile at reference 0
// (masked scores are -inf; NaN ones are left out). In logarithms: with 64
// exponentials from a rolled loop over tensor memory an evaluation took the
// warp some 6000 cycles, and 2 x 2048 tokens whose norms spread by e^1 734 us
// instead of 595 (by e^0.2 583 and 593: the longer code costs that much).
TQ_DEV float tw_largest(const float (&x)[64], const float* lg, float row_inv) {
  const f2 scale = make_float2(row_inv, row_inv);
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int c = 0; c < 64; c += 4) {
    const float4 l = *reinterpret_cast<const float4*>(lg + c);
    const f2 u = fma2(make_float2(x[c], x[c + 1]), scale, make_float2(l.x, l.y));
    const f2 v = fma2(make_float2(x[c + 2], x[c + 3]), scale, make_float2(l.z, l.w));
    m0 = tw_max3(m0, u.x, u.y);
    m1 = tw_max3(m1, v.x, v.y);
  }
  return fmaxf(m0, m1);
}

template <int N>
TQ_DEV void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
TQ_DEV void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(TwCfg<D, KB, VB>::WARPS * 32, 1)
    window_tc_kernel(const __grid_constant__ AwArgs a) {
  using C = TwCfg<D, KB, VB>;
  constexpr int MT = C::MT, NBUF = C::NBUF;
  constexpr int PK = D * KB / 8, PV = D * VB / 8;
  extern __shared__ uint8_t raw_smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int b = blockIdx.z;
  const int c_split = blockIdx.x / a.hkv, hk = blockIdx.x - c_split * a.hkv;
  const bool halves = MT == 2 && a.halves;
  const AwSeq sq = aw_sequence(a, b, blockIdx.x == 0 && blockIdx.y == 0 && tid == 0);
  const int rows = sq.n * a.g, r0 = blockIdx.y * (128 * MT);
  if (r0 >= rows) return;

  // ---- the tiles of this CTA
  const int r1 = min(r0 + 128 * MT, rows) - 1;
  const int p_lo = aw_position(sq, r0 / a.g), p_hi = aw_position(sq, r1 / a.g);
  const AwBlocks bl = aw_blocks(p_lo, p_hi, a.window, a.sinks);
  const int tiles = (bl.n + 3) / 4, n_cta = halves ? a.n_split / 2 : a.n_split;
  const int share = (tiles + n_cta - 1) / n_cta;
  const int tile0 = c_split * share, cnt = max(0, min(share, tiles - tile0));

  const uint32_t raw = smem_u32(raw_smem), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = raw_smem + (base - raw);
  const uint32_t bar = base + C::BAR;
  const uint32_t k_full = bar, k_empty = k_full + 8 * NBUF, v_full = k_empty + 8 * NBUF, v_empty = v_full + 8 * NBUF,
                 n_full = v_empty + 8 * NBUF, s_full = n_full + 8 * TW_SLOTS,  // [MT][2]
                 p_full = s_full + 16 * MT, o_done = p_full + 16 * MT, mma_end = o_done + 16 * MT, q_full = mma_end + 8 * MT;
  if (tid == 0) {
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(k_full + 8 * i, 128 + 32);  // the key warps and the norm warp
      mbar_init(k_empty + 8 * i, halves ? 1 : MT);  // the issuers that read it
      mbar_init(v_full + 8 * i, 128);
      mbar_init(v_empty + 8 * i, halves ? 1 : MT);
    }
    for (int i = 0; i < TW_SLOTS; ++i) mbar_init(n_full + 8 * i, 32);
    for (int i = 0; i < 2 * MT; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(o_done + 8 * i, 1);
    }
    for (int i = 0; i < MT; ++i) {
      mbar_init(mma_end + 8 * i, 1);
      mbar_init(q_full + 8 * i, 128);
    }
    fence_mbar_init();
  }
  constexpr int MMA_WARP = C::SM_WARPS + 8;
  if (warp == MMA_WARP) {
    tmem_alloc(base + C::SLOT, TW_TMEM);
    tmem_relinquish();
  }
  // ---- tables: pairs of codes -> two fp16 levels, 16 copies
  {
    uint32_t* t = reinterpret_cast<uint32_t*>(sm + C::T0);
    for (int e = tid; e < C::K_TAB / 4; e += blockDim.x) {
      const int f = e >> 4;
      t[e] = a.k_lev[f & ((1 << KB) - 1)] | (uint32_t)a.k_lev[f >> KB] << 16;
    }
    t += C::K_TAB / 4;
    for (int e = tid; e < C::V_TAB / 4; e += blockDim.x) {
      const int f = e >> 4;
      t[e] = a.v_lev[f & ((1 << VB) - 1)] | (uint32_t)a.v_lev[f >> VB] << 16;
    }
  }
  // ---- query rows, as they are, into the space of the key and value operands
  // (row r at r x 2 d bytes, 16-byte chunks swizzled within 128 bytes)
  static_assert(C::NBUF * 2 * C::KV == 128 * MT * D * 2, "room for the raw query rows");
  {
    constexpr int CH = D / 8;  // chunks of a row
    const int n_rows = min(128 * MT, rows - r0);
    for (int e = tid; e < n_rows * CH; e += C::WARPS * 32) {
      const int rr = e / CH, c = e % CH;
      const int i = (r0 + rr) / a.g, h = r0 + rr - i * a.g;
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.q + ((sq.q0 + i) * a.hq + hk * a.g + h) * D) + c);
      *reinterpret_cast<uint4*>(sm + C::K0 + rr * (2 * D) + ((c & ~7) << 4) + (((c ^ rr) & 7) << 4)) = w;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(sm + C::SLOT), 0);
  // row tile t: scores / weights at columns 256 t + {0, 64}, accumulator at 256 t + 128
  constexpr uint32_t FULL = 0xffffffffu;

  if (warp >= C::SM_WARPS && warp < MMA_WARP) {
    regs_down<C::R_CV>();
    const bool keys = warp < C::SM_WARPS + 4;
    const int w4 = (warp - C::SM_WARPS) & 3;
    // the query rows must have been read before operands take their place
    bool ok = true;
    for (int t = 0; t < MT; ++t) ok = ok && tw_wait<TW_NAP>(q_full + 8 * t, 0, TW_TRIES);
    ok = __all_sync(FULL, ok);
    if (!ok && lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
    auto entry = [&](int i, int q) {  // table entry of block q of tile i
      return aw_block_entry(a, b, aw_block(bl, min(4 * (tile0 + i) + q, bl.n - 1)));
    };
    if (keys) {
      // ---- key codes -> K operands: row 16 w4 + lane % 16, half (lane / 16) of its dims
      constexpr int HB = PK / 2, HW = HB / 4;
      const int row = 16 * w4 + (lane & 15), half = lane >> 4;
      [[maybe_unused]] const uint32_t lut = base + C::T0 + (lane & 15) * 4u;
      [[maybe_unused]] const uint32_t k_lo = a.k_lev[0] | (uint32_t)a.k_lev[1] << 16,
                                      k_hi = a.k_lev[2] | (uint32_t)a.k_lev[3] << 16;
      [[maybe_unused]] const TwLevels16 k_t = tw_table16(a.k_lev);
      uint32_t cw[HW];
      int next = 0;  // table entry of the tile after the loaded one
      auto fetch = [&](int i) {
        const int j = aw_block(bl, min(4 * (tile0 + i) + w4, bl.n - 1));
        const int64_t c_row = (aw_entry_row(a, b, next) + min(row & 15, sq.ctx - 1 - j * ATT_BLOCK)) * a.hkv + hk;
        aw_load<HB, HW>(cw, a.k_packed + c_row * PK, half * HB, PK);
        if (i + 1 < cnt) next = entry(i + 1, w4);
      };
      if (cnt > 0) {
        next = entry(0, w4);
        fetch(0);
      }
      for (int i = 0; i < cnt && ok; ++i) {
        const int buf = i % NBUF;
        if (i >= NBUF) ok = __all_sync(FULL, tw_wait<TW_NAP>(k_empty + 8 * buf, ((i / NBUF) - 1) & 1, TW_TRIES));
        if (!ok) {
          if (lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
          break;
        }
        uint8_t* dst = sm + C::K0 + buf * C::KV + row * 128;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {  // 8 dims each
          uint32_t w[4];
          if constexpr (KB == 2) {
            const uint32_t codes = cw[c / 2] >> (16 * (c & 1));
            uint32_t p[4];  // levels of codes q, q + 4
#pragma unroll
            for (int q = 0; q < 4; ++q) p[q] = tw_levels2(codes >> (2 * q), k_lo, k_hi);
            w[0] = __byte_perm(p[0], p[1], 0x5410);
            w[1] = __byte_perm(p[2], p[3], 0x5410);
            w[2] = __byte_perm(p[0], p[1], 0x7632);
            w[3] = __byte_perm(p[2], p[3], 0x7632);
          } else if constexpr (KB == 4) {
            tw_levels8(cw[c], k_t, w);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = lds32(aw_bits<2 * KB>(cw, (4 * c + k) * 2 * KB) * 64u + lut);
          }
          const int chunk = half * (D / 16) + c;  // 16-byte chunk of the row: atom chunk / 8
          *reinterpret_cast<uint4*>(dst + (chunk >> 3) * (TW_TP * 128) + (((chunk & 7) ^ (row & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (i + 1 < cnt) fetch(i + 1);
        fence_proxy_async_smem();
        mbar_arrive(k_full + 8 * buf);
      }
    } else {
      // ---- value codes -> V operands: positions 8 pg ..., dims 8 dg ... of a thread
      constexpr int DG = D / 8, PASS = D == 256 ? 2 : 1;  // 128 threads cover 128 / DG groups of 8 positions
      const int t = w4 * 32 + lane, dg = t % DG, pg0 = t / DG;
      const bool on = D > 64 || pg0 < 8;
      [[maybe_unused]] const uint32_t lut = base + C::T0 + C::K_TAB * (KB == VB ? 0 : 1) + (lane & 15) * 4u;
      [[maybe_unused]] const uint32_t v_lo = a.v_lev[0] | (uint32_t)a.v_lev[1] << 16,
                                      v_hi = a.v_lev[2] | (uint32_t)a.v_lev[3] << 16;
      [[maybe_unused]] const TwLevels16 v_t = tw_table16(a.v_lev);
      uint32_t vw[PASS][8];
      int next[PASS];
      auto fetch = [&](int i) {
#pragma unroll
        for (int q = 0; q < PASS; ++q) {
          const int pg = pg0 + q * (128 / DG);
          const int j = aw_block(bl, min(4 * (tile0 + i) + (pg >> 1), bl.n - 1));
          const int64_t row0 = aw_entry_row(a, b, next[q]);
          const int most = sq.ctx - 1 - j * ATT_BLOCK;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t w[1];
            const int64_t v_row = (row0 + min(8 * (pg & 1) + k, most)) * a.hkv + hk;
            aw_load<VB, 1>(w, a.v_packed + v_row * PV, dg * VB, PV);
            vw[q][k] = w[0];
          }
          if (i + 1 < cnt) next[q] = entry(i + 1, pg >> 1);
        }
      };
      if (cnt > 0 && on) {
#pragma unroll
        for (int q = 0; q < PASS; ++q) next[q] = entry(0, (pg0 + q * (128 / DG)) >> 1);
        fetch(0);
      }
      for (int i = 0; i < cnt && ok; ++i) {
        const int buf = i % NBUF;
        if (i >= NBUF) ok = __all_sync(FULL, tw_wait<TW_NAP>(v_empty + 8 * buf, ((i / NBUF) - 1) & 1, TW_TRIES));
        if (!ok) {
          if (lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
          break;
        }
        if (on) {
#pragma unroll
          for (int q = 0; q < PASS; ++q) {
            const int pg = pg0 + q * (128 / DG);
            uint8_t* dst = sm + C::V0 + buf * C::KV + dg * 128 + ((pg ^ (dg & 7)) << 4);
            if constexpr (VB == 2) {
              uint32_t pair[4];  // code bytes of two positions, interleaved: dims 0-3, then 4-7
#pragma unroll
              for (int k = 0; k < 4; ++k) pair[k] = __byte_perm(vw[q][2 * k], vw[q][2 * k + 1], 0x5140);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                uint32_t e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = tw_levels2(pair[k] >> (16 * (j >> 2) + 2 * (j & 3)), v_lo, v_hi);
                *reinterpret_cast<uint4*>(dst + j * DG * 128) = make_uint4(e[0], e[1], e[2], e[3]);
              }
            } else if constexpr (VB == 4) {
              constexpr uint32_t LOWS = 0x0f0f0f0fu;
#pragma unroll
              for (int odd = 0; odd < 2; ++odd) {  // dims 8 dg + odd, + 2, + 4, + 6
                uint32_t e[4][4];                  // of position pair k: its words for the four dims
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // codes of two positions side by side, dim by dim
                  const uint32_t x = vw[q][2 * k], y = vw[q][2 * k + 1];
                  tw_levels8(odd ? ((x >> 4) & LOWS) | (y & ~LOWS) : (x & LOWS) | ((y << 4) & ~LOWS), v_t, e[k]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  *reinterpret_cast<uint4*>(dst + (2 * j + odd) * DG * 128) =
                      make_uint4(e[0][j], e[1][j], e[2][j], e[3][j]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {  // dims 8 dg + 2 j, + 1
                uint32_t l[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) l[k] = lds32(((vw[q][k] >> (2 * VB * j)) & ((1u << 2 * VB) - 1u)) * 64u + lut);
                uint32_t e[4], o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  e[k] = __byte_perm(l[2 * k], l[2 * k + 1], 0x5410);
                  o[k] = __byte_perm(l[2 * k], l[2 * k + 1], 0x7632);
                }
                *reinterpret_cast<uint4*>(dst + (2 * j) * DG * 128) = make_uint4(e[0], e[1], e[2], e[3]);
                *reinterpret_cast<uint4*>(dst + (2 * j + 1) * DG * 128) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          }
          if (i + 1 < cnt) fetch(i + 1);
        }
        fence_proxy_async_smem();
        mbar_arrive(v_full + 8 * buf);
      }
    }
  } else if (warp >= MMA_WARP) {
    // ---- MMA issuer of row tile t
    regs_down<C::R_MMA>();
    const int t = warp - MMA_WARP;
    if (t < MT) {
      constexpr uint32_t ID_S = umma_idesc_f16(128, TW_TP), ID_O = umma_idesc_f16(128, D);
      const uint32_t s0 = tmem + 256u * t, o0 = s0 + 128u;
      const uint64_t q_desc = umma_desc_sw128(base + C::Q0 + 2 * t * C::Q_PART);
      const uint64_t k_desc = umma_desc_sw128(base + C::K0), v_desc = umma_desc_sw128(base + C::V0);
      const bool active = halves || r0 + 128 * t < rows;  // a row tile without rows only signals
      const int n = halves ? (cnt + 1 - t) / 2 : cnt;
      // the whole warp waits, one elected lane issues
      bool ok = __all_sync(FULL, tw_wait(q_full + 8 * t, 0, TW_TRIES));
      for (int j = 0; j <= n && ok; ++j) {  // this row tile's j-th tile of positions
        if (j < n) {
          const int i = halves ? 2 * j + t : j, buf = i % NBUF;
          ok = __all_sync(FULL, tw_wait(k_full + 8 * buf, (i / NBUF) & 1, TW_TRIES));
          if (!ok) break;
          tc_fence_after();
          const uint32_t s = s0 + 64u * (j & 1);
          if (elect_one()) {
            if (active) {
              const uint64_t kd = k_desc + ((uint32_t)(buf * C::KV) >> 4);
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                  umma_f16(s, q_desc + ((part * C::Q_PART + (ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                           kd + (((ks >> 2) * (TW_TP * 128) + (ks & 3) * 32) >> 4), ID_S, part + ks > 0);
            }
            umma_commit(s_full + 16 * t + 8 * (j & 1));
            umma_commit(k_empty + 8 * buf);
          }
          __syncwarp();
        }
        if (j > 0) {
          const int u = j - 1, i = halves ? 2 * u + t : u, buf = i % NBUF;
          ok = __all_sync(FULL, tw_wait(v_full + 8 * buf, (i / NBUF) & 1, TW_TRIES) &&
                                    tw_wait(p_full + 16 * t + 8 * (u & 1), (u >> 1) & 1, TW_TRIES));
          if (!ok) break;
          tc_fence_after();
          const uint32_t p = s0 + 64u * (u & 1);
          if (elect_one()) {
            if (active) {
              const uint64_t vd = v_desc + ((uint32_t)(buf * C::KV) >> 4);
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int ks = 0; ks < TW_TP / 16; ++ks)
                  umma_f16_ts(o0, p + (uint32_t)(32 * part + 8 * ks), vd + ((ks * 32) >> 4), ID_O,
                              part + ks > 0 || u > 0);
            }
            umma_commit(o_done + 16 * t + 8 * (u & 1));
            umma_commit(v_empty + 8 * buf);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
      if (elect_one()) umma_commit(mma_end + 8 * t);
      __syncwarp();
      if (!tw_wait(mma_end + 8 * t, 0, TW_TRIES) && lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
    } else if (t == 2) {
      // ---- norms and positions of the tiles, two positions per lane. A slot is
      // free again when the product two tiles back has read its keys: its
      // issuer had the weights of the tile two before that one in its row
      // tile's order, which is at most six tiles back.
      const int q = lane >> 4;
      float nk[2], nv[2];
      int next[2];
      auto entry = [&](int i, int h) {
        return aw_block_entry(a, b, aw_block(bl, min(4 * (tile0 + i) + 2 * h + q, bl.n - 1)));
      };
      auto fetch = [&](int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = aw_block(bl, min(4 * (tile0 + i) + 2 * h + q, bl.n - 1));
          const int64_t n_row =
              (aw_entry_row(a, b, next[h]) + min(lane & 15, sq.ctx - 1 - j * ATT_BLOCK)) * a.hkv + hk;
          nk[h] = __ldg(a.k_norms + n_row);
          nv[h] = __ldg(a.v_norms + n_row);
          if (i + 1 < cnt) next[h] = entry(i + 1, h);
        }
      };
      if (cnt > 0) {
        next[0] = entry(0, 0);
        next[1] = entry(0, 1);
        fetch(0);
      }
      float v_most = 0.f, v_up = 1.f, v_inv = 1.f;
      for (int i = 0; i < cnt; ++i) {
        const int buf = i % NBUF;
        if (i >= NBUF && !__all_sync(FULL, tw_wait<TW_NAP>(k_empty + 8 * buf, ((i / NBUF) - 1) & 1, TW_TRIES))) {
          if (lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
          break;
        }
        TwSlot& s = reinterpret_cast<TwSlot*>(sm + C::N0)[i % TW_SLOTS];
        float most = 0.f, least = INFINITY;
        int t_min = INT_MAX, t_max = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = 4 * (tile0 + i) + 2 * h + q;
          const int at = m < bl.n ? aw_block(bl, m) * ATT_BLOCK : INT_MAX - 64;
          // a norm that no row sees takes no part in the power of two, whatever it is
          const bool seen = aw_seen(at + (lane & 15), p_lo, p_hi, a.window, a.sinks);
          if (!seen) nv[h] = 0.f;
          const float v = fabsf(nv[h]);
          if (v < INFINITY) {
            most = fmaxf(most, v);
            if (seen) least = fminf(least, v);
          }
          t_min = min(t_min, at);
          t_max = max(t_max, at + ATT_BLOCK - 1);
          if ((lane & 15) == 0) s.blk_t[2 * h + q] = at;
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
          most = fmaxf(most, __shfl_xor_sync(FULL, most, m));
          least = fminf(least, __shfl_xor_sync(FULL, least, m));
        }
        t_min = min(t_min, __shfl_xor_sync(FULL, t_min, 16));
        t_max = max(t_max, __shfl_xor_sync(FULL, t_max, 16));
        if (most > v_most) {
          v_most = most;
          v_up = aw_pow2_for<5>(most, v_inv);  // weights reach 2^8: 2^14 in fp16
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool fine = fabsf(nv[h]) < INFINITY;
          s.nk[32 * h + lane] = nk[h];
          const float n = fine ? nv[h] * v_up : 0.f;
          s.nv[32 * h + lane] = n;
          s.lg[32 * h + lane] = __log2f(fabsf(n));
          const uint32_t odd = __ballot_sync(FULL, !fine);
          if (lane == 0) s.odd[h] = odd;
        }
        if (lane == 0) {
          s.t_min = t_min;
          s.t_max = t_max;
          s.v_up = v_up;
          s.v_inv = v_inv;
          s.nv_min = least * v_up;
          s.head = (float)min(13 - ((int)(__float_as_uint(most * v_up) >> 23) - 127), 30);
        }
        if (i + 1 < cnt) fetch(i + 1);
        mbar_arrive(n_full + 8 * (i % TW_SLOTS));
        mbar_arrive(k_full + 8 * buf);
      }
    }
  } else {
    regs_up<C::R_SM>();
    // ---- rotated queries, one row per softmax thread
    const int mt = warp >> 2;  // row tile
    const int r_tile = tid & 127, r_cta = halves ? r_tile : tid, r = r0 + r_cta;
    const bool row_ok = r < rows;
    const int q_i = row_ok ? r / a.g : 0, q_h = row_ok ? r - q_i * a.g : 0;
    const int64_t out_row = (sq.q0 + q_i) * a.hq + hk * a.g + q_h;
    float row_inv = 1.f;
    if (row_ok) {
      const uint8_t* src = sm + C::K0 + r_cta * (2 * D);
      const int sw = (r_cta & 7) << 4;
      f2 s2 = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int e = 0; e < D / 8; ++e) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + ((e & ~7) << 4) + (((e & 7) << 4) ^ sw));
        const uint32_t hw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hw[c]));
          s2 = fma2(f, f, s2);
        }
      }
      const float ss = s2.x + s2.y;
      // no rotated coordinate exceeds sqrt(d) |q|: that bound is put just below 2^15
      const float up = aw_pow2_for<14>(sqrtf(ss * (float)D) * a.q_scale, row_inv);
      const float qs = a.q_scale * up;
#pragma unroll 1
      for (int hf = 0; hf < D / 64; ++hf) {
        f2 x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int m = 0; m < D / 64; ++m) {
          const float sg1 = (__popc(m & hf) & 1) ? -1.f : 1.f;
          const f2 sg = make_float2(sg1, sg1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + (m << 7) + ((e << 4) ^ sw));
            const uint32_t hw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t s = hw[c] ^ a.k_sign_h2[32 * m + 4 * e + c];
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&s));
              x[4 * e + c] = fma2(sg, f, x[4 * e + c]);
            }
          }
        }
        wht64(x);
        uint8_t* dst = sm + C::Q0 + 2 * mt * C::Q_PART + hf * 16384 + r_tile * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const f2 u = mul2(x[4 * c + k], make_float2(qs, qs));
            hi[k] = pack_half2(u.x, u.y);
            const f2 r = sub2(u, __half22float2(*reinterpret_cast<const __half2*>(&hi[k])));
            lo[k] = pack_half2(r.x, r.y);
          }
          const int off = (c ^ (r_tile & 7)) << 4;
          *reinterpret_cast<uint4*>(dst + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + C::Q_PART + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    }
    if (!row_ok) {  // rows behind the last: scores of 0
      uint4* dst = reinterpret_cast<uint4*>(sm + C::Q0 + 2 * mt * C::Q_PART + r_tile * 128);
      for (int e = 0; e < 2 * (D / 64); ++e)
#pragma unroll
        for (int c = 0; c < 8; ++c) dst[e * (16384 / 16) + c] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    mbar_arrive(q_full + 8 * mt);
    // ---- softmax of one row per thread
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s0 = tmem + 256u * mt + lane_base, o0 = s0 + 128u;
    const int rw0 = r0 + 32 * (halves ? warp & 3 : warp), rw1 = min(rw0 + 31, rows - 1);  // rows of this warp
    const bool any_row = rw0 < rows;
    const int pw_lo = any_row ? aw_position(sq, rw0 / a.g) : -1, pw_hi = any_row ? aw_position(sq, rw1 / a.g) : -1;
    const int p_row = row_ok ? aw_position(sq, q_i) : pw_hi;
    float m_ref = -INFINITY, l_sum = 0.f, v_inv = 1.f;
    // a lower bound of the largest |weight x norm| of the row so far (infinite
    // before the row's first position: no reason to move)
    float w_low = INFINITY;
    bool ok = true;
    const int n = halves ? (cnt + 1 - mt) / 2 : cnt;
    for (int j = 0; j < n; ++j) {
      const int i = halves ? 2 * j + mt : j;
      ok = tw_wait(s_full + 16 * mt + 8 * (j & 1), (j >> 1) & 1, TW_TRIES) &&
           tw_wait(n_full + 8 * (i % TW_SLOTS), (i / TW_SLOTS) & 1, TW_TRIES);
      ok = __all_sync(FULL, ok);
      if (!ok) {
        if (lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t sp = s0 + 64u * (j & 1);
      if (any_row) {
        const TwSlot& slot = reinterpret_cast<const TwSlot*>(sm + C::N0)[i % TW_SLOTS];
        float x[64];
        {
          uint32_t u[32], v[32];
          tmem_ld32(sp, u);
          tmem_ld32(sp + 32u, v);
          tmem_wait_ld();
          tmem_regs_after_wait(u);
          tmem_regs_after_wait(v);
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(u[c]), x[c + 32] = __uint_as_float(v[c]);
        }
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 n = *reinterpret_cast<const float4*>(slot.nk + c);
          const f2 u = mul2(make_float2(x[c], x[c + 1]), make_float2(n.x, n.y));
          const f2 v = mul2(make_float2(x[c + 2], x[c + 3]), make_float2(n.z, n.w));
          x[c] = u.x, x[c + 1] = u.y, x[c + 2] = v.x, x[c + 3] = v.y;
        }
        // whether some position is masked for some row of the warp
        const bool hidden =
            !(slot.t_max <= pw_lo && (slot.t_max < a.sinks || slot.t_min > pw_hi - a.window));
        if (hidden) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t seen = tw_visible16(slot.blk_t[h], p_row, a.window, a.sinks);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (!(seen >> c & 1u)) x[16 * h + c] = -INFINITY;
          }
        }
        float mx0 = x[0], mx1 = x[1], mx2 = x[2], mx3 = x[3];
#pragma unroll
        for (int c = 4; c < 60; c += 8) {
          mx0 = tw_max3(mx0, x[c], x[c + 1]);
          mx1 = tw_max3(mx1, x[c + 2], x[c + 3]);
          mx2 = tw_max3(mx2, x[c + 4], x[c + 5]);
          mx3 = tw_max3(mx3, x[c + 6], x[c + 7]);
        }
        mx0 = tw_max3(mx0, x[60], x[61]);
        mx1 = tw_max3(mx1, x[62], x[63]);
        const float mx = fmaxf(tw_max3(mx0, mx1, mx2), mx3) * row_inv;
        const float v_fix = slot.v_up * v_inv;  // over the power of two of the tile before
        v_inv = slot.v_inv;
        w_low *= v_fix;
        // the reference follows products that could pass 2^14, and ones that are small
        const bool move = mx > m_ref + slot.head || w_low < AW_SMALL;
        if (__any_sync(FULL, move || v_fix != 1.0f)) {
          float fix = v_fix;
          const float top = fmaxf(m_ref, mx);
          float most = slot.nv_min;  // at least, where the largest score is new
          if (__any_sync(FULL, move && !(mx > m_ref && most >= AW_SMALL)))
            most = aw_exp2(tw_largest(x, slot.lg, row_inv) - top);
          if (move) {
            const float old = aw_exp2(m_ref - top);  // 0 from -inf
            most = fmaxf(most, w_low * old);  // (inf * 0 = NaN is left out)
            const float to = aw_reference(top, l_sum * old, most), f = aw_exp2(m_ref - to);
            l_sum *= f;
            fix *= f;
            m_ref = to;
            w_low = most;
          }
          if (j > 0) {
            // the previous product must be in the accumulator before it is
            // rescaled. (Even and odd tiles have barriers of their own: a wait
            // may be the first in many tiles, and this one's earlier phases
            // ended before the scores of tile j - 1 were complete.)
            const bool done = __all_sync(
                FULL, tw_wait(o_done + 16 * mt + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, TW_TRIES));
            if (!done) {
              if (lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t u[16];
              tmem_ld16(o0 + (uint32_t)c0, u);
              tmem_wait_ld();
              tmem_regs_after_wait(u);
#pragma unroll
              for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(__uint_as_float(u[c]) * fix);
              tmem_st16(o0 + (uint32_t)c0, u);
            }
          }
        }
        const float ref = m_ref == -INFINITY ? 0.f : m_ref;
        l_sum += tw_weights(x, slot.nv, row_inv, ref, sp);
        if (slot.odd[0] | slot.odd[1]) {  // value norms that are infinite or NaN: NaN for the rows that see one
#pragma unroll 1
          for (int c = 0; c < TW_TP; ++c)
            if ((slot.odd[c >> 5] >> (c & 31) & 1u) &&
                aw_visible(slot.blk_t[c >> 4] + (c & 15), p_row, a.window, a.sinks))
              l_sum = __int_as_float(0x7fc00000);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(p_full + 16 * mt + 8 * (j & 1));
    }
    // ---- results
    if (ok) {
      // every product is done; and, also where there is none (no row of the
      // CTA sees a position), the tile's other softmax warps have written
      // their query rows into the space that the results below go to: the
      // issuer signals after q_full
      ok = __all_sync(FULL, tw_wait(mma_end + 8 * mt, 0, TW_TRIES));
      if (!ok && lane == 0) record_error(a.err, TQ_DEVERR_TIMEOUT);
      tc_fence_after();
    }
    if (any_row && ok) {
      const int64_t idx = out_row * a.n_split + (halves ? 2 * c_split + mt : c_split);
      if (a.n_split > 1 && row_ok) {
        a.ws_m[idx] = m_ref;
        a.ws_l[idx] = l_sum;
      }
      // NaN where the sum is NaN, 0 where no position was seen
      const float scale = a.n_split > 1 ? v_inv : (l_sum > 0.f ? v_inv * a.o_scale / l_sum : (l_sum == l_sum ? 0.f : l_sum));
      // rows of the warp are put together in the row tile's query operand
      // (no product reads it any more; 4 d bytes per row, 16-byte chunks
      // swizzled within 128 bytes) and leave in whole lines
      uint8_t* stage = sm + C::Q0 + 2 * mt * C::Q_PART + 32 * (warp & 3) * (4 * D);
#pragma unroll 1
      for (int hf = 0; hf < D / 64; ++hf) {
        f2 x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = make_float2(0.f, 0.f);
        if (n > 0) {
#pragma unroll 1
          for (int m = a.n_split > 1 ? hf : 0; m < (a.n_split > 1 ? hf + 1 : D / 64); ++m) {
            const float sg1 = a.n_split > 1 || !(__popc(m & hf) & 1) ? 1.f : -1.f;
            const f2 sg = make_float2(sg1, sg1);
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += 16) {
              uint32_t u[16];
              tmem_ld16(o0 + (uint32_t)(64 * m + c0), u);
              tmem_wait_ld();
              tmem_regs_after_wait(u);
#pragma unroll
              for (int c = 0; c < 16; c += 2)
                x[(c0 + c) / 2] =
                    fma2(sg, make_float2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), x[(c0 + c) / 2]);
            }
          }
        }
        if (a.n_split == 1) wht64(x);
        // column 64 hf + e is dim 8 (e % DG) + JN hf + e / DG: JN neighbouring dims per group
        constexpr int DG = D / 8, JN = 64 / DG;
        auto at_col = [&](int e) { return e & 1 ? x[e / 2].y : x[e / 2].x; };
#pragma unroll
        for (int dg = 0; dg < DG; ++dg) {
          const int dim = 8 * dg + JN * hf;
#pragma unroll
          for (int j = 0; j < JN; j += 2) {
            const float u = at_col(j * DG + dg) * scale, v = at_col((j + 1) * DG + dg) * scale;
            const int at = (a.n_split > 1 ? 4 : 2) * (dim + j);
            uint8_t* dst = stage + lane * (4 * D) + (at & ~112) + ((at ^ (lane << 4)) & 112);
            if (a.n_split > 1) *reinterpret_cast<float2*>(dst) = make_float2(u, v);
            else *reinterpret_cast<uint32_t*>(dst) = pack_half2(u, v) ^ a.v_sign_h2[(dim + j) / 2];
          }
        }
      }
      __syncwarp();
      auto leave = [&](auto chunks_, uint8_t* to, int64_t row_to) {
        constexpr int chunks = decltype(chunks_)::value;  // of 16 bytes, per row
#pragma unroll 8
        for (int it = 0; it < chunks; ++it) {
          const int e = it * 32 + lane, rr = e / chunks, c = e % chunks;
          const int64_t at = __shfl_sync(FULL, row_to, rr) * (16 * chunks) + 16 * c;
          const uint4 w =
              *reinterpret_cast<const uint4*>(stage + rr * (4 * D) + ((c & ~7) << 4) + (((c ^ rr) & 7) << 4));
          if (rw0 + rr < rows) *reinterpret_cast<uint4*>(to + at) = w;
        }
      };
      if (a.n_split > 1)
        leave(std::integral_constant<int, D / 4>(), reinterpret_cast<uint8_t*>(a.ws_acc), idx);
      else
        leave(std::integral_constant<int, D / 8>(), reinterpret_cast<uint8_t*>(a.out), out_row);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    __syncwarp();
    tmem_dealloc(tmem, TW_TMEM);
  }
}

template <int D, int KB, int VB>
static cudaError_t launch_tc_t(const AwArgs& a, cudaStream_t st) {
  using C = TwCfg<D, KB, VB>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = aw_allow_smem(reinterpret_cast<const void*>(window_tc_kernel<D, KB, VB>), C::BYTES, done);
  if (e != cudaSuccess) return e;
  const int64_t gx = (int64_t)(a.halves ? a.n_split / 2 : a.n_split) * a.hkv, gy = ((int64_t)a.max_q * a.g + 128 * C::MT - 1) / (128 * C::MT);
  if (gx > 0x7fffffff || gy > 65535) return cudaErrorNotSupported;
  window_tc_kernel<D, KB, VB><<<dim3((unsigned)gx, (unsigned)gy, a.B), C::WARPS * 32, C::BYTES, st>>>(a);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_tc_d(const AwArgs& a, int kb, int vb, cudaStream_t st) {
#define TQ_TW_CASE(KB_, VB_) \
  if (kb == KB_ && vb == VB_) return launch_tc_t<D, KB_, VB_>(a, st);
  TQ_TW_CASE(2, 2) TQ_TW_CASE(2, 3) TQ_TW_CASE(2, 4) TQ_TW_CASE(3, 2) TQ_TW_CASE(3, 3) TQ_TW_CASE(3, 4)
  TQ_TW_CASE(4, 2) TQ_TW_CASE(4, 3) TQ_TW_CASE(4, 4)
#undef TQ_TW_CASE
  return cudaErrorInvalidValue;
}

}  // namespace tq

using namespace tq;

int tq_window_tc_rows(int d) { return d == 256 ? 128 : 256; }

cudaError_t tq_launch_window_tc(const AwArgs& a, int d, int kb, int vb, cudaStream_t st) {
  if (d == 64) return launch_tc_d<64>(a, kb, vb, st);
  if (d == 128) return launch_tc_d<128>(a, kb, vb, st);
  return launch_tc_d<256>(a, kb, vb, st);
}
