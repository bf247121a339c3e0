// Orthogonalised updates: Newton-Schulz steps on a batch of matrices (the gradients of the expert weights).
//
//   X_0 = g / (|g|_F + eps);   A = X X^T,  X <- a X + (b A + c A A) X   (X is p x q with p <= q);   out = scale X
//
// Three matrix products a step.  A and A A are symmetric, so only the tiles on and above the diagonal are computed and
// each is stored twice, once transposed: p^2 q + p^3 + 2 p^2 q operations a step instead of 2 p^2 q + 2 p^3 + 2 p^2 q.
// Bound by the matrix instructions: a step at p = 2048, q = 7168 is 99 GFLOP on 59 MB.  A product whose tiles do not fill
// the last round of the 256 compute units shares those tiles' reductions among workgroups and joins them in a launch of its
// own (8 x 2048 x 7168: 288 tiles of 256 x 256, X X^T from 369 to 251 + 11 us); see shape().
//
// Number formats.  Operands are fp16 (11 bits; the products then run at the bf16 rate with an eighth of its rounding
// error), accumulated in fp32.  Everything carries a factor S = 2^12: entries of an orthogonal-like p x q matrix are near
// 1 / sqrt(q) and those of A off its diagonal smaller still, which unscaled would be subnormal in fp16, while the largest
// possible entries (|X| <= 3, |A| <= 9, |B| <= 12, from the entry point's bounds on the coefficients) stay below 2^16.
// X itself is kept as hi + lo, two fp16 values (22 bits): the term a X magnifies singular values near zero by
// a^steps (485 for the usual coefficients), and with X rounded to 11 bits each step it would magnify that rounding with
// them (a gradient of rank 1 then comes out 15% wrong, of rank 16 4%; measured in fp64 models of both).  Rounding the
// operands of the products does not have this effect: an error in A or B multiplies X from the left, and leaves its row
// space alone.  The last step, which magnifies by a alone, does without lo.  bf16 results of 64 x 1000 to 2048 x 7168 are 1.86
// to 2.11e-3 of the norm off, of rank 1, 3 and 16 1.92 to 2.05e-3; their rounding alone is 1.66e-3.
// SPLIT (fp32 outputs, and bf16 outputs of matrices so small that the launches are what is paid for) gives hi and lo to the
// operands too and sums lo hi + hi lo + hi hi: three products, the same tiles.
//
// Layout: X is held transposed only, X^T [Q][P] (two, used in turn: an update's tiles read one and write the other; lo in
// place where it is no operand), A and B [P][P]; P and Q are p and q rounded up to the tile size and zero-filled, which the
// iteration keeps, so no product has a bound to check.  a sits on B's diagonal: X^T <- X^T (a + b A + c A A) + a lo.  A A and
// X^T B reduce along rows of both operands; X X^T reduces over the rows of X^T, through the transposing LDS load.  Holding X
// in both orientations instead cost an update 10 bytes per value for 6 (8 x 2048 x 7168: 615 us for 494).
#include <type_traits>
#include <utility>

#include "common.h"
#include "gemm_tile.h"
#include "kernels.h"

namespace moe {
namespace orth {

constexpr float S = 4096.0f;

// 16 bytes at the elements' own alignment: one wide access
typedef float f32x4_e4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x4_e2_t __attribute__((ext_vector_type(4), aligned(2)));

enum Mode { GRAM = 0, POLY = 1, UPDATE = 2, FINAL = 3 };

// Tiles.  0: 64 x 64 over 4 wavefronts (32 x 32 each); 1: 128 x 128 over 4 (64 x 64 each); 2: 256 x 256 over 8
// (128 x 64 each); 3: 256 x 192 over 8 (64 x 96 each), for X^T B where it fills the last round better (P = 1536, Q = 4096,
// 4 matrices: 512 tiles instead of 384 on 256 compute units, 102 us instead of 117; 1 x 2304 x 4096 in all 603 instead of
// 637), and 4, the same turned, for the last product.  A stage holds RB bytes of the reduction for every tile row of each operand array (hi, and lo with
// SPLIT); NS stages are in flight or in use.  The small tiles' stages leave room for a second workgroup on a compute unit:
// with SPLIT two stages of 64 x 64 instead of four took three matrices of 1001 x 333 from 186 to 163 us.
template <int SIZE, bool SPLIT>
struct Cfg;
template <>
struct Cfg<0, false> {
  static constexpr int RB = 128, NS = 3, BM = 64, BN = 64, WM = 2, WN = 2;
};
template <>
struct Cfg<1, false> {
  static constexpr int RB = 64, NS = 4, BM = 128, BN = 128, WM = 2, WN = 2;
};
template <>
struct Cfg<2, false> {
  static constexpr int RB = 128, NS = 2, BM = 256, BN = 256, WM = 2, WN = 4;
};
template <>
struct Cfg<0, true> {
  static constexpr int RB = 128, NS = 2, BM = 64, BN = 64, WM = 2, WN = 2;
};
template <>
struct Cfg<1, true> {
  static constexpr int RB = 64, NS = 2, BM = 128, BN = 128, WM = 2, WN = 2;
};
template <>
struct Cfg<2, true> {
  static constexpr int RB = 64, NS = 2, BM = 256, BN = 256, WM = 2, WN = 4;
};
template <>
struct Cfg<3, false> {
  static constexpr int RB = 128, NS = 2, BM = 256, BN = 192, WM = 4, WN = 2;
};
template <>
struct Cfg<4, false> {
  static constexpr int RB = 128, NS = 2, BM = 192, BN = 256, WM = 2, WN = 4;
};
constexpr int TILE_M[4] = {64, 128, 256, 256}, TILE_N[4] = {64, 128, 256, 192};

struct Args {
  // operands: hi and (SPLIT) lo, fp16.  GRAM: [K][rows] per matrix of the batch (the reduction runs over rows); else [rows][K]
  const uint8_t *M0, *M1, *N0, *N1;
  int64_t m_batch, n_batch;  // bytes between matrices
  int m_ld, n_ld;            // values per row
  int K;                     // reduction length (values), a multiple of 64
  int mt, nt;                // row and column tiles (symmetric products: mt == nt)
  // results and the elementwise operand, hi and lo, [rows][ld]; symmetric products also store the mirrored tile
  const uint8_t *E0, *E1;
  uint8_t *R0, *R1;
  int ld;
  int64_t r_batch;           // bytes between matrices
  float alpha, beta, diag;   // result = alpha * E + beta * product + diag on the diagonal (POLY)
  _Float16* rest_of_diag;    // without SPLIT: what B's diagonal loses to its rounding, [P] per matrix (POLY writes, B X adds)
  bool b_is_m;               // FINAL: B is the operand M
  // the first `whole` tiles are one workgroup each; `parts` workgroups share each of the rest
  int whole, parts;
  float* partial;            // [rest * parts][tile values]
  // FINAL: out [m][n], the result's rows and columns
  uint8_t* out;
  int m, n;
  bool out_bf16;
};

// fp16 pair of a value: hi = rounded, lo = the rest rounded
MOE_DEV void split16(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

MOE_DEV void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------------------------------------
// Stages.  An operand whose reduction is contiguous (A, B, and X^T in B X) lies in a stage as B rows of RB bytes, in the
// layout of the grouped products (gemm_tile.h).  X X^T reduces over the rows of X^T [Q][P]: a stage then holds RB / 2 of
// those rows, B values of each, and the fragments are read with the transposing LDS load: 16 lanes read 4 rows x 16 values,
// 8 bytes each, and lane l gets the 4 values of column l.  One such load of a wavefront covers rows k .. k + 3 and
// k + 8 .. k + 11 of 32 columns; a row's 64-byte chunks (32 columns) are stored at chunk ^ (row & 3) (64-value rows:
// chunk ^ (row / 2 & 1)), so that the four rows that are served together fall on distinct banks.
// ---------------------------------------------------------------------------------------------------------
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
template <int B>
MOE_DEV int swz_t(int row) {
  return B >= 128 ? row & 3 : (row >> 1) & 1;
}
template <int ROWB>
MOE_DEV f16x8_t frag_t(tile::lds_u8_t* p, int imm) {
  union {
    i16x4_t h[2];
    f16x8_t f;
  } u;
  u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p + imm));
  u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p + imm + 4 * ROWB));
  return u.f;
}

// acc += the products of one stage; SPLIT: lo hi + hi lo + hi hi, the lo array of an operand ARR bytes behind its hi array.
// ao, bo: byte offsets of this lane's fragments: per reduction step (rows of RB bytes) or per 32 columns (transposed).
template <int RB, int MB, int NB>
MOE_DEV void mma_stage_split(const uint8_t* As, const uint8_t* Bs, int ARR, const int (&arow)[MB], const int (&brow)[NB],
                             const tile::FragOff& ao, const tile::FragOff& bo, f32x16_t (&acc)[MB][NB]) {
#pragma unroll
  for (int s = 0; s < RB / 32; ++s) {
    tile::lds_u8_t* av = tile::to_lds(As) + ao.o[s];
    tile::lds_u8_t* bv = tile::to_lds(Bs) + bo.o[s];
    f16x8_t bh[NB], bl[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      bh[j] = __builtin_bit_cast(f16x8_t, tile::lds_at(bv, (brow[j] - brow[0]) * RB));
      bl[j] = __builtin_bit_cast(f16x8_t, tile::lds_at(bv, ARR + (brow[j] - brow[0]) * RB));
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const f16x8_t ah = __builtin_bit_cast(f16x8_t, tile::lds_at(av, (arow[i] - arow[0]) * RB));
      const f16x8_t al = __builtin_bit_cast(f16x8_t, tile::lds_at(av, ARR + (arow[i] - arow[0]) * RB));
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = mfma_32x32x16(al, bh[j], acc[i][j]);
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = mfma_32x32x16(ah, bl[j], acc[i][j]);
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = mfma_32x32x16(ah, bh[j], acc[i][j]);
    }
  }
}

template <int RB, int B, bool SPLIT, int MB, int NB>
MOE_DEV void mma_stage_t(const uint8_t* As, const uint8_t* Bs, const uint32_t (&ao)[MB], const uint32_t (&bo)[NB],
                         f32x16_t (&acc)[MB][NB]) {
  constexpr int STEPS = RB / 32, ROWB = 2 * B, STEP = 16 * ROWB, ARR = B * RB;
  tile::lds_u8_t *av[MB], *bv[NB];
#pragma unroll
  for (int i = 0; i < MB; ++i) av[i] = tile::to_lds(As) + ao[i];
#pragma unroll
  for (int j = 0; j < NB; ++j) bv[j] = tile::to_lds(Bs) + bo[j];
  if constexpr (SPLIT) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      f16x8_t bh[NB], bl[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        bh[j] = frag_t<ROWB>(bv[j], s * STEP);
        bl[j] = frag_t<ROWB>(bv[j], ARR + s * STEP);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const f16x8_t ah = frag_t<ROWB>(av[i], s * STEP), al = frag_t<ROWB>(av[i], ARR + s * STEP);
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma_32x32x16(al, bh[j], acc[i][j]);
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma_32x32x16(ah, bl[j], acc[i][j]);
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma_32x32x16(ah, bh[j], acc[i][j]);
      }
    }
  } else {
    // fragments double-buffered in registers: step s + 1's loads go between step s's products
    f16x8_t fa[2][MB], fb[2][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[0][i] = frag_t<ROWB>(av[i], 0);
#pragma unroll
    for (int j = 0; j < NB; ++j) fb[0][j] = frag_t<ROWB>(bv[j], 0);
    sched_fence();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = s & 1;
      if (s + 1 < STEPS) {
#pragma unroll
        for (int i = 0; i < MB; ++i) fa[c ^ 1][i] = frag_t<ROWB>(av[i], (s + 1) * STEP);
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[c ^ 1][j] = frag_t<ROWB>(bv[j], (s + 1) * STEP);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma_32x32x16(fa[c][i], fb[c][j], acc[i][j]);
      if (s + 1 < STEPS) {
#pragma unroll
        for (int q = 0; q < MB + NB; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
      }
      sched_fence();
    }
  }
}

struct TileAt {
  int e, mi, ni;  // matrix, row tile, column tile
};
template <int MODE>
MOE_DEV TileAt tile_at(const Args& a, int L) {
  TileAt r;
  if constexpr (MODE == GRAM || MODE == POLY) {
    // tile t of the upper triangle, column by column: t = ni (ni + 1) / 2 + mi, mi <= ni
    const int per = a.nt * (a.nt + 1) / 2;
    r.e = L / per;
    const int t = L % per;
    r.ni = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (r.ni * (r.ni + 1) / 2 > t) --r.ni;
    while ((r.ni + 1) * (r.ni + 2) / 2 <= t) ++r.ni;
    r.mi = t - r.ni * (r.ni + 1) / 2;
  } else {
    // groups of 4 row tiles, column tiles next, row tiles fastest: the tiles that an XCD runs at once share operands
    const int per = a.mt * a.nt;
    r.e = L / per;
    const int t = L % per;
    const int g = t / (4 * a.nt), q = t % (4 * a.nt);
    const int gm = min(4, a.mt - g * 4);
    r.ni = q / gm;
    r.mi = g * 4 + q % gm;
  }
  r.e = uniform_int(r.e);
  r.mi = uniform_int(r.mi);
  r.ni = uniform_int(r.ni);
  return r;
}

// What follows a product for one 32 x W block of a wavefront (W = WTN columns), through the wavefront's own LDS block, so
// that every global access is 16 bytes per lane: by rows for the result (and the elementwise operand, loaded ahead by the
// caller), by columns for a mirrored one.
// Accumulator element v of a lane: row (v / 4) * 8 + 4 * (lane / 32) + v % 4, column lane % 32.
template <int MODE, int W, bool SPLIT>
struct Epilogue {
  static constexpr bool SYM = MODE == GRAM || MODE == POLY;
  // elementwise operand: A for B = b A + c A A; of X its lo part, but in the last step (hi comes with the product: B carries
  // a on its diagonal, and with SPLIT the lo part does too)
  static constexpr bool E_HI = MODE == POLY, E_LO = SPLIT ? MODE == POLY : MODE == UPDATE;
  static constexpr int NB = W / 32, PITCH = W + 4;                       // floats per row of the LDS block
  static constexpr int LPR = W / 8, RPP = 64 / LPR, PASS = 32 / RPP;     // lanes per row, rows per pass, passes
  struct Elem {
    f16x8_t h[E_HI ? PASS : 1], l[E_LO ? PASS : 1];
  };

  static MOE_DEV void load(const Args& a, int e, int row0, int col0, Elem& x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int it = 0; it < PASS; ++it) {
      const int64_t at = e * a.r_batch + ((int64_t)(row0 + it * RPP + lane / LPR) * a.ld + col0 + lane % LPR * 8) * 2;
      if constexpr (E_HI) x.h[it] = *reinterpret_cast<const f16x8_t*>(a.E0 + at);
      if constexpr (E_LO) x.l[it] = *reinterpret_cast<const f16x8_t*>(a.E1 + at);
    }
  }

  // 8 values of a row of out from column gc on, at the elements' own alignment; a row's last ones go one by one
  static MOE_DEV void store_out(const Args& a, int64_t o, int gc, const float (&v)[8]) {
    if (gc + 8 <= a.n) {
      if (a.out_bf16) {
        i32x4_t w;
#pragma unroll
        for (int d = 0; d < 4; ++d)
          w[d] = (int)((uint32_t)f32_to_bf16_bits(v[2 * d]) | ((uint32_t)f32_to_bf16_bits(v[2 * d + 1]) << 16));
        *reinterpret_cast<i32x4_e2_t*>(a.out + o * 2) = w;
      } else {
#pragma unroll
        for (int d = 0; d < 2; ++d)
          *reinterpret_cast<f32x4_e4_t*>(a.out + o * 4 + 16 * d) =
              (f32x4_t){v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]};
      }
      return;
    }
#pragma unroll
    for (int x = 0; x < 7; ++x)
      if (gc + x < a.n) {
        if (a.out_bf16)
          reinterpret_cast<uint16_t*>(a.out)[o + x] = f32_to_bf16_bits(v[x]);
        else
          reinterpret_cast<float*>(a.out)[o + x] = v[x];
      }
  }
  static MOE_DEV void store_pair(const Args& a, int64_t at, const float (&v)[8]) {
    f16x8_t h, l;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      _Float16 hi, lo;
      split16(v[x], hi, lo);
      h[x] = hi;
      l[x] = lo;
    }
    *reinterpret_cast<f16x8_t*>(a.R0 + at) = h;
    if constexpr (SPLIT)
      *reinterpret_cast<f16x8_t*>(a.R1 + at) = l;
    else if (MODE == UPDATE && a.R1 != nullptr)
      *reinterpret_cast<f16x8_t*>(a.R1 + at) = l;
  }

  // block at (row0, col0) of matrix e; mirror: also store it transposed
  static MOE_DEV void run(const Args& a, int e, int row0, int col0, bool mirror, const f32x16_t (&acc)[NB], const Elem& el,
                          float* sc) {
    const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) sc[((v >> 2) * 8 + 4 * lh + (v & 3)) * PITCH + j * 32 + lr] = acc[j][v];
    wave_lds_fence();
#pragma unroll
    for (int it = 0; it < PASS; ++it) {
      const int r = it * RPP + lane / LPR, c = lane % LPR * 8;
      float v[8];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const f32x4_t q = *reinterpret_cast<const f32x4_t*>(&sc[r * PITCH + c + 4 * d]);
#pragma unroll
        for (int x = 0; x < 4; ++x) v[4 * d + x] = a.beta * q[x];
      }
      if constexpr (E_HI || E_LO) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float ev = 0.0f;
          if constexpr (E_HI) ev += (float)el.h[it][x];
          if constexpr (E_LO) ev += (float)el.l[it][x];
          v[x] = __builtin_fmaf(a.alpha, ev, v[x]);
        }
      }
      if constexpr (MODE == POLY) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (row0 + r == col0 + c + x) {
            v[x] += a.diag;
            if constexpr (!SPLIT) {
              _Float16 hi;
              split16(v[x], hi, a.rest_of_diag[(int64_t)e * a.ld + row0 + r]);
            }
          }
      }
      if constexpr (MODE == FINAL) {
        const int gr = row0 + r, gc = col0 + c;
        if (gr < a.m && gc < a.n) store_out(a, ((int64_t)e * a.m + gr) * a.n + gc, gc, v);
      } else {
        store_pair(a, e * a.r_batch + ((int64_t)(row0 + r) * a.ld + col0 + c) * 2, v);
      }
      if (SYM && mirror)
#pragma unroll
        for (int d = 0; d < 2; ++d)
          *reinterpret_cast<f32x4_t*>(&sc[r * PITCH + c + 4 * d]) =
              (f32x4_t){v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]};
    }
    wave_lds_fence();
    if (!SYM || !mirror) return;
#pragma unroll
    for (int it = 0; it < W / 16; ++it) {
      const int c = it * 16 + lane / 4, r = lane % 4 * 8;
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = sc[(r + x) * PITCH + c];
      store_pair(a, e * a.r_batch + ((int64_t)(col0 + c) * a.ld + row0 + r) * 2, v);
    }
    wave_lds_fence();
  }
};

template <int MODE, int SIZE, bool SPLIT>
__global__ __launch_bounds__((64 * Cfg<SIZE, SPLIT>::WM * Cfg<SIZE, SPLIT>::WN)) void product_kernel(const Args a) {
  using C_ = Cfg<SIZE, SPLIT>;
  constexpr int RB = C_::RB, NS = C_::NS, BM = C_::BM, BN = C_::BN, WM = C_::WM, WN = C_::WN, NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN, MB = WTM / 32, NB = WTN / 32;
  constexpr int RPI = 1024 / RB;         // rows one wavefront load instruction fills
  constexpr int INM = BM / (NW * RPI), INN = BN / (NW * RPI);  // load instructions per wavefront and operand array
  constexpr int ARRM = BM * RB, ARRN = BN * RB;                // bytes of an operand array in a stage
  constexpr int NA = SPLIT ? 4 : 2;                            // operand arrays, half of them M's
  constexpr int N_AT = NA / 2 * ARRM, STAGE = N_AT + NA / 2 * ARRN, NL = NA / 2 * (INM + INN), CPR = RB / 16;
  constexpr int EW = WTN % 64 == 0 ? WTN : 32;                 // columns that the epilogue takes at a time
  using Epi = Epilogue<MODE, EW, SPLIT>;
  constexpr int EPI = NW * 32 * Epi::PITCH * 4;
  constexpr int SMEM = NS * STAGE > EPI ? NS * STAGE : EPI;
  constexpr bool SYM = Epi::SYM, TR = MODE == GRAM;
  static_assert(BM == BN || (!SYM && !SPLIT), "rectangular tiles: X B only");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SMEM];

  const int lane = threadIdx.x & 63, wid = uniform_int(threadIdx.x >> 6);
  const int wm = wid / WN, wn = wid % WN;
  const int lr = lane & 31, lh = lane >> 5;

  // ---- workgroup -> tile (each XCD takes one contiguous range of the whole tiles) and part of its reduction
  int L = blockIdx.x, part = 0, parts = 1;
  if (L < a.whole) {
    L = tile::xcd_tile_index(a.whole, L);
  } else {
    parts = a.parts;
    part = (L - a.whole) % parts;
    L = a.whole + (L - a.whole) / parts;
  }
  const TileAt at = tile_at<MODE>(a, L);
  const int e = at.e, m0 = at.mi * BM, n0 = at.ni * BN;
  // this workgroup's stages, and a stage's step in memory (bytes)
  const int nk_all = a.K * 2 / RB;
  const int k0 = uniform_int((int)((int64_t)nk_all * part / parts));
  const int nk = uniform_int((int)((int64_t)nk_all * (part + 1) / parts)) - k0;
  const int64_t m_row = (int64_t)a.m_ld * 2, n_row = (int64_t)a.n_ld * 2;
  const int64_t m_step = TR ? m_row * (RB / 2) : RB, n_step = TR ? n_row * (RB / 2) : RB;
  const int64_t moff = e * a.m_batch + k0 * m_step + (TR ? m0 * 2 : m0 * m_row);
  const int64_t noff = e * a.n_batch + k0 * n_step + (TR ? n0 * 2 : n0 * n_row);
  const uint8_t* base[NA];
  base[0] = uniform_ptr(a.M0 + moff);
  base[NA / 2] = uniform_ptr(a.N0 + noff);
  if constexpr (SPLIT) {
    base[1] = uniform_ptr(a.M1 + moff);
    base[3] = uniform_ptr(a.N1 + noff);
  }
  uint32_t m_off[INM], n_off[INN];
  auto offset = [&](int instr, int64_t row_bytes) {  // of this lane's 16 bytes of an operand array
    int r, at;                                       // row, and byte in it
    if constexpr (TR) {
      constexpr int PIECES = BM / 8;
      r = instr * (64 / PIECES) + lane / PIECES;
      const int piece = lane % PIECES;
      at = (((piece / 4) ^ swz_t<BM>(r)) * 4 + piece % 4) * 16;
    } else {
      r = instr * RPI + lane / CPR;
      at = ((lane % CPR) ^ tile::swz<RB>(r)) * 16;
    }
    return (uint32_t)(r * row_bytes + at);
  };
#pragma unroll
  for (int q = 0; q < INM; ++q) m_off[q] = offset(wid * INM + q, m_row);
#pragma unroll
  for (int q = 0; q < INN; ++q) n_off[q] = offset(wid * INN + q, n_row);
  auto load_stage = [&](uint8_t* dst, int kt) {
#pragma unroll
    for (int x = 0; x < NA / 2; ++x) {
      const uint8_t* p = uniform_ptr(base[x] + kt * m_step);
#pragma unroll
      for (int q = 0; q < INM; ++q) load_lds16(p, m_off[q], dst + x * ARRM + (wid * INM + q) * 1024);
    }
#pragma unroll
    for (int x = 0; x < NA / 2; ++x) {
      const uint8_t* p = uniform_ptr(base[NA / 2 + x] + kt * n_step);
#pragma unroll
      for (int q = 0; q < INN; ++q) load_lds16(p, n_off[q], dst + N_AT + x * ARRN + (wid * INN + q) * 1024);
    }
  };

  f32x16_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  int arow[MB], brow[NB];
#pragma unroll
  for (int i = 0; i < MB; ++i) arow[i] = wm * WTM + i * 32 + lr;
#pragma unroll
  for (int j = 0; j < NB; ++j) brow[j] = wn * WTN + j * 32 + lr;
  const tile::FragOff ao = tile::frag_offsets<RB, RB / 32>(arow[0], lh, 2);
  const tile::FragOff bo = tile::frag_offsets<RB, RB / 32>(brow[0], lh, 2);

  uint32_t at_m[MB], at_n[NB];  // transposed fragments
  {
    const int k = (lane >> 5) * 8 + (lane >> 2 & 3), in = (lane >> 4 & 1) * 32 + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < MB; ++i) at_m[i] = (uint32_t)(k * 2 * BM + ((wm * MB + i) ^ swz_t<BM>(k)) * 64 + in);
#pragma unroll
    for (int j = 0; j < NB; ++j) at_n[j] = (uint32_t)(k * 2 * BM + ((wn * NB + j) ^ swz_t<BM>(k)) * 64 + in);
  }

  const int row0 = m0 + wm * WTM, col0 = n0 + wn * WTN;
  // Without SPLIT, B's rounding to fp16 is the largest error, most of it on the diagonal, where B is of the size of a.  The
  // 32 x 32 blocks of this wavefront's part of the diagonal get two more products each, by a fragment that is the rest of the
  // diagonal and zero elsewhere: 1/64 more matrix instructions at P = 2048 (16 more us of 4500 for 8 x 2048 x 7168), and
  // 2.11e-3 of the norm off instead of 2.7e-3 at 363 x 3263.
  constexpr bool DIAG = !SPLIT && (MODE == UPDATE || MODE == FINAL);
  constexpr int DB = DIAG ? (MB > NB ? MB : NB) : 1;
  const bool b_is_m = SIZE == 4 || (SIZE < 3 && MODE == FINAL && a.b_is_m);
  _Float16 rest[DB];
  if constexpr (DIAG)
#pragma unroll
    for (int x = 0; x < DB; ++x) {
      const int blocks = b_is_m ? MB : NB, first = b_is_m ? row0 : col0;
      rest[x] = x < blocks ? a.rest_of_diag[(int64_t)e * a.m_ld + first + x * 32 + lr] : (_Float16)0.0f;
    }
  auto diagonal = [&](const uint8_t* As, const uint8_t* Bs, int first_k) {
    if constexpr (DIAG) {
#pragma unroll
      for (int x = 0; x < DB; ++x) {
        const int kk = (b_is_m ? row0 : col0) + x * 32 - first_k;  // of the block, in this stage
        if (x >= (b_is_m ? MB : NB) || kk < 0 || kk >= RB / 2) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          f16x8_t d;
#pragma unroll
          for (int y = 0; y < 8; ++y) d[y] = lr == t * 16 + lh * 8 + y ? rest[x] : (_Float16)0.0f;
          const int s1 = RB == 128 ? t + 2 : t;
          if (b_is_m) {
            if (x < MB)
#pragma unroll
              for (int j = 0; j < NB; ++j)
                acc[x < MB ? x : 0][j] = mfma_32x32x16(
                    d,
                    __builtin_bit_cast(f16x8_t, tile::lds_at(tile::to_lds(Bs) + (kk >= 32 ? bo.o[s1] : bo.o[t]),
                                                             (brow[j] - brow[0]) * RB)),
                    acc[x < MB ? x : 0][j]);
          } else if (x < NB) {
#pragma unroll
            for (int i = 0; i < MB; ++i)
              acc[i][x < NB ? x : 0] = mfma_32x32x16(
                  __builtin_bit_cast(f16x8_t, tile::lds_at(tile::to_lds(As) + (kk >= 32 ? ao.o[s1] : ao.o[t]),
                                                           (arow[i] - arow[0]) * RB)),
                  d, acc[i][x < NB ? x : 0]);
          }
        }
      }
    }
  };
  typename Epi::Elem el[2];
  if constexpr (SIZE == 0)
    if (parts == 1) Epi::load(a, e, row0, col0, el[0]);

  // slices 0 .. NS-2 in flight; each iteration waits for its own slice, meets the other wavefronts (the buffer read
  // last iteration is then free), refills it with slice kt + NS - 1 (clamped: loaded, never read) and computes slice kt
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) load_stage(smem + s * STAGE, min(s, nk - 1));
  if constexpr (DIAG)  // the rest of the diagonal has arrived: no stage waits for it, and so for the slices behind it
#pragma unroll
    for (int x = 0; x < DB; ++x) asm volatile("" : "+v"(rest[x]));
  int cb = 0, fb = NS - 1;
  auto step = [&](int kt, auto with_diagonal) {
    wait_vmcnt<(NS - 2) * NL>();
    __syncthreads();
    load_stage(smem + fb * STAGE, min(kt + NS - 1, nk - 1));
    const uint8_t* As = smem + cb * STAGE;
    if constexpr (TR)
      mma_stage_t<RB, BM, SPLIT, MB, NB>(As, As + N_AT, at_m, at_n, acc);
    else if constexpr (SPLIT)
      mma_stage_split<RB, MB, NB>(As, As + N_AT, ARRM, arow, brow, ao, bo, acc);
    else
      tile::mma_stage_bf16<RB, MB, NB, f16x8_t>(As, As + N_AT, arow, brow, ao, bo, acc);
    if constexpr (decltype(with_diagonal)::value) diagonal(As, As + N_AT, (k0 + kt) * (RB / 2));
    cb = cb + 1 == NS ? 0 : cb + 1;
    fb = fb + 1 == NS ? 0 : fb + 1;
  };
  if constexpr (DIAG) {  // three loops, so that the stages without a part of the diagonal ask nothing
    constexpr int KS = RB / 2;
    const int first = b_is_m ? row0 : col0, end = first + (b_is_m ? WTM : WTN);
    const int d0 = uniform_int(max(0, min(nk, first / KS - k0))), d1 = uniform_int(max(d0, min(nk, (end + KS - 1) / KS - k0)));
    int kt = 0;
    for (; kt < d0; ++kt) step(kt, std::false_type{});
    for (; kt < d1; ++kt) step(kt, std::true_type{});
    for (; kt < nk; ++kt) step(kt, std::false_type{});
  } else {
    for (int kt = 0; kt < nk; ++kt) step(kt, std::false_type{});
  }

  // ---- a shared tile: every part leaves its sums in memory, in the accumulators' order (16 bytes per lane side by side),
  // for the launch that joins them
  if (parts > 1) {
    float* mine = a.partial + ((int64_t)(L - a.whole) * parts + part) * (BM * BN) + wid * (WTM * WTN) + lane * 4;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4_t*>(mine + ((i * NB + j) * 4 + q) * 256) =
              (f32x4_t){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    wait_vmcnt0();  // no load into this workgroup's LDS is outstanding when it ends
    return;
  }

  // ---- epilogue, 32 rows at a time; the elementwise operand of a block is loaded while the block before is worked on (the
  // small tiles' before the product)
  const bool mirror = SYM && at.mi != at.ni;
  if constexpr (SIZE > 0) Epi::load(a, at.e, row0, col0, el[0]);
  wait_vmcnt0();
  __syncthreads();  // no load into LDS in flight, no wavefront still reading a stage: the epilogue reuses the buffers
  float* sc = reinterpret_cast<float*>(smem) + wid * 32 * Epi::PITCH;
  constexpr int PIECES = WTN / EW;
#pragma unroll
  for (int u = 0; u < MB * PIECES; ++u) {
    const int i = u / PIECES, c = u % PIECES * EW, next = (u + 1) / PIECES;
    if (next < MB) Epi::load(a, at.e, row0 + next * 32, col0 + (u + 1) % PIECES * EW, el[(u + 1) & 1]);
    f32x16_t block[Epi::NB];
#pragma unroll
    for (int x = 0; x < Epi::NB; ++x) block[x] = acc[i][c / 32 + x];
    Epi::run(a, at.e, row0 + i * 32, col0 + c, mirror, block, el[u & 1], sc);
  }
}

// The shared tiles: adds the parts' sums in the order of the parts and finishes the tile.  One wavefront per 32 x WTN block.
template <int MODE, int SIZE, bool SPLIT>
__global__ __launch_bounds__(256) void join_kernel(const Args a) {
  using C_ = Cfg<SIZE, SPLIT>;
  constexpr int B = C_::BM, WTM = B / C_::WM, WTN = B / C_::WN, MB = WTM / 32, NB = WTN / 32;
  constexpr int BLOCKS = C_::WM * C_::WN * MB;  // of a tile
  using Epi = Epilogue<MODE, WTN, SPLIT>;
  __shared__ float smem[4 * 32 * Epi::PITCH];
  const int lane = threadIdx.x & 63, w4 = uniform_int(threadIdx.x >> 6);
  const int blk = blockIdx.x * 4 + w4, rest = blk / BLOCKS, wid = blk % BLOCKS / MB, i = blk % MB;
  const TileAt at = tile_at<MODE>(a, a.whole + rest);
  const int row0 = at.mi * B + wid / C_::WN * WTM + i * 32, col0 = at.ni * B + wid % C_::WN * WTN;
  typename Epi::Elem el;
  Epi::load(a, at.e, row0, col0, el);
  const float* p = a.partial + (int64_t)rest * a.parts * (B * B) + wid * (WTM * WTN) + i * NB * 1024 + lane * 4;
  f32x16_t acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[j][v] = 0.0f;
  for (int x = 0; x < a.parts; ++x, p += B * B)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t t = *reinterpret_cast<const f32x4_t*>(p + (j * 4 + q) * 256);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[j][4 * q + v] += t[v];
      }
  Epi::run(a, at.e, row0, col0, Epi::SYM && at.mi != at.ni, acc, el, smem + w4 * 32 * Epi::PITCH);
}

// Sides of at most 128 (P = 64 or 128): B = a + b A + c A A and X^T <- X^T B in one launch.  A workgroup makes the 64
// rows of B that its 64 x 64 tile needs from all of A in LDS (twice the tile's own work at P = 128, but nothing to wait for),
// which saves the launch between the two products.  Small batches are bound by launches, 4 to 6 us each: 8 x 128 x 256 in
// fp32 takes 64 us with 12 of them and took 75 us with 17; plan_of() has the other side.
template <int MODE, int P, bool SPLIT>
__global__ __launch_bounds__(256) void narrow_kernel(const Args a, const uint8_t* A0, const uint8_t* A1, int64_t a_batch,
                                                     bool b_first, float pa, float pb, float pc) {
  constexpr int RB = 128, ST = P / 64;  // stages of 64 reduction values
  constexpr int NA = SPLIT ? 2 : 1;
  constexpr int A_ARR = P * RB, X_ARR = 64 * RB;             // one stage's rows, hi or lo
  constexpr int A_ALL = ST * NA * A_ARR, X_ALL = ST * NA * X_ARR;
  using Epi = Epilogue<MODE, 32, SPLIT>;
  constexpr int EPI = 4 * 32 * Epi::PITCH * 4;
  constexpr int FIRST = A_ALL > EPI ? A_ALL : EPI;           // A, then the epilogue's blocks
  __shared__ __attribute__((aligned(1024))) uint8_t smem[FIRST + 2 * X_ALL];
  __shared__ _Float16 rest[64];  // without SPLIT: what B's diagonal loses to its rounding
  uint8_t *sa = smem, *sx = smem + FIRST, *sb = sx + X_ALL;  // [stage][hi, lo][row][RB]

  const int lane = threadIdx.x & 63, wid = uniform_int(threadIdx.x >> 6), wm = wid >> 1, wn = wid & 1;
  const int lr = lane & 31, lh = lane >> 5;
  const TileAt at = tile_at<MODE>(a, tile::xcd_tile_index(gridDim.x, blockIdx.x));
  const int e = at.e, row0 = at.mi * 64 + wm * 32, col0 = at.ni * 64 + wn * 32;  // of the result
  const int m0 = (b_first ? at.ni : at.mi) * 64, n0 = (b_first ? at.mi : at.ni) * 64;  // rows of X^T and of B
  const int64_t row_bytes = (int64_t)P * 2;
  typename Epi::Elem el;
  Epi::load(a, e, row0, col0, el);
  // rows of 128 bytes, 8 per load instruction
  auto load_rows = [&](const uint8_t* src, uint8_t* dst, int rows) {
    const uint8_t* p = uniform_ptr(src);
    for (int i = wid; i < rows / 8; i += 4) {
      const int r = i * 8 + lane / 8;
      load_lds16(p, (uint32_t)(r * row_bytes + (((lane % 8) ^ tile::swz<RB>(r)) << 4)), dst + i * 1024);
    }
  };
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    load_rows(A0 + e * a_batch + s * RB, sa + s * NA * A_ARR, P);
    load_rows(a.M0 + e * a.m_batch + m0 * row_bytes + s * RB, sx + s * NA * X_ARR, 64);
    if constexpr (SPLIT) {
      load_rows(A1 + e * a_batch + s * RB, sa + (s * NA + 1) * A_ARR, P);
      load_rows(a.M1 + e * a.m_batch + m0 * row_bytes + s * RB, sx + (s * NA + 1) * X_ARR, 64);
    }
  }
  wait_vmcnt0();
  __syncthreads();

  // B^T: rows k (all P, half to each wm), columns the tile's 64 rows of B (32 to each wn)
  constexpr int MB = ST;
  f32x16_t acc[MB][1];
  int krow[MB], irow[1] = {n0 + wn * 32 + lr};
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    krow[i] = wm * (P / 2) + i * 32 + lr;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][0][v] = 0.0f;
  }
  const tile::FragOff ko = tile::frag_offsets<RB, RB / 32>(krow[0], lh, 2);
  const tile::FragOff io = tile::frag_offsets<RB, RB / 32>(irow[0], lh, 2);
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    const uint8_t* p = sa + s * NA * A_ARR;
    if constexpr (SPLIT)
      mma_stage_split<RB, MB, 1>(p, p, A_ARR, krow, irow, ko, io, acc);
    else
      tile::mma_stage_bf16<RB, MB, 1, f16x8_t>(p, p, krow, irow, ko, io, acc);
  }
  // accumulator values 4 q .. 4 q + 3 of a lane: B[i][k .. k + 3], i = irow, 8 bytes of row i
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = wm * (P / 2) + i * 32 + q * 8 + 4 * lh, r = irow[0], rb = wn * 32 + lr;
      const int st = k / 64, ch = k % 64 / 8;
      typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
      const f16x4_t ah = *reinterpret_cast<const f16x4_t*>(sa + st * NA * A_ARR + r * RB +
                                                           ((ch ^ tile::swz<RB>(r)) << 4) + 8 * lh);
      f16x4_t al = {0, 0, 0, 0}, bh, bl;
      if constexpr (SPLIT)
        al = *reinterpret_cast<const f16x4_t*>(sa + (st * NA + 1) * A_ARR + r * RB + ((ch ^ tile::swz<RB>(r)) << 4) +
                                               8 * lh);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float v = __builtin_fmaf(pb, (float)ah[x] + (float)al[x], pc * acc[i][0][4 * q + x]);
        v += k + x == r ? pa : 0.0f;
        _Float16 hi, lo;
        split16(v, hi, lo);
        if constexpr (!SPLIT)
          if (k + x == r) rest[rb] = lo;
        bh[x] = hi;
        bl[x] = lo;
      }
      uint8_t* d = sb + st * NA * X_ARR + rb * RB + ((ch ^ tile::swz<RB>(rb)) << 4) + 8 * lh;
      *reinterpret_cast<f16x4_t*>(d) = bh;
      if constexpr (SPLIT) *reinterpret_cast<f16x4_t*>(d + X_ARR) = bl;
    }
  __syncthreads();  // B is whole, and A is read no more

  f32x16_t out[1][1];
  int jrow[1] = {wm * 32 + lr}, brow[1] = {wn * 32 + lr};
#pragma unroll
  for (int v = 0; v < 16; ++v) out[0][0][v] = 0.0f;
  const tile::FragOff jo = tile::frag_offsets<RB, RB / 32>(jrow[0], lh, 2);
  const tile::FragOff bo = tile::frag_offsets<RB, RB / 32>(brow[0], lh, 2);
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    const uint8_t *pm = (b_first ? sb : sx) + s * NA * X_ARR, *pn = (b_first ? sx : sb) + s * NA * X_ARR;
    if constexpr (SPLIT)
      mma_stage_split<RB, 1, 1>(pm, pn, X_ARR, jrow, brow, jo, bo, out);
    else
      tile::mma_stage_bf16<RB, 1, 1, f16x8_t>(pm, pn, jrow, brow, jo, bo, out);
  }
  if constexpr (!SPLIT) {
    // the rest of the diagonal: rows n0 + 32 w .. of B against the same values of k, in stage n0 / 64
    const int w = b_first ? wm : wn;
    const _Float16 mine = rest[w * 32 + lr];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f16x8_t d;
#pragma unroll
      for (int y = 0; y < 8; ++y) d[y] = lr == t * 16 + lh * 8 + y ? mine : (_Float16)0.0f;
      const tile::FragOff& xo = b_first ? bo : jo;
      const f16x8_t f = __builtin_bit_cast(
          f16x8_t, tile::lds_at(tile::to_lds(sx + n0 / 64 * X_ARR) + (w == 1 ? xo.o[t + 2] : xo.o[t]), 0));
      out[0][0] = b_first ? mfma_32x32x16(d, f, out[0][0]) : mfma_32x32x16(f, d, out[0][0]);
    }
  }
  Epi::run(a, e, row0, col0, false, out[0], el, reinterpret_cast<float*>(sa) + wid * 32 * Epi::PITCH);
}

// Four consecutive values of g from index i on, at the elements' own alignment (one wide access), zeros from `end` on
typedef uint16_t u16x4_e2_t __attribute__((ext_vector_type(4), aligned(2)));
MOE_DEV f32x4_t load_g4(const uint8_t* g, bool bf16, int64_t i, int64_t end) {
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (bf16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(g) + i;
    if (i + 4 <= end) {
      const u16x4_e2_t q = *reinterpret_cast<const u16x4_e2_t*>(p);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = __uint_as_float((uint32_t)q[x] << 16);
    } else {
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (i + x < end) v[x] = __uint_as_float((uint32_t)p[x] << 16);
    }
  } else {
    const float* p = reinterpret_cast<const float*>(g) + i;
    if (i + 4 <= end) {
      v = *reinterpret_cast<const f32x4_e4_t*>(p);
    } else {
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (i + x < end) v[x] = p[x];
    }
  }
  return v;
}

// part[e][chunk] = sum of the squares of the chunk's values, in fp64 (squares of fp32 values neither overflow nor vanish);
// `step` values per chunk, a multiple of 4
__global__ __launch_bounds__(256) void square_sum_kernel(const uint8_t* __restrict__ g, bool bf16, int64_t count,
                                                         int64_t step, int chunks, double* __restrict__ part) {
  __shared__ double red[4];
  const int64_t e = blockIdx.x / chunks;
  const int64_t lo = blockIdx.x % chunks * step, hi = lo + step < count ? lo + step : count;
  const int64_t base = e * count, end = base + hi;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  int64_t i = base + lo + threadIdx.x * 4;
  for (; i + 3 * 1024 + 4 <= end; i += 4 * 1024) {  // four loads in flight
    f32x4_t v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = load_g4(g, bf16, i + u * 1024, end);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[x] = __builtin_fma((double)v[u][x], (double)v[u][x], s[x]);
  }
  for (; i < end; i += 1024) {
    const f32x4_t v = load_g4(g, bf16, i, end);
#pragma unroll
    for (int x = 0; x < 4; ++x) s[x] = __builtin_fma((double)v[x], (double)v[x], s[x]);
  }
  double t = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) t += __shfl_xor(t, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

struct PrepArgs {
  const uint8_t* g;
  bool bf16;
  int m, n;          // of g
  int rt, ct;        // 64 x 64 tiles of the padded matrix, in g's orientation
  const double* part;
  int chunks;
  float eps;
  bool turn;         // g's rows are the result's columns
  uint8_t *y0, *y1;  // hi and lo
  int ld;            // values per row
  int64_t batch_bytes;
};

// S g / (|g| + eps) as hi and lo, [Q][P], zero-filled past m x n
__global__ __launch_bounds__(256) void prepare_kernel(const PrepArgs a) {
  __shared__ float t[64][65];
  __shared__ double red[4];
  const int per = a.rt * a.ct;
  const int64_t e = blockIdx.x / per;
  const int r0 = blockIdx.x % per / a.ct * 64, c0 = blockIdx.x % per % a.ct * 64;
  const int tid = threadIdx.x;
  double s = tid < a.chunks ? a.part[e * a.chunks + tid] : 0.0;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((tid & 63) == 0) red[tid >> 6] = s;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = k * 16 + tid / 16, c = tid % 16 * 4;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r0 + r < a.m && c0 + c < a.n) {
      const int64_t row = (e * a.m + r0 + r) * a.n;
      v = load_g4(a.g, a.bf16, row + c0 + c, row + a.n);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) t[r][c + x] = v[x];
  }
  __syncthreads();
  // The quotient as a fraction in [1/2, 1) and a power of two, so that a gradient whose norm passes fp32's range, either
  // way, still gives its X; the fraction's rounding to fp32 is below the 22 bits that X keeps.
  int power;
  const float fraction = (float)frexp((double)S / (sqrt(red[0] + red[1] + red[2] + red[3]) + (double)a.eps), &power);
#pragma unroll
  for (int k = 0; k < 2; ++k) {  // 8 values of a row of the result each
    const int q = k * 256 + tid, r = q / 8, c = q % 8 * 8;
    f16x8_t h, l;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float v = ldexpf((a.turn ? t[c + x][r] : t[r][c + x]) * fraction, power);
      _Float16 hi, lo;
      split16(v, hi, lo);
      h[x] = hi;
      l[x] = lo;
    }
    const int64_t at = e * a.batch_bytes +
                       (a.turn ? (int64_t)(c0 + r) * a.ld + r0 + c : (int64_t)(r0 + r) * a.ld + c0 + c) * 2;
    *reinterpret_cast<f16x8_t*>(a.y0 + at) = h;
    *reinterpret_cast<f16x8_t*>(a.y1 + at) = l;
  }
}

constexpr int CUS = 256, MOST_PARTS = 8;

// How one product is laid over the GPU: the tile size (index of TILE), the tiles that are one workgroup each, and the
// parts of each of the others.
struct Shape {
  int size, whole, parts, rest;
  double us;  // estimate
};

// Microseconds of a product, to choose by: a launch of its own, then for every 256 tiles (one per compute unit; two smaller
// tiles that share one take as long as one after the other) the reduction and the epilogue.  Measured on kernels of 24 to
// 8192 tiles, K = 512 to 14336; one 256 x 256 tile holds 16 of 64 x 64, so per value the sizes cost 22 : 37 : 67.
// Columns: 64 x 64, 128 x 128, 256 x 256, 256 x 192.
constexpr double PER_K[2][4] = {{4.2e-3, 9.2e-3, 22e-3, 17.5e-3}, {8.5e-3, 27e-3, 72e-3}};  // [SPLIT]
constexpr double EPI_SYM[2][3] = {{1.0, 4.0, 10.0}, {1.5, 6.0, 15.0}};
constexpr double EPI_UPDATE[2][4] = {{1.0, 5.0, 19.0, 14.5}, {1.5, 7.0, 28.0}};
constexpr double LAUNCH_US = 4.5, BYTES_PER_US = 4e6;

static Shape shape(int64_t batch, int rows, int cols, int K, bool sym, bool split) {
  Shape best{};
  best.us = 1e30;
  for (int size = 0; size < (sym || split ? 3 : 4); ++size) {
    const int tm = TILE_M[size], tn = TILE_N[size];
    if (rows % tm != 0 || cols % tn != 0) continue;
    const int64_t nt = cols / tn, tiles = (sym ? nt * (nt + 1) / 2 : (int64_t)(rows / tm) * nt) * batch;
    const double epi = sym ? EPI_SYM[split][size] : EPI_UPDATE[split][size], red = K * PER_K[split][size];
    const int64_t full = tiles / CUS;
    const int rest = (int)(tiles % CUS);
    const int stages = K / (size == 1 || (size == 2 && split) ? 32 : 64);
    // the tiles of the last, partial round: whole, or each shared by `parts` workgroups and joined by another launch
    int parts = rest > 0 ? CUS / rest : 1;
    if (parts > MOST_PARTS) parts = MOST_PARTS;
    if (parts > stages / 4) parts = stages / 4;
    if (size == 3) parts = 1;  // chosen where it fills its last round: nothing to share
    for (int x = 1; x <= (parts < 1 ? 1 : parts); ++x) {
      const double bytes = 2.0 * rest * x * tm * tn * sizeof(float);
      const double us = LAUNCH_US + full * (red + epi) +
                        (rest == 0 ? 0.0 : x == 1 ? red + epi : red / x + LAUNCH_US + bytes / BYTES_PER_US);
      if (us < best.us) {
        best.us = us;
        best.size = size;
        best.parts = x;
        best.rest = x > 1 ? rest : 0;
        best.whole = (int)(tiles - best.rest);
      }
    }
  }
  return best;
}
static size_t partial_bytes(const Shape& z) {
  return (size_t)z.rest * z.parts * TILE_M[z.size] * TILE_N[z.size] * sizeof(float);
}

struct Plan {
  int p, q, P, Q;
  bool split, flip, narrow;
  double us;  // of a step, estimated
  int chunks;
  int64_t chunk_values;
  Shape gram, poly, update;
  size_t x_bytes, a_bytes;  // one fp16 array of the whole batch
  size_t part_bytes, partial, diag_bytes, total;
};

static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

static Plan plan_of(int64_t batch, int m, int n, bool split) {
  Plan z{};
  z.split = split;
  z.flip = m > n;
  z.p = z.flip ? n : m;
  z.q = z.flip ? m : n;
  // padding to multiples of the tile sizes (384: of 128 and 192): the least sum of the estimates
  z.us = 1e30;
  for (const auto [to_p, to_q] : {std::pair{64, 64}, {128, 128}, {256, 256}, {384, 256}}) {
    const int P = (z.p + to_p - 1) / to_p * to_p, Q = (z.q + to_q - 1) / to_q * to_q;
    const Shape gram = shape(batch, P, P, Q, true, split), poly = shape(batch, P, P, P, true, split),
                update = shape(batch, Q, P, P, false, split);
    if (gram.us + poly.us + update.us < z.us) {
      z.us = gram.us + poly.us + update.us;
      z.P = P;
      z.Q = Q;
      z.gram = gram;
      z.poly = poly;
      z.update = update;
    }
  }
  // One launch for the last two products of a step: always at P = 64 (16 x 64 x 8192: 141 us against 162); at P = 128 while
  // the rows of B that every tile makes for itself cost less than the launch: to four tiles per compute unit (16 x 128 x
  // 2048: 120 us against 127; 64 x 128 x 1024: 157 against 148), with SPLIT to one (8 x 128 x 256: 64 us against 75;
  // 2 x 128 x 8192: 156 against 152).
  const int64_t narrow_tiles = (int64_t)(z.Q / 64) * (z.P / 64) * batch;
  z.narrow = z.P == 64 || (z.P == 128 && narrow_tiles <= (split ? CUS : 4 * CUS));
  if (z.narrow) z.us -= LAUNCH_US;
  const int64_t count = (int64_t)m * n;
  // chunks of 4096 values or more, 256 at most: a workgroup of the next kernel adds one per thread
  z.chunks = (int)(count / 4096 < 1 ? 1 : count / 4096 > 256 ? 256 : count / 4096);
  z.chunk_values = ((count + z.chunks - 1) / z.chunks + 3) / 4 * 4;
  z.x_bytes = (size_t)batch * z.P * z.Q * 2;
  z.a_bytes = (size_t)batch * z.P * z.P * 2;
  z.part_bytes = up256((size_t)batch * z.chunks * sizeof(double));
  for (const Shape* t : {&z.gram, &z.poly, &z.update})
    if (partial_bytes(*t) > z.partial) z.partial = partial_bytes(*t);
  z.diag_bytes = split ? 0 : up256((size_t)batch * z.P * 2);
  z.total = z.part_bytes + z.partial + z.diag_bytes + (split ? 4 : 3) * z.x_bytes + (split ? 4 : 2) * z.a_bytes;
  return z;
}

// bf16 results take the split form where the estimates are close: it brings them to their own rounding (1.7e-3 of the norm
// off; 1.9 to 2.1e-3 without it), and a 64 x 64 takes 67 us either way, where 4 x 100 x 1000 takes 91 us instead of 71.
static Plan plan(int64_t batch, int m, int n, bool out_bf16) {
  const Plan split = plan_of(batch, m, n, true);
  if (!out_bf16) return split;
  const Plan whole = plan_of(batch, m, n, false);
  return split.us <= 1.2 * whole.us ? split : whole;
}

template <int MODE, int SIZE, bool SPLIT>
static void launch_sized(const Args& a, const Shape& z, hipStream_t s) {
  using C_ = Cfg<SIZE, SPLIT>;
  hipLaunchKernelGGL((product_kernel<MODE, SIZE, SPLIT>), dim3((unsigned)(z.whole + z.rest * z.parts)),
                     dim3(64 * C_::WM * C_::WN), 0, s, a);
  // 32-row blocks of a tile, joined by a launch of their own: SIZE 0: 2 x 2 x 1, 1: 2 x 2 x 2, 2: 2 x 4 x 4; four to a workgroup
  constexpr int GROUPS = C_::WM * C_::WN * (C_::BM / C_::WM / 32) / 4;
  if constexpr (SIZE < 3)
    if (z.rest > 0)
      hipLaunchKernelGGL((join_kernel<MODE, SIZE, SPLIT>), dim3((unsigned)(z.rest * GROUPS)), dim3(256), 0, s, a);
}

template <int MODE, bool SPLIT>
static void launch_product(const Args& a0, const Shape& z, int rows, int cols, hipStream_t s) {
  Args a = a0;
  a.mt = rows / (a.b_is_m ? TILE_N : TILE_M)[z.size];
  a.nt = cols / (a.b_is_m ? TILE_M : TILE_N)[z.size];
  a.whole = z.whole;
  a.parts = z.parts;
  if constexpr (!SPLIT && (MODE == UPDATE || MODE == FINAL))
    if (z.size == 3) {
      if constexpr (MODE == FINAL)
        if (a.b_is_m) return launch_sized<FINAL, 4, false>(a, z, s);
      return launch_sized<MODE, 3, false>(a, z, s);
    }
  if (z.size == 2)
    launch_sized<MODE, 2, SPLIT>(a, z, s);
  else if (z.size == 1)
    launch_sized<MODE, 1, SPLIT>(a, z, s);
  else
    launch_sized<MODE, 0, SPLIT>(a, z, s);
}

template <int MODE, bool SPLIT>
static void launch_narrow(const Args& a0, int rows, int cols, bool b_first, int P, int64_t batch, const uint8_t* A0,
                          const uint8_t* A1, float pa, float pb, float pc, hipStream_t s) {
  Args a = a0;
  a.mt = rows / 64;
  a.nt = cols / 64;
  if (b_first) {  // the kernel takes X^T as M and its tiles' rows of B from A
    a.M0 = a0.N0;
    a.M1 = a0.N1;
    a.m_batch = a0.n_batch;
  }
  const dim3 grid((unsigned)(a.mt * a.nt * batch));
  const int64_t ab = (int64_t)P * P * 2;
  if (P == 128)
    hipLaunchKernelGGL((narrow_kernel<MODE, 128, SPLIT>), grid, dim3(256), 0, s, a, A0, A1, ab, b_first, pa, pb, pc);
  else
    hipLaunchKernelGGL((narrow_kernel<MODE, 64, SPLIT>), grid, dim3(256), 0, s, a, A0, A1, ab, b_first, pa, pb, pc);
}

template <bool SPLIT>
static void run(const OrthLaunch& p, const Plan& z, hipStream_t s) {
  uint8_t* ws = reinterpret_cast<uint8_t*>(p.workspace);
  auto take = [&](size_t bytes) {
    uint8_t* r = ws;
    ws += bytes;
    return r;
  };
  double* part = reinterpret_cast<double*>(take(z.part_bytes));
  float* partial = reinterpret_cast<float*>(take(z.partial));
  _Float16* rest_of_diag = reinterpret_cast<_Float16*>(take(z.diag_bytes));
  uint8_t *y0[2] = {take(z.x_bytes), take(z.x_bytes)}, *y1[2];
  y1[0] = take(z.x_bytes);
  y1[1] = SPLIT ? take(z.x_bytes) : y1[0];  // not an operand without SPLIT: updated in place
  uint8_t *a0 = take(z.a_bytes), *b0 = take(z.a_bytes), *a1 = nullptr, *b1 = nullptr;
  if constexpr (SPLIT) {
    a1 = take(z.a_bytes);
    b1 = take(z.a_bytes);
  }
  const uint8_t* g = reinterpret_cast<const uint8_t*>(p.g);
  hipLaunchKernelGGL(square_sum_kernel, dim3((unsigned)(p.batch * z.chunks)), dim3(256), 0, s, g, p.g_bf16,
                     (int64_t)p.m * p.n, z.chunk_values, z.chunks, part);
  PrepArgs r{};
  r.g = g;
  r.bf16 = p.g_bf16;
  r.m = p.m;
  r.n = p.n;
  r.rt = (z.flip ? z.Q : z.P) / 64;
  r.ct = (z.flip ? z.P : z.Q) / 64;
  r.part = part;
  r.chunks = z.chunks;
  r.eps = p.eps;
  r.turn = !z.flip;
  r.y0 = y0[0];
  r.y1 = y1[0];
  r.ld = z.P;
  r.batch_bytes = (int64_t)z.P * z.Q * 2;
  hipLaunchKernelGGL(prepare_kernel, dim3((unsigned)(p.batch * r.rt * r.ct)), dim3(256), 0, s, r);

  const int64_t xb = (int64_t)z.P * z.Q * 2, ab = (int64_t)z.P * z.P * 2;
  for (int k = 0; k < p.steps; ++k) {
    const int cur = k & 1, nxt = cur ^ 1;
    Args q{};
    q.partial = partial;
    q.rest_of_diag = rest_of_diag;
    q.M0 = q.N0 = y0[cur];  // A = X X^T
    q.M1 = q.N1 = y1[cur];
    q.m_batch = q.n_batch = xb;
    q.m_ld = q.n_ld = z.P;
    q.K = z.Q;
    q.R0 = a0;
    q.R1 = a1;
    q.ld = z.P;
    q.r_batch = ab;
    q.beta = 1.0f / S;
    launch_product<GRAM, SPLIT>(q, z.gram, z.P, z.P, s);
    q.M0 = q.N0 = q.E0 = a0;  // B = a + b A + c A A
    q.M1 = q.N1 = q.E1 = a1;
    q.m_batch = q.n_batch = ab;
    q.K = z.P;
    q.R0 = b0;
    q.R1 = b1;
    q.alpha = p.b;
    q.beta = p.c / S;
    q.diag = p.a * S;
    if (!z.narrow) launch_product<POLY, SPLIT>(q, z.poly, z.P, z.P, s);
    q.M0 = y0[cur];  // X^T <- X^T B
    q.M1 = y1[cur];
    q.m_batch = xb;
    q.N0 = b0;
    q.N1 = b1;
    q.E1 = y1[cur];
    q.R0 = y0[nxt];
    q.R1 = SPLIT || k + 2 < p.steps ? y1[nxt] : nullptr;  // the last step's X is hi alone without SPLIT
    q.r_batch = xb;
    if (k + 1 < p.steps) {
      q.alpha = p.a;
      q.beta = 1.0f / S;
      if (z.narrow)
        launch_narrow<UPDATE, SPLIT>(q, z.Q, z.P, false, z.P, p.batch, a0, a1, p.a * S, p.b, p.c / S, s);
      else
        launch_product<UPDATE, SPLIT>(q, z.update, z.Q, z.P, s);
    } else {
      q.alpha = p.a * (p.scale / S);
      q.beta = p.scale / S / S;
      q.out = reinterpret_cast<uint8_t*>(p.out);
      q.m = p.m;
      q.n = p.n;
      q.out_bf16 = p.out_bf16;
      if (!z.flip) {  // the last product as B X: its rows are then out's
        std::swap(q.M0, q.N0);
        std::swap(q.M1, q.N1);
        std::swap(q.m_batch, q.n_batch);
        q.b_is_m = true;
      }
      const int rows = z.flip ? z.Q : z.P, cols = z.flip ? z.P : z.Q;
      if (z.narrow)
        launch_narrow<FINAL, SPLIT>(q, rows, cols, !z.flip, z.P, p.batch, a0, a1, p.a * S, p.b, p.c / S, s);
      else
        launch_product<FINAL, SPLIT>(q, z.update, rows, cols, s);
    }
  }
}

}  // namespace orth

size_t orthogonalize_workspace(int64_t batch, int m, int n, bool out_bf16) {
  const orth::Plan z = orth::plan(batch, m, n, out_bf16);
  // the largest grid has a workgroup of 256 per 64 x 64 values, and a grid less than 2^32 threads
  return batch * (z.P / 64) * (z.Q / 64) < (1 << 24) ? z.total : 0;
}

void launch_orthogonalize(const OrthLaunch& p, hipStream_t s) {
  const orth::Plan z = orth::plan(p.batch, p.m, p.n, p.out_bf16);
  if (z.split)
    orth::run<true>(p, z, s);
  else
    orth::run<false>(p, z, s);
}

}  // namespace moe
