// Orthogonalised updates: Newton-Schulz steps on a batch of matrices (the gradients of the expert weights).
//
//   X_0 = g / (|g|_F + eps);   A = X X^T,  X <- a X + (b A + c A A) X   (X is p x q with p <= q);   out = scale X
//
// Three matrix products a step.  A and A A are symmetric, so only the tiles on and above the diagonal are computed and
// each is stored twice, once transposed: p^2 q + p^3 + 2 p^2 q operations a step instead of 2 p^2 q + 2 p^3 + 2 p^2 q.
// Bound by the matrix instructions: a step at p = 2048, q = 7168 is 99 GFLOP on 59 MB.
//
// Number formats.  Operands are fp16 (11 bits; the products then run at the bf16 rate with an eighth of its rounding
// error), accumulated in fp32.  Everything carries a factor S = 2^12: entries of an orthogonal-like p x q matrix are near
// 1 / sqrt(q) and those of A off its diagonal smaller still, which unscaled would be subnormal in fp16, while the largest
// possible entries (|X| <= 3, |A| <= 9, |B| <= 12, from the entry point's bounds on the coefficients) stay below 2^16.
// X itself is kept as hi + lo, two fp16 values (22 bits): the term a X magnifies singular values near zero by
// a^steps (485 for the usual coefficients), and with X rounded to 11 bits each step it would magnify that rounding with
// them (a gradient of rank 1 then comes out 15% wrong, of rank 16 4%; measured in fp64 models of both).  Rounding the
// operands of the products does not have this effect: an error in A or B multiplies X from the left, and leaves its row
// space alone.
// SPLIT (fp32 outputs) gives hi and lo to the operands too and sums lo hi + hi lo + hi hi: three passes over the reduction
// with the same tiles.
//
// Layout: X [P][Q] hi and lo, its transpose [Q][P] (two, used in turn: a step's tiles read one and write the other), A and
// B [P][P]; P and Q are p and q rounded up to the tile size and zero-filled, which the iteration keeps, so no product has
// a bound to check.  Every product is C[i][j] = sum_k M[i][k] N[j][k] with both reductions contiguous: X X^T from X
// twice, A A from A twice (symmetric), B X from B and the transpose of X.
#include "common.h"
#include "gemm_tile.h"
#include "kernels.h"

namespace moe {
namespace orth {

constexpr float S = 4096.0f;

enum Mode { GRAM = 0, POLY = 1, UPDATE = 2, FINAL = 3 };

// 256 x 256 tiles over 8 wavefronts (128 x 64 each), two stages of 64 reduction values; 128 x 128 over 4 wavefronts
// (64 x 64 each), four stages of 32 values: two workgroups share a compute unit.
template <int BIG>
struct Cfg;
template <>
struct Cfg<0> {
  static constexpr int RB = 64, NS = 4, BM = 128, BN = 128, WM = 2, WN = 2;
};
template <>
struct Cfg<1> {
  static constexpr int RB = 128, NS = 2, BM = 256, BN = 256, WM = 2, WN = 4;
};

struct Args {
  // operands: hi and (SPLIT) lo, [rows][K] fp16 per matrix of the batch
  const uint8_t *M0, *M1, *N0, *N1;
  int64_t m_batch, n_batch;  // bytes between matrices
  int K;                     // reduction length (values), a multiple of the tile size
  int mt, nt;                // row and column tiles (symmetric products: mt == nt)
  // results and the elementwise operand: hi and lo, [rows][ld]; the transposed result T0 (T1: SPLIT) [cols][ld_t]
  const uint8_t *E0, *E1;
  uint8_t *R0, *R1, *T0, *T1;
  int ld, ld_t;
  int64_t r_batch, t_batch;  // bytes between matrices
  float alpha, beta;         // result = alpha * E + beta * product
  // FINAL: out [m][n], row i of X is row i of out (flip: column i)
  uint8_t* out;
  int m, n;
  bool flip, out_bf16, out_vec;
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

template <int MODE, int BIG, bool SPLIT>
__global__ __launch_bounds__((64 * Cfg<BIG>::WM * Cfg<BIG>::WN)) void product_kernel(const Args a) {
  using C_ = Cfg<BIG>;
  constexpr int RB = C_::RB, NS = C_::NS, BM = C_::BM, BN = C_::BN, WM = C_::WM, WN = C_::WN, NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN, MB = WTM / 32, NB = WTN / 32;
  constexpr int RPI = 1024 / RB;  // rows one wavefront load instruction fills
  constexpr int A_INS = BM / (NW * RPI), B_INS = BN / (NW * RPI), NL = A_INS + B_INS;
  constexpr int STAGE = (BM + BN) * RB, CPR = RB / 16;
  constexpr int PITCH = 68;  // floats per row of a wavefront's 32 x 64 epilogue block
  constexpr int SMEM = NS * STAGE > NW * 32 * PITCH * 4 ? NS * STAGE : NW * 32 * PITCH * 4;
  constexpr bool SYM = MODE == GRAM || MODE == POLY;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SMEM];

  const int lane = threadIdx.x & 63, wid = uniform_int(threadIdx.x >> 6);
  const int wm = wid / WN, wn = wid % WN;
  const int lr = lane & 31, lh = lane >> 5;

  // ---- workgroup -> (matrix, row tile, column tile); each XCD takes one contiguous range of the tiles
  const int L = tile::xcd_tile_index(gridDim.x, blockIdx.x);
  int e, mi, ni;
  if constexpr (SYM) {
    // tile t of the upper triangle, column by column: t = ni (ni + 1) / 2 + mi, mi <= ni
    const int per = a.nt * (a.nt + 1) / 2;
    e = L / per;
    const int t = L % per;
    ni = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (ni * (ni + 1) / 2 > t) --ni;
    while ((ni + 1) * (ni + 2) / 2 <= t) ++ni;
    mi = t - ni * (ni + 1) / 2;
  } else {
    // groups of 4 row tiles, column tiles next, row tiles fastest: the tiles that an XCD runs at once share operands
    const int per = a.mt * a.nt;
    e = L / per;
    const int t = L % per;
    const int g = t / (4 * a.nt), r = t % (4 * a.nt);
    const int gm = min(4, a.mt - g * 4);
    ni = r / gm;
    mi = g * 4 + r % gm;
  }
  e = uniform_int(e);
  const int m0 = uniform_int(mi) * BM, n0 = uniform_int(ni) * BN;
  const int64_t Kb = (int64_t)a.K * 2;
  const int nk1 = (int)(Kb / RB);            // stages of one pass over the reduction
  const int nk = SPLIT ? 3 * nk1 : nk1;

  const int64_t moff = e * a.m_batch + m0 * Kb, noff = e * a.n_batch + n0 * Kb;
  const uint8_t* mb[2] = {uniform_ptr(a.M0 + moff), SPLIT ? uniform_ptr(a.M1 + moff) : nullptr};
  const uint8_t* nb[2] = {uniform_ptr(a.N0 + noff), SPLIT ? uniform_ptr(a.N1 + noff) : nullptr};
  uint32_t a_off[A_INS], b_off[B_INS];
#pragma unroll
  for (int q = 0; q < A_INS; ++q) {
    const int r = (wid * A_INS + q) * RPI + lane / CPR;
    a_off[q] = (uint32_t)(r * Kb + (((lane % CPR) ^ tile::swz<RB>(r)) << 4));
  }
#pragma unroll
  for (int q = 0; q < B_INS; ++q) {
    const int r = (wid * B_INS + q) * RPI + lane / CPR;
    b_off[q] = (uint32_t)(r * Kb + (((lane % CPR) ^ tile::swz<RB>(r)) << 4));
  }
  auto load_stage = [&](uint8_t* dst, int kt) {
    const uint8_t *ab = mb[0], *bb = nb[0];
    int k = kt;
    if constexpr (SPLIT) {  // passes: lo hi, hi lo, hi hi (small terms first)
      if (kt < nk1) {
        ab = mb[1];
      } else if (kt < 2 * nk1) {
        bb = nb[1];
        k = kt - nk1;
      } else {
        k = kt - 2 * nk1;
      }
    }
    ab = uniform_ptr(ab + (int64_t)k * RB);
    bb = uniform_ptr(bb + (int64_t)k * RB);
#pragma unroll
    for (int q = 0; q < A_INS; ++q) load_lds16(ab, a_off[q], dst + (wid * A_INS + q) * 1024);
#pragma unroll
    for (int q = 0; q < B_INS; ++q) load_lds16(bb, b_off[q], dst + BM * RB + (wid * B_INS + q) * 1024);
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

  // slices 0 .. NS-2 in flight; each iteration waits for its own slice, meets the other wavefronts (the buffer read
  // last iteration is then free), refills it with slice kt + NS - 1 (clamped: loaded, never read) and computes slice kt
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) load_stage(smem + s * STAGE, min(s, nk - 1));
  int cb = 0, fb = NS - 1;
  for (int kt = 0; kt < nk; ++kt) {
    wait_vmcnt<(NS - 2) * NL>();
    __syncthreads();
    load_stage(smem + fb * STAGE, min(kt + NS - 1, nk - 1));
    const uint8_t* As = smem + cb * STAGE;
    tile::mma_stage_bf16<RB, MB, NB, f16x8_t>(As, As + BM * RB, arow, brow, ao, bo, acc);
    cb = cb + 1 == NS ? 0 : cb + 1;
    fb = fb + 1 == NS ? 0 : fb + 1;
  }
  wait_vmcnt0();
  __syncthreads();  // no load in flight, no wavefront still reading a stage: the epilogue reuses the buffers

  // ---- epilogue, 32 rows x 64 columns of a wavefront at a time through its own part of LDS, so that every global
  // access is 16 bytes per lane: by rows for the result (and the elementwise operand), by columns for the transpose.
  // Accumulator element v of a lane: row (v / 4) * 8 + 4 * (lane / 32) + v % 4, column lane % 32.
  float* sc = reinterpret_cast<float*>(smem) + wid * 32 * PITCH;
  const bool mirror = MODE == UPDATE || (SYM && mi != ni);
  const int64_t rb = e * a.r_batch;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        sc[((v >> 2) * 8 + 4 * lh + (v & 3)) * PITCH + j * 32 + lr] = acc[i][j][v];
    wave_lds_fence();
    const int row0 = m0 + wm * WTM + i * 32, col0 = n0 + wn * WTN;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int r = it * 8 + lane / 8, c = lane % 8 * 8;
      float v[8];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const f32x4_t q = *reinterpret_cast<const f32x4_t*>(&sc[r * PITCH + c + 4 * d]);
#pragma unroll
        for (int x = 0; x < 4; ++x) v[4 * d + x] = a.beta * q[x];
      }
      const int64_t at = rb + ((int64_t)(row0 + r) * a.ld + col0 + c) * 2;
      if constexpr (MODE != GRAM) {
        const f16x8_t h = *reinterpret_cast<const f16x8_t*>(a.E0 + at);
        f16x8_t l;
        if constexpr (MODE != POLY || SPLIT) l = *reinterpret_cast<const f16x8_t*>(a.E1 + at);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float ev = (float)h[x];
          if constexpr (MODE != POLY || SPLIT) ev += (float)l[x];
          v[x] = __builtin_fmaf(a.alpha, ev, v[x]);
        }
      }
      if constexpr (MODE == FINAL) {
        if (!a.flip) {
          const int gr = row0 + r, gc = col0 + c;
          if (gr < a.m && gc < a.n) {
            const int64_t o = ((int64_t)e * a.m + gr) * a.n + gc;
            if (a.out_vec) {  // n a multiple of 8: the 8 values are all inside, and aligned
              if (a.out_bf16) {
                i32x4_t w;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                  w[d] = (int)((uint32_t)f32_to_bf16_bits(v[2 * d]) | ((uint32_t)f32_to_bf16_bits(v[2 * d + 1]) << 16));
                *reinterpret_cast<i32x4_t*>(a.out + o * 2) = w;
              } else {
#pragma unroll
                for (int d = 0; d < 2; ++d)
                  *reinterpret_cast<f32x4_t*>(a.out + o * 4 + 16 * d) =
                      (f32x4_t){v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]};
              }
            } else {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if (gc + x < a.n) {
                  if (a.out_bf16)
                    reinterpret_cast<uint16_t*>(a.out)[o + x] = f32_to_bf16_bits(v[x]);
                  else
                    reinterpret_cast<float*>(a.out)[o + x] = v[x];
                }
            }
          }
        }
      } else {
        f16x8_t h, l;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          _Float16 hi, lo;
          split16(v[x], hi, lo);
          h[x] = hi;
          l[x] = lo;
        }
        *reinterpret_cast<f16x8_t*>(a.R0 + at) = h;
        if constexpr (MODE == UPDATE || SPLIT) *reinterpret_cast<f16x8_t*>(a.R1 + at) = l;
      }
      if (MODE != FINAL ? mirror : a.flip) {
#pragma unroll
        for (int d = 0; d < 2; ++d)
          *reinterpret_cast<f32x4_t*>(&sc[r * PITCH + c + 4 * d]) =
              (f32x4_t){v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]};
      }
    }
    wave_lds_fence();
    if (MODE != FINAL ? mirror : a.flip) {
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int c = it * 16 + lane / 4, r = lane % 4 * 8;
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = sc[(r + x) * PITCH + c];
        if constexpr (MODE == FINAL) {
          const int gr = col0 + c, gc = row0 + r;  // row and first column of out
          if (gr < a.m) {
            const int64_t o = ((int64_t)e * a.m + gr) * a.n + gc;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (gc + x < a.n) {
                if (a.out_bf16)
                  reinterpret_cast<uint16_t*>(a.out)[o + x] = f32_to_bf16_bits(v[x]);
                else
                  reinterpret_cast<float*>(a.out)[o + x] = v[x];
              }
          }
        } else {
          f16x8_t h, l;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            _Float16 hi, lo;
            split16(v[x], hi, lo);
            h[x] = hi;
            l[x] = lo;
          }
          const int64_t at = e * a.t_batch + ((int64_t)(col0 + c) * a.ld_t + row0 + r) * 2;
          *reinterpret_cast<f16x8_t*>(a.T0 + at) = h;
          if constexpr (SPLIT) *reinterpret_cast<f16x8_t*>(a.T1 + at) = l;
        }
      }
      wave_lds_fence();
    }
  }
}

MOE_DEV float load_g(const uint8_t* g, bool bf16, int64_t i) {
  if (bf16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(g)[i] << 16);
  return reinterpret_cast<const float*>(g)[i];
}

// part[e][chunk] = sum of the squares of the chunk's values, in fp64 (squares of fp32 values neither overflow nor vanish)
__global__ __launch_bounds__(256) void square_sum_kernel(const uint8_t* __restrict__ g, bool bf16, int64_t count,
                                                         int chunks, double* __restrict__ part) {
  __shared__ double red[4];
  const int64_t e = blockIdx.x / chunks;
  const int ch = blockIdx.x % chunks;
  const int64_t step = (count + chunks - 1) / chunks, lo = ch * step, hi = lo + step < count ? lo + step : count;
  const int64_t base = e * count;
  double s = 0.0;
  for (int64_t i = lo + threadIdx.x; i < hi; i += 256) {
    const double v = load_g(g, bf16, base + i);
    s = __builtin_fma(v, v, s);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
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
  // natural (g's rows contiguous) and transposed destinations, either hi/lo; lo may be NULL
  uint8_t *n0, *n1, *t0, *t1;
  int ld_n, ld_t;    // values per row
  int64_t batch_bytes;
};

// S g / (|g| + eps) as hi and lo, in both orientations, zero-filled past m x n
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
  for (int k = 0; k < 16; ++k) {
    const int r = k * 4 + tid / 64, c = tid % 64;
    t[r][c] = r0 + r < a.m && c0 + c < a.n ? load_g(a.g, a.bf16, (e * a.m + r0 + r) * a.n + c0 + c) : 0.0f;
  }
  __syncthreads();
  // the quotient in fp64: a gradient whose norm passes fp32's range, either way, still gives its X
  const double inv = (double)S / (sqrt(red[0] + red[1] + red[2] + red[3]) + (double)a.eps);
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // k < 2: rows of g, else columns; 8 values each
    const int q = (k & 1) * 256 + tid, r = q / 8, c = q % 8 * 8;
    f16x8_t h, l;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float v = (float)((double)(k < 2 ? t[r][c + x] : t[c + x][r]) * inv);
      _Float16 hi, lo;
      split16(v, hi, lo);
      h[x] = hi;
      l[x] = lo;
    }
    uint8_t *d0 = k < 2 ? a.n0 : a.t0, *d1 = k < 2 ? a.n1 : a.t1;
    const int64_t at = e * a.batch_bytes +
                       (k < 2 ? (int64_t)(r0 + r) * a.ld_n + c0 + c : (int64_t)(c0 + r) * a.ld_t + r0 + c) * 2;
    *reinterpret_cast<f16x8_t*>(d0 + at) = h;
    if (d1 != nullptr) *reinterpret_cast<f16x8_t*>(d1 + at) = l;
  }
}

struct Plan {
  int p, q, P, Q;
  bool flip, big;
  int chunks;
  size_t x_bytes, a_bytes;  // one fp16 array of the whole batch
  size_t part_bytes, total;
};

static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

static Plan plan(int64_t batch, int m, int n, bool split) {
  Plan z{};
  z.flip = m > n;
  z.p = z.flip ? n : m;
  z.q = z.flip ? m : n;
  // 256 x 256 tiles where the update's tiles fill the 256 compute units, 128 x 128 otherwise
  z.big = (int64_t)((z.p + 255) / 256) * ((z.q + 255) / 256) * batch >= 256;
  const int tl = z.big ? 256 : 128;
  z.P = (z.p + tl - 1) / tl * tl;
  z.Q = (z.q + tl - 1) / tl * tl;
  const int64_t count = (int64_t)m * n;
  z.chunks = (int)(count / 4096 < 1 ? 1 : count / 4096 > 256 ? 256 : count / 4096);
  z.x_bytes = (size_t)batch * z.P * z.Q * 2;
  z.a_bytes = (size_t)batch * z.P * z.P * 2;
  z.part_bytes = up256((size_t)batch * z.chunks * sizeof(double));
  z.total = z.part_bytes + (split ? 6 : 4) * z.x_bytes + (split ? 4 : 2) * z.a_bytes;
  return z;
}

template <int MODE, bool SPLIT>
static void launch_product(const Args& a0, bool big, int rows, int cols, int64_t batch, hipStream_t s) {
  Args a = a0;
  const int tl = big ? 256 : 128;
  a.mt = rows / tl;
  a.nt = cols / tl;
  const int64_t per = MODE == GRAM || MODE == POLY ? (int64_t)a.nt * (a.nt + 1) / 2 : (int64_t)a.mt * a.nt;
  const dim3 grid((unsigned)(per * batch));
  if (big)
    hipLaunchKernelGGL((product_kernel<MODE, 1, SPLIT>), grid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((product_kernel<MODE, 0, SPLIT>), grid, dim3(256), 0, s, a);
}

template <bool SPLIT>
static void run(const OrthLaunch& p, hipStream_t s) {
  const Plan z = plan(p.batch, p.m, p.n, SPLIT);
  uint8_t* ws = reinterpret_cast<uint8_t*>(p.workspace);
  auto take = [&](size_t bytes) {
    uint8_t* r = ws;
    ws += bytes;
    return r;
  };
  double* part = reinterpret_cast<double*>(take(z.part_bytes));
  uint8_t *x0 = take(z.x_bytes), *x1 = take(z.x_bytes);
  uint8_t *t0[2] = {take(z.x_bytes), take(z.x_bytes)}, *t1[2] = {nullptr, nullptr};
  uint8_t *a0 = take(z.a_bytes), *b0 = take(z.a_bytes), *a1 = nullptr, *b1 = nullptr;
  if constexpr (SPLIT) {
    t1[0] = take(z.x_bytes);
    t1[1] = take(z.x_bytes);
    a1 = take(z.a_bytes);
    b1 = take(z.a_bytes);
  }
  const uint8_t* g = reinterpret_cast<const uint8_t*>(p.g);
  hipLaunchKernelGGL(square_sum_kernel, dim3((unsigned)(p.batch * z.chunks)), dim3(256), 0, s, g, p.g_bf16,
                     (int64_t)p.m * p.n, z.chunks, part);
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
  r.n0 = z.flip ? t0[0] : x0;
  r.n1 = z.flip ? t1[0] : x1;
  r.t0 = z.flip ? x0 : t0[0];
  r.t1 = z.flip ? x1 : t1[0];
  r.ld_n = z.flip ? z.P : z.Q;
  r.ld_t = z.flip ? z.Q : z.P;
  r.batch_bytes = (int64_t)z.P * z.Q * 2;
  hipLaunchKernelGGL(prepare_kernel, dim3((unsigned)(p.batch * r.rt * r.ct)), dim3(256), 0, s, r);

  const int64_t xb = (int64_t)z.P * z.Q * 2, ab = (int64_t)z.P * z.P * 2;
  for (int k = 0; k < p.steps; ++k) {
    const int cur = k & 1, nxt = cur ^ 1;
    Args q{};
    q.M0 = q.N0 = x0;  // A = X X^T
    q.M1 = q.N1 = x1;
    q.m_batch = q.n_batch = xb;
    q.K = z.Q;
    q.R0 = q.T0 = a0;
    q.R1 = q.T1 = a1;
    q.ld = q.ld_t = z.P;
    q.r_batch = q.t_batch = ab;
    q.beta = 1.0f / S;
    launch_product<GRAM, SPLIT>(q, z.big, z.P, z.P, p.batch, s);
    q.M0 = q.N0 = q.E0 = a0;  // B = b A + c A A
    q.M1 = q.N1 = q.E1 = a1;
    q.m_batch = q.n_batch = ab;
    q.K = z.P;
    q.R0 = q.T0 = b0;
    q.R1 = q.T1 = b1;
    q.alpha = p.b;
    q.beta = p.c / S;
    launch_product<POLY, SPLIT>(q, z.big, z.P, z.P, p.batch, s);
    q.M0 = b0;  // X <- a X + B X
    q.M1 = b1;
    q.N0 = t0[cur];
    q.N1 = t1[cur];
    q.n_batch = xb;
    q.E0 = q.R0 = x0;
    q.E1 = q.R1 = x1;
    q.ld = z.Q;
    q.r_batch = q.t_batch = xb;
    q.T0 = t0[nxt];
    q.T1 = t1[nxt];
    q.ld_t = z.P;
    q.alpha = p.a;
    q.beta = 1.0f / S;
    if (k + 1 < p.steps) {
      launch_product<UPDATE, SPLIT>(q, z.big, z.P, z.Q, p.batch, s);
    } else {
      q.alpha = p.a * (p.scale / S);
      q.beta = p.scale / S / S;
      q.out = reinterpret_cast<uint8_t*>(p.out);
      q.m = p.m;
      q.n = p.n;
      q.flip = z.flip;
      q.out_bf16 = p.out_bf16;
      q.out_vec = p.n % 8 == 0 && (uintptr_t)p.out % 16 == 0;
      launch_product<FINAL, SPLIT>(q, z.big, z.P, z.Q, p.batch, s);
    }
  }
}

}  // namespace orth

size_t orthogonalize_workspace(int64_t batch, int m, int n, bool out_bf16) {
  return orth::plan(batch, m, n, !out_bf16).total;
}

void launch_orthogonalize(const OrthLaunch& p, hipStream_t s) {
  if (p.out_bf16)
    orth::run<false>(p, s);
  else
    orth::run<true>(p, s);
}

}  // namespace moe
