// Layer norm and RMS norm of token rows, forward and backward, in front of the layer.
//
//   s = x, or x + residual rounded once to the rows' type (the stored sum is what is normalised);
//   m = mean(s) (0 for RMS norm), r = (mean((s - m)^2) + eps)^(-1/2), z = (s - m) r, y = z w + b.
//   backward, t = dy w:  ds = r (t - [mean(t)] - z mean(t z)) + dsum,   dw = sum over rows dy z,  db = sum dy
//   (the bracket for layer norm only).
//
// Bound by memory: forward reads x (and residual) and writes y (and s) once, backward reads dy and s (and dsum) and
// writes ds once; a row stays in registers between its statistics and its result.  TPR threads share a row, 16
// columns each (TPR = 16 .. 1024 by powers of two; bf16 rows 24 where fewer threads then idle; above 16384 columns forward ones
// 64, and wide backward ones take a form of their own), so a thread has two to four 16-byte loads of each operand in flight
// and the two sums of a row cost one or two exchanges: in a wavefront by lane shuffles, across wavefronts through LDS.
// Rows of any width, stride and alignment take the same 16-byte accesses, at the element's alignment; only a row's last
// few elements go one by one.
// Statistics: the mean first, then the squares of the differences, both in fp32 from registers: no cancellation of
// E[s^2] - m^2.
//
// The weight's gradient: a persistent grid of G workgroups walks the rows, each thread keeping its columns' sums in
// fp32 registers; the groups of a workgroup are added through LDS, each workgroup writes one partial row, and a second
// launch adds the G partial rows in a fixed order.  No atomics: results do not change from run to run.
//
// Measured, 16384 x 4096 bf16: forward 53 us (5.1 TB/s), backward with both parameters' gradients 81 us (5.0 TB/s), where a
// device copy of that size runs at 5.4 TB/s.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace norm {

struct FwdArgs {
  const uint8_t* x;
  const uint8_t* res;  // NULL: none
  int64_t ldx, ldr;    // elements
  int64_t T;
  int H;
  const uint8_t* w;
  const uint8_t* b;  // NULL: none
  bool w_bf16, rms, y_fp8;
  float eps;
  uint8_t* sum;  // stored sum, with res
  uint8_t* y;
  float* ys;  // fp8: scale per row and 128 columns
  float *mean, *rstd;  // either may be NULL
};

struct BwdArgs {
  const uint8_t* dy;
  const uint8_t* s;
  const uint8_t* dsum;  // NULL: none
  int64_t ld_dy, ld_s, ld_dsum;
  int64_t T;
  int H;
  const uint8_t* w;
  bool w_bf16, rms;
  const float *mean, *rstd;
  uint8_t* dx;
  float* part;  // [2][G][H]: weight partials, then bias partials
  float *dw, *db;  // where one workgroup is all: the results themselves
  float* sums;     // wide rows: [T][2], mean(t) and mean(t z)
};

// 16 bytes of a row (VEC = 16 / ESZ elements), at the elements' own alignment: one wide access, which the memory system
// splits where it crosses a line.  TAIL: H is no multiple of VEC (a variant of its own: the code costs registers).  Then the
// thread with a row's last few elements either loads them one by one (SINGLE), or loads the row's last 16 bytes, and
// settle16 moves the elements to their places where they are used, zeros behind them.  bf16 rows take the second form, in
// both directions (seven loads otherwise: forward 9717 x 1741 42.7 -> 34.6 us, backward 4252 x 10362 97 -> 72), fp32 rows
// backward only, where loads run ahead of their use (32627 x 642 92 -> 77; forward 2000 x 15001 52 -> 53 or more), and
// there without a condition on the load, which would wait for it (78 -> 133).  Rows of less than 16 bytes go one by one.
typedef int i32x4_e4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x4_e2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef int i32x2_e2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef int i32_e2_t __attribute__((aligned(2)));

template <int ESZ, bool TAIL, bool SINGLE>
MOE_DEV i32x4_t fetch_row16(const uint8_t* row, int c, int H) {
  constexpr int VEC = 16 / ESZ;
  i32x4_t q = {0, 0, 0, 0};
  if (TAIL && (SINGLE ? c + VEC > H : H < VEC)) {
    const uint8_t* p = row + (uint32_t)(c * ESZ);
#pragma unroll
    for (int e = 0; e < VEC - 1; ++e)
      if (c + e < H) {
        if constexpr (ESZ == 4)
          q[e] = reinterpret_cast<const int*>(p)[e];
        else
          q[e / 2] |= (int)((uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1)));
      }
  } else if ((TAIL && ESZ == 4) || c < H) {
    const uint8_t* p = row + (uint32_t)((TAIL && !SINGLE && c + VEC > H ? H - VEC : c) * ESZ);
    if constexpr (ESZ == 4)
      q = *reinterpret_cast<const i32x4_e4_t*>(p);
    else
      q = *reinterpret_cast<const i32x4_e2_t*>(p);
  }
  return q;
}
template <int ESZ, bool TAIL, bool SINGLE>
MOE_DEV void settle16(i32x4_t& q, int c, int H) {
  constexpr int VEC = 16 / ESZ;
  if (!TAIL || SINGLE || H < VEC || c + VEC <= H || (ESZ == 2 && c >= H)) return;
  const int k = VEC - H % VEC;             // elements in front of this thread's own, the same in every thread
  const int words = ESZ == 4 ? k : k / 2;  // 0 .. 3
  if (words & 1) q = (i32x4_t){q[1], q[2], q[3], 0};
  if (words & 2) q = (i32x4_t){q[2], q[3], 0, 0};
  if (ESZ == 2 && (k & 1))
#pragma unroll
    for (int d = 0; d < 4; ++d) q[d] = (int)__builtin_amdgcn_alignbit(d < 3 ? (uint32_t)q[d + 1] : 0u, (uint32_t)q[d], 16);
  if (ESZ == 4 && c >= H) q = (i32x4_t){0, 0, 0, 0};
}
template <int ESZ, bool TAIL>
MOE_DEV i32x4_t load_row16(const uint8_t* row, int c, int H) {
  i32x4_t q = fetch_row16<ESZ, TAIL, ESZ == 4>(row, c, H);
  settle16<ESZ, TAIL, ESZ == 4>(q, c, H);
  return q;
}
template <int ESZ>
MOE_DEV float element(const i32x4_t& q, int e) {
  if constexpr (ESZ == 4) return __int_as_float(q[e]);
  const uint32_t u = (uint32_t)q[e / 2];
  return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
}
template <int ESZ, bool TAIL, int VEC>
MOE_DEV void store_row16(uint8_t* row, int c, int H, const float (&v)[VEC]) {
  if (c >= H) return;
  uint8_t* p = row + (uint32_t)(c * ESZ);
  i32x4_t q;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (ESZ == 4)
      q[d] = __float_as_int(v[d]);
    else
      q[d] = (int)((uint32_t)f32_to_bf16_bits(v[2 * d]) | ((uint32_t)f32_to_bf16_bits(v[2 * d + 1]) << 16));
  }
  if (!TAIL || c + VEC <= H) {
    if constexpr (ESZ == 4)
      *reinterpret_cast<i32x4_e4_t*>(p) = q;
    else
      *reinterpret_cast<i32x4_e2_t*>(p) = q;
    return;
  }
  if constexpr (ESZ == 4) {
#pragma unroll
    for (int e = 0; e < VEC - 1; ++e)
      if (c + e < H) reinterpret_cast<float*>(p)[e] = v[e];
  } else {  // the last H % VEC elements as 8, 4 and 2 bytes
    const int words = H % VEC / 2;
    if (words & 2) *reinterpret_cast<i32x2_e2_t*>(p) = (i32x2_t){q[0], q[1]};
    if (words & 1) *reinterpret_cast<i32_e2_t*>(p + (words & 2) * 4) = words & 2 ? q[2] : q[0];
    if (H & 1)
      *reinterpret_cast<uint16_t*>(p + words * 4) =
          (uint16_t)(words == 0 ? q[0] : words == 1 ? q[1] : words == 2 ? q[2] : q[3]);
  }
}
// VEC columns of the weight or bias: fp32 or bf16 by a launch-uniform flag; 0 past H
template <int VEC, bool TAIL>
MOE_DEV void load_param(const uint8_t* p, bool bf16, int c, int H, float (&v)[VEC]) {
  if (bf16 && VEC == 8) {
    const i32x4_t q = load_row16<2, TAIL>(p, c, H);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = element<2>(q, e);
  } else if (bf16) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      v[e] = c + e < H ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[c + e] << 16) : 0.0f;
  } else {
#pragma unroll
    for (int d = 0; d < VEC / 4; ++d) {
      const i32x4_t q = load_row16<4, TAIL>(p, c + 4 * d, H);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * d + e] = element<4>(q, e);
    }
  }
}

// The row group of this thread; one per wavefront or several wavefronts per group: a scalar, and the row's addresses with it.
template <int TPR>
MOE_DEV int row_group() {
  if constexpr (TPR >= 64) return uniform_int(threadIdx.x / TPR);
  return threadIdx.x / TPR;
}

// Sum of one or two values over the TPR threads of a row, to all of them, in a fixed order.  `red` has a slot per
// wavefront and value; `flip` alternates its two halves, so a slot is rewritten only after the barrier that follows
// its last read.
template <int TPR, int THREADS, int N>
MOE_DEV void row_sum(float (&v)[N], float (*red)[THREADS / 64 * 2], int& flip) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o >= 1; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wid = threadIdx.x >> 6;
    float* slot = red[flip];
    flip ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) slot[wid * 2 + k] = v[k];
    __syncthreads();
    const int w0 = wid / W * W;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.0f;
#pragma unroll
    for (int q = 0; q < W; ++q)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += slot[(w0 + q) * 2 + k];
  }
}

template <int ESZ, int NV, int TPR, bool TAIL>
__global__ __launch_bounds__((TPR < 256 ? 256 : TPR)) void norm_fwd_kernel(const FwdArgs a) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR, VEC = 16 / ESZ;
  __shared__ float red[2][THREADS / 64 * 2];
  int flip = 0;
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + row_group<TPR>();
  const bool live = row < a.T;
  const int64_t rr = live ? row : a.T - 1;  // surplus threads compute the last row and store nothing
  i32x4_t raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) raw[i] = fetch_row16<ESZ, TAIL, ESZ == 4>(a.x + rr * a.ldx * ESZ, (i * TPR + t) * VEC, a.H);
  float v[NV][VEC];
  if (a.res != nullptr) {
    i32x4_t res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) res[i] = fetch_row16<ESZ, TAIL, ESZ == 4>(a.res + rr * a.ldr * ESZ, (i * TPR + t) * VEC, a.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      settle16<ESZ, TAIL, ESZ == 4>(raw[i], (i * TPR + t) * VEC, a.H);
      settle16<ESZ, TAIL, ESZ == 4>(res[i], (i * TPR + t) * VEC, a.H);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = element<ESZ>(raw[i], e) + element<ESZ>(res[i], e);
        if constexpr (ESZ == 2) v[i][e] = __uint_as_float((uint32_t)f32_to_bf16_bits(v[i][e]) << 16);
      }
      if (live) store_row16<ESZ, TAIL, VEC>(a.sum + row * a.H * ESZ, (i * TPR + t) * VEC, a.H, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      settle16<ESZ, TAIL, ESZ == 4>(raw[i], (i * TPR + t) * VEC, a.H);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = element<ESZ>(raw[i], e);
    }
  }
  const float h = (float)a.H;
  float m = 0.0f;
  if (!a.rms) {
    float s1[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s1[0] += v[i][e];
    row_sum<TPR, THREADS, 1>(s1, red, flip);
    m = s1[0] / h;
  }
  float s2[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[i][e] = (i * TPR + t) * VEC + (TAIL ? e : 0) < a.H ? v[i][e] - m : 0.0f;
      s2[0] = __builtin_fmaf(v[i][e], v[i][e], s2[0]);
    }
  row_sum<TPR, THREADS, 1>(s2, red, flip);
  const float r = 1.0f / sqrtf(s2[0] / h + a.eps);
  if (t == 0 && live) {
    if (a.mean != nullptr && !a.rms) a.mean[row] = m;
    if (a.rstd != nullptr) a.rstd[row] = r;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    float w[VEC], y[VEC];
    load_param<VEC, TAIL>(a.w, a.w_bf16, c, a.H, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) y[e] = v[i][e] * r * w[e];
    if (a.b != nullptr) {
      load_param<VEC, TAIL>(a.b, a.w_bf16, c, a.H, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] += w[e];
    }
    if (a.y_fp8) {
      // one scale per 128 columns: 128 / VEC consecutive lanes (16 for bf16 rows, 32 for fp32 rows); H % 128 == 0
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(y[e]));  // past H: 0 or NaN, which is not counted
#pragma unroll
      for (int o = 64 / VEC; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
      const float q448 = amax / 448.0f, sc = q448 > 0.0f ? q448 : 1.0f;  // 0 too where amax is below 448 * 2^-150
      if (c < a.H && live) {
        uint32_t code[VEC / 4];
        if (sc > 0x1p-80f && sc < 0x1p100f) {
          // y / sc as q + (y - q sc) / sc: the difference is exact and the second term corrects q's last bit, so this
          // rounds as the division does, at three operations a value for ten or more (8192 x 7168 with a residual 96 ->
          // 80 us, without one 65 -> 47).  |y / sc| is at most 448 and its last bit: no clamp; NaN converts to NaN.
          const float rc = 1.0f / sc;
#pragma unroll
          for (int q = 0; q < VEC / 4; ++q) {
            float d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v0 = y[q * 4 + e], q0 = v0 * rc;
              d[e] = __builtin_fmaf(__builtin_fmaf(-q0, sc, v0), rc, q0);
            }
            const int low = __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], 0, false);
            code[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(d[2], d[3], low, true);
          }
        } else {
#pragma unroll
          for (int q = 0; q < VEC / 4; ++q) {
            float d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = y[q * 4 + e] / sc;
            code[q] = f32x2_to_e4m3x2(d[0], d[1]) | (f32x2_to_e4m3x2(d[2], d[3]) << 16);
#pragma unroll
            for (int e = 0; e < 4; ++e)  // the clamp of the conversion takes NaN for a number: its code is set here
              if (d[e] != d[e]) code[q] = (code[q] & ~(0xFFu << (8 * e))) | (0x7Fu << (8 * e));
          }
        }
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.y + row * a.H + c);
        if constexpr (VEC == 8)
          *reinterpret_cast<i32x2_t*>(dst) = (i32x2_t){(int)code[0], (int)code[1]};
        else
          dst[0] = code[0];
        if (c % 128 == 0) a.ys[row * (a.H / 128) + c / 128] = sc;
      }
    } else if (live) {
      store_row16<ESZ, TAIL, VEC>(a.y + row * a.H * ESZ, c, a.H, y);
    }
  }
}

// BIAS: whether the bias's gradient is wanted (its sums take as many registers as the weight's)
template <int ESZ, int NV, int TPR, bool TAIL, bool BIAS>
__global__ __launch_bounds__((TPR < 256 ? 256 : TPR)) void norm_bwd_kernel(const BwdArgs a) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR, VEC = 16 / ESZ, WAVES = THREADS / 64;
  constexpr int COLS = TPR * NV * VEC;
  // wavefronts that hold the same columns: their sums meet in LDS
  constexpr int SHARE = TPR < 64 ? WAVES : RPB, PER = WAVES / SHARE;
  __shared__ float red[2][THREADS / 64 * 2];
  __shared__ float comb[SHARE > 1 ? SHARE * COLS : 1];
  int flip = 0;
  const int t = threadIdx.x % TPR, sub = row_group<TPR>();
  const float h = (float)a.H;
  float dw[NV][VEC], db[BIAS ? NV : 1][VEC], w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      dw[i][e] = 0.0f;
      if constexpr (BIAS) db[i][e] = 0.0f;
    }
    load_param<VEC, TAIL>(a.w, a.w_bf16, (i * TPR + t) * VEC, a.H, w[i]);
  }
  const int64_t step = (int64_t)gridDim.x * RPB;
  i32x4_t qy[NV], qs[NV];  // the next row, loaded while the one before is summed
  float m = 0.0f, r = 0.0f;
  auto fetch = [&](int64_t r0) {
    const int64_t row = r0 + sub < a.T ? r0 + sub : a.T - 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      qy[i] = fetch_row16<ESZ, TAIL, false>(a.dy + row * a.ld_dy * ESZ, c, a.H);
      qs[i] = fetch_row16<ESZ, TAIL, false>(a.s + row * a.ld_s * ESZ, c, a.H);
    }
    if (!a.rms) m = a.mean[row];
    r = a.rstd[row];
  };
  int64_t r0 = (int64_t)blockIdx.x * RPB;
  if (r0 < a.T) fetch(r0);
  for (; r0 < a.T; r0 += step) {
    const int64_t row = r0 + sub;
    const bool live = row < a.T;
    float z[NV][VEC], tw[NV][VEC];
    const float rs = r;
    float c12[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      settle16<ESZ, TAIL, false>(qy[i], (i * TPR + t) * VEC, a.H);
      settle16<ESZ, TAIL, false>(qs[i], (i * TPR + t) * VEC, a.H);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const bool in = (i * TPR + t) * VEC + (TAIL ? e : 0) < a.H && live;
        const float dy = in ? element<ESZ>(qy[i], e) : 0.0f;
        z[i][e] = in ? (element<ESZ>(qs[i], e) - m) * rs : 0.0f;
        dw[i][e] = __builtin_fmaf(dy, z[i][e], dw[i][e]);
        if constexpr (BIAS) db[i][e] += dy;
        tw[i][e] = dy * w[i][e];
        c12[0] += tw[i][e];
        c12[1] = __builtin_fmaf(tw[i][e], z[i][e], c12[1]);
      }
    }
    i32x4_t qd[NV];
    if (a.dsum != nullptr) {
      const int64_t rr = live ? row : a.T - 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) qd[i] = fetch_row16<ESZ, TAIL, false>(a.dsum + rr * a.ld_dsum * ESZ, (i * TPR + t) * VEC, a.H);
    }
    if (r0 + step < a.T) fetch(r0 + step);
    row_sum<TPR, THREADS, 2>(c12, red, flip);
    const float c1 = a.rms ? 0.0f : c12[0] / h, c2 = c12[1] / h;
    if (live)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float d[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] = (tw[i][e] - c1 - z[i][e] * c2) * rs;
        if (a.dsum != nullptr) {
          settle16<ESZ, TAIL, false>(qd[i], (i * TPR + t) * VEC, a.H);
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[e] += element<ESZ>(qd[i], e);
        }
        store_row16<ESZ, TAIL, VEC>(a.dx + row * a.H * ESZ, (i * TPR + t) * VEC, a.H, d);
      }
  }
  // one partial row per workgroup: the row groups of a wavefront are added by lane exchanges, the wavefronts in LDS
#pragma unroll
  for (int k = 0; k < (BIAS ? 2 : 1); ++k) {
    float* out = gridDim.x == 1 ? (k == 0 ? a.dw : a.db) : a.part + ((int64_t)k * gridDim.x + blockIdx.x) * a.H;
    float v[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = k == 0 ? dw[i][e] : db[BIAS ? i : 0][e];
#pragma unroll
        for (int o = TPR; o < 64; o <<= 1) v[i][e] += __shfl_xor(v[i][e], o, 64);
      }
    if constexpr (SHARE > 1) {
      if (k > 0) __syncthreads();
      const int share = (threadIdx.x >> 6) / PER;
      if (TPR >= 64 || (threadIdx.x & 63) < TPR)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) comb[share * COLS + (i * TPR + t) * VEC + e] = v[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < COLS; c += THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < SHARE; ++q) s += comb[q * COLS + c];
        if (c < a.H) out[c] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int d = 0; d < VEC / 4; ++d)
          store_row16<4, TAIL, 4>(reinterpret_cast<uint8_t*>(out), (i * TPR + t) * VEC + 4 * d, a.H,
                            reinterpret_cast<const float(&)[4]>(v[i][4 * d]));
    }
  }
}

// Wide rows: a thread would hold more columns' sums than it has registers (with them spilled, 3640 x 18432 took 3.3 ms; this
// form takes 0.14).  The rows' two sums in a launch of their own, then the rest column by column: five passes over
// rows instead of three.
template <int ESZ, bool TAIL>
__global__ __launch_bounds__(256) void norm_bwd_sums_kernel(const BwdArgs a) {
  constexpr int VEC = 16 / ESZ;
  __shared__ float red[2][8];
  int flip = 0;
  const int64_t row = blockIdx.x;
  const float m = a.rms ? 0.0f : a.mean[row], r = a.rstd[row];
  float c12[2] = {0.0f, 0.0f};
#pragma unroll 2
  for (int c = (int)threadIdx.x * VEC; c < a.H; c += 256 * VEC) {
    const i32x4_t qy = load_row16<ESZ, TAIL>(a.dy + row * a.ld_dy * ESZ, c, a.H);
    const i32x4_t qs = load_row16<ESZ, TAIL>(a.s + row * a.ld_s * ESZ, c, a.H);
    float w[VEC];
    load_param<VEC, TAIL>(a.w, a.w_bf16, c, a.H, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const bool in = !TAIL || c + e < a.H;
      const float z = in ? (element<ESZ>(qs, e) - m) * r : 0.0f;
      const float tw = element<ESZ>(qy, e) * w[e];
      c12[0] += tw;
      c12[1] = __builtin_fmaf(tw, z, c12[1]);
    }
  }
  row_sum<256, 256, 2>(c12, red, flip);
  if (threadIdx.x == 0) {
    a.sums[2 * row] = a.rms ? 0.0f : c12[0] / (float)a.H;
    a.sums[2 * row + 1] = c12[1] / (float)a.H;
  }
}

constexpr int SPAN = 4096;  // columns of a workgroup of the kernel below

// blockIdx.x: column span, blockIdx.y: row group; one partial row span per workgroup
template <int ESZ, bool TAIL, bool BIAS>
__global__ __launch_bounds__(256) void norm_bwd_span_kernel(const BwdArgs a) {
  constexpr int VEC = 16 / ESZ, NV = ESZ;
  const int c0 = blockIdx.x * SPAN, G = gridDim.y;
  float dw[NV][VEC], db[BIAS ? NV : 1][VEC], w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      dw[i][e] = 0.0f;
      if constexpr (BIAS) db[i][e] = 0.0f;
      w[i][e] = 0.0f;
    }
    const int c = c0 + (i * 256 + (int)threadIdx.x) * VEC;
    load_param<VEC, TAIL>(a.w, a.w_bf16, c, a.H, w[i]);
  }
  for (int64_t row = blockIdx.y; row < a.T; row += G) {
    const float m = a.rms ? 0.0f : a.mean[row], r = a.rstd[row], c1 = a.sums[2 * row], c2 = a.sums[2 * row + 1];
    i32x4_t qy[NV], qs[NV], qd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + (i * 256 + (int)threadIdx.x) * VEC;
      qy[i] = load_row16<ESZ, TAIL>(a.dy + row * a.ld_dy * ESZ, c, a.H);
      qs[i] = load_row16<ESZ, TAIL>(a.s + row * a.ld_s * ESZ, c, a.H);
      if (a.dsum != nullptr) qd[i] = load_row16<ESZ, TAIL>(a.dsum + row * a.ld_dsum * ESZ, c, a.H);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + (i * 256 + (int)threadIdx.x) * VEC;
      float d[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const bool in = c + (TAIL ? e : 0) < a.H;
        const float dy = element<ESZ>(qy[i], e), z = in ? (element<ESZ>(qs[i], e) - m) * r : 0.0f;
        dw[i][e] = __builtin_fmaf(dy, z, dw[i][e]);
        if constexpr (BIAS) db[i][e] += dy;
        d[e] = (dy * w[i][e] - c1 - z * c2) * r;
        if (a.dsum != nullptr) d[e] += element<ESZ>(qd[i], e);
      }
      store_row16<ESZ, TAIL, VEC>(a.dx + row * a.H * ESZ, c, a.H, d);
    }
  }
#pragma unroll
  for (int k = 0; k < (BIAS ? 2 : 1); ++k) {
    float* out = a.part + ((int64_t)k * G + blockIdx.y) * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int d = 0; d < VEC / 4; ++d)
        store_row16<4, TAIL, 4>(reinterpret_cast<uint8_t*>(out), c0 + (i * 256 + (int)threadIdx.x) * VEC + 4 * d, a.H,
                                reinterpret_cast<const float(&)[4]>((k == 0 ? dw[i] : db[BIAS ? i : 0])[4 * d]));
  }
}

// out[c] = sum over the G partial rows, in a fixed order: 32 columns (8 threads of 4) and 32 row lanes per workgroup.
// blockIdx.y: 0 the weight's partials, 1 the bias's.  G = 0 (no rows) writes zeros.
__global__ __launch_bounds__(256) void norm_reduce_kernel(const float* __restrict__ part, int G, int H,
                                                          float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float red[32][33];
  const int q = threadIdx.x & 7, g0 = threadIdx.x >> 3, c = blockIdx.x * 32 + q * 4;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(part + (int64_t)blockIdx.y * G * H);
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int g = g0; g < G; g += 32) {
    const i32x4_t v = load_row16<4, true>(p + (int64_t)g * H * 4, c, H);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += __int_as_float(v[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[g0][q * 4 + e] = s[e];
  __syncthreads();
  const int col = blockIdx.x * 32 + (int)threadIdx.x;
  if (threadIdx.x < 32 && col < H) {
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < 32; ++g) v += red[g][threadIdx.x];
    (blockIdx.y == 0 ? dw : db)[col] = v;
  }
}

// 16 columns per thread: the power of two TPR with 16 TPR >= H
static int threads_per_row(int H) {
  int t = 16;
  while (t < 1024 && t * 16 < H) t *= 2;
  return t;
}
// bf16 rows: half the threads with 24 columns each where that holds the row and leaves fewer threads without any.  Forward
// (2304 columns 4.7 -> 5.4 TB/s, 5120 4.8 -> 5.4, 9216 4.35 -> 5.3) whenever it does; backward, which has half as many
// wavefronts then, up to 5/8 of the width (2304 columns 4.0 -> 5.1 TB/s, 4608 4.8 -> 5.1; 6144 loses, 5.3 -> 4.9), and
// instead of 1024 threads always (9216 3.4 -> 5.1).  fp32 rows, whose threads have four loads each already, lose (forward,
// 5120 5.1 -> 4.9).
static int threads_per_row(int H, bool f32, bool backward) {
  const int t = threads_per_row(H);
  return !f32 && t >= 128 && H <= (backward && t < 1024 ? 10 : 12) * t ? t / 2 : t;
}

enum Kind { FWD, BWD, BWD_BIAS };

// Whether the backward pass takes the form of wide rows.  512 threads hold rows of up to 8192 columns (bf16: 12288) with
// their sums in registers (4.5 to 5.1 TB/s); of 1024 threads each has half the registers, which bf16 rows without a bias's
// sums fit (3.8 TB/s at 16384 columns) and others spill out of (1.2 to 2.3); the form of wide rows runs at 2.8 whatever the
// width.
static bool wide(int H, bool f32, bool bias) {
  return H > 16384 || (H > 8192 && f32) || (H > 12288 && bias);
}
static int64_t wide_groups(int64_t T, int H) {
  const int64_t most = 1024 / ((H + SPAN - 1) / SPAN);
  return T < most ? T : most;
}

template <int ESZ, Kind KIND, bool TAIL, int NV, int TPR, typename Args>
static void launch_tail(const Args& a, unsigned grid, hipStream_t s) {
  constexpr int TH = TPR < 256 ? 256 : TPR;
  if constexpr (KIND == FWD)
    hipLaunchKernelGGL((norm_fwd_kernel<ESZ, NV, TPR, TAIL>), dim3(grid), dim3(TH), 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<ESZ, NV, TPR, TAIL, KIND == BWD_BIAS>), dim3(grid), dim3(TH), 0, s, a);
}

template <int ESZ, Kind KIND, int NV, int TPR, typename Args>
static void launch_tpr(const Args& a, unsigned grid, hipStream_t s) {
  if (a.H % (16 / ESZ) != 0)
    launch_tail<ESZ, KIND, true, NV, TPR>(a, grid, s);
  else
    launch_tail<ESZ, KIND, false, NV, TPR>(a, grid, s);
}

template <int ESZ, Kind KIND, typename Args>
static void launch_shape(const Args& a, int tpr, unsigned grid, hipStream_t s) {
  constexpr int NV = ESZ;  // 16 columns per thread
  if constexpr (KIND == FWD)
    if (a.H > 16384) return launch_tpr<ESZ, KIND, 4 * NV, 1024>(a, grid, s);
  if constexpr (ESZ == 2)
    if (a.H > 16 * tpr) {  // 24 columns per thread
      switch (tpr) {
        case 64: return launch_tpr<ESZ, KIND, 3, 64>(a, grid, s);
        case 128: return launch_tpr<ESZ, KIND, 3, 128>(a, grid, s);
        case 256: return launch_tpr<ESZ, KIND, 3, 256>(a, grid, s);
        default: return launch_tpr<ESZ, KIND, 3, 512>(a, grid, s);
      }
    }
  if constexpr (KIND == FWD || (KIND == BWD && ESZ == 2))  // else wide()
    if (tpr == 1024) return launch_tpr<ESZ, KIND, NV, 1024>(a, grid, s);
  switch (tpr) {
    case 16: return launch_tpr<ESZ, KIND, NV, 16>(a, grid, s);
    case 32: return launch_tpr<ESZ, KIND, NV, 32>(a, grid, s);
    case 64: return launch_tpr<ESZ, KIND, NV, 64>(a, grid, s);
    case 128: return launch_tpr<ESZ, KIND, NV, 128>(a, grid, s);
    case 256: return launch_tpr<ESZ, KIND, NV, 256>(a, grid, s);
    default: return launch_tpr<ESZ, KIND, NV, 512>(a, grid, s);
  }
}

template <int ESZ, bool TAIL>
static void launch_wide(const BwdArgs& a, bool bias, int G, hipStream_t s) {
  hipLaunchKernelGGL((norm_bwd_sums_kernel<ESZ, TAIL>), dim3((unsigned)a.T), dim3(256), 0, s, a);
  const dim3 grid((unsigned)((a.H + SPAN - 1) / SPAN), (unsigned)G);
  if (bias)
    hipLaunchKernelGGL((norm_bwd_span_kernel<ESZ, TAIL, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_span_kernel<ESZ, TAIL, false>), grid, dim3(256), 0, s, a);
}

}  // namespace norm

// Workgroups of the backward pass.  Two of 256 threads or one larger one per compute unit: with the next row on its way
// while a row is summed that many keep the memory busy, and the partial rows stay a few percent of the traffic
// (16384 x 4096 bf16 with bias: 512 workgroups 81 us, 1024 95 us, 256 128 us).  And no more than leaves each four passes
// over its rows (2048 x 4096: 512 workgroups 18.5 us, 1024 19.8 us), but at least one per compute unit.
static int64_t backward_groups(int64_t T, int tpr) {
  const int rpb = tpr < 256 ? 256 / tpr : 1;
  const int64_t most = tpr <= 256 ? 512 : 256;
  const int64_t need = (T + rpb - 1) / rpb;
  if (T > 0 && need <= 4) return 1;  // a few passes of one workgroup cost less than a second launch
  int64_t g = need / 4;
  if (g < 256) g = need < 256 ? need : 256;
  return g < most ? g : most;
}

// Partial rows, and for wide rows the sums of every row: what the largest of the forms that rows of H columns can take needs.
size_t norm_backward_floats(int64_t T, int H) {
  size_t most = 0;
  for (int f32 = 0; f32 < 2; ++f32)
    for (int bias = 0; bias < 2; ++bias) {
      const bool wide = norm::wide(H, f32, bias);
      const size_t G = wide ? norm::wide_groups(T, H) : backward_groups(T, norm::threads_per_row(H, f32, true));
      const size_t floats = 2 * G * (size_t)H + (wide ? 2 * (size_t)T : 0);
      if (floats > most) most = floats;
    }
  return most;
}

void launch_norm(const NormLaunch& p, hipStream_t s) {
  norm::FwdArgs a{};
  a.x = (const uint8_t*)p.x;
  a.res = (const uint8_t*)p.residual;
  a.ldx = p.ldx;
  a.ldr = p.ldr;
  a.T = p.T;
  a.H = p.H;
  a.w = (const uint8_t*)p.weight;
  a.b = (const uint8_t*)p.bias;
  a.w_bf16 = p.w_bf16;
  a.rms = p.rms;
  a.y_fp8 = p.y_fp8;
  a.eps = p.eps;
  a.sum = (uint8_t*)p.sum;
  a.y = (uint8_t*)p.y;
  a.ys = p.y_scales;
  a.mean = p.mean;
  a.rstd = p.rstd;
  const bool f32 = p.dtype == MOE_DTYPE_F32;
  int tpr = norm::threads_per_row(p.H, f32, false);
  if (p.y_fp8 && f32 && tpr < 32) tpr = 32;  // a 128-column block of fp32 rows spans 32 lanes
  const int rpb = tpr < 256 ? 256 / tpr : 1;
  const int64_t most = (1ll << 31) / (tpr < 256 ? 256 : tpr) * rpb;  // rows of a launch: a grid has less than 2^32 threads
  const size_t es = f32 ? 4 : 2;
  for (int64_t left = p.T; left > 0; left -= a.T) {
    a.T = left < most ? left : most;
    const unsigned grid = (unsigned)((a.T + rpb - 1) / rpb);
    if (f32)
      norm::launch_shape<4, norm::FWD>(a, tpr, grid, s);
    else
      norm::launch_shape<2, norm::FWD>(a, tpr, grid, s);
    a.x += a.T * a.ldx * es;
    if (a.res != nullptr) {
      a.res += a.T * a.ldr * es;
      a.sum += a.T * a.H * es;
    }
    a.y += a.T * a.H * (a.y_fp8 ? 1 : es);
    if (a.y_fp8) a.ys += a.T * (a.H / 128);
    if (a.mean != nullptr) a.mean += a.T;
    if (a.rstd != nullptr) a.rstd += a.T;
  }
}

void launch_norm_backward(const NormLaunch& p, hipStream_t s) {
  norm::BwdArgs a{};
  a.dy = (const uint8_t*)p.dy;
  a.s = (const uint8_t*)p.x;
  a.dsum = (const uint8_t*)p.residual;
  a.ld_dy = p.ld_dy;
  a.ld_s = p.ldx;
  a.ld_dsum = p.ldr;
  a.T = p.T;
  a.H = p.H;
  a.w = (const uint8_t*)p.weight;
  a.w_bf16 = p.w_bf16;
  a.rms = p.rms;
  a.mean = p.mean;
  a.rstd = p.rstd;
  a.dx = (uint8_t*)p.dx;
  a.part = p.part;
  a.dw = p.dweight;
  a.db = p.dbias;
  const bool f32 = p.dtype == MOE_DTYPE_F32;
  const int tpr = norm::threads_per_row(p.H, f32, true);
  const bool bias = p.dbias != nullptr, wide = norm::wide(p.H, f32, bias);
  const int G = (int)(wide ? norm::wide_groups(p.T, p.H) : backward_groups(p.T, tpr));
  if (G > 0 && wide) {
    a.sums = p.part + 2 * (size_t)G * p.H;
    const bool tail = p.H % (f32 ? 4 : 8) != 0;
    if (f32)
      tail ? norm::launch_wide<4, true>(a, bias, G, s) : norm::launch_wide<4, false>(a, bias, G, s);
    else
      tail ? norm::launch_wide<2, true>(a, bias, G, s) : norm::launch_wide<2, false>(a, bias, G, s);
  } else if (G > 0) {
    if (f32)
      bias ? norm::launch_shape<4, norm::BWD_BIAS>(a, tpr, G, s) : norm::launch_shape<4, norm::BWD>(a, tpr, G, s);
    else
      bias ? norm::launch_shape<2, norm::BWD_BIAS>(a, tpr, G, s) : norm::launch_shape<2, norm::BWD>(a, tpr, G, s);
  }
  if (G == 1 && !wide) return;  // it has written the sums themselves
  hipLaunchKernelGGL(norm::norm_reduce_kernel, dim3((unsigned)((p.H + 31) / 32), p.dbias != nullptr ? 2 : 1),
                     dim3(256), 0, s, p.part, G, p.H, p.dweight, p.dbias);
}

}  // namespace moe
