// Layer norm and RMS norm of token rows, forward and backward, in front of the layer.
//
//   s = x, or x + residual rounded once to the rows' type (the stored sum is what is normalised);
//   m = mean(s) (0 for RMS norm), r = (mean((s - m)^2) + eps)^(-1/2), z = (s - m) r, y = z w + b.
//   backward, t = dy w:  ds = r (t - [mean(t)] - z mean(t z)) + dsum,   dw = sum over rows dy z,  db = sum dy
//   (the bracket for layer norm only).
//
// Bound by memory: forward reads x (and residual) and writes y (and s) once, backward reads dy and s (and dsum) and
// writes ds once; a row stays in registers between its statistics and its result.  TPR threads share a row, 16
// columns each (TPR = 16 .. 1024 by powers of two; rows above 16384 columns take 64 per thread), so a thread has two
// to four 16-byte loads of each operand in flight and the two sums of a row cost one or two exchanges: in a wavefront
// by lane shuffles, across wavefronts through LDS.  Rows whose width, strides or base addresses are not multiples of
// 16 bytes take the same code with single-element accesses (VEC = 1, the wavefront's 64 lanes side by side).
// Statistics: the mean first, then the squares of the differences, both in fp32 from registers: no cancellation of
// E[s^2] - m^2.
//
// The weight's gradient: a persistent grid of G workgroups walks the rows, each thread keeping its columns' sums in
// fp32 registers; the groups of a workgroup are added through LDS, each workgroup writes one partial row, and a second
// launch adds the G partial rows in a fixed order.  No atomics: results do not change from run to run.
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
  bool want_bias;
};

// VEC consecutive elements as fp32: bf16 (ESZ 2) or fp32 (ESZ 4)
template <int ESZ, int VEC>
MOE_DEV void load_vec(const uint8_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = ESZ == 4 ? *reinterpret_cast<const float*>(p)
                    : __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
  } else {
    constexpr int ND = VEC * ESZ / 4;  // dwords: 2, 4 or 8
    int q[ND];
    if constexpr (ND == 2) {
      const i32x2_t d = *reinterpret_cast<const i32x2_t*>(p);
      q[0] = d[0];
      q[1] = d[1];
    } else {
#pragma unroll
      for (int k = 0; k < ND / 4; ++k) {
        const i32x4_t d = reinterpret_cast<const i32x4_t*>(p)[k];
#pragma unroll
        for (int x = 0; x < 4; ++x) q[4 * k + x] = d[x];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (ESZ == 4) {
        v[e] = __int_as_float(q[e]);
      } else {
        const uint32_t u = (uint32_t)q[e / 2];
        v[e] = __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
      }
    }
  }
}
template <int ESZ, int VEC>
MOE_DEV void store_vec(uint8_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (ESZ == 4)
      *reinterpret_cast<float*>(p) = v[0];
    else
      *reinterpret_cast<uint16_t*>(p) = f32_to_bf16_bits(v[0]);
  } else {
    constexpr int NW = VEC * ESZ / 16;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      i32x4_t q;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if constexpr (ESZ == 4)
          q[d] = __float_as_int(v[k * 4 + d]);
        else
          q[d] = (int)((uint32_t)f32_to_bf16_bits(v[k * 8 + 2 * d]) |
                       ((uint32_t)f32_to_bf16_bits(v[k * 8 + 2 * d + 1]) << 16));
      }
      reinterpret_cast<i32x4_t*>(p)[k] = q;
    }
  }
}
// weight or bias columns: fp32 or bf16 by a launch-uniform flag
template <int VEC>
MOE_DEV void load_param(const uint8_t* p, bool bf16, int c, float (&v)[VEC]) {
  if (bf16)
    load_vec<2, VEC>(p + (int64_t)c * 2, v);
  else
    load_vec<4, VEC>(p + (int64_t)c * 4, v);
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

template <int ESZ, int VEC, int NV, int TPR>
__global__ __launch_bounds__((TPR < 256 ? 256 : TPR)) void norm_fwd_kernel(const FwdArgs a) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  __shared__ float red[2][THREADS / 64 * 2];
  int flip = 0;
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < a.T;
  const int64_t rr = live ? row : a.T - 1;  // surplus threads compute the last row and store nothing
  float v[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[i][e] = 0.0f;
    if (c < a.H) load_vec<ESZ, VEC>(a.x + (rr * a.ldx + c) * ESZ, v[i]);
  }
  if (a.res != nullptr) {
    float u[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[i][e] = 0.0f;
      if (c < a.H) load_vec<ESZ, VEC>(a.res + (rr * a.ldr + c) * ESZ, u[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] += u[i][e];
        if constexpr (ESZ == 2) v[i][e] = __uint_as_float((uint32_t)f32_to_bf16_bits(v[i][e]) << 16);
      }
      if (c < a.H && live) store_vec<ESZ, VEC>(a.sum + (row * a.H + c) * ESZ, v[i]);
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
  for (int i = 0; i < NV; ++i) {
    const bool in = (i * TPR + t) * VEC < a.H;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = in ? v[i][e] - m : 0.0f;
      s2[0] = __builtin_fmaf(d, d, s2[0]);
    }
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
    const bool in = c < a.H;
    float w[VEC], y[VEC];
    if (in) {
      load_param<VEC>(a.w, a.w_bf16, c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = (v[i][e] - m) * r * w[e];
      if (a.b != nullptr) {
        load_param<VEC>(a.b, a.w_bf16, c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] += w[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = 0.0f;
    }
    if constexpr (VEC > 1) {
      if (a.y_fp8) {
        // one scale per 128 columns: 128 / VEC consecutive lanes (16 for bf16 rows, 32 for fp32 rows)
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(y[e]));
#pragma unroll
        for (int o = 64 / VEC; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
        const float sc = amax > 0.0f ? amax / 448.0f : 1.0f;
        if (in && live) {
          uint32_t code[VEC / 4];
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
          uint32_t* dst = reinterpret_cast<uint32_t*>(a.y + row * a.H + c);
#pragma unroll
          for (int q = 0; q < VEC / 4; ++q) dst[q] = code[q];
          if (c % 128 == 0) a.ys[row * (a.H / 128) + c / 128] = sc;
        }
        continue;
      }
    }
    if (in && live) store_vec<ESZ, VEC>(a.y + (row * a.H + c) * ESZ, y);
  }
}

template <int ESZ, int VEC, int NV, int TPR>
__global__ __launch_bounds__((TPR < 256 ? 256 : TPR)) void norm_bwd_kernel(const BwdArgs a) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  __shared__ float red[2][THREADS / 64 * 2];
  __shared__ float comb[RPB > 1 ? TPR * NV * VEC : 1];  // sums of one column range, the groups added one by one
  int flip = 0;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv_h = 1.0f / (float)a.H;
  float dw[NV][VEC], db[NV][VEC], w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = w[i][e] = 0.0f;
    if (c < a.H) load_param<VEC>(a.w, a.w_bf16, c, w[i]);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.T; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + sub;
    const bool live = row < a.T;
    const int64_t rr = live ? row : a.T - 1;
    float z[NV][VEC], dy[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) z[i][e] = dy[i][e] = 0.0f;
      if (c < a.H && live) {
        load_vec<ESZ, VEC>(a.dy + (rr * a.ld_dy + c) * ESZ, dy[i]);
        load_vec<ESZ, VEC>(a.s + (rr * a.ld_s + c) * ESZ, z[i]);
      }
    }
    const float m = a.rms ? 0.0f : a.mean[rr];
    const float r = a.rstd[rr];
    float c12[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * TPR + t) * VEC < a.H && live;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        z[i][e] = in ? (z[i][e] - m) * r : 0.0f;
        dw[i][e] = __builtin_fmaf(dy[i][e], z[i][e], dw[i][e]);
        db[i][e] += dy[i][e];
        const float tw = dy[i][e] * w[i][e];
        c12[0] += tw;
        c12[1] = __builtin_fmaf(tw, z[i][e], c12[1]);
      }
    }
    row_sum<TPR, THREADS, 2>(c12, red, flip);
    const float c1 = a.rms ? 0.0f : c12[0] * inv_h, c2 = c12[1] * inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c < a.H && live) {
        float d[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] = (dy[i][e] * w[i][e] - c1 - z[i][e] * c2) * r;
        if (a.dsum != nullptr) {
          float u[VEC];
          load_vec<ESZ, VEC>(a.dsum + (row * a.ld_dsum + c) * ESZ, u);
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[e] += u[e];
        }
        store_vec<ESZ, VEC>(a.dx + (row * a.H + c) * ESZ, d);
      }
    }
  }
  // one partial row per workgroup
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k == 1 && !a.want_bias) break;
    float* out = a.part + ((int64_t)k * gridDim.x + blockIdx.x) * a.H;
    if constexpr (RPB > 1) {
      for (int g = RPB - 1; g >= 0; --g) {
        __syncthreads();
        if (sub == g) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const int c = (i * TPR + t) * VEC + e;
              const float v = (k == 0 ? dw[i][e] : db[i][e]) + (g == RPB - 1 ? 0.0f : comb[c]);
              if (g > 0)
                comb[c] = v;
              else if (c < a.H)
                out[c] = v;
            }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int c = (i * TPR + t) * VEC + e;
          if (c < a.H) out[c] = k == 0 ? dw[i][e] : db[i][e];
        }
    }
  }
}

// out[c] = sum over the G partial rows, in a fixed order: 32 columns and 32 row lanes per workgroup.  blockIdx.y: 0 the
// weight's partials, 1 the bias's.  G = 0 (no rows) writes zeros.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* __restrict__ part, int G, int H,
                                                           float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g0 = threadIdx.x >> 5;
  const float* p = part + (int64_t)blockIdx.y * G * H;
  float s = 0.0f;
  if (c < H)
    for (int g = g0; g < G; g += 32) s += p[(int64_t)g * H + c];
  red[g0][threadIdx.x & 31] = s;
  __syncthreads();
  if (threadIdx.x < 32 && c < H) {
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < 32; ++g) v += red[g][threadIdx.x];
    (blockIdx.y == 0 ? dw : db)[c] = v;
  }
}

// 16 columns per thread: the power of two TPR with 16 TPR >= H
static int threads_per_row(int H) {
  int t = 16;
  while (t < 1024 && t * 16 < H) t *= 2;
  return t;
}
static int rows_per_block(int H) {
  const int t = threads_per_row(H);
  return t < 256 ? 256 / t : 1;
}

template <int ESZ, int VEC, bool BWD, typename Args>
static void launch_shape(const Args& a, int tpr, unsigned grid, hipStream_t s) {
#define MOE_NORM_LAUNCH(NV, TPR)                                                                        \
  do {                                                                                                  \
    constexpr int TH = TPR < 256 ? 256 : TPR;                                                           \
    if constexpr (BWD)                                                                                  \
      hipLaunchKernelGGL((norm_bwd_kernel<ESZ, VEC, NV, TPR>), dim3(grid), dim3(TH), 0, s, a);          \
    else                                                                                                \
      hipLaunchKernelGGL((norm_fwd_kernel<ESZ, VEC, NV, TPR>), dim3(grid), dim3(TH), 0, s, a);          \
  } while (0)
  if (a.H > 16384) {
    MOE_NORM_LAUNCH(64 / VEC, 1024);
    return;
  }
  switch (tpr) {
    case 16: MOE_NORM_LAUNCH(16 / VEC, 16); break;
    case 32: MOE_NORM_LAUNCH(16 / VEC, 32); break;
    case 64: MOE_NORM_LAUNCH(16 / VEC, 64); break;
    case 128: MOE_NORM_LAUNCH(16 / VEC, 128); break;
    case 256: MOE_NORM_LAUNCH(16 / VEC, 256); break;
    case 512: MOE_NORM_LAUNCH(16 / VEC, 512); break;
    default: MOE_NORM_LAUNCH(16 / VEC, 1024); break;
  }
#undef MOE_NORM_LAUNCH
}

static bool vec_ok(const void* p, int64_t ld, int esz) {
  return p == nullptr || (((uintptr_t)p % 16) == 0 && (ld * esz) % 16 == 0);
}

}  // namespace norm

// Workgroups of the backward pass: at most four of 256 threads' worth per compute unit (256 of them), so the partial
// rows stay a few percent of the traffic.
int norm_backward_groups(int64_t T, int H) {
  const int rpb = norm::rows_per_block(H);
  const int tpr = norm::threads_per_row(H);
  const int64_t most = tpr <= 256 ? 1024 : tpr == 512 ? 512 : 256;
  const int64_t need = (T + rpb - 1) / rpb;
  return (int)(need < most ? need : most);
}

bool norm_vector_ok(const NormLaunch& p) {
  const int esz = p.dtype == MOE_DTYPE_F32 ? 4 : 2, wsz = p.w_bf16 ? 2 : 4;
  const int vec = 16 / esz;
  return p.H % vec == 0 && (p.H * wsz) % 16 == 0 && norm::vec_ok(p.x, p.ldx, esz) &&
         norm::vec_ok(p.residual, p.ldr, esz) && norm::vec_ok(p.dy, p.ld_dy, esz) &&
         norm::vec_ok(p.weight, 0, wsz) && norm::vec_ok(p.bias, 0, wsz) && norm::vec_ok(p.sum, p.H, esz) &&
         norm::vec_ok(p.y, 0, 1) && norm::vec_ok(p.dx, 0, 1);
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
  int tpr = norm::threads_per_row(p.H);
  const bool f32 = p.dtype == MOE_DTYPE_F32;
  if (p.y_fp8 && f32 && tpr < 32) tpr = 32;  // a 128-column block of fp32 rows spans 32 lanes
  const int rpb = tpr < 256 ? 256 / tpr : 1;
  const unsigned grid = (unsigned)((p.T + rpb - 1) / rpb);
  const bool vec = norm_vector_ok(p);
  if (f32)
    vec ? norm::launch_shape<4, 4, false>(a, tpr, grid, s) : norm::launch_shape<4, 1, false>(a, tpr, grid, s);
  else
    vec ? norm::launch_shape<2, 8, false>(a, tpr, grid, s) : norm::launch_shape<2, 1, false>(a, tpr, grid, s);
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
  a.want_bias = p.dbias != nullptr;
  const int tpr = norm::threads_per_row(p.H);
  const int G = norm_backward_groups(p.T, p.H);
  if (G > 0) {
    const bool vec = norm_vector_ok(p);
    if (p.dtype == MOE_DTYPE_F32)
      vec ? norm::launch_shape<4, 4, true>(a, tpr, G, s) : norm::launch_shape<4, 1, true>(a, tpr, G, s);
    else
      vec ? norm::launch_shape<2, 8, true>(a, tpr, G, s) : norm::launch_shape<2, 1, true>(a, tpr, G, s);
  }
  hipLaunchKernelGGL(norm::norm_reduce_kernel, dim3((unsigned)((p.H + 31) / 32), p.dbias != nullptr ? 2 : 1),
                     dim3(1024), 0, s, p.part, G, p.H, p.dweight, p.dbias);
}

}  // namespace moe
