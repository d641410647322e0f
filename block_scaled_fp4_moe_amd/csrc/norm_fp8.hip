// rms_norm_fp8 and swiglu_fp8: the producers of 1x128 quantized activations.
//
// rms_norm_fp8: v = x + residual; y = v * weight / sqrt(mean v^2 + eps); per
// 128 values s = max(amax/448, 2^-64), code = E4M3(y/s).  One pass: a workgroup
// owns a row and keeps v in registers between the sum of squares and the
// quantization, so each input byte is read once (rows above 16384 columns twice).
// Bound by HBM at prefill sizes, 8192 x 7168 bfloat16 with a residual 86 us = 4.8 TB/s
// (a bare stream of the same four bytes read to three written: 5.8); by launch and three
// latencies (load, cross-wave sum, store) at decode sizes, 8 x 7168 5.0 us.
//
// swiglu_fp8: h = g / (1 + e^-g) * u, quantized the same way, in float32 and in 64 bits where
// a code hangs on it.  Bound by HBM, 73728 x 2048 bfloat16 137 us = 5.5 TB/s with four bytes
// read for one written (a bare stream: 6.3); by the launch at decode sizes, 72 x 2048 3.8 us.
//
// In both, a lane holds 8 consecutive values and the 16 lanes of a DPP row one
// 128-value block, so the block maximum takes four DPP steps and no LDS.
#include "fp8_block.h"

#include <numeric>

namespace fp4moe {
namespace {

struct NormParams {
  const void *x, *residual, *weight;
  void *residual_out, *y_out;
  uint8_t* codes;
  float* scales;
  int64_t ldx, ldr, ldro, ldy, ldc, scale_row, scale_blk;
  int K;
  float eps;
};

// Sum over the 64 lanes, in every lane: DPP adds within rows of 16 (rotations), then
// the four rows' sums.
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](auto ctrl) {
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  add(std::integral_constant<int, 0x128>{});
  add(std::integral_constant<int, 0x124>{});
  add(std::integral_constant<int, 0x122>{});
  add(std::integral_constant<int, 0x121>{});
  auto row = [&](int l) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
  };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// 1/sqrt(m) to about one unit: the instruction's value and one Newton step on it.  The
// instruction takes a subnormal m for zero: small ones are brought up by 2^64 before.
__device__ __forceinline__ float rsqrt_refined(float m) {
  const bool small = m < 0x1p-100f;
  m = small ? m * 0x1p64f : m;
  float r = __builtin_amdgcn_rsqf(m);
  const float e = fmaf(-m * r, r, 1.f);
  // m = 0 or infinity: r is infinity or 0 and e a NaN; a NaN m stays one
  r = (r > 0.f && r < __builtin_inff()) ? fmaf(0.5f * r, e, r) : r;
  return small ? r * 0x1p32f : r;
}

// Scale and codes of a block of y = v*inv*w.  The row's factor inv cancels in
//   y/s = 448 * (v*w) / max(v*w),
// so the codes are taken from the products p = v*w with their rounding errors e
// (exact, by fma), and 448/max as a float32 pair: one rounding before the
// conversion in place of five at no more operations, and a value next to a
// boundary between two codes falls on the right side more often.
__device__ __forceinline__ float quant8_norm(const float* v, const float* w, float inv, uint32_t* c) {
  float p[8], e[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = v[i] * w[i];
    e[i] = fmaf(v[i], w[i], -p[i]);
    top = max(top, __float_as_uint(p[i]) & 0x7fffffffu);
  }
  top = row16_max(top);
  const float m = __uint_as_float(top);
  // what the largest product's float32 value leaves out
  float lo = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    lo = fabsf(p[i]) == m ? fmaxf(lo, copysignf(1.f, p[i]) * e[i]) : lo;
  lo = row16_fmax(lo);
  const float t = m * inv, te = fmaf(m, inv, -t) + lo * inv;
  const float s = __fdiv_rn(t, 448.f) + te * (1.f / 448.f);
  // zeros, tiny or huge products, a row without a finite norm: the formula as it stands
  if (!(m >= 0x1p-80f && m <= 0x1p100f && s > 0x1p-64f && s < 0x1p100f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = (v[i] * inv) * w[i];
    return quant8_e4m3(p, c);
  }
  const float f = __fdiv_rn(448.f, m);
  const float fe = fmaf(-f, lo, fmaf(-f, m, 448.f)) * __builtin_amdgcn_rcpf(m);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fmaf(p[i], f, fmaf(e[i], f, p[i] * fe));
  e4m3_codes(q, c);
  return s;
}

// NT threads a row, at most PIECES 8-value pieces a thread; the row stays in registers
// between the sum of squares and the quantization.  All loads, the weight's among
// them, are issued before the first wait.
template <class T, bool VEC, bool STREAM, int NT, int PIECES>
__global__ __launch_bounds__(NT) void rms_norm_kernel(NormParams p, int M) {
  using E = typename T::type;
  __shared__ float part[NT / 64];
  const int tid = threadIdx.x;
  const E* wt = static_cast<const E*>(p.weight);
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const E* x = static_cast<const E*>(p.x) + row * p.ldx;
    const E* res = p.residual ? static_cast<const E*>(p.residual) + row * p.ldr : nullptr;
    float v[PIECES][8], w[PIECES][8];
    auto load_row = [&](const E* q, float (&to)[PIECES][8]) {
#pragma unroll
      for (int j = 0; j < PIECES; ++j) {
        const int k = (tid + j * NT) * 8;
        if (k < p.K) {
          load8<T, VEC>(q + k, p.K - k, to[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) to[j][i] = 0.f;
        }
      }
    };
    load_row(x, v);
    if (res) {
      float r[PIECES][8];
      load_row(res, r);
      load_row(wt, w);
#pragma unroll
      for (int j = 0; j < PIECES; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += r[j][i];
    } else {
      load_row(wt, w);
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    if (p.residual_out) {
      E* ro = static_cast<E*>(p.residual_out) + row * p.ldro;
#pragma unroll
      for (int j = 0; j < PIECES; ++j) {
        const int k = (tid + j * NT) * 8;
        if (k < p.K) store8<T, VEC, STREAM>(ro + k, p.K - k, v[j]);
      }
    }
    float sum = wave_sum(ss);
    if constexpr (NT > 64) {
      if ((tid & 63) == 0) part[tid >> 6] = sum;
      __syncthreads();
      double all = 0.0;
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) all += (double)part[i];
      sum = (float)all;
    }
    const float inv = rsqrt_refined(sum / (float)p.K + p.eps);
    E* y = p.y_out ? static_cast<E*>(p.y_out) + row * p.ldy : nullptr;
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const int k = (tid + j * NT) * 8;
      if (y && k < p.K) {
        float yv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) yv[i] = (v[j][i] * inv) * w[j][i];
        store8<T, VEC, STREAM>(y + k, p.K - k, yv);
      }
      if (p.codes) {
        // lanes past the row's end hold zeros, whose quotients can only be NaN where
        // the whole row's are
        uint32_t c[2];
        const float s = quant8_norm(v[j], w[j], inv, c);
        if (k < p.K) {
          store_codes(p.codes + row * p.ldc + k, p.K - k, VEC, c);
          if ((tid & 15) == 0) p.scales[row * p.scale_row + (int64_t)(k >> 7) * p.scale_blk] = s;
        }
      }
    }
    if constexpr (NT > 64) __syncthreads();   // the next row writes part again
  }
}

// Rows too wide for registers: x and residual are read a second time, from the caches,
// by the threads that read them first (which write residual_out then: it may be
// either of them).
template <class T, bool VEC>
__global__ __launch_bounds__(1024) void rms_norm_wide_kernel(NormParams p, int M) {
  using E = typename T::type;
  __shared__ float part[16];
  const int tid = threadIdx.x;
  const E* wt = static_cast<const E*>(p.weight);
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const E* x = static_cast<const E*>(p.x) + row * p.ldx;
    const E* res = p.residual ? static_cast<const E*>(p.residual) + row * p.ldr : nullptr;
    auto load_v = [&](int k, float* v) {
      float r[8];
      load8<T, VEC>(x + k, p.K - k, v);
      if (res) {
        load8<T, VEC>(res + k, p.K - k, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
    };
    float ss = 0.f;
    for (int k = tid * 8; k < p.K; k += 8192) {
      float v[8];
      load_v(k, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    }
    const float mine = wave_sum(ss);
    if ((tid & 63) == 0) part[tid >> 6] = mine;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) all += (double)part[i];
    const float inv = rsqrt_refined((float)all / (float)p.K + p.eps);
    // whole blocks of 128: every lane of a DPP row takes the same turns
    for (int k = tid * 8; k - (tid & 15) * 8 < p.K; k += 8192) {
      float v[8], w[8];
      if (k < p.K) {
        load_v(k, v);
        load8<T, VEC>(wt + k, p.K - k, w);
        if (p.residual_out)
          store8<T, VEC, false>(static_cast<E*>(p.residual_out) + row * p.ldro + k, p.K - k, v);
        if (p.y_out) {
          float yv[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) yv[i] = (v[i] * inv) * w[i];
          store8<T, VEC, false>(static_cast<E*>(p.y_out) + row * p.ldy + k, p.K - k, yv);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f, w[i] = 0.f;
      }
      if (p.codes) {
        uint32_t c[2];
        const float s = quant8_norm(v, w, inv, c);
        if (k < p.K) {
          store_codes(p.codes + row * p.ldc + k, p.K - k, VEC, c);
          if ((tid & 15) == 0) p.scales[row * p.scale_row + (int64_t)(k >> 7) * p.scale_blk] = s;
        }
      }
    }
    __syncthreads();   // the next row writes part again
  }
}

// e^-g for SiLU: 2^t with t = -g*log2(e) carried as a rounded product and its
// remainder, because the rounding of t alone would cost |t| * 2^-24 of relative
// error; then 1/(1 + e^-g).
//
// Lanes with a gate beyond +-80 (or a NaN) are added to `far`: their block takes the 64-bit
// form.  The remainder is left out there, and from -87.3 on the reciprocal is
// subnormal, which the instruction returns as zero.  (The comparison is the select's own,
// and the masks are joined by the scalar unit.)
__device__ __forceinline__ float silu(float g, uint64_t& far) {
  const float L = 1.44269502f, L_lo = 1.92596299e-8f;   // log2(e) in two parts
  const float t = -g * L;
  const float lo = fmaf(-g, L, -t) - g * L_lo;
  float e = __builtin_amdgcn_exp2f(t);
  const float c = e * (lo * 0.693147181f);
  const bool beyond = !(fabsf(g) <= 80.f);
  far |= __ballot(beyond);
  e = beyond ? e : e + c;                               // there the remainder may be inf - inf
  const float d = 1.f + e;
  float r = __builtin_amdgcn_rcpf(d);
  return g * r;
}

// The same in 64 bits and for any gate, to about 2^-32: 2^n * 2^f with n the integer next to
// -g*log2(e), and 2^f = e^(f ln 2) by its series up to the eighth power (|f| <= 1/2 leaves
// (ln 2/2)^9/9!).  The exponent's gate is cut at 700: beyond, 1 + e^-g is 1.  Gates below
// -108.67, whose SiLU is less than half of the smallest float32, give -0, and -infinity
// gives -infinity * 0 = NaN, as the formula does.
__device__ __forceinline__ double silu64(float g) {
  const double t = -1.4426950408889634 * (double)__builtin_amdgcn_fmed3f(g, -700.f, 700.f);
  const double n = __builtin_rint(t), f = t - n;
  double e = 1.3215486790144307e-06;
  e = fma(e, f, 1.5252733804059841e-05);
  e = fma(e, f, 1.5403530393381608e-04);
  e = fma(e, f, 1.3333558146428443e-03);
  e = fma(e, f, 9.6181291076284772e-03);
  e = fma(e, f, 5.5504108664821580e-02);
  e = fma(e, f, 2.4022650695910072e-01);
  e = fma(e, f, 6.9314718055994531e-01);
  e = fma(e, f, 1.0);
  const double d = 1.0 + __builtin_amdgcn_ldexp(e, (int)n);
  const double r = __builtin_amdgcn_rcp(d), q = fma(fma(-d, r, 1.0), r, r);
  return (double)g * (g < -108.67f ? 0.0 : q);
}

// Whether a block's largest magnitude (its bits) lies in 2^-55 .. 2^100.
__device__ __forceinline__ bool usual(uint32_t m) { return m >= 0x24000000u && m <= 0x71800000u; }

// Scale and codes of a block of h = silu(g)*u from 64-bit values.
__device__ __forceinline__ float quant8_swiglu64(const float* g, const float* u, uint32_t* c) {
  double h[8];
  float p[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = silu64(g[i]) * (double)u[i];
    p[i] = (float)h[i];
    top = max(top, __float_as_uint(p[i]) & 0x7fffffffu);
  }
  top = row16_max(top);
  if (!usual(top)) return quant8_e4m3(p, c);
  const float m = __uint_as_float(top);
  float lo = -__builtin_inff();     // what the largest value's float32 form leaves out
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float rest = (float)(h[i] - (double)p[i]);
    lo = fabsf(p[i]) == m ? fmaxf(lo, copysignf(1.f, p[i]) * rest) : lo;
  }
  const double top64 = (double)m + (double)row16_fmax(lo);
  double r = __builtin_amdgcn_rcp(top64);
  r = fma(fma(-top64, r, 1.0), r, r);
  const double f = 448.0 * r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // A quotient that float32 rounds onto the middle itself goes to the side it came from,
    // unless it is the middle but for this computation's error (gates equal to the largest
    // value's cancel, which happens with 16-bit inputs): that goes to the even code.
    const double q = h[i] * f, rest = q - (double)(float)q;
    uint32_t b = __float_as_uint((float)q);
    if ((b & 0xfffffu) == 0x80000u && fabs(rest) > fabs(q) * 0x1p-30) b += (rest > 0.0) == (q > 0.0) ? 1 : -1;
    p[i] = __uint_as_float(b);
  }
  e4m3_codes(p, c);
  return (float)(top64 * (1.0 / 448.0));
}

// Scale and codes of a block of h = silu(g)*u.  Float32 arithmetic is off by up to nine units
// of a quotient's last place (the exponential and the reciprocals one each, the other
// operations a half, twice for the quotient's two sides), which changes its code
// only where it lies that close to the middle between two codes: a block that holds such a
// quotient (one in 300 does) is computed in 64 bits instead.  In 64 bits
// throughout, 73728 x 2048 takes 246 us, so 137, in float32 alone 136 with one code in a
// million on the wrong side.  (Not looked at: quotients below 2^-6, whose codes are a fixed small
// step apart, and blocks with infinities or NaN or without a value of 2^-55 .. 2^100.)
__device__ __forceinline__ float quant8_swiglu(const float* g, const float* u, uint32_t* c) {
  float h[8];
  uint32_t m = 0;
  uint64_t far = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = silu(g[i], far) * u[i];
    m = max(m, __float_as_uint(h[i]) & 0x7fffffffu);
  }
  m = row16_max(m);
  // the block's own lanes decide, so that a row's result does not depend on its neighbours
  auto own = [](uint64_t lanes) { return ((lanes >> (threadIdx.x & 48)) & 0xffff) != 0; };
  if (far && own(far)) return quant8_swiglu64(g, u, c);
  if (!usual(m)) return quant8_e4m3(h, c);
  const float f = 448.f * __builtin_amdgcn_rcpf(__uint_as_float(m));
  constexpr uint32_t kUnits = 12;
  uint32_t near = ~0u;              // units above the middle of two codes less kUnits
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] *= f;
    near = min(near, (__float_as_uint(h[i]) - (0x80000u - kUnits)) & 0xfffffu);
  }
  const uint64_t hit = __ballot(near <= 2 * kUnits);
  if (hit && own(hit)) return quant8_swiglu64(g, u, c);
  e4m3_codes(h, c);
  return __fdiv_rn(__uint_as_float(m), 448.f);
}

template <class T, bool VEC, bool STREAM>
__global__ __launch_bounds__(256) void swiglu_kernel(const typename T::type* __restrict__ gu, int M,
                                                     int I, int blocks, int64_t ldg,
                                                     const int32_t* __restrict__ row_count,
                                                     uint8_t* __restrict__ codes, int64_t ldc,
                                                     float* __restrict__ scales, int64_t scale_row,
                                                     int64_t scale_blk) {
  const int rows = row_count ? min(M, max(*row_count, 0)) : M;
  const int total = rows * blocks;
  // 16 lanes a block, 16 blocks a workgroup
  for (int64_t b = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); b < total;
       b += (int64_t)gridDim.x * 16) {
    const int row = (int)((uint32_t)b / (uint32_t)blocks);
    const int blk = (int)b - row * blocks;
    const int k = blk * 128 + (threadIdx.x & 15) * 8;
    const typename T::type* g = gu + (int64_t)row * ldg + k;
    float gv[8], uv[8];
    if (k < I) {
      load8<T, VEC, STREAM>(g, I - k, gv);
      load8<T, VEC, STREAM>(g + I, I - k, uv);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) gv[i] = 0.f, uv[i] = 0.f;
    }
    uint32_t c[2];
    const float s = quant8_swiglu(gv, uv, c);
    if (k < I) {
      store_codes(codes + (int64_t)row * ldc + k, I - k, VEC, c);
      if ((threadIdx.x & 15) == 0) scales[row * scale_row + blk * scale_blk] = s;
    }
  }
}

template <class T, bool VEC, bool STREAM>
void launch_norm(const NormParams& p, int M, hipStream_t s) {
  const dim3 grid((unsigned)(M < (1 << 20) ? M : 1 << 20));   // a HIP grid holds fewer than 2^32 threads
  // One piece a thread where a row fits: measured at 8192 rows of 7168 (bfloat16,
  // residual), 512 threads x 2 pieces 92 us, 256 x 4 125, 128 x 7 149, 64 x 14 238; a row
  // on every CU or fewer: 1024 x 1 4.5 us at 8 rows, 512 x 2 4.8, 256 x 4 6.6.
#define FP8BLOCK_NORM(NT, PIECES) \
  hipLaunchKernelGGL((rms_norm_kernel<T, VEC, STREAM, NT, PIECES>), grid, dim3(NT), 0, s, p, M)
  if (p.K <= 512) FP8BLOCK_NORM(64, 1);
  else if (p.K <= 1024) FP8BLOCK_NORM(128, 1);
  else if (p.K <= 2048) FP8BLOCK_NORM(256, 1);
  else if (p.K <= 4096) FP8BLOCK_NORM(512, 1);
  else if (p.K <= 8192 && M <= 256) FP8BLOCK_NORM(1024, 1);
  else if (p.K <= 8192) FP8BLOCK_NORM(512, 2);
  else if (p.K <= 16384) FP8BLOCK_NORM(1024, 2);
  else hipLaunchKernelGGL((rms_norm_wide_kernel<T, VEC>), grid, dim3(1024), 0, s, p, M);
#undef FP8BLOCK_NORM
}

template <class T>
int norm_typed(const fp8block_norm_args* a, const NormParams& p, hipStream_t s) {
  constexpr int64_t E = sizeof(typename T::type);
  auto ok = [](const void* q, int64_t stride_bytes, uintptr_t n) {
    return !q || (((uintptr_t)q | (uintptr_t)stride_bytes) & (n - 1)) == 0;
  };
  const bool vec = a->K % 8 == 0 && ok(a->x, a->ldx * E, 16) && ok(a->residual, a->ldr * E, 16) &&
                   ok(a->weight, 0, 16) && ok(a->residual_out, a->ldro * E, 16) &&
                   ok(a->y_out, a->ldy * E, 16) && ok(a->codes, a->ldc, 8);
  // Results too large for the caches go past them: 8192 x 7168 bfloat16 (117 MB) 83 us
  // streamed, 90 not; 8192 x 2048 (34 MB) 27.6, 25.3.
  const bool stream = (int64_t)a->M * a->K * E > (64 << 20);
  if (!vec) launch_norm<T, false, false>(p, a->M, s);
  else if (stream) launch_norm<T, true, true>(p, a->M, s);
  else launch_norm<T, true, false>(p, a->M, s);
  return check_launch("rms_norm_fp8");
}

template <class T>
int swiglu_typed(const void* gu, int M, int I, int64_t ldg, const int32_t* row_count,
                 uint8_t* codes, int64_t ldc, float* scales, int64_t scale_row, int64_t scale_blk,
                 hipStream_t s) {
  using E = typename T::type;
  const bool vec = I % 8 == 0 && (((uintptr_t)gu | (uintptr_t)(ldg * sizeof(E)) |
                                   (uintptr_t)(I * sizeof(E))) & 15) == 0 &&
                   (((uintptr_t)codes | (uintptr_t)ldc) & 7) == 0;
  const int blocks = (I + 127) / 128;
  const int64_t want = ((int64_t)M * blocks + 15) / 16;
  const dim3 grid((unsigned)(want < 256 * 64 ? want : 256 * 64));
  const E* g = static_cast<const E*>(gu);
  // An input larger than the last cache (256 MB) is read past it: right after its
  // producer, bfloat16 I = 2048, 537 MB 113 us streamed and 137 not, 268 MB 62 and 69,
  // 201 MB 48 and 48, 101 MB 27 and 25.
  const bool stream = (int64_t)M * I * 2 * (int64_t)sizeof(E) >= (256 << 20);
#define FP8BLOCK_SWIGLU(VEC, STREAM)                                                            \
  hipLaunchKernelGGL((swiglu_kernel<T, VEC, STREAM>), grid, dim3(256), 0, s, g, M, I, blocks,   \
                     ldg, row_count, codes, ldc, scales, scale_row, scale_blk)
  if (!vec) FP8BLOCK_SWIGLU(false, false);
  else if (stream) FP8BLOCK_SWIGLU(true, true);
  else FP8BLOCK_SWIGLU(true, false);
#undef FP8BLOCK_SWIGLU
  return check_launch("swiglu_fp8");
}

bool aligned(const void* p, int dtype) {
  return ((uintptr_t)p & (dtype == FP8BLOCK_F32 ? 3 : 1)) == 0;
}

// Whether the scales of M rows of K columns lie at places of their own.  Two elements
// meet where i * row = j * blk with 0 < i < M and 0 < j < blocks, first at
// i = blk / gcd, j = row / gcd (a stride of zero: at the next row or block).
bool scales_apart(int64_t M, int64_t K, int64_t row, int64_t blk) {
  const int64_t blocks = (K + 127) / 128;
  if (M <= 1 || blocks <= 1) return (M <= 1 || row > 0) && (blocks <= 1 || blk > 0);
  if (row == 0 || blk == 0) return false;
  const int64_t g = std::gcd(row, blk);
  return blk / g >= M || row / g >= blocks;
}

// `rows` pieces of `width` bytes, `pitch` apart.
struct Piece {
  uintptr_t at;
  int64_t rows, pitch, width;
  uintptr_t end() const { return at + (rows - 1) * pitch + width; }
};

// Whether two of them have a byte in common (null ones: no).  Exact where their pitches are
// equal or one is a single row (columns of one buffer do not meet); otherwise whether the
// ranges do.
bool meet(const Piece& a, const Piece& b) {
  if (!a.at || !b.at || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const Piece &low = a.at <= b.at ? a : b, &high = a.at <= b.at ? b : a;
  if (low.rows <= 1) return true;                      // the other one starts inside it
  const int64_t d = (int64_t)((high.at - low.at) % (uintptr_t)low.pitch);
  return d < low.width || d + high.width > low.pitch;
}

// Scales as rows, or, where the rows of a block lie together, as blocks.
Piece scale_piece(const float* at, int64_t M, int64_t K, int64_t row, int64_t blk) {
  const int64_t blocks = (K + 127) / 128;
  const int64_t across = (blocks - 1) * blk + 1, down = (M - 1) * row + 1;
  const uintptr_t p = (uintptr_t)at;
  if (across <= row) return {p, M, row * 4, across * 4};
  if (down <= blk) return {p, blocks, blk * 4, down * 4};
  return {p, 1, 0, ((M - 1) * row + across) * 4};
}

// residual_out and y_out each lie on x or residual, row for row, or apart from every
// input; codes and scales apart from everything.  Rows are read and written by
// workgroups in any order, so anything else would be a race.
const char* overlap(const fp8block_norm_args* a) {
  const int64_t E = a->dtype == FP8BLOCK_F32 ? 4 : 2;
  auto rows = [&](const void* p, int64_t ld, int64_t e) {
    return Piece{(uintptr_t)p, a->M, ld * e, a->K * e};
  };
  const Piece in[] = {rows(a->x, a->ldx, E), rows(a->residual, a->ldr, E)};
  const Piece weight = {(uintptr_t)a->weight, 1, 0, a->K * E};
  const Piece out[] = {rows(a->residual_out, a->ldro, E), rows(a->y_out, a->ldy, E)};
  const Piece code[] = {rows(a->codes, a->ldc, 1),
                        scale_piece(a->scales, a->M, a->K, a->scale_row, a->scale_blk)};
  const char* names[] = {"residual_out", "y_out", "codes", "scales"};
  for (int o = 0; o < 2; ++o) {
    for (const Piece& i : in) {
      const bool same = out[o].at == i.at && (a->M == 1 || out[o].pitch == i.pitch);
      if (!same && meet(out[o], i)) return names[o];
    }
    if (meet(out[o], weight)) return names[o];
    for (const Piece& i : in)
      if (meet(code[o], i)) return names[2 + o];
    if (meet(code[o], weight) || meet(code[o], out[0]) || meet(code[o], out[1])) return names[2 + o];
  }
  if (meet(code[0], code[1])) return names[3];
  return meet(out[0], out[1]) ? names[1] : nullptr;
}

}  // namespace
}  // namespace fp4moe

using namespace fp4moe;

extern "C" int rms_norm_fp8(const fp8block_norm_args* a, void* stream) {
  FP4MOE_REQUIRE(a, "rms_norm_fp8: null args");
  FP4MOE_REQUIRE(a->dtype >= FP8BLOCK_BF16 && a->dtype <= FP8BLOCK_F32, "rms_norm_fp8: dtype=%d",
                 a->dtype);
  FP4MOE_REQUIRE(a->M >= 0 && a->K >= 1 && a->K <= 65536,
                 "rms_norm_fp8: M=%d K=%d (K at most 65536)", a->M, a->K);
  FP4MOE_REQUIRE(a->eps >= 0.f, "rms_norm_fp8: eps=%g", (double)a->eps);
  if (a->M == 0) return FP4MOE_OK;
  FP4MOE_REQUIRE(a->x && a->weight, "rms_norm_fp8: null pointer");
  FP4MOE_REQUIRE(!a->codes == !a->scales, "rms_norm_fp8: codes and scales come together");
  FP4MOE_REQUIRE(a->codes || a->y_out || a->residual_out, "rms_norm_fp8: null outputs");
  FP4MOE_REQUIRE(a->ldx >= a->K && (!a->residual || a->ldr >= a->K) &&
                     (!a->residual_out || a->ldro >= a->K) && (!a->y_out || a->ldy >= a->K) &&
                     (!a->codes || a->ldc >= a->K),
                 "rms_norm_fp8: a row stride is below K=%d", a->K);
  FP4MOE_REQUIRE(!a->scales || (a->scale_row >= 0 && a->scale_blk >= 0),
                 "rms_norm_fp8: negative scale stride");
  FP4MOE_REQUIRE(!a->scales || scales_apart(a->M, a->K, a->scale_row, a->scale_blk),
                 "rms_norm_fp8: scale strides %lld, %lld put scales on top of each other",
                 (long long)a->scale_row, (long long)a->scale_blk);
  FP4MOE_REQUIRE(aligned(a->x, a->dtype) && aligned(a->residual, a->dtype) &&
                     aligned(a->weight, a->dtype) && aligned(a->residual_out, a->dtype) &&
                     aligned(a->y_out, a->dtype) && ((uintptr_t)a->scales & 3) == 0,
                 "rms_norm_fp8: a pointer is not aligned to its element");
  const char* on = overlap(a);
  FP4MOE_REQUIRE(!on, "rms_norm_fp8: %s overlaps an input or another output", on);
  FP4MOE_CHECK_DEVICE();
  NormParams p;
  p.x = a->x, p.residual = a->residual, p.weight = a->weight;
  p.residual_out = a->residual_out, p.y_out = a->y_out;
  p.codes = a->codes, p.scales = a->scales;
  p.ldx = a->ldx, p.ldr = a->ldr, p.ldro = a->ldro, p.ldy = a->ldy, p.ldc = a->ldc;
  p.scale_row = a->scale_row, p.scale_blk = a->scale_blk;
  p.K = a->K, p.eps = a->eps;
  hipStream_t s = as_stream(stream);
  if (a->dtype == FP8BLOCK_BF16) return norm_typed<TBf16>(a, p, s);
  if (a->dtype == FP8BLOCK_F16) return norm_typed<TF16>(a, p, s);
  return norm_typed<TF32>(a, p, s);
}

extern "C" int swiglu_fp8(int dtype, const void* gate_up, int M, int I, int64_t ldg,
                          const int32_t* row_count, uint8_t* codes, int64_t ldc, float* scales,
                          int64_t scale_row, int64_t scale_blk, void* stream) {
  FP4MOE_REQUIRE(dtype >= FP8BLOCK_BF16 && dtype <= FP8BLOCK_F32, "swiglu_fp8: dtype=%d", dtype);
  FP4MOE_REQUIRE(M >= 0 && I >= 1 && I <= (1 << 30) &&
                     (int64_t)M * ((I + 127) / 128) < (int64_t)1 << 31,
                 "swiglu_fp8: M=%d I=%d", M, I);
  if (M == 0) return FP4MOE_OK;
  FP4MOE_REQUIRE(gate_up && codes && scales, "swiglu_fp8: null pointer");
  FP4MOE_REQUIRE(ldg >= 2 * (int64_t)I && ldc >= I, "swiglu_fp8: ldg=%lld ldc=%lld for I=%d",
                 (long long)ldg, (long long)ldc, I);
  FP4MOE_REQUIRE(scale_row >= 0 && scale_blk >= 0, "swiglu_fp8: negative scale stride");
  FP4MOE_REQUIRE(scales_apart(M, I, scale_row, scale_blk),
                 "swiglu_fp8: scale strides %lld, %lld put scales on top of each other",
                 (long long)scale_row, (long long)scale_blk);
  FP4MOE_REQUIRE(aligned(gate_up, dtype) && ((uintptr_t)scales & 3) == 0 &&
                     ((uintptr_t)row_count & 3) == 0,
                 "swiglu_fp8: a pointer is not aligned to its element");
  FP4MOE_CHECK_DEVICE();
  hipStream_t s = as_stream(stream);
  if (dtype == FP8BLOCK_BF16)
    return swiglu_typed<TBf16>(gate_up, M, I, ldg, row_count, codes, ldc, scales, scale_row,
                               scale_blk, s);
  if (dtype == FP8BLOCK_F16)
    return swiglu_typed<TF16>(gate_up, M, I, ldg, row_count, codes, ldc, scales, scale_row,
                              scale_blk, s);
  return swiglu_typed<TF32>(gate_up, M, I, ldg, row_count, codes, ldc, scales, scale_row,
                            scale_blk, s);
}
