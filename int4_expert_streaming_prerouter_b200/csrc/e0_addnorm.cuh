// Residual addition + RMSNorm with an optional 8-bit output (e0_add_rmsnorm).
//
//   h' = bf16(h + delta)                              (the exact sum rounded once)
//   x  = bf16(h' gamma / sqrt(mean(h'^2) + eps))      (evaluated in 64 bits, rounded once)
//   per token and group G of consecutive channels:  a = max |x_G|,  scale = a / M  (fp32),
//   q = x M / a to the nearest int8 (M = 127) or e4m3 (M = 448), ties to even
//
// Every rounding is that of the exact value, so the outputs do not depend on how the row is
// split over threads.  The 64-bit arithmetic is only done where it decides: a value is first
// computed in fp32 with an error of at most 3 ulp, and only one that lies within 4 ulp of a
// bf16 rounding border (9 of 65536) is computed again in 64 bits.  q is decided from
// x M / a, not from x / scale: the border t between two codes is compared as |x| M against
// t a, two products of few significant bits that fp32 holds exactly.
#pragma once
#include "e0_device.cuh"

namespace e0 {

struct AddNormArgs {
  const uint16_t *h;
  long long h_stride;
  const void *delta;        // bf16 or fp32 [T, d], or nullptr
  int delta_f32;
  long long delta_stride;
  const uint16_t *gamma;
  float eps;
  int T, d;
  uint16_t *h_out;
  long long h_out_stride;
  uint16_t *x;
  long long x_stride;
  uint8_t *q8;
  long long q8_stride;
  int q8_e4m3;              // 0: int8, 1: e4m3
  int q8_group;             // 64, 128 or 0 (one group a row)
  float *q8_scale;          // [T, groups]
  int groups;
};

// bf16(a + b) of the exact sum.  Rounding the fp32 sum differs from it only where that sum is a
// border between two bf16 values and not exact: what was lost (exact in fp32, by the order of the
// subtractions) then tells the side.
__device__ __forceinline__ uint16_t add_bf16(float a, float b) {
  const float s = a + b;
  uint32_t u = __float_as_uint(s);
  if ((u & 0xFFFFu) == 0x8000u) {
    const float bb = s - a, lost = (a - (s - bb)) + (b - bb);
    if (lost != 0.f) u += (lost > 0.f) == (s > 0.f) ? 1u : 0xFFFFFFFFu;
  }
  return f2bf(__uint_as_float(u));
}

// bf16(h g rinv), rinv in 64 bits and rinv_f its fp32 rounding.  The fp32 product carries three
// roundings of half an ulp each, so it is off by at most 3 ulp.
// (The 64-bit form stays a call: inlined at every element it would be most of the code.)
__device__ __noinline__ uint32_t norm_bf16_64(float h, float g, double rinv) { return d2bf((double)h * (double)g * rinv); }

__device__ __forceinline__ uint32_t norm_bf16(float h, float g, double rinv, float rinv_f) {
  const float p = h * rinv_f * g;
  const uint32_t u = __float_as_uint(p);
  const uint32_t e = (u >> 23) & 255u;
  if ((u & 0xFFFFu) - 0x7FFCu <= 8u || e - 16u > 222u) return norm_bf16_64(h, g, rinv);
  return f2bf(p);
}

// The exact factor that brings a group whose largest magnitude is `a` into the range where
// the products below neither overflow nor underflow.
__device__ __forceinline__ float q8_range(float a) {
  return a < 0x1p-60f ? 0x1p70f : (a > 0x1p60f ? 0x1p-70f : 1.0f);
}

// x M / a moved off a rounding border in the direction of the exact quotient: p approximates
// it to 2^-22 relative, t is the border next to it.
__device__ __forceinline__ float q8_settle(float p, float t, float xm, float a) {
  const float ta = t * a;
  const float up = __uint_as_float(__float_as_uint(t) + 64u), dn = __uint_as_float(__float_as_uint(t) - 64u);
  return xm > ta ? up : (xm < ta ? dn : t);
}

// code of x (already times q8_range) for inv ~ M / a
__device__ __forceinline__ uint32_t q8_int8(float x, float inv, float a) {
  float p = fabsf(x) * inv;
  const float t = rintf(p - 0.5f) + 0.5f;              // the border k + 1/2 nearest to p
  if (fabsf(p - t) < 0x1p-14f) p = q8_settle(p, t, fabsf(x) * 127.0f, a);
  const int q = (int)rintf(p);
  return (uint32_t)(x < 0.f ? -q : q) & 255u;
}

__device__ __forceinline__ uint32_t q8_e4m3(float x, float inv, float a) {
  float p = fabsf(x) * inv;
  float t;
  if (p >= 0x1p-6f) {                                   // three bits below the leading one
    t = __uint_as_float((__float_as_uint(p) & 0xFFF00000u) | 0x00080000u);
  } else {                                              // spacing 2^-9
    t = (rintf(p * 512.0f - 0.5f) + 0.5f) * 0x1p-9f;
  }
  if (fabsf(p - t) <= 0x1p-18f * t) p = q8_settle(p, t, fabsf(x) * 448.0f, a);
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(p));
  return (uint32_t)r | (x < 0.f ? 0x80u : 0u);
}

// One row per block; thread i holds the 8-element chunks i, i + blockDim, ... (V of them) in
// registers, so every input is read once.  VEC: rows and strides allow 16-byte accesses and
// d % 8 == 0; otherwise each element is accessed by itself.
template <int V, bool VEC>
__global__ void __launch_bounds__(1024) k_add_rmsnorm(AddNormArgs A) {
  __shared__ double red[32];
  __shared__ uint32_t redm[32];
  const long long row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
  const int d = A.d;
  const uint16_t *h = A.h + row * A.h_stride;
  float hv[V][8];
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int c = 8 * (tid + v * (int)blockDim.x);
    if (VEC) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (c < d) w = *reinterpret_cast<const uint4 *>(h + c);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        hv[v][2 * j] = __uint_as_float(ws[j] << 16);
        hv[v][2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) hv[v][j] = c + j < d ? bf(h[c + j]) : 0.f;
    }
  }
  if (A.delta) {
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int c = 8 * (tid + v * (int)blockDim.x);
      float dv[8];
#pragma unroll
      for (int j = 0; j < 8; j++) dv[j] = 0.f;
      if (A.delta_f32) {
        const float *p = (const float *)A.delta + row * A.delta_stride + c;
        if (VEC) {
          if (c < d) {
            const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
            dv[0] = a.x; dv[1] = a.y; dv[2] = a.z; dv[3] = a.w;
            dv[4] = b.x; dv[5] = b.y; dv[6] = b.z; dv[7] = b.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++)
            if (c + j < d) dv[j] = p[j];
        }
      } else {
        const uint16_t *p = (const uint16_t *)A.delta + row * A.delta_stride + c;
        if (VEC) {
          if (c < d) {
            const uint4 w = *reinterpret_cast<const uint4 *>(p);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
              dv[2 * j] = __uint_as_float(ws[j] << 16);
              dv[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++)
            if (c + j < d) dv[j] = bf(p[j]);
        }
      }
      uint16_t o[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        o[j] = add_bf16(hv[v][j], dv[j]);
        hv[v][j] = bf(o[j]);
      }
      if (A.h_out) {
        uint16_t *p = A.h_out + row * A.h_out_stride + c;
        if (VEC) {
          if (c < d)
            *reinterpret_cast<uint4 *>(p) = make_uint4(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16,
                                                       o[4] | (uint32_t)o[5] << 16, o[6] | (uint32_t)o[7] << 16);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++)
            if (c + j < d) p[j] = o[j];
        }
      }
    }
  } else if (A.h_out && A.h_out != A.h) {
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int c = 8 * (tid + v * (int)blockDim.x);
      uint16_t *p = A.h_out + row * A.h_out_stride + c;
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; j++) o[j] = __float_as_uint(hv[v][j]) >> 16;
      if (VEC) {
        if (c < d)
          *reinterpret_cast<uint4 *>(p) = make_uint4(o[0] | o[1] << 16, o[2] | o[3] << 16, o[4] | o[5] << 16, o[6] | o[7] << 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (c + j < d) p[j] = (uint16_t)o[j];
      }
    }
  }
  if (!A.x && !A.q8) return;
  // sum of squares in 64 bits: a bf16's square and their sum keep every bit that matters
  double ss = 0.0;
#pragma unroll
  for (int v = 0; v < V; v++)
#pragma unroll
    for (int j = 0; j < 8; j++) ss = fma((double)hv[v][j], (double)hv[v][j], ss);
  ss = warp_sum(ss);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  ss = 0.0;
  for (int w = 0; w < nwarp; w++) ss += red[w];         // the same order on every thread
  const double rinv = rsqrt(ss / d + (double)A.eps);
  const float rinv_f = (float)rinv;
  uint32_t rowmax = 0;
  uint32_t xb[V][4];
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int c = 8 * (tid + v * (int)blockDim.x);
    float g[8];
    if (VEC) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (c < d) w = __ldg(reinterpret_cast<const uint4 *>(A.gamma + c));
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        g[2 * j] = __uint_as_float(ws[j] << 16);
        g[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) g[j] = c + j < d ? bf(A.gamma[c + j]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const uint32_t b0 = c + 2 * j < d ? norm_bf16(hv[v][2 * j], g[2 * j], rinv, rinv_f) : 0u;
      const uint32_t b1 = c + 2 * j + 1 < d ? norm_bf16(hv[v][2 * j + 1], g[2 * j + 1], rinv, rinv_f) : 0u;
      xb[v][j] = b0 | (b1 << 16);
    }
    if (A.x) {
      uint16_t *p = A.x + row * A.x_stride + c;
      if (VEC) {
        if (c < d) *reinterpret_cast<uint4 *>(p) = make_uint4(xb[v][0], xb[v][1], xb[v][2], xb[v][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (c + j < d) p[j] = (uint16_t)(xb[v][j >> 1] >> (16 * (j & 1)));
      }
    }
  }
  if (!A.q8) return;
  // largest magnitude of each group, compared as integers so that a NaN is the largest
  uint32_t gm[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) m = max(m, max(xb[v][j] & 0x7FFFu, (xb[v][j] >> 16) & 0x7FFFu));
    if (A.q8_group) {
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
      if (A.q8_group == 128) m = max(m, __shfl_xor_sync(0xffffffffu, m, 8));
    }
    gm[v] = m;
    rowmax = max(rowmax, m);
  }
  if (!A.q8_group) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rowmax = max(rowmax, __shfl_xor_sync(0xffffffffu, rowmax, o));
    if (lane == 0) redm[warp] = rowmax;
    __syncthreads();
    for (int w = 0; w < nwarp; w++) rowmax = max(rowmax, redm[w]);
#pragma unroll
    for (int v = 0; v < V; v++) gm[v] = rowmax;
  }
  const float M = A.q8_e4m3 ? 448.0f : 127.0f;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int c = 8 * (tid + v * (int)blockDim.x);
    if (c >= d) continue;
    const float a = bf(gm[v]);
    const bool ok = gm[v] < 0x7F80u;
    const float scale = ok ? a / M : __uint_as_float(0x7FC00000u);
    if (A.q8_group ? c % A.q8_group == 0 : c == 0)
      A.q8_scale[row * A.groups + (A.q8_group ? c / A.q8_group : 0)] = scale;
    const float f = q8_range(a), af = a * f;
    const float inv = ok && a > 0.f ? M / af : 0.f;
    uint32_t q[2] = {0, 0};
    if (inv > 0.f) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float xv = __uint_as_float(j & 1 ? xb[v][j >> 1] & 0xFFFF0000u : xb[v][j >> 1] << 16) * f;
        const uint32_t code = A.q8_e4m3 ? q8_e4m3(xv, inv, af) : q8_int8(xv, inv, af);
        q[j >> 2] |= code << (8 * (j & 3));
      }
    }
    uint8_t *p = A.q8 + row * A.q8_stride + c;
    if (VEC) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (c + j < d) p[j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
    }
  }
}

}  // namespace e0
