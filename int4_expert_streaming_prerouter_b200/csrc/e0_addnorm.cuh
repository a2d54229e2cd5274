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
//
// Measured (a captured launch among others): 16384 rows of 2048 with e4m3 and scales 63.2 us (4.8
// TB/s; issue slots bound it, 79 % of them taken by conversions and border tests), 64 rows of 4096
// in int8 4.2 us, one row 2.8 us (a launch and its latency).
#pragma once
#include "e0_bf16.cuh"
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
  double inv_d;
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

// bf16(a + b) of the exact sum, b of 24 bits.  Rounding the fp32 sum differs from it only where that
// sum is a border between two bf16 values and not exact: what was lost (exact in fp32, by the order
// of the subtractions) then tells the side.  With b a bf16 the sum is exact, or so much nearer to
// the larger than to a border that plain rounding is right.
__device__ __forceinline__ float add_settled(float a, float b) {
  const float s = a + b;
  uint32_t u = __float_as_uint(s);
  if ((u & 0xFFFFu) == 0x8000u) {
    const float bb = s - a, lost = (a - (s - bb)) + (b - bb);
    if (lost != 0.f) u += (lost > 0.f) == (s > 0.f) ? 1u : 0xFFFFFFFFu;
  }
  return __uint_as_float(u);
}
// {lo, hi} of two fp32 numbers in bf16
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// bf16(h g rinv), rinv in 64 bits and rinv_f its fp32 rounding.  The fp32 product carries three
// roundings of half an ulp each, so it is off by at most 3 ulp.
// That holds where nothing on the way is below fp32's normal numbers, 2^-126.  rinv_f is NaN where rinv
// itself is (norm_rinv), and h rinv can be only where the result is below 2^-111 or gamma is 2^15 or more.
// (The 64-bit form stays a call: inlined at every element it would be most of the code.)
__device__ __forceinline__ float norm_rinv(double rinv) { return rinv >= 0x1p-126 ? (float)rinv : __uint_as_float(0x7FC00000u); }
__device__ __noinline__ uint32_t norm_bf16_64(float h, float g, double rinv) { return d2bf((double)h * (double)g * rinv); }

// 8 channels of h and gamma (bf16) normed; the largest of their magnitudes (as bf16 bits: a NaN is the
// largest) goes to `most`.  Results within 4 ulp of a border, or not in [2^-111, 2^112) (where the
// fp32 product, or the 2^-133 spacing of small bf16 numbers, would need care), or under a gamma of 2^15
// or more are done again.
__device__ __forceinline__ uint4 norm_bf16x8(uint4 h, uint4 g, double rinv, float rinv_f, uint32_t &most) {
  const uint32_t hs[4] = {h.x, h.y, h.z, h.w}, gs[4] = {g.x, g.y, g.z, g.w};
  uint32_t o[4], border = 0xFFFFFFFFu, low = 0xFFFFFFFFu, high = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const float p0 = bf_lo(hs[j]) * rinv_f * bf_lo(gs[j]), p1 = bf_hi(hs[j]) * rinv_f * bf_hi(gs[j]);
    o[j] = bf16x2(p0, p1);
    // the 16 dropped bits of both, plus 0x8004: at most 8 next to a border, or 9 with the carry of
    // the lower half
    border = __vminu2(border, __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x5410) + 0x80048004u);
    low = __vminu2(low, o[j] & 0x7FFF7FFFu);
    high = __vmaxu2(high, o[j] & 0x7FFF7FFFu);
  }
  most = max(high & 0xFFFFu, high >> 16);
  bool again = min(border & 0xFFFFu, border >> 16) <= 9u || most >= 0x7780u;
  if (min(low & 0xFFFFu, low >> 16) < 0x0800u) {
    // (a zero is what it is)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const uint32_t lo = o[j] & 0x7FFFu, hi = (o[j] >> 16) & 0x7FFFu;
      again |= (lo < 0x0800u && bf_lo(hs[j]) * bf_lo(gs[j]) != 0.f) || (hi < 0x0800u && bf_hi(hs[j]) * bf_hi(gs[j]) != 0.f);
    }
  }
  if ((gs[0] | gs[1] | gs[2] | gs[3]) & 0x40004000u) {
    // (a gamma of 2 or more: rare enough to look closer at)
#pragma unroll
    for (int j = 0; j < 4; j++) again |= (gs[j] & 0x7FFFu) >= 0x4700u || (gs[j] & 0x7FFF0000u) >= 0x47000000u;
  }
  if (again) {
    most = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const uint32_t lo = norm_bf16_64(bf_lo(hs[j]), bf_lo(gs[j]), rinv), hi = norm_bf16_64(bf_hi(hs[j]), bf_hi(gs[j]), rinv);
      o[j] = lo | hi << 16;
      most = max(most, max(lo & 0x7FFFu, hi & 0x7FFFu));
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The exact factor that brings a group whose largest magnitude is `a` into the range where
// the products below neither overflow nor underflow.
__device__ __forceinline__ float q8_range(float a) {
  return a < 0x1p-60f ? 0x1p70f : (a > 0x1p60f ? 0x1p-70f : 1.0f);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// p rounded to 18 significant bits (Veltkamp's splitting, each operation rounded by itself).
__device__ __forceinline__ float to_18_bits(float p) {
  const float c = __fmul_rn(p, 65.0f);
  return __fsub_rn(c, __fsub_rn(c, p));
}

// The codes of 8 channels; f, inv ~ M / a with x f inv = x M / a.  A quotient x M / a that is not a border
// t between two codes differs from it by 2^-16 t or more: |x| M and t a are products of 8 bits by 7 (M) and
// of 8 bits (t; 5 for e4m3) by 8, so in units of their last bit they are whole numbers below 2^16.  The fp32
// product below is off by less than 2^-21, so rounding it to 18 bits gives t where x M / a = t, and a number
// on the right side of t otherwise; rounding that to a code, ties to even, rounds x M / a.
__device__ __forceinline__ uint2 q8_codes(uint4 x, float f, float inv, int e4m3) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
  float p[8];
#pragma unroll
  for (int j = 0; j < 8; j++) p[j] = to_18_bits((j & 1 ? bf_hi(xs[j >> 1]) : bf_lo(xs[j >> 1])) * f * inv);
  if (e4m3) return make_uint2(e4m3x2(p[0], p[1]) | e4m3x2(p[2], p[3]) << 16, e4m3x2(p[4], p[5]) | e4m3x2(p[6], p[7]) << 16);
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; j++) c[j] = __float_as_uint(p[j] + 12582912.0f);      // 1.5 2^23: the integer is in the low bits
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

// 8 channels from c on (those past d are zero), one by one
__device__ __forceinline__ uint4 load8_single(const uint16_t *p, int c, int d) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (c + j < d) w[j >> 1] |= (uint32_t)p[c + j] << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8_single(uint16_t *p, int c, int d, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (c + j < d) p[c + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}

constexpr int addnorm_threads(int V) { return V == 4 ? 1024 : 512; }

// One row per block; thread i holds the 8-channel chunks i, i + blockDim, ... (V of them) in
// registers, so every input is read once.  VEC: rows and strides allow 16-byte
// accesses and d % 8 == 0; otherwise each element is accessed by itself.
template <int V, bool VEC>
__global__ void __launch_bounds__(addnorm_threads(V)) k_add_rmsnorm(const __grid_constant__ AddNormArgs A) {
  __shared__ double red[32];
  __shared__ uint32_t redm[32];
  const long long row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, nwarp = blockDim.x >> 5, d = A.d;
  const uint16_t *h = A.h + row * A.h_stride;
  uint4 x[V];
  auto at = [&](int v) { return 8 * (tid + v * (int)blockDim.x); };
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int c = at(v);
    if (VEC)
      x[v] = c < d ? __ldcs(reinterpret_cast<const uint4 *>(h + c)) : make_uint4(0, 0, 0, 0);
    else
      x[v] = load8_single(h, c, d);
  }
  if (A.delta && !A.delta_f32) {
    const uint16_t *p = (const uint16_t *)A.delta + row * A.delta_stride;
    uint4 e[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int c = at(v);
      if (VEC)
        e[v] = c < d ? __ldcs(reinterpret_cast<const uint4 *>(p + c)) : make_uint4(0, 0, 0, 0);
      else
        e[v] = load8_single(p, c, d);
    }
#pragma unroll
    for (int v = 0; v < V; v++)
      x[v] = make_uint4(bf16x2(bf_lo(x[v].x) + bf_lo(e[v].x), bf_hi(x[v].x) + bf_hi(e[v].x)),
                        bf16x2(bf_lo(x[v].y) + bf_lo(e[v].y), bf_hi(x[v].y) + bf_hi(e[v].y)),
                        bf16x2(bf_lo(x[v].z) + bf_lo(e[v].z), bf_hi(x[v].z) + bf_hi(e[v].z)),
                        bf16x2(bf_lo(x[v].w) + bf_lo(e[v].w), bf_hi(x[v].w) + bf_hi(e[v].w)));
  } else if (A.delta) {
    const float *p = (const float *)A.delta + row * A.delta_stride;
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int c = at(v);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      if (VEC) {
        if (c < d) {
          a = __ldcs(reinterpret_cast<const float4 *>(p + c));
          b = __ldcs(reinterpret_cast<const float4 *>(p + c + 4));
        }
      } else {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] = c + j < d ? p[c + j] : 0.f;
        a = make_float4(w[0], w[1], w[2], w[3]);
        b = make_float4(w[4], w[5], w[6], w[7]);
      }
      x[v] = make_uint4(bf16x2(add_settled(bf_lo(x[v].x), a.x), add_settled(bf_hi(x[v].x), a.y)),
                        bf16x2(add_settled(bf_lo(x[v].y), a.z), add_settled(bf_hi(x[v].y), a.w)),
                        bf16x2(add_settled(bf_lo(x[v].z), b.x), add_settled(bf_hi(x[v].z), b.y)),
                        bf16x2(add_settled(bf_lo(x[v].w), b.z), add_settled(bf_hi(x[v].w), b.w)));
    }
  }
  auto store = [&](uint16_t *out, long long stride) {
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int c = at(v);
      if (VEC) {
        if (c < d) *reinterpret_cast<uint4 *>(out + row * stride + c) = x[v];
      } else {
        store8_single(out + row * stride, c, d, x[v]);
      }
    }
  };
  if (A.h_out && (A.delta || A.h_out != A.h)) store(A.h_out, A.h_out_stride);
  if (!A.x && !A.q8) return;
  // sum of squares in 64 bits: a bf16's square and their sum keep every bit that matters
  double ss = 0.0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const uint32_t w[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const double lo = (double)bf_lo(w[j]), hi = (double)bf_hi(w[j]);
      ss = fma(lo, lo, fma(hi, hi, ss));
    }
  }
  ss = warp_sum(ss);
  if (nwarp > 1) {
    if (lane == 0) red[tid >> 5] = ss;
    __syncthreads();
    // the same order on every thread: lane by lane over the warps, at most 32
    ss = lane < nwarp ? red[lane] : 0.0;
    ss = warp_sum(ss);
  }
  const double rinv = rsqrt(fma(ss, A.inv_d, (double)A.eps));
  const float rinv_f = norm_rinv(rinv);
  uint32_t gm[V], rowmax = 0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int c = at(v);
    uint4 g = make_uint4(0, 0, 0, 0);
    if (VEC) {
      if (c < d) g = __ldg(reinterpret_cast<const uint4 *>(A.gamma + c));
    } else {
      g = load8_single(A.gamma, c, d);
    }
    // (past the end, h and gamma are zero: a NaN or 0 that is neither stored nor counted)
    gm[v] = 0;
    if (c < d) x[v] = norm_bf16x8(x[v], g, rinv, rinv_f, gm[v]);
    if (!VEC && c < d && c + 8 > d) {
      // the ragged last chunk: zero what lies past the end
      const int n = d - c;
      const uint32_t keep[4] = {n > 1 ? 0xFFFFFFFFu : 0xFFFFu, n > 3 ? 0xFFFFFFFFu : n > 2 ? 0xFFFFu : 0u,
                                n > 5 ? 0xFFFFFFFFu : n > 4 ? 0xFFFFu : 0u, n > 6 ? 0xFFFFu : 0u};
      x[v] = make_uint4(x[v].x & keep[0], x[v].y & keep[1], x[v].z & keep[2], x[v].w & keep[3]);
      const uint32_t m = __vmaxu2(__vmaxu2(x[v].x & 0x7FFF7FFFu, x[v].y & 0x7FFF7FFFu),
                                  __vmaxu2(x[v].z & 0x7FFF7FFFu, x[v].w & 0x7FFF7FFFu));
      gm[v] = max(m & 0xFFFFu, m >> 16);
    }
  }
  if (A.x) store(A.x, A.x_stride);
  if (!A.q8) return;
#pragma unroll
  for (int v = 0; v < V; v++) {
    uint32_t m = gm[v];
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
    rowmax = __reduce_max_sync(0xffffffffu, rowmax);
    if (nwarp > 1) {
      if (lane == 0) redm[tid >> 5] = rowmax;
      __syncthreads();
#pragma unroll 4
      for (int w = 0; w < nwarp; w++) rowmax = max(rowmax, redm[w]);
    }
#pragma unroll
    for (int v = 0; v < V; v++) gm[v] = rowmax;
  }
  const float M = A.q8_e4m3 ? 448.0f : 127.0f;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int c = at(v);
    if (c >= d) continue;
    const float a = bf(gm[v]);
    const bool ok = gm[v] < 0x7F80u;
    if (A.q8_group ? (c & (A.q8_group - 1)) == 0 : c == 0)
      A.q8_scale[row * A.groups + (A.q8_group ? c / A.q8_group : 0)] = ok ? a / M : __uint_as_float(0x7FC00000u);
    const float f = q8_range(a), af = a * f;
    const float inv = ok && a > 0.f ? __fdividef(M, af) : 0.f;      // off by 2 ulp at most
    uint2 q = make_uint2(0, 0);
    if (inv > 0.f) q = q8_codes(x[v], f, inv, A.q8_e4m3);
    uint8_t *p = A.q8 + row * A.q8_stride + c;
    if (VEC) {
      *reinterpret_cast<uint2 *>(p) = q;
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (c + j < d) p[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
    }
  }
}

}  // namespace e0
