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
// (The 64-bit form stays a call: inlined at every element it would be most of the code.)
__device__ __noinline__ uint32_t norm_bf16_64(float h, float g, double rinv) { return d2bf((double)h * (double)g * rinv); }

// 8 channels of h and gamma (bf16) normed; the largest of their magnitudes (as bf16 bits: a NaN is the
// largest) goes to `most`.  Results within 4 ulp of a border, or not in [2^-111, 2^112) (where the
// fp32 product, or the 2^-133 spacing of small bf16 numbers, would need care), are done again.
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
  if (min(border & 0xFFFFu, border >> 16) <= 9u || (min(low & 0xFFFFu, low >> 16) < 0x0800u && rinv_f > 0.f) || most >= 0x7780u) {
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

// x M / a moved off a rounding border in the direction of the exact quotient: p approximates
// it to 2^-22 relative, t is the border next to it.
__device__ __forceinline__ float q8_settle(float t, float xm, float a) {
  const float ta = t * a;
  const float up = __uint_as_float(__float_as_uint(t) + 64u), dn = __uint_as_float(__float_as_uint(t) - 64u);
  return xm > ta ? up : (xm < ta ? dn : t);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The codes of 8 channels x (already times q8_range), each decided at its border; a call, like the
// 64-bit form above, since few chunks need it.
__device__ __noinline__ uint2 q8_settled(uint4 x, float f, float inv, float a, int e4m3) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[2] = {0, 0};
#pragma unroll 1
  for (int j = 0; j < 8; j++) {
    const uint32_t w = j < 2 ? xs[0] : j < 4 ? xs[1] : j < 6 ? xs[2] : xs[3];
    const float v = (j & 1 ? bf_hi(w) : bf_lo(w)) * f;
    float p = fabsf(v) * inv;
    uint32_t code;
    if (e4m3) {
      // the border: three bits below the leading one, or (below 2^-6) odd multiples of 2^-10
      const float t = p >= 0x1p-6f ? __uint_as_float((__float_as_uint(p) & 0xFFF00000u) | 0x00080000u)
                                   : (rintf(p * 512.0f - 0.5f) + 0.5f) * 0x1p-9f;
      if (fabsf(p - t) <= 0x1p-18f * t) p = q8_settle(t, fabsf(v) * 448.0f, a);
      code = (e4m3x2(p, 0.f) & 0x7Fu) | (v < 0.f ? 0x80u : 0u);
    } else {
      const float t = rintf(p - 0.5f) + 0.5f;              // the border k + 1/2 nearest to p
      if (fabsf(p - t) < 0x1p-14f) p = q8_settle(t, fabsf(v) * 127.0f, a);
      const int c = (int)rintf(p);
      code = (uint32_t)(v < 0.f ? -c : c) & 255u;
    }
    q[j >> 2] |= code << (8 * (j & 3));
  }
  return make_uint2(q[0], q[1]);
}

// The codes of 8 channels: where x times an inv a little larger and a little smaller (by more than
// its error) round to the same codes, those; else each is decided at its border.
__device__ __forceinline__ uint2 q8_codes(uint4 x, float f, float inv, float a, int e4m3) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
  uint2 q;
  bool same = f == 1.0f;
  if (e4m3) {
    const float up = inv * (1.0f + 0x1p-19f), dn = inv * (1.0f - 0x1p-19f);
    uint32_t u[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      u[j] = e4m3x2(bf_lo(xs[j]) * up, bf_hi(xs[j]) * up);
      w[j] = e4m3x2(bf_lo(xs[j]) * dn, bf_hi(xs[j]) * dn);
    }
    q = make_uint2(u[0] | u[1] << 16, u[2] | u[3] << 16);
    same &= q.x == (w[0] | w[1] << 16) && q.y == (w[2] | w[3] << 16);
  } else {
    // + 1.5 2^23: the integer is in the low bits
    const float up = inv * (1.0f + 0x1p-20f), dn = inv * (1.0f - 0x1p-20f);
    uint32_t u[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float v = j & 1 ? bf_hi(xs[j >> 1]) : bf_lo(xs[j >> 1]);
      u[j] = __float_as_uint(fmaf(v, up, 12582912.0f));
      w[j] = __float_as_uint(fmaf(v, dn, 12582912.0f));
    }
    auto pack = [](const uint32_t *c) { return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410); };
    q = make_uint2(pack(u), pack(u + 4));
    same &= q.x == pack(w) && q.y == pack(w + 4);
  }
  return same ? q : q8_settled(x, f, inv, a, e4m3);
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
    ss = 0.0;
#pragma unroll 4
    for (int w = 0; w < nwarp; w++) ss += red[w];       // the same order on every thread
  }
  const double rinv = rsqrt(ss / d + (double)A.eps);
  const float rinv_f = (float)rinv;
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
    if (inv > 0.f) q = q8_codes(x[v], f, inv, af, A.q8_e4m3);
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
