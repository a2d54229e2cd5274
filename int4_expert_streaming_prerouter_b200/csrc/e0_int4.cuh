// Products of a few tokens with a matrix in the int4 affine group format (e0_int4_linear).
//
//   W[n, k] = s[n, k / g] q[n, k] + m[n, k / g],  g = 64 or 128
//   y[t, n] = sum_k W[n, k] x[t, k]
//           = sum over groups G of 64:  s sum_{k in G} q x  +  m sum_{k in G} x
//
// The inner sums run on the tensor cores (mma.sync m16n8k16, fp16 operands, fp32
// accumulation): 16 weight rows by 8 tokens by 16 channels.  A weight word holds 8 codes
// n0..n7; masked in place, the pairs (n0, n4) and, after a shift by 8, (n2, n6) read as the
// fp16 subnormals q 2^-24, the pairs (n1, n5) and (n3, n7) as q 2^-20.  So a code costs 5
// integer instructions per 8 and no conversion, and every product q x is exact.  s and m are
// applied per group in fp32, on the fp32 sums.
//
// The activations are brought to fp16 per token and group of 64 by a power of two that takes
// the largest of the group to [2^15, 2^16): exact for every bf16 value down to 2^-28 of the
// group's largest, and off by at most 2^-36 of the largest below that.  8-bit activations are
// exact.  Against 64 bits the fp32 logits of 2048 channels are off by 1.1e-7 of their size, as fp32
// sums of the products in another order are.
#pragma once
#include <cooperative_groups.h>
#include "e0_device.cuh"

namespace e0 {

// ---------------------------------------------------------------------------------------
// Shared-memory and copy instructions
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32u(uint32_t a) { return __float_as_uint(lds32(a)); }
__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// the first `bytes` (0..N) from src, zeros behind
template <int N>
__device__ __forceinline__ void cp_async_part(uint32_t dst, const void *src, int bytes) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Barrier of a team of wk warps (a power of two below 16): ids 1, 2 for teams of 8, 3..6 of 4, 7..14 of 2, so that
// teams of different sizes may be under way at once.
__device__ __forceinline__ void bar_team(int wk, int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(16 / wk - 1 + team), "r"(wk * 32) : "memory");
}

// The warp's number, as a value that the compiler knows to be the same in every lane: what follows from
// it (tiles, addresses of rows, loop counts) then stays on the uniform units.
__device__ __forceinline__ int warp_id() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// chunk c (of 16 bytes) of row r of 128 bytes lies at chunk c ^ row_swz(r): the lanes of a load, whether 16 or 8
// bytes each, fall into distinct banks
__device__ __forceinline__ int row_swz(int r) { return ((r & 1) << 2) ^ (r & 2); }

__device__ __forceinline__ float dot8(uint4 w, float4 x, float4 y, float s) {
  s = fmaf(__uint_as_float(w.x << 16), x.x, fmaf(__uint_as_float(w.x & 0xFFFF0000u), x.y, s));
  s = fmaf(__uint_as_float(w.y << 16), x.z, fmaf(__uint_as_float(w.y & 0xFFFF0000u), x.w, s));
  s = fmaf(__uint_as_float(w.z << 16), y.x, fmaf(__uint_as_float(w.z & 0xFFFF0000u), y.y, s));
  return fmaf(__uint_as_float(w.w << 16), y.z, fmaf(__uint_as_float(w.w & 0xFFFF0000u), y.w, s));
}

__device__ __forceinline__ void mma_bf16_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bf16 rows times 8 bf16 columns, 32 channels: a, b the lane's rows l / 4 and l / 4 + 8 at
// channel 8 (l & 3), x its column there.
__device__ __forceinline__ void bf16_mul(uint4 a, uint4 b, uint4 x, float (&acc)[4]) {
  mma_bf16_acc(acc, a.x, b.x, a.y, b.y, x.x, x.y);
  mma_bf16_acc(acc, a.z, b.z, a.w, b.w, x.z, x.w);
}

// ---------------------------------------------------------------------------------------
// Activations as matrix operands
// ---------------------------------------------------------------------------------------
// One token's group of 64 channels takes 128 bytes: word w (0, 1) at 64 w, then lane t (0..3)
// at 16 t, then the 8 channels 16 t + 8 w + {0, 4, 1, 5, 2, 6, 3, 7}, the odd ones divided by
// 16 (their codes sit 4 bits higher).  Lane t of a matrix instruction reads its operands of a
// word in one 16-byte access.  `sv` holds, for each group and pair of tokens, {factor of the
// first, of the second, sum of the first, of the second}.  factor and sum carry 2^-12, by which
// the end result is divided once: a group of bf16's largest numbers times codes of 15 comes to
// 2^138, with it to less than fp32's largest.
enum { ACT_BF16 = 0, ACT_INT8 = 1, ACT_E4M3 = 2 };
constexpr float kActUnit = 4096.0f;
constexpr int kActPad = 64;               // per token, so that the tokens of a load fall into distinct banks

__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float sum8(const float *v) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// Where a token's group goes: its 128 bytes and its place in `sv`.
struct ActDst {
  uint8_t *op;
  float *sv;
  int pitch, pairs;
  __device__ __forceinline__ void put(int tok, int grp, int i, uint4 w, float factor, float sum) const {
    *reinterpret_cast<uint4 *>(op + (size_t)tok * pitch + grp * 128 + (i & 1) * 64 + (i >> 1) * 16) = w;
    if (i == 0) {
      float *p = sv + ((size_t)grp * pairs + (tok >> 1)) * 4 + (tok & 1);
      p[0] = factor;
      p[2] = sum;
    }
  }
};

// The values of 8 int8 or e4m3 codes.
__device__ __forceinline__ void q8_values(uint2 w, bool e4m3, float (&v)[8]) {
  const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const uint32_t two = (ws[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
    if (e4m3) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
      asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[2 * j]), "=f"(v[2 * j + 1]) : "r"(h2));
    } else {
      v[2 * j] = (float)(int8_t)(two & 0xFFu);
      v[2 * j + 1] = (float)(int8_t)(two >> 8);
    }
  }
}

// Eight lanes (i = 0..7) bring one token's group of 64 channels, 8 each (16 bytes of bf16, or 8 of
// codes with their scale), into place.  All 32 lanes of the warp call these together.
__device__ __forceinline__ void act_group_bf16(uint4 w, int i, int tok, int grp, const ActDst &D) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  float v[8], m = 0.f;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    v[2 * j] = __uint_as_float(ws[j] << 16);
    v[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
    m = fmaxf(m, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
  // largest in [2^(eb-127), 2^(eb-126)) -> [2^15, 2^16); an infinity or a NaN stays one in its place
  // and in the sum, so the token's outputs are not finite
  const uint32_t eb = max(__float_as_uint(m) >> 23, 15u);
  const float up = __uint_as_float((269u - eb) << 23), up16 = up * 0.0625f, factor = __uint_as_float((eb - 3) << 23);
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] *= j & 1 ? up16 : up;
  // the sum, of the numbers in range (exact, but for what is 2^-24 of the largest and less), back by
  // 2^(eb-142) / kActUnit in two factors, as one would be below fp32's normal numbers
  const float s8 = fmaf(16.0f, (v[1] + v[3]) + (v[5] + v[7]), (v[0] + v[2]) + (v[4] + v[6]));
  const float s = group_sum(s8, 8) * 0x1p-24f * factor;
  static_assert(kActUnit == 4096.0f, "factor is 2^(eb - 142) 2^24 / kActUnit, the factor of the sum 2^(eb - 142) / kActUnit");
  D.put(tok, grp, i, make_uint4(half2_of(v[0], v[4]), half2_of(v[1], v[5]), half2_of(v[2], v[6]), half2_of(v[3], v[7])), factor, s);
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Codes times 32 (odd channels times 2): exact in fp16; the factor is scale 2^24 / 2^5 / 2^12.
__device__ __forceinline__ void act_group_int8(uint2 w, float scale, int i, int tok, int grp, const ActDst &D) {
  constexpr uint32_t X32 = 0x50005000u, X2 = 0x40004000u;             // 32, 2
  constexpr uint32_t O32 = 0xF880F880u, O2 = 0xE880E880u;             // -1152 * 32, -1152 * 2
  // a byte b + 128 under 0x64 is the fp16 number 1024 + 128 + b
  const uint32_t x = w.x ^ 0x80808080u, y = w.y ^ 0x80808080u;
  const uint32_t u = __byte_perm(x, y, 0x5140), v = __byte_perm(x, y, 0x7362);   // channels 0 4 1 5, 2 6 3 7
  const uint4 p = make_uint4(hfma2(__byte_perm(u, 0x64646464u, 0x4140), X32, O32), hfma2(__byte_perm(u, 0x64646464u, 0x4342), X2, O2),
                             hfma2(__byte_perm(v, 0x64646464u, 0x4140), X32, O32), hfma2(__byte_perm(v, 0x64646464u, 0x4342), X2, O2));
  int n = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, 0));
  n += __shfl_xor_sync(0xffffffffu, n, 1);
  n += __shfl_xor_sync(0xffffffffu, n, 2);
  n += __shfl_xor_sync(0xffffffffu, n, 4);
  D.put(tok, grp, i, p, scale * (0x1p19f / kActUnit), (float)n * (scale * (1.0f / kActUnit)));
}

__device__ __forceinline__ void act_group_e4m3(uint2 w, float scale, int i, int tok, int grp, const ActDst &D) {
  constexpr uint32_t X32 = 0x50005000u, X2 = 0x40004000u;
  uint32_t h[4];
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const uint32_t two = ((j < 2 ? w.x : w.y) >> (16 * (j & 1))) & 0xFFFFu;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[j]) : "h"((uint16_t)two));
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[2 * j]), "=f"(v[2 * j + 1]) : "r"(h[j]));
  }
  const uint32_t none = 0x80008000u;                                   // -0: x y + -0 = x y
  const uint4 p = make_uint4(hfma2(__byte_perm(h[0], h[2], 0x5410), X32, none), hfma2(__byte_perm(h[0], h[2], 0x7632), X2, none),
                             hfma2(__byte_perm(h[1], h[3], 0x5410), X32, none), hfma2(__byte_perm(h[1], h[3], 0x7632), X2, none));
  const float s = group_sum(sum8(v), 8);
  D.put(tok, grp, i, p, scale * (0x1p19f / kActUnit), s * (scale * (1.0f / kActUnit)));
}

// ---------------------------------------------------------------------------------------
// e0_int4_linear
// ---------------------------------------------------------------------------------------
// A block (one an SM, 16 warps) holds the activations of its tokens in shared memory and takes a
// contiguous share of the rows in tiles of 16; each warp (or a team of wk warps that splits K, where
// there are few tiles) streams its tiles through a ring of its own by cp.async, a stage of 256
// channels.  Where the activations are many (tokens times K), so that every block would spend more on
// bringing them to fp16 than on its weights, or they do not fit, the blocks of a cluster split K, and
// each adds up a part of the rows over the cluster's shared memory.
//
// Measured (a captured launch among others): 2048 x 2048 with LoRA at one token 6.3 us, 5120 x 2048 at
// 8 int8 tokens 6.1, 65521 x 2048 at one token 18.5 (3.9 TB/s), 8192 x 4096 at 32 e4m3 tokens 20.4.
// The small ones are the latency of a launch, the activations (3.3 us before the first tile) and one
// tile; 65521 rows by the weights and the wait for the first activations; 32 tokens by latency (a tile
// of four stages a warp, one stage ahead: no unit above half its rate, issue slots 47 %, shared-memory
// wavefronts 40 %, tensor pipe 22 %, on 132 of the SMs).  Ring depths 3 and 2: pair 18.3 us at
// one token and 65521 rows, with a depth of 2 19.9 (4: no change); wide needs the room for activations.
//
// Two forms.  Pair (up to 4 tokens, N = 1): the 8 columns of a matrix instruction are 4 tokens
// restricted to one group of 64 and the same 4 restricted to the next (zeros elsewhere), so a lane
// takes 16 consecutive bytes of a row and one fold serves both groups.  Wide (N tiles of 8 tokens): 8
// bytes of a row a lane, a fold per group.  The accumulators of a lane are rows l / 4 and l / 4 + 8,
// tokens 2 (l & 3), + 1 of a tile (pair: tokens 2 (l & 1), + 1, after adding lanes l and l + 2).
// (65521 x 2048: at 4 tokens pair 19.2 us, wide 20.6; at 8 two pair tiles 28.9, wide 21.9.)
struct LinearArgs {
  const uint8_t *codes;          // [N, K / 2]
  const uint8_t *scale, *min;    // [N, K / g] bf16
  int N, K;
  const uint16_t *A, *B;         // LoRA [r, K], [N, r], or nullptr
  int r, b16;                    // b16: rows of B begin at 16 bytes and r is a multiple of 8
  float c;
  const void *x;                 // [T, K]
  int x_type;
  long long x_stride;            // elements
  const float *x_scale;          // [T, K / x_group], or nullptr
  int x_shift, x_groups;         // scale k >> x_shift of x_groups belongs to channel k
  int T;
  void *y;                       // [T, N]
  int y_f32;
  long long y_stride;
  int S, kc;                     // blocks of a cluster, channels a block (a multiple of 256 and 128 cs where S > 1)
  int pass;                      // rows between two exchanges of a cluster (a multiple of 16)
  int cs;                        // 128-channel steps to a slot of scales: 8, 4, 2; 0: 2, fetched one by one
  int tok;                       // tokens of a block
};

constexpr int kLinThreads = 512, kLinWarps = kLinThreads / 32;
constexpr int kLinStage = 16 * 128, kLinSlot = 16 * 32;
constexpr int lin_depth(bool wide) { return wide ? 2 : 3; }
constexpr int lin_ring(bool wide) { return lin_depth(wide) * (kLinStage + kLinSlot); }
__host__ __device__ inline int lin_blocks(int kc) { return (kc + 255) / 256; }
// shared memory: zeros | t | partial sums | rings | activations of nt tokens | sums of a pass (S > 1)
__host__ __device__ inline size_t lin_fixed(bool wide, int N) {
  return 128 + 32 * (size_t)(wide ? 8 : 4) * N * 4 + (size_t)kLinWarps * 16 * (wide ? 8 : 4) * N * 4 + (size_t)kLinWarps * lin_ring(wide);
}
__host__ __device__ inline size_t lin_acts(int nt, int kc) {
  return (size_t)nt * (lin_blocks(kc) * 512 + kActPad) + (size_t)lin_blocks(kc) * 4 * ((nt + 1) / 2) * 16;
}

__device__ __forceinline__ void mma_f16_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same without a sum to add to
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// One fold: the sums p of a group (pair: of a lane's group of two) with its scales and mins, the
// low (sel 0x1044) or high (0x3244) halves of the words.  sv: {factors, sums} of a lane's two tokens.
template <int N>
__device__ __forceinline__ void lin_fold(const float (&p)[N][4], uint32_t wsa, uint32_t wma, uint32_t wsb, uint32_t wmb,
                                         uint32_t sel, const uint32_t (&sv)[N], float (&acc)[N][4]) {
  auto pick = [&](uint32_t w) { return __uint_as_float(__byte_perm(w, 0u, sel)); };
  const float sa = pick(wsa), sb = pick(wsb), ma = pick(wma), mb = pick(wmb);
#pragma unroll
  for (int q = 0; q < N; q++) {
    const uint4 f = lds128(sv[q]);
    const float f0 = __uint_as_float(f.x), f1 = __uint_as_float(f.y), v0 = __uint_as_float(f.z), v1 = __uint_as_float(f.w);
    acc[q][0] = fmaf(sa, p[q][0] * f0, fmaf(ma, v0, acc[q][0]));
    acc[q][1] = fmaf(sa, p[q][1] * f1, fmaf(ma, v1, acc[q][1]));
    acc[q][2] = fmaf(sb, p[q][2] * f0, fmaf(mb, v0, acc[q][2]));
    acc[q][3] = fmaf(sb, p[q][3] * f1, fmaf(mb, v1, acc[q][3]));
  }
}

// A lane's columns: operands x, and {factors, sums} sv, advanced by 128 channels at a time.
template <int N>
struct LinCol {
  uint32_t x[N], sv[N], step, svs;
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int q = 0; q < N; q++) {
      x[q] += step;
      sv[q] += 2 * svs;
    }
  }
};

// 128 channels: the lane's codes at shared address w0 (pair: 16 bytes; wide: 8 bytes, those of the
// second group at w1), those of 8 rows further 1024 bytes on; words of scales and mins.  hi: the
// scales are the high halves (one scale for both groups); otherwise a half each.
template <bool WIDE, int N, bool G128>
__device__ __forceinline__ void lin_mul128(uint32_t w0, uint32_t w1, uint32_t wsa, uint32_t wma, uint32_t wsb, uint32_t wmb,
                                           bool hi, const LinCol<N> &X, float (&acc)[N][4]) {
  constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
  const int t = threadIdx.x & 3;
  if (WIDE) {
#pragma unroll
    for (int g = 0; g < 2; g++) {
      const uint2 wa = lds64(g ? w1 : w0), wb = lds64((g ? w1 : w0) + 1024);
      float p[N][4];
#pragma unroll
      for (int w = 0; w < 2; w++) {
        const uint32_t xa = w ? wa.y : wa.x, xb = w ? wb.y : wb.x, ya = xa >> 8, yb = xb >> 8;
#pragma unroll
        for (int q = 0; q < N; q++) {
          const uint4 x = lds128(X.x[q] + g * 128 + w * 64);
          if (w == 0) mma_f16_first(p[q], xa & LO, xb & LO, xa & HI, xb & HI, x.x, x.y);
          else mma_f16_acc(p[q], xa & LO, xb & LO, xa & HI, xb & HI, x.x, x.y);
          mma_f16_acc(p[q], ya & LO, yb & LO, ya & HI, yb & HI, x.z, x.w);
        }
      }
      uint32_t sv[N];
#pragma unroll
      for (int q = 0; q < N; q++) sv[q] = X.sv[q] + g * X.svs;
      lin_fold<N>(p, wsa, wma, wsb, wmb, (G128 ? hi : g) ? 0x3244u : 0x1044u, sv, acc);
    }
  } else {
    const uint4 wa = lds128(w0), wb = lds128(w0 + 1024);
    // (two chains of dependent instructions, joined at the fold)
    static_assert(WIDE || N == 1, "one tile of tokens");
    float p[N][4], p2[4];
#pragma unroll
    for (int w = 0; w < 4; w++) {
      const uint32_t xa = w == 0 ? wa.x : w == 1 ? wa.y : w == 2 ? wa.z : wa.w;
      const uint32_t xb = w == 0 ? wb.x : w == 1 ? wb.y : w == 2 ? wb.z : wb.w, ya = xa >> 8, yb = xb >> 8;
#pragma unroll
      for (int q = 0; q < N; q++) {
        // chunk 4 (t & 1) + w of the group: word w & 1, lane 2 (t & 1) + w / 2 of it
        const uint4 x = lds128(X.x[q] + (w & 1) * 64 + (w >> 1) * 16);
        if (w == 0) mma_f16_first(p[q], xa & LO, xb & LO, xa & HI, xb & HI, x.x, x.y);
        else mma_f16_acc(p[q], xa & LO, xb & LO, xa & HI, xb & HI, x.x, x.y);
        if (w == 0) mma_f16_first(p2, ya & LO, yb & LO, ya & HI, yb & HI, x.z, x.w);
        else mma_f16_acc(p2, ya & LO, yb & LO, ya & HI, yb & HI, x.z, x.w);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) p[0][i] += p2[i];
    lin_fold<N>(p, wsa, wma, wsb, wmb, (G128 ? hi : t >> 1) ? 0x3244u : 0x1044u, X.sv, acc);
  }
}

// y[tok][row] = v
__device__ __forceinline__ void lin_store(const LinearArgs &L, int tok, int row, float v) {
  const long long at = (long long)tok * L.y_stride + row;
  if (L.y_f32)
    ((float *)L.y)[at] = v;
  else
    ((uint16_t *)L.y)[at] = f2bf(v);
}

// c B t of one row and token (t: 32 floats in shared memory)
__device__ __forceinline__ float lin_lora(const LinearArgs &L, int row, const float *t) {
  const uint16_t *b = L.B + (long long)row * L.r;
  float s = 0.f;
  if (L.b16) {
#pragma unroll 2
    for (int j = 0; j < L.r; j += 8)
      s = dot8(__ldg(reinterpret_cast<const uint4 *>(b + j)), *reinterpret_cast<const float4 *>(t + j),
               *reinterpret_cast<const float4 *>(t + j + 4), s);
  } else {
#pragma unroll 2
    for (int j = 0; j < L.r; j++) s = fmaf(bf(b[j]), t[j], s);
  }
  return L.c * s;
}

template <bool WIDE, int N, bool G128>
__global__ void __launch_bounds__(kLinThreads, 1) k_int4_linear(const __grid_constant__ LinearArgs L) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int TOK = N * (WIDE ? 8 : 4), DEPTH = lin_depth(WIDE);
  const int tid = threadIdx.x, lane = tid & 31, warp = warp_id(), r = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % L.S, part = blockIdx.x / L.S, parts = gridDim.x / L.S;
  const int t0 = blockIdx.y * L.tok, nt = min(L.tok, L.T - t0);
  // (the last blocks of a cluster may have fewer channels, or none)
  const int k0 = min(rank * L.kc, L.K), kc = min(L.kc, L.K - k0), NB = lin_blocks(kc), NB1 = max(NB, 1),
            NBmost = lin_blocks(L.kc);
  const int row_lo = (int)((long long)L.N * part / parts), row_hi = (int)((long long)L.N * (part + 1) / parts);
  // shared memory
  float *lt = reinterpret_cast<float *>(smem + 128);                 // [TOK][32]
  float *red = lt + TOK * 32;                                        // [16 warps][TOK][16 rows]
  const uint32_t ring = smem_at(red + kLinWarps * 16 * TOK) + warp * lin_ring(WIDE);
  uint8_t *ops = reinterpret_cast<uint8_t *>(red + kLinWarps * 16 * TOK) + kLinWarps * lin_ring(WIDE);
  const int pitch = NB * 512 + kActPad, pairs = (nt + 1) / 2;
  const ActDst D{ops, reinterpret_cast<float *>(ops + (size_t)nt * pitch), pitch, pairs};
  float *sums = reinterpret_cast<float *>(ops + lin_acts(min(L.tok, L.T), L.kc));   // S > 1: [pass / 16][nt][16 rows]
  const uint32_t zero = smem_at(smem);
  if (tid < 32) reinterpret_cast<uint32_t *>(smem)[tid] = 0;

  // ---- the ring: slots of scales, then the stages
  const uint32_t slots = ring, slots_end = slots + DEPTH * kLinSlot, end = slots_end + DEPTH * kLinStage;
  const int cr = lane >> 3, cc = lane & 7, sr = lane >> 1, cs = L.cs ? L.cs : 2;
  const uint32_t cdst = cr * 128 + ((cc ^ row_swz(cr)) << 4), sdst = sr * 32 + (lane & 1) * 16;
  const int Gn = L.K / (G128 ? 128 : 64);                            // scales of a row
  int lj = 0, jobs = 0, lb = 0, b0 = 0, b1 = 0, step = 1, tile0 = 0, tiles = 0, base = 0, top = 0;
  const uint8_t *cp = nullptr, *sp = nullptr;
  int o[4] = {};
  uint32_t lst = slots_end, lsl = slots;
  // tile q of the pass: rows base + 16 q .., at most to top
  auto issue = [&]() {
    if (lj < jobs) {
      if (lb == b0) {
        const int row = base + (tile0 + lj * step) * 16, nr = min(16, top - row);
        cp = L.codes + (long long)row * (L.K / 2) + k0 / 2 + b0 * 128 + cc * 16;
#pragma unroll
        for (int i = 0; i < 4; i++) o[i] = min(cr + 4 * i, nr - 1) * (L.K / 2);
        sp = (lane & 1 ? L.min : L.scale) + ((long long)(row + min(sr, nr - 1)) * Gn + (k0 + (2 * b0 & -cs) * 128) / (G128 ? 128 : 64)) * 2;
      }
      if (lb == b0 || (2 * lb & (cs - 1)) == 0) {
        const int ch = (2 * lb & -cs) * 128, bytes = min(cs * 128, kc - ch) / (G128 ? 128 : 64) * 2;
        if (L.cs == 0) {
          // rows of an odd number of groups, or no aligned base: one by one
          const uint16_t *p = reinterpret_cast<const uint16_t *>(sp);
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 4; i++)
            if (2 * i < bytes) w[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(lsl + sdst), "r"(w[0]), "r"(w[1]) : "memory");
        } else if (cs * (G128 ? 2 : 4) == 16) {
          cp_async_part<16>(lsl + sdst, sp, bytes);
        } else if (cs * (G128 ? 2 : 4) == 8) {
          cp_async_part<8>(lsl + sdst, sp, bytes);
        } else {
          cp_async_part<4>(lsl + sdst, sp, bytes);
        }
        sp += cs * (G128 ? 2 : 4);
        lsl = lsl + kLinSlot == slots_end ? slots : lsl + kLinSlot;
      }
      if ((lb + 1) * 256 <= kc) {
#pragma unroll
        for (int i = 0; i < 4; i++) cp_async16(lst + cdst + i * 512, cp + o[i]);
      } else {
        const int bytes = lb * 256 + cc * 32 < kc ? 16 : 0;
#pragma unroll
        for (int i = 0; i < 4; i++) cp_async_part<16>(lst + cdst + i * 512, bytes ? cp + o[i] : L.codes, bytes);
      }
      cp += 128;
      lst = lst + kLinStage == end ? slots_end : lst + kLinStage;
      if (++lb == b1) {
        lb = b0;
        lj++;
      }
    }
    cp_async_commit();
  };
  int wk = 1, team = 0, sub = 0;
  // the tiles of rows [lo, hi): warps to a tile so that the last round is full, no more than there
  // are blocks of K (the same in every block of a cluster); a warp without a block adds nothing
  auto begin = [&](int lo, int hi) {
    base = lo;
    top = hi;
    tiles = (hi - lo + 15) / 16;
    int best = 1 << 30, lg = 0;
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int cost = (((tiles << g) + 15) >> 4 << (4 - g)) + 2 * g;
      if ((1 << g) <= NBmost && cost < best) {
        best = cost;
        lg = g;
      }
    }
    wk = 1 << lg;
    team = warp >> lg;
    sub = warp & (wk - 1);
    step = kLinWarps >> lg;
    tile0 = team;
    jobs = (tiles - team + step - 1) >> (4 - lg);
    b0 = lb = NB * sub >> lg;
    b1 = NB * (sub + 1) >> lg;
    lj = b0 < b1 ? 0 : jobs;
    __syncwarp();
    issue();
  };
  // ---- the tiles
  const int swz = row_swz(r);
  const uint32_t w_at = r * 128 + (((WIDE ? t >> 1 : t) ^ swz) << 4) + (WIDE ? (t & 1) * 8 : 0);
  const uint32_t w_at1 = r * 128 + (((2 + (t >> 1)) ^ swz) << 4) + (t & 1) * 8;
  const bool mine = WIDE || (t >> 1) == (r >> 2);
  LinCol<N> X0;
  X0.step = mine ? 256 : 0;
  X0.svs = pairs * 16;
#pragma unroll
  for (int q = 0; q < N; q++) {
    const int tok = min(WIDE ? 8 * q + r : 4 * q + (r & 3), nt - 1), pair = min(WIDE ? 4 * q + t : 2 * q + (t & 1), pairs - 1);
    X0.x[q] = mine ? smem_at(D.op) + tok * pitch + (WIDE ? t * 16 : (t >> 1) * 128 + (t & 1) * 32) : zero;
    X0.sv[q] = smem_at(D.sv) + pair * 16 + (WIDE ? 0 : (t >> 1) * X0.svs);
  }
  uint32_t st = slots_end, sl = slots_end - kLinSlot;
  const int pass = L.S > 1 ? L.pass : row_hi - row_lo;
#pragma unroll 1
  for (int lo = row_lo; lo < row_hi; lo += pass) {
    const int hi = min(lo + pass, row_hi);
    begin(lo, hi);
    if (lo == row_lo) {
      // ---- the activations of this block's channels, zeros behind the last: a warp takes 256 of a
      // token, 8 lanes to a group of 64; four of them are under way at once, the first four between the
      // weights' first two steps (all of the weights' steps before them: 19.1 us for 65521 x 2048 at one
      // token, here 18.4; all behind them: 17.4, but 7.8 for 5120 x 2048 at 8 tokens instead of 7.2)
      {
        const int i = lane & 7, wide = L.x_type == ACT_BF16 ? 1 : 0;
        // the 16 units that the warps take at once, in tokens and blocks: quotients by a reciprocal, half a
        // unit from a whole number
        const float per = __fdividef(1.0f, (float)NB1);
        const int dct = (int)((kLinWarps + 0.5f) * per), dcb = kLinWarps - dct * NB1, ct0 = (int)((warp + 0.5f) * per);
        int ct = NB > 0 ? ct0 : nt, cb = warp - ct0 * NB1;
        const char *px = (const char *)L.x + (((t0 + ct) * L.x_stride + k0 + cb * 256 + lane * 8) << wide);
        const long long dpx = (dct * L.x_stride + dcb * 256) << wide, wrap = (L.x_stride - NB * 256) << wide;
        const float *ps = L.x_scale + (t0 + ct) * (long long)L.x_groups;
        int u = 2;
#pragma unroll 1
        do {
          uint4 w[4];
          float s[4];
          int tk[4], gr[4];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const int k = cb * 256 + lane * 8;
            w[j] = make_uint4(0, 0, 0, 0);
            s[j] = 1.f;
            tk[j] = ct;
            gr[j] = cb * 4 + (lane >> 3);
            if (ct < nt && k < kc) {
              if (wide) {
                w[j] = __ldg(reinterpret_cast<const uint4 *>(px));
              } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(px));
                w[j].x = v.x;
                w[j].y = v.y;
                s[j] = __ldg(ps + ((k0 + k) >> L.x_shift));
              }
            }
            ct += dct;
            cb += dcb;
            px += dpx;
            ps += dct * L.x_groups;
            if (cb >= NB) {
              cb -= NB;
              ct++;
              px += wrap;
              ps += L.x_groups;
            }
          }
          if (u < DEPTH) issue();
          u = DEPTH;
#pragma unroll
          for (int j = 0; j < 4; j++) {
            if (tk[j] >= nt) break;                     // (the same for the whole warp)
            if (L.x_type == ACT_BF16) act_group_bf16(w[j], i, tk[j], gr[j], D);
            else if (L.x_type == ACT_INT8) act_group_int8(make_uint2(w[j].x, w[j].y), s[j], i, tk[j], gr[j], D);
            else act_group_e4m3(make_uint2(w[j].x, w[j].y), s[j], i, tk[j], gr[j], D);
          }
        } while (ct < nt);
      }
      // ---- t = A x of this block's channels, K split over the warps: 16 ranks by 8 tokens at a time
      if (L.A) {
        const int G = kc / 64;
#pragma unroll 1
        for (int u = 0; u < (L.r + 15) / 16 * ((nt + 7) / 8); u++) {
          const int q = u / ((nt + 7) / 8) * 16, tt = u % ((nt + 7) / 8) * 8;
          const uint16_t *ra = L.A + (long long)min(q + r, L.r - 1) * L.K + k0 + t * 8;
          const uint16_t *rb = L.A + (long long)min(q + r + 8, L.r - 1) * L.K + k0 + t * 8;
          const int tok = min(tt + r, nt - 1);
          const long long xa = (long long)(t0 + tok) * L.x_stride + k0 + t * 8;
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
          for (int g = G * warp / kLinWarps; g < G * (warp + 1) / kLinWarps; g++) {
            float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const int k = g * 64 + h * 32;
              uint4 x;
              if (L.x_type == ACT_BF16) {
                x = __ldg(reinterpret_cast<const uint4 *>((const uint16_t *)L.x + xa + k));
              } else {
                float v[8];
                q8_values(__ldg(reinterpret_cast<const uint2 *>((const uint8_t *)L.x + xa + k)), L.x_type == ACT_E4M3, v);
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; j++) w[j] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xFFFF0000u);
                x = make_uint4(w[0], w[1], w[2], w[3]);            // codes are exact in bf16
              }
              bf16_mul(__ldg(reinterpret_cast<const uint4 *>(ra + k)), __ldg(reinterpret_cast<const uint4 *>(rb + k)), x, p);
            }
            // columns 2 t, 2 t + 1 are tokens of their own scales
            float s0 = 1.f, s1 = 1.f;
            if (L.x_type != ACT_BF16) {
              const int gs = (k0 + g * 64) >> L.x_shift, ng = L.x_groups;
              s0 = __ldg(L.x_scale + (long long)(t0 + min(tt + 2 * t, nt - 1)) * ng + gs);
              s1 = __ldg(L.x_scale + (long long)(t0 + min(tt + 2 * t + 1, nt - 1)) * ng + gs);
            }
            acc[0] = fmaf(s0, p[0], acc[0]);
            acc[1] = fmaf(s1, p[1], acc[1]);
            acc[2] = fmaf(s0, p[2], acc[2]);
            acc[3] = fmaf(s1, p[3], acc[3]);
          }
          float *p = red + warp * 128 + r * 8 + 2 * t;               // TOK >= 4: 16 warps of 64 floats or more
          if (TOK >= 8) {
            p[0] = acc[0];
            p[1] = acc[1];
            p[64] = acc[2];
            p[65] = acc[3];
          } else if (t < 2) {                                        // 4 tokens: columns 0..3
            p = red + warp * 64 + r * 4 + 2 * t;
            p[0] = acc[0];
            p[1] = acc[1];
            p[32] = acc[2];
            p[33] = acc[3];
          }
          __syncthreads();
          constexpr int W = TOK >= 8 ? 8 : 4;
          if (tid < 16 * W) {
            const int row = q + tid / W, tk = tt + tid % W;
            if (row < L.r && tk < nt) {
              float s = 0.f;
#pragma unroll
              for (int w = 0; w < kLinWarps; w++) s += red[w * 16 * W + tid];
              lt[tk * 32 + row] = s;
            }
          }
          __syncthreads();
        }
      }
      __syncthreads();
    } else if (DEPTH > 2) {
      issue();
    }
#pragma unroll 1
    for (int j = 0; j < jobs; j++) {
      const int row = lo + (tile0 + j * step) * 16;
      float acc[N][4];
#pragma unroll
      for (int q = 0; q < N; q++) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
      LinCol<N> X = X0;
#pragma unroll
      for (int q = 0; q < N; q++) {
        X.x[q] += 2 * b0 * X.step;
        X.sv[q] += 4 * b0 * X.svs;
      }
#pragma unroll 1
      for (int b = b0; b < b1; b++) {
        cp_async_wait_but<DEPTH - 2>();
        __syncwarp();                     // the block has arrived, and every lane has left the one before
        issue();
        const int at = 2 * b & (cs - 1);
        if (b == b0 || at == 0) sl = sl + kLinSlot == slots_end ? slots : sl + kLinSlot;
        const uint32_t sc = sl + r * 32 + at * (G128 ? 2 : 4);
        uint2 sa, ma, sb, mb;
        if (G128) {
          sa.x = sa.y = lds32u(sc);
          ma.x = ma.y = lds32u(sc + 16);
          sb.x = sb.y = lds32u(sc + 256);
          mb.x = mb.y = lds32u(sc + 272);
        } else {
          sa = lds64(sc);
          ma = lds64(sc + 16);
          sb = lds64(sc + 256);
          mb = lds64(sc + 272);
        }
        lin_mul128<WIDE, N, G128>(st + w_at, st + w_at1, sa.x, ma.x, sb.x, mb.x, false, X, acc);
        X.advance();
        // chunk c + 4 lies 64 bytes from chunk c, on the side that the permutation leaves
        lin_mul128<WIDE, N, G128>(st + (w_at ^ 64), st + (w_at1 ^ 64), sa.y, ma.y, sb.y, mb.y, true, X, acc);
        X.advance();
        st = st + kLinStage == end ? slots_end : st + kLinStage;
      }
      // pair: lanes l and l + 2 hold the same two tokens and take one each; wide: both tokens
      float *mine_at = red + warp * 16 * TOK;
#pragma unroll
      for (int q = 0; q < N; q++) {
        if (!WIDE)
#pragma unroll
          for (int i = 0; i < 4; i++) acc[q][i] += __shfl_xor_sync(0xffffffffu, acc[q][i], 2);
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); h++) {
          const int odd = WIDE ? h : t >> 1, tok = WIDE ? 8 * q + 2 * t + h : 4 * q + 2 * (t & 1) + odd;
          mine_at[tok * 16 + r] = odd ? acc[q][1] : acc[q][0];
          mine_at[tok * 16 + r + 8] = odd ? acc[q][3] : acc[q][2];
        }
      }
      if (wk > 1) bar_team(wk, team); else __syncwarp();
      float *p = red + team * wk * 16 * TOK;
#pragma unroll 1
      for (int u = sub * 32 + lane; u < 16 * nt; u += wk * 32) {
        const int tok = u >> 4, n = row + (u & 15);
        float v = p[u];
#pragma unroll 1
        for (int w = 1; w < wk; w++) v += p[w * 16 * TOK + u];
        v *= kActUnit;
        if (n >= hi) continue;
        if (L.A) v += lin_lora(L, n, lt + tok * 32);
        if (L.S > 1)
          sums[(tile0 + j * step) * 16 * nt + u] = v;       // joined below
        else
          lin_store(L, t0 + tok, n, v);
      }
      if (wk > 1) bar_team(wk, team); else __syncwarp();
    }
    if (L.S > 1) {
      cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
      cluster.sync();
#pragma unroll 1
      for (int u = rank * kLinThreads + tid; u < tiles * 16 * nt; u += L.S * kLinThreads) {
        const int q = u / (16 * nt), at = u - q * 16 * nt, n = lo + q * 16 + (at & 15);
        if (n >= hi) continue;
        float v = 0.f;
#pragma unroll 2
        for (int w = 0; w < L.S; w++) v += cluster.map_shared_rank(sums, w)[u];
        lin_store(L, t0 + (at >> 4), n, v);
      }
      cluster.sync();
    }
  }
}

}  // namespace e0
