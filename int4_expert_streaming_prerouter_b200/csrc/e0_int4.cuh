// Products of a few tokens with a matrix in the int4 affine group format (e0_int4_linear),
// and the pieces it shares with the few-token MoE layer.
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
// exact.
#pragma once
#include "e0_device.cuh"

namespace e0 {

// ---------------------------------------------------------------------------------------
// Activations as matrix operands
// ---------------------------------------------------------------------------------------
// One token's group of 64 channels takes 128 bytes: word w (0, 1) at 64 w, then lane t (0..3)
// at 16 t, then the 8 channels 16 t + 8 w + {0, 4, 1, 5, 2, 6, 3, 7}, the odd ones divided by
// 16 (their codes sit 4 bits higher).  Lane t of a matrix instruction reads its operands of a
// word in one 16-byte access.  `sv` holds, for each group and pair of tokens, {factor of the
// first, of the second, sum of the first, of the second}.  factor and sum carry 2^-9, which
// the end result is multiplied with once, so that no factor overflows.
constexpr float kActUnit = 512.0f;
constexpr int kActPad = 64;               // per token, so that 8 tokens fall into distinct banks

__host__ __device__ inline int act_pitch(int groups) { return groups * 128 + kActPad; }
__host__ __device__ inline int act_sv_bytes(int groups, int tokens) { return groups * ((tokens + 1) / 2) * 16; }

__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint4 act_pack(const float *v) {
  constexpr float o = 0.0625f;
  return make_uint4(half2_of(v[0], v[4]), half2_of(v[1] * o, v[5] * o), half2_of(v[2], v[6]),
                    half2_of(v[3] * o, v[7] * o));
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

// Eight lanes (i = 0..7) bring one token's group of 64 bf16 channels, 8 each, into place.
// All 32 lanes of the warp call it together.
__device__ __forceinline__ void act_group_bf16(uint4 w, int i, int tok, int grp, const ActDst &D, bool put) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  float v[8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    m = max(m, max(ws[j] & 0x7FFFu, (ws[j] >> 16) & 0x7FFFu));
    v[2 * j] = __uint_as_float(ws[j] << 16);
    v[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
  }
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
  // largest in [2^(eb-127), 2^(eb-126)) -> [2^15, 2^16); a group with a NaN or an infinity
  // keeps it (eb = 255 makes the factor infinite), so its outputs are not finite
  const uint32_t eb = max(m >> 7, 15u);
  const float up = __uint_as_float((269u - eb) << 23), factor = __uint_as_float(eb << 23);
  float s = sum8(v) * (1.0f / kActUnit);
  s = group_sum(s, 8);
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] *= up;
  if (put) D.put(tok, grp, i, act_pack(v), factor, s);
}

// The same for 8-bit channels (int8, or e4m3) with a scale: 8 bytes a lane.
__device__ __forceinline__ void act_group_q8(uint2 w, bool e4m3, float scale, int i, int tok, int grp,
                                             const ActDst &D, bool put) {
  float v[8];
  const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const uint32_t two = (ws[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
    if (e4m3) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
      float lo, hi;
      asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(lo), "=f"(hi) : "r"(h2));
      v[2 * j] = lo;
      v[2 * j + 1] = hi;
    } else {
      v[2 * j] = (float)(int8_t)(two & 0xFFu);
      v[2 * j + 1] = (float)(int8_t)(two >> 8);
    }
  }
  float s = group_sum(sum8(v), 8) * (scale * (1.0f / kActUnit));
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] *= 64.0f;            // q 2^6: the factor is scale 2^24 / 2^6 / 2^9
  if (put) D.put(tok, grp, i, act_pack(v), scale * 512.0f, s);
}

// ---------------------------------------------------------------------------------------
// 16 weight rows by 8 NT tokens
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void mma_f16_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One weight row as a lane sees it: its codes (already at the lane's 8 bytes of a group of 64),
// scales and mins.
struct Int4Row {
  const uint8_t *c;
  const uint16_t *s, *m;
};

__device__ __forceinline__ unsigned long long f2mul(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Sums over the tokens of a lane's two rows: accumulator columns 2 t, 2 t + 1 of each n-tile.
template <int NT>
struct Int4Acc {
  unsigned long long a[NT], b[NT];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; n++) a[n] = b[n] = 0ull;
  }
};

// Adds groups [g0, g1) (of 64 channels) of rows `ra` (row l / 4 of the tile) and `rb` (row
// l / 4 + 8).  gs: 0 when the scales are per 64, 1 when per 128.  col[n]: the lane's token
// (column l / 4 of n-tile n) at its 16 bytes (16 (l & 3)) of group 0; sv[n]: the pair of
// tokens 2 (l & 3), 2 (l & 3) + 1 of n-tile n in group 0, `svs` bytes from group to group.
template <int NT>
__device__ __forceinline__ void int4_rows(const Int4Row &ra, const Int4Row &rb, int g0, int g1, int gs,
                                          const uint8_t *const (&col)[NT], const uint8_t *const (&sv)[NT], int svs,
                                          Int4Acc<NT> &acc) {
  constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
#pragma unroll 4
  for (int g = g0; g < g1; g++) {
    const uint2 wa = __ldg(reinterpret_cast<const uint2 *>(ra.c + (size_t)g * 32));
    const uint2 wb = __ldg(reinterpret_cast<const uint2 *>(rb.c + (size_t)g * 32));
    const float sa = bf(__ldg(ra.s + (g >> gs))), ma = bf(__ldg(ra.m + (g >> gs)));
    const float sb = bf(__ldg(rb.s + (g >> gs))), mb = bf(__ldg(rb.m + (g >> gs)));
    float p[NT][4];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int j = 0; j < 4; j++) p[n][j] = 0.f;
    const uint32_t wa2[2] = {wa.x, wa.y}, wb2[2] = {wb.x, wb.y};
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const uint32_t xa = wa2[w], xb = wb2[w], ya = xa >> 8, yb = xb >> 8;
#pragma unroll
      for (int n = 0; n < NT; n++) {
        const uint4 x = *reinterpret_cast<const uint4 *>(col[n] + g * 128 + w * 64);
        mma_f16_acc(p[n], xa & LO, xb & LO, xa & HI, xb & HI, x.x, x.y);
        mma_f16_acc(p[n], ya & LO, yb & LO, ya & HI, yb & HI, x.z, x.w);
      }
    }
    const unsigned long long sa2 = pk2(sa, sa), ma2 = pk2(ma, ma), sb2 = pk2(sb, sb), mb2 = pk2(mb, mb);
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(sv[n] + (size_t)g * svs);
      acc.a[n] = f2fma(sa2, f2mul(pk2(p[n][0], p[n][1]), f.x), f2fma(ma2, f.y, acc.a[n]));
      acc.b[n] = f2fma(sb2, f2mul(pk2(p[n][2], p[n][3]), f.x), f2fma(mb2, f.y, acc.b[n]));
    }
  }
}

// ---------------------------------------------------------------------------------------
// 16 weight rows by up to 8 tokens: two groups to a matrix instruction
// ---------------------------------------------------------------------------------------
// With few tokens the 8 columns of a matrix instruction hold 4 tokens twice: columns 0..3 the
// tokens restricted to a group of 64, columns 4..7 restricted to the next one (zero elsewhere).
// A lane then takes 16 consecutive bytes of a row, its four lanes cover two groups, the sums of
// the two come out in different columns, and there is one fold for both.  The lane (row l / 4,
// t = l & 3) holds tokens 2 (t & 1), 2 (t & 1) + 1 of group t / 2 in its accumulators; lanes t
// and t + 2 are added at the end.
//
// A block is 256 channels of 16 rows: 4 loads of codes and 4 of scales and mins a lane.

struct PairBlk {
  uint4 a[2], b[2];
  uint2 sa, ma, sb, mb;
};

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Block b of rows whose codes start at the lane's 16 bytes of the row.  G128: scales per 128
// (two a block) instead of per 64 (four).
template <bool G128>
__device__ __forceinline__ void pair_load(PairBlk &B, const Int4Row &ra, const Int4Row &rb, int b) {
  B.a[0] = ldg_stream(ra.c + (size_t)b * 128);
  B.a[1] = ldg_stream(ra.c + (size_t)b * 128 + 64);
  B.b[0] = ldg_stream(rb.c + (size_t)b * 128);
  B.b[1] = ldg_stream(rb.c + (size_t)b * 128 + 64);
  if (G128) {
    B.sa.x = __ldg(reinterpret_cast<const uint32_t *>(ra.s + b * 2));
    B.ma.x = __ldg(reinterpret_cast<const uint32_t *>(ra.m + b * 2));
    B.sb.x = __ldg(reinterpret_cast<const uint32_t *>(rb.s + b * 2));
    B.mb.x = __ldg(reinterpret_cast<const uint32_t *>(rb.m + b * 2));
  } else {
    B.sa = __ldg(reinterpret_cast<const uint2 *>(ra.s + b * 4));
    B.ma = __ldg(reinterpret_cast<const uint2 *>(ra.m + b * 4));
    B.sb = __ldg(reinterpret_cast<const uint2 *>(rb.s + b * 4));
    B.mb = __ldg(reinterpret_cast<const uint2 *>(rb.m + b * 4));
  }
}

// The lane's view of the activations of NP times 4 tokens (n of them, at rows `at`.. of D;
// `at` even).  zero: 128 bytes of zeros in shared memory, 16-byte aligned.
template <int NP>
struct PairCol {
  const uint8_t *col[NP], *sv[NP];
  int step, svs;
  uint32_t sel;
  __device__ __forceinline__ PairCol(const ActDst &D, int at, int n, const uint8_t *zero) {
    const int lane = threadIdx.x & 31, t = lane & 3, c = lane >> 2;
    const bool mine = (t >> 1) == (c >> 2);
    step = mine ? 256 : 0;
    svs = D.pairs * 16;
    sel = t >> 1 ? 0x3244u : 0x1044u;
#pragma unroll
    for (int q = 0; q < NP; q++) {
      col[q] = mine ? D.op + (size_t)(at + min(4 * q + (c & 3), n - 1)) * D.pitch + (t >> 1) * 128 + (t & 1) * 32 : zero;
      sv[q] = reinterpret_cast<const uint8_t *>(D.sv) + (at / 2 + min(2 * q + (t & 1), (n - 1) / 2)) * 16 + (t >> 1) * svs;
    }
  }
};

template <int NP, bool G128>
__device__ __forceinline__ void pair_mul(const PairBlk &B, int b, const PairCol<NP> &X, Int4Acc<NP> &acc) {
  constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const uint32_t wa[4] = {B.a[j].x, B.a[j].y, B.a[j].z, B.a[j].w}, wb[4] = {B.b[j].x, B.b[j].y, B.b[j].z, B.b[j].w};
    float p[NP][4];
#pragma unroll
    for (int q = 0; q < NP; q++) p[q][0] = p[q][1] = p[q][2] = p[q][3] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; w++) {
      const uint32_t xa = wa[w], xb = wb[w], ya = xa >> 8, yb = xb >> 8;
#pragma unroll
      for (int q = 0; q < NP; q++) {
        const uint4 x = *reinterpret_cast<const uint4 *>(X.col[q] + (2 * b + j) * X.step + (w & 1) * 64 + (w >> 1) * 16);
        mma_f16_acc(p[q], xa & LO, xb & LO, xa & HI, xb & HI, x.x, x.y);
        mma_f16_acc(p[q], ya & LO, yb & LO, ya & HI, yb & HI, x.z, x.w);
      }
    }
    const uint32_t sel = G128 ? (j ? 0x3244u : 0x1044u) : X.sel;
    auto pick = [&](const uint2 &v) {
      const float f = __uint_as_float(__byte_perm(G128 || j == 0 ? v.x : v.y, 0u, sel));
      return pk2(f, f);
    };
    const unsigned long long sa = pick(B.sa), ma = pick(B.ma), sb = pick(B.sb), mb = pick(B.mb);
#pragma unroll
    for (int q = 0; q < NP; q++) {
      const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(X.sv[q] + (4 * b + 2 * j) * X.svs);
      acc.a[q] = f2fma(sa, f2mul(pk2(p[q][0], p[q][1]), f.x), f2fma(ma, f.y, acc.a[q]));
      acc.b[q] = f2fma(sb, f2mul(pk2(p[q][2], p[q][3]), f.x), f2fma(mb, f.y, acc.b[q]));
    }
  }
}

// Adds lanes t and t + 2: every lane then holds the sums of tokens 2 (t & 1), 2 (t & 1) + 1.
template <int NP>
__device__ __forceinline__ void pair_join(Int4Acc<NP> &acc) {
#pragma unroll
  for (int q = 0; q < NP; q++) {
    acc.a[q] = f2add(acc.a[q], __shfl_xor_sync(0xffffffffu, acc.a[q], 2));
    acc.b[q] = f2add(acc.b[q], __shfl_xor_sync(0xffffffffu, acc.b[q], 2));
  }
}

// A warp's jobs one after another, each blocks [b0, b1) of 16 rows, with the loads of the next
// blocks in flight, across the end of a job too.  rows(j, ra, rb) gives job j's rows,
// cols(j) its activations, done(j, acc) takes its sums.
template <int NP, bool G128, class Rows, class Cols, class Done>
__device__ __forceinline__ void pair_stream(int jobs, int b0, int b1, Rows rows, Cols cols, Done done) {
  if (jobs <= 0 || b0 >= b1) return;
  constexpr int D = NP == 1 ? 3 : 2;      // two tiles of tokens leave registers for one less
  PairBlk buf[D];
  Int4Row ra, rb;
  int lj = 0, lb = b0;                    // the next block to load
  auto load = [&](PairBlk &B) {
    if (lj >= jobs) return;
    if (lb == b0) rows(lj, ra, rb);
    pair_load<G128>(B, ra, rb, lb);
    if (++lb == b1) {
      lb = b0;
      lj++;
    }
  };
#pragma unroll
  for (int u = 0; u < D - 1; u++) load(buf[u]);
  Int4Acc<NP> acc;
  acc.clear();
  PairCol<NP> X = cols(0);
  for (int j = 0, b = b0;;) {
#pragma unroll
    for (int u = 0; u < D; u++) {
      load(buf[(u + D - 1) % D]);
      pair_mul<NP, G128>(buf[u], b, X, acc);
      if (++b == b1) {
        pair_join(acc);
        done(j, acc);
        if (++j == jobs) return;
        acc.clear();
        X = cols(j);
        b = b0;
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// e0_int4_linear
// ---------------------------------------------------------------------------------------
enum { ACT_BF16 = 0, ACT_INT8 = 1, ACT_E4M3 = 2 };

struct LinearArgs {
  const uint8_t *codes;       // [N, K / 2]
  const uint16_t *scale, *min;   // [N, K / g]
  int N, K, gs;               // gs: 0 for g = 64, 1 for g = 128
  const uint16_t *A, *B;      // LoRA [r, K], [N, r], or nullptr
  int r;
  float c;
  const void *x;              // [T, K]
  int x_type;
  long long x_stride;         // elements
  const float *x_scale;       // [T, K / x_group], or nullptr
  int x_group;                // channels to a scale
  int T;
  void *y;                    // [T, N]
  int y_f32;
  long long y_stride;
  int kc;                     // groups of 64 to a chunk of the activations
};

constexpr int kLinThreads = 256;
constexpr int kLinRows = 16;

template <int NT>
__global__ void __launch_bounds__(kLinThreads) k_int4_linear(LinearArgs L) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int TT = 8 * NT, NW = kLinThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.y * TT, nt = min(TT, L.T - t0);
  const int row0 = blockIdx.x * kLinRows;
  const int G = L.K / 64, pitch = act_pitch(L.kc);
  ActDst D{smem, reinterpret_cast<float *>(smem + TT * pitch), pitch, TT / 2};
  float *red = reinterpret_cast<float *>(smem);        // [NW][16][TT], after the last chunk
  __shared__ float lt[TT][32];
  // rows past the end read the last row and are not stored
  auto row_at = [&](int r) {
    const long long n = min(row0 + r, L.N - 1);
    return Int4Row{L.codes + n * (L.K / 2) + (lane & 3) * 8, L.scale + n * (G >> L.gs), L.min + n * (G >> L.gs)};
  };
  const Int4Row ra = row_at(lane >> 2), rb = row_at((lane >> 2) + 8);
  Int4Acc<NT> acc;
  acc.clear();
  const uint8_t *col[NT], *sv[NT];
#pragma unroll
  for (int n = 0; n < NT; n++) {
    col[n] = D.op + min(8 * n + (lane >> 2), nt - 1) * pitch + (lane & 3) * 16;
    sv[n] = reinterpret_cast<const uint8_t *>(D.sv) + (4 * n + (lane & 3)) * 16;
  }
  for (int c0 = 0; c0 < G; c0 += L.kc) {
    const int gc = min(L.kc, G - c0);
    __syncthreads();
    // activations of the chunk: 8 lanes to a token's group
    for (int u0 = 0; u0 < nt * gc; u0 += kLinThreads / 8) {
      const int u = u0 + tid / 8, i = tid & 7;
      const bool in = u < nt * gc;
      const int tok = in ? u / gc : 0, grp = in ? u % gc : 0;
      const long long k = (long long)(c0 + grp) * 64 + i * 8, base = (long long)(t0 + tok) * L.x_stride;
      if (L.x_type == ACT_BF16) {
        act_group_bf16(*reinterpret_cast<const uint4 *>((const uint16_t *)L.x + base + k), i, tok, grp, D, in);
      } else {
        const float s = L.x_scale[(long long)(t0 + tok) * (L.K / L.x_group) + k / L.x_group];
        act_group_q8(*reinterpret_cast<const uint2 *>((const uint8_t *)L.x + base + k), L.x_type == ACT_E4M3, s, i, tok,
                     grp, D, in);
      }
    }
    __syncthreads();
    const int per = (gc + NW - 1) / NW, g0 = min(warp * per, gc), g1 = min(g0 + per, gc);
    const Int4Row pa{ra.c + (size_t)c0 * 32, ra.s + (c0 >> L.gs), ra.m + (c0 >> L.gs)};
    const Int4Row pb{rb.c + (size_t)c0 * 32, rb.s + (c0 >> L.gs), rb.m + (c0 >> L.gs)};
    int4_rows<NT>(pa, pb, g0, g1, L.gs, col, sv, TT / 2 * 16, acc);
  }
  // LoRA: t = A x, one warp to a (token, rank) pair at a time
  if (L.A) {
    for (int u = warp; u < nt * L.r; u += NW) {
      const int tok = u / L.r, rr = u % L.r;
      const long long base = (long long)(t0 + tok) * L.x_stride;
      float s = 0.f;
      for (int k = lane; k < L.K; k += 32) {
        float xv;
        if (L.x_type == ACT_BF16) {
          xv = bf(((const uint16_t *)L.x)[base + k]);
        } else {
          const uint8_t b = ((const uint8_t *)L.x)[base + k];
          if (L.x_type == ACT_INT8) {
            xv = (float)(int8_t)b;
          } else {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)b));
            asm("{.reg .f16 a, b; mov.b32 {a, b}, %1; cvt.f32.f16 %0, a;}" : "=f"(xv) : "r"(h2));
          }
          xv *= L.x_scale[(long long)(t0 + tok) * (L.K / L.x_group) + k / L.x_group];
        }
        s = fmaf(bf(L.A[(long long)rr * L.K + k]), xv, s);
      }
      s = warp_sum(s);
      if (lane == 0) lt[tok][rr] = s;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; n++) {
    float *p = red + (size_t)warp * 16 * TT + (lane >> 2) * TT + 8 * n + 2 * (lane & 3);
    *reinterpret_cast<unsigned long long *>(p) = acc.a[n];
    *reinterpret_cast<unsigned long long *>(p + 8 * TT) = acc.b[n];
  }
  __syncthreads();
  for (int o = tid; o < 16 * nt; o += kLinThreads) {
    const int tok = o / 16, r = o % 16, n = row0 + r;
    if (n >= L.N) continue;
    float s = 0.f;
    for (int w = 0; w < NW; w++) s += red[(size_t)w * 16 * TT + r * TT + tok];
    s *= kActUnit;
    if (L.A) {
      float b = 0.f;
      for (int j = 0; j < L.r; j++) b = fmaf(bf(L.B[(long long)n * L.r + j]), lt[tok][j], b);
      s = fmaf(L.c, b, s);
    }
    const long long at = (long long)(t0 + tok) * L.y_stride + n;
    if (L.y_f32)
      ((float *)L.y)[at] = s;
    else
      ((uint16_t *)L.y)[at] = f2bf(s);
  }
}

}  // namespace e0
