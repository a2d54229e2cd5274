// A whole MoE layer for up to 64 tokens in one cooperative launch (e0_moe_layer_few):
// residual addition, RMSNorm, router, top-k or given routing, int4 experts, the shared expert
// with its unmerged LoRA, weighted combine.
//
// Three phases with a grid-wide barrier between them, one block per SM:
//   1. x = bf16(RMSNorm(bf16(h + delta))) of 1, 2 or 4 tokens in shared memory; a share of the rows
//      [W_r; A_g; A_u] times them (mma.sync m16n8k16 bf16, K split over the warps).
//   2. every block takes the top-k of all tokens (of more than 16 tokens: of its own, and a barrier
//      hands the result round) and groups the (token, slot) assignments by
//      expert into segments of at most 8 tokens (the shared expert is one more expert
//      that every token has); it then computes an equal share, by cost, of the tiles of 8
//      intermediate indices of all segments: 8 gate and 8 up rows, SwiGLU, a = bf16(silu(g) u).
//   3. every block computes an equal share of the output rows for all segments and combines
//      them per token in slot order, routed experts first, so y does not depend on timing.
// Each expert's weights are read once per 8 tokens that chose it, from L2 after the first time.
//
// Measured (256 experts, d = 2048, I = 512, 4 a token, LoRA of rank 16; a captured launch among
// others): 21.3 us for 1 token, 22.3 for 2, 39 for 8, 51 for 16, 99 for 64 (291 MB of weights, 2.9
// TB/s); 64 tokens over 16 experts 55.7.
// One token is a chain of latencies (the norm and router 4.3, two barriers of 1.3, the plan 2.8,
// gate and up 3 to 4.5, down and combine 4.5); 64 are the streams' instructions (gate and up about 41
// us, 4.7 TB/s, down about 29 us) and 30 us of norm, routing, sums and three barriers: over the whole
// launch issue slots and shared-memory wavefronts 51 %, integer pipe 35 %, tensor pipe 16 %.
//
// A launch with few tokens is a chain of latencies, code fetches among them: the streaming loops
// exist in two forms for each of the two products and no more, and what they call at the end
// of a tile is a function.  (724 KB of code with 12 inlined forms took 42 us for 5 tokens of
// d = 256, most of it waiting for instructions.)
//
// Products: bf16 matrix instructions on the activations as they are.  A weight word holds 8 codes
// n0..n7; masked in place, the pairs (n0, n4) and, after a shift by 8, (n2, n6) read as the bf16
// subnormals q 2^-133, the pairs (n1, n5) and (n3, n7) as q 2^-129; one bf16 product with a power of
// two brings each to q 2^-6, the most that a power of two within bf16 reaches.  So a code's products
// q x 2^-6 are exact and the fp32 sums carry nothing beside them; the sums of x, which come with the
// activations, carry 2^-6 too, and the end result is multiplied by 64.
// Rows of x and a are stored with each 8 channels in the order 0 4 1 5 2 6 3 7, so that 16 bytes
// are the operands that meet one word of codes.
#pragma once
#include <cooperative_groups.h>
#include "e0_addnorm.cuh"
#include "e0_int4.cuh"
#include "e0_kernels.cuh"

namespace e0 {

constexpr int kFewMaxT = 64;
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewMaxA = kFewMaxT * (kMaxK + 1);                // assignments
constexpr int kFewMaxSeg = kMaxE + 1 + kFewMaxA / 8;            // segments
constexpr int kFewSeg = 8;                                      // tokens to a segment
constexpr int kFewPad = 16;                                     // bytes between rows: 8 rows in distinct banks
constexpr int kFewNorm = 4;                                     // tokens that a block of phase 1 norms, at most

constexpr float kFewUnit = 64.0f;                               // what sums of products and of x are divided by

struct FewArgs {
  const uint16_t *h, *delta;
  const uint16_t *gamma, *router;
  const uint8_t *experts, *shared;
  const uint16_t *Ag, *Bg, *Au, *Bu, *Ad, *Bd;
  Blob bl;
  int T, d, E, I, k, r;
  double inv_d;
  float eps, c;
  const int32_t *route;
  uint16_t *h_out, *y;
  float *yf;
  int32_t *idx;
  float *gates;
  // workspace
  uint16_t *xb;               // [T][d], channels in operand order
  float *xv;                  // [T][d / 64] sums of x / kFewUnit
  float *logits;              // [T][E]
  float *lt;                  // [T][2][r]
  int32_t *rsel;              // [T][k] routing and gates, where one block routes for all
  float *rgate;
  uint16_t *a;                // [T][k + 1][I], channels in operand order
  float *a8;                  // [T][k + 1][I / 8] sums of a / kFewUnit
  int *err;
  int lora16;                 // rows of LoRA B begin at 16 bytes
  int tpb;                    // tokens that a block of phase 1 norms
  int gu_rows;                // activation rows that fit the staging area of phase 2
  int out_bytes, dn_rows, dn_ring;   // phase 3: bytes of the results; rows whose sums fit; bytes of a warp's ring
};

struct FewPlan {
  FewArgs args;                   // a copy that functions read at shared memory's latency
  float gate[kFewMaxT * kMaxK];
  unsigned long long tok[kMaxE];  // the tokens that chose an expert, one bit each
  unsigned long long scan[kFewWarps];
  uint16_t sel[kFewMaxT * kMaxK];
  uint16_t first[kMaxE + 1];      // place of an expert's first assignment
  uint16_t place[kFewMaxA];       // place of assignment t (k + 1) + j
  uint16_t asg[kFewMaxA];         // assignment at a place
  uint16_t seg_exp[kFewMaxSeg];
  uint16_t seg_at[kFewMaxSeg + 1];
  uint16_t seg_n[kFewMaxSeg];
  int nseg, nplace, n4;           // segments of experts with at most 4 tokens come first
  double part[kFewWarps];
};

__host__ __device__ inline size_t few_plan_bytes() { return (sizeof(FewPlan) + 127) & ~(size_t)127; }
constexpr int kFewZeroBytes = 128;
constexpr int kFewRedBytes = kFewWarps * 16 * kFewSeg * 4;       // partial sums of 16 warps: 16 rows x 8 tokens
constexpr int kFewTdBytes = 16384;                              // parts of t_d (few_td): at most 128 rows of kMaxR
// bytes of an activation row of phase 2 with its sums
__host__ __device__ inline int few_row_bytes(int channels) { return channels * 2 + kFewPad + channels / 64 * 4; }

// mma_bf16_acc without a sum to add to
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 channels 0..7 -> 0 4 1 5 2 6 3 7 and back (pairs of a 16-byte chunk)
__device__ __forceinline__ uint4 operand_order(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}
__device__ __forceinline__ uint4 natural_order(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                    __byte_perm(v.z, v.w, 0x7632));
}

// ---------------------------------------------------------------------------------------
// int4 rows times bf16 columns: 16 rows, blocks of 256 channels (the last may be 128)
// ---------------------------------------------------------------------------------------
// Two forms.  Pair: 4 tokens; the 8 columns of a matrix instruction
// are 4 tokens restricted to one group of 64 and the same 4 restricted to the next, so a lane takes 16
// consecutive bytes of a row and one fold serves both groups.  Wide: 8 tokens, 8 bytes of a row a
// lane, a fold per group.  (Segments of 5 to 8 tokens as two pair tiles: 61.3 us for 64 tokens over 16
// experts, wide 56.3; segments of 16 would need rings that leave no room for the results.)  The accumulators of a lane are rows l / 4 and l / 4 + 8,
// tokens 2 (l & 3), + 1 of a tile (pair: tokens 2 (l & 1), + 1, after adding lanes l and l + 2).
//
// Each warp streams its weights through a ring of its own in shared memory by cp.async, a block to
// a stage.  Phase 2: 256 channels, 16 rows of 128 bytes of codes (their 16-byte chunks permuted by
// row, so that either form reads without bank conflicts); the activations, which every tile needs
// again, are staged apart.  Phase 3: 128 channels, 64 bytes of codes a row and the activations of
// the segment's tokens, which are used once.  The scales and mins of 512 channels (256, 128 where a
// row is no multiple of that), 16 bytes each a row, have slots of their own: fetched block by block,
// each would be 4 or 8 bytes of a 32-byte sector.
constexpr int kFewStage = 16 * 128;
constexpr int kFewDepth = 3;
constexpr int kFewSlot = 16 * 32;
constexpr int kFewRing = kFewDepth * (kFewStage + kFewSlot), kFewRingBytes = kFewWarps * kFewRing;
constexpr int kFewDnHead = 16 * 64, kFewDnRow = 256 + 16;
constexpr int few_dn_stage(int tokens) { return kFewDnHead + tokens * kFewDnRow; }
constexpr int few_dn_depth(int tokens) { return tokens <= 4 ? 3 : 2; }
constexpr int few_dn_ring(int tokens) { return few_dn_depth(tokens) * (few_dn_stage(tokens) + kFewSlot); }

// Activation rows in shared memory: bf16 rows `pitch` bytes apart, and their sums by group.
struct FewOps {
  uint32_t x, v;              // shared addresses
  int pitch, vp;              // bytes between rows of x and of v
};

// A lane's columns: n tokens at row `at` of x and `vat` of the sums; advanced by 128 channels at a time.
template <bool WIDE>
struct FewCol {
  uint32_t x, v0, v1;
  uint32_t step;              // bytes from 128 channels to the next: 256, or 0 at the zeros
  __device__ __forceinline__ void set(const FewOps &O, int at, int vat, int n, uint32_t zero) {
    const int lane = threadIdx.x & 31, t = lane & 3, c = lane >> 2;
    const bool mine = WIDE || (t >> 1) == (c >> 2);
    step = mine ? 256 : 0;
    const int tok = WIDE ? c : c & 3, pair = WIDE ? 2 * t : 2 * (t & 1);
    x = mine ? O.x + (at + min(tok, n - 1)) * O.pitch + (WIDE ? t * 32 : t * 64) : zero;
    v0 = O.v + (vat + min(pair, n - 1)) * O.vp + (WIDE ? 0 : (t >> 1) * 4);
    v1 = O.v + (vat + min(pair + 1, n - 1)) * O.vp + (WIDE ? 0 : (t >> 1) * 4);
  }
  __device__ __forceinline__ void advance(uint32_t xs) {
    x += xs;
    v0 += 8;
    v1 += 8;
  }
};

// Pair i of a word's 8 codes as q 2^-6, in operand order.  (As 128 + q, by one mask and one or, a pair
// is an instruction less, but 128 times the sum of x then stands in the fp32 sums: 4 of their bits.)
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  const uint32_t v = (w >> (i & 2 ? 8 : 0)) & (i & 1 ? 0x00F000F0u : 0x000F000Fu);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(i & 1 ? 0x7D007D00u : 0x7F007F00u));   // 2^123, 2^127
  return r;
}

// One fold: the sums p of a group (pair: of a lane's group of two) with its scales and mins, the
// low (sel 0x1044) or high (0x3244) halves of the words.  v0, v1: addresses of the tokens' sums.
__device__ __forceinline__ void few_fold(const float (&p)[4], uint32_t wsa, uint32_t wma, uint32_t wsb, uint32_t wmb,
                                         uint32_t sel, uint32_t v0, uint32_t v1, float (&acc)[4]) {
  auto pick = [&](uint32_t w) { return __uint_as_float(__byte_perm(w, 0u, sel)); };
  const float sa = pick(wsa), sb = pick(wsb), ma = pick(wma), mb = pick(wmb), x0 = lds32(v0), x1 = lds32(v1);
  acc[0] = fmaf(sa, p[0], fmaf(ma, x0, acc[0]));
  acc[1] = fmaf(sa, p[1], fmaf(ma, x1, acc[1]));
  acc[2] = fmaf(sb, p[2], fmaf(mb, x0, acc[2]));
  acc[3] = fmaf(sb, p[3], fmaf(mb, x1, acc[3]));
}

// 128 channels: the lane's codes at shared address w0 (pair: 16 bytes; wide: 8 bytes, those of the
// second group at w1), `HALF` bytes on those of 8 rows further; scale words (s, m of rows l / 4,
// l / 4 + 8) of the two groups.
template <bool WIDE, int HALF>
__device__ __forceinline__ void few_mul128(uint32_t w0, uint32_t w1, uint32_t wsa, uint32_t wma, uint32_t wsb, uint32_t wmb,
                                           const FewCol<WIDE> &X, float (&acc)[4]) {
  const int t = threadIdx.x & 3;
  if (WIDE) {
#pragma unroll
    for (int g = 0; g < 2; g++) {
      const uint2 wa = lds64(g ? w1 : w0), wb = lds64((g ? w1 : w0) + HALF);
      float p[4];
#pragma unroll
      for (int w = 0; w < 2; w++) {
        const uint32_t xa = w ? wa.y : wa.x, xb = w ? wb.y : wb.x;
        const uint32_t a0 = code_pair(xa, 0), a1 = code_pair(xa, 1), a2 = code_pair(xa, 2), a3 = code_pair(xa, 3);
        const uint32_t b0 = code_pair(xb, 0), b1 = code_pair(xb, 1), b2 = code_pair(xb, 2), b3 = code_pair(xb, 3);
        const uint4 x = lds128(X.x + g * 128 + w * 16);
        if (w == 0) mma_bf16_first(p, a0, b0, a1, b1, x.x, x.y);
        else mma_bf16_acc(p, a0, b0, a1, b1, x.x, x.y);
        mma_bf16_acc(p, a2, b2, a3, b3, x.z, x.w);
      }
      few_fold(p, wsa, wma, wsb, wmb, g ? 0x3244u : 0x1044u, X.v0 + g * 4, X.v1 + g * 4, acc);
    }
  } else {
    const uint4 wa = lds128(w0), wb = lds128(w0 + HALF);
    // (two chains of dependent instructions, joined at the fold)
    float p[4], p2[4];
#pragma unroll
    for (int w = 0; w < 4; w++) {
      const uint32_t xa = w == 0 ? wa.x : w == 1 ? wa.y : w == 2 ? wa.z : wa.w;
      const uint32_t xb = w == 0 ? wb.x : w == 1 ? wb.y : w == 2 ? wb.z : wb.w;
      const uint32_t a0 = code_pair(xa, 0), a1 = code_pair(xa, 1), a2 = code_pair(xa, 2), a3 = code_pair(xa, 3);
      const uint32_t b0 = code_pair(xb, 0), b1 = code_pair(xb, 1), b2 = code_pair(xb, 2), b3 = code_pair(xb, 3);
      const uint4 x = lds128(X.x + w * 16);
      if (w == 0) mma_bf16_first(p, a0, b0, a1, b1, x.x, x.y);
      else mma_bf16_acc(p, a0, b0, a1, b1, x.x, x.y);
      if (w == 0) mma_bf16_first(p2, a2, b2, a3, b3, x.z, x.w);
      else mma_bf16_acc(p2, a2, b2, a3, b3, x.z, x.w);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) p[i] += p2[i];
    few_fold(p, wsa, wma, wsb, wmb, t >> 1 ? 0x3244u : 0x1044u, X.v0, X.v1, acc);
  }
}

// A number whose order as an unsigned integer is the order of the floats, and back; a NaN is the
// lowest but one (0 is what has been taken).
__device__ __forceinline__ uint32_t few_key(float f) {
  const uint32_t u = __float_as_uint(f == f ? (f == 0.f ? 0.f : f) : -INFINITY);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float few_key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// Top-k of E <= 256 keys (lane l holds those of l, l + 32, ...; 0 past the end) over a warp,
// descending, equal values by lower index.  Lane j < k gets the j-th index and its key.
__device__ __forceinline__ int few_topk(uint32_t (&key)[kMaxE / 32], int k, int lane, uint32_t &mine_key) {
  int mine = 0;
#pragma unroll 1
  for (int s = 0; s < k; s++) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < kMaxE / 32; i++) m = max(m, key[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    uint32_t at = 0x7fffffffu;
#pragma unroll
    for (int i = kMaxE / 32 - 1; i >= 0; i--)
      if (key[i] == m) at = lane + 32 * i;
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == s) {
      mine = (int)at;
      mine_key = m;
    }
#pragma unroll
    for (int i = 0; i < kMaxE / 32; i++)
      if ((uint32_t)(lane + 32 * i) == at) key[i] = 0;
  }
  return mine;
}

// ---------------------------------------------------------------------------------------
// Phase 1
// ---------------------------------------------------------------------------------------
// The block's tokens (at most 4) normed into rows at `area` (operand order) with their sums, h'
// behind them, then the block's rows of [router; A_g; A_u].  Every block of the same tokens norms
// them again, which costs less than a grid-wide barrier; so a block has few tokens, and more (up to
// 4) only until its share of the rows is 2 or less.  (256 experts, d = 2048, one token a block
// against four: 26.6 and 23.8 us for 2 tokens, 42.2 and 40.5 for 8, 114 and 102 for 64, 8 tokens a
// block 42.3 for 8; 16 experts, d = 256: 20.2 and 22.8 for 5.)
struct FewTok {
  int ntb, tb, member, members, t0, nt;
  __device__ __forceinline__ explicit FewTok(const FewArgs &A) {
    ntb = (A.T + A.tpb - 1) / A.tpb;
    tb = blockIdx.x % ntb;
    member = blockIdx.x / ntb;
    members = ((int)gridDim.x - tb + ntb - 1) / ntb;
    t0 = tb * A.tpb;
    nt = min(A.tpb, A.T - t0);
  }
};
__device__ __forceinline__ void few_phase1(const FewArgs &A, FewPlan &P, uint8_t *area, float *red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = warp_id(), d = A.d;
  const FewTok K(A);
  const int pitch = d * 2 + kFewPad, vbytes = d / 64 * 4;
  uint8_t *hs = area + kFewNorm * (pitch + vbytes);
  // the first 16 rows are fetched before they are needed: 4 chunks of 32 channels a warp
  const int R = A.E + (A.Ag ? 2 * A.r : 0);
  const int r0 = (int)((long long)R * K.member / K.members), r1 = (int)((long long)R * (K.member + 1) / K.members);
  auto row_ptr = [&](int row) -> const uint16_t * {
    if (row < A.E) return A.router + (size_t)row * d;
    row -= A.E;
    return row < A.r ? A.Ag + (size_t)row * d : A.Au + (size_t)(row - A.r) * d;
  };
  const int nb = d / 32, b0 = nb * warp / kFewWarps, b1 = nb * (warp + 1) / kFewWarps;
  constexpr int PRE = 4;
  uint4 wa[PRE], wb[PRE];
  auto fetch = [&](int q, int b) {
    const uint16_t *ra = row_ptr(min(q + (lane >> 2), r1 - 1)) + (lane & 3) * 8;
    const uint16_t *rb = row_ptr(min(q + (lane >> 2) + 8, r1 - 1)) + (lane & 3) * 8;
    // rows past the share are not fetched: they would be the last row again
    const bool two = q + 8 < r1;
#pragma unroll
    for (int i = 0; i < PRE; i++) {
      wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
      if (b + i < b1) {
        wa[i] = __ldg(reinterpret_cast<const uint4 *>(ra + (b + i) * 32));
        if (two) wb[i] = __ldg(reinterpret_cast<const uint4 *>(rb + (b + i) * 32));
      }
    }
  };
  if (r0 < r1) fetch(r0, b0);
  // 16 warps over nt tokens, 4 to 16 warps each
  const int wpt = K.nt > 2 ? 4 : K.nt > 1 ? 8 : 16, tok = warp / wpt, sub = warp % wpt;
  const bool mine = tok < K.nt;
  uint8_t *xs = area + tok * pitch;
  const int c0 = (sub * 32 + lane) * 8, cl = min(c0, d - 8);
  uint4 gm = __ldg(reinterpret_cast<const uint4 *>(A.gamma + cl));
  double ss = 0.0;
  if (mine) {
    const uint16_t *h = A.h + (size_t)(K.t0 + tok) * d, *dl = A.delta ? A.delta + (size_t)(K.t0 + tok) * d : nullptr;
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 hv = *reinterpret_cast<const uint4 *>(h + cl), dv = dl ? *reinterpret_cast<const uint4 *>(dl + cl) : none;
#pragma unroll 1
    for (int c = c0; c < d; c += wpt * 256) {
      uint32_t ws[4] = {hv.x, hv.y, hv.z, hv.w};
      const uint32_t es[4] = {dv.x, dv.y, dv.z, dv.w};
      const int cn = min(c + wpt * 256, d - 8);     // the next, while this one is worked on
      hv = *reinterpret_cast<const uint4 *>(h + cn);
      if (dl) dv = *reinterpret_cast<const uint4 *>(dl + cn);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (dl) ws[j] = bf16x2(bf_lo(ws[j]) + bf_lo(es[j]), bf_hi(ws[j]) + bf_hi(es[j]));
        const double lo = (double)__uint_as_float(ws[j] << 16), hi = (double)__uint_as_float(ws[j] & 0xFFFF0000u);
        ss = fma(lo, lo, fma(hi, hi, ss));
      }
      *reinterpret_cast<uint4 *>(xs + c * 2) = make_uint4(ws[0], ws[1], ws[2], ws[3]);
    }
  }
  ss = warp_sum(ss);
  if (lane == 0) P.part[warp] = ss;
  __syncthreads();
  if (mine) {
    // (lanes l, l + wpt, ... hold the same: a butterfly over wpt of them)
    ss = P.part[tok * wpt + (lane & (wpt - 1))];
    for (int o = wpt >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double rinv = rsqrt(fma(ss, A.inv_d, (double)A.eps));
    const float rinv_f = norm_rinv(rinv);
#pragma unroll 1
    for (int c = c0; c < d; c += wpt * 256) {
      const uint4 w = *reinterpret_cast<const uint4 *>(xs + c * 2);
      uint32_t most;
      const uint4 o = norm_bf16x8(w, gm, rinv, rinv_f, most);
      gm = __ldg(reinterpret_cast<const uint4 *>(A.gamma + min(c + wpt * 256, d - 8)));
      float v = ((bf_lo(o.x) + bf_hi(o.x)) + (bf_lo(o.y) + bf_hi(o.y))) + ((bf_lo(o.z) + bf_hi(o.z)) + (bf_lo(o.w) + bf_hi(o.w)));
      v = group_sum(v * (1.0f / kFewUnit), 8);                          // d is a multiple of 256: whole warps
      const uint4 xv = operand_order(o);
      *reinterpret_cast<uint4 *>(xs + c * 2) = xv;
      if ((lane & 7) == 0) *reinterpret_cast<float *>(area + kFewNorm * pitch + tok * vbytes + c / 64 * 4) = v;
      if (K.member == 0) {
        *reinterpret_cast<uint4 *>(A.xb + (size_t)(K.t0 + tok) * d + c) = xv;
        if ((lane & 7) == 0) A.xv[(size_t)(K.t0 + tok) * (d / 64) + c / 64] = v;
        if (A.h_out) *reinterpret_cast<uint4 *>(hs + ((size_t)tok * d + c) * 2) = w;
      }
    }
  }
  __syncthreads();
  const uint32_t x = smem_at(area) + min(lane >> 2, K.nt - 1) * pitch + (lane & 3) * 16;
#pragma unroll 1
  for (int q = r0; q < r1; q += 16) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int b = b0; b < b1; b += PRE) {
      if (q != r0 || b != b0) fetch(q, b);
#pragma unroll
      for (int i = 0; i < PRE; i++)
        if (b + i < b1) bf16_mul(wa[i], wb[i], natural_order(lds128(x + (b + i) * 64)), acc);
    }
    float *p = red + warp * 128 + (lane >> 2) * 8 + 2 * (lane & 3);
    p[0] = acc[0];
    p[1] = acc[1];
    p[64] = acc[2];
    p[65] = acc[3];
    __syncthreads();
    if (tid < 128) {
      const int row = q + (tid >> 3), tk = tid & 7;
      if (row < r1 && tk < K.nt) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; w++) s += red[w * 128 + tid];
        if (row < A.E)
          A.logits[(size_t)(K.t0 + tk) * A.E + row] = s;
        else
          A.lt[(size_t)(K.t0 + tk) * 2 * A.r + (row - A.E)] = s;
      }
    }
    __syncthreads();
  }
}

// h' of the block's tokens to h_out, after every block has read h (h_out may be h).
__device__ __forceinline__ void few_residual(const FewArgs &A, const uint8_t *area) {
  const FewTok K(A);
  if (K.member) return;
  const uint8_t *hs = area + kFewNorm * (A.d * 2 + kFewPad + A.d / 64 * 4);
#pragma unroll 1
  for (int c = threadIdx.x * 8; c < K.nt * A.d; c += kFewThreads * 8)
    *reinterpret_cast<uint4 *>(A.h_out + (size_t)K.t0 * A.d + c) = *reinterpret_cast<const uint4 *>(hs + c * 2);
}

// ---------------------------------------------------------------------------------------
// Routing of every token and the segments of (token, slot) assignments by expert
// ---------------------------------------------------------------------------------------
// The given expert of lane j < k for token t, -1 where the token has none.
__device__ __forceinline__ int few_given(const FewArgs &A, int t) {
  const int lane = threadIdx.x & 31;
  return A.route != nullptr && t < A.T && lane < A.k ? __ldg(A.route + (size_t)t * A.k + lane) : -1;
}

// A warp takes one token, whose given experts are `e` (few_given): lane j < k gets its j-th expert and
// gate.  `say`: report bad routing.
__device__ __forceinline__ void few_route(const FewArgs &A, int t, bool say, int &e, float &gate) {
  const int lane = threadIdx.x & 31, k = A.k, E = A.E;
  const float *lg = A.logits + (size_t)t * E;
  float l = -INFINITY;
  if (__shfl_sync(0xffffffffu, e, 0) < 0) {
    uint32_t key[kMaxE / 32], mine = 0;
    float f[kMaxE / 32];
#pragma unroll
    for (int i = 0; i < kMaxE / 32; i++) f[i] = lane + 32 * i < E ? lg[lane + 32 * i] : 0.f;
    unsigned nan = 0;
#pragma unroll
    for (int i = 0; i < kMaxE / 32; i++) {
      nan |= f[i] != f[i];
      key[i] = lane + 32 * i < E ? few_key(f[i]) : 0u;
    }
    e = few_topk(key, k, lane, mine);
    // (with a NaN among the logits the gates are the NaNs that they come to)
    const bool look = __any_sync(0xffffffffu, nan);
    if (lane < k) l = look ? lg[e] : few_key_value(mine);
  } else {
    int bad = 0;
    if (e < 0 || e >= E) {
      bad = DERR_INDEX;
      e = 0;
    }
    if (lane < k) l = lg[e];
    const unsigned same = __match_any_sync(0xffffffffu, lane < k ? e : -1 - lane);
    if (same & (same - 1)) bad |= DERR_DUP;
    if (say && lane < k && bad && A.err) atomicOr(A.err, bad);
  }
  float mx = l;
#pragma unroll
  for (int o = kMaxK / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ex = lane < k ? expf(l - mx) : 0.f;
  gate = ex / group_sum(ex, kMaxK);
}

// Up to this many tokens, every block routes all of them, a warp a token; beyond, each token is
// routed by one block and a second grid-wide barrier (1.3 us) hands the result round.
constexpr int kFewRouteAll = kFewWarps;

__device__ __forceinline__ void few_route_share(const FewArgs &A) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x >= 32) return;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x) {
    int e = few_given(A, t);
    float g;
    few_route(A, t, true, e, g);
    if (lane < A.k) {
      A.rsel[t * A.k + lane] = e;
      A.rgate[t * A.k + lane] = g;
    }
  }
}

// Relative cost of a tile in phase 2: segments of experts of at most 4 tokens, of more.  (1.25, 1.5,
// 1.75, 2 to 1: 106, 102, 99.9, 100.4 us at 64 tokens; 40.1, 40.4, 39.4, 38.9 at 8.)
constexpr int kFewCost4 = 1, kFewCost8 = 2;

// given: few_given of the token that has the warp's number
__device__ __forceinline__ void few_plan(const FewArgs &A, FewPlan &P, int given) {
  const int tid = threadIdx.x, lane = tid & 31, warp = warp_id();
  const int k = A.k, T = A.T, E = A.E;
  static_assert(kFewMaxT * kMaxK <= kFewThreads && kMaxE < kFewThreads, "an assignment, an expert a thread");
  if (tid < kMaxE) P.tok[tid] = 0;
  if (T <= kFewRouteAll) {
    if (warp < T) {
      int e = given;
      float g;
      few_route(A, warp, blockIdx.x == 0, e, g);
      if (lane < k) {
        P.sel[warp * k + lane] = (uint16_t)e;
        P.gate[warp * k + lane] = g;
      }
    }
  } else if (tid < T * k) {
    P.sel[tid] = (uint16_t)A.rsel[tid];
    P.gate[tid] = A.rgate[tid];
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid < T * k) {
    if (A.idx) A.idx[tid] = P.sel[tid];
    if (A.gates) A.gates[tid] = P.gate[tid];
  }
  // The rank of a token among those of its expert is a count of bits, so every block comes to
  // the same segments (an expert with more tokens than a segment holds has several, which
  // different blocks work on).
  if (tid < T * k) atomicOr(&P.tok[P.sel[tid]], 1ull << (tid / k));
  __syncthreads();
  // Places and segments by one prefix sum over the experts, a thread each: experts of at most 4
  // tokens first, then the others.  A class takes 20 bits: 10 of places, 10 of segments (at most
  // 576 and 329).
  const int n = tid < E ? __popcll(P.tok[tid]) : tid == E ? T : 0, cls = n <= 4 ? 0 : 1;
  const int ns = (n + kFewSeg - 1) / kFewSeg;
  const unsigned long long own = (unsigned long long)(n | (ns << 10)) << (20 * cls);
  unsigned long long sum = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) P.scan[warp] = sum;
  __syncthreads();
  unsigned long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kFewWarps; w++) {
    if (w == warp) before = total;
    total += P.scan[w];
  }
  before += sum - own;
  auto places = [](unsigned long long v, int c) { return (int)(v >> (20 * c)) & 1023; };
  auto segs = [](unsigned long long v, int c) { return (int)(v >> (20 * c + 10)) & 1023; };
  int at = places(before, cls), sg = segs(before, cls);
  if (cls) {
    at += places(total, 0);
    sg += segs(total, 0);
  }
  if (n > 0) P.first[tid] = (uint16_t)at;
#pragma unroll 1
  for (int i = 0; i < ns; i++) {
    P.seg_exp[sg + i] = (uint16_t)tid;
    P.seg_at[sg + i] = (uint16_t)(at + i * kFewSeg);
    P.seg_n[sg + i] = (uint16_t)min(kFewSeg, n - i * kFewSeg);
  }
  const int n4 = segs(total, 0), nseg = n4 + segs(total, 1);
  if (tid == 0) {
    P.n4 = n4;
    P.nseg = nseg;
  }
  __syncthreads();
  if (tid == 0) {
    P.nplace = P.seg_at[nseg - 1] + P.seg_n[nseg - 1];   // an expert given twice to a token has one place
    P.seg_at[nseg] = (uint16_t)P.nplace;
  }
#pragma unroll 1
  for (int i = tid; i < T * (k + 1); i += kFewThreads) {
    const int t = i / (k + 1), j = i % (k + 1);
    const int e = j < k ? P.sel[t * k + j] : E;
    const int to = P.first[e] + (j < k ? __popcll(P.tok[e] & ((1ull << t) - 1)) : t);
    P.place[i] = (uint16_t)to;
    // an expert given twice to a token (reported above) is computed once
    bool again = false;
#pragma unroll 1
    for (int q = 0; q < j && j < k; q++) again |= P.sel[t * k + q] == e;
    if (!again) P.asg[to] = (uint16_t)i;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------------------
// Streaming
// ---------------------------------------------------------------------------------------
// The tiles of a warp (or of a team of wk warps that split K): gate/up, every `step`th of a list
// of tiles of 8 indices, `per` to a segment; down, every `step`th segment.
template <bool GU>
struct FewCursor {
  int s, i, left;                 // segment, tile of it, tiles left
  __device__ __forceinline__ void next(int step, int per) {
    left--;
    if (GU) {
      i += step;
#pragma unroll 1
      while (i >= per) {
        i -= per;
        s++;
      }
    } else {
      s += step;
    }
  }
};

struct FewPart {                  // what a warp does of K, and where its team stands
  int b0, b1, wk, team, sub;
};

// SwiGLU of one token (a lane's index l / 4 of tile i8 of segment s), with the shared expert's
// LoRA; a to the workspace in operand order, and the sum of the tile's 8.  g, u: in units of kFewUnit.
__device__ __noinline__ void few_emit(const FewPlan &P, int s, int i8, int tok, float g, float u) {
  const FewArgs &A = P.args;
  const int q = (int)(threadIdx.x & 31) >> 2, n = P.seg_n[s], i = i8 * 8 + q;
  const int asg = P.asg[P.seg_at[s] + min(tok, n - 1)];
  g *= kFewUnit;
  u *= kFewUnit;
  if (P.seg_exp[s] == A.E && A.Ag) {
    const float *lt = A.lt + (size_t)(asg / (A.k + 1)) * 2 * A.r;
    const uint16_t *bg = A.Bg + (size_t)i * A.r, *bu = A.Bu + (size_t)i * A.r;
    float lg = 0.f, lu = 0.f;
    if ((A.r & 7) == 0 && A.lora16) {
#pragma unroll 2
      for (int j = 0; j < A.r; j += 8) {
        const uint4 wg = __ldg(reinterpret_cast<const uint4 *>(bg + j)), wu = __ldg(reinterpret_cast<const uint4 *>(bu + j));
        const float4 *tg = reinterpret_cast<const float4 *>(lt + j), *tu = reinterpret_cast<const float4 *>(lt + A.r + j);
        lg = dot8(wg, tg[0], tg[1], lg);
        lu = dot8(wu, tu[0], tu[1], lu);
      }
    } else {
#pragma unroll 2
      for (int j = 0; j < A.r; j++) {
        lg = fmaf(bf(bg[j]), lt[j], lg);
        lu = fmaf(bf(bu[j]), lt[A.r + j], lu);
      }
    }
    g = fmaf(A.c, lg, g);
    u = fmaf(A.c, lu, u);
  }
  const uint32_t bits = f2bf(g / (1.0f + expf(-g)) * u);
  float sum = bf(bits) * (1.0f / kFewUnit);
  sum += __shfl_xor_sync(0xffffffffu, sum, 4);
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
  if (tok < n) {
    A.a[(size_t)asg * A.I + i8 * 8 + ((q & 3) * 2 + (q >> 2))] = (uint16_t)bits;
    if (q == 0) A.a8[(size_t)asg * (A.I / 8) + i8] = sum;
  }
}

// The join of a team's partial sums (red: [warp][16 rows][8 tokens]).
__device__ __noinline__ void few_join(const FewPlan &P, int s, int i8, int wk, int team, int sub, const float *red) {
  const int lane = threadIdx.x & 31, n = P.seg_n[s];
  bar_team(wk, team);
  // 4 tokens of 8 indices to a warp at a time: lane = token + 4 index
  const float *base = red + team * wk * 16 * kFewSeg + (lane >> 2) * kFewSeg;
#pragma unroll 1
  for (int t0 = sub * 4; t0 < n; t0 += wk * 4) {
    const int tok = t0 + (lane & 3), tk = min(tok, n - 1);
    float g = 0.f, u = 0.f;
#pragma unroll 2
    for (int w = 0; w < wk; w++) {
      g += base[w * 16 * kFewSeg + tk];
      u += base[w * 16 * kFewSeg + 8 * kFewSeg + tk];
    }
    few_emit(P, s, i8, tok, g, u);
  }
  bar_team(wk, team);
}

// Streams a warp's tiles, blocks ahead across the end of a tile too.  Down: rows r0.. (nr of
// them).  Sums go through few_emit / few_join, or (down) to
// out[place][16].
template <bool GU, bool WIDE>
__device__ __forceinline__ void few_stream(const FewArgs &A, const FewPlan &P, const FewOps &O, int p0, FewCursor<GU> C,
                                           int step, int per, const FewPart &W, int r0, int nr, uint32_t zero,
                                           uint32_t ring, float *out) {
  if (C.left <= 0) return;
  constexpr int TOK = WIDE ? 8 : 4, STAGE = GU ? kFewStage : few_dn_stage(TOK);
  const int lane = threadIdx.x & 31, t = lane & 3, r = lane >> 2, warp = warp_id();
  constexpr int stages = GU ? kFewDepth : few_dn_depth(TOK);
  const int K = GU ? A.d : A.I;
  const uint32_t slots = ring, slots_end = slots + stages * kFewSlot;     // of scales, then the stages
  const uint32_t stages_at = slots_end, end = stages_at + stages * STAGE;
  const int cs = K % 512 == 0 ? 4 : K % 256 == 0 ? 2 : 1;                 // 128 channels to a slot
  // what this lane copies of a block.  Phase 2: chunk l & 7 of rows l / 8 + 4 i, the scales or mins
  // of row l / 2.  Phase 3: chunk l & 3 of rows l / 4 and l / 4 + 8, the same of row l / 2, and
  // chunk l & 15 of tokens l / 16 + 2 i.  The pointers run on from block to block.
  const int cr = GU ? lane >> 3 : r, cc = GU ? lane & 7 : t, sr = lane >> 1;
  const uint32_t cdst = GU ? cr * 128 + ((cc ^ row_swz(cr)) << 4) : cr * 64 + ((cc ^ (cr & 2)) << 4);
  const uint32_t sdst = sr * 32 + (lane & 1) * 16;
  FewCursor<GU> L = C;
  int lb = W.b0;
  uint32_t lst = stages_at, lsl = slots;
  const uint8_t *cp = nullptr, *sp = nullptr;     // codes of the first row, scales or mins
  const uint8_t *xp[GU ? 1 : TOK / 2];
  // phase 2: 4 rows on, and from gate to up; phase 3: 8 rows on (the last row again past the end)
  const int row4 = 4 * (K / 2), up = (int)(A.bl.uc - A.bl.gc);
  const int row8 = GU ? 0 : (min(cr + 8, nr - 1) - min(cr, nr - 1)) * (K / 2);
  // a lane's place in the blob of the first index or row
  const int c_at = GU ? (int)A.bl.gc + cr * (K / 2) + W.b0 * 128 + cc * 16
                      : (int)A.bl.dc + (r0 + min(cr, nr - 1)) * (K / 2) + W.b0 * 64 + cc * 16;
  const int s_at = GU ? (int)(lane & 1 ? A.bl.gm : A.bl.gs) + (sr < 8 ? 0 : up) + (sr & 7) * (K / 32) + ((2 * W.b0) & -cs) * 4
                      : (int)(lane & 1 ? A.bl.dm : A.bl.ds) + (r0 + min(sr, nr - 1)) * (K / 32) + (W.b0 & -cs) * 4;
  int xn = 0;                                     // tokens of the segment
  auto issue = [&]() {
    if (L.left > 0) {
      if (lb == W.b0) {
        const int e = P.seg_exp[L.s];
        const uint8_t *blob = e < A.E ? A.experts + (long long)e * A.bl.bytes : A.shared;
        cp = blob + c_at;
        sp = blob + s_at;
        if (GU) {
          cp += L.i * 8 * (K / 2);
          sp += L.i * 8 * (K / 32);
        } else {
          xn = P.seg_n[L.s];
          const int at = P.seg_at[L.s];
#pragma unroll
          for (int i = 0; i < TOK / 2; i++) {
            const int tok = min((lane >> 4) + 2 * i, xn - 1);
            xp[GU ? 0 : i] = reinterpret_cast<const uint8_t *>(A.a + (size_t)(P.asg[at + tok] * A.I) + W.b0 * 128) + (lane & 15) * 16;
          }
        }
      }
      if (lb == W.b0 || ((GU ? 2 * lb : lb) & (cs - 1)) == 0) {
        if (cs == 4) cp_async16(lsl + sdst, sp);
        else if (cs == 2) cp_async_small<8>(lsl + sdst, sp);
        else cp_async_small<4>(lsl + sdst, sp);
        sp += cs * 4;
        lsl = lsl + kFewSlot == slots_end ? slots : lsl + kFewSlot;
      }
      cp_async16(lst + cdst, cp);
      if (GU) {
        cp_async16(lst + cdst + 512, cp + row4);
        const uint8_t *cu = cp + up;
        cp_async16(lst + cdst + 1024, cu);
        cp_async16(lst + cdst + 1536, cu + row4);
        cp += 128;
      } else {
        cp_async16(lst + cdst + 512, cp + row8);
        cp += 64;
        const uint32_t xd = lst + kFewDnHead + (lane >> 4) * kFewDnRow + (lane & 15) * 16;
#pragma unroll
        for (int i = 0; i < TOK / 2; i++)
          if (2 * i < xn) {                       // (the whole warp; with an odd last token half of it)
            if ((lane >> 4) + 2 * i < xn) cp_async16(xd + 2 * i * kFewDnRow, xp[GU ? 0 : i]);
            xp[GU ? 0 : i] += 256;
          }
      }
      lst = lst + STAGE == end ? stages_at : lst + STAGE;
      if (++lb == W.b1) {
        lb = W.b0;
        L.next(step, per);
      }
    }
    cp_async_commit();
  };
  __syncwarp();                           // every lane has left the ring's last use
#pragma unroll 1
  for (int u = 1; u < stages; u++) issue();
  uint32_t st = stages_at, sl = slots_end - kFewSlot;
  // the lane's codes in a stage: pair, chunk t (and, phase 2, 4 + t); wide, the 8 bytes of groups
  // 0 and 1 (and 2 and 3, 64 bytes on before the permutation)
  const int swz = GU ? row_swz(r) : r & 2, pitch = GU ? 128 : 64;
  const uint32_t o0 = r * pitch + (((WIDE ? t >> 1 : t) ^ swz) << 4) + (WIDE ? (t & 1) * 8 : 0);
  const uint32_t o1 = r * pitch + (((2 + (t >> 1)) ^ swz) << 4) + (t & 1) * 8;
  FewCol<WIDE> X;
#pragma unroll 1
  for (; C.left > 0; C.next(step, per)) {
    const int n = P.seg_n[C.s], at = P.seg_at[C.s];
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    X.set(O, GU ? at - p0 : 0, at - p0, n, zero);
    X.x += GU ? 2 * W.b0 * X.step : 0;
    X.v0 += (GU ? 16 : 8) * W.b0;
    X.v1 += (GU ? 16 : 8) * W.b0;
#pragma unroll 1
    for (int b = W.b0; b < W.b1; b++) {
      cp_async_wait_but<stages - 2>();
      __syncwarp();                       // the block has arrived, and every lane has left the one before
      issue();
      const int at128 = (GU ? 2 * b : b) & (cs - 1);
      if (b == W.b0 || at128 == 0) sl = sl + kFewSlot == slots_end ? slots : sl + kFewSlot;
      const uint32_t sc = sl + r * 32 + at128 * 4;
      if (GU) {
        const uint2 s0 = lds64(sc), m0 = lds64(sc + 16), s8 = lds64(sc + 256), m8 = lds64(sc + 272);
        few_mul128<WIDE, 1024>(st + o0, st + o1, s0.x, m0.x, s8.x, m8.x, X, acc);
        X.advance(X.step);
        // chunk c + 4 lies 64 bytes from chunk c, on the side that the permutation leaves
        few_mul128<WIDE, 1024>(st + (o0 ^ 64), st + (o1 ^ 64), s0.y, m0.y, s8.y, m8.y, X, acc);
        X.advance(X.step);
      } else {
        FewCol<WIDE> Y = X;               // the stage's own columns
        Y.x += X.step ? st : 0u;
        few_mul128<WIDE, 512>(st + o0, st + o1, lds32u(sc), lds32u(sc + 16), lds32u(sc + 256), lds32u(sc + 272), Y, acc);
        X.advance(0);
      }
      st = st + STAGE == end ? stages_at : st + STAGE;
    }
    // pair: lanes l and l + 2 hold the same two tokens and take one each; wide: both tokens
    if (!WIDE)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
#pragma unroll
    for (int j = 0; j < (WIDE ? 2 : 1); j++) {
      const int odd = WIDE ? j : t >> 1, tok = WIDE ? 2 * t + j : 2 * (t & 1) + odd;
      const float va = odd ? acc[1] : acc[0], vb = odd ? acc[3] : acc[2];
      if (!GU) {
        if (tok < n) {
          float *p = out + (size_t)(at + tok) * 16 + r;
          p[0] = va;
          p[8] = vb;
        }
      } else if (W.wk == 1) {
        few_emit(P, C.s, C.i, tok, va, vb);
      } else if (tok < n) {
        float *p = out + (warp * 16 + r) * kFewSeg + tok;
        p[0] = va;
        p[8 * kFewSeg] = vb;
      }
    }
    if (GU && W.wk > 1) few_join(P, C.s, C.i, W.wk, W.team, W.sub, out);
  }
}

// ---------------------------------------------------------------------------------------
// Phase 2
// ---------------------------------------------------------------------------------------
// Copies of the x rows of the assignments at places [p0, p1) and their sums by group of 64.
__device__ __forceinline__ FewOps few_stage(const FewArgs &A, const FewPlan &P, int p0, int p1, uint8_t *area) {
  const int n = p1 - p0, G = A.d / 64, pitch = A.d * 2 + kFewPad, lane = threadIdx.x & 31;
  const FewOps O{smem_at(area), smem_at(area + (size_t)n * pitch), pitch, G * 4};
#pragma unroll 1
  for (int r = threadIdx.x >> 5; r < n; r += kFewWarps) {
    const int tok = P.asg[p0 + r] / (A.k + 1);
    const uint16_t *x = A.xb + (size_t)tok * A.d;
#pragma unroll 1
    for (int c = lane; c < A.d / 8; c += 32) cp_async16(O.x + r * pitch + c * 16, x + c * 8);
    // d is a multiple of 256: G of 4
    if (lane < G / 4) cp_async16(O.v + r * O.vp + lane * 16, A.xv + (size_t)tok * G + lane * 4);
  }
  return O;
}

// Tile at which block b's share begins: an equal share of the cost of all tiles.  (At most 329
// segments of 512 tiles of cost 2: 32 bits.)
__device__ __forceinline__ void few_bound(const FewPlan &P, int per, int b, int &s, int &f) {
  const unsigned c1 = (unsigned)(P.n4 * per) * kFewCost4, c2 = (unsigned)((P.nseg - P.n4) * per) * kFewCost8;
  const unsigned pos = (unsigned)((unsigned long long)(c1 + c2) * b / gridDim.x);
  const unsigned tile = pos < c1 ? pos / kFewCost4 : P.n4 * per + (pos - c1) / kFewCost8;
  s = tile / per;
  f = tile % per;
}

__device__ __forceinline__ void few_phase2(const FewArgs &A, const FewPlan &P, uint8_t *area, uint32_t zero, uint32_t ring, float *red) {
  const int per = A.I / 8, NB = A.d / 256, warp = warp_id();
  int sl, fl, sh, fh;
  few_bound(P, per, blockIdx.x, sl, fl);
  few_bound(P, per, blockIdx.x + 1, sh, fh);
  const int s_end = fh > 0 ? sh + 1 : sh;             // one past the last segment
  const int n4 = P.n4;
#pragma unroll 1
  for (int s0 = sl; s0 < s_end;) {
    int s1 = s0 + 1;
#pragma unroll 1
    while (s1 < s_end && P.seg_at[s1 + 1] - P.seg_at[s0] <= A.gu_rows) s1++;
    const int p0 = P.seg_at[s0];
    __syncthreads();
    const FewOps O = few_stage(A, P, p0, P.seg_at[s1], area);
    cp_async_wait();
    __syncthreads();
    // the tiles of segments [a, b) of these: warps to a tile by their number, no more than there
    // are blocks of K
    auto share = [&](int a, int b, FewCursor<true> &C, FewPart &W) {
      a = max(a, s0);
      b = min(b, s1);
      const int f0 = a == sl ? fl : 0, f1 = b == s_end && fh > 0 ? fh : per;
      const int tiles = a < b ? (b - a - 1) * per - f0 + f1 : 0;
      int lg = tiles <= 2 ? 3 : tiles <= 4 ? 2 : tiles <= 8 ? 1 : 0;
      while ((1 << lg) > NB) lg--;
      const int wk = 1 << lg, sub = warp & (wk - 1), team = warp >> lg, teams = kFewWarps >> lg;
      W = FewPart{NB * sub >> lg, NB * (sub + 1) >> lg, wk, team, sub};
      C = FewCursor<true>{a, f0 + team, (tiles - team + teams - 1) / teams};
      while (C.i >= per) {
        C.i -= per;
        C.s++;
      }
      return teams;
    };
    FewCursor<true> C;
    FewPart W;
    if (n4 < s1) {
      const int step = share(n4, P.nseg, C, W);
      few_stream<true, true>(A, P, O, p0, C, step, per, W, 0, 0, zero, ring, red);
    }
    if (s0 < n4) {
      const int step = share(0, n4, C, W);
      few_stream<true, false>(A, P, O, p0, C, step, per, W, 0, 0, zero, ring, red);
    }
    s0 = s1;
  }
}

// ---------------------------------------------------------------------------------------
// Phase 3
// ---------------------------------------------------------------------------------------
// t_d = A_d a_s of every token: 16 rows by 8 tokens, K split over the warps that are left.  td holds a part's T rows
// of kMaxR behind another's: split * T <= 16 / ntt * 8 ntt = 128 rows.
__device__ __forceinline__ int few_td(const FewArgs &A, float *td) {
  const int lane = threadIdx.x & 31, warp = warp_id(), k1 = A.k + 1;
  const int rt = (A.r + 15) / 16, ntt = (A.T + 7) / 8, nb = A.I / 32;
  const int split = min(nb, kFewWarps / (rt * ntt)), u = warp;
  if (u < rt * ntt * split) {
    const int q = u / split / ntt * 16, t0 = u / split % ntt * 8, part = u % split;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const uint16_t *ra = A.Ad + (size_t)min(q + (lane >> 2), A.r - 1) * A.I + (lane & 3) * 8;
    const uint16_t *rb = A.Ad + (size_t)min(q + (lane >> 2) + 8, A.r - 1) * A.I + (lane & 3) * 8;
    const uint16_t *x = A.a + ((size_t)min(t0 + (lane >> 2), A.T - 1) * k1 + A.k) * A.I + (lane & 3) * 8;
#pragma unroll 4
    for (int b = nb * part / split; b < nb * (part + 1) / split; b++)
      bf16_mul(__ldg(reinterpret_cast<const uint4 *>(ra + b * 32)), __ldg(reinterpret_cast<const uint4 *>(rb + b * 32)),
               natural_order(*reinterpret_cast<const uint4 *>(x + b * 32)), acc);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int row = q + (lane >> 2) + 8 * (j >> 1), t = t0 + 2 * (lane & 3) + (j & 1);
      if (row < A.r && t < A.T) td[(part * A.T + t) * kMaxR + row] = acc[j];
    }
  }
  return split;
}

// area: t_d, the results, the sums of the activations, the rings
__device__ __forceinline__ void few_phase3(const FewArgs &A, const FewPlan &P, uint8_t *area, uint32_t zero) {
  const int tid = threadIdx.x, warp = warp_id();
  const int lo = (int)((long long)A.d * blockIdx.x / gridDim.x), hi = (int)((long long)A.d * (blockIdx.x + 1) / gridDim.x);
  if (lo >= hi) return;
  const int G = A.I / 64, NB = A.I / 128, k1 = A.k + 1, nplace = P.nplace;
  float *td = reinterpret_cast<float *>(area), *out = reinterpret_cast<float *>(area + kFewTdBytes);
  float *sums = reinterpret_cast<float *>(area + kFewTdBytes + A.out_bytes);
  const uint32_t ring = smem_at(sums) + ((A.dn_rows * G * 4 + 15) & ~15) + warp * A.dn_ring;
  bool first = true;
#pragma unroll 1
  for (int r0 = lo; r0 < hi; r0 += 16) {
    const int nr = min(16, hi - r0);
    // parts of K: more where there are few segments to keep the warps busy
    int lg = 0;
    while (lg < 2 && (P.nseg << (lg + 1)) <= kFewWarps && (2 << lg) <= NB && (2 << lg) * nplace * 64 <= A.out_bytes) lg++;
    // 16 warps are a multiple of the parts, so a warp stays with one part
    const int parts = 1 << lg, part = warp & (parts - 1), team = warp >> lg, step = kFewWarps >> lg;
    const FewPart W{NB * part >> lg, NB * (part + 1) >> lg, 1, 0, 0};
    float *o = out + (size_t)part * nplace * 16;
#pragma unroll 1
    for (int s0 = 0; s0 < P.nseg;) {
      int s1 = P.nseg;
      if (nplace > A.dn_rows) {
        s1 = s0 + 1;
#pragma unroll 1
        while (s1 < P.nseg && P.seg_at[s1 + 1] - P.seg_at[s0] <= A.dn_rows) s1++;
      }
      const int p0 = P.seg_at[s0], p1 = P.seg_at[s1];
      __syncthreads();
      // sums by group of 64 of the tiles' sums (u / G by its reciprocal: u < 2^16); a thread's first
      // is on its way while t_d is formed
      const uint32_t rg = 0xFFFFFFFFu / G + 1;
      const int nsum = (p1 - p0) * G;
      auto tile_sums = [&](int u, float4 &v, float4 &w) {
        const int p = __umulhi(u, rg), g = u - p * G;
        const float4 *q = reinterpret_cast<const float4 *>(A.a8 + (size_t)P.asg[p0 + p] * (A.I / 8) + g * 8);
        v = q[0];
        w = q[1];
      };
      float4 v0, w0;
      if (tid < nsum) tile_sums(tid, v0, w0);
      const int split = A.Ad && first ? few_td(A, td) : 0;
      if (tid < nsum) sums[tid] = ((v0.x + v0.y) + (v0.z + v0.w)) + ((w0.x + w0.y) + (w0.z + w0.w));
#pragma unroll 4
      for (int u = tid + kFewThreads; u < nsum; u += kFewThreads) {
        float4 v, w;
        tile_sums(u, v, w);
        sums[u] = ((v.x + v.y) + (v.z + v.w)) + ((w.x + w.y) + (w.z + w.w));
      }
      __syncthreads();
      if (split > 1) {
        // each column is read and written by one thread, and read by others after the barrier below
#pragma unroll 1
        for (int u = tid; u < A.T * kMaxR; u += kFewThreads) {
          float v = td[u];
#pragma unroll 4
          for (int w = 1; w < split; w++) v += td[w * A.T * kMaxR + u];
          td[u] = v;
        }
      }
      first = false;
      const FewOps O{kFewDnHead, smem_at(sums), kFewDnRow, G * 4};
      const int m4 = max(s0, min(s1, P.n4));
      auto cursor = [&](int a, int b) { return FewCursor<false>{a + team, 0, (b - a - team + step - 1) >> (4 - lg)}; };
      if (m4 < s1) few_stream<false, true>(A, P, O, p0, cursor(m4, s1), step, 0, W, r0, nr, zero, ring, o);
      if (s0 < m4) few_stream<false, false>(A, P, O, p0, cursor(s0, m4), step, 0, W, r0, nr, zero, ring, o);
      s0 = s1;
    }
    __syncthreads();
#pragma unroll 1
    for (int u = tid; u < 16 * A.T; u += kFewThreads) {
      const int t = u / 16, q = u % 16, row = r0 + q;
      if (q >= nr) continue;
      float y = 0.f;
#pragma unroll 1
      for (int j = 0; j <= A.k; j++) {
        const float *p = out + (size_t)P.place[t * k1 + j] * 16 + q;
        float v = p[0];
#pragma unroll 1
        for (int w = 1; w < parts; w++) v += p[(size_t)w * nplace * 16];
        v *= kFewUnit;
        y = j < A.k ? fmaf(P.gate[t * A.k + j], v, y) : y + v;
      }
      if (A.Ad) {
        const uint16_t *bd = A.Bd + (size_t)row * A.r;
        const float *tv = td + t * kMaxR;
        float b = 0.f;
        if ((A.r & 7) == 0 && A.lora16) {
#pragma unroll 2
          for (int j = 0; j < A.r; j += 8)
            b = dot8(__ldg(reinterpret_cast<const uint4 *>(bd + j)), *reinterpret_cast<const float4 *>(tv + j),
                     *reinterpret_cast<const float4 *>(tv + j + 4), b);
        } else {
#pragma unroll 2
          for (int j = 0; j < A.r; j++) b = fmaf(bf(bd[j]), tv[j], b);
        }
        y = fmaf(A.c, b, y);
      }
      A.y[(size_t)t * A.d + row] = f2bf(y);
      if (A.yf) A.yf[(size_t)t * A.d + row] = y;
    }
  }
}

__global__ void __launch_bounds__(kFewThreads, 1) k_moe_few(const __grid_constant__ FewArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  FewPlan &P = *reinterpret_cast<FewPlan *>(smem);
  uint8_t *zero = smem + few_plan_bytes(), *red_area = zero + kFewZeroBytes, *rings = red_area + kFewRedBytes;
  uint8_t *area = rings + kFewRingBytes;          // phase 1, which streams nothing, takes the rings too
  float *red = reinterpret_cast<float *>(red_area);
  const uint32_t ring = smem_at(rings) + (threadIdx.x >> 5) * kFewRing;
  if (threadIdx.x < kFewZeroBytes / 4) reinterpret_cast<uint32_t *>(zero)[threadIdx.x] = 0;
  static_assert(sizeof(FewArgs) % 4 == 0 && sizeof(FewArgs) / 4 <= kFewThreads, "one word of the arguments a thread");
  if (threadIdx.x < sizeof(FewArgs) / 4)
    reinterpret_cast<uint32_t *>(&P.args)[threadIdx.x] = reinterpret_cast<const uint32_t *>(&A)[threadIdx.x];
  cooperative_groups::grid_group grid = cooperative_groups::this_grid();
  const int given = few_given(A, threadIdx.x >> 5);
  few_phase1(A, P, rings, red);
  grid.sync();
  if (A.h_out) few_residual(A, rings);
  if (A.T > kFewRouteAll) {
    few_route_share(A);
    grid.sync();
  }
  few_plan(A, P, given);
  few_phase2(A, P, area, smem_at(zero), ring, red);
  grid.sync();
  few_phase3(A, P, red_area, smem_at(zero));
}

}  // namespace e0
