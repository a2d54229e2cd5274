// A whole MoE layer for up to 64 tokens in one cooperative launch (e0_moe_layer_few):
// residual addition, RMSNorm, router, top-k or given routing, int4 experts, the shared expert
// with its unmerged LoRA, weighted combine.
//
// Three phases with a grid-wide barrier between them, one block per SM:
//   1. x = bf16(RMSNorm(bf16(h + delta))) of 8 tokens in shared memory; a share of the rows
//      [W_r; A_g; A_u] times them (mma.sync m16n8k16 bf16, K split over the warps).
//   2. every block takes the top-k of all tokens and groups the (token, slot) assignments by
//      expert into segments of at most `seg_cap` tokens (the shared expert is one more expert
//      that every token has); it then computes an equal share of the intermediate indices of
//      all segments: a gate and an up row each, SwiGLU, a = bf16(silu(g) u).
//   3. every block computes an equal share of the output rows for all segments and combines
//      them per token in slot order, routed experts first, so y does not depend on timing.
// Each expert's weights are read once per 32 tokens that chose it (16 or 8 where wide
// activations leave less shared memory).
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
constexpr int kFewMaxPos = kFewMaxA + kFewMaxSeg + 1;           // places, each segment padded to even

struct FewArgs {
  const uint16_t *h, *delta;
  const uint16_t *gamma, *router;
  const uint8_t *experts, *shared;
  const uint16_t *Ag, *Bg, *Au, *Bu, *Ad, *Bd;
  Blob bl;
  int T, d, E, I, k, r;
  float eps, c;
  const int32_t *route;
  uint16_t *h_out, *y;
  float *yf;
  int32_t *idx;
  float *gates;
  // workspace
  uint16_t *xb;               // [T][d]
  float *logits;              // [T][E]
  float *lt;                  // [T][2][r]
  uint16_t *a;                // [T][k + 1][I]
  int *err;
  int seg_cap;                // tokens to a segment: 8, 16 or 32
  int gu_rows, dn_rows;       // activation rows that fit the staging area in phases 2 and 3
  int parts_bytes;            // bytes of the down-projection results in phase 3
};

struct FewPlan {
  float gate[kFewMaxT * kMaxK];
  uint16_t sel[kFewMaxT * kMaxK];
  unsigned long long tok[kMaxE];  // the tokens that chose an expert, one bit each
  uint16_t first[kMaxE + 1];      // place of an expert's first assignment
  uint16_t place[kFewMaxA];       // place of assignment t (k + 1) + j
  int16_t asg[kFewMaxPos];        // assignment at a place, -1 for padding
  uint16_t seg_exp[kFewMaxSeg];
  uint16_t seg_at[kFewMaxSeg + 1];
  uint16_t seg_n[kFewMaxSeg];
  int nseg, nplace;
  double part[kFewWarps];
};

__host__ __device__ inline size_t few_plan_bytes() { return (sizeof(FewPlan) + 127) & ~(size_t)127; }
constexpr int kFewRedBytes = kFewWarps * 16 * 32 * 4;            // partial sums of 16 warps: 16 rows x 32 tokens

__device__ __forceinline__ void bar_team(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void mma_bf16_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bf16 rows times 8 bf16 columns over channels [k0, k1) (multiples of 32): ra, rb the
// lane's rows l / 4 and l / 4 + 8, x its column, each at channel 8 (l & 3).
__device__ __forceinline__ void bf16_rows(const uint16_t *ra, const uint16_t *rb, const uint16_t *x, int k0, int k1,
                                          float (&acc)[4]) {
#pragma unroll 4
  for (int k = k0; k < k1; k += 32) {
    const uint4 a = *reinterpret_cast<const uint4 *>(ra + k), b = *reinterpret_cast<const uint4 *>(rb + k);
    const uint4 v = *reinterpret_cast<const uint4 *>(x + k);
    mma_bf16_acc(acc, a.x, b.x, a.y, b.y, v.x, v.y);
    mma_bf16_acc(acc, a.z, b.z, a.w, b.w, v.z, v.w);
  }
}

// Top-k of E <= 256 logits over a warp, descending, equal values by lower index; a NaN counts
// as the lowest value, so every index is valid.
__device__ __forceinline__ void few_topk(const float *v, int E, int k, int lane, int *out) {
  float vals[kMaxE / 32];
  unsigned left = 0;
#pragma unroll
  for (int i = 0; i < kMaxE / 32; i++) {
    const int e = lane + 32 * i;
    vals[i] = -INFINITY;
    if (e < E) {
      const float f = v[e];
      vals[i] = f == f ? f : -INFINITY;
      left |= 1u << i;
    }
  }
#pragma unroll
  for (int s = 0; s < kMaxK; s++) {
    if (s >= k) break;
    float bv = -INFINITY;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kMaxE / 32; i++)
      if (((left >> i) & 1u) && (be == 0x7fffffff || vals[i] > bv)) {
        bv = vals[i];
        be = lane + 32 * i;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (ov > bv || (ov == bv && oe < be)) {
        bv = ov;
        be = oe;
      }
    }
    out[s] = be;
    if ((be & 31) == lane) left &= ~(1u << (be >> 5));
  }
}

// Phase 1: the block's 8 tokens (8 tb ..) normed into xs, then its rows.
__device__ __forceinline__ void few_phase1(const FewArgs &A, FewPlan &P, uint8_t *area, float *red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ntb = (A.T + 7) / 8, tb = blockIdx.x % ntb, member = blockIdx.x / ntb;
  const int members = ((int)gridDim.x - tb + ntb - 1) / ntb;
  const int t0 = tb * 8, nt = min(8, A.T - t0), d = A.d;
  uint16_t *xs = reinterpret_cast<uint16_t *>(area);
  const int pitch = d + kActPad / 2;
  // 16 warps over nt tokens, 2 to 16 warps each
  const int wpt = nt > 4 ? 2 : nt > 2 ? 4 : nt > 1 ? 8 : 16, tok = warp / wpt, sub = warp % wpt;
  const bool mine = tok < nt;
  const uint16_t *h = A.h + (size_t)(t0 + tok) * d, *dl = A.delta ? A.delta + (size_t)(t0 + tok) * d : nullptr;
  auto load8 = [&](int c, float *v) {
    const uint4 w = *reinterpret_cast<const uint4 *>(h + c);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[2 * j] = __uint_as_float(ws[j] << 16);
      v[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
    }
  };
  double ss = 0.0;
  if (mine)
    for (int c = (sub * 32 + lane) * 8; c < d; c += wpt * 256) {
      float v[8];
      load8(c, v);
      if (dl) {
        const uint4 w = *reinterpret_cast<const uint4 *>(dl + c);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 8; j++)
          v[j] = bf(add_bf16(v[j], __uint_as_float(j & 1 ? ws[j >> 1] & 0xFFFF0000u : ws[j >> 1] << 16)));
      }
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; j++) o[j] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xFFFF0000u);
      const uint4 hv = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4 *>(xs + (size_t)tok * pitch + c) = hv;
#pragma unroll
      for (int j = 0; j < 8; j++) ss = fma((double)v[j], (double)v[j], ss);
    }
  ss = warp_sum(ss);
  if (lane == 0) P.part[warp] = ss;
  __syncthreads();
  if (mine) {
    ss = 0.0;
    for (int w = 0; w < wpt; w++) ss += P.part[tok * wpt + w];
    const double rinv = 1.0 / sqrt(ss / d + (double)A.eps);
    const float rinv_f = (float)rinv;
    for (int c = (sub * 32 + lane) * 8; c < d; c += wpt * 256) {
      uint4 *at = reinterpret_cast<uint4 *>(xs + (size_t)tok * pitch + c);
      const uint4 w = *at, g = __ldg(reinterpret_cast<const uint4 *>(A.gamma + c));
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w}, gs[4] = {g.x, g.y, g.z, g.w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t b0 = norm_bf16(__uint_as_float(ws[j] << 16), __uint_as_float(gs[j] << 16), rinv, rinv_f);
        const uint32_t b1 = norm_bf16(__uint_as_float(ws[j] & 0xFFFF0000u), __uint_as_float(gs[j] & 0xFFFF0000u), rinv, rinv_f);
        o[j] = b0 | (b1 << 16);
      }
      const uint4 xv = make_uint4(o[0], o[1], o[2], o[3]);
      *at = xv;
      if (member == 0) *reinterpret_cast<uint4 *>(A.xb + (size_t)(t0 + tok) * d + c) = xv;
    }
  }
  __syncthreads();
  // rows [router; A_g; A_u] of this member
  const int R = A.E + (A.Ag ? 2 * A.r : 0);
  const int r0 = (int)((long long)R * member / members), r1 = (int)((long long)R * (member + 1) / members);
  auto row_ptr = [&](int row) -> const uint16_t * {
    if (row < A.E) return A.router + (size_t)row * d;
    row -= A.E;
    return row < A.r ? A.Ag + (size_t)row * d : A.Au + (size_t)(row - A.r) * d;
  };
  const int nb = d / 32, k0 = nb * warp / kFewWarps * 32, k1 = nb * (warp + 1) / kFewWarps * 32;
  const uint16_t *x = xs + (size_t)min(lane >> 2, nt - 1) * pitch + (lane & 3) * 8;
  for (int q = r0; q < r1; q += 16) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const uint16_t *ra = row_ptr(min(q + (lane >> 2), r1 - 1)) + (lane & 3) * 8;
    const uint16_t *rb = row_ptr(min(q + (lane >> 2) + 8, r1 - 1)) + (lane & 3) * 8;
    bf16_rows(ra, rb, x, k0, k1, acc);
    float *p = red + warp * 128 + (lane >> 2) * 8 + 2 * (lane & 3);
    p[0] = acc[0];
    p[1] = acc[1];
    p[64] = acc[2];
    p[65] = acc[3];
    __syncthreads();
    if (tid < 128) {
      const int row = q + (tid >> 3), tk = tid & 7;
      if (row < r1 && tk < nt) {
        float s = 0.f;
        for (int w = 0; w < kFewWarps; w++) s += red[w * 128 + tid];
        if (row < A.E)
          A.logits[(size_t)(t0 + tk) * A.E + row] = s;
        else
          A.lt[(size_t)(t0 + tk) * 2 * A.r + (row - A.E)] = s;
      }
    }
    __syncthreads();
  }
}

// h' = bf16(h + delta) to h_out, after every block has read h (h_out may be h).
__device__ __forceinline__ void few_residual(const FewArgs &A) {
  const size_t n = (size_t)A.T * A.d;
  for (size_t c = ((size_t)blockIdx.x * kFewThreads + threadIdx.x) * 8; c < n; c += (size_t)gridDim.x * kFewThreads * 8) {
    const uint4 w = *reinterpret_cast<const uint4 *>(A.h + c);
    uint4 o = w;
    if (A.delta) {
      const uint4 e = *reinterpret_cast<const uint4 *>(A.delta + c);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w}, es[4] = {e.x, e.y, e.z, e.w};
      uint32_t os[4];
#pragma unroll
      for (int j = 0; j < 4; j++)
        os[j] = add_bf16(__uint_as_float(ws[j] << 16), __uint_as_float(es[j] << 16)) |
                (uint32_t)add_bf16(__uint_as_float(ws[j] & 0xFFFF0000u), __uint_as_float(es[j] & 0xFFFF0000u)) << 16;
      o = make_uint4(os[0], os[1], os[2], os[3]);
    }
    *reinterpret_cast<uint4 *>(A.h_out + c) = o;
  }
}

// Routing of every token and the segments of (token, slot) assignments by expert.
__device__ __forceinline__ void few_plan(const FewArgs &A, FewPlan &P) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int k = A.k, T = A.T, E = A.E;
  for (int e = tid; e < kMaxE; e += kFewThreads) P.tok[e] = 0;
  for (int t = warp; t < T; t += kFewWarps) {
    const float *lg = A.logits + (size_t)t * E;
    int sel[kMaxK];
    const bool own = A.route == nullptr || A.route[(size_t)t * k] < 0;
    int bad = 0;
    if (own) {
      few_topk(lg, E, k, lane, sel);
    } else {
#pragma unroll
      for (int j = 0; j < kMaxK; j++) {
        if (j >= k) break;
        int e = A.route[(size_t)t * k + j];
        if (e < 0 || e >= E) {
          bad |= DERR_INDEX;
          e = 0;
        }
        sel[j] = e;
      }
#pragma unroll
      for (int j = 0; j < kMaxK; j++)
#pragma unroll
        for (int q = 0; q < j; q++)
          if (j < k && sel[j] == sel[q]) bad |= DERR_DUP;
    }
    float ex[kMaxK], mx = -INFINITY, sum = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxK; j++) {
      if (j >= k) break;
      ex[j] = lg[sel[j]];
      mx = fmaxf(mx, ex[j]);
    }
#pragma unroll
    for (int j = 0; j < kMaxK; j++) {
      if (j >= k) break;
      ex[j] = expf(ex[j] - mx);
      sum += ex[j];
    }
#pragma unroll
    for (int j = 0; j < kMaxK; j++) {
      if (j >= k || lane != j) continue;
      const float g = ex[j] / sum;
      P.sel[t * k + j] = (uint16_t)sel[j];
      P.gate[t * k + j] = g;
      if (blockIdx.x == 0) {
        if (A.idx) A.idx[(size_t)t * k + j] = sel[j];
        if (A.gates) A.gates[(size_t)t * k + j] = g;
      }
    }
    if (bad && lane == 0 && blockIdx.x == 0 && A.err) atomicOr(A.err, bad);
  }
  __syncthreads();
  // The rank of a token among those of its expert is a count of bits, so every block comes to
  // the same segments (an expert with more tokens than a segment holds has several, which
  // different blocks work on).
  for (int i = tid; i < T * k; i += kFewThreads) atomicOr(&P.tok[P.sel[i]], 1ull << (i / k));
  __syncthreads();
  if (warp == 0) {
    // places (each segment padded to even) and segments: prefix sums over the experts
    int place = 0, seg = 0;
    for (int e0 = 0; e0 <= E; e0 += 32) {
      const int e = e0 + lane, n = e < E ? __popcll(P.tok[e]) : e == E ? T : 0;
      const int ns = (n + A.seg_cap - 1) / A.seg_cap, np = (n + 1) & ~1;
      int ps = np, ss = ns;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, ps, o), b = __shfl_up_sync(0xffffffffu, ss, o);
        if (lane >= o) {
          ps += a;
          ss += b;
        }
      }
      const int at = place + ps - np, sg = seg + ss - ns;
      if (e <= E) P.first[e] = (uint16_t)at;
      for (int i = 0; i < ns; i++) {
        P.seg_exp[sg + i] = (uint16_t)e;
        P.seg_at[sg + i] = (uint16_t)(at + i * A.seg_cap);
        P.seg_n[sg + i] = (uint16_t)min(A.seg_cap, n - i * A.seg_cap);
      }
      if (n & 1) P.asg[at + n] = -1;
      place += __shfl_sync(0xffffffffu, ps, 31);
      seg += __shfl_sync(0xffffffffu, ss, 31);
    }
    if (lane == 0) {
      P.nseg = seg;
      P.nplace = place;
      P.seg_at[seg] = (uint16_t)place;
    }
  }
  __syncthreads();
  for (int i = tid; i < T * (k + 1); i += kFewThreads) {
    const int t = i / (k + 1), j = i % (k + 1);
    const int e = j < k ? P.sel[t * k + j] : E;
    const int at = P.first[e] + (j < k ? __popcll(P.tok[e] & ((1ull << t) - 1)) : t);
    P.place[i] = (uint16_t)at;
    // an expert given twice to a token (reported above) is computed once
    bool again = false;
    for (int q = 0; q < j && j < k; q++) again |= P.sel[t * k + q] == e;
    if (!again) P.asg[at] = (int16_t)i;
  }
  __syncthreads();
}

// Brings the bf16 rows of the assignments at places [p0, p1) into the staging area as matrix
// operands; src(assignment) is a row of 64 G channels.
template <class F>
__device__ __forceinline__ ActDst few_stage(const FewPlan &P, int p0, int p1, int G, uint8_t *area, F src) {
  const int n = p1 - p0, pitch = act_pitch(G);
  ActDst D{area, reinterpret_cast<float *>(area + (size_t)n * pitch), pitch, (n + 1) / 2};
  const int i = threadIdx.x & 7;
  for (int u0 = 0; u0 < n * G; u0 += kFewThreads / 8) {
    const int u = u0 + (int)threadIdx.x / 8;
    const bool in = u < n * G;
    const int row = in ? u / G : 0, g = in ? u % G : 0, asg = P.asg[p0 + row];
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in && asg >= 0) w = *reinterpret_cast<const uint4 *>(src(asg) + g * 64 + i * 8);
    act_group_bf16(w, i, row, g, D, in);
  }
  return D;
}

// One team's tile of phase 2: 8 intermediate indices i0.. (n8 of them) of a segment.
template <int NT>
__device__ __forceinline__ void few_gate_up(const FewArgs &A, const FewPlan &P, const ActDst &D, int p0, int seg, int i0,
                                            int n8, int team, int wk, float *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % wk;
  const int G = A.d / 64, e = P.seg_exp[seg], n = P.seg_n[seg], at = P.seg_at[seg] - p0;
  const uint8_t *blob = e < A.E ? A.experts + (long long)e * A.bl.bytes : A.shared;
  const int row = i0 + min(lane >> 2, n8 - 1);
  const Int4Row ra{blob + A.bl.gc + (size_t)row * (A.d / 2) + (lane & 3) * 8,
                   reinterpret_cast<const uint16_t *>(blob + A.bl.gs) + (size_t)row * G,
                   reinterpret_cast<const uint16_t *>(blob + A.bl.gm) + (size_t)row * G};
  const Int4Row rb{blob + A.bl.uc + (size_t)row * (A.d / 2) + (lane & 3) * 8,
                   reinterpret_cast<const uint16_t *>(blob + A.bl.us) + (size_t)row * G,
                   reinterpret_cast<const uint16_t *>(blob + A.bl.um) + (size_t)row * G};
  const uint8_t *col[NT], *sv[NT];
#pragma unroll
  for (int q = 0; q < NT; q++) {
    col[q] = D.op + (size_t)(at + min(8 * q + (lane >> 2), n - 1)) * D.pitch + (lane & 3) * 16;
    sv[q] = reinterpret_cast<const uint8_t *>(D.sv) + (at / 2 + min(4 * q + (lane & 3), (n - 1) / 2)) * 16;
  }
  Int4Acc<NT> acc;
  acc.clear();
  int4_rows<NT>(ra, rb, G * sub / wk, G * (sub + 1) / wk, 0, col, sv, D.pairs * 16, acc);
  float *mine = red + warp * 16 * 32;
#pragma unroll
  for (int q = 0; q < NT; q++) {
    float *p = mine + (lane >> 2) * 32 + 8 * q + 2 * (lane & 3);
    *reinterpret_cast<unsigned long long *>(p) = acc.a[q];
    *reinterpret_cast<unsigned long long *>(p + 8 * 32) = acc.b[q];
  }
  if (wk > 1) bar_team(1 + team, wk * 32); else __syncwarp();
  const float *base = red + team * wk * 16 * 32;
  for (int o = sub * 32 + lane; o < 8 * n; o += wk * 32) {
    const int q = o & 7, tok = o >> 3;
    if (q >= n8) continue;
    float g = 0.f, u = 0.f;
    for (int w = 0; w < wk; w++) {
      g += base[w * 16 * 32 + q * 32 + tok];
      u += base[w * 16 * 32 + (8 + q) * 32 + tok];
    }
    g *= kActUnit;
    u *= kActUnit;
    const int asg = P.asg[P.seg_at[seg] + tok], i = i0 + q;
    if (e == A.E && A.Ag) {
      const float *lt = A.lt + (size_t)(asg / (A.k + 1)) * 2 * A.r;
      float lg = 0.f, lu = 0.f;
      for (int j = 0; j < A.r; j++) {
        lg = fmaf(bf(A.Bg[(size_t)i * A.r + j]), lt[j], lg);
        lu = fmaf(bf(A.Bu[(size_t)i * A.r + j]), lt[A.r + j], lu);
      }
      g = fmaf(A.c, lg, g);
      u = fmaf(A.c, lu, u);
    }
    A.a[(size_t)asg * A.I + i] = f2bf(g / (1.0f + expf(-g)) * u);
  }
  if (wk > 1) bar_team(1 + team, wk * 32); else __syncwarp();
}

// Phase 2: this block's share of all (segment, intermediate index) units.
__device__ __forceinline__ void few_phase2(const FewArgs &A, const FewPlan &P, uint8_t *area, float *red) {
  const int warp = threadIdx.x >> 5, I = A.I, G = A.d / 64;
  const long long units = (long long)P.nseg * I;
  const int lo = (int)(units * blockIdx.x / gridDim.x), hi = (int)(units * (blockIdx.x + 1) / gridDim.x);
  for (int s0 = lo / I; s0 * I < hi && lo < hi;) {
    int s1 = s0 + 1;
    while (s1 * I < hi && P.seg_at[s1 + 1] - P.seg_at[s0] <= A.gu_rows) s1++;
    const int p0 = P.seg_at[s0], p1 = P.seg_at[s1];
    __syncthreads();
    const uint16_t *xb = A.xb;
    const int k1 = A.k + 1, d = A.d;
    const ActDst D = few_stage(P, p0, p1, G, area, [=](int asg) { return xb + (size_t)(asg / k1) * d; });
    __syncthreads();
    int tiles = 0;
    for (int s = s0; s < s1; s++) tiles += (min(hi, (s + 1) * I) - max(lo, s * I) + 7) / 8;
    // warps to a tile (K split): all of them where there are few tiles
    const int wk = tiles <= 1 ? 16 : tiles <= 2 ? 8 : tiles <= 4 ? 4 : tiles <= 8 ? 2 : 4;
    const int team = warp / wk, teams = kFewWarps / wk;
    int s = s0, base = 0;
    for (int q = team; q < tiles; q += teams) {
      int i0, i1;
      for (;;) {
        i0 = max(lo, s * I) - s * I;
        i1 = min(hi, (s + 1) * I) - s * I;
        const int nq = (i1 - i0 + 7) / 8;
        if (q < base + nq) break;
        base += nq;
        s++;
      }
      const int i = i0 + (q - base) * 8, n8 = min(8, i1 - i), n = P.seg_n[s];
      if (n <= 8)
        few_gate_up<1>(A, P, D, p0, s, i, n8, team, wk, red);
      else if (n <= 16)
        few_gate_up<2>(A, P, D, p0, s, i, n8, team, wk, red);
      else
        few_gate_up<4>(A, P, D, p0, s, i, n8, team, wk, red);
    }
    s0 = s1;
  }
}

// One warp's part of phase 3: 16 output rows (nr of them) of a segment over a part of K.
template <int NT>
__device__ __forceinline__ void few_down(const FewArgs &A, const FewPlan &P, const ActDst &D, int p0, int seg, int r0,
                                         int nr, int g0, int g1, float *out) {
  const int lane = threadIdx.x & 31;
  const int G = A.I / 64, e = P.seg_exp[seg], n = P.seg_n[seg], at = P.seg_at[seg] - p0;
  const uint8_t *blob = e < A.E ? A.experts + (long long)e * A.bl.bytes : A.shared;
  auto row_at = [&](int q) {
    const int row = r0 + min(q, nr - 1);
    return Int4Row{blob + A.bl.dc + (size_t)row * (A.I / 2) + (lane & 3) * 8,
                   reinterpret_cast<const uint16_t *>(blob + A.bl.ds) + (size_t)row * G,
                   reinterpret_cast<const uint16_t *>(blob + A.bl.dm) + (size_t)row * G};
  };
  const uint8_t *col[NT], *sv[NT];
#pragma unroll
  for (int q = 0; q < NT; q++) {
    col[q] = D.op + (size_t)(at + min(8 * q + (lane >> 2), n - 1)) * D.pitch + (lane & 3) * 16;
    sv[q] = reinterpret_cast<const uint8_t *>(D.sv) + (at / 2 + min(4 * q + (lane & 3), (n - 1) / 2)) * 16;
  }
  Int4Acc<NT> acc;
  acc.clear();
  int4_rows<NT>(row_at(lane >> 2), row_at((lane >> 2) + 8), g0, g1, 0, col, sv, D.pairs * 16, acc);
#pragma unroll
  for (int q = 0; q < NT; q++)
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int tok = 8 * q + 2 * (lane & 3) + j;
      if (tok < n) {
        float *p = out + (size_t)(P.seg_at[seg] + tok) * 16 + (lane >> 2);
        p[0] = __uint_as_float((uint32_t)(acc.a[q] >> (32 * j)));
        p[8] = __uint_as_float((uint32_t)(acc.b[q] >> (32 * j)));
      }
    }
}

// Phase 3: this block's share of the output rows.
__device__ __forceinline__ void few_phase3(const FewArgs &A, const FewPlan &P, uint8_t *area, float *td) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = (int)((long long)A.d * blockIdx.x / gridDim.x), hi = (int)((long long)A.d * (blockIdx.x + 1) / gridDim.x);
  if (lo >= hi) return;
  const int G = A.I / 64, k1 = A.k + 1;
  float *out = reinterpret_cast<float *>(area);
  uint8_t *stage = area + A.parts_bytes;
  // t_d = A_d a_s of every token, 16 rows by 8 tokens a warp
  if (A.Ad) {
    const int rt = (A.r + 15) / 16, ntt = (A.T + 7) / 8;
    for (int u = warp; u < rt * ntt; u += kFewWarps) {
      const int q = u / ntt * 16, t0 = u % ntt * 8;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const uint16_t *ra = A.Ad + (size_t)min(q + (lane >> 2), A.r - 1) * A.I + (lane & 3) * 8;
      const uint16_t *rb = A.Ad + (size_t)min(q + (lane >> 2) + 8, A.r - 1) * A.I + (lane & 3) * 8;
      const uint16_t *x = A.a + ((size_t)min(t0 + (lane >> 2), A.T - 1) * k1 + A.k) * A.I + (lane & 3) * 8;
      bf16_rows(ra, rb, x, 0, A.I, acc);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int row = q + (lane >> 2) + 8 * (j >> 1), t = t0 + 2 * (lane & 3) + (j & 1);
        if (row < A.r && t < A.T) td[t * kMaxR + row] = acc[j];
      }
    }
  }
  for (int r0 = lo; r0 < hi; r0 += 16) {
    const int nr = min(16, hi - r0);
    // parts of K: more where there are few segments to keep the warps busy
    int parts = 1;
    while (parts < 4 && P.nseg * parts * 2 <= 2 * kFewWarps && 2 * parts <= G &&
           2 * parts * P.nplace * 64 <= A.parts_bytes)
      parts *= 2;
    for (int s0 = 0; s0 < P.nseg;) {
      int s1 = s0 + 1;
      while (s1 < P.nseg && P.seg_at[s1 + 1] - P.seg_at[s0] <= A.dn_rows) s1++;
      const int p0 = P.seg_at[s0], p1 = P.seg_at[s1];
      __syncthreads();
      const uint16_t *a = A.a;
      const int I = A.I;
      const ActDst D = few_stage(P, p0, p1, G, stage, [=](int asg) { return a + (size_t)asg * I; });
      __syncthreads();
      for (int u = warp; u < (s1 - s0) * parts; u += kFewWarps) {
        const int s = s0 + u / parts, part = u % parts, n = P.seg_n[s];
        float *o = out + (size_t)part * P.nplace * 16;
        const int g0 = G * part / parts, g1 = G * (part + 1) / parts;
        if (n <= 8)
          few_down<1>(A, P, D, p0, s, r0, nr, g0, g1, o);
        else if (n <= 16)
          few_down<2>(A, P, D, p0, s, r0, nr, g0, g1, o);
        else
          few_down<4>(A, P, D, p0, s, r0, nr, g0, g1, o);
      }
      s0 = s1;
    }
    __syncthreads();
    for (int o = tid; o < 16 * A.T; o += kFewThreads) {
      const int t = o / 16, q = o % 16, row = r0 + q;
      if (q >= nr) continue;
      float y = 0.f;
      for (int j = 0; j <= A.k; j++) {
        const float *p = out + (size_t)P.place[t * k1 + j] * 16 + q;
        float v = p[0];
        for (int w = 1; w < parts; w++) v += p[(size_t)w * P.nplace * 16];
        v *= kActUnit;
        y = j < A.k ? fmaf(P.gate[t * A.k + j], v, y) : y + v;
      }
      if (A.Ad) {
        float b = 0.f;
        for (int j = 0; j < A.r; j++) b = fmaf(bf(A.Bd[(size_t)row * A.r + j]), td[t * kMaxR + j], b);
        y = fmaf(A.c, b, y);
      }
      A.y[(size_t)t * A.d + row] = f2bf(y);
      if (A.yf) A.yf[(size_t)t * A.d + row] = y;
    }
  }
}

__global__ void __launch_bounds__(kFewThreads, 1) k_moe_few(FewArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  FewPlan &P = *reinterpret_cast<FewPlan *>(smem);
  uint8_t *red_area = smem + few_plan_bytes(), *area = red_area + kFewRedBytes;
  float *red = reinterpret_cast<float *>(red_area);
  cooperative_groups::grid_group grid = cooperative_groups::this_grid();
  few_phase1(A, P, area, red);
  grid.sync();
  if (A.h_out) few_residual(A);
  few_plan(A, P);
  few_phase2(A, P, area, red);
  grid.sync();
  few_phase3(A, P, area, red);
}

}  // namespace e0
