// norm.cu -- layer norm of irreps rows (include/cgtp.h: cgtp_norm_*).
//
// Every block of every row is normalised by itself.  Block of N values, c = 1
// for 0e blocks and 0 otherwise:
//   mu = c mean(x), r = (mean((x - mu)^2) + eps)^(-1/2), xh = r (x - mu)
//   y = xh w + b
// Backward, a = w g:   dx = r (a - c mean(a) - xh mean(a xh))
//   dw[u] = sum_rows sum_m g xh,  db[u] = sum_rows g
// Second order, J z = r (P z - xh mean(z xh)), P z = z - c mean(z), k = h_w g:
//   gg = w J h + h_w xh + h_b
//   gx = r^2 (xh (3 al be - ga) - be P a - al P h) + J k
//   gw[u] = sum_rows sum_m g J h
// with al = mean(a xh), be = mean(h xh), ga = mean(P h a).
//
// Split.  The unit of work is one block of one row.  A unit of up to 4 V values
// a thread stays in registers: a group of 1..T threads (a power of two, chosen
// per irreps block) loads it once, forms its sums by shuffles (and, above a
// warp, through shared memory), and writes the result, so every array moves once.
// A CTA works for one irreps block and walks over rows, so a thread keeps the
// same columns: the weights lie expanded to columns in shared memory, and the
// weights' gradients add up there in slots that only their thread touches;
// each CTA leaves one partial sum a channel, and a second launch adds these
// (no atomics; the order is fixed by n).  Blocks wider than 16,384 values take
// kernels that read a unit several times.
//
// Alignment.  Values move 16 bytes at a time.  Where a block's rows start
// anywhere (D, its offset or its length no multiple of 4), the rows of a CTA are
// P = 4 / gcd(D, 4) apart, so that all of them start at the same o = 0..3 floats
// behind a 16-byte border: value i of the unit is then value i + o of whole
// float4s, the same thread's in every row, and only the first and the last
// float4 are moved value by value.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <string>

#include "internal.hpp"

namespace cgtp {

namespace {

constexpr int kMaxBlocks = 32;

struct NormBlock {
  int off, len, d;  // first column, values, values per channel (2l+1)
  int ch, sc;       // first channel; first 0e channel, -1 for blocks that are not centred
};

struct NormTable {
  int D, nblocks, C, S;  // row width, blocks, channels, 0e channels
  float eps;
  NormBlock b[kMaxBlocks];
};

enum { kForward = 0, kBackward = 1, kDouble = 2 };

// Inputs and outputs of one call; bias is b (forward) or h_b (double).
struct NormArgs {
  const float *x, *w, *bias, *g, *hx, *hw;
  float *out, *out2;  // y | grad_x | gg, gx
};

// How one irreps block is worked on in a launch.
struct NormSeg {
  int off, len, d, ch, sc;
  unsigned magic;  // i / d = umulhi(i, magic); 0 for d = 1
  int tlog, vec;   // log2 of the group's threads; every row of it whole float4s
  int slots;       // float4s a thread has of a unit, at most
  int period;      // rows of a CTA are so many apart (1, 2 or 4)
  int cta0, ncta;  // its CTAs, a multiple of period: CTA c has the rows c mod period
  int fin0;        // its first CTA in the closing launch
  int64_t part;    // its partial sums: [ncta][mul] of the weight, then of the bias
};

struct NormPlan {
  int D, nseg;
  float eps;
  int direct;  // one CTA a block: no partial sums, the gradients are written at once
  NormSeg s[kMaxBlocks];
};

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ int channel_of(int i, unsigned magic) { return magic ? (int)__umulhi(i, magic) : i; }

// Barrier of group g of 2^TLOG threads (64 at least).  Immediate numbers: a
// number in a register would reserve all sixteen barriers for every CTA.
template <int TLOG>
__device__ __forceinline__ void group_barrier(int g) {
  switch (g) {
#define CGTP_GROUP(i) \
  case i: asm volatile("bar.sync %0, %1;" ::"n"(1 + i), "n"(1 << TLOG) : "memory"); break;
    CGTP_GROUP(0) CGTP_GROUP(1) CGTP_GROUP(2) CGTP_GROUP(3)
#undef CGTP_GROUP
  }
}

// Sums of K values over a group of 2^TLOG threads, the same bits in each of
// them.  Above a warp: the warps' sums through red (two buffers in turn, so
// that one barrier a call is enough), added by a butterfly of their own.
template <int TLOG, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float* red, int& turn) {
#pragma unroll
  for (int o = (TLOG < 5 ? TLOG : 5) - 1; o >= 0; --o)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], 1 << o);
  if constexpr (TLOG > 5) {
    constexpr int nw = 1 << (TLOG - 5);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = warp & ~(nw - 1);
    float* buf = red + turn;
    turn ^= 32 * 8;
    float4* mine = reinterpret_cast<float4*>(buf + warp * 8);
    if (lane == 0) {
      mine[0] = make_float4(v[0], v[K > 1 ? 1 : 0], v[K > 2 ? 2 : 0], v[K > 3 ? 3 : 0]);
      if constexpr (K > 4) mine[1].x = v[4];
    }
    group_barrier<TLOG>(warp >> (TLOG - 5));
    const float4* theirs = reinterpret_cast<const float4*>(buf + (w0 + (lane & (nw - 1))) * 8);
    const float4 t = theirs[0];
    v[0] = t.x;
    if constexpr (K > 1) v[1] = t.y;
    if constexpr (K > 2) v[2] = t.z;
    if constexpr (K > 3) v[3] = t.w;
    if constexpr (K > 4) v[4] = theirs[1].x;
#pragma unroll
    for (int o = TLOG - 6; o >= 0; --o)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], 1 << o);
  }
}

__device__ __forceinline__ void take4(float (&v)[4], const float4 t) {
  v[0] = t.x;
  v[1] = t.y;
  v[2] = t.z;
  v[3] = t.w;
}

// Four values at p: all of them where whole, else those in `some` (the others
// are 0).
template <bool SHIFT>
__device__ __forceinline__ void load4(const float* p, bool whole, unsigned some, float* v) {
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (whole) {
    t = __ldg(reinterpret_cast<const float4*>(p));
  } else if (SHIFT && some) {
    if (some & 1) t.x = __ldg(p);
    if (some & 2) t.y = __ldg(p + 1);
    if (some & 4) t.z = __ldg(p + 2);
    if (some & 8) t.w = __ldg(p + 3);
  }
  v[0] = t.x;
  v[1] = t.y;
  v[2] = t.z;
  v[3] = t.w;
}

template <bool SHIFT>
__device__ __forceinline__ void store4(float* p, bool whole, unsigned some, const float (&v)[4]) {
  if (whole) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (SHIFT && some) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (some >> j & 1) p[j] = v[j];
  }
}

__device__ __forceinline__ void add_to(float4& acc, const float4 v) {
  float4 t = acc;
  t.x += v.x;
  t.y += v.y;
  t.z += v.z;
  t.w += v.w;
  acc = t;
}

// The rows of one CTA.  Shared: w (and, by the operator, bias / h_w, h_b)
// expanded to columns; acc, acc2: the sums of the weight's and the bias's
// gradient, slot (q, thread).  CENTRED: a 0e block.
//
// Value j of a thread's slot q is value (q W + lane) 4 + j of the unit's
// float4s, which start o values before the unit.  Lanes without a slot hold
// zeros there and compute along, without branches: zeros add nothing to the
// sums (centred values are masked), and what they leave in acc is not read.
//
// The group's size W = 2^TLOG is a constant, so that a thread's slots are
// immediate offsets from one address an array: with W a variable the addresses
// and conditions were four fifths of the instructions (73 a value, now 33), and the
// backward was bound by their issue (Lmax 3 output: 93 us, now 74).
//
// What bounds it (B200, 6,144 rows of 256x0e+352x1o+384x2e+320x3o): the backward
// moves its 403 MB at 5.5 TB/s, 84 % of the measured copy rate, with 32 warps an
// SM; the forward of 768 rows of 52,864 columns 325 MB at 5.3 TB/s, 82 %; the
// double backward of 6,144 x 704 (in L2) 86 MB in 17.5 us, held by the latency that
// 16 warps an SM of 119 registers leave open (24 warps of 80 registers took 5 % more,
// 32 of 64 20 %, for their spills).  Few rows cost their launches: 2.5 us and 7 us.
// Rows that start anywhere, 6,143 x 5,456: forward 54 us, backward 84, double 203 (on
// 16-byte borders 52, 74, 134); with 32 values a thread the double backward spills (504
// bytes stored, 1,060 loaded): 768 rows of Lmax 6 312 us, on 16-byte borders 188.
template <int OP, int T, int V, bool SHIFT, bool CENTRED, int TLOG>
__device__ __forceinline__ void norm_rows(const NormSeg& s, int o, int D, float eps, int64_t n, const NormArgs& a,
                                          bool dw, bool db, const float4* sw, const float4* s2, const float4* s3,
                                          float4* acc, float4* acc2, float* red) {
  constexpr int W = 1 << TLOG, groups = T >> TLOG;
  const int lane = threadIdx.x & (W - 1);
  const int cta = blockIdx.x - s.cta0, period = SHIFT ? s.period : 1, cls = SHIFT ? cta % period : 0;
  const int len = s.len, slots = s.slots;
  unsigned valid = 0;  // SHIFT: bit 4 q + j: the value belongs to the unit
  if (SHIFT) {
#pragma unroll
    for (int e = 0; e < 4 * V; ++e) {
      const int i = ((e >> 2) * W + lane) * 4 + (e & 3) - o;
      valid |= (unsigned)(i >= 0 && i < len) << e;
    }
  }
  const int last = (len >> 2) - lane;  // not SHIFT: slot q exists where q W < last
  const int step = (SHIFT ? s.ncta / period : s.ncta) * groups;
  const int rows = (int)(SHIFT ? (n - cls + period - 1) / period : n);  // of this CTA's class
  const float inv = 1.f / (float)len;
  sw += lane;
  s2 += lane;
  s3 += lane;
  acc += threadIdx.x;
  acc2 += threadIdx.x;
  int turn = 0;
  int left = rows - (SHIFT ? cta / period : cta) * groups;  // rows from the CTA's first one on
  const int group = threadIdx.x >> TLOG;
  int64_t at = ((int64_t)(rows - left + group) * period + cls) * D + s.off - o + 4 * lane;
  const int64_t stride = (int64_t)step * period * D;
  for (; left > 0; left -= step, at += stride) {  // the same trips for every thread of the CTA
    const bool row = group < left;
    float x[4 * V], g[OP == kForward ? 1 : 4 * V], h[OP == kDouble ? 4 * V : 1];
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (q < slots) {
        const unsigned some = SHIFT && row ? valid >> (4 * q) & 15 : 0;
        const bool whole = SHIFT ? some == 15 : row && q * W < last;
        load4<SHIFT>(a.x + at + 4 * q * W, whole, some, x + 4 * q);
        if constexpr (OP != kForward) load4<SHIFT>(a.g + at + 4 * q * W, whole, some, g + 4 * q);
        if constexpr (OP == kDouble)
          load4<SHIFT>(a.hx + at + 4 * q * W, a.hx && whole, a.hx ? some : 0, h + 4 * q);
      }
    float mean = 0.f, ma = 0.f, mh = 0.f, mk = 0.f;
    if (CENTRED) {  // means of x, a = w g, h, k = h_w g
      constexpr int K = OP == kForward ? 1 : OP == kBackward ? 2 : 4;
      float t[K] = {};
#pragma unroll
      for (int q = 0; q < V; ++q)
        if (q < slots) {
          float w[4], k[4];
          if (OP != kForward) take4(w, sw[q * W]);
          if (OP == kDouble) take4(k, s2[q * W]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * q + j;
            t[0] += x[e];
            if constexpr (OP != kForward) t[1] = fmaf(g[e], w[j], t[1]);
            if constexpr (OP == kDouble) {
              t[2] += h[e];
              t[3] = fmaf(g[e], k[j], t[3]);
            }
          }
        }
      group_sum<TLOG>(t, red, turn);
      mean = t[0] * inv;
      if constexpr (OP != kForward) ma = t[1] * inv;
      if constexpr (OP == kDouble) {
        mh = t[2] * inv;
        mk = t[3] * inv;
      }
    }
    // sums of xc^2; a xc; h xc, k xc, P h a
    constexpr int K = OP == kForward ? 1 : OP == kBackward ? 2 : 5;
    float t[K] = {};
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (q < slots) {
        float w[4], k[4];
        if (OP != kForward) take4(w, sw[q * W]);
        if (OP == kDouble) take4(k, s2[q * W]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * q + j;
          const bool in = SHIFT ? valid >> e & 1 : q * W < last;
          if (CENTRED) x[e] = in ? x[e] - mean : 0.f;
          t[0] = fmaf(x[e], x[e], t[0]);
          if constexpr (OP == kBackward) t[1] = fmaf(g[e] * w[j], x[e], t[1]);
          if constexpr (OP == kDouble) {
            if (CENTRED) h[e] = in ? h[e] - mh : 0.f;
            const float aa = g[e] * w[j];
            t[1] = fmaf(aa, x[e], t[1]);
            t[2] = fmaf(h[e], x[e], t[2]);
            t[3] = fmaf(g[e] * k[j], x[e], t[3]);
            t[4] = fmaf(h[e], aa, t[4]);
          }
        }
      }
    group_sum<TLOG>(t, red, turn);
    const float r = rsqrtf(fmaf(t[0], inv, eps));
    // From here on by xc = xh / r: what projects on xh is sum(z xc) xc / (sum(xc^2) + N
    // eps), without the rounding of r twice.
    float along = 0.f, shift = 0.f, ph = 0.f, rb = 0.f, rl = 0.f, rc = 0.f;
    if constexpr (OP != kForward) {
      const float over = 1.f / fmaf((float)len, eps, t[0]);
      if constexpr (OP == kBackward) {  // grad_x = r (a - mean(a)) - (sum(a xc) over) xh; r^2 a may leave FP32
        along = -(t[1] * over);
        shift = -r * ma;
      }
      // gx = r (r (cx xh - be P a - al P h) + P k - de xh): only xh = r xc meets r once
      // more before the sum, since r^2 and r^3 leave FP32 where eps is small
      if constexpr (OP == kDouble) {
        const float al = t[1] * inv * r, be = t[2] * inv * r, ga = t[4] * inv;
        ph = -(t[2] * over);
        along = -(t[3] * over);
        rc = r * (3.f * al * be - ga);
        rb = -r * be;
        rl = -r * al;
        shift = -(rb * ma + mk);
      }
    }
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (q < slots) {
        const unsigned some = SHIFT && row ? valid >> (4 * q) & 15 : 0;
        const bool whole = SHIFT ? some == 15 : row && q * W < last;
        float w[4], y[4];
        take4(w, sw[q * W]);
        if constexpr (OP == kForward) {
          float b[4];
          if (CENTRED) take4(b, s2[q * W]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float xh = x[4 * q + j] * r;
            y[j] = CENTRED ? fmaf(xh, w[j], b[j]) : xh * w[j];
          }
          store4<SHIFT>(a.out + at + 4 * q * W, whole, some, y);
        } else if constexpr (OP == kBackward) {
          float p[4], gq[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * q + j;
            gq[j] = g[e];
            x[e] *= r;
            p[j] = g[e] * x[e];
            y[j] = fmaf(x[e], along, CENTRED ? fmaf(g[e], w[j] * r, shift) : g[e] * (w[j] * r));
          }
          if (a.out) store4<SHIFT>(a.out + at + 4 * q * W, whole, some, y);
          if (dw) add_to(acc[q * T], make_float4(p[0], p[1], p[2], p[3]));
          if (CENTRED && db) add_to(acc2[q * T], make_float4(gq[0], gq[1], gq[2], gq[3]));
        } else {
          float k[4], b[4], z[4], p[4];
          take4(k, s2[q * W]);
          if (CENTRED) take4(b, s3[q * W]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * q + j;
            const float xh = x[e] * r, jh = r * fmaf(ph, x[e], h[e]);
            y[j] = fmaf(w[j], jh, CENTRED ? fmaf(k[j], xh, b[j]) : k[j] * xh);
            const float c = fmaf(rb, w[j], k[j]);  // of g
            const float lin = fmaf(rl, h[e], fmaf(x[e], along, CENTRED ? fmaf(xh, rc, shift) : xh * rc));
            z[j] = r * fmaf(c, g[e], lin);
            p[j] = g[e] * jh;
          }
          if (a.out) store4<SHIFT>(a.out + at + 4 * q * W, whole, some, y);
          if (a.out2) store4<SHIFT>(a.out2 + at + 4 * q * W, whole, some, z);
          if (dw) add_to(acc[q * T], make_float4(p[0], p[1], p[2], p[3]));
        }
      }
  }
}

// The group sizes that are built: 4, 16, 32, 64, 128 and 256 threads for CTAs
// of 256 (16 values a thread), 4, 32, 128 and 512 for CTAs of 512 (32 values).
__host__ __device__ constexpr bool width_built(int tlog, int T) {
  return T == 256 ? tlog == 2 || (tlog >= 4 && tlog <= 8) : tlog == 2 || tlog == 5 || tlog == 7 || tlog == 9;
}

template <int OP, int T, int V, bool SHIFT, int TLOG = 2, class... Rest>
__device__ __forceinline__ void norm_width(const NormSeg& s, Rest... rest) {
  if (s.tlog == TLOG) {
    if constexpr (width_built(TLOG, T)) {
      if (s.sc >= 0)
        norm_rows<OP, T, V, SHIFT, true, TLOG>(s, rest...);
      else
        norm_rows<OP, T, V, SHIFT, false, TLOG>(s, rest...);
    }
  } else if constexpr ((2 << TLOG) <= T) {
    norm_width<OP, T, V, SHIFT, TLOG + 1>(s, rest...);
  }
}

// Shared floats of one CTA: the expanded parameters of a block of `len` values
// (each padded to whole slots of its group), the accumulators, the sums.
constexpr int kRed = 2 * 32 * 8;
__host__ __device__ constexpr int expanded_arrays(int op, bool centred) {
  return 1 + (op == kForward && centred) + (op == kDouble) + (op == kDouble && centred);
}
__host__ __device__ inline int expanded(int len, int tlog, int vec) {
  const int slot = 4 << tlog;  // a group's values of one slot
  return (len + (vec ? 0 : 3) + slot - 1) / slot * slot;
}

// SHIFT: some block's rows start or end inside a float4.
template <int OP, int T, int V, bool SHIFT, int MIN>
__global__ void __launch_bounds__(T, MIN) norm_kernel(const __grid_constant__ NormPlan p, int64_t n,
                                                      const __grid_constant__ NormArgs a, float* __restrict__ part,
                                                      float* __restrict__ dw, float* __restrict__ db) {
  grid_dependency_wait();
  grid_launch_dependents();
  extern __shared__ float4 smem4[];
  float* smem = reinterpret_cast<float*>(smem4);
  int q = 0;
  while (q + 1 < p.nseg && (int)blockIdx.x >= p.s[q + 1].cta0) ++q;
  const NormSeg s = p.s[q];
  const int size = expanded(s.len, s.tlog, s.vec);
  // floats from a 16-byte border to this CTA's units (every array starts on one)
  const int o = SHIFT ? (int)(((int64_t)((blockIdx.x - s.cta0) % s.period) * p.D + s.off) & 3) : 0;
  float* sw = smem;
  const bool centred = s.sc >= 0;
  float* s2 = sw + size;  // forward: bias of a centred block; double: h_w
  float* s3 = s2 + size;  // double: h_b of a centred block
  float4* acc = reinterpret_cast<float4*>(smem + expanded_arrays(OP, centred) * size);
  const bool want_w = OP != kForward && dw, want_b = OP == kBackward && db && centred;
  float4* acc2 = acc + (want_w ? T * V : 0);
  float* red = reinterpret_cast<float*>(acc2 + (want_b ? T * V : 0));
  for (int i = threadIdx.x; i < size; i += T) {
    const bool in = i >= o && i < o + s.len;
    const int c = in ? channel_of(i - o, s.magic) : 0;
    sw[i] = !in ? 0.f : a.w ? __ldg(a.w + s.ch + c) : 1.f;
    if (OP == kForward && centred) s2[i] = in && a.bias ? __ldg(a.bias + s.sc + c) : 0.f;
    if (OP == kDouble) s2[i] = in && a.hw ? __ldg(a.hw + s.ch + c) : 0.f;
    if (OP == kDouble && centred) s3[i] = in && a.bias ? __ldg(a.bias + s.sc + c) : 0.f;
  }
  if (OP != kForward) {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = threadIdx.x; i < (want_w ? T * V : 0) + (want_b ? T * V : 0); i += T) acc[i] = zero;
  }
  __syncthreads();
  const float4 *sw4 = smem4, *s24 = sw4 + size / 4, *s34 = s24 + size / 4;
  norm_width<OP, T, V, SHIFT>(s, o, p.D, p.eps, n, a, want_w, want_b, sw4, s24, s34, acc, acc2, red);
  if (OP == kForward || (!want_w && !want_b)) return;
  // this CTA's sums: over its groups, halving them, then over a channel's components
  const int mul = s.len / s.d, width = 1 << s.tlog, cta = blockIdx.x - s.cta0;
  for (int h = T / 2; h >= width; h >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < h)
      for (int k = 0; k < s.slots; ++k) {
        if (want_w) add_to(acc[k * T + threadIdx.x], acc[k * T + threadIdx.x + h]);
        if (want_b) add_to(acc2[k * T + threadIdx.x], acc2[k * T + threadIdx.x + h]);
      }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < mul; c += T) {
    float v = 0.f, b = 0.f;
    for (int k = 0; k < s.d; ++k) {
      const int i = c * s.d + k + o;
      const int at = ((i >> 2 >> s.tlog) * T + ((i >> 2) & (width - 1))) * 4 + (i & 3);
      if (want_w) v += reinterpret_cast<float*>(acc)[at];
      if (want_b) b += reinterpret_cast<float*>(acc2)[at];
    }
    if (p.direct) {
      if (want_w) dw[s.ch + c] = v;
      if (want_b) db[s.sc + c] = b;
    } else {
      if (want_w) part[s.part + (int64_t)cta * mul + c] = v;
      if (want_b) part[s.part + (int64_t)(s.ncta + cta) * mul + c] = b;
    }
  }
}

// The closing sums: a CTA takes 32 channels of one block; its warps share the
// CTAs' partial sums, eight loads in flight each, which are then added in warp
// order.
constexpr int kFinish = 1024;

__global__ void __launch_bounds__(kFinish) norm_finish_kernel(const __grid_constant__ NormPlan p,
                                                              const float* __restrict__ part, float* __restrict__ dw,
                                                              float* __restrict__ db) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kWarps = kFinish / 32;
  int q = 0;
  while (q + 1 < p.nseg && (int)blockIdx.x >= p.s[q + 1].fin0) ++q;
  const NormSeg s = p.s[q];
  const int mul = s.len / s.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = (mul + 31) / 32, tile = blockIdx.x - s.fin0;
  const bool bias = tile >= tiles;
  const int c = (bias ? tile - tiles : tile) * 32 + lane;
  float* out = bias ? (db ? db + s.sc : nullptr) : (dw ? dw + s.ch : nullptr);
  if (!out) return;
  float v = 0.f;
  if (c < mul) {
    const float* src = part + s.part + (bias ? (int64_t)s.ncta * mul : 0) + c;
    for (int k0 = warp; k0 < s.ncta; k0 += 8 * kWarps) {
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = k0 + j * kWarps;
        t[j] = k < s.ncta ? src[(int64_t)k * mul] : 0.f;
      }
      v += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
    }
  }
  __shared__ float sums[kWarps][33];
  sums[warp][lane] = v;
  __syncthreads();
  // warp w adds the partial sums of channel w
  v = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int mine = (bias ? tile - tiles : tile) * 32 + warp;
  if (lane == 0 && mine < mul) out[mine] = v;
}

// ---- blocks wider than the registers of a CTA: one CTA a unit, several reads, and one
// CTA a channel for the weights, which reads columns.  768 rows of 40000x0e (123 MB an
// array), us: forward 154, backward 569, double backward 893: 4, 10 and 9.5 times what the bytes take

constexpr int kWide = 256;

__device__ __forceinline__ float cta_sum(float v, float* red, int& turn) {
  float t[1] = {v};
  group_sum<8>(t, red, turn);
  return t[0];
}

// mean (0 unless centred) and 1 / sqrt(variance + eps) of one block
__device__ __forceinline__ void block_stats(const float* x, const NormBlock& b, float eps, float* red, int& turn,
                                            float* mu, float* r) {
  const float inv = 1.f / (float)b.len;
  float m = 0.f;
  if (b.sc >= 0) {
    for (int i = threadIdx.x; i < b.len; i += kWide) m += x[i];
    m = cta_sum(m, red, turn) * inv;
  }
  float v = 0.f;
  for (int i = threadIdx.x; i < b.len; i += kWide) {
    const float t = x[i] - m;
    v = fmaf(t, t, v);
  }
  *mu = m;
  *r = 1.f / sqrtf(cta_sum(v, red, turn) * inv + eps);
}

__global__ void __launch_bounds__(kWide) wide_forward_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                             const float* __restrict__ x, const float* __restrict__ w,
                                                             const float* __restrict__ bias, float* __restrict__ y) {
  __shared__ float red[kRed];
  int turn = 0;
  for (int64_t u = blockIdx.x; u < n * t.nblocks; u += gridDim.x) {
    const NormBlock b = t.b[u % t.nblocks];
    const int64_t at = u / t.nblocks * t.D + b.off;
    float mu, r;
    block_stats(x + at, b, t.eps, red, turn, &mu, &r);
    for (int i = threadIdx.x; i < b.len; i += kWide) {
      const int c = i / b.d;
      const float v = (x[at + i] - mu) * r * (w ? w[b.ch + c] : 1.f);
      y[at + i] = b.sc >= 0 && bias ? v + bias[b.sc + c] : v;
    }
  }
}

// stats[u] = (mu, r, mean(h) if centred, mean(h xh)) of unit u = row * nblocks + block
__global__ void __launch_bounds__(kWide) wide_backward_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                              const float* __restrict__ x, const float* __restrict__ w,
                                                              const float* __restrict__ g, float* __restrict__ dx,
                                                              float4* __restrict__ stats) {
  __shared__ float red[kRed];
  int turn = 0;
  for (int64_t u = blockIdx.x; u < n * t.nblocks; u += gridDim.x) {
    const NormBlock b = t.b[u % t.nblocks];
    const int64_t at = u / t.nblocks * t.D + b.off;
    float mu, r;
    block_stats(x + at, b, t.eps, red, turn, &mu, &r);
    if (threadIdx.x == 0 && stats) stats[u] = make_float4(mu, r, 0.f, 0.f);
    if (!dx) continue;
    float sa = 0.f, sax = 0.f;
    for (int i = threadIdx.x; i < b.len; i += kWide) {
      const float a = g[at + i] * (w ? w[b.ch + i / b.d] : 1.f);
      sa += a;
      sax = fmaf(a, (x[at + i] - mu) * r, sax);
    }
    const float inv = 1.f / (float)b.len;
    const float ma = b.sc >= 0 ? cta_sum(sa, red, turn) * inv : 0.f;
    const float al = cta_sum(sax, red, turn) * inv;
    for (int i = threadIdx.x; i < b.len; i += kWide) {
      const float a = g[at + i] * (w ? w[b.ch + i / b.d] : 1.f);
      dx[at + i] = r * (a - ma - (x[at + i] - mu) * r * al);
    }
  }
}

__global__ void __launch_bounds__(kWide) wide_double_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                            const float* __restrict__ x, const float* __restrict__ w,
                                                            const float* __restrict__ g, const float* __restrict__ hx,
                                                            const float* __restrict__ hw, const float* __restrict__ hb,
                                                            float* __restrict__ gg, float* __restrict__ gx,
                                                            float4* __restrict__ stats) {
  __shared__ float red[kRed];
  int turn = 0;
  for (int64_t u = blockIdx.x; u < n * t.nblocks; u += gridDim.x) {
    const NormBlock b = t.b[u % t.nblocks];
    const int64_t at = u / t.nblocks * t.D + b.off;
    const float inv = 1.f / (float)b.len;
    float mu, r;
    block_stats(x + at, b, t.eps, red, turn, &mu, &r);
    float sa = 0.f, sh = 0.f, sk = 0.f;
    if (b.sc >= 0) {
      for (int i = threadIdx.x; i < b.len; i += kWide) {
        const int c = b.ch + i / b.d;
        sa = fmaf(g[at + i], w ? w[c] : 1.f, sa);
        if (hx) sh += hx[at + i];
        if (hw) sk = fmaf(g[at + i], hw[c], sk);
      }
      sa = cta_sum(sa, red, turn) * inv;
      sh = cta_sum(sh, red, turn) * inv;
      sk = cta_sum(sk, red, turn) * inv;
    }
    float sax = 0.f, shx = 0.f, skx = 0.f, sha = 0.f;
    for (int i = threadIdx.x; i < b.len; i += kWide) {
      const int c = b.ch + i / b.d;
      const float xh = (x[at + i] - mu) * r, gi = g[at + i];
      const float a = gi * (w ? w[c] : 1.f), h = hx ? hx[at + i] - sh : 0.f;
      sax = fmaf(a, xh, sax);
      shx = fmaf(h, xh, shx);
      sha = fmaf(h, a, sha);
      if (hw) skx = fmaf(gi * hw[c], xh, skx);
    }
    const float al = cta_sum(sax, red, turn) * inv, be = cta_sum(shx, red, turn) * inv,
                ga = cta_sum(sha, red, turn) * inv, de = cta_sum(skx, red, turn) * inv;
    if (threadIdx.x == 0 && stats) stats[u] = make_float4(mu, r, sh, be);
    const float cx = 3.f * al * be - ga;
    for (int i = threadIdx.x; i < b.len; i += kWide) {
      const int c = b.ch + i / b.d;
      const float xh = (x[at + i] - mu) * r, gi = g[at + i], wi = w ? w[c] : 1.f, hwi = hw ? hw[c] : 0.f;
      const float h = hx ? hx[at + i] - sh : 0.f;
      if (gg) {
        float v = fmaf(hwi, xh, wi * r * (h - xh * be));
        if (b.sc >= 0 && hb) v += hb[b.sc + i / b.d];
        gg[at + i] = v;
      }
      if (gx)
        gx[at + i] = r * (r * (xh * cx - be * (gi * wi - sa) - al * h) + (gi * hwi - sk - xh * de));
    }
  }
}

// One CTA per channel: the sums over rows and components of g xh or g J h, and
// of g for 0e channels.  stats as written above.
__global__ void __launch_bounds__(kWide) wide_weight_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                            const float* __restrict__ x, const float* __restrict__ g,
                                                            const float* __restrict__ hx, bool second,
                                                            const float4* __restrict__ stats, float* __restrict__ dw,
                                                            float* __restrict__ db) {
  __shared__ float red[kRed];
  int turn = 0;
  const int ch = blockIdx.x;
  int q = 0;
  while (q + 1 < t.nblocks && t.b[q + 1].ch <= ch) ++q;
  const NormBlock b = t.b[q];
  const int c = ch - b.ch;
  float sw = 0.f, sb = 0.f;
  for (int64_t i = threadIdx.x; i < n * b.d; i += kWide) {
    const int64_t row = i / b.d, at = row * t.D + b.off + c * b.d + (i - row * b.d);
    const float4 s = stats[row * t.nblocks + q];
    const float xh = (x[at] - s.x) * s.y;
    const float v = second ? (hx ? s.y * (hx[at] - s.z - xh * s.w) : 0.f) : xh;
    sw = fmaf(g[at], v, sw);
    sb += g[at];
  }
  sw = cta_sum(sw, red, turn);
  sb = cta_sum(sb, red, turn);
  if (threadIdx.x == 0) {
    if (dw) dw[ch] = sw;
    if (db && b.sc >= 0) db[b.sc + c] = sb;
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

cgtp_status norm_checks(cgtp_norm norm, int64_t n) {
  if (!norm) return fail(CGTP_ERR_NULL, "norm is NULL");
  if (n < 0 || n >= (int64_t(1) << 31)) return fail(CGTP_ERR_SIZE, "n out of range");
  return CGTP_OK;
}

cgtp_status norm_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned16(p)) return fail(CGTP_ERR_ALIGN, "float arrays must be 16-byte aligned");
  return CGTP_OK;
}

constexpr int kSms = 148;
constexpr int kNarrow = 4096;    // values a group of 256 threads holds, 16 a thread
constexpr int kMiddle = 16384;   // values a group of 512 threads holds, 32 a thread
constexpr size_t kMaxShared = 227 * 1024;
constexpr int64_t kDirectTrips = 4;

bool whole(const NormTable& t, const NormBlock& b) { return t.D % 4 == 0 && b.off % 4 == 0 && b.len % 4 == 0; }

// Does every block fit `most` values, wherever its rows start?
bool fits(const NormTable& t, int most) {
  for (int q = 0; q < t.nblocks; ++q)
    if (t.b[q].len + (whole(t, t.b[q]) ? 0 : 3) > most) return false;
  return true;
}

bool any_shift(const NormTable& t) {
  for (int q = 0; q < t.nblocks; ++q)
    if (!whole(t, t.b[q])) return true;
  return false;
}

// Resident CTAs an SM, by registers (the launch bounds below).
constexpr int resident(int op, bool narrow, bool shift) {
  return narrow ? (op == kForward ? 4 : op == kBackward ? (shift ? 3 : 4) : 2) : (op == kForward ? (shift ? 1 : 2) : 1);
}

// The division of n rows among the CTAs; *floats: the partial sums' size,
// *shared: bytes of shared memory.  False where some block does not fit a
// CTA's registers or shared memory (the kernels for wide blocks run then).
//
// One wave of CTAs.  A CTA's trip over one row a group costs about its threads' slots
// and two slots' time more for the sums, so the blocks' CTAs are chosen for the
// smallest bound on trips x cost that one wave meets.
bool norm_plan(const NormTable& t, int op, int64_t n, NormPlan& p, int64_t* floats, size_t* shared) {
  if (!fits(t, kMiddle)) return false;
  const bool narrow = fits(t, kNarrow), shift = any_shift(t);
  const int T = narrow ? 256 : 512, V = narrow ? 4 : 8;
  p.D = t.D;
  p.nseg = t.nblocks;
  p.eps = t.eps;
  int64_t trips[kMaxBlocks];  // of a class of rows, by one CTA
  int cost[kMaxBlocks];
  int64_t work = 0, longest = 1;
  for (int q = 0; q < t.nblocks; ++q) {
    const NormBlock& b = t.b[q];
    NormSeg& s = p.s[q];
    s.off = b.off;
    s.len = b.len;
    s.d = b.d;
    s.ch = b.ch;
    s.sc = b.sc;
    s.magic = b.d == 1 ? 0u : (unsigned)((uint64_t(1) << 32) / b.d + 1);
    s.vec = whole(t, b);
    s.period = t.D % 4 == 0 ? 1 : t.D % 2 == 0 ? 2 : 4;
    const int values = b.len + (s.vec ? 0 : 3);
    s.tlog = 0;
    while (!width_built(s.tlog, T) || (4 * V << s.tlog) < values) ++s.tlog;
    s.slots = (values + (4 << s.tlog) - 1) >> (2 + s.tlog);
    const int64_t groups = T >> s.tlog, rows = (n + s.period - 1) / s.period;
    trips[q] = (rows + groups - 1) / groups;
    cost[q] = s.slots + 2;
    work += trips[q] * s.period * cost[q];
    longest = std::max(longest, trips[q]);
  }
  const int64_t target = kSms * resident(op, narrow, shift);
  // few rows: one CTA a block writes the gradients itself, without a second launch
  p.direct = op != kForward && longest <= kDirectTrips && t.D % 4 == 0;
  for (int64_t bound = std::max<int64_t>(work / target, 1);; bound += bound / 16 + 1) {
    int64_t total = 0;
    for (int q = 0; q < t.nblocks; ++q) {
      const int64_t each = std::max<int64_t>(bound / cost[q], 1);
      p.s[q].ncta = p.direct ? 1 : (int)(p.s[q].period * std::min<int64_t>((trips[q] + each - 1) / each, target));
      total += p.s[q].ncta;
    }
    if (total <= target || bound >= longest * (V + 2)) break;
  }
  int cta = 0, fin = 0;
  int64_t part = 0;
  size_t most = 0;
  for (int q = 0; q < t.nblocks; ++q) {
    NormSeg& s = p.s[q];
    const bool two = op == kBackward && s.sc >= 0;
    const int mul = s.len / s.d;
    s.cta0 = cta;
    cta += s.ncta;
    s.fin0 = fin;
    fin += (mul + 31) / 32 * (two ? 2 : 1);
    s.part = part;
    part += (int64_t)s.ncta * mul * (two ? 2 : 1);
    size_t here = (size_t)expanded_arrays(op, s.sc >= 0) * expanded(s.len, s.tlog, s.vec) + kRed;
    if (op != kForward) here += (size_t)4 * T * V * (two ? 2 : 1);
    most = std::max(most, here * sizeof(float));
  }
  *floats = part;
  *shared = most;
  return most <= kMaxShared;
}

size_t norm_workspace(const NormTable& t, int64_t n) {
  int64_t bytes = 0, floats;
  size_t shared;
  NormPlan p;
  for (int op : {kBackward, kDouble})
    bytes = std::max(bytes, norm_plan(t, op, n, p, &floats, &shared) ? floats * (int64_t)sizeof(float)
                                                                     : n * t.nblocks * (int64_t)sizeof(float4));
  return ((size_t)bytes + 255) & ~size_t(255);
}

cgtp_status norm_workspace_check(const NormTable& t, int64_t n, const void* ws, size_t bytes) {
  const size_t need = norm_workspace(t, n);
  if (!ws || bytes < need) return fail(CGTP_ERR_WORKSPACE, "workspace of " + std::to_string(need) + " bytes required");
  if ((uintptr_t)ws & 255) return fail(CGTP_ERR_ALIGN, "workspace must be 256-byte aligned");
  return CGTP_OK;
}

template <class... KArgs, class... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t shared, cudaStream_t s,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <int OP, int T, int V, bool SHIFT, int MIN>
cudaError_t launch_rows(const NormPlan& p, int64_t n, const NormArgs& a, size_t shared, float* dw, float* db,
                        float* part, cudaStream_t s) {
  auto kernel = norm_kernel<OP, T, V, SHIFT, MIN>;
  if (shared > 48 * 1024) {
    // always the same value: threads with other sizes do not undo it
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxShared);
    if (e != cudaSuccess) return e;
  }
  const NormSeg& last = p.s[p.nseg - 1];
  return launch_dependent(kernel, (unsigned)(last.cta0 + last.ncta), T, shared, s, p, n, a, part, dw, db);
}

template <int OP>
cudaError_t launch_norm(const NormTable& t, int64_t n, const NormArgs& a, float* dw, float* db, void* workspace,
                        cudaStream_t s) {
  NormPlan p;
  int64_t floats;
  size_t shared;
  if (!norm_plan(t, OP, n, p, &floats, &shared)) {
    float4* stats = (float4*)workspace;
    const unsigned grid = (unsigned)std::min<int64_t>(n * t.nblocks, kSms * 8);
    if (OP == kForward) wide_forward_kernel<<<grid, kWide, 0, s>>>(t, n, a.x, a.w, a.bias, a.out);
    if (OP == kBackward) wide_backward_kernel<<<grid, kWide, 0, s>>>(t, n, a.x, a.w, a.g, a.out, stats);
    if (OP == kDouble)
      wide_double_kernel<<<grid, kWide, 0, s>>>(t, n, a.x, a.w, a.g, a.hx, a.hw, a.bias, a.out, a.out2, stats);
    if (stats)
      wide_weight_kernel<<<(unsigned)t.C, kWide, 0, s>>>(t, n, a.x, a.g, a.hx, OP == kDouble, stats, dw, db);
    return cudaGetLastError();
  }
  float* part = (float*)workspace;
  const bool narrow = fits(t, kNarrow), shift = any_shift(t);
  auto rows = narrow ? (shift ? launch_rows<OP, 256, 4, true, resident(OP, true, true)>
                              : launch_rows<OP, 256, 4, false, resident(OP, true, false)>)
                     : (shift ? launch_rows<OP, 512, 8, true, resident(OP, false, true)>
                              : launch_rows<OP, 512, 8, false, resident(OP, false, false)>);
  const cudaError_t e = rows(p, n, a, shared, dw, db, part, s);
  if (e != cudaSuccess || (!dw && !db) || p.direct) return e;
  int fin = 0;
  for (int q = 0; q < t.nblocks; ++q)
    fin += (t.b[q].len / t.b[q].d + 31) / 32 * (OP == kBackward && t.b[q].sc >= 0 ? 2 : 1);
  return launch_dependent(norm_finish_kernel, (unsigned)fin, kFinish, 0, s, p, (const float*)part, dw, db);
}

}  // namespace

}  // namespace cgtp

struct cgtp_norm_s {
  cgtp::NormTable t;
};

using namespace cgtp;

extern "C" {

cgtp_status cgtp_norm_create(const char* irreps, double eps, cgtp_norm* out) {
  if (!out) return fail(CGTP_ERR_NULL, "out is NULL");
  *out = nullptr;
  if (!irreps) return fail(CGTP_ERR_NULL, "irreps string is NULL");
  try {
    std::vector<Irrep> v;
    std::string err;
    if (!parse_irreps(irreps, v, err)) return fail(CGTP_ERR_IRREPS_PARSE, err);
    // a normal float: the backward divides by the sum of squares plus N eps
    if (!((float)eps >= FLT_MIN) || !std::isfinite((float)eps))
      return fail(CGTP_ERR_SIZE, "eps must be a positive normal FP32 number");
    if (v.size() > kMaxBlocks) return fail(CGTP_ERR_SIZE, "more than 32 irreps blocks");
    NormTable t;
    std::memset(&t, 0, sizeof t);
    t.eps = (float)eps;
    int64_t off = 0;
    for (const Irrep& ir : v) {
      if (ir.mul <= 0) return fail(CGTP_ERR_IRREPS_PARSE, "multiplicities must be positive");
      if (ir.l > 6) return fail(CGTP_ERR_LMAX, "an irrep degree exceeds 6");
      NormBlock& b = t.b[t.nblocks++];
      const bool scalar = ir.l == 0 && ir.parity > 0;
      b.off = (int)off;
      b.d = 2 * ir.l + 1;
      b.len = ir.mul * b.d;
      b.ch = t.C;
      b.sc = scalar ? t.S : -1;
      t.C += ir.mul;
      if (scalar) t.S += ir.mul;
      off += b.len;
      if (off >= (1 << 30)) return fail(CGTP_ERR_SIZE, "irreps too wide");
    }
    t.D = (int)off;
    auto h = std::make_unique<cgtp_norm_s>();
    h->t = t;
    *out = h.release();
  } catch (const std::exception& e) {
    return fail(CGTP_ERR_OOM, std::string("exception in norm create: ") + e.what());
  }
  return CGTP_OK;
}

cgtp_status cgtp_norm_destroy(cgtp_norm norm) {
  delete norm;
  return CGTP_OK;
}

cgtp_status cgtp_norm_info(cgtp_norm norm, int64_t* d, int64_t* n_weight, int64_t* n_bias) {
  if (!norm) return fail(CGTP_ERR_NULL, "norm is NULL");
  if (d) *d = norm->t.D;
  if (n_weight) *n_weight = norm->t.C;
  if (n_bias) *n_bias = norm->t.S;
  return CGTP_OK;
}

cgtp_status cgtp_norm_forward(cgtp_norm norm, int64_t n, const float* x, const float* weight, const float* bias,
                              float* y, cgtp_stream stream) {
  NvtxRange nvtx_range("cgtp_norm_forward");
  cgtp_status st = norm_checks(norm, n);
  if (st != CGTP_OK) return st;
  if (n == 0) return CGTP_OK;
  if (!x || !y) return fail(CGTP_ERR_NULL, "x or y is NULL");
  if ((st = norm_aligned({x, weight, bias, y})) != CGTP_OK) return st;
  CGTP_CUDA_TRY(launch_norm<kForward>(norm->t, n, {x, weight, bias, nullptr, nullptr, nullptr, y, nullptr},
                                      nullptr, nullptr, nullptr, (cudaStream_t)stream));
  return CGTP_OK;
}

cgtp_status cgtp_norm_workspace_size(cgtp_norm norm, int64_t n, size_t* bytes) {
  cgtp_status st = norm_checks(norm, n);
  if (st != CGTP_OK) return st;
  if (!bytes) return fail(CGTP_ERR_NULL, "bytes is NULL");
  *bytes = norm_workspace(norm->t, n);
  return CGTP_OK;
}

cgtp_status cgtp_norm_backward(cgtp_norm norm, int64_t n, const float* x, const float* weight, const float* grad_y,
                               float* grad_x, float* grad_weight, float* grad_bias, void* workspace,
                               size_t workspace_bytes, cgtp_stream stream) {
  NvtxRange nvtx_range("cgtp_norm_backward");
  cgtp_status st = norm_checks(norm, n);
  if (st != CGTP_OK) return st;
  const NormTable& t = norm->t;
  cudaStream_t s = (cudaStream_t)stream;
  if (n > 0 && (!x || !grad_y)) return fail(CGTP_ERR_NULL, "x or grad_y is NULL");
  if ((st = norm_aligned({x, weight, grad_y, grad_x, grad_weight, grad_bias})) != CGTP_OK) return st;
  if (t.S == 0) grad_bias = nullptr;
  const bool params = grad_weight || grad_bias;
  if (n == 0) {
    if (grad_weight) CGTP_CUDA_TRY(cudaMemsetAsync(grad_weight, 0, (size_t)t.C * 4, s));
    if (grad_bias) CGTP_CUDA_TRY(cudaMemsetAsync(grad_bias, 0, (size_t)t.S * 4, s));
    return CGTP_OK;
  }
  if (!params && !grad_x) return CGTP_OK;
  if (params && (st = norm_workspace_check(t, n, workspace, workspace_bytes)) != CGTP_OK) return st;
  CGTP_CUDA_TRY(launch_norm<kBackward>(t, n, {x, weight, nullptr, grad_y, nullptr, nullptr, grad_x, nullptr},
                                       grad_weight, grad_bias, params ? workspace : nullptr, s));
  return CGTP_OK;
}

cgtp_status cgtp_norm_double_backward(cgtp_norm norm, int64_t n, const float* x, const float* weight,
                                      const float* grad_y, const float* h_x, const float* h_weight,
                                      const float* h_bias, float* gg, float* gx, float* gweight, void* workspace,
                                      size_t workspace_bytes, cgtp_stream stream) {
  NvtxRange nvtx_range("cgtp_norm_double_backward");
  cgtp_status st = norm_checks(norm, n);
  if (st != CGTP_OK) return st;
  const NormTable& t = norm->t;
  cudaStream_t s = (cudaStream_t)stream;
  if (n > 0 && (!x || !grad_y)) return fail(CGTP_ERR_NULL, "x or grad_y is NULL");
  if ((st = norm_aligned({x, weight, grad_y, h_x, h_weight, h_bias, gg, gx, gweight})) != CGTP_OK) return st;
  if (n == 0) {
    if (gweight) CGTP_CUDA_TRY(cudaMemsetAsync(gweight, 0, (size_t)t.C * 4, s));
    return CGTP_OK;
  }
  if (!gg && !gx && !gweight) return CGTP_OK;
  if (gweight && (st = norm_workspace_check(t, n, workspace, workspace_bytes)) != CGTP_OK) return st;
  CGTP_CUDA_TRY(launch_norm<kDouble>(t, n, {x, weight, h_bias, grad_y, h_x, h_weight, gg, gx}, gweight, nullptr,
                                     gweight ? workspace : nullptr, s));
  return CGTP_OK;
}

}  // extern "C"
