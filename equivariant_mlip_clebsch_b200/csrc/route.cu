// route.cu -- routing of edges to experts (include/cgtp.h: cgtp_router_*).
//
// A row's logits l over n experts give scores s = softmax(l) or sigmoid(l); v =
// s + bias is compared, within the best groups, and the k best experts get the
// weights scale s_j (over the chosen ones' sum, if renormalised).
//
// The choice has to be that of 64 bits: scores next to one another differ by
// less than FP32's rounding.  A row is decided in FP32 (by a thread where rows are
// many, else by a warp) as far as its error bound lets it; the rest is decided by a
// warp in 64 bits.  That rest is rare where scores or biases are spread (60 of 172,050
// rows of 64 experts in 8 groups, sigmoid, random biases).  It is not where a row's
// scores next to the cut are all small, since the bound does not shrink with them, or
// equal: 172,050 x 64, softmax in 8 groups without a bias, normal logits of deviation
// 1.5 63 us, of 5 139 us, of 10 453 us, all equal 638 us.
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <algorithm>
#include <memory>
#include <string>

#include "internal.hpp"

namespace cgtp {

namespace {

constexpr int kMaxExperts = 512, kMaxGroups = 32, kMaxK = 32;
constexpr unsigned kAll = 0xffffffffu;

struct RouteSpec {
  int n, k, sigmoid, groups, top_groups, group_best, renormalise;
  float scale;
};

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The hardware's 2^x and 1 / x (2 ulp and 1 ulp), subnormals as zero: without
// the steps around them that keep subnormals.
__device__ __forceinline__ float quick_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float quick_sigmoid(float l) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + quick_exp(-l)));
  return y;
}

template <class X>
__device__ __forceinline__ X warp_sum(X v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ bool there(float l) { return l > -FLT_MAX; }

__device__ __forceinline__ int ordered(float v) {  // an integer in the order of the values
  const int i = __float_as_int(v);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// One row by one warp with every compared value in 64 bits, v [n] in shared
// memory of the warp's own.  Lane j returns the j-th choice and its weight (-1 and
// 0 where nothing is left).
//
// It runs for few rows, each at the end of a CTA that others wait for, and what
// it costs there is the fetch of its instructions: so it is one function of loops
// that are not unrolled (inlined and unrolled, the 60 such rows of 172,050 took 16
// of the 68 us of the whole forward).
__device__ __noinline__ double exp_64(double x) { return exp(x); }

__device__ __noinline__ void route_row(const RouteSpec* spec, const float* row, const float* bias, double* v,
                                       int* id_out, float* w_out) {
  const RouteSpec p = *spec;
  const int lane = threadIdx.x & 31, size = p.n / p.groups;
  int most = INT_MIN;
#pragma unroll 1
  for (int e = lane; e < p.n; e += 32)
    if (there(row[e])) most = max(most, ordered(fminf(row[e], FLT_MAX)));
  most = __reduce_max_sync(kAll, most);
  const double top = most == INT_MIN ? 0.0 : (double)unordered(most);
  double total = 0.0;
#pragma unroll 1
  for (int e = lane; e < p.n; e += 32) {
    const double l = (double)fminf(row[e], FLT_MAX), x = exp_64(p.sigmoid ? -l : l - top);
    const double s = !there(row[e]) ? -1.0 : p.sigmoid ? 1.0 / (1.0 + x) : x;
    v[e] = s;
    if (s >= 0.0) total += s;
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
#pragma unroll 1
  for (int e = lane; e < p.n; e += 32) {
    double x = v[e];
    if (x < 0.0) {
      x = -INFINITY;
    } else if (!bias && p.groups == 1) {
      x = (double)fminf(row[e], FLT_MAX);  // the scores' order, which they lose where they saturate
    } else {
      x = (p.sigmoid ? x : x / total) + (bias ? (double)bias[e] : 0.0);
      if (!(x > -INFINITY)) x = -INFINITY;
    }
    v[e] = x;
  }
  __syncwarp();
  // the warp's best pair: the largest value, of equal ones the lowest index
  auto meet = [&](double& b, int& at) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double w = __shfl_xor_sync(kAll, b, o);
      const int j = __shfl_xor_sync(kAll, at, o);
      if (w > b || (w == b && j < at)) {
        b = w;
        at = j;
      }
    }
  };
  if (p.groups > 1) {  // lane g scores group g; a group's rank is the number of better ones
    double b1 = -INFINITY, b2 = -INFINITY;
    if (lane < p.groups)
#pragma unroll 4
      for (int i = 0; i < size; ++i) {
        const double x = v[lane * size + i];
        b2 = x > b1 ? b1 : x > b2 ? x : b2;
        b1 = x > b1 ? x : b1;
      }
    const double score = p.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    int rank = 0;
#pragma unroll 4
    for (int g = 0; g < p.groups; ++g) {
      const double other = __shfl_sync(kAll, score, g);
      rank += other > score || (other == score && g < lane);
    }
    const unsigned kept = __ballot_sync(kAll, lane < p.groups && rank < p.top_groups);
#pragma unroll 1
    for (int e = lane; e < p.n; e += 32)
      if (!(kept >> (e / size) & 1)) v[e] = -INFINITY;
    __syncwarp();
  }
  int id = -1;
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    double b = -INFINITY;
    int at = kMaxExperts;
#pragma unroll 1
    for (int e = lane; e < p.n; e += 32)
      if (v[e] > b) {
        b = v[e];
        at = e;
      }
    meet(b, at);
    if (at == kMaxExperts) break;
    if (lane == j) id = at;
    __syncwarp();
    if (lane == 0) v[at] = -INFINITY;
    __syncwarp();
  }
  // The weights.  Renormalised ones relative to the largest chosen logit (for
  // the sigmoid where that is negative): the chosen scores may all lie below
  // the smallest float.
  const double l = id >= 0 ? (double)fminf(row[id], FLT_MAX) : 0.0;
  double m = top;
  if (p.renormalise) {
    m = (double)unordered(__reduce_max_sync(kAll, id >= 0 ? ordered((float)l) : ordered(-FLT_MAX)));
    if (p.sigmoid) m = fmin(m, 0.0);
  } else if (p.sigmoid) {
    m = 0.0;
  }
  // softmax e^(l - m); sigmoid e^(l - m) / (1 + e^l), for positive l (m = 0) 1 / (1 + e^-l)
  const double x = exp_64(p.sigmoid ? -fabs(l) : l - m);
  double w = p.sigmoid ? (l > 0.0 ? 1.0 : exp_64(l - m)) / (1.0 + x) : x;
  if (id < 0) w = 0.0;
  double sum = w;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (!p.renormalise) sum = p.sigmoid ? 1.0 : total;
  *id_out = id;
  *w_out = id < 0 ? 0.f : (float)((double)p.scale * (w / sum));
  __syncwarp();
}

// ---- one row by one warp in FP32: false where two compared values are closer
// than their error (then route_row decides)

// The error of a compared value.
//   sigmoid: 1 / (1 + 2^(-l log2 e)): the exponent's two roundings and the function's error
//   give s (1 - s) (|l| 2^-23 + 2^-22) < 1e-7, the reciprocal 1 ulp: |ds| < 2e-7
//   softmax: exp(l - top) off by < 2.7e-7 in the same way; the sum's relative
//   error, in eight partial sums at least, (n / 8 + 4) 2^-24, is common to all
//   scores <= 1
//   adding the bias rounds by 2^-24 |v|
// A difference of two is off by twice that; a group's score adds two values.
__device__ __forceinline__ float value_error(int n, bool sigmoid) {
  return sigmoid ? 4e-7f : 6e-7f + (float)(n / 8 + 4) * 6e-8f;
}

// The score of a group of two available values.  Biases of the lowest float leave
// their sum available, but below what FP32 holds; as the lowest float it is close to
// any other such group, and 64 bits decide between them.
__device__ __forceinline__ float pair_score(float b1, float b2) { return fmaxf(b1 + b2, -FLT_MAX); }

// The weight of a warp's row: lane j has the j-th choice (-1: none) and its
// logit; the row's largest logit and one over its softmax's sum.
__device__ __forceinline__ float row_weight(const RouteSpec& p, int id, float l, float top, float over) {
  float w = 0.f;
  if (!p.renormalise) {
    if (id >= 0) w = p.sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - top) * over;
  } else {  // relative to the largest: see route_row
    float m = unordered(__reduce_max_sync(kAll, id >= 0 ? ordered(l) : INT_MIN));
    if (p.sigmoid) m = fminf(m, 0.f);
    if (id >= 0) w = !p.sigmoid ? expf(l - m) : l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - m) / (1.f + expf(l));
    const float sum = warp_sum(w);
    if (id >= 0) w /= sum;
  }
  return p.scale * w;
}

template <int PER>
__device__ __forceinline__ bool route_row_fast(const RouteSpec& p, const float* row, const float* bias, int* id_out,
                                               float* w_out) {
  constexpr int kLow = INT_MIN;
  const int lane = threadIdx.x & 31, size = p.n / p.groups;
  const bool by_logit = !bias && p.groups == 1;
  const int none = ordered(-INFINITY);
  float l[PER];
  int v[PER], best = kLow;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = q * 32 + lane;
    l[q] = e < p.n ? fminf(__ldg(row + e), FLT_MAX) : -FLT_MAX;  // fminf drops a NaN ...
    if (e < p.n && !there(__ldg(row + e))) l[q] = -FLT_MAX;      // ... which rules the expert out
    best = max(best, ordered(l[q]));
  }
  const float top = unordered(__reduce_max_sync(kAll, best));
  float s[PER], total = 0.f;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    s[q] = !there(l[q]) ? 0.f : p.sigmoid ? quick_sigmoid(l[q]) : quick_exp(l[q] - top);
    total += s[q];
  }
  float over = 1.f;
  if (!p.sigmoid) {
    total = warp_sum(total);
    over = total > 0.f ? 1.f / total : 0.f;
  }
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    v[q] = none;
    if (there(l[q])) {
      const float b = bias ? __ldg(bias + q * 32 + lane) : 0.f;
      const float x = by_logit ? l[q] + 0.f : s[q] * over + b;  // + 0: -0 and 0 are one value, and so one integer
      if (x > -INFINITY) v[q] = ordered(x);
    }
  }
  const float wide = 2.f * value_error(p.n, p.sigmoid);
  auto apart = [&](float a, float b) { return by_logit ? a > b : a - b > wide + 1.2e-7f * (fabsf(a) + fabsf(b)); };
  // the largest value of the experts from..to - 1 and its lowest index, which is then taken out
  auto take = [&](int from, int to, int& at) {
    int m = none;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * 32 + lane;
      if (e >= from && e < to) m = max(m, v[q]);
    }
    m = __reduce_max_sync(kAll, m);
    int i = INT_MAX;
#pragma unroll
    for (int q = PER - 1; q >= 0; --q) {
      const int e = q * 32 + lane;
      if (e >= from && e < to && v[q] == m) i = e;
    }
    at = __reduce_min_sync(kAll, i);
    return unordered(m);
  };
  auto drop = [&](int at) {
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (q * 32 + lane == at) v[q] = none;
  };
  if (p.groups > 1) {
    float mine = -INFINITY;  // lane g: the score of group g
    for (int g = 0; g < p.groups; ++g) {
      int at, m = none;
      const float b1 = take(g * size, (g + 1) * size, at);
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int e = q * 32 + lane;
        if (e >= g * size && e < (g + 1) * size && e != at) m = max(m, v[q]);
      }
      float sum = b1;
      if (p.group_best == 2) {
        const float b2 = unordered(__reduce_max_sync(kAll, m));
        if (b2 > -INFINITY) sum = pair_score(b1, b2);
      }
      if (lane == g) mine = sum;
    }
    unsigned kept = 0;
    float last = INFINITY;
    int score = ordered(mine);
    for (int r = 0; r < p.top_groups; ++r) {
      const int m = __reduce_max_sync(kAll, score);
      if (m == none) break;
      const int at = __ffs(__ballot_sync(kAll, score == m)) - 1;
      kept |= 1u << at;
      last = unordered(m);
      if (lane == at) score = none;
    }
    const float next = unordered(__reduce_max_sync(kAll, score));
    if (next > -INFINITY && !(last - next > 2.f * wide + 2.4e-7f * (fabsf(last) + fabsf(next)))) return false;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * 32 + lane;
      if (e < p.n && !(kept >> (e / size) & 1)) v[q] = none;
    }
  }
  // equal logits and biases are equal values here, of which take() gives the lowest index first
  auto same = [&](int a, int b) {
    return __ldg(row + a) == __ldg(row + b) && (!bias || __ldg(bias + a) == __ldg(bias + b));
  };
  int id = -1, before = -1;
  float last = INFINITY;
  for (int j = 0; j < p.k; ++j) {
    int at;
    const float x = take(0, p.n, at);
    if (!(x > -INFINITY)) break;
    if (before >= 0 && !apart(last, x) && !same(before, at)) return false;
    drop(at);
    if (lane == j) id = at;
    before = at;
    last = x;
  }
  for (;;) {  // those not chosen
    int at;
    const float x = take(0, p.n, at);
    if (!(x > -INFINITY) || before < 0 || apart(last, x)) break;
    if (!same(before, at)) return false;
    drop(at);
  }
  *id_out = id;
  *w_out = row_weight(p, id, id >= 0 ? fminf(__ldg(row + max(id, 0)), FLT_MAX) : 0.f, top, over);
  return true;
}

// ---- forward, one warp a row, eight rows a CTA (few rows, many experts, k > 8).
// Every choice is a reduction over all of the row's values, so many rows are slow here:
// 40,000 x 256 in 8 groups, k = 8, 164 us; 172,050 x 64, k = 16, 855 us, 13 and 51
// times what their bytes take; 1,000 x 64, k = 8, 10.5 us

template <int PER>
__global__ void __launch_bounds__(256) route_warp_kernel(const __grid_constant__ RouteSpec p, int64_t n, const float* __restrict__ logits,
                                                         const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights, float* __restrict__ gates,
                                                         int64_t ld, int32_t* __restrict__ counts) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int S = PER < 16 ? 9 : 8;  // 48 KB in all at 512 experts
  __shared__ float tile[PER * 32 * S];  // gates of eight rows, [expert][S]
  __shared__ double exact[8][PER * 32];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  for (int64_t t0 = (int64_t)blockIdx.x * 8; t0 < n; t0 += (int64_t)gridDim.x * 8) {
    const int64_t t = t0 + r;
    if (t < n) {  // whole warps
      int id;
      float w;
      if (!route_row_fast<PER>(p, logits + t * p.n, bias, &id, &w))
        route_row(&p, logits + t * p.n, bias, exact[r], &id, &w);
      if (lane < p.k) {
        if (ids) ids[t * p.k + lane] = id;
        if (weights) weights[t * p.k + lane] = w;
        if (counts && id >= 0) atomicAdd(counts + id, 1);
      }
      if (gates) {
#pragma unroll
        for (int q = 0; q < PER; ++q) tile[(q * 32 + lane) * S + r] = 0.f;
        __syncwarp();
        if (id >= 0) tile[id * S + r] = w;
      }
    }
    if (gates) {
      __syncthreads();
      for (int i = threadIdx.x; i < p.n * 8; i += 256)
        if (t0 + (i & 7) < n) gates[(int64_t)(i >> 3) * ld + t0 + (i & 7)] = tile[(i >> 3) * S + (i & 7)];
      __syncthreads();
    }
  }
}

// ---- forward, one thread a row (many rows)

// Rows of a CTA's tile.  64 / 128, us: 172,050 x 128, k = 8: 117 / 137; x 96: 84 / 90; x 64
// in 8 groups: 49.5 / 49; 400,000 x 16, k = 2: 28.7 / 27.2.
constexpr int kTile = 64;
constexpr int kThreadExperts = 128;  // the widest row of this form
constexpr int kThreadK = 8;

// A key whose order as an integer is the value's, its low bits replaced so that of
// equal values the lowest index is the largest; mask = 2^bits - 1 >= experts - 1.
__device__ __forceinline__ int key_of(float v, int e, int mask) {
  int i = __float_as_int(v);
  i ^= (i >> 31) & 0x7fffffff;
  return (i & ~mask) | (mask - e);
}

// The largest value that a key's order allows.
__device__ __forceinline__ float key_top(int key, int mask) {
  int i = key | mask;
  i ^= (i >> 31) & 0x7fffffff;
  return __int_as_float(i);
}

// A falling list of L = 2^i + 1 keys: the places from the back meet a falling list
// b of n <= L from its front, and the larger ones, the best L of both, are put in
// order (a bitonic merge whose first place stands alone).
template <int L>
__device__ __forceinline__ void merge_keys(int (&a)[L], const int* b, int n) {
  auto meet = [&](int i, int j) {
    const int most = max(a[i], a[j]);
    a[j] = min(a[i], a[j]);
    a[i] = most;
  };
#pragma unroll
  for (int i = 0; i < n; ++i) a[L - 1 - i] = max(a[L - 1 - i], b[i]);
  meet(0, L - 1);
#pragma unroll
  for (int m = (L - 1) / 2; m > 0; m /= 2)
#pragma unroll
    for (int i = 1; i < L; ++i)
      if (((i - 1) & m) == 0) meet(i, i + m);
}

__device__ __forceinline__ void sort_four(int (&b)[4]) {
  auto meet = [&](int i, int j) {
    const int most = max(b[i], b[j]);
    b[j] = min(b[i], b[j]);
    b[i] = most;
  };
  meet(0, 1);
  meet(2, 3);
  meet(0, 2);
  meet(1, 3);
  meet(1, 2);
}

// A row's choice in FP32, by one thread.  Two compared values are off by at
// most twice value_error against one another; where a decision is closer than that
// the row is looked at again (two experts of equal logit and bias are in their
// right order already) and, if that does not settle it, decided in 64 bits by the
// whole warp: the few experts that may be among the k best, one a lane.  The k + 1 best are found as integer keys (two instructions a
// place and expert) that hold the index in their
// low bits; the keys' order is put right from the values themselves.
//
// Two threads share a row, each with one half of every group: the second also
// clears the row's gates while the first chooses the groups.  The tile lies
// by experts, [expert][row], so that a thread's experts are constant offsets from
// one address.
//
// What bounds it (B200, 172,050 x 64 in 8 groups, k = 8): 51 us for 99 MB.  Some 5,300
// instructions for 32 rows take 62 % of the issue slots; the largest stall is the
// barriers at which the second half waits while the first merges the lists and decides;
// and the last of 2.3 waves is not full.  64 registers hold all but 36 to 56 bytes a
// thread, which spill.  A warp a row in 64 bits took 1,954 us.
template <int K, bool SIGMOID, bool BY_LOGIT>
__global__ void __launch_bounds__(2 * kTile, 512 / kTile) route_thread_kernel(
    const __grid_constant__ RouteSpec p, int64_t n, const float* __restrict__ logits, const float* __restrict__ bias,
    int32_t* __restrict__ ids, float* __restrict__ weights, float* __restrict__ gates, int64_t ld,
    int32_t* __restrict__ counts, unsigned magic) {
  grid_dependency_wait();
  grid_launch_dependents();
  extern __shared__ float4 smem4[];
  float* smem = reinterpret_cast<float*>(smem4);
  constexpr int S = kTile + 1;  // odd: neither filling nor reading meets one bank
  const int tid = threadIdx.x & (kTile - 1), half = threadIdx.x / kTile, lane = tid & 31, N = p.n;
  double* exact = reinterpret_cast<double*>(smem4);  // [kTile / 32][N] of the warps that decide
  float* sb = smem + kTile / 16 * N;                 // [N] bias, in whole float4s
  float* tile = sb + (N + 3) / 4 * 4;                // [N][S]
  int* hist = reinterpret_cast<int*>(tile + N * S);  // [N]
  unsigned* skept = reinterpret_cast<unsigned*>(hist + N);  // [kTile] groups kept, then [4][kTile] experts chosen
  float* swap = reinterpret_cast<float*>(skept + 4 * kTile);  // [swap_rows][kTile], what the halves tell one another
  for (int e = threadIdx.x; e < N; e += 2 * kTile) {
    const float b = bias ? __ldg(bias + e) : 0.f;
    sb[e] = b >= -INFINITY ? b : -INFINITY;  // a NaN rules the expert out too
    hist[e] = 0;
  }
  int mask = 1;
  while (mask < N - 1) mask = 2 * mask + 1;
  const float base = value_error(N, SIGMOID);
  const int size = N / p.groups, split = (size + 1) / 2;
  const int from = half ? split : 0, to = half ? size : split;  // this thread's part of a group
  const bool fours = size % 8 == 0;                             // both parts are whole fours
  // a thread's float4s of a tile are 8 kTile values apart: so many rows and columns
  const int fill_r = N == 1 ? 0 : (int)__umulhi(threadIdx.x * 4, magic), fill_c = threadIdx.x * 4 - fill_r * N;
  const int step_c = 8 * kTile % N, step_at = step_c * S + 8 * kTile / N;
  for (int64_t t0 = (int64_t)blockIdx.x * kTile; t0 < n; t0 += (int64_t)gridDim.x * kTile) {
    const int rows = (int)min((int64_t)kTile, n - t0);
    __syncthreads();  // the tile of the round before is read
    const float* src = logits + t0 * N;  // rows N values from a 16-byte border
    if (N % 4 == 0) {
      int c = fill_c;
      float* dst = tile + c * S + fill_r;
#pragma unroll 4
      for (int i = threadIdx.x * 4; i < rows * N; i += 8 * kTile) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(src + i));
        dst[0] = f.x;
        dst[S] = f.y;
        dst[2 * S] = f.z;
        dst[3 * S] = f.w;
        c += step_c;
        dst += step_at;
        if (c >= N) {
          c -= N;
          dst -= N * S - 1;
        }
      }
    } else {
#pragma unroll 8
      for (int i = threadIdx.x; i < rows * N; i += 2 * kTile) {
        const int r = N == 1 ? i : (int)__umulhi(i, magic);
        tile[(i - r * N) * S + r] = __ldg(src + i);
      }
    }
    __syncthreads();
    // Rows behind the last: whatever lies in their columns is computed with and not written.
    const bool live = tid < rows;
    const int64_t t = t0 + tid;
    float* col = tile + tid;                                  // expert e of this row at col[e S]
    const float* row = logits + (t0 + (live ? tid : 0)) * N;  // the same in memory
    float top = -FLT_MAX, total = 0.f;
    if (!SIGMOID && !(BY_LOGIT && (p.renormalise || p.sigmoid))) {
      const int e0 = half ? (N + 1) / 2 : 0, e1 = half ? N : (N + 1) / 2;
#pragma unroll 8
      for (int e = e0; e < e1; ++e) top = fmaxf(top, there(col[e * S]) ? fminf(col[e * S], FLT_MAX) : -FLT_MAX);
      swap[half * kTile + tid] = top;
      __syncthreads();
      top = fmaxf(top, swap[(1 - half) * kTile + tid]);
      float part[4] = {};
      for (int e = e0; e < e1; e += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float l = e + j < e1 ? col[(e + j) * S] : -FLT_MAX;
          const float x = there(l) ? quick_exp(fminf(l, FLT_MAX) - top) : 0.f;
          part[j] += x;
          // from here on the tile holds these, -1 where the expert is out
          if (!BY_LOGIT && e + j < e1) col[(e + j) * S] = there(l) ? x : -1.f;
        }
      total = (part[0] + part[1]) + (part[2] + part[3]);
      __syncthreads();
      swap[half * kTile + tid] = total;
      __syncthreads();
      total = swap[tid] + swap[kTile + tid];
      __syncthreads();
    }
    const float over = total > 0.f ? 1.f / total : 0.f;
    auto score = [&](float x) {  // from the tile; -1 where the expert is out
      if (!SIGMOID) return x < 0.f ? -1.f : x * over;
      const float s = quick_sigmoid(x);
      return there(x) ? s : -1.f;
    };
    auto biased = [&](float s, float b) { return s < 0.f ? -INFINITY : s + b; };
    // what is compared, from the tile: logits, with groups (once they are scored) scores
    auto value = [&](float x, float b) {
      if (BY_LOGIT) return there(x) ? fminf(x, FLT_MAX) : -INFINITY;
      return biased(p.groups > 1 ? x : score(x), b);
    };
    const float wide = 2.f * base;  // bound on the error of a difference of two values, with 2^-23 of each
    auto apart = [&](float a, float b) { return BY_LOGIT ? a > b : a - b > wide + 1.2e-7f * (fabsf(a) + fabsf(b)); };
    bool doubt = false, hard = false;  // hard: 64 bits from the start
    unsigned kept = 1;
    int key[K + 1];
#pragma unroll
    for (int j = 0; j <= K; ++j) key[j] = INT_MIN;
    auto insert = [&](int x) {
#pragma unroll
      for (int j = 0; j <= K; ++j) {
        const int a = max(x, key[j]);
        x = min(x, key[j]);
        key[j] = a;
      }
    };
    // four experts from e on; a long list takes them sorted (40 instructions for a
    // list of nine, 72 one by one)
    auto insert_four = [&](const float* c, int e) {
      int x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = key_of(value(c[j * S], sb[e + j]), e + j, mask);
      if constexpr (K >= 4) {
        sort_four(x);
        merge_keys(key, x, 4);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) insert(x[j]);
      }
    };
    if (p.groups > 1) {
      // the groups' scores, half of the groups by each half
      const int mid = (p.groups + 1) / 2, last_group = half ? p.groups : mid;
      for (int g = half ? mid : 0; g < last_group; ++g) {
        float b1 = -INFINITY, b2 = -INFINITY;
        float* c = col + g * size * S;
        const float* b = sb + g * size;
        auto look = [&](float* at, float bi) {
          const float x = *at, s = SIGMOID ? quick_sigmoid(x) : x * over;
          const bool in = SIGMOID ? there(x) : x >= 0.f;
          const float v = in ? s + bi : -INFINITY;
          *at = in ? s : -1.f;  // from here on the tile holds the scores
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
        };
        if (size % 4 == 0) {
#pragma unroll 1
          for (int i = 0; i < size; i += 4, c += 4 * S, b += 4) {
            const float4 bi = *reinterpret_cast<const float4*>(b);
            look(c, bi.x);
            look(c + S, bi.y);
            look(c + 2 * S, bi.z);
            look(c + 3 * S, bi.w);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < size; ++i, c += S, ++b) look(c, *b);
        }
        swap[g * kTile + tid] = p.group_best == 2 && b2 > -INFINITY ? pair_score(b1, b2) : b1;
      }
      __syncthreads();
      if (!half) {
        kept = 0;
        float last = INFINITY;
        for (int r = 0; r < p.top_groups; ++r) {
          float best = -INFINITY;
          int at = -1;
#pragma unroll 4
          for (int g = 0; g < p.groups; ++g) {
            const float x = swap[g * kTile + tid];
            if (x > best) {
              best = x;
              at = g;
            }
          }
          if (at >= 0) {
            kept |= 1u << at;
            last = best;
            swap[at * kTile + tid] = -INFINITY;
          }
        }
        float next = -INFINITY;
#pragma unroll 4
        for (int g = 0; g < p.groups; ++g) next = fmaxf(next, swap[g * kTile + tid]);
        hard = next > -INFINITY && !(last - next > 2.f * wide + 2.4e-7f * (fabsf(last) + fabsf(next)));
        skept[tid] = kept;
      }
      __syncthreads();
      kept = skept[tid];
      for (unsigned left = kept; left; left &= left - 1) {
        int e = (__ffs(left) - 1) * size + from;
        const int end = e + to - from;
        const float* c = col + e * S;
        if (fours) {
          for (; e < end; e += 4, c += 4 * S) insert_four(c, e);
        } else {
#pragma unroll 1
          for (; e < end; ++e, c += S) insert(key_of(value(*c, sb[e]), e, mask));
        }
      }
    } else {
      const float* c = col + from * S;
      if (fours) {
        for (int e = from; e < to; e += 4, c += 4 * S) insert_four(c, e);
      } else {
#pragma unroll 1
        for (int e = from; e < to; ++e, c += S) insert(key_of(value(*c, sb[e]), e, mask));
      }
    }
    if (half) {
#pragma unroll
      for (int j = 0; j <= K; ++j) swap[j * kTile + tid] = __int_as_float(key[j]);
    }
    __syncthreads();
    if (!half) {
      int other[K + 1];
#pragma unroll
      for (int j = 0; j <= K; ++j) other[j] = __float_as_int(swap[j * kTile + tid]);
      merge_keys(key, other, K + 1);
      // the values behind the keys, as they were compared
      float val[K + 1];
      int idx[K + 1];
#pragma unroll
      for (int j = 0; j <= K; ++j) {
        const bool some = key[j] != INT_MIN;
        idx[j] = some ? mask - (key[j] & mask) : 0;
        const float v = value(col[idx[j] * S], sb[idx[j]]);
        val[j] = some ? v : -INFINITY;
      }
      const float outside = key[K] != INT_MIN ? key_top(key[K], mask) : -INFINITY;  // no smaller key has more
#pragma unroll
      for (int j = K; j > 0; --j) {  // neighbours that the keys' cut bits put the wrong way round
        const bool wrong = val[j] > val[j - 1];
        const float a = val[j];
        val[j] = wrong ? val[j - 1] : a;
        val[j - 1] = wrong ? a : val[j - 1];
        const int b = idx[j];
        idx[j] = wrong ? idx[j - 1] : b;
        idx[j - 1] = wrong ? b : idx[j - 1];
      }
      // The smallest gap: inside the k first, and from the smallest of them (also
      // while two are the wrong way round) to the rest of the list, which one pass need
      // not have put in order, and to the experts behind its last key, at most
      // `outside`.  (Where fewer than k are left, the list holds them all; a difference
      // with -inf is inf or a NaN, which fminf drops.)
      float lastv = INFINITY, gap = INFINITY, rest = val[K] > -INFINITY ? outside : -INFINITY;
      int lastid = -1;
#pragma unroll
      for (int j = 0; j <= K; ++j) {
        const bool in = j < p.k && val[j] > -INFINITY;
        lastv = in ? fminf(lastv, val[j]) : lastv;
        lastid = in ? idx[j] : lastid;
        if (j > 0) gap = in ? fminf(gap, val[j - 1] - val[j]) : gap;
        rest = j < p.k ? rest : fmaxf(rest, val[j]);
      }
      gap = fminf(gap, lastv - rest);
      const float size_of = fmaxf(fabsf(val[0]), lastid >= 0 ? fabsf(lastv) : 0.f);
      // every pair is closer to zero than size_of, or apart by more than it
      const bool close = lastid >= 0 && !(BY_LOGIT ? gap > 0.f : gap > wide + 2.4e-7f * size_of);
      if (close && live && !hard) {
        auto same = [&](int a, int b) { return a < b && __ldg(row + a) == __ldg(row + b) && sb[a] == sb[b]; };
#pragma unroll
        for (int j = 0; j + 1 < K; ++j)
          if (j + 1 < p.k && val[j + 1] > -INFINITY && !apart(val[j], val[j + 1])) doubt |= !same(idx[j], idx[j + 1]);
        for (unsigned left = kept; left; left &= left - 1) {
          const int e0 = (__ffs(left) - 1) * size;
          for (int e = e0; e < e0 + size; ++e) {
            const float v = value(col[e * S], sb[e]);
            if (v > -INFINITY && !apart(lastv, v)) {
              bool chosen = false;
#pragma unroll
              for (int j = 0; j < K; ++j) chosen |= j < p.k && idx[j] == e;
              if (!chosen) doubt |= !same(lastid, e);
            }
          }
        }
      }
      // weights of the chosen, in order: from the scores where the tile holds them
      const bool scored = p.groups > 1 || !(SIGMOID || BY_LOGIT);
      float w[K], sum = 0.f, most = -FLT_MAX, least = 1.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (j >= p.k || !(val[j] > -INFINITY)) idx[j] = -1;
        w[j] = idx[j] < 0 ? 0.f : col[idx[j] * S];
        most = idx[j] < 0 ? most : fmaxf(most, w[j]);
        least = idx[j] < 0 ? least : fminf(least, w[j]);
      }
      // Small scores are formed again from their logits: the quick exponential of x is off
      // by |x| 2^-23 of itself, and gives 0 below the smallest normal float.
      const bool again = scored && lastid >= 0 && least < 1e-13f;
      if (again) {
        most = -FLT_MAX;
#pragma unroll
        for (int j = 0; j < K; ++j) {
          w[j] = idx[j] < 0 ? 0.f : __ldg(row + idx[j]);
          most = idx[j] < 0 ? most : fmaxf(most, w[j]);
        }
      }
      if (scored && !again) {
        // the scores stand in w
      } else if (SIGMOID || (BY_LOGIT && p.sigmoid)) {
        most = p.renormalise ? fminf(most, 0.f) : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const float x = fminf(w[j], FLT_MAX);
          const float a = x > 0.f || !p.renormalise ? __fdividef(1.f, 1.f + expf(-x))
                                                    : __fdividef(expf(x - most), 1.f + expf(x));
          w[j] = idx[j] < 0 ? 0.f : a;
        }
      } else {
        most = p.renormalise ? fminf(most, FLT_MAX) : top;
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const float a = expf(fminf(w[j], FLT_MAX) - most);
          w[j] = idx[j] < 0 ? 0.f : a;
        }
      }
#pragma unroll
      for (int j = 0; j < K; ++j) sum += w[j];
      // a softmax's scores are divided by their sum already where groups were scored
      const float f = p.renormalise                           ? (sum > 0.f ? p.scale / sum : 0.f)
                      : p.sigmoid || (p.groups > 1 && !again) ? p.scale
                                                              : p.scale * over;
#pragma unroll
      for (int j = 0; j < K; ++j) w[j] *= f;
      if (p.renormalise && idx[0] >= 0 && (K == 1 || idx[K > 1] < 0)) w[0] = p.scale;  // a single one: not by rounding
      doubt = (doubt || hard) && live;
      if (live && !doubt) {
        if (K % 4 == 0 && p.k == K) {
#pragma unroll
          for (int j = 0; j + 3 < K; j += 4) {
            if (ids) *reinterpret_cast<int4*>(ids + t * K + j) = make_int4(idx[j], idx[j + 1], idx[j + 2], idx[j + 3]);
            if (weights) *reinterpret_cast<float4*>(weights + t * K + j) = make_float4(w[j], w[j + 1], w[j + 2], w[j + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (j < p.k) {
              if (ids) ids[t * p.k + j] = idx[j];
              if (weights) weights[t * p.k + j] = w[j];
            }
        }
      }
      // gates: the chosen's weights to the tile, their places to a mask of 128 bits
      unsigned chosen[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (idx[j] >= 0 && live && !doubt) {
          col[idx[j] * S] = w[j];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (32 * q < N) chosen[q] |= idx[j] >> 5 == q ? 1u << (idx[j] & 31) : 0u;
          if (counts) atomicAdd(hist + idx[j], 1);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (32 * q < N) skept[q * kTile + tid] = chosen[q];
      __syncwarp();
      for (unsigned left = __ballot_sync(kAll, doubt); left; left &= left - 1) {
        const int from_lane = __ffs(left) - 1, r = (tid & ~31) + from_lane;
        const float* rowr = logits + (t0 + r) * N;
        const float* colr = tile + r;
        const float lastr = __shfl_sync(kAll, lastv, from_lane);
        const unsigned keptr = __shfl_sync(kAll, kept, from_lane);
        const float topr = __shfl_sync(kAll, top, from_lane), overr = __shfl_sync(kAll, over, from_lane);
        // the experts that may be among the k best: one a lane
        int* cand = reinterpret_cast<int*>(exact + (tid >> 5) * N);
        int m = 0;
        if (!__shfl_sync(kAll, (int)hard, from_lane)) {
#pragma unroll 1
          for (int e0 = 0; e0 < N; e0 += 32) {
            const int e = e0 + lane;
            float v = -INFINITY;
            if (e < N && keptr >> (e / size) & 1) {
              const float x = colr[e * S];
              v = BY_LOGIT ? (there(x) ? fminf(x, FLT_MAX) : -INFINITY)
                           : biased(p.groups > 1 ? x
                                    : !SIGMOID   ? (x < 0.f ? -1.f : x * overr)
                                    : there(x)   ? quick_sigmoid(x)
                                                 : -1.f,
                                    sb[e]);
            }
            const bool may = v > -INFINITY && !apart(lastr, v);
            const unsigned who = __ballot_sync(kAll, may);
            const int at = m + __popc(who & ((1u << lane) - 1));
            if (may && at < 32) cand[at] = e;
            m += __popc(who);
          }
          __syncwarp();
        }
        int id;
        float wj;
        if (m >= 1 && m <= 32) {
          const int e = lane < m ? cand[lane] : 0;
          const double l = (double)fminf(__ldg(rowr + e), FLT_MAX);
          double v = l, total64 = 0.0;
          if (!BY_LOGIT) {
            if (!SIGMOID) {
#pragma unroll 1
              for (int q = lane; q < N; q += 32) {
                const float x = __ldg(rowr + q);
                if (there(x)) total64 += exp_64((double)fminf(x, FLT_MAX) - (double)topr);
              }
              total64 = warp_sum(total64);
            }
            const double x = exp_64(SIGMOID ? -l : l - (double)topr);
            v = (SIGMOID ? 1.0 / (1.0 + x) : x / total64) + (bias ? (double)__ldg(bias + e) : 0.0);
          }
          int rank = 0;
#pragma unroll 1
          for (int c = 0; c < m; ++c) {
            const double other = __shfl_sync(kAll, v, c);
            rank += other > v || (other == v && c < lane);  // candidates ascend
          }
          __syncwarp();
          if (lane < m) cand[rank] = e;
          __syncwarp();
          id = lane < p.k && lane < m ? cand[lane] : -1;
          __syncwarp();
          wj = row_weight(p, id, id >= 0 ? fminf(__ldg(rowr + id), FLT_MAX) : 0.f, topr, overr);
        } else {
          route_row(&p, rowr, bias, exact + (tid >> 5) * N, &id, &wj);
        }
        if (lane < p.k) {
          if (ids) ids[(t0 + r) * p.k + lane] = id;
          if (weights) weights[(t0 + r) * p.k + lane] = wj;
          if (id >= 0) {
            tile[id * S + r] = wj;
            atomicOr(skept + (id >> 5) * kTile + r, 1u << (id & 31));
            if (counts) atomicAdd(hist + id, 1);
          }
        }
      }
    }
    if (gates) {  // each half writes half of the experts, a warp 32 rows of one expert
      __syncthreads();
      if (live) {
        const int mid = (N / 2 + 7) / 8 * 8, e0 = half ? mid : 0, e1 = half ? N : min(mid, N);
        float* out = gates + t0 + e0 * ld;
        for (int e = e0; e < e1; e += 8) {  // eights do not cross a word of the mask
          const unsigned bits = skept[(e >> 5) * kTile + tid] >> (e & 31);
          const float* from_tile = col + e * S;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e + j < e1) {
              out[tid] = bits & 1u << j ? from_tile[j * S] : 0.f;
              out += ld;
            }
        }
      }
    }
  }
  if (counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < N; e += 2 * kTile)
      if (hist[e]) atomicAdd(counts + e, hist[e]);
  }
}

// ---- backward where only the chosen experts' logits have a gradient: one
// thread a row; the gradient is built in shared memory and written in whole
// lines.  A chosen expert's logit and gate gradient are one sector each, and an SM
// holds few requests of one sector: where the row is not much longer than its
// choices and the arrays are large, the whole rows are read and the places picked
// in shared memory.  Measured, single sectors / whole, us: 172,050 x 64, k = 8: 79 /
// 35; 60,000 x 128: 37 / 30; 60,000 x 64: 12.5 / 12.9; 10,000 x 64: 5.9 / 7.2.  What is
// left of the first is latency: its 132 MB pass at 3.8 TB/s.

constexpr int kRows = 128;               // rows of a CTA's tile, at most
constexpr int64_t kWholeRows = 1 << 22;  // values of an array

template <int K>
__global__ void __launch_bounds__(2 * kRows, K <= 8 ? 5 : 2) route_chosen_backward_kernel(
    RouteSpec p, int64_t n, const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ grad_weights, const float* __restrict__ grad_gates, int64_t ld,
    float* __restrict__ grad_logits, unsigned magic) {
  grid_dependency_wait();
  grid_launch_dependents();
  extern __shared__ float4 smem4[];
  float* smem = reinterpret_cast<float*>(smem4);
  const int N = p.n, R = blockDim.x / 2, half = threadIdx.x / R, tid = threadIdx.x - half * R, odd = N | 1;
  const bool whole = N <= 16 * p.k && n * N >= kWholeRows;
  for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < n; t0 += (int64_t)gridDim.x * R) {
    const int rows = (int)min((int64_t)R, n - t0);
    const bool live = tid < rows, mine = live && !half;  // the second half helps to move whole rows
    const int64_t t = t0 + tid;
    int id[K];
    float l[K], d[K];
#pragma unroll
    for (int j = 0; j < K; ++j) id[j] = mine && j < p.k ? __ldg(ids + t * p.k + j) : -1;
    if (!whole) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const bool in = (unsigned)id[j] < (unsigned)N;
        l[j] = in ? __ldg(logits + t * N + id[j]) : -FLT_MAX;
        d[j] = in && grad_gates ? __ldg(grad_gates + (int64_t)id[j] * ld + t) : 0.f;
      }
      __syncthreads();  // the tile of the round before is written out
    } else {
      // the logits' rows, one piece of memory, on their way while the gates' are read
      if (N % 4 == 0 && threadIdx.x == 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(logits + t0 * N), "r"(rows * N * 4) : "memory");
      __syncthreads();
      if (grad_gates) {  // expert e of this row at smem[e R + tid]
        const float* src = grad_gates + t0 + half * ld;
        if (live)
#pragma unroll 16
          for (int e = half; e < N; e += 2, src += 2 * ld) smem[e * R + tid] = __ldg(src + tid);
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < K; ++j) d[j] = (unsigned)id[j] < (unsigned)N && grad_gates ? smem[id[j] * R + tid] : 0.f;
      __syncthreads();
      const float* src = logits + t0 * N;
      if (N % 4 == 0) {
#pragma unroll 8
        for (int i = threadIdx.x * 4; i < rows * N; i += R * 8) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(src + i));
          const int r = (int)__umulhi(i, magic);
          float* dst = smem + r * odd + i - r * N;
          dst[0] = f.x;
          dst[1] = f.y;
          dst[2] = f.z;
          dst[3] = f.w;
        }
      } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < rows * N; i += 2 * R) {
          const int r = N == 1 ? i : (int)__umulhi(i, magic);
          smem[r * odd + i - r * N] = __ldg(src + i);
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < K; ++j) l[j] = (unsigned)id[j] < (unsigned)N ? smem[tid * odd + id[j]] : -FLT_MAX;
      __syncthreads();
    }
    for (int i = threadIdx.x; i < (rows * N + 3) / 4; i += 2 * R) smem4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    if (mine) {
      float* out = smem + tid * N;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if ((unsigned)id[j] < (unsigned)N && grad_weights) d[j] += __ldg(grad_weights + t * p.k + j);
        if (!there(l[j])) {  // out of range, out for the row, or NaN
          id[j] = -1;
          d[j] = 0.f;
        }
        l[j] = fminf(l[j], FLT_MAX);
      }
      float m = 0.f, sum = 0.f, dot = 0.f;
      if (p.renormalise) {
        m = -FLT_MAX;
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (id[j] >= 0) m = fmaxf(m, l[j]);
        if (p.sigmoid) m = fminf(m, 0.f);
      }
      // scores, the renormalised ones relative to exp(m) and then shares that add to
      // one (a single one is 1, and its gradient 0)
      float share[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        share[j] = 0.f;
        if (id[j] >= 0) {
          const float x = l[j];
          share[j] = !p.sigmoid                   ? expf(x - m)
                     : x > 0.f || !p.renormalise ? 1.f / (1.f + expf(-x))
                                                  : expf(x - m) / (1.f + expf(x));
          sum += share[j];
        }
      }
      // Renormalised, d_j - sum(share d): where one share is nearly 1 its d and the sum
      // cancel.  So by differences: pair by pair, or for many places from the d of a share
      // above a half, d_j - ref - sum(share (d - ref)).
      if (p.renormalise) {
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (id[j] >= 0) {
            share[j] /= sum;
            dot = fmaf(d[j], share[j], dot);
          }
        if constexpr (K > 8) {
          float ref = 0.f;
          dot = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (id[j] >= 0 && share[j] > 0.5f) ref = d[j];
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (id[j] >= 0) {
              d[j] -= ref;
              dot = fmaf(d[j], share[j], dot);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (id[j] >= 0) {
          float x = d[j] - dot;
          if (K <= 8 && p.renormalise) {
            x = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i) x = fmaf(share[i], d[j] - d[i], x);
          }
          x *= p.scale * share[j];
          if (p.sigmoid) x *= 1.f / (1.f + expf(l[j]));
          out[id[j]] += x;
        }
    }
    __syncthreads();
    float* dst = grad_logits + t0 * N;
    for (int i = threadIdx.x; i < rows * N / 4; i += 2 * R) reinterpret_cast<float4*>(dst)[i] = smem4[i];
    for (int i = (rows * N & ~3) + threadIdx.x; i < rows * N; i += 2 * R) dst[i] = smem[i];
  }
}

// ---- backward of the softmax as it is, whose sum reaches every logit: L
// lanes a row, lane i the experts i, i + L, ...; lane j also the row's j-th choice.
// (34,244 x 16, k = 2: 5.2 us; by one thread a row over a tile 8.5.)

template <int L, int PER>
__global__ void __launch_bounds__(256) route_every_backward_kernel(
    RouteSpec p, int64_t n, const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ grad_weights, const float* __restrict__ grad_gates, int64_t ld,
    float* __restrict__ grad_logits) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int rows = 256 / L;
  const int lane = threadIdx.x & (L - 1), N = p.n;
  for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < n; t0 += (int64_t)gridDim.x * rows) {  // whole CTAs
    const int64_t t = t0 + threadIdx.x / L;
    const bool live = t < n;
    const float* row = logits + (live ? t : n - 1) * N;
    int id = live && lane < p.k ? __ldg(ids + t * p.k + lane) : -1;
    if ((unsigned)id >= (unsigned)N) id = -1;
    float l[PER], top = -FLT_MAX;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      l[q] = q * L + lane < N ? __ldg(row + q * L + lane) : -FLT_MAX;
      if (there(l[q])) top = fmaxf(top, fminf(l[q], FLT_MAX));
    }
    float d = 0.f, lj = id >= 0 ? __ldg(row + id) : -FLT_MAX;
    if (id >= 0 && grad_weights) d += __ldg(grad_weights + t * p.k + lane);
    if (id >= 0 && grad_gates) d += __ldg(grad_gates + (int64_t)id * ld + t);
    if (!there(lj)) id = -1;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    float total = 0.f;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      l[q] = there(l[q]) ? expf(fminf(l[q], FLT_MAX) - top) : 0.f;
      total += l[q];
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    const float over = total > 0.f ? 1.f / total : 0.f;
    float dot = 0.f;
    // d_i - sum(s d) cancels for a score near 1.  So where one is above a half (it is exp(0)
    // / total), with c its d or, if it is not chosen, 0: d_i - c - sum(s (d - c)).  A row that
    // has a warp (L = 32) and no such score takes fewer instructions: 20,000 x 512 21 us,
    // all rows by differences 25; 300,000 x 16 takes 31 either way.
    if (L < 32 || __any_sync(kAll, total < 2.f)) {
      float c = id >= 0 && total < 2.f && fminf(lj, FLT_MAX) == top ? d : 0.f, each[PER];
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) c += __shfl_xor_sync(kAll, c, o);
#pragma unroll
      for (int q = 0; q < PER; ++q) each[q] = 0.f;
      for (int j = 0; j < p.k; ++j) {
        const int i = __shfl_sync(kAll, id, j, L);
        const float x = __shfl_sync(kAll, d, j, L);
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (i == q * L + lane) each[q] += x;
      }
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        each[q] -= c;
        dot = fmaf(l[q], each[q], dot);
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
#pragma unroll
      for (int q = 0; q < PER; ++q) l[q] = p.scale * (l[q] * over) * (each[q] - dot * over);
    } else {
      const float term = id >= 0 ? p.scale * d * (expf(fminf(lj, FLT_MAX) - top) * over) : 0.f;
      dot = term;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
#pragma unroll
      for (int q = 0; q < PER; ++q) l[q] *= -dot * over;
      for (int j = 0; j < p.k; ++j) {
        const int i = __shfl_sync(kAll, id, j, L);
        const float x = __shfl_sync(kAll, term, j, L);
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (i == q * L + lane) l[q] += x;
      }
    }
    if (live)
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (q * L + lane < N) grad_logits[t * N + q * L + lane] = l[q];
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

cgtp_status route_checks(cgtp_router r, int64_t n) {
  if (!r) return fail(CGTP_ERR_NULL, "router is NULL");
  if (n < 0 || n >= (int64_t(1) << 31)) return fail(CGTP_ERR_SIZE, "n out of range");
  return CGTP_OK;
}

constexpr int kSms = 148;

template <class... KArgs, class... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), int64_t grid, unsigned block, size_t shared, cudaStream_t s,
                             Args... args) {
  if (shared > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
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

// i / n = umulhi(i, magic) for i < 2^16 (a tile's values), n > 1
unsigned divide_by(int n) { return (unsigned)((uint64_t(1) << 32) / n + 1); }

struct RouteOut {
  int32_t* ids;
  float *weights, *gates;
  int64_t ld;
  int32_t* counts;
};

template <int PER>
cudaError_t forward_warps(const RouteSpec& p, int64_t n, const float* logits, const float* bias, const RouteOut& o,
                          cudaStream_t s) {
  return launch_dependent(route_warp_kernel<PER>, std::min<int64_t>((n + 7) / 8, kSms * 8), 256, 0, s, p, n, logits,
                          bias, o.ids, o.weights, o.gates, o.ld, o.counts);
}

template <int K>
cudaError_t forward_threads(const RouteSpec& p, int64_t n, const float* logits, const float* bias, const RouteOut& o,
                            cudaStream_t s) {
  const int swap_rows = std::max(std::max(K + 1, 2), p.groups);
  const size_t shared = sizeof(float) * ((size_t)(kTile + 1) * p.n + (kTile / 16 + 2) * p.n + 4 + (size_t)(4 + swap_rows) * kTile);
  // Short rows: the resident CTAs go on from tile to tile, since starting one (the biases,
  // its counts into the whole) weighs beside a tile; long ones: a CTA a tile, so that
  // those with rows to decide in 64 bits hold up no others.  Measured, going on / a
  // CTA a tile, us: 300,000 x 8: 17.3 / 20.7; 400,000 x 16: 27 / 31; 500,000 x 32: 54 / 55;
  // 172,050 x 48: 25.9 / 26.8; 300,000 x 64, k = 4: 85 / 76; 172,050 x 96: 110 / 90.
  const int64_t grid = std::min<int64_t>((n + kTile - 1) / kTile, kSms * (p.n <= 32 ? 512 / kTile : 128));
  auto kernel = !bias && p.groups == 1 ? route_thread_kernel<K, false, true>
                : p.sigmoid            ? route_thread_kernel<K, true, false>
                                       : route_thread_kernel<K, false, false>;
  return launch_dependent(kernel, grid, 2 * kTile, shared, s, p, n, logits, bias, o.ids, o.weights, o.gates, o.ld,
                          o.counts, divide_by(p.n));
}

template <int K>
cudaError_t backward_chosen(const RouteSpec& p, int64_t n, const float* logits, const int32_t* ids, const float* gw,
                            const float* gg, int64_t ld, float* out, cudaStream_t s) {
  const unsigned rows = p.n <= 64 ? kRows : p.n <= 256 ? 64 : 32;  // tiles of 33 to 66 KB
  return launch_dependent(route_chosen_backward_kernel<K>, std::min<int64_t>((n + rows - 1) / rows, kSms * 64), 2 * rows,
                          sizeof(float) * rows * (p.n | 1), s, p, n, logits, ids, gw, gg, ld, out, divide_by(p.n));
}

template <int L, int PER>
cudaError_t backward_every(const RouteSpec& p, int64_t n, const float* logits, const int32_t* ids, const float* gw,
                           const float* gg, int64_t ld, float* out, cudaStream_t s) {
  constexpr int rows = 256 / L;
  return launch_dependent(route_every_backward_kernel<L, PER>, std::min<int64_t>((n + rows - 1) / rows, kSms * 32), 256,
                          0, s, p, n, logits, ids, gw, gg, ld, out);
}

cudaError_t launch_backward(const RouteSpec& p, int64_t n, const float* logits, const int32_t* ids, const float* gw,
                            const float* gg, int64_t ld, float* out, cudaStream_t s) {
  auto run = backward_chosen<kMaxK>;
  if (!p.sigmoid && !p.renormalise) {
    run = p.n <= 4     ? backward_every<4, 1>
          : p.n <= 8   ? backward_every<8, 1>
          : p.n <= 16  ? backward_every<16, 1>
          : p.n <= 32  ? backward_every<32, 1>
          : p.n <= 64  ? backward_every<32, 2>
          : p.n <= 128 ? backward_every<32, 4>
          : p.n <= 256 ? backward_every<32, 8>
                       : backward_every<32, 16>;
  } else if (p.k <= 8) {
    run = p.k == 1   ? backward_chosen<1>
          : p.k == 2 ? backward_chosen<2>
          : p.k <= 4 ? backward_chosen<4>
                     : backward_chosen<8>;
  }
  return run(p, n, logits, ids, gw, gg, ld, out, s);
}

cudaError_t launch_forward(const RouteSpec& p, int64_t n, const float* logits, const float* bias, const RouteOut& o,
                           cudaStream_t s) {
  // A thread's row is one long chain, whatever their number; warps take their rows
  // side by side until the SMs are full.  Measured, threads / warps, us: 64 experts, k =
  // 8: 1,000 rows 12.4 / 10.5, 4,000 12.4 / 20.5, 20,000 20.6 / 75; 128 experts, k = 8:
  // 4,000 31 / 16, 10,000 31 / 31, 60,000 53 / 152; 32 experts, k = 2: 1,000 8.2 / 6.3,
  // 4,000 8.3 / 10.4; 16 experts, k = 8: 1,000 9.7 / 8.2, 4,000 11.9 / 12.4.
  if (p.k <= kThreadK && p.n <= kThreadExperts && n >= std::max(1500, p.n * p.n / 2)) {
    if (p.k == 1) return forward_threads<1>(p, n, logits, bias, o, s);
    if (p.k == 2) return forward_threads<2>(p, n, logits, bias, o, s);
    if (p.k <= 4) return forward_threads<4>(p, n, logits, bias, o, s);
    return forward_threads<8>(p, n, logits, bias, o, s);
  }
  if (p.n <= 32) return forward_warps<1>(p, n, logits, bias, o, s);
  if (p.n <= 64) return forward_warps<2>(p, n, logits, bias, o, s);
  if (p.n <= 128) return forward_warps<4>(p, n, logits, bias, o, s);
  if (p.n <= 256) return forward_warps<8>(p, n, logits, bias, o, s);
  return forward_warps<16>(p, n, logits, bias, o, s);
}

}  // namespace

}  // namespace cgtp

struct cgtp_router_s {
  cgtp::RouteSpec p;
};

using namespace cgtp;

extern "C" {

cgtp_status cgtp_router_create(int n_experts, int k, int score, int n_groups, int top_groups, int group_best,
                               int renormalise, double scale, cgtp_router* out) {
  if (!out) return fail(CGTP_ERR_NULL, "out is NULL");
  *out = nullptr;
  if (n_experts < 1 || n_experts > kMaxExperts) return fail(CGTP_ERR_SIZE, "n_experts must be in 1..512");
  if (score != CGTP_ROUTE_SOFTMAX && score != CGTP_ROUTE_SIGMOID) return fail(CGTP_ERR_SIZE, "unknown score");
  if (n_groups < 1 || n_groups > kMaxGroups || n_experts % n_groups)
    return fail(CGTP_ERR_SIZE, "n_groups must be in 1..32 and divide n_experts");
  if (top_groups < 1 || top_groups > n_groups) return fail(CGTP_ERR_SIZE, "top_groups must be in 1..n_groups");
  if (group_best != 1 && group_best != 2) return fail(CGTP_ERR_SIZE, "group_best must be 1 or 2");
  if (k < 1 || k > kMaxK || k > top_groups * (n_experts / n_groups))
    return fail(CGTP_ERR_SIZE, "k must be in 1..32 and at most the experts of top_groups groups");
  if (!((float)scale > 0.f) || !std::isfinite((float)scale))
    return fail(CGTP_ERR_SIZE, "scale must be positive and finite");
  try {
    auto h = std::make_unique<cgtp_router_s>();
    h->p = RouteSpec{n_experts, k, score == CGTP_ROUTE_SIGMOID, n_groups, top_groups, group_best, renormalise != 0,
                     (float)scale};
    *out = h.release();
  } catch (...) {
    return fail(CGTP_ERR_OOM, "host allocation failed");
  }
  return CGTP_OK;
}

cgtp_status cgtp_router_destroy(cgtp_router router) {
  delete router;
  return CGTP_OK;
}

cgtp_status cgtp_router_forward(cgtp_router router, int64_t n, const float* logits, const float* bias, int32_t* ids,
                                float* weights, float* gates, int64_t ld, int32_t* counts, cgtp_stream stream) {
  NvtxRange nvtx_range("cgtp_router_forward");
  cgtp_status st = route_checks(router, n);
  if (st != CGTP_OK) return st;
  const RouteSpec& p = router->p;
  cudaStream_t s = (cudaStream_t)stream;
  if (gates && (ld < n || ld % 4)) return fail(CGTP_ERR_SIZE, "ld must be at least n and a multiple of 4");
  if (n > 0 && !logits) return fail(CGTP_ERR_NULL, "logits is NULL");
  for (const void* q : {(const void*)logits, (const void*)bias, (const void*)ids, (const void*)weights,
                        (const void*)gates, (const void*)counts})
    if (q && !aligned16(q)) return fail(CGTP_ERR_ALIGN, "arrays must be 16-byte aligned");
  if (counts) CGTP_CUDA_TRY(cudaMemsetAsync(counts, 0, (size_t)p.n * 4, s));
  if (n == 0 || (!ids && !weights && !gates && !counts)) return CGTP_OK;
  CGTP_CUDA_TRY(launch_forward(p, n, logits, bias, {ids, weights, gates, ld, counts}, s));
  return CGTP_OK;
}

cgtp_status cgtp_router_backward(cgtp_router router, int64_t n, const float* logits, const int32_t* ids,
                                 const float* grad_weights, const float* grad_gates, int64_t ld, float* grad_logits,
                                 cgtp_stream stream) {
  NvtxRange nvtx_range("cgtp_router_backward");
  cgtp_status st = route_checks(router, n);
  if (st != CGTP_OK) return st;
  if (grad_gates && ld < n) return fail(CGTP_ERR_SIZE, "ld must be at least n");
  if (n == 0) return CGTP_OK;
  if (!logits || !ids || !grad_logits) return fail(CGTP_ERR_NULL, "logits, ids or grad_logits is NULL");
  for (const void* q : {(const void*)logits, (const void*)ids, (const void*)grad_weights, (const void*)grad_gates,
                        (const void*)grad_logits})
    if (q && !aligned16(q)) return fail(CGTP_ERR_ALIGN, "arrays must be 16-byte aligned");
  CGTP_CUDA_TRY(launch_backward(router->p, n, logits, ids, grad_weights, grad_gates, ld, grad_logits,
                                (cudaStream_t)stream));
  return CGTP_OK;
}

}  // extern "C"
