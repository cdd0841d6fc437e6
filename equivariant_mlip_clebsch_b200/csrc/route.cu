// route.cu -- routing of edges to experts (include/cgtp.h: cgtp_router_*).
//
// A row's logits l over n experts give scores s = softmax(l) or sigmoid(l); v =
// s + bias is compared, within the best groups, and the k best experts get the
// weights scale s_j (over the chosen ones' sum, if renormalised).
//
// The choice has to be that of 64 bits: scores next to one another differ by
// less than FP32's rounding.  With many rows a thread takes a row and decides in
// FP32 what its error bound lets it decide; the rare rest, and every row where
// rows are few or wide, is decided by a warp in 64 bits.
#include <cuda_runtime.h>

#include <cfloat>
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

template <class X>
__device__ __forceinline__ X warp_sum(X v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The best (largest value, lowest index) of the warp's pairs.
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(kAll, v, o);
    const int j = __shfl_xor_sync(kAll, i, o);
    if (w > v || (w == v && j < i)) {
      v = w;
      i = j;
    }
  }
}

__device__ __forceinline__ bool there(float l) { return l > -FLT_MAX; }

// One row by one warp with every compared value in 64 bits; lane i holds the
// experts i, i + 32, ... (PER of them).  Lane j returns the j-th choice and
// its weight (-1 and 0 where nothing is left).
template <int PER>
__device__ __forceinline__ void route_row(const RouteSpec& p, const float* row, const float* bias, int* id_out,
                                          float* w_out) {
  const int lane = threadIdx.x & 31, size = p.n / p.groups;
  double s[PER], v[PER];
  float top = -FLT_MAX;
  unsigned on = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = q * 32 + lane;
    const float l = e < p.n ? row[e] : -FLT_MAX;
    if (there(l)) {
      on |= 1u << q;
      top = fmaxf(top, fminf(l, FLT_MAX));
    }
    s[q] = (double)fminf(l, FLT_MAX);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  double total = 0.0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    s[q] = !(on >> q & 1) ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-s[q])) : exp(s[q] - (double)top);
    total += s[q];
  }
  if (!p.sigmoid) {
    total = warp_sum(total);
#pragma unroll
    for (int q = 0; q < PER; ++q) s[q] = total > 0.0 ? s[q] / total : 0.0;
  }
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    v[q] = -INFINITY;
    if (on >> q & 1) {
      // without bias and groups the logits' own order, which the scores lose where they saturate
      v[q] = bias ? s[q] + (double)bias[q * 32 + lane]
             : p.groups > 1 ? s[q]
                            : (double)fminf(row[q * 32 + lane], FLT_MAX);
      if (!(v[q] > -INFINITY)) v[q] = -INFINITY;
    }
  }
  if (p.groups > 1) {
    double mine = -INFINITY;  // lane g: the score of group g
    for (int g = 0; g < p.groups; ++g) {
      double sum = -INFINITY;
      int taken = -1;
      for (int r = 0; r < p.group_best; ++r) {
        double b = -INFINITY;
        int at = kMaxExperts;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          const int e = q * 32 + lane;
          if (e >= g * size && e < (g + 1) * size && e != taken && v[q] > b) {
            b = v[q];
            at = e;
          }
        }
        warp_best(b, at);
        if (b > -INFINITY) sum = r == 0 ? b : sum + b;
        taken = at;
      }
      if (lane == g) mine = sum;
    }
    unsigned kept = 0;
    for (int r = 0; r < p.top_groups; ++r) {
      double b = lane < p.groups && !(kept >> lane & 1) ? mine : -INFINITY;
      int at = b > -INFINITY ? lane : 64;
      warp_best(b, at);
      if (at < 32) kept |= 1u << at;
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * 32 + lane;
      if (e < p.n && !(kept >> (e / size) & 1)) v[q] = -INFINITY;
    }
  }
  int id = -1;
  for (int j = 0; j < p.k; ++j) {
    double b = -INFINITY;
    int at = kMaxExperts;
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (v[q] > b) {
        b = v[q];
        at = q * 32 + lane;
      }
    warp_best(b, at);
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (q * 32 + lane == at) v[q] = -INFINITY;
    if (lane == j && at < kMaxExperts) id = at;
  }
  // The weights.  Renormalised ones relative to the largest chosen logit (for
  // the sigmoid where that is negative): the chosen scores may all lie below
  // the smallest float.
  const double l = id >= 0 ? (double)fminf(row[id], FLT_MAX) : 0.0;
  double w = 0.0;
  if (!p.renormalise) {
    if (id >= 0) w = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / total;
  } else {
    double m = id >= 0 ? l : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
    if (p.sigmoid) m = fmin(m, 0.0);
    if (id >= 0) w = !p.sigmoid ? exp(l - m) : l <= 0.0 ? exp(l - m) / (1.0 + exp(l)) : 1.0 / (1.0 + exp(-l));
    const double sum = warp_sum(w);
    if (id >= 0) w /= sum;
  }
  *id_out = id;
  *w_out = (float)((double)p.scale * w);
}

// ---- forward, one warp a row, eight rows a CTA (few rows, many experts, k > 8)

template <int PER>
__global__ void __launch_bounds__(256) route_warp_kernel(RouteSpec p, int64_t n, const float* __restrict__ logits,
                                                         const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights, float* __restrict__ gates,
                                                         int64_t ld, int32_t* __restrict__ counts) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ float tile[PER * 32 * 9];  // gates of eight rows, [expert][9]
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  for (int64_t t0 = (int64_t)blockIdx.x * 8; t0 < n; t0 += (int64_t)gridDim.x * 8) {
    const int64_t t = t0 + r;
    if (t < n) {  // whole warps
      int id;
      float w;
      route_row<PER>(p, logits + t * p.n, bias, &id, &w);
      if (lane < p.k) {
        if (ids) ids[t * p.k + lane] = id;
        if (weights) weights[t * p.k + lane] = w;
        if (counts && id >= 0) atomicAdd(counts + id, 1);
      }
      if (gates) {
#pragma unroll
        for (int q = 0; q < PER; ++q) tile[(q * 32 + lane) * 9 + r] = 0.f;
        __syncwarp();
        if (id >= 0) tile[id * 9 + r] = w;
      }
    }
    if (gates) {
      __syncthreads();
      for (int i = threadIdx.x; i < p.n * 8; i += 256)
        if (t0 + (i & 7) < n) gates[(int64_t)(i >> 3) * ld + t0 + (i & 7)] = tile[(i >> 3) * 9 + (i & 7)];
      __syncthreads();
    }
  }
}

// ---- forward, one thread a row (many rows)

constexpr int kRows = 128;         // rows of a CTA's tile
constexpr int kThreadExperts = 128;  // the widest row of this form
constexpr int kThreadK = 8;

__device__ __forceinline__ float quick_sigmoid(float l) { return __fdividef(1.f, 1.f + __expf(-l)); }

// A row's choice in FP32, by one thread.  Two compared values are off by at
// most `tol` against one another; where a decision is closer than that the row
// is marked (unless the two have equal logits and biases) and decided again in
// 64 bits by the whole warp.
//   sigmoid: 1 / (1 + __expf(-l)): the exponent's rounding and the function's error
//   give s (1 - s) (|l| 2^-24 + 2^-22) < 8e-8, the division 2 ulp: |ds| < 2e-7
//   softmax: exp(l - top) off by < 2.7e-7 in the same way; the sum's relative
//   error, eight partial sums, (n / 8 + 4) 2^-24, is common to all scores <= 1
//   adding the bias rounds by 2^-24 |v|
// and a group's score adds two such values.
template <int K, bool SIGMOID, bool BY_LOGIT>
__global__ void __launch_bounds__(kRows) route_thread_kernel(RouteSpec p, int64_t n, const float* __restrict__ logits,
                                                             const float* __restrict__ bias,
                                                             int32_t* __restrict__ ids, float* __restrict__ weights,
                                                             float* __restrict__ gates, int64_t ld,
                                                             int32_t* __restrict__ counts, unsigned magic) {
  grid_dependency_wait();
  grid_launch_dependents();
  extern __shared__ float smem[];
  const int stride = p.n | 1, tid = threadIdx.x, lane = tid & 31;
  float* tile = smem;                                // [kRows][stride]
  float* sb = tile + kRows * stride;                 // [n] bias
  int* hist = reinterpret_cast<int*>(sb + p.n);      // [n]
  float* gsc = reinterpret_cast<float*>(hist + p.n);  // [groups][kRows]
  for (int e = tid; e < p.n; e += kRows) {
    sb[e] = bias ? __ldg(bias + e) : 0.f;
    hist[e] = 0;
  }
  const float base = SIGMOID ? 4e-7f : 6e-7f + (float)(p.n / 8 + 4) * 6e-8f;
  const int size = p.n / p.groups;
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < n; t0 += (int64_t)gridDim.x * kRows) {
    const int rows = (int)min((int64_t)kRows, n - t0);
    __syncthreads();  // the tile of the round before is read
    const float* src = logits + t0 * p.n;  // kRows p.n values from a 16-byte border
    for (int i = tid * 4; i < rows * p.n; i += kRows * 4) {
      float x[4];
      if (i + 3 < rows * p.n) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(src + i));
        x[0] = f.x;
        x[1] = f.y;
        x[2] = f.z;
        x[3] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = i + j < rows * p.n ? __ldg(src + i + j) : 0.f;
      }
      int r = p.n == 1 ? i : (int)__umulhi(i, magic), c = i - r * p.n;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r < rows) tile[r * stride + c] = x[j];
        if (++c == p.n) {
          c = 0;
          ++r;
        }
      }
    }
    __syncthreads();
    const bool live = tid < rows;
    const int64_t t = t0 + tid;
    const float* row = tile + (live ? tid : 0) * stride;
    float top = -FLT_MAX, total = 0.f;
    if (!SIGMOID && !(BY_LOGIT && (p.renormalise || p.sigmoid))) {
      for (int e = 0; e < p.n; ++e) top = fmaxf(top, there(row[e]) ? fminf(row[e], FLT_MAX) : -FLT_MAX);
      float part[8] = {};
      for (int e = 0; e < p.n; e += 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float l = e + j < p.n ? row[e + j] : -FLT_MAX;
          part[j] += there(l) ? __expf(fminf(l, FLT_MAX) - top) : 0.f;
        }
      total = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
    }
    const float over = total > 0.f ? 1.f / total : 0.f;
    auto value = [&](int e) {  // what is compared; -inf where the expert is out
      const float l = row[e];
      if (BY_LOGIT) return there(l) ? fminf(l, FLT_MAX) : -INFINITY;
      const float s = SIGMOID ? quick_sigmoid(l) : __expf(fminf(l, FLT_MAX) - top) * over;
      return there(l) ? fmaxf(s + sb[e], -INFINITY) : -INFINITY;  // fmaxf drops a NaN
    };
    bool doubt = false;
    unsigned kept = 1;
    if (p.groups > 1) {
      for (int g = 0; g < p.groups; ++g) {
        float b1 = -INFINITY, b2 = -INFINITY;
        for (int i = 0; i < size; ++i) {
          const float v = value(g * size + i);
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
        }
        gsc[g * kRows + tid] = p.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
      }
      kept = 0;
      float last = INFINITY;
      for (int r = 0; r < p.top_groups; ++r) {
        float best = -INFINITY;
        int at = -1;
        for (int g = 0; g < p.groups; ++g) {
          const float x = gsc[g * kRows + tid];
          if (!(kept >> g & 1) && x > best) {
            best = x;
            at = g;
          }
        }
        if (at >= 0) {
          kept |= 1u << at;
          last = best;
        }
      }
      float next = -INFINITY;
      for (int g = 0; g < p.groups; ++g)
        if (!(kept >> g & 1)) next = fmaxf(next, gsc[g * kRows + tid]);
      doubt = next > -INFINITY && !(last - next > 4.f * base + 2.4e-7f * (fabsf(last) + fabsf(next)));
    }
    float val[K + 1];
    int idx[K + 1];
#pragma unroll
    for (int j = 0; j <= K; ++j) {
      val[j] = -INFINITY;
      idx[j] = -1;
    }
    for (unsigned left = kept; left; left &= left - 1) {
      const int e0 = (__ffs(left) - 1) * size;
      for (int i = 0; i < size; ++i) {
        float v = value(e0 + i);
        int at = e0 + i;
        if (v > val[K]) {
          bool up = false;  // from its place on, all move down by one: equal ones keep their order
#pragma unroll
          for (int j = 0; j <= K; ++j) {
            up |= v > val[j];
            const float a = up ? v : val[j];
            const int b = up ? at : idx[j];
            v = up ? val[j] : v;
            at = up ? idx[j] : at;
            val[j] = a;
            idx[j] = b;
          }
        }
      }
    }
    // close decisions
    auto apart = [&](float a, float b) { return BY_LOGIT ? a > b : a - b > 2.f * base + 1.2e-7f * (fabsf(a) + fabsf(b)); };
    bool close = false;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < p.k && val[j + 1] > -INFINITY && !apart(val[j], val[j + 1])) close = true;
    if (close && !doubt && !BY_LOGIT) {
      // equal logits and biases are in their right order already
      int lastid = -1;
      float lastv = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j < p.k && idx[j] >= 0) {
          if (j + 1 < p.k && idx[j + 1] >= 0 && !apart(val[j], val[j + 1]))
            doubt |= !(row[idx[j]] == row[idx[j + 1]] && sb[idx[j]] == sb[idx[j + 1]]);
          lastid = idx[j];
          lastv = val[j];
        }
      for (unsigned left = kept; left; left &= left - 1) {
        const int e0 = (__ffs(left) - 1) * size;
        for (int i = 0; i < size; ++i) {
          const int e = e0 + i;
          const float v = value(e);
          bool chosen = false;
#pragma unroll
          for (int j = 0; j < K; ++j) chosen |= j < p.k && idx[j] == e;
          if (!chosen && v > -INFINITY && !apart(lastv, v)) doubt |= !(row[e] == row[lastid] && sb[e] == sb[lastid]);
        }
      }
    }
    doubt = doubt && live;
    // weights of the chosen, in order
    float w[K];
    {
      float m = -FLT_MAX, sum = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (j >= p.k) idx[j] = -1;
        w[j] = idx[j] >= 0 ? fminf(row[max(idx[j], 0)], FLT_MAX) : 0.f;
        if (idx[j] >= 0) m = fmaxf(m, w[j]);
      }
      if (SIGMOID || (BY_LOGIT && p.sigmoid)) {
        m = p.renormalise ? fminf(m, 0.f) : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (idx[j] >= 0)
            w[j] = w[j] > 0.f || !p.renormalise ? 1.f / (1.f + expf(-w[j])) : expf(w[j] - m) / (1.f + expf(w[j]));
      } else {
        m = p.renormalise ? m : top;
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (idx[j] >= 0) w[j] = expf(w[j] - m);
      }
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (idx[j] >= 0) sum += w[j];
      const float f = !p.renormalise ? (p.sigmoid ? p.scale : p.scale * over) : sum > 0.f ? p.scale / sum : 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) w[j] = idx[j] >= 0 ? w[j] * f : 0.f;
    }
    if (live && !doubt) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j < p.k) {
          if (ids) ids[t * p.k + j] = idx[j];
          if (weights) weights[t * p.k + j] = w[j];
          if (counts && idx[j] >= 0) atomicAdd(hist + idx[j], 1);
        }
    }
    if (gates && live) {
      for (int e = 0; e < p.n; ++e) gates[(int64_t)e * ld + t] = 0.f;  // a warp writes 32 rows of one expert
      if (!doubt) {
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (idx[j] >= 0) gates[(int64_t)idx[j] * ld + t] = w[j];
      }
    }
    __syncwarp();
    for (unsigned left = __ballot_sync(kAll, doubt); left; left &= left - 1) {
      const int r = __ffs(left) - 1;
      const int64_t tr = t0 + (tid & ~31) + r;
      int id;
      float wj;
      route_row<kThreadExperts / 32>(p, tile + ((tid & ~31) + r) * stride, bias, &id, &wj);
      if (lane < p.k) {
        if (ids) ids[tr * p.k + lane] = id;
        if (weights) weights[tr * p.k + lane] = wj;
        if (id >= 0) {
          if (counts) atomicAdd(hist + id, 1);
          if (gates) gates[(int64_t)id * ld + tr] = wj;
        }
      }
    }
  }
  if (counts) {
    __syncthreads();
    for (int e = tid; e < p.n; e += kRows)
      if (hist[e]) atomicAdd(counts + e, hist[e]);
  }
}

// ---- backward, one thread a row: the gradient is built in shared memory and
// written in whole lines

__global__ void __launch_bounds__(kRows) route_backward_kernel(RouteSpec p, int64_t n, const float* __restrict__ logits,
                                                               const int32_t* __restrict__ ids,
                                                               const float* __restrict__ grad_weights,
                                                               const float* __restrict__ grad_gates, int64_t ld,
                                                               float* __restrict__ grad_logits, unsigned magic) {
  grid_dependency_wait();
  grid_launch_dependents();
  extern __shared__ float smem[];
  const int stride = p.n | 1, tid = threadIdx.x, R = blockDim.x;
  const bool every = !p.sigmoid && !p.renormalise;  // the softmax's sum reaches every logit
  for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < n; t0 += (int64_t)gridDim.x * R) {
    const int rows = (int)min((int64_t)R, n - t0);
    __syncthreads();
    if (every) {
      const float* src = logits + t0 * p.n;
      for (int i = tid; i < rows * p.n; i += R) {
        const int r = p.n == 1 ? i : (int)__umulhi(i, magic);
        smem[r * stride + i - r * p.n] = __ldg(src + i);
      }
    } else {
      for (int i = tid; i < rows * stride; i += R) smem[i] = 0.f;
    }
    __syncthreads();
    if (tid < rows) {
      const int64_t t = t0 + tid;
      const float* row = logits + t * p.n;
      float* out = smem + tid * stride;
      auto chosen = [&](int j, float& l, float& d) {
        const int id = __ldg(ids + t * p.k + j);
        if ((unsigned)id >= (unsigned)p.n) return -1;
        l = __ldg(row + id);
        if (!there(l)) return -1;
        l = fminf(l, FLT_MAX);
        d = (grad_weights ? __ldg(grad_weights + t * p.k + j) : 0.f) +
            (grad_gates ? __ldg(grad_gates + (int64_t)id * ld + t) : 0.f);
        return id;
      };
      float l, d;
      if (every) {
        float top = -FLT_MAX, total = 0.f, dot = 0.f;
        for (int e = 0; e < p.n; ++e) top = fmaxf(top, there(out[e]) ? fminf(out[e], FLT_MAX) : -FLT_MAX);
        for (int e = 0; e < p.n; ++e) total += there(out[e]) ? expf(fminf(out[e], FLT_MAX) - top) : 0.f;
        const float over = total > 0.f ? 1.f / total : 0.f;
        for (int j = 0; j < p.k; ++j)
          if (chosen(j, l, d) >= 0) dot = fmaf(d, expf(l - top) * over, dot);
        dot *= p.scale;
        for (int e = 0; e < p.n; ++e)
          out[e] = there(out[e]) ? -(expf(fminf(out[e], FLT_MAX) - top) * over) * dot : 0.f;
        for (int j = 0; j < p.k; ++j) {
          const int id = chosen(j, l, d);
          if (id >= 0) out[id] += p.scale * d * (expf(l - top) * over);
        }
      } else {
        float m = p.sigmoid ? 0.f : -FLT_MAX, sum = 0.f, dot = 0.f;
        if (p.renormalise) {
          float top = -FLT_MAX;
          for (int j = 0; j < p.k; ++j)
            if (chosen(j, l, d) >= 0) top = fmaxf(top, l);
          m = p.sigmoid ? fminf(top, 0.f) : top;
        }
        // a score relative to exp(m)
        auto score = [&](float x) {
          if (!p.sigmoid) return expf(x - m);
          return x > 0.f || !p.renormalise ? 1.f / (1.f + expf(-x)) : expf(x - m) / (1.f + expf(x));
        };
        if (p.renormalise) {
          for (int j = 0; j < p.k; ++j)
            if (chosen(j, l, d) >= 0) {
              const float s = score(l);
              sum += s;
              dot = fmaf(d, s, dot);
            }
          sum = sum > 0.f ? 1.f / sum : 0.f;
          dot *= sum;
        }
        for (int j = 0; j < p.k; ++j) {
          const int id = chosen(j, l, d);
          if (id < 0) continue;
          float x = p.scale * score(l);
          x *= p.renormalise ? sum * (d - dot) : d;
          if (p.sigmoid) x *= 1.f / (1.f + expf(l));
          out[id] += x;
        }
      }
    }
    __syncthreads();
    float* dst = grad_logits + t0 * p.n;
    for (int i = tid; i < rows * p.n; i += R) {
      const int r = p.n == 1 ? i : (int)__umulhi(i, magic);
      dst[i] = smem[r * stride + i - r * p.n];
    }
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
  const size_t shared = sizeof(float) * ((size_t)kRows * (p.n | 1) + 2 * p.n + (p.groups > 1 ? p.groups * kRows : 0));
  const int64_t grid = std::min<int64_t>((n + kRows - 1) / kRows, kSms * 8);
  auto kernel = !bias && p.groups == 1 ? route_thread_kernel<K, false, true>
                : p.sigmoid            ? route_thread_kernel<K, true, false>
                                       : route_thread_kernel<K, false, false>;
  return launch_dependent(kernel, grid, kRows, shared, s, p, n, logits, bias, o.ids, o.weights, o.gates, o.ld,
                          o.counts, divide_by(p.n));
}

cudaError_t launch_forward(const RouteSpec& p, int64_t n, const float* logits, const float* bias, const RouteOut& o,
                           cudaStream_t s) {
  if (p.k <= kThreadK && p.n <= kThreadExperts && (n >= kSms * kRows || p.n <= 16)) {
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
  const RouteSpec& p = router->p;
  const unsigned rows = p.n <= 64 ? kRows : p.n <= 256 ? 64 : 32;  // tiles of 33 to 66 KB
  const int64_t grid = std::min<int64_t>((n + rows - 1) / rows, kSms * 12);
  CGTP_CUDA_TRY(launch_dependent(route_backward_kernel, grid, rows, sizeof(float) * rows * (p.n | 1),
                                 (cudaStream_t)stream, p, n, logits, ids, grad_weights, grad_gates, ld, grad_logits,
                                 divide_by(p.n)));
  return CGTP_OK;
}

}  // extern "C"
