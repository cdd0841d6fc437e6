// route.cu -- routing of edges to experts (include/cgtp.h: cgtp_router_*).
//
// A row's logits l over n experts give scores s = softmax(l) or sigmoid(l); v =
// s + bias is compared, within the best groups, and the k best experts get the
// weights scale s_j (over the chosen ones' sum, if renormalised).
//
// One warp takes one row, lane i the experts i, i + 32, ...; the values that
// are compared are held in 64 bits (scores next to one another differ by less
// than the rounding of FP32).
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
constexpr int kPer = kMaxExperts / 32;
constexpr unsigned kAll = 0xffffffffu;

struct RouteSpec {
  int n, k, sigmoid, groups, top_groups, group_best, renormalise;
  float scale;
};

__device__ __forceinline__ double warp_sum(double v) {
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

__global__ void __launch_bounds__(128) route_forward_kernel(RouteSpec p, int64_t n, const float* __restrict__ logits,
                                                            const float* __restrict__ bias,
                                                            int32_t* __restrict__ ids, float* __restrict__ weights,
                                                            float* __restrict__ gates, int64_t ld,
                                                            int32_t* __restrict__ counts) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 4;
  const int size = p.n / p.groups;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); t < n; t += warps) {
    double s[kPer], v[kPer];
    float top = -FLT_MAX;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int e = q * 32 + lane;
      const float l = e < p.n ? fminf(logits[t * p.n + e], FLT_MAX) : -FLT_MAX;
      const bool on = e < p.n && there(logits[t * p.n + e]);
      s[q] = on ? (double)l : -INFINITY;
      if (on) top = fmaxf(top, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    double total = 0.0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const bool on = s[q] > -INFINITY;
      v[q] = on ? 0.0 : -INFINITY;
      s[q] = !on ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-s[q])) : exp(s[q] - (double)top);
      total += s[q];
    }
    if (!p.sigmoid) {
      total = warp_sum(total);
#pragma unroll
      for (int q = 0; q < kPer; ++q) s[q] = total > 0.0 ? s[q] / total : 0.0;
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int e = q * 32 + lane;
      if (v[q] == 0.0) {
        v[q] = bias ? s[q] + (double)bias[e] : s[q];
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
          for (int q = 0; q < kPer; ++q) {
            const int e = q * 32 + lane;
            if (e / size == g && e != taken && v[q] > b) {
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
      for (int q = 0; q < kPer; ++q) {
        const int e = q * 32 + lane;
        if (e < p.n && !(kept >> (e / size) & 1)) v[q] = -INFINITY;
      }
    }
    int id = -1;  // lane j: the j-th choice
    double sj = 0.0;
    for (int j = 0; j < p.k; ++j) {
      double b = -INFINITY;
      int at = kMaxExperts;
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (v[q] > b) {
          b = v[q];
          at = q * 32 + lane;
        }
      warp_best(b, at);
      double sb = 0.0;
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (q * 32 + lane == at) {
          sb = s[q];
          v[q] = -INFINITY;
        }
      sb = warp_sum(sb);
      if (lane == j && at < kMaxExperts) {
        id = at;
        sj = sb;
      }
    }
    const double sum = warp_sum(sj);
    const double w = id < 0 ? 0.0 : p.renormalise ? (sum > 0.0 ? sj / sum : 0.0) : sj;
    const float wj = (float)((double)p.scale * w);
    if (lane < p.k) {
      if (ids) ids[t * p.k + lane] = id;
      if (weights) weights[t * p.k + lane] = wj;
      if (counts && id >= 0) atomicAdd(counts + id, 1);
    }
    if (gates)
      for (int q = 0; q < kPer; ++q) {
        const int e = q * 32 + lane;
        float gate = 0.f;
        for (int j = 0; j < p.k; ++j) {
          const int i = __shfl_sync(kAll, id, j);
          const float x = __shfl_sync(kAll, wj, j);
          if (i == e) gate = x;
        }
        if (e < p.n) gates[(int64_t)e * ld + t] = gate;
      }
  }
}

__global__ void __launch_bounds__(128) route_backward_kernel(RouteSpec p, int64_t n, const float* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ grad_weights,
                                                             const float* __restrict__ grad_gates, int64_t ld,
                                                             float* __restrict__ grad_logits) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 4;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); t < n; t += warps) {
    const float* row = logits + t * p.n;
    int id = lane < p.k ? ids[t * p.k + lane] : -1;
    if ((unsigned)id >= (unsigned)p.n || !there(row[id])) id = -1;
    const double l = id >= 0 ? (double)fminf(row[id], FLT_MAX) : 0.0;
    double d = 0.0;
    if (id >= 0 && grad_weights) d += (double)grad_weights[t * p.k + lane];
    if (id >= 0 && grad_gates) d += (double)grad_gates[(int64_t)id * ld + t];
    const bool every = !p.sigmoid && !p.renormalise;
    float top = id >= 0 ? (float)l : -FLT_MAX;
    double total = 1.0;
    if (every)
      for (int e = lane; e < p.n; e += 32)
        if (there(row[e])) top = fmaxf(top, fminf(row[e], FLT_MAX));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    if (every) {
      total = 0.0;
      for (int e = lane; e < p.n; e += 32)
        if (there(row[e])) total += exp((double)fminf(row[e], FLT_MAX) - (double)top);
      total = warp_sum(total);
    }
    double s = 0.0;
    if (id >= 0) s = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / total;
    double dl;
    double dot = 0.0;
    if (p.renormalise) {
      const double sum = warp_sum(s);
      const double q = sum > 0.0 ? s / sum : 0.0;
      dl = p.scale * q * (d - warp_sum(d * q));
      if (p.sigmoid) dl *= 1.0 - s;
    } else if (p.sigmoid) {
      dl = p.scale * d * s * (1.0 - s);
    } else {
      dl = p.scale * d * s;
      dot = warp_sum(dl);
    }
    for (int e0 = 0; e0 < p.n; e0 += 32) {
      const int e = e0 + lane;
      double out = 0.0;
      for (int j = 0; j < p.k; ++j) {
        const int i = __shfl_sync(kAll, id, j);
        const double x = __shfl_sync(kAll, dl, j);
        if (i == e) out += x;
      }
      if (e < p.n) {
        if (every && there(row[e])) out -= exp((double)fminf(row[e], FLT_MAX) - (double)top) / total * dot;
        grad_logits[t * p.n + e] = (float)out;
      }
    }
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

cgtp_status route_checks(cgtp_router r, int64_t n) {
  if (!r) return fail(CGTP_ERR_NULL, "router is NULL");
  if (n < 0 || n >= (int64_t(1) << 31)) return fail(CGTP_ERR_SIZE, "n out of range");
  return CGTP_OK;
}

unsigned row_grid(int64_t n) { return (unsigned)std::min<int64_t>((n + 3) / 4, 148 * 16); }

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
  route_forward_kernel<<<row_grid(n), 128, 0, s>>>(p, n, logits, bias, ids, weights, gates, ld, counts);
  CGTP_CUDA_TRY(cudaGetLastError());
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
  route_backward_kernel<<<row_grid(n), 128, 0, (cudaStream_t)stream>>>(router->p, n, logits, ids, grad_weights,
                                                                      grad_gates, ld, grad_logits);
  CGTP_CUDA_TRY(cudaGetLastError());
  return CGTP_OK;
}

}  // extern "C"
