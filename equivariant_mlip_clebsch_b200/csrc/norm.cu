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
// One warp takes one block of one row and reads it three times (from L2 after
// the first); the weights' gradients are a second kernel over the rows with
// the statistics of the first.
#include <cuda_runtime.h>

#include <algorithm>
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// mean (0 unless centred) and 1 / sqrt(variance + eps) of one block
__device__ __forceinline__ void block_stats(const float* x, const NormBlock& b, float eps, int lane, float* mu,
                                            float* r) {
  const float inv = 1.f / (float)b.len;
  float m = 0.f;
  if (b.sc >= 0) {
    for (int i = lane; i < b.len; i += 32) m += x[i];
    m = warp_sum(m) * inv;
  }
  float v = 0.f;
  for (int i = lane; i < b.len; i += 32) {
    const float t = x[i] - m;
    v = fmaf(t, t, v);
  }
  *mu = m;
  *r = 1.f / sqrtf(warp_sum(v) * inv + eps);
}

__global__ void __launch_bounds__(256) norm_forward_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                           const float* __restrict__ x, const float* __restrict__ w,
                                                           const float* __restrict__ bias, float* __restrict__ y) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < n * t.nblocks; u += warps) {
    const NormBlock b = t.b[u % t.nblocks];
    const int64_t at = u / t.nblocks * t.D + b.off;
    float mu, r;
    block_stats(x + at, b, t.eps, lane, &mu, &r);
    for (int i = lane; i < b.len; i += 32) {
      const int c = i / b.d;
      const float v = (x[at + i] - mu) * r * (w ? w[b.ch + c] : 1.f);
      y[at + i] = b.sc >= 0 && bias ? v + bias[b.sc + c] : v;
    }
  }
}

// stats[u] = (mu, r, mean(h) if centred, mean(h xh)) of unit u = row * nblocks + block
__global__ void __launch_bounds__(256) norm_backward_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                            const float* __restrict__ x, const float* __restrict__ w,
                                                            const float* __restrict__ g, float* __restrict__ dx,
                                                            float4* __restrict__ stats) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < n * t.nblocks; u += warps) {
    const NormBlock b = t.b[u % t.nblocks];
    const int64_t at = u / t.nblocks * t.D + b.off;
    float mu, r;
    block_stats(x + at, b, t.eps, lane, &mu, &r);
    if (lane == 0 && stats) stats[u] = make_float4(mu, r, 0.f, 0.f);
    if (!dx) continue;
    float sa = 0.f, sax = 0.f;
    for (int i = lane; i < b.len; i += 32) {
      const float a = g[at + i] * (w ? w[b.ch + i / b.d] : 1.f);
      sa += a;
      sax = fmaf(a, (x[at + i] - mu) * r, sax);
    }
    const float inv = 1.f / (float)b.len;
    const float ma = b.sc >= 0 ? warp_sum(sa) * inv : 0.f;
    const float al = warp_sum(sax) * inv;
    for (int i = lane; i < b.len; i += 32) {
      const float a = g[at + i] * (w ? w[b.ch + i / b.d] : 1.f);
      dx[at + i] = r * (a - ma - (x[at + i] - mu) * r * al);
    }
  }
}

__global__ void __launch_bounds__(256) norm_double_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                          const float* __restrict__ x, const float* __restrict__ w,
                                                          const float* __restrict__ g, const float* __restrict__ hx,
                                                          const float* __restrict__ hw, const float* __restrict__ hb,
                                                          float* __restrict__ gg, float* __restrict__ gx,
                                                          float4* __restrict__ stats) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < n * t.nblocks; u += warps) {
    const NormBlock b = t.b[u % t.nblocks];
    const int64_t at = u / t.nblocks * t.D + b.off;
    const float inv = 1.f / (float)b.len;
    float mu, r;
    block_stats(x + at, b, t.eps, lane, &mu, &r);
    float sa = 0.f, sh = 0.f, sk = 0.f;
    if (b.sc >= 0) {
      for (int i = lane; i < b.len; i += 32) {
        const int c = b.ch + i / b.d;
        sa = fmaf(g[at + i], w ? w[c] : 1.f, sa);
        if (hx) sh += hx[at + i];
        if (hw) sk = fmaf(g[at + i], hw[c], sk);
      }
      sa = warp_sum(sa) * inv;
      sh = warp_sum(sh) * inv;
      sk = warp_sum(sk) * inv;
    }
    float sax = 0.f, shx = 0.f, skx = 0.f, sha = 0.f;
    for (int i = lane; i < b.len; i += 32) {
      const int c = b.ch + i / b.d;
      const float xh = (x[at + i] - mu) * r, gi = g[at + i];
      const float a = gi * (w ? w[c] : 1.f), h = hx ? hx[at + i] - sh : 0.f;
      sax = fmaf(a, xh, sax);
      shx = fmaf(h, xh, shx);
      sha = fmaf(h, a, sha);
      if (hw) skx = fmaf(gi * hw[c], xh, skx);
    }
    const float al = warp_sum(sax) * inv, be = warp_sum(shx) * inv, ga = warp_sum(sha) * inv,
                de = warp_sum(skx) * inv;
    if (lane == 0 && stats) stats[u] = make_float4(mu, r, sh, be);
    const float cx = 3.f * al * be - ga;
    for (int i = lane; i < b.len; i += 32) {
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

// One CTA per channel: the sums over rows and components of g xh (h null) or
// g J h, and of g for 0e channels.  stats as written above.
__global__ void __launch_bounds__(256) norm_weight_kernel(const __grid_constant__ NormTable t, int64_t n,
                                                          const float* __restrict__ x, const float* __restrict__ g,
                                                          const float* __restrict__ hx, bool second,
                                                          const float4* __restrict__ stats, float* __restrict__ dw,
                                                          float* __restrict__ db) {
  const int ch = blockIdx.x;
  int q = 0;
  while (q + 1 < t.nblocks && t.b[q + 1].ch <= ch) ++q;
  const NormBlock b = t.b[q];
  const int c = ch - b.ch;
  float sw = 0.f, sb = 0.f;
  for (int64_t i = threadIdx.x; i < n * b.d; i += 256) {
    const int64_t row = i / b.d, at = row * t.D + b.off + c * b.d + (i - row * b.d);
    const float4 s = stats[row * t.nblocks + q];
    const float xh = (x[at] - s.x) * s.y;
    const float v = second ? (hx ? s.y * (hx[at] - s.z - xh * s.w) : 0.f) : xh;
    sw = fmaf(g[at], v, sw);
    sb += g[at];
  }
  __shared__ float part[2][8];
  sw = warp_sum(sw);
  sb = warp_sum(sb);
  if ((threadIdx.x & 31) == 0) {
    part[0][threadIdx.x >> 5] = sw;
    part[1][threadIdx.x >> 5] = sb;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    sw = sb = 0.f;
    for (int k = 0; k < 8; ++k) {
      sw += part[0][k];
      sb += part[1][k];
    }
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

size_t norm_workspace(const NormTable& t, int64_t n) { return ((size_t)n * t.nblocks * sizeof(float4) + 255) & ~size_t(255); }

cgtp_status norm_workspace_check(const NormTable& t, int64_t n, const void* ws, size_t bytes) {
  const size_t need = norm_workspace(t, n);
  if (!ws || bytes < need) return fail(CGTP_ERR_WORKSPACE, "workspace of " + std::to_string(need) + " bytes required");
  if ((uintptr_t)ws & 255) return fail(CGTP_ERR_ALIGN, "workspace must be 256-byte aligned");
  return CGTP_OK;
}

unsigned unit_grid(const NormTable& t, int64_t n) {
  return (unsigned)std::min<int64_t>((n * t.nblocks + 7) / 8, 148 * 8);
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
    if (!((float)eps > 0.f) || !std::isfinite((float)eps)) return fail(CGTP_ERR_SIZE, "eps must be positive and finite");
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
  norm_forward_kernel<<<unit_grid(norm->t, n), 256, 0, (cudaStream_t)stream>>>(norm->t, n, x, weight, bias, y);
  CGTP_CUDA_TRY(cudaGetLastError());
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
  float4* stats = params ? (float4*)workspace : nullptr;
  norm_backward_kernel<<<unit_grid(t, n), 256, 0, s>>>(t, n, x, weight, grad_y, grad_x, stats);
  if (params)
    norm_weight_kernel<<<(unsigned)t.C, 256, 0, s>>>(t, n, x, grad_y, nullptr, false, stats, grad_weight, grad_bias);
  CGTP_CUDA_TRY(cudaGetLastError());
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
  float4* stats = gweight ? (float4*)workspace : nullptr;
  norm_double_kernel<<<unit_grid(t, n), 256, 0, s>>>(t, n, x, weight, grad_y, h_x, h_weight, h_bias, gg, gx, stats);
  if (gweight)
    norm_weight_kernel<<<(unsigned)t.C, 256, 0, s>>>(t, n, x, grad_y, h_x, true, stats, gweight, nullptr);
  CGTP_CUDA_TRY(cudaGetLastError());
  return CGTP_OK;
}

}  // extern "C"
