// The norms after and before a block of a residual network, with the block's
// gate and the residual's scale in the same pass, and their gradient.
//
// For one token with the block's output b, the residual x, gate g, weights p
// (after the block) and w (before the next one), each of D values:
//   u = b r1 p, r1 = (mean(b^2) + eps)^(-1/2)   (without the norm after: u = b p)
//   h = alpha x + beta g u
//   n = h r2 w, r2 = (mean(h^2) + eps)^(-1/2)
// and backward, from dh (h's gradient from what comes later) and dn, with
// m = h r2, y = b r1 (or b), v = dn w:
//   t = dh + r2 (v - m mean(v m)),   dx = alpha t
//   s = beta g t,  z = s p,  db = r1 (z - y mean(z y))   (or z)
//   dg = beta t u (summed over the row for a gate of the token)
//   dw = sum over tokens of dn m,  dp = sum over tokens of s y.
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int BN_ANY_THREADS = 256;
constexpr int BN_MAX_BLOCKS = 608;  // of a gradient launch, each with its own sums of dp and dw
constexpr long long BN_MAX_DIM = 1 << 20;

enum Gate { NO_GATE, TOKEN_GATE, VALUE_GATE };

struct BlockNormParams {
  const void *branch, *x;          // x: the residual, or (gradient) the new residual h
  void *h, *n;                     // forward
  const void *dh, *dn;             // gradient
  void *dbranch, *dx;
  const void *gate;
  void* dgate;
  const void *branch_weight, *weight;
  long long branch_ld, x_ld, h_ld, n_ld, dh_ld, dn_ld, dbranch_ld, dx_ld, gate_ld, dgate_ld;
  long long tokens, dim;
  int gate_kind, post, weight_fp32, norm;  // norm: whether n is wanted
  float alpha, beta, eps;
  float* partial;                  // gradient: [blocks][2][dim], dp and dw
};

template <typename T>
__device__ __forceinline__ float weight_of(const BlockNormParams& p, const void* w, long long d) {
  if (!w) return 1.0f;
  return p.weight_fp32 ? static_cast<const float*>(w)[d] : to_float(static_cast<const T*>(w)[d]);
}

// Sums of a and b over the block, in all of its threads.
__device__ __forceinline__ float2 block_sum(float2 v, float2* parts) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  __syncthreads();
  if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = v;
  __syncthreads();
  float2 sum = make_float2(0.0f, 0.0f);
  for (int w = 0; w < BN_ANY_THREADS / 32; ++w) sum = add2(sum, parts[w]);
  return sum;
}

// Value by value, a block a row, which it reads once for each of the formulas'
// sums: rows of any width, stride and alignment.
template <typename T, typename R>
__global__ void __launch_bounds__(BN_ANY_THREADS) ns_block_norm_any_kernel(const __grid_constant__ BlockNormParams p) {
  __shared__ float2 parts[BN_ANY_THREADS / 32];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const float inv_dim = 1.0f / p.dim;
  for (long long t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const T* b = p.branch ? static_cast<const T*>(p.branch) + t * p.branch_ld : nullptr;
    const R* x = static_cast<const R*>(p.x) + t * p.x_ld;
    const T* gv = p.gate_kind == VALUE_GATE ? static_cast<const T*>(p.gate) + t * p.gate_ld : nullptr;
    R* const h_out = p.h ? static_cast<R*>(p.h) + t * p.h_ld : nullptr;
    T* const n_out = p.n ? static_cast<T*>(p.n) + t * p.n_ld : nullptr;
    const float beta = p.gate_kind == TOKEN_GATE ? p.beta * static_cast<const float*>(p.gate)[t] : p.beta;
    float r1 = 1.0f, r2 = 1.0f;
    if (b && p.post) {
      float2 sum = make_float2(0.0f, 0.0f);
      for (long long d = threadIdx.x; d < p.dim; d += BN_ANY_THREADS) sum.x = fmaf(to_float(b[d]), to_float(b[d]), sum.x);
      r1 = rsqrtf(fmaf(block_sum(sum, parts).x, inv_dim, p.eps));
    }
    auto h_at = [&](long long d) {
      float h = p.alpha * to_float(x[d]);
      if (!b) return h;
      const float u = to_float(b[d]) * r1 * weight_of<T>(p, p.branch_weight, d);
      return fmaf(beta, gv ? to_float(gv[d]) * u : u, h);
    };
    if (n_out) {
      float2 sum = make_float2(0.0f, 0.0f);
      for (long long d = threadIdx.x; d < p.dim; d += BN_ANY_THREADS) {
        const float h = h_at(d);
        sum.x = fmaf(h, h, sum.x);
      }
      r2 = rsqrtf(fmaf(block_sum(sum, parts).x, inv_dim, p.eps));
    }
    for (long long d = threadIdx.x; d < p.dim; d += BN_ANY_THREADS) {
      const float h = h_at(d), w = weight_of<T>(p, p.weight, d);
      if (h_out) h_out[d] = from_float<R>(h);
      if (n_out) n_out[d] = from_float<T>(h * r2 * w);
    }
  }
}

template <typename T, typename R>
__global__ void __launch_bounds__(BN_ANY_THREADS) ns_block_norm_grad_any_kernel(const __grid_constant__ BlockNormParams p) {
  __shared__ float2 parts[BN_ANY_THREADS / 32];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const float inv_dim = 1.0f / p.dim;
  float* const dp = p.partial ? p.partial + static_cast<long long>(blockIdx.x) * 2 * p.dim : nullptr;
  float* const dw = dp ? dp + p.dim : nullptr;
  if (dp)
    for (long long d = threadIdx.x; d < 2 * p.dim; d += BN_ANY_THREADS) dp[d] = 0.0f;
  __syncthreads();
  for (long long t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const T* b = p.branch ? static_cast<const T*>(p.branch) + t * p.branch_ld : nullptr;
    const R* h = static_cast<const R*>(p.x) + t * p.x_ld;
    const R* dh = p.dh ? static_cast<const R*>(p.dh) + t * p.dh_ld : nullptr;
    const T* dn = p.dn ? static_cast<const T*>(p.dn) + t * p.dn_ld : nullptr;
    const T* gv = p.gate_kind == VALUE_GATE ? static_cast<const T*>(p.gate) + t * p.gate_ld : nullptr;
    const float gt = p.gate_kind == TOKEN_GATE ? static_cast<const float*>(p.gate)[t] : 1.0f;
    float2 sum = make_float2(0.0f, 0.0f);
    if (dn || (b && p.post)) {
      for (long long d = threadIdx.x; d < p.dim; d += BN_ANY_THREADS) {
        const float hv = to_float(h[d]), bv = b ? to_float(b[d]) : 0.0f;
        sum = fma2(make_float2(hv, bv), make_float2(hv, bv), sum);
      }
      sum = block_sum(sum, parts);
    }
    const float r2 = dn ? rsqrtf(fmaf(sum.x, inv_dim, p.eps)) : 1.0f;
    const float r1 = b && p.post ? rsqrtf(fmaf(sum.y, inv_dim, p.eps)) : 1.0f;
    float mean_vm = 0.0f;
    if (dn) {
      sum = make_float2(0.0f, 0.0f);
      for (long long d = threadIdx.x; d < p.dim; d += BN_ANY_THREADS)
        sum.x = fmaf(to_float(dn[d]) * weight_of<T>(p, p.weight, d), to_float(h[d]) * r2, sum.x);
      mean_vm = block_sum(sum, parts).x * inv_dim;
    }
    auto t_at = [&](long long d) {
      float v = dh ? to_float(dh[d]) : 0.0f;
      if (dn) v = fmaf(r2, to_float(dn[d]) * weight_of<T>(p, p.weight, d) - to_float(h[d]) * r2 * mean_vm, v);
      return v;
    };
    sum = make_float2(0.0f, 0.0f);
    if (b && (p.post || (p.dgate && p.gate_kind == TOKEN_GATE))) {
      for (long long d = threadIdx.x; d < p.dim; d += BN_ANY_THREADS) {
        const float tb = p.beta * t_at(d), y = to_float(b[d]) * r1, yp = y * weight_of<T>(p, p.branch_weight, d);
        sum.x = fmaf(tb * (gv ? to_float(gv[d]) : gt), yp, sum.x);
        sum.y = fmaf(tb, yp, sum.y);
      }
      sum = block_sum(sum, parts);
      if (threadIdx.x == 0 && p.dgate && p.gate_kind == TOKEN_GATE) static_cast<float*>(p.dgate)[t] = sum.y;
    }
    const float mean_zy = sum.x * inv_dim;
    // a column's inputs are read by the thread that writes there, so that outputs may take their place
    for (long long d = threadIdx.x; d < p.dim; d += BN_ANY_THREADS) {
      const float tv = t_at(d), m = to_float(h[d]) * r2, dnv = dn ? to_float(dn[d]) : 0.0f;
      const float bv = b ? to_float(b[d]) : 0.0f, g = gv ? to_float(gv[d]) : gt;
      if (dp) dw[d] = fmaf(dnv, m, dw[d]);
      if (p.dx) static_cast<R*>(p.dx)[t * p.dx_ld + d] = from_float<R>(p.alpha * tv);
      if (!b) continue;
      const float tb = p.beta * tv, s = tb * g, y = bv * r1, pw = weight_of<T>(p, p.branch_weight, d);
      if (dp) dp[d] = fmaf(s, y, dp[d]);
      if (p.dgate && p.gate_kind == VALUE_GATE) static_cast<T*>(p.dgate)[t * p.dgate_ld + d] = from_float<T>(tb * y * pw);
      if (p.dbranch)
        static_cast<T*>(p.dbranch)[t * p.dbranch_ld + d] = from_float<T>(p.post ? r1 * (s * pw - y * mean_zy) : s * pw);
    }
  }
}

struct BlockNormSumParams {
  const float* partial;  // [blocks][2 * dim]
  float* out[2];
  long long dim;
  int blocks;
};

// The weights' gradients: sums of the blocks' partial sums, in a fixed order: 32
// columns a block, whose 32 warps split the partial sums.
__global__ void __launch_bounds__(1024) ns_block_norm_sum_kernel(const __grid_constant__ BlockNormSumParams p) {
  __shared__ float part[32][33];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + lane;
  float sum = 0.0f;
  if (col < 2 * p.dim) {
#pragma unroll 8
    for (int b = warp; b < p.blocks; b += 32) sum += p.partial[b * 2 * p.dim + col];
  }
  part[warp][lane] = sum;
  __syncthreads();
  sum = warp_sum(part[lane][warp]);  // warp w: column w's parts
  const long long c = static_cast<long long>(blockIdx.x) * 32 + warp;
  if (lane || c >= 2 * p.dim) return;
  float* out = p.out[c >= p.dim];
  if (out) out[c >= p.dim ? c - p.dim : c] = sum;
}

template <typename T, typename R>
cudaError_t launch_block_norm(bool grad, const BlockNormParams& p, int nsm, int* blocks, cudaStream_t st) {
  *blocks = static_cast<int>(std::min<long long>(p.tokens, std::min(nsm * 4, BN_MAX_BLOCKS)));
  if (grad) return launch_pdl(ns_block_norm_grad_any_kernel<T, R>, dim3(*blocks), dim3(BN_ANY_THREADS), 0, st, p);
  return launch_pdl(ns_block_norm_any_kernel<T, R>, dim3(*blocks), dim3(BN_ANY_THREADS), 0, st, p);
}

}  // namespace
}  // namespace nsk

using namespace nsorch;

namespace {

cudaError_t run_block_norm(bool grad, int dtype, int residual_dtype, const nsk::BlockNormParams& p, int nsm, int* blocks,
                           cudaStream_t st) {
  return counted(K_BLOCK_NORM, st, [&] {
    if (dtype == NS_DT_FP32) return nsk::launch_block_norm<float, float>(grad, p, nsm, blocks, st);
    if (dtype == NS_DT_BF16)
      return residual_dtype == NS_DT_FP32 ? nsk::launch_block_norm<__nv_bfloat16, float>(grad, p, nsm, blocks, st)
                                          : nsk::launch_block_norm<__nv_bfloat16, __nv_bfloat16>(grad, p, nsm, blocks, st);
    return residual_dtype == NS_DT_FP32 ? nsk::launch_block_norm<__half, float>(grad, p, nsm, blocks, st)
                                        : nsk::launch_block_norm<__half, __half>(grad, p, nsm, blocks, st);
  });
}

int check_types(int dtype, int residual_dtype, int weight_dtype) {
  if (!nsk::dtype_ok(dtype)) return NS_ERR_ARG;
  if (residual_dtype != dtype && residual_dtype != NS_DT_FP32) return NS_ERR_ARG;
  if (weight_dtype != dtype && weight_dtype != NS_DT_FP32) return NS_ERR_ARG;
  return NS_OK;
}

// The sizes and numbers that both directions share.
int check_sizes(int64_t tokens, int64_t dim, int gate_kind, const void* branch, const void* gate, int post_norm, float alpha,
                float beta, float eps) {
  if (tokens < 0 || dim < 0 || gate_kind < 0 || gate_kind > 2) return NS_ERR_ARG;
  if (post_norm != 0 && post_norm != 1) return NS_ERR_ARG;
  if (!(eps >= 0.0f) || !(alpha - alpha == 0.0f) || !(beta - beta == 0.0f)) return NS_ERR_ARG;
  if (dim > nsk::BN_MAX_DIM) return NS_ERR_UNSUPPORTED;
  if (tokens > (int64_t{1} << 40) / std::max<int64_t>(1, dim)) return NS_ERR_SHAPE;
  if (tokens > 0 && dim > 0 && branch && gate_kind != nsk::NO_GATE && !gate) return NS_ERR_ARG;
  return NS_OK;
}

// Whether a matrix can be there: an aligned address, rows that do not overlap.
int check_matrix(const void* p, int64_t ld, int dtype, int64_t dim) {
  if (!p) return NS_OK;
  if (!nsk::element_aligned(p, nsk::elem_bytes(dtype))) return NS_ERR_ARG;
  return ld < dim ? NS_ERR_SHAPE : NS_OK;
}

int check_gate(const void* p, int64_t ld, int kind, int dtype, int64_t dim) {
  if (kind == nsk::NO_GATE) return NS_OK;
  if (kind == nsk::TOKEN_GATE) return nsk::element_aligned(p, 4) ? NS_OK : NS_ERR_ARG;
  return check_matrix(p, ld, dtype, dim);
}

}  // namespace

extern "C" {

int ns_block_norm(const void* branch, const void* residual, void* residual_out, void* out, const int64_t* strides,
                  int dtype, int residual_dtype, int64_t tokens, int64_t dim, const void* branch_weight,
                  const void* weight, int weight_dtype, const void* gate, int gate_kind, int post_norm,
                  float residual_scale, float branch_scale, float eps, void* stream) {
  int rc = check_types(dtype, residual_dtype, weight_dtype);
  if (rc != NS_OK) return rc;
  if (!strides) return NS_ERR_ARG;
  if ((rc = check_sizes(tokens, dim, gate_kind, branch, gate, post_norm, residual_scale, branch_scale, eps)) != NS_OK) return rc;
  if (tokens == 0 || dim == 0 || (!residual_out && !out)) return NS_OK;
  if (!residual) return NS_ERR_ARG;
  const int w = nsk::elem_bytes(weight_dtype);
  if (!nsk::element_aligned(branch_weight, w) || !nsk::element_aligned(weight, w)) return NS_ERR_ARG;
  if ((rc = check_matrix(branch, strides[0], dtype, dim)) != NS_OK) return rc;
  if ((rc = check_matrix(residual, strides[1], residual_dtype, dim)) != NS_OK) return rc;
  if ((rc = check_matrix(residual_out, strides[2], residual_dtype, dim)) != NS_OK) return rc;
  if ((rc = check_matrix(out, strides[3], dtype, dim)) != NS_OK) return rc;
  if (branch && (rc = check_gate(gate, strides[4], gate_kind, dtype, dim)) != NS_OK) return rc;
  nsk::BlockNormParams p = {};
  p.branch = branch;
  p.x = residual;
  p.h = residual_out;
  p.n = out;
  p.branch_ld = strides[0];
  p.x_ld = strides[1];
  p.h_ld = strides[2];
  p.n_ld = strides[3];
  p.gate_ld = strides[4];
  p.gate_kind = branch ? gate_kind : nsk::NO_GATE;
  p.gate = p.gate_kind == nsk::NO_GATE ? nullptr : gate;
  p.branch_weight = branch_weight;
  p.weight = weight;
  p.weight_fp32 = weight_dtype == NS_DT_FP32;
  p.tokens = tokens;
  p.dim = dim;
  p.post = post_norm;
  p.alpha = residual_scale;
  p.beta = branch_scale;
  p.eps = eps;
  int dev, nsm, blocks;
  unsigned int* status;
  if ((rc = device_setup(&dev, &status, &nsm)) != NS_OK) return rc;
  const cudaError_t e = run_block_norm(false, dtype, residual_dtype, p, nsm, &blocks, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

int ns_block_norm_grad_workspace_bytes(int64_t dim, uint64_t* bytes) {
  if (!bytes || dim < 0) return NS_ERR_ARG;
  if (dim > nsk::BN_MAX_DIM) return NS_ERR_UNSUPPORTED;
  *bytes = sizeof(float) * 2 * nsk::BN_MAX_BLOCKS * static_cast<uint64_t>(dim);
  return NS_OK;
}

int ns_block_norm_grad(const void* grad_residual_out, const void* grad_out, const void* branch, const void* residual_out,
                       void* grad_branch, void* grad_residual, const int64_t* strides, int dtype, int residual_dtype,
                       int64_t tokens, int64_t dim, const void* branch_weight, const void* weight, int weight_dtype,
                       const void* gate, int gate_kind, float* grad_branch_weight, float* grad_weight, void* grad_gate,
                       int post_norm, float residual_scale, float branch_scale, float eps, void* workspace,
                       uint64_t workspace_bytes, void* stream) {
  int rc = check_types(dtype, residual_dtype, weight_dtype);
  if (rc != NS_OK) return rc;
  if (!strides) return NS_ERR_ARG;
  if ((rc = check_sizes(tokens, dim, gate_kind, branch, gate, post_norm, residual_scale, branch_scale, eps)) != NS_OK) return rc;
  if (dim == 0) return NS_OK;
  if (!nsk::element_aligned(grad_branch_weight, 4) || !nsk::element_aligned(grad_weight, 4)) return NS_ERR_ARG;
  const bool sums = grad_branch_weight || grad_weight;
  if (sums && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
               workspace_bytes < sizeof(float) * 2 * nsk::BN_MAX_BLOCKS * static_cast<uint64_t>(dim)))
    return NS_ERR_WORKSPACE;
  if (tokens > 0) {
    if (!residual_out || (!grad_residual_out && !grad_out)) return NS_ERR_ARG;
    if (!branch && (grad_branch || grad_branch_weight || grad_gate)) return NS_ERR_ARG;
    if (grad_gate && gate_kind == nsk::NO_GATE) return NS_ERR_ARG;
    const int w = nsk::elem_bytes(weight_dtype);
    if (!nsk::element_aligned(branch_weight, w) || !nsk::element_aligned(weight, w)) return NS_ERR_ARG;
    if ((rc = check_matrix(branch, strides[0], dtype, dim)) != NS_OK) return rc;
    if ((rc = check_matrix(residual_out, strides[1], residual_dtype, dim)) != NS_OK) return rc;
    if ((rc = check_matrix(grad_branch, strides[2], dtype, dim)) != NS_OK) return rc;
    if ((rc = check_matrix(grad_residual, strides[3], residual_dtype, dim)) != NS_OK) return rc;
    if ((rc = check_matrix(grad_residual_out, strides[4], residual_dtype, dim)) != NS_OK) return rc;
    if ((rc = check_matrix(grad_out, strides[5], dtype, dim)) != NS_OK) return rc;
    if (branch && (rc = check_gate(gate, strides[6], gate_kind, dtype, dim)) != NS_OK) return rc;
    if (branch && (rc = check_gate(grad_gate, strides[7], gate_kind, dtype, dim)) != NS_OK) return rc;
  }
  int dev, nsm, blocks = 0;
  unsigned int* status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens > 0) {
    nsk::BlockNormParams p = {};
    p.branch = branch;
    p.x = residual_out;
    p.dh = grad_residual_out;
    p.dn = grad_out;
    p.dbranch = grad_branch;
    p.dx = grad_residual;
    p.branch_ld = strides[0];
    p.x_ld = strides[1];
    p.dbranch_ld = strides[2];
    p.dx_ld = strides[3];
    p.dh_ld = strides[4];
    p.dn_ld = strides[5];
    p.gate_ld = strides[6];
    p.dgate_ld = strides[7];
    p.gate_kind = branch ? gate_kind : nsk::NO_GATE;
    p.gate = p.gate_kind == nsk::NO_GATE ? nullptr : gate;
    p.dgate = grad_gate;
    p.branch_weight = branch_weight;
    p.weight = weight;
    p.weight_fp32 = weight_dtype == NS_DT_FP32;
    p.tokens = tokens;
    p.dim = dim;
    p.post = post_norm;
    p.alpha = residual_scale;
    p.beta = branch_scale;
    p.eps = eps;
    p.partial = sums ? static_cast<float*>(workspace) : nullptr;
    if ((rc = device_setup(&dev, &status, &nsm)) != NS_OK) return rc;
    if (run_block_norm(true, dtype, residual_dtype, p, nsm, &blocks, st) != cudaSuccess) return NS_ERR_CUDA;
  }
  if (!sums) return NS_OK;
  if ((rc = device_setup(&dev, &status, &nsm)) != NS_OK) return rc;
  nsk::BlockNormSumParams sp = {static_cast<const float*>(workspace), {grad_branch_weight, grad_weight}, dim, blocks};
  const cudaError_t e = counted(K_BLOCK_NORM, st, [&] {
    return nsk::launch_pdl(nsk::ns_block_norm_sum_kernel, dim3(static_cast<unsigned>((2 * dim + 31) / 32)), dim3(1024), 0, st, sp);
  });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

}  // extern "C"
