// A whole mixture-of-experts layer for a few tokens: each token's experts, their
// gated products and the weighted sum, in two kernels.
//
//   h_s = silu(G_e x_t) * (U_e x_t)     for slot s = (t, j) with expert e
//   y_t = sum over j of w_tj D_e h_s
// with silu(a) = a / (1 + exp(-a)). The hidden values h stay in fp32 between the
// kernels.
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int MF_THREADS = 256;
constexpr int MF_WARPS = MF_THREADS / 32;
constexpr int MF_MAX_TOKENS = 256;

struct MoeFewParams {
  const void *x, *gate_up, *down;
  void* y;
  const void* ids;
  int id_bytes, tokens, k, experts;
  long long x_ld, y_ld, dim, ffn;
  const float* weights;
  float* hidden;  // [tokens * k][ffn]
  unsigned int* status;
};

// The expert of a slot, -1 if it goes nowhere.
__device__ __forceinline__ int expert_of(const MoeFewParams& p, int slot) {
  const long long e = load_index(p.ids, p.id_bytes, slot);
  if (e >= p.experts) atomicOr(p.status, NS_DEV_BAD_INDEX);
  return e < 0 || e >= p.experts ? -1 : static_cast<int>(e);
}

// A warp a hidden value of a slot.
template <typename T>
__global__ void __launch_bounds__(MF_THREADS) ns_moe_few_hidden_kernel(const __grid_constant__ MoeFewParams p) {
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int slot = blockIdx.y, lane = threadIdx.x & 31, e = expert_of(p, slot);
  const long long f = static_cast<long long>(blockIdx.x) * MF_WARPS + threadIdx.x / 32;
  if (e < 0 || f >= p.ffn) return;
  const T* x = static_cast<const T*>(p.x) + (slot / p.k) * p.x_ld;
  const T* g = static_cast<const T*>(p.gate_up) + (2 * e * p.ffn + f) * p.dim;
  const T* u = g + p.ffn * p.dim;
  float a = 0.0f, b = 0.0f;
  for (long long d = lane; d < p.dim; d += 32) {
    const float v = to_float(x[d]);
    a = fmaf(to_float(g[d]), v, a);
    b = fmaf(to_float(u[d]), v, b);
  }
  a = warp_sum(a);
  b = warp_sum(b);
  if (lane == 0) p.hidden[slot * p.ffn + f] = a / (1.0f + expf(-a)) * b;
}

// A warp a value of y.
template <typename T>
__global__ void __launch_bounds__(MF_THREADS) ns_moe_few_sum_kernel(const __grid_constant__ MoeFewParams p) {
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int t = blockIdx.y, lane = threadIdx.x & 31;
  const long long d = static_cast<long long>(blockIdx.x) * MF_WARPS + threadIdx.x / 32;
  if (d >= p.dim) return;
  float y = 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int slot = t * p.k + j, e = expert_of(p, slot);
    if (e < 0) continue;
    const T* w = static_cast<const T*>(p.down) + (e * p.dim + d) * p.ffn;
    const float* h = p.hidden + slot * p.ffn;
    float sum = 0.0f;
    for (long long f = lane; f < p.ffn; f += 32) sum = fmaf(to_float(w[f]), h[f], sum);
    y = fmaf(p.weights ? p.weights[slot] : 1.0f, warp_sum(sum), y);
  }
  if (lane == 0) static_cast<T*>(p.y)[t * p.y_ld + d] = from_float<T>(y);
}

template <typename T>
int launch_few(const MoeFewParams& p, cudaStream_t st) {
  const auto blocks = [](long long n) { return static_cast<unsigned>((n + MF_WARPS - 1) / MF_WARPS); };
  cudaError_t e = nsorch::counted(nsorch::K_MOE, st, [&] {
    return launch_pdl(ns_moe_few_hidden_kernel<T>, dim3(blocks(p.ffn), p.tokens * p.k), dim3(MF_THREADS), 0, st, p);
  });
  if (e != cudaSuccess) return NS_ERR_CUDA;
  e = nsorch::counted(nsorch::K_MOE, st, [&] {
    return launch_pdl(ns_moe_few_sum_kernel<T>, dim3(blocks(p.dim), p.tokens), dim3(MF_THREADS), 0, st, p);
  });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

}  // namespace
}  // namespace nsk

using namespace nsorch;

namespace {

int check_few(int64_t tokens, int k, int64_t dim, int64_t ffn) {
  if (tokens < 0 || k < 1 || dim < 0 || ffn < 1) return NS_ERR_ARG;
  if (k > 32 || tokens > nsk::MF_MAX_TOKENS) return NS_ERR_UNSUPPORTED;
  // a matrix of an expert has fewer than 2^40 values
  if (dim >= (int64_t{1} << 20) || ffn >= (int64_t{1} << 20)) return NS_ERR_UNSUPPORTED;
  return NS_OK;
}

uint64_t few_workspace(int64_t tokens, int k, int64_t ffn) {
  return sizeof(float) * static_cast<uint64_t>(tokens) * k * static_cast<uint64_t>(ffn);
}

}  // namespace

extern "C" {

int ns_moe_few_tokens_workspace_bytes(int64_t tokens, int k, int64_t dim, int64_t ffn, uint64_t* bytes) {
  if (!bytes) return NS_ERR_ARG;
  const int rc = check_few(tokens, k, dim, ffn);
  if (rc == NS_OK) *bytes = few_workspace(tokens, k, ffn);
  return rc;
}

int ns_moe_few_tokens(const void* x, int64_t x_stride, int dtype, int64_t tokens, int k, int64_t dim, int64_t ffn,
                      int experts, const void* expert_ids, int id_bytes, const float* weights, const void* gate_up,
                      const void* down, void* y, int64_t y_stride, void* workspace, uint64_t workspace_bytes,
                      void* stream) {
  if (!nsk::dtype_ok(dtype) || (id_bytes != 4 && id_bytes != 8) || experts < 1) return NS_ERR_ARG;
  int rc = check_few(tokens, k, dim, ffn);
  if (rc != NS_OK) return rc;
  if (experts > 1024) return NS_ERR_UNSUPPORTED;
  if (tokens == 0 || dim == 0) return NS_OK;
  if (!x || !expert_ids || !y || !gate_up || !down) return NS_ERR_ARG;
  const int b = nsk::elem_bytes(dtype);
  for (const void* q : {x, gate_up, down, static_cast<const void*>(y)})
    if (!nsk::element_aligned(q, b)) return NS_ERR_ARG;
  if (!nsk::element_aligned(expert_ids, id_bytes) || !nsk::element_aligned(weights, 4)) return NS_ERR_ARG;
  if (x_stride < dim || y_stride < dim) return NS_ERR_SHAPE;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < few_workspace(tokens, k, ffn))
    return NS_ERR_WORKSPACE;
  nsk::MoeFewParams p = {};
  p.x = x;
  p.gate_up = gate_up;
  p.down = down;
  p.y = y;
  p.ids = expert_ids;
  p.id_bytes = id_bytes;
  p.tokens = static_cast<int>(tokens);
  p.k = k;
  p.experts = experts;
  p.x_ld = x_stride;
  p.y_ld = y_stride;
  p.dim = dim;
  p.ffn = ffn;
  p.weights = weights;
  p.hidden = static_cast<float*>(workspace);
  int dev, nsm;
  if ((rc = device_setup(&dev, &p.status, &nsm)) != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == NS_DT_BF16) return nsk::launch_few<__nv_bfloat16>(p, st);
  if (dtype == NS_DT_FP16) return nsk::launch_few<__half>(p, st);
  return nsk::launch_few<float>(p, st);
}

}  // extern "C"
