// Distillation from a teacher's top logits: the loss of each token, and its
// gradient in the student's logits.
//
// For a token with student logits s over V entries, the teacher's K values z
// at entries i, a temperature tau and a weight w:
//   p_j = exp(z_j / tau - Z), Z = logsumexp_j(z_j / tau), or the teacher's own
//         log-sum-exp over all its entries where that is given
//   lse = logsumexp_v(s_v / tau)
//   loss = w sum_j p_j (log p_j - s_{i_j} / tau + lse)
//   dloss/ds_v = (w / tau) (P exp(s_v / tau - lse) - sum_{j: i_j = v} p_j), P = sum_j p_j
// Entries with i_j < 0 or z_j = -inf are left out. A token whose weight is 0
// or that has no entry left has loss 0, lse 0 and a zero gradient, and its
// logits are not read, so nothing in them (NaN included) reaches the outputs.
// The maximum, the sums and the logarithm are in fp32; a gradient value is
// rounded once, when it is stored.
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int DISTILL_THREADS = 512;
constexpr int DISTILL_WARPS = DISTILL_THREADS / 32;
constexpr int DISTILL_MAX_TOP = 1024;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct DistillParams {
  const void* logits;
  long long logits_ld;
  void* grad;           // null: no gradient
  long long grad_ld;
  long long vocab;
  const void* teacher;  // [tokens][top]
  int teacher_dtype;
  const void* ids;
  int id_bytes, top;
  const float* weights;      // null: 1
  const float* teacher_lse;  // null: over the top entries
  float inv_tau;
  float* loss;          // null: the log-sum-exp is given
  float* lse;
  unsigned int* status;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Maximum and sum of exp2((x - max) c) of what was seen so far.
struct Online {
  float m = -INFINITY, s = 0.0f;
  __device__ __forceinline__ void join(float m2, float s2) {
    const float n = fmaxf(m, m2);
    if (n == -INFINITY) {
      s += s2;  // 0, or NaN
      return;
    }
    s = s * exp2_fast(m - n) + s2 * exp2_fast(m2 - n);
    m = n;
  }
};

// Elements before the first 16-byte boundary of p, at most n.
template <typename T>
__device__ __forceinline__ long long head_of(const T* p, long long n) {
  const long long h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
  return h < n ? h : n;
}

// One block takes one token: the teacher's entries into shared memory, one
// pass over the logits for the log-sum-exp, and one for the gradient.
template <typename T>
__global__ void __launch_bounds__(DISTILL_THREADS) ns_distill_kernel(const __grid_constant__ DistillParams p) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float tp[DISTILL_MAX_TOP];      // p_j
  __shared__ float ts[DISTILL_MAX_TOP];      // the student's logit at the entry
  __shared__ int ti[DISTILL_MAX_TOP];        // the entry, -1 if left out
  __shared__ float red_m[DISTILL_WARPS], red_s[DISTILL_WARPS];
  __shared__ float sh_mass, sh_lse2;
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const long long t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(p.logits) + t * p.logits_ld;
  T* grad = static_cast<T*>(p.grad) + t * p.grad_ld;
  const float weight = p.weights ? p.weights[t] : 1.0f;
  const float c = p.inv_tau * LOG2E;  // logits to powers of two

  // teacher: values times c, then probabilities
  float zmax = -INFINITY;
  bool refused = false;
  for (int j = tid; j < p.top; j += DISTILL_THREADS) {
    const long long i = t * p.top + j, id = load_index(p.ids, p.id_bytes, i);
    float z = -INFINITY;
    if (id >= p.vocab) refused = true;
    if (id >= 0 && id < p.vocab && weight != 0.0f)
      z = p.teacher_dtype == NS_DT_FP32   ? static_cast<const float*>(p.teacher)[i]
          : p.teacher_dtype == NS_DT_BF16 ? to_float(static_cast<const __nv_bfloat16*>(p.teacher)[i])
                                          : to_float(static_cast<const __half*>(p.teacher)[i]);
    const bool in = !(z == -INFINITY);
    ti[j] = in ? static_cast<int>(id) : -1;
    tp[j] = z;
    if (in) ts[j] = to_float(row[id]);
    zmax = z != z ? z : fmaxf(zmax, z);
  }
  if (refused) atomicOr(p.status, NS_DEV_BAD_INDEX);
  const int any = __syncthreads_or(zmax != -INFINITY);
  if (!any) {
    // nothing to learn from: zeros, without a look at the logits
    if (p.loss && tid == 0) {
      p.loss[t] = 0.0f;
      p.lse[t] = 0.0f;
    }
    if (p.grad) {
      const long long head = head_of(grad, p.vocab), words = (p.vocab - head) / V;
      for (long long i = tid; i < head; i += DISTILL_THREADS) grad[i] = from_float<T>(0.0f);
      for (long long i = tid; i < words; i += DISTILL_THREADS)
        store_vec<T, V>(grad + head + i * V, zero_vec<T, V>());
      for (long long i = head + words * V + tid; i < p.vocab; i += DISTILL_THREADS) grad[i] = from_float<T>(0.0f);
    }
    return;
  }
  if (warp == 0) {
    // log-sum-exp of the entries left, unless the teacher's own is given
    // (relative to their maximum, so that values near the type's lowest stay finite)
    float z0 = 0.0f, zlog;
    if (p.teacher_lse) {
      zlog = p.teacher_lse[t];
    } else {
      z0 = -INFINITY;
      for (int j = lane; j < p.top; j += 32) z0 = fmaxf(z0, tp[j]);
      z0 = warp_max(z0);
      float sum = 0.0f;
      for (int j = lane; j < p.top; j += 32) sum += ti[j] >= 0 ? expf((tp[j] - z0) * p.inv_tau) : 0.0f;
      zlog = logf(warp_sum(sum));
    }
    float mass = 0.0f, part = 0.0f;
    for (int j = lane; j < p.top; j += 32) {
      const float logp = (tp[j] - z0) * p.inv_tau - zlog;
      const float pr = ti[j] >= 0 ? expf(logp) : 0.0f;
      if (pr != 0.0f) part += pr * (logp - ts[j] * p.inv_tau);
      mass += pr;
      tp[j] = pr;
    }
    mass = warp_sum(mass);
    part = warp_sum(part);
    if (lane == 0) {
      sh_mass = mass;
      sh_lse2 = part;  // kept here until the log-sum-exp is known
    }
  }

  const long long head = head_of(row, p.vocab), words = (p.vocab - head) / V, tail = head + words * V;
  float lse2;
  if (p.loss) {
    Online o;
    for (long long i = tid; i < words; i += DISTILL_THREADS) {
      const Vec<T, V> x = load_vec<T, V>(row + head + i * V);
      float v[V], m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        v[k] = to_float(x.v[k]) * c;
        m = fmaxf(m, v[k]);
      }
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int k = 0; k < V; ++k) s += exp2_fast(v[k] - base);
      o.join(m, s);
    }
    for (long long i = tid; i < head + (p.vocab - tail); i += DISTILL_THREADS) {
      const float v = to_float(row[i < head ? i : tail + i - head]) * c;
      o.join(v, v == -INFINITY ? 0.0f : exp2_fast(v - v));
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) o.join(__shfl_xor_sync(0xffffffffu, o.m, k), __shfl_xor_sync(0xffffffffu, o.s, k));
    if (lane == 0) {
      red_m[warp] = o.m;
      red_s[warp] = o.s;
    }
    __syncthreads();
    Online all;
    for (int k = 0; k < DISTILL_WARPS; ++k) all.join(red_m[k], red_s[k]);
    lse2 = all.m + log2f(all.s);
    if (tid == 0) {
      p.loss[t] = weight * (sh_lse2 + sh_mass * (lse2 * LN2));
      p.lse[t] = lse2 * LN2;
    }
  } else {
    lse2 = p.lse[t] * LOG2E;
    __syncthreads();
  }
  if (!p.grad) return;

  const float scale = weight * p.inv_tau, mass = scale * sh_mass;
  const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(grad)) & 15) == 0;
  if (same) {
    for (long long i = tid; i < words; i += DISTILL_THREADS) {
      Vec<T, V> x = load_vec<T, V>(row + head + i * V);
#pragma unroll
      for (int k = 0; k < V; ++k) x.v[k] = from_float<T>(mass * exp2_fast(fmaf(to_float(x.v[k]), c, -lse2)));
      store_vec<T, V>(grad + head + i * V, x);
    }
    for (long long i = tid; i < head + (p.vocab - tail); i += DISTILL_THREADS) {
      const long long v = i < head ? i : tail + i - head;
      grad[v] = from_float<T>(mass * exp2_fast(fmaf(to_float(row[v]), c, -lse2)));
    }
  } else {
    for (long long v = tid; v < p.vocab; v += DISTILL_THREADS)
      grad[v] = from_float<T>(mass * exp2_fast(fmaf(to_float(row[v]), c, -lse2)));
  }
  __syncthreads();
  // the teacher's entries, each with all probabilities that name it
  for (int j = tid; j < p.top; j += DISTILL_THREADS) {
    const int id = ti[j];
    if (id < 0) continue;
    float sum = 0.0f;
    for (int i = 0; i < p.top; ++i) sum += ti[i] == id ? tp[i] : 0.0f;
    grad[id] = from_float<T>(mass * exp2_fast(fmaf(ts[j], c, -lse2)) - scale * sum);
  }
}

}  // namespace
}  // namespace nsk

using namespace nsorch;

namespace {

bool dtype_ok(int dtype) { return dtype == NS_DT_BF16 || dtype == NS_DT_FP16 || dtype == NS_DT_FP32; }

int run_distill(const void* logits, int64_t logits_stride, int dtype, int64_t tokens, int64_t vocab,
                const void* teacher_values, int teacher_dtype, const void* teacher_ids, int id_bytes, int top,
                const float* weights, const float* teacher_lse, float temperature, float* loss, float* lse,
                void* grad_logits, int64_t grad_stride, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype) || (id_bytes != 4 && id_bytes != 8)) return NS_ERR_ARG;
  if (tokens < 0 || vocab < 1 || top < 1 || !(temperature > 0.0f) || temperature > 3.0e38f) return NS_ERR_ARG;
  if (top > nsk::DISTILL_MAX_TOP) return NS_ERR_UNSUPPORTED;
  if (vocab > INT_MAX || tokens > INT_MAX || logits_stride < vocab || (grad_logits && grad_stride < vocab))
    return NS_ERR_SHAPE;
  if (tokens == 0) return NS_OK;
  if (!logits || !teacher_values || !teacher_ids || !lse) return NS_ERR_ARG;
  if (grad_logits == logits && grad_stride != logits_stride) return NS_ERR_ARG;
  nsk::DistillParams p = {};
  p.logits = logits;
  p.logits_ld = logits_stride;
  p.grad = grad_logits;
  p.grad_ld = grad_stride;
  p.vocab = vocab;
  p.teacher = teacher_values;
  p.teacher_dtype = teacher_dtype;
  p.ids = teacher_ids;
  p.id_bytes = id_bytes;
  p.top = top;
  p.weights = weights;
  p.teacher_lse = teacher_lse;
  p.inv_tau = 1.0f / temperature;
  p.loss = loss;
  p.lse = lse;
  int dev, nsm;
  const int rc = device_setup(&dev, &p.status, &nsm);
  if (rc != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(tokens)), block(nsk::DISTILL_THREADS);
  const cudaError_t e = counted(K_DISTILL, st, [&] {
    if (dtype == NS_DT_BF16) return nsk::launch_pdl(nsk::ns_distill_kernel<__nv_bfloat16>, grid, block, 0, st, p);
    if (dtype == NS_DT_FP16) return nsk::launch_pdl(nsk::ns_distill_kernel<__half>, grid, block, 0, st, p);
    return nsk::launch_pdl(nsk::ns_distill_kernel<float>, grid, block, 0, st, p);
  });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

}  // namespace

extern "C" {

int ns_distill_loss(const void* logits, int64_t logits_stride, int dtype, int64_t tokens, int64_t vocab,
                    const void* teacher_values, int teacher_dtype, const void* teacher_ids, int id_bytes, int top,
                    const float* weights, const float* teacher_lse, float temperature, float* loss, float* lse,
                    void* grad_logits, int64_t grad_stride, void* stream) {
  if (tokens > 0 && !loss) return NS_ERR_ARG;
  return run_distill(logits, logits_stride, dtype, tokens, vocab, teacher_values, teacher_dtype, teacher_ids,
                     id_bytes, top, weights, teacher_lse, temperature, loss, lse, grad_logits, grad_stride, stream);
}

int ns_distill_grad(const void* logits, int64_t logits_stride, int dtype, int64_t tokens, int64_t vocab,
                    const void* teacher_values, int teacher_dtype, const void* teacher_ids, int id_bytes, int top,
                    const float* weights, const float* teacher_lse, float temperature, const float* lse,
                    void* grad_logits, int64_t grad_stride, void* stream) {
  if (tokens > 0 && !grad_logits) return NS_ERR_ARG;
  return run_distill(logits, logits_stride, dtype, tokens, vocab, teacher_values, teacher_dtype, teacher_ids,
                     id_bytes, top, weights, teacher_lse, temperature, nullptr, const_cast<float*>(lse), grad_logits,
                     grad_stride, stream);
}

}  // extern "C"
