// The global norm of many tensors' gradients, and clipping by it.
//
//   norm = sqrt(sum of g^2 over every value of every tensor)
//   c = min(1, max_norm / (norm + eps)),  out = c g
//
// A tensor is cut into chunks of CHUNK_WORDS aligned 16-byte words (the values
// before the first word belong to its first chunk, those after the last to its
// last), and the blocks of a grid that fits the card take the chunks of all
// tensors in turn. The tensors' addresses and sizes are kernel arguments, so
// that a call needs no copy and can be captured.
//
// Bound by memory: the norm reads each value once (2.0 GB in 280-285 us, 7.1
// TB/s); clipping reads it once more, because no value can be written before all
// were read (1.14 GB normed and clipped into other tensors in 523 us, 6.5 TB/s).
#include <algorithm>
#include <climits>
#include <cmath>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int GN_THREADS = 256;
constexpr int GN_WORDS = 8;                      // 16-byte words of a chunk that a lane takes
// Blocks of an SM. Reading alone wants much on its way (2.0 GB normed at 7.1 TB/s with 4 blocks of 8 words a lane, 6.2
// with 8 of 4), reading beside writing little: clipped at 6.6 TB/s with 3 blocks of 4 words at a time, 4.7 with 8 of 4
// and 3.4 with 6 of 8.
constexpr int GN_BLOCKS = 4, GN_CLIP_BLOCKS = 3, GN_CLIP_WORDS = 4;
// Of the block that joins the partial sums: few enough to stand on an SM beside the norm's blocks and wait there (23
// tensors of 5.4 MB normed in 5.2 us, with 1024 threads 7.1).
constexpr int GN_TOTAL_THREADS = 128;
constexpr int CHUNK_WORDS = GN_THREADS * GN_WORDS;
constexpr int GN_TENSORS = 512;                  // of a launch
constexpr int GN_MAX_BLOCKS = 2048;              // partial sums of a launch

struct GradTable {
  const void* src[GN_TENSORS];
  long long size[GN_TENSORS];  // values * 4 + type
  int first[GN_TENSORS + 1];   // chunks of the tensors before
  int tensors, chunks;
};

struct GradNormParams {
  GradTable in;
  double* partial;  // [blocks]
};

struct GradClipParams {
  GradTable in;
  void* out[GN_TENSORS];
  const float* norm;
  float max_norm, eps;
};

struct GradTotalParams {
  const double* partial;
  int n;
  float* norm;
};

// The tensor of chunk c.
__device__ __forceinline__ int tensor_of(const GradTable& g, int c) {
  int low = 0, high = g.tensors;
  while (high - low > 1) {
    const int mid = (low + high) / 2;
    if (g.first[mid] <= c)
      low = mid;
    else
      high = mid;
  }
  return low;
}

// One chunk of a tensor: `words` aligned words from `at` on, and (first and last
// chunk) the values at its ends.
template <typename T>
struct Chunk {
  const T* at;
  int words;
  const T* head;
  int heads;
  const T* tail;
  int tails;
  __device__ __forceinline__ Chunk(const T* p, long long n, int k) {
    constexpr int V = 16 / sizeof(T);
    const long long h = head_of(p, n), all = (n - h) / V, from = static_cast<long long>(k) * CHUNK_WORDS;
    at = p + h + from * V;
    words = static_cast<int>(min(static_cast<long long>(CHUNK_WORDS), all - from));
    head = p;
    heads = k == 0 ? static_cast<int>(h) : 0;
    tail = p + h + all * V;
    tails = from + CHUNK_WORDS >= all ? static_cast<int>(n - h - all * V) : 0;
  }
};

// The sum of a lane's squares in 64 bits, for those that leave fp32's range.
template <typename T>
__device__ __noinline__ double wide_sum(const Chunk<T> c) {
  constexpr int V = 16 / sizeof(T);
  double sum = 0.0;
  for (int i = threadIdx.x; i < c.words; i += GN_THREADS) {
    const Vec<T, V> x = load_vec<T, V>(c.at + static_cast<long long>(i) * V);
    for (int j = 0; j < V; ++j) {
      const double v = get(x, j);
      sum += v * v;
    }
  }
  const int i = threadIdx.x;
  if (i < c.heads) sum += static_cast<double>(to_float(c.head[i])) * to_float(c.head[i]);
  if (i < c.tails) sum += static_cast<double>(to_float(c.tail[i])) * to_float(c.tail[i]);
  return sum;
}

// A lane's share of a chunk's sum of squares: at most 80 values, in fp32 (two
// values at a time). A sum that is not finite, or so small that squares may have
// vanished though values are there, is formed again in 64 bits.
template <typename T>
__device__ __forceinline__ double chunk_sum(const T* p, long long n, int k) {
  constexpr int V = 16 / sizeof(T);
  const Chunk<T> c(p, n, k);
  Vec<T, V> x[GN_WORDS];
#pragma unroll
  for (int w = 0; w < GN_WORDS; ++w) {
    const int i = w * GN_THREADS + threadIdx.x;
    x[w] = i < c.words ? load_vec<T, V>(c.at + i * V) : zero_vec<T, V>();
  }
  float2 s[2] = {};
  uint32_t any = 0;
#pragma unroll
  for (int w = 0; w < GN_WORDS; ++w) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 v = make_float2(get(x[w], j), get(x[w], j + 1));
      s[(j / 2) & 1] = fma2(v, v, s[(j / 2) & 1]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) any |= x[w].w[j];
  }
  const int i = threadIdx.x;
  float ends = 0.0f;
  if (i < c.heads) ends = to_float(c.head[i]);
  if (i < c.tails) s[1].x = fmaf(to_float(c.tail[i]), to_float(c.tail[i]), s[1].x);
  const float sum = fmaf(ends, ends, (s[0].x + s[0].y) + (s[1].x + s[1].y));
  // 2^-100 over 80 squares: what fp32's smallest values took away is below 2^-24 of it
  if (sum > 0x1p-100f && sum < INFINITY) return sum;
  const uint32_t sign = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
  if (!(any & ~sign) && c.heads + c.tails == 0) return 0.0;
  return wide_sum(c);
}

__global__ void __launch_bounds__(GN_THREADS, GN_BLOCKS) ns_grad_norm_kernel(const __grid_constant__ GradNormParams p) {
  __shared__ double part[GN_THREADS / 32];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  double sum = 0.0;
  for (int c = blockIdx.x; c < p.in.chunks; c += gridDim.x) {
    const int t = tensor_of(p.in, c), k = c - p.in.first[t], type = static_cast<int>(p.in.size[t] & 3);
    const long long n = p.in.size[t] >> 2;
    if (type == NS_DT_BF16)
      sum += chunk_sum(static_cast<const __nv_bfloat16*>(p.in.src[t]), n, k);
    else if (type == NS_DT_FP16)
      sum += chunk_sum(static_cast<const __half*>(p.in.src[t]), n, k);
    else
      sum += chunk_sum(static_cast<const float*>(p.in.src[t]), n, k);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < GN_THREADS / 32; ++w) sum += part[w];
  p.partial[blockIdx.x] = sum;
}

// The partial sums in a fixed order, and the root.
__global__ void __launch_bounds__(GN_TOTAL_THREADS) ns_grad_total_kernel(const __grid_constant__ GradTotalParams p) {
  __shared__ double part[32];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  double sum = 0.0;
  for (int i = threadIdx.x; i < p.n; i += GN_TOTAL_THREADS) sum += p.partial[i];
  for (int round = 0; round < 2; ++round) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (round) break;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = threadIdx.x % 32 < GN_TOTAL_THREADS / 32 ? part[threadIdx.x % 32] : 0.0;
  }
  if (threadIdx.x == 0) *p.norm = static_cast<float>(sqrt(sum));
}

// A value times the scale, in fp32's or the scale's bits, whichever are more.
template <typename F>
__device__ __forceinline__ float scaled(float x, F scale) {
  return static_cast<float>(x * scale);
}

template <typename T, typename F>
__device__ __forceinline__ void clip_chunk(const T* p, T* out, long long n, int k, F scale) {
  constexpr int V = 16 / sizeof(T);
  const Chunk<T> c(p, n, k);
  T* const to = out + (c.at - p);
  if ((reinterpret_cast<uintptr_t>(to) & 15) == 0) {
#pragma unroll
    for (int w0 = 0; w0 < GN_WORDS; w0 += GN_CLIP_WORDS) {
      Vec<T, V> x[GN_CLIP_WORDS];
#pragma unroll
      for (int w = 0; w < GN_CLIP_WORDS; ++w) {
        const int i = (w0 + w) * GN_THREADS + threadIdx.x;
        if (i < c.words) x[w] = load_vec<T, V>(c.at + i * V);
      }
#pragma unroll
      for (int w = 0; w < GN_CLIP_WORDS; ++w) {
        const int i = (w0 + w) * GN_THREADS + threadIdx.x;
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = scaled(get(x[w], j), scale);
        if (i < c.words) store_vec<T, V>(to + i * V, pack<T, V>(f));
      }
    }
  } else {  // the two start at different places of a word
    for (int i = threadIdx.x; i < c.words * V; i += GN_THREADS) to[i] = from_float<T>(scaled(to_float(c.at[i]), scale));
  }
  const int i = threadIdx.x;
  if (i < c.heads) out[i] = from_float<T>(scaled(to_float(c.head[i]), scale));
  if (i < c.tails) out[c.tail - p + i] = from_float<T>(scaled(to_float(c.tail[i]), scale));
}

// Chunk k of tensor t.
template <typename F>
__device__ __forceinline__ void clip_tensor(const GradClipParams& p, int t, int k, F scale) {
  const int type = static_cast<int>(p.in.size[t] & 3);
  const long long n = p.in.size[t] >> 2;
  if (type == NS_DT_BF16)
    clip_chunk(static_cast<const __nv_bfloat16*>(p.in.src[t]), static_cast<__nv_bfloat16*>(p.out[t]), n, k, scale);
  else if (type == NS_DT_FP16)
    clip_chunk(static_cast<const __half*>(p.in.src[t]), static_cast<__half*>(p.out[t]), n, k, scale);
  else
    clip_chunk(static_cast<const float*>(p.in.src[t]), static_cast<float*>(p.out[t]), n, k, scale);
}
__device__ __noinline__ void clip_tensor_wide(const GradClipParams& p, int t, int k, double scale) { clip_tensor(p, t, k, scale); }

// From the last chunk back: the norm read it last, so that L2 still holds some. A
// scale below fp32's normal range would lose bits there (a norm of 3e38 clipped to
// 1e-4: 2e-3 of every value) and is multiplied in 64 bits.
__global__ void __launch_bounds__(GN_THREADS, GN_CLIP_BLOCKS) ns_grad_clip_kernel(const __grid_constant__ GradClipParams p) {
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const double norm = static_cast<double>(*p.norm) + p.eps, wide = norm <= p.max_norm ? 1.0 : p.max_norm / norm;  // NaN stays visible
  const float scale = static_cast<float>(wide);
  for (int i = p.in.chunks - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
    const int t = tensor_of(p.in, i), k = i - p.in.first[t];
    if (scale == 1.0f && p.in.src[t] == p.out[t]) continue;
    if (wide > 0.0 && wide < 0x1p-126)
      clip_tensor_wide(p, t, k, wide);
    else
      clip_tensor(p, t, k, scale);
  }
}

// Chunks of a tensor.
long long chunks_of(const void* p, int64_t n, int dtype) {
  const int b = elem_bytes(dtype), V = 16 / b;
  const int64_t head = std::min<int64_t>(n, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / b);
  return std::max<int64_t>(1, ((n - head) / V + CHUNK_WORDS - 1) / CHUNK_WORDS);
}

// Adds tensors i, i + 1, ... < count to a launch's table, as many as it holds;
// the first that it does not. `outs` and `to`: the tensors' outputs, if any.
int fill_table(GradTable& g, const void* const* grads, const int64_t* numels, const int* dtypes, int i, int count,
               void* const* outs, void** to) {
  long long chunks = 0;
  g.tensors = 0;
  for (; i < count && g.tensors < GN_TENSORS; ++i) {
    if (numels[i] == 0) continue;
    g.src[g.tensors] = grads[i];
    g.size[g.tensors] = numels[i] * 4 + dtypes[i];
    if (outs) to[g.tensors] = outs[i];
    g.first[g.tensors++] = static_cast<int>(chunks);
    chunks += chunks_of(grads[i], numels[i], dtypes[i]);
  }
  g.first[g.tensors] = g.chunks = static_cast<int>(chunks);
  return i;
}

}  // namespace
}  // namespace nsk

using namespace nsorch;

namespace {

// More than any card holds; the chunks of a launch fit an int.
constexpr int64_t kMostBytes = int64_t{1} << 43;
constexpr int kMostTensors = 1 << 20;

int check_tensors(const void* const* grads, const int64_t* numels, const int* dtypes, int count) {
  if (count < 0 || (count > 0 && (!grads || !numels || !dtypes))) return NS_ERR_ARG;
  if (count > kMostTensors) return NS_ERR_UNSUPPORTED;
  int64_t bytes = 0;
  for (int i = 0; i < count; ++i) {
    if (!nsk::dtype_ok(dtypes[i]) || numels[i] < 0) return NS_ERR_ARG;
    if (numels[i] == 0) continue;
    if (!grads[i] || !nsk::element_aligned(grads[i], nsk::elem_bytes(dtypes[i]))) return NS_ERR_ARG;
    if (numels[i] > kMostBytes / 4 || (bytes += numels[i] * nsk::elem_bytes(dtypes[i])) > kMostBytes) return NS_ERR_SHAPE;
  }
  return NS_OK;
}

uint64_t norm_workspace(int count) {
  const int launches = std::max(1, (count + nsk::GN_TENSORS - 1) / nsk::GN_TENSORS);
  return sizeof(double) * static_cast<uint64_t>(nsk::GN_MAX_BLOCKS) * launches;
}

}  // namespace

extern "C" {

int ns_grad_norm_workspace_bytes(int count, uint64_t* bytes) {
  if (!bytes || count < 0) return NS_ERR_ARG;
  if (count > kMostTensors) return NS_ERR_UNSUPPORTED;
  *bytes = norm_workspace(count);
  return NS_OK;
}

int ns_grad_norm(const void* const* grads, const int64_t* numels, const int* dtypes, int count, float* norm,
                 void* workspace, uint64_t workspace_bytes, void* stream) {
  int rc = check_tensors(grads, numels, dtypes, count);
  if (rc != NS_OK) return rc;
  if (!norm || !nsk::element_aligned(norm, 4)) return NS_ERR_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < norm_workspace(count))
    return NS_ERR_WORKSPACE;
  int dev, nsm;
  unsigned int* status;
  rc = device_setup(&dev, &status, &nsm);
  if (rc != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int most = std::min(nsm * nsk::GN_BLOCKS, nsk::GN_MAX_BLOCKS);
  nsk::GradTotalParams total = {static_cast<const double*>(workspace), 0, norm};
  nsk::GradNormParams p;
  for (int i = 0; i < count;) {
    i = nsk::fill_table(p.in, grads, numels, dtypes, i, count, nullptr, nullptr);
    if (p.in.tensors == 0) break;
    const int blocks = std::min(p.in.chunks, most);
    p.partial = static_cast<double*>(workspace) + total.n;
    total.n += blocks;
    const cudaError_t e = counted(K_GRAD, st, [&] {
      return nsk::launch_pdl(nsk::ns_grad_norm_kernel, dim3(blocks), dim3(nsk::GN_THREADS), 0, st, p);
    });
    if (e != cudaSuccess) return NS_ERR_CUDA;
  }
  const cudaError_t e =
      counted(K_GRAD, st, [&] { return nsk::launch_pdl(nsk::ns_grad_total_kernel, dim3(1), dim3(nsk::GN_TOTAL_THREADS), 0, st, total); });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

int ns_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes, int count,
                 const float* norm, float max_norm, float eps, void* stream) {
  int rc = check_tensors(grads, numels, dtypes, count);
  if (rc != NS_OK) return rc;
  if (count > 0 && !outs) return NS_ERR_ARG;
  if (!norm || !nsk::element_aligned(norm, 4) || !(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(eps)) return NS_ERR_ARG;
  for (int i = 0; i < count; ++i)
    if (numels[i] > 0 && (!outs[i] || !nsk::element_aligned(outs[i], nsk::elem_bytes(dtypes[i])))) return NS_ERR_ARG;
  int dev, nsm;
  unsigned int* status;
  nsk::GradClipParams p;
  p.norm = norm;
  p.max_norm = max_norm;
  p.eps = eps;
  bool ready = false;
  for (int i = 0; i < count;) {
    i = nsk::fill_table(p.in, grads, numels, dtypes, i, count, outs, p.out);
    if (p.in.tensors == 0) break;
    if (!ready && (rc = device_setup(&dev, &status, &nsm)) != NS_OK) return rc;
    ready = true;
    const int blocks = std::min(p.in.chunks, nsm * nsk::GN_CLIP_BLOCKS);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = counted(K_GRAD, st, [&] {
      return nsk::launch_pdl(nsk::ns_grad_clip_kernel, dim3(blocks), dim3(nsk::GN_THREADS), 0, st, p);
    });
    if (e != cudaSuccess) return NS_ERR_CUDA;
  }
  return NS_OK;
}

}  // extern "C"
