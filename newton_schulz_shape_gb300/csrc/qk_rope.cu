// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradient.
//
// For one head x of D values at position pos, with weight g and the rotation
// R over the first `rot_dim` of them:
//   r = (mean(x^2) + eps)^(-1/2),  y = R_pos (x r g)
// and backward, with u = R_pos^T dy and h = u g:
//   dx = r (h - x r^2 mean(h x)),  dg = sum over tokens and heads of u x r.
// The rotation turns pairs (a, b) -> (a c - b s, b c + a s); the pairs are
// (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved.
//
// Every value is read and written once, so the kernels are bound by memory.
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int QK_THREADS = 256;
constexpr int QK_WARPS = QK_THREADS / 32;
constexpr int QK_ANY_THREADS = 128;
constexpr int QK_MAX_DIM = 1024;
constexpr int QK_MAX_BLOCKS = 1024;  // blocks of a gradient launch, each with its own sums of dg

struct QkSide {
  const void* x;
  const void* dy;     // gradient only
  void* out;          // y, or dx
  const void* weight; // null: 1
  long long x_token, x_head, dy_token, dy_head, out_token, out_head;  // strides in elements
  int heads;
};

struct QkParams {
  QkSide side[2];     // queries, keys
  long long tokens;
  int dim, rot_dim, interleaved, weight_fp32;
  float eps;
  const float* table; // [table_rows][rot_dim]: cosines, then sines
  long long table_rows;
  const void* positions;  // null: the token's index
  int position_bytes;
  long long q_warps;  // forward: warps on the queries, the rest are on the keys
  float* partial;     // gradient: [blocks][2][dim]
  unsigned int* status;
};

// The table row of token t, null if its position is outside the table.
__device__ __forceinline__ const float* table_row(const QkParams& p, long long t) {
  const long long pos = p.positions ? load_index(p.positions, p.position_bytes, t) : t;
  if (pos < 0 || pos >= p.table_rows) {
    atomicOr(p.status, NS_DEV_BAD_INDEX);
    return nullptr;
  }
  return p.table + pos * p.rot_dim;
}

template <typename T>
__device__ __forceinline__ float weight_at(const QkParams& p, const void* w, int d) {
  if (!w) return 1.0f;
  return p.weight_fp32 ? static_cast<const float*>(w)[d] : to_float(static_cast<const T*>(w)[d]);
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a lane knows of its 16 bytes of every head: V values from d0 on.
template <typename T>
struct Lane {
  static constexpr int V = 16 / sizeof(T);
  int d0;
  bool on;       // inside the head
  bool rotated;  // inside the rotated part
  int partner;   // lane that holds the other values of the pairs (i, i + rot_dim / 2)
  int angle;     // first angle of the lane's values
  float sign;    // of the partner's sine term, forward
};

template <typename T, int G>
__device__ __forceinline__ Lane<T> lane_of(const QkParams& p, int lane) {
  constexpr int V = Lane<T>::V;
  Lane<T> l;
  const int chunk = lane % G, half = p.rot_dim / 2;
  l.d0 = chunk * V;
  l.on = l.d0 < p.dim;
  l.rotated = l.d0 < p.rot_dim;
  const bool first = l.d0 < half;
  l.partner = l.rotated && !p.interleaved ? lane + (first ? half / V : -(half / V)) : lane;
  l.angle = p.interleaved ? l.d0 / 2 : (first ? l.d0 : l.d0 - half);
  l.sign = first ? -1.0f : 1.0f;
  return l;
}

template <typename T>
__device__ __forceinline__ Vec<T, Lane<T>::V> from_partner(const Vec<T, Lane<T>::V>& x, int lane) {
  Vec<T, Lane<T>::V> y;
  const uint4 a = *reinterpret_cast<const uint4*>(&x);
  uint4 b;
  b.x = __shfl_sync(0xffffffffu, a.x, lane);
  b.y = __shfl_sync(0xffffffffu, a.y, lane);
  b.z = __shfl_sync(0xffffffffu, a.z, lane);
  b.w = __shfl_sync(0xffffffffu, a.w, lane);
  *reinterpret_cast<uint4*>(&y) = b;
  return y;
}

// The lane's cosines and sines of one table row: V of each, or V / 2 when the
// pairs are interleaved.
template <typename T>
__device__ __forceinline__ void load_angles(const QkParams& p, const Lane<T>& l, const float* row,
                                            float (&c)[Lane<T>::V], float (&s)[Lane<T>::V]) {
  constexpr int V = Lane<T>::V;
  if (!row || !l.rotated) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
    return;
  }
  const float* cr = row + l.angle;
  const float* sr = cr + p.rot_dim / 2;
  if (p.interleaved) {
    const Vec<float, V / 2> a = load_vec<float, V / 2>(cr), b = load_vec<float, V / 2>(sr);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      c[i] = get(a, i);
      s[i] = get(b, i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const Vec<float, 4> a = load_vec<float, 4>(cr + i), b = load_vec<float, 4>(sr + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[i + j] = get(a, j);
        s[i + j] = get(b, j);
      }
    }
  }
}

// Position in the pairs (token, head) of one side, in token order.
struct Place {
  long long t;
  int h;
  __device__ __forceinline__ Place(long long pair, int heads) : t(pair / heads), h(static_cast<int>(pair - t * heads)) {}
  __device__ __forceinline__ void step(int n, int heads) {
    h += n;
    while (h >= heads) {
      h -= heads;
      ++t;
    }
  }
};

// Forward: G lanes hold one head, 16 bytes each; a warp takes U rounds of
// 32 / G consecutive heads.
template <typename T, int G, int U>
__global__ void __launch_bounds__(QK_THREADS) ns_qk_kernel(const __grid_constant__ QkParams p) {
  constexpr int V = Lane<T>::V;
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  long long w = static_cast<long long>(blockIdx.x) * QK_WARPS + (threadIdx.x >> 5);
  const int which = w < p.q_warps ? 0 : 1;
  if (which) w -= p.q_warps;
  const QkSide& side = p.side[which];
  const long long pairs = p.tokens * side.heads;
  const long long first = w * (U * (32 / G)) + lane / G;
  if (w * (U * (32 / G)) >= pairs) return;
  const Lane<T> l = lane_of<T, G>(p, lane);

  Vec<T, V> x[U];
  {
    Place at(first, side.heads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = zero_vec<T, V>();
      if (l.on && first + u * (32 / G) < pairs)
        x[u] = load_vec<T, V>(static_cast<const T*>(side.x) + at.t * side.x_token + at.h * side.x_head + l.d0);
      at.step(32 / G, side.heads);
    }
  }
  float g[V], gp[V];  // the lane's weights and its partner's
#pragma unroll
  for (int i = 0; i < V; ++i) {
    g[i] = l.on ? weight_at<T>(p, side.weight, l.d0 + i) : 0.0f;
    gp[i] = __shfl_sync(0xffffffffu, g[i], l.partner);
  }
  Place at(first, side.heads);
  long long angles_of = -1;
  const float* row = nullptr;
  float c[V], s[V];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool live = first + u * (32 / G) < pairs;
    if (live && p.rot_dim && at.t != angles_of) {
      row = table_row(p, at.t);
      load_angles<T>(p, l, row, c, s);
      angles_of = at.t;
    }
    float xf[V], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      xf[i] = get(x[u], i);
      sum = fmaf(xf[i], xf[i], sum);
    }
    sum = group_sum<G>(sum);
    const float r = rsqrtf(sum / p.dim + p.eps);
    float y[V];
    if (p.interleaved && l.rotated) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float a = xf[i] * r * g[i], b = xf[i + 1] * r * g[i + 1];
        y[i] = a * c[i / 2] - b * s[i / 2];
        y[i + 1] = b * c[i / 2] + a * s[i / 2];
      }
    }
    const Vec<T, V> other = from_partner<T>(x[u], l.partner);
    if (!p.interleaved || !l.rotated) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float a = xf[i] * r * g[i];
        const float b = get(other, i) * r * gp[i];
        y[i] = l.rotated ? a * c[i] + l.sign * (b * s[i]) : a;
      }
    }
    if (live && l.on && (row || !p.rot_dim))
      store_vec<T, V>(static_cast<T*>(side.out) + at.t * side.out_token + at.h * side.out_head + l.d0, pack<T, V>(y));
    at.step(32 / G, side.heads);
  }
}

// Gradient: the same lanes, in a grid that stays on the card; a lane keeps the
// sums of its V columns of dg, which a block joins in a fixed order.
template <typename T, int G, int U>
__global__ void __launch_bounds__(QK_THREADS) ns_qk_grad_kernel(const __grid_constant__ QkParams p) {
  constexpr int V = Lane<T>::V;
  __shared__ float joined[QK_WARPS][G * V];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<T> l = lane_of<T, G>(p, lane);
  for (int which = 0; which < 2; ++which) {
    const QkSide& side = p.side[which];
    const long long pairs = p.tokens * side.heads;
    float g[V], dg[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      g[i] = l.on ? weight_at<T>(p, side.weight, l.d0 + i) : 0.0f;
      dg[i] = 0.0f;
    }
    const long long stride = static_cast<long long>(gridDim.x) * QK_WARPS * (U * (32 / G));
    for (long long base = (static_cast<long long>(blockIdx.x) * QK_WARPS + warp) * (U * (32 / G)); base < pairs;
         base += stride) {
      const long long first = base + lane / G;
      Vec<T, V> x[U], dy[U];
      {
        Place at(first, side.heads);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[u] = zero_vec<T, V>();
          dy[u] = zero_vec<T, V>();
          if (l.on && first + u * (32 / G) < pairs) {
            x[u] = load_vec<T, V>(static_cast<const T*>(side.x) + at.t * side.x_token + at.h * side.x_head + l.d0);
            dy[u] = load_vec<T, V>(static_cast<const T*>(side.dy) + at.t * side.dy_token + at.h * side.dy_head + l.d0);
          }
          at.step(32 / G, side.heads);
        }
      }
      Place at(first, side.heads);
      long long angles_of = -1;
      const float* row = nullptr;
      float c[V], s[V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        bool live = first + u * (32 / G) < pairs;
        if (live && p.rot_dim && at.t != angles_of) {
          row = table_row(p, at.t);
          load_angles<T>(p, l, row, c, s);
          angles_of = at.t;
        }
        if (p.rot_dim && !row) live = false;
        const Vec<T, V> other = from_partner<T>(dy[u], l.partner);
        float xf[V], t[V], sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xf[i] = get(x[u], i);
          t[i] = get(dy[u], i);
        }
        if (l.rotated) {
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
              const float a = t[i], b = t[i + 1];
              t[i] = a * c[i / 2] + b * s[i / 2];
              t[i + 1] = b * c[i / 2] - a * s[i / 2];
            }
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] = t[i] * c[i] - l.sign * (get(other, i) * s[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sum = fmaf(xf[i], xf[i], sum);
          dot = fmaf(t[i] * g[i], xf[i], dot);
        }
        sum = group_sum<G>(sum);
        dot = group_sum<G>(dot);
        const float r = rsqrtf(sum / p.dim + p.eps);
        const float m = r * r * (dot / p.dim);
        if (live && l.on) {
          float dx[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dg[i] = fmaf(t[i], xf[i] * r, dg[i]);
            dx[i] = r * (t[i] * g[i] - xf[i] * m);
          }
          store_vec<T, V>(static_cast<T*>(side.out) + at.t * side.out_token + at.h * side.out_head + l.d0,
                          pack<T, V>(dx));
        }
        at.step(32 / G, side.heads);
      }
    }
    if (!p.partial) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int o = G; o < 32; o <<= 1) dg[i] += __shfl_xor_sync(0xffffffffu, dg[i], o);
      if (lane < G) joined[warp][lane * V + i] = dg[i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.dim; d += QK_THREADS) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < QK_WARPS; ++k) sum += joined[k][d];
      p.partial[(static_cast<long long>(blockIdx.x) * 2 + which) * p.dim + d] = sum;
    }
    __syncthreads();
  }
}

// Any head width, alignment and rotation: a warp takes one head through shared
// memory, value by value.
template <typename T, bool GRAD>
__global__ void __launch_bounds__(QK_ANY_THREADS) ns_qk_any_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ float any_smem[];
  constexpr int WARPS = QK_ANY_THREADS / 32;
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.dim, half = p.rot_dim / 2;
  float* xs = any_smem + warp * (GRAD ? 3 : 1) * D;  // x; then dy, and the sums of dg
  float* us = xs + D;
  float* dg = xs + 2 * D;
  for (int which = 0; which < 2; ++which) {
    const QkSide& side = p.side[which];
    const long long pairs = p.tokens * side.heads;
    if (GRAD)
      for (int d = lane; d < D; d += 32) dg[d] = 0.0f;
    for (long long pair = static_cast<long long>(blockIdx.x) * WARPS + warp; pair < pairs;
         pair += static_cast<long long>(gridDim.x) * WARPS) {
      const Place at(pair, side.heads);
      const float* row = p.rot_dim ? table_row(p, at.t) : nullptr;
      if (p.rot_dim && !row) continue;
      const T* x = static_cast<const T*>(side.x) + at.t * side.x_token + at.h * side.x_head;
      T* out = static_cast<T*>(side.out) + at.t * side.out_token + at.h * side.out_head;
      __syncwarp();
      float sum = 0.0f;
      for (int d = lane; d < D; d += 32) {
        const float v = to_float(x[d]);
        xs[d] = v;
        sum = fmaf(v, v, sum);
      }
      sum = warp_sum(sum);
      const float r = rsqrtf(sum / D + p.eps);
      // partner, cosine and sine of value d; the sine's sign is the forward's
      auto turn = [&](int d, int* other, float* c, float* s) {
        const bool second = p.interleaved ? d & 1 : d >= half;
        *other = p.interleaved ? d ^ 1 : (second ? d - half : d + half);
        const int a = p.interleaved ? d >> 1 : (second ? d - half : d);
        *c = row[a];
        *s = second ? row[half + a] : -row[half + a];
      };
      if (!GRAD) {
        __syncwarp();
        for (int d = lane; d < D; d += 32) {
          float y = xs[d] * r * weight_at<T>(p, side.weight, d);
          if (d < p.rot_dim) {
            int o;
            float c, s;
            turn(d, &o, &c, &s);
            y = y * c + xs[o] * r * weight_at<T>(p, side.weight, o) * s;
          }
          out[d] = from_float<T>(y);
        }
      } else {
        const T* dy = static_cast<const T*>(side.dy) + at.t * side.dy_token + at.h * side.dy_head;
        float dot = 0.0f;
        for (int d = lane; d < D; d += 32) {
          float u = to_float(dy[d]);
          if (d < p.rot_dim) {
            int o;
            float c, s;
            turn(d, &o, &c, &s);
            u = u * c - to_float(dy[o]) * s;
          }
          us[d] = u;
          dot = fmaf(u * weight_at<T>(p, side.weight, d), xs[d], dot);
          dg[d] = fmaf(u, xs[d] * r, dg[d]);
        }
        dot = warp_sum(dot);
        const float m = r * r * (dot / D);
        __syncwarp();  // dx may take the place of dy
        for (int d = lane; d < D; d += 32)
          out[d] = from_float<T>(r * (us[d] * weight_at<T>(p, side.weight, d) - xs[d] * m));
      }
    }
    if (GRAD && p.partial) {
      __syncthreads();
      for (int d = threadIdx.x; d < D; d += QK_ANY_THREADS) {
        float sum = 0.0f;
        for (int k = 0; k < WARPS; ++k) sum += any_smem[(k * 3 + 2) * D + d];
        p.partial[(static_cast<long long>(blockIdx.x) * 2 + which) * D + d] = sum;
      }
      __syncthreads();
    }
  }
}

struct QkSumParams {
  const float* partial;  // [blocks][2 * dim]
  float* out[2];
  int blocks, dim;
};

// dg: sums of the blocks' partial sums, in a fixed order.
__global__ void __launch_bounds__(256) ns_qk_sum_kernel(const __grid_constant__ QkSumParams p) {
  __shared__ float part[8][32];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < 2 * p.dim)
    for (int b = warp; b < p.blocks; b += 8) sum += p.partial[static_cast<long long>(b) * 2 * p.dim + col];
  part[warp][lane] = sum;
  __syncthreads();
  if (warp || col >= 2 * p.dim) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) sum += part[k][lane];
  float* out = p.out[col >= p.dim];
  if (out) out[col >= p.dim ? col - p.dim : col] = sum;
}

template <typename T, int G>
cudaError_t launch_lanes(bool grad, QkParams& p, int nsm, int* blocks, cudaStream_t st) {
  constexpr int U = 4, PER = U * (32 / G);
  const long long qw = (p.tokens * p.side[0].heads + PER - 1) / PER, kw = (p.tokens * p.side[1].heads + PER - 1) / PER;
  if (grad) {
    const long long want = (std::max(qw, kw) + QK_WARPS - 1) / QK_WARPS;
    *blocks = static_cast<int>(std::max<long long>(1, std::min<long long>(want, std::min(nsm * 4, QK_MAX_BLOCKS))));
    return launch_pdl(ns_qk_grad_kernel<T, G, 2>, dim3(*blocks), dim3(QK_THREADS), 0, st, p);
  }
  p.q_warps = qw;
  const long long n = (qw + kw + QK_WARPS - 1) / QK_WARPS;
  if (n > INT_MAX) return cudaErrorInvalidValue;
  return launch_pdl(ns_qk_kernel<T, G, U>, dim3(static_cast<unsigned>(n)), dim3(QK_THREADS), 0, st, p);
}

template <typename T>
cudaError_t launch_qk(bool grad, bool lanes, QkParams& p, int nsm, int* blocks, cudaStream_t st) {
  constexpr int V = Lane<T>::V;
  if (lanes) {
    const int need = p.dim / V;
    if (need <= 4) return launch_lanes<T, 4>(grad, p, nsm, blocks, st);
    if (need <= 8) return launch_lanes<T, 8>(grad, p, nsm, blocks, st);
    if (need <= 16) return launch_lanes<T, 16>(grad, p, nsm, blocks, st);
    return launch_lanes<T, 32>(grad, p, nsm, blocks, st);
  }
  constexpr int WARPS = QK_ANY_THREADS / 32;
  const long long pairs = p.tokens * std::max(p.side[0].heads, p.side[1].heads);
  *blocks = static_cast<int>(std::min<long long>((pairs + WARPS - 1) / WARPS, std::min(nsm * 6, QK_MAX_BLOCKS)));
  const size_t smem = sizeof(float) * WARPS * (grad ? 3 : 1) * p.dim;
  if (grad) return launch_pdl(ns_qk_any_kernel<T, true>, dim3(*blocks), dim3(QK_ANY_THREADS), smem, st, p);
  return launch_pdl(ns_qk_any_kernel<T, false>, dim3(*blocks), dim3(QK_ANY_THREADS), smem, st, p);
}

}  // namespace
}  // namespace nsk

using namespace nsorch;

namespace {

// Whether every head of a side is reached in aligned 16-byte words.
bool words_ok(const void* base, int64_t token, int64_t head, int bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 15) == 0 && token * bytes % 16 == 0 && head * bytes % 16 == 0;
}

int run_qk(bool grad, const void* const* x, const void* const* dy, void* const* out, const int64_t* strides,
           int dtype, int64_t tokens, const int* heads, int head_dim, int rot_dim, int interleaved,
           const void* const* weight, int weight_dtype, float* const* grad_weight, float eps, const float* table,
           int64_t table_rows, const void* positions, int position_bytes, void* workspace, uint64_t workspace_bytes,
           void* stream) {
  if (dtype != NS_DT_BF16 && dtype != NS_DT_FP16 && dtype != NS_DT_FP32) return NS_ERR_ARG;
  if (weight_dtype != dtype && weight_dtype != NS_DT_FP32) return NS_ERR_ARG;
  if (tokens < 0 || heads[0] < 0 || heads[1] < 0 || head_dim < 1 || rot_dim < 0 || table_rows < 0 || !(eps >= 0.0f) || !strides)
    return NS_ERR_ARG;
  if (rot_dim > head_dim || rot_dim % 2) return NS_ERR_SHAPE;
  if (head_dim > nsk::QK_MAX_DIM) return NS_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return NS_ERR_ARG;
  if (rot_dim > 0 && !table) return NS_ERR_ARG;
  if (positions && position_bytes != 4 && position_bytes != 8) return NS_ERR_ARG;
  const int most = std::max(heads[0], heads[1]);
  if (most > 0 && tokens > INT64_MAX / 4 / most / head_dim) return NS_ERR_SHAPE;
  const bool sums = grad && (grad_weight[0] || grad_weight[1]);
  for (int i = 0; i < 2; ++i) {
    if (tokens == 0 || heads[i] == 0) continue;
    if (!x[i] || !out[i] || (grad && !dy[i])) return NS_ERR_ARG;
  }
  if (sums && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
               workspace_bytes < sizeof(float) * 2 * nsk::QK_MAX_BLOCKS * static_cast<uint64_t>(head_dim)))
    return NS_ERR_WORKSPACE;
  if ((tokens == 0 || most == 0) && !sums) return NS_OK;
  nsk::QkParams p = {};
  const int b = dtype == NS_DT_FP32 ? 4 : 2, V = 16 / b;
  bool lanes = head_dim % V == 0 && head_dim / V <= 32 && rot_dim % (interleaved ? V : 2 * V) == 0 &&
               (reinterpret_cast<uintptr_t>(table) & 15) == 0;
  // strides: (token, head) of x, of out and, for the gradient, of dy; queries then keys of each
  for (int i = 0; i < 2; ++i) {
    nsk::QkSide& s = p.side[i];
    s.x = x[i];
    s.out = out[i];
    s.dy = grad ? dy[i] : nullptr;
    s.weight = weight[i];
    s.heads = heads[i];
    s.x_token = strides[2 * i];
    s.x_head = strides[2 * i + 1];
    s.out_token = strides[4 + 2 * i];
    s.out_head = strides[5 + 2 * i];
    if (grad) {
      s.dy_token = strides[8 + 2 * i];
      s.dy_head = strides[9 + 2 * i];
    }
    if (heads[i] == 0) continue;
    lanes = lanes && words_ok(s.x, s.x_token, s.x_head, b) && words_ok(s.out, s.out_token, s.out_head, b) &&
            (!grad || words_ok(s.dy, s.dy_token, s.dy_head, b));
  }
  p.tokens = tokens;
  p.dim = head_dim;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved;
  p.weight_fp32 = weight_dtype == NS_DT_FP32;
  p.eps = eps;
  p.table = table;
  p.table_rows = table_rows;
  p.positions = positions;
  p.position_bytes = position_bytes;
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  int dev, nsm;
  const int rc = device_setup(&dev, &p.status, &nsm);
  if (rc != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int blocks = 0;
  if (tokens > 0 && most > 0) {
    const cudaError_t e = counted(K_QK, st, [&] {
      if (dtype == NS_DT_BF16) return nsk::launch_qk<__nv_bfloat16>(grad, lanes, p, nsm, &blocks, st);
      if (dtype == NS_DT_FP16) return nsk::launch_qk<__half>(grad, lanes, p, nsm, &blocks, st);
      return nsk::launch_qk<float>(grad, lanes, p, nsm, &blocks, st);
    });
    if (e != cudaSuccess) return NS_ERR_CUDA;
  }
  if (!sums) return NS_OK;
  nsk::QkSumParams sp = {p.partial, {grad_weight[0], grad_weight[1]}, blocks, head_dim};
  const cudaError_t e = counted(K_QK, st, [&] {
    return nsk::launch_pdl(nsk::ns_qk_sum_kernel, dim3((2 * head_dim + 31) / 32), dim3(256), 0, st, sp);
  });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

}  // namespace

extern "C" {

int ns_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const int64_t* strides, int dtype,
                    int64_t tokens, int q_heads, int k_heads, int head_dim, int rot_dim, int interleaved,
                    const void* q_weight, const void* k_weight, int weight_dtype, float eps, const float* table,
                    int64_t table_rows, const void* positions, int position_bytes, void* stream) {
  const void* x[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int heads[2] = {q_heads, k_heads};
  const void* weight[2] = {q_weight, k_weight};
  return run_qk(false, x, nullptr, out, strides, dtype, tokens, heads, head_dim, rot_dim, interleaved, weight,
                weight_dtype, nullptr, eps, table, table_rows, positions, position_bytes, nullptr, 0, stream);
}

int ns_qk_norm_rope_grad_workspace_bytes(int head_dim, uint64_t* bytes) {
  if (!bytes || head_dim < 1) return NS_ERR_ARG;
  if (head_dim > nsk::QK_MAX_DIM) return NS_ERR_UNSUPPORTED;
  *bytes = sizeof(float) * 2 * nsk::QK_MAX_BLOCKS * static_cast<uint64_t>(head_dim);
  return NS_OK;
}

int ns_qk_norm_rope_grad(const void* grad_q_out, const void* grad_k_out, const void* q, const void* k, void* grad_q,
                         void* grad_k, const int64_t* strides, int dtype, int64_t tokens, int q_heads, int k_heads,
                         int head_dim, int rot_dim, int interleaved, const void* q_weight, const void* k_weight,
                         int weight_dtype, float* grad_q_weight, float* grad_k_weight, float eps,
                         const float* table, int64_t table_rows, const void* positions, int position_bytes,
                         void* workspace, uint64_t workspace_bytes, void* stream) {
  const void* x[2] = {q, k};
  const void* dy[2] = {grad_q_out, grad_k_out};
  void* out[2] = {grad_q, grad_k};
  const int heads[2] = {q_heads, k_heads};
  const void* weight[2] = {q_weight, k_weight};
  float* grad_weight[2] = {grad_q_weight, grad_k_weight};
  return run_qk(true, x, dy, out, strides, dtype, tokens, heads, head_dim, rot_dim, interleaved, weight, weight_dtype,
                grad_weight, eps, table, table_rows, positions, position_bytes, workspace, workspace_bytes, stream);
}

}  // extern "C"
