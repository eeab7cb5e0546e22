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
//
// Every value is read and written once, so large calls are bound by memory. A
// row stays in registers from its first sum to its last: a team of warps shares
// it, 8 or 16 values a lane, and copies the row that it takes next to shared
// memory while it computes one. (With two or three rows on their way the reads
// and the writes disturb each other: 16384 rows of 4096 bf16 with an fp32
// residual 134 us, with one 121.)
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int BN_WARPS = 16;        // of a block at most
constexpr size_t BN_SMEM = 224 * 1024;
// Blocks of an SM, by the registers and the copies of their rows.
constexpr int bn_blocks(bool grad, int values) { return grad || values > 8 ? 1 : 2; }
constexpr int BN_ANY_THREADS = 256;
constexpr int BN_MAX_BLOCKS = 608;  // of a gradient launch, each with its own sums of dp and dw
// Of a block that joins partial sums: few enough to stand beside the gradient's blocks and wait there (200 rows of 8192
// bf16 backward 15.8 us, with 32 warps 17.0).
constexpr int BN_SUM_WARPS = 8;
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
  int gate_kind, post, weight_fp32;
  float alpha, beta, eps;
  float* partial;                  // gradient: [blocks][2][dim], dp and dw
  // rows in registers: inputs and outputs by their place, with steps from row to row in bytes
  const void* src[5];
  void* dst[3];
  int src_step[5], dst_step[3], place[5], wide[5];
  int warps, teams;                // of a row, rows of a block
  int stage;                       // 16-byte words of a warp's part of a row
  int places;                      // rows of a warp in shared memory: the one in use, and the next where there is room
};

template <typename T>
__device__ __forceinline__ float weight_of(const BlockNormParams& p, const void* w, long long d) {
  if (!w) return 1.0f;
  return p.weight_fp32 ? static_cast<const float*>(w)[d] : to_float(static_cast<const T*>(w)[d]);
}

// ----------------------------------------------------------- rows in registers
// The warps that share a row. Sums go through shared memory, where every other
// one has its own place, so that one barrier is enough.
struct RowTeam {
  int warps, warp, id, lane, turn;
  float* parts;  // [2][warps][4]
  __device__ __forceinline__ RowTeam(const BlockNormParams& p, float* of_block)
      : warps(p.warps), warp((threadIdx.x >> 5) % p.warps), id((threadIdx.x >> 5) / p.warps), lane(threadIdx.x & 31), turn(0),
        parts(of_block + id * p.warps * 8) {}
  static __device__ __forceinline__ float from(float x, int distance) { return __shfl_xor_sync(0xffffffffu, x, distance); }
  // N values, each summed over the team's lanes, in all of them. Half of the lanes go on with one half of the values:
  // three take 6 exchanges in a warp and 6 among the warps, where one after the other they took 30.
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
    static_assert(N <= 3, "places");
    constexpr int S = N == 3 ? 4 : N;  // places of a warp; place i is summed in lane i * 32 / S
    float x;
    if constexpr (N == 1) {
      x = v[0] + from(v[0], 16);
      x += from(x, 8);
    } else if constexpr (N == 2) {
      const bool upper = lane & 16;
      x = (upper ? v[1] : v[0]) + from(upper ? v[0] : v[1], 16);
      x += from(x, 8);
    } else {
      const bool upper = lane & 16, odd = lane & 8;
      const float a = (upper ? v[2] : v[0]) + from(upper ? v[0] : v[2], 16), b = (upper ? 0.0f : v[1]) + from(upper ? v[1] : 0.0f, 16);
      x = (odd ? b : a) + from(odd ? a : b, 8);
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) x += from(x, o);
    if (warps == 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x, i * 32 / S);
      return;
    }
    float* const to = parts + turn * warps * 4;
    turn ^= 1;
    if (lane % (32 / S) == 0) to[warp * S + lane / (32 / S)] = x;
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(32 * warps) : "memory");
    x = lane < warps * S ? to[lane] : 0.0f;
    if (S == 4 && warps > 8) x += lane + 32 < warps * S ? to[lane + 32] : 0.0f;
#pragma unroll
    for (int o = S; o < 32; o <<= 1) x += from(x, o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = N == 1 ? x : __shfl_sync(0xffffffffu, x, i);
  }
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Places of a warp's rows in shared memory, and their addresses in memory.
enum Input { IN_DN = 0, IN_BRANCH = 0, IN_X = 1, IN_DH = 2, IN_GRAD_BRANCH = 3, IN_GATE = 4, INPUTS = 5 };
enum Output { OUT_N = 0, OUT_H = 1, OUT_DBRANCH = 0, OUT_DX = 1, OUT_DGATE = 2, OUTPUTS = 3 };

// NV values of a lane: units of V, a unit's values side by side, units 32 * V *
// warps apart. Columns past the last are zero throughout.
template <typename T, typename R, int NV, bool GRAD, bool FULL>
struct Lanes {
  static constexpr int N = NV / 2, V = 16 / sizeof(T), U = NV / V, RW = sizeof(R) / sizeof(T);  // RW: words of a unit of R
  const BlockNormParams& p;
  const RowTeam& team;
  uint4* ring;         // the warp's
  const uint4* zeros;  // for inputs that are not there
  const float* weight; // the block's, [2][columns of a row]
  int dim, fill, take;

  __device__ __forceinline__ Lanes(const BlockNormParams& params, const RowTeam& t, uint4* smem)
      : p(params), team(t), ring(smem + (threadIdx.x >> 5) * 2 * params.stage), dim(static_cast<int>(params.dim)),
        fill(0), take(0) {
    uint4* const behind = smem + p.warps * p.teams * 2 * p.stage;
    zeros = behind;
    weight = reinterpret_cast<float*>(behind + 32 * U * RW);
  }
  // Fills what the copies leave: zeros, the weights (by the block's first team). The block's call.
  __device__ __forceinline__ void prepare() const {
    uint4* const z = const_cast<uint4*>(zeros);
    for (int i = threadIdx.x; i < 32 * U * RW; i += blockDim.x) z[i] = make_uint4(0, 0, 0, 0);
    if (team.id == 0) {
      put_weights(p.branch_weight, 0);
      put_weights(p.weight, 1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (of_warp(u) + 32 * V <= dim) continue;
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        const bool x = first(u) >= dim && j == 0, r = of_warp(u) + (j * 32 + team.lane) * (V / RW) >= dim;
        for (int at = 0; at <= p.stage; at += p.stage)
          for (int k = 0; k < INPUTS; ++k)
            if (p.src[k] && (p.wide[k] ? r : x)) ring[at + p.place[k] + u * (p.wide[k] ? RW : 1) * 32 + (p.wide[k] ? place<RW>(j * 32 + team.lane) : team.lane)] = make_uint4(0, 0, 0, 0);
      }
    }
    __syncthreads();
  }
  // Where values i to i + 3 of the lane's unit u have their weights: those of 32 lanes side by side.
  __device__ __forceinline__ int quad(int u, int i) const { return of_warp(u) + i / 4 * 128 + team.lane * 4; }
  __device__ __forceinline__ void put_weights(const void* w, int which) const {
    float* const to = const_cast<float*>(weight) + which * team.warps * 32 * NV;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = first(u) < dim ? 1.0f : 0.0f;
      if (w && first(u) < dim) {
        if (sizeof(T) == 2 && p.weight_fp32) {
#pragma unroll
          for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(f + i) = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + first(u) + i);
        } else {
          const Vec<T, V> x = load_vec<T, V>(static_cast<const T*>(w) + first(u));
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = get(x, i);
        }
      }
#pragma unroll
      for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(to + quad(u, i)) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
  }
  // Which inputs and outputs there are.
  __device__ __forceinline__ bool in(int k) const { return FULL ? k < IN_GATE : p.src[k] != nullptr; }
  __device__ __forceinline__ bool out(int k) const { return FULL ? k < OUT_DGATE : p.dst[k] != nullptr; }
  // Place of word w of a unit of W words a lane. The gradient reads two words side by side without conflicts (16384 rows
  // of 2048 bf16 with an fp32 residual 101 us against 106); forward, where memory alone is the limit, the plain order is
  // the faster one (65 against 69).
  template <int W>
  static __device__ __forceinline__ int place(int w) {
    return GRAD && W == 2 ? w ^ ((w >> 3) & 1) : w;
  }
  // First value of the warp's unit u, of the lane's.
  __device__ __forceinline__ int of_warp(int u) const { return (u * team.warps + team.warp) * 32 * V; }
  __device__ __forceinline__ int first(int u) const { return of_warp(u) + team.lane * V; }
  // The warp's part of a row of input k on its way.
  template <typename E>
  __device__ __forceinline__ void fetch(int k, int t) const {
    constexpr int W = sizeof(E) / sizeof(T), VE = 16 / sizeof(E);  // words of a unit, values of a word
    if (!in(k)) return;
    const char* const row = static_cast<const char*>(p.src[k]) + static_cast<long long>(t) * p.src_step[k];
    uint4* const to = ring + fill + p.place[k];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int d = of_warp(u) + (j * 32 + team.lane) * VE;
        if (d < dim) nsptx::cp_async16(to + u * W * 32 + place<W>(j * 32 + team.lane), row + d * static_cast<int>(sizeof(E)));
      }
  }
  __device__ __forceinline__ void fetched() {
    nsptx::cp_async_commit();
    fill = p.stage - fill;
  }
  // The row on its way is there, for all lanes of the warp; and all have read the one before.
  __device__ __forceinline__ void wait(int) const {
    nsptx::cp_async_wait<0>();
    __syncwarp();
  }
  __device__ __forceinline__ void taken() { take = p.stage - take; }
  template <typename E>
  __device__ __forceinline__ void get_row(int k, float2 (&v)[N]) const {
    constexpr int W = sizeof(E) / sizeof(T), VE = 16 / sizeof(E);
    const uint4* const from = in(k) ? ring + take + p.place[k] : zeros;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        Vec<E, VE> x;
        *reinterpret_cast<uint4*>(&x) = from[u * W * 32 + place<W>(team.lane * W + j)];
#pragma unroll
        for (int i = 0; i < VE; i += 2) v[(u * V + j * VE + i) / 2] = make_float2(get(x, i), get(x, i + 1));
      }
  }
  template <typename E>
  __device__ __forceinline__ void put_row(int k, int t, const float2 (&v)[N]) const {
    constexpr int W = sizeof(E) / sizeof(T), VE = 16 / sizeof(E);
    if (!out(k)) return;
    char* const to = static_cast<char*>(p.dst[k]) + static_cast<long long>(t) * p.dst_step[k];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      E* const row = reinterpret_cast<E*>(to + first(u) * static_cast<int>(sizeof(E)));
      if constexpr (W == 2) {  // 32 bytes at once
        if (first(u) < dim)
          asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row), "f"(v[u * 4].x), "f"(v[u * 4].y),
                       "f"(v[u * 4 + 1].x), "f"(v[u * 4 + 1].y), "f"(v[u * 4 + 2].x), "f"(v[u * 4 + 2].y), "f"(v[u * 4 + 3].x),
                       "f"(v[u * 4 + 3].y)
                       : "memory");
      } else {
        float f[VE];
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          f[i] = v[(u * V + i) / 2].x;
          f[i + 1] = v[(u * V + i) / 2].y;
        }
        if (first(u) < dim) store_vec<E, VE>(row, pack<E, VE>(f));
      }
    }
  }
  // A lane's sums of the weights' gradients to their columns of [2][dim].
  __device__ __forceinline__ void join(float* to, const float2 (&dp)[N], const float2 (&dw)[N]) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (first(u) >= dim) continue;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        *reinterpret_cast<float2*>(to + first(u) + 2 * i) = dp[u * V / 2 + i];
        *reinterpret_cast<float2*>(to + dim + first(u) + 2 * i) = dw[u * V / 2 + i];
      }
    }
  }
  // A token's own gate, on its way with the row; 1 where there are none.
  __device__ __forceinline__ void fetch_gate(int t) const {
    if (p.gate_kind == TOKEN_GATE && team.lane == 0) nsptx::cp_async4(ring + fill + p.stage - 1, static_cast<const float*>(p.gate) + t);
  }
  __device__ __forceinline__ float gate() const {
    return p.gate_kind == TOKEN_GATE ? *reinterpret_cast<const float*>(ring + take + p.stage - 1) : 1.0f;
  }
  // Weights of the lane's columns: of the branch (0), of the norm after (1).
  __device__ __forceinline__ void weights(int which, float2 (&v)[N]) const {
    const float* const from = weight + which * team.warps * 32 * NV;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(from + quad(u, i));
        v[(u * V + i) / 2] = make_float2(f.x, f.y);
        v[(u * V + i) / 2 + 1] = make_float2(f.z, f.w);
      }
  }
};

// The same for rows of any width, stride and alignment: a warp has 32 * NV columns
// side by side, copies the aligned 16-byte words that cover them and takes them
// from shared memory value by value. (Value by value from memory 8196 rows of 2047
// bf16 took 313 us backward and 59 forward, so 91 and 46; 5003 rows of 1001 fp16
// without a branch, which L2 holds, took 8.0 us, so 9.2.) Bound by instructions.
template <typename T, typename R, int NV, bool GRAD>
struct Singles {
  static constexpr int N = NV / 2;
  const BlockNormParams& p;
  const RowTeam& team;
  uint4* ring;          // the warp's
  const float* weight;  // the block's, [2][columns of a row]
  int first, count;     // columns of the warp
  int fill, take, row;

  __device__ __forceinline__ Singles(const BlockNormParams& params, const RowTeam& t, uint4* smem)
      : p(params), team(t), ring(smem + (threadIdx.x >> 5) * p.places * p.stage),
        weight(reinterpret_cast<float*>(smem + p.warps * p.teams * p.places * p.stage)), first(t.warp * 32 * NV),
        count(min(static_cast<int>(p.dim) - first, 32 * NV)), fill(0), take(0), row(0) {}
  // Words of a warp's columns of E, wherever they start.
  template <typename E>
  static constexpr int WORDS_OF = 2 * NV * sizeof(E) + 1;
  __device__ __forceinline__ void prepare() const {
    float* const to = const_cast<float*>(weight);
    const int columns = 32 * NV * team.warps;
    for (int i = threadIdx.x; i < columns; i += blockDim.x) {
      to[i] = i < p.dim ? weight_of<T>(p, p.branch_weight, i) : 0.0f;
      to[columns + i] = i < p.dim ? weight_of<T>(p, p.weight, i) : 0.0f;
    }
    __syncthreads();
  }
  template <typename E>
  __device__ __forceinline__ const char* columns_of(int k, int t) const {
    return static_cast<const char*>(p.src[k]) + static_cast<long long>(t) * p.src_step[k] + first * static_cast<int>(sizeof(E));
  }
  // The words begin in the row or, from the second row on, in the one before or between the two. What is before the
  // first row is not the matrix's: its word there is put together from its values.
  template <typename E>
  __device__ __forceinline__ void fetch(int k, int t) const {
    if (!p.src[k]) return;
    const char* const from = columns_of<E>(k, t);
    const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15), bytes = skip + count * static_cast<int>(sizeof(E));
    uint4* const to = ring + fill + p.place[k];
#pragma unroll
    for (int w0 = 0; w0 < WORDS_OF<E>; w0 += 32) {
      const int w = w0 + team.lane;
      const char* const q = from - skip + 16 * w;
      if (16 * w >= bytes) break;
      if (q >= static_cast<const char*>(p.src[k])) {
        nsptx::cp_async16_upto(to + w, q, min(16, bytes - 16 * w));
      } else {
        for (int i = 0; i < count && skip + i * static_cast<int>(sizeof(E)) < 16; ++i)
          *reinterpret_cast<E*>(reinterpret_cast<char*>(to) + skip + i * sizeof(E)) = reinterpret_cast<const E*>(from)[i];
      }
    }
  }
  __device__ __forceinline__ void fetched() {
    nsptx::cp_async_commit();
    fill = p.places == 2 ? p.stage - fill : 0;
  }
  __device__ __forceinline__ void wait(int t) {
    nsptx::cp_async_wait<0>();
    __syncwarp();
    row = t;
  }
  __device__ __forceinline__ void taken() { take = p.places == 2 ? p.stage - take : 0; }
  template <typename E>
  __device__ __forceinline__ void get_row(int k, float2 (&v)[N]) const {
    const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(columns_of<E>(k, row)) & 15);
    const E* const from = reinterpret_cast<const E*>(reinterpret_cast<const char*>(ring + take + p.place[k]) + skip);
    float f[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) f[i] = p.src[k] && i * 32 + team.lane < count ? to_float(from[i * 32 + team.lane]) : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
  }
  template <typename E>
  __device__ __forceinline__ void put_row(int k, int t, const float2 (&v)[N]) const {
    if (!p.dst[k]) return;
    E* const to = reinterpret_cast<E*>(static_cast<char*>(p.dst[k]) + static_cast<long long>(t) * p.dst_step[k]) + first;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * 32 + team.lane < count) to[i * 32 + team.lane] = from_float<E>(i % 2 ? v[i / 2].y : v[i / 2].x);
  }
  __device__ __forceinline__ void fetch_gate(int t) const {
    if (p.gate_kind == TOKEN_GATE && team.lane == 0) nsptx::cp_async4(ring + fill + p.stage - 1, static_cast<const float*>(p.gate) + t);
  }
  __device__ __forceinline__ float gate() const {
    return p.gate_kind == TOKEN_GATE ? *reinterpret_cast<const float*>(ring + take + p.stage - 1) : 1.0f;
  }
  __device__ __forceinline__ void weights(int which, float2 (&v)[N]) const {
    const float* const from = weight + which * team.warps * 32 * NV + first + team.lane;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(from[2 * i * 32], from[(2 * i + 1) * 32]);
  }
  // A lane's sums of the weights' gradients to their columns of [2][dim].
  __device__ __forceinline__ void join(float* to, const float2 (&dp)[N], const float2 (&dw)[N]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * 32 + team.lane >= count) continue;
      to[first + i * 32 + team.lane] = i % 2 ? dp[i / 2].y : dp[i / 2].x;
      to[p.dim + first + i * 32 + team.lane] = i % 2 ? dw[i / 2].y : dw[i / 2].x;
    }
  }
};

template <typename T, typename R, int NV, bool WORDS>
__global__ void __launch_bounds__(32 * BN_WARPS, bn_blocks(false, NV)) ns_block_norm_kernel(const __grid_constant__ BlockNormParams p) {
  extern __shared__ uint4 rows_smem[];
  __shared__ float parts[BN_WARPS * 8];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  constexpr int N = NV / 2;
  RowTeam team(p, parts);
  typename std::conditional<WORDS, Lanes<T, R, NV, false, false>, Singles<T, R, NV, false>>::type lanes(p, team, rows_smem);
  const float inv_dim = 1.0f / p.dim;
  const float2 alpha = both(p.alpha);
  const bool gated = p.gate_kind == VALUE_GATE;
  const int tokens = static_cast<int>(p.tokens), stride = gridDim.x * p.teams, t0 = blockIdx.x * p.teams + team.id;
  auto fetch = [&](int t) {
    if (t < tokens) {
      lanes.template fetch<T>(IN_BRANCH, t);
      lanes.template fetch<R>(IN_X, t);
      lanes.template fetch<T>(IN_GATE, t);
      lanes.fetch_gate(t);
    }
    lanes.fetched();
  };
  fetch(t0);
  lanes.prepare();
  for (int t = t0; t < tokens; t += stride) {
    lanes.wait(t);
    if (WORDS || p.places == 2) fetch(t + stride);
    float2 b[N], h[N];
    const float2 beta = both(p.beta * lanes.gate());
    float2 w[N];
    lanes.template get_row<T>(IN_BRANCH, b);
    lanes.template get_row<R>(IN_X, h);
    if (p.branch) {
      lanes.weights(0, w);
      float r1[1] = {1.0f};
      if (p.post) {
        float2 s = both(0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) s = fma2(b[i], b[i], s);
        r1[0] = s.x + s.y;
        team.sum(r1);
        r1[0] = rsqrtf(fmaf(r1[0], inv_dim, p.eps));
      }
#pragma unroll
      for (int i = 0; i < N; ++i) b[i] = mul2(mul2(b[i], both(r1[0])), w[i]);
      if (gated) {
        float2 g[N];
        lanes.template get_row<T>(IN_GATE, g);
#pragma unroll
        for (int i = 0; i < N; ++i) b[i] = mul2(b[i], g[i]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] = fma2(beta, b[i], mul2(alpha, h[i]));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] = mul2(alpha, h[i]);
    }
    lanes.taken();
    if (!WORDS && p.places == 1) {
      __syncwarp();
      fetch(t + stride);
    }
    lanes.template put_row<R>(OUT_H, t, h);
    if (!p.n) continue;
    lanes.weights(1, w);
    float2 s = both(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) s = fma2(h[i], h[i], s);
    float r2[1] = {s.x + s.y};
    team.sum(r2);
    r2[0] = rsqrtf(fmaf(r2[0], inv_dim, p.eps));
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = mul2(mul2(h[i], both(r2[0])), w[i]);
    lanes.template put_row<T>(OUT_N, t, h);
  }
}

template <typename T, typename R, int NV, bool WORDS, bool FULL>
__global__ void __launch_bounds__(32 * BN_WARPS, bn_blocks(true, NV)) ns_block_norm_grad_kernel(const __grid_constant__ BlockNormParams p) {
  extern __shared__ uint4 rows_smem[];
  __shared__ float parts[BN_WARPS * 8];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  constexpr int N = NV / 2;
  RowTeam team(p, parts);
  typename std::conditional<WORDS, Lanes<T, R, NV, true, FULL>, Singles<T, R, NV, true>>::type lanes(p, team, rows_smem);
  const float inv_dim = 1.0f / p.dim;
  const bool gated = !FULL && p.gate_kind == VALUE_GATE, has_dn = FULL || p.dn, has_dx = FULL || p.dx, has_branch = FULL || p.branch, post = FULL || p.post;
  const int tokens = static_cast<int>(p.tokens), stride = gridDim.x * p.teams, t0 = blockIdx.x * p.teams + team.id;
  auto fetch = [&](int t) {
    if (t < tokens) {
      lanes.template fetch<T>(IN_DN, t);
      lanes.template fetch<R>(IN_X, t);
      lanes.template fetch<R>(IN_DH, t);
      lanes.template fetch<T>(IN_GRAD_BRANCH, t);
      lanes.template fetch<T>(IN_GATE, t);
      lanes.fetch_gate(t);
    }
    lanes.fetched();
  };
  float2 dp[N], dw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dp[i] = dw[i] = both(0.0f);
  fetch(t0);
  lanes.prepare();
  for (int t = t0; t < tokens; t += stride) {
    lanes.wait(t);
    if (WORDS || p.places == 2) fetch(t + stride);
    float2 v[N], h[N], d[N], b[N], w[N];
    const float gt = lanes.gate();
    lanes.weights(1, w);
    lanes.template get_row<T>(IN_DN, v);
    lanes.template get_row<R>(IN_X, h);
    lanes.template get_row<R>(IN_DH, d);
    lanes.template get_row<T>(IN_GRAD_BRANCH, b);
    float2 s0 = both(0.0f), s1 = s0, s2 = s0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s0 = fma2(h[i], h[i], s0);
      s1 = fma2(mul2(v[i], w[i]), h[i], s1);
      s2 = fma2(b[i], b[i], s2);
    }
    float sum[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
    team.sum(sum);
    if (has_dn) {
      const float r = rsqrtf(fmaf(sum[0], inv_dim, p.eps)), mean = sum[1] * r * inv_dim;
      const float2 r2 = both(r), minus = both(-mean);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 m = mul2(h[i], r2);
        dw[i] = fma2(v[i], m, dw[i]);
        d[i] = fma2(r2, fma2(m, minus, mul2(v[i], w[i])), d[i]);  // t
      }
    }
    if (has_dx) {
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] = mul2(d[i], both(p.alpha));
      lanes.template put_row<R>(OUT_DX, t, h);
    }
    if (has_branch) {
      const float r1 = post ? rsqrtf(fmaf(sum[2], inv_dim, p.eps)) : 1.0f;
      lanes.weights(0, w);
      float2 g[N];
      if (gated) {
        lanes.template get_row<T>(IN_GATE, g);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = both(gt);
      }
      s0 = s1 = both(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 tb = mul2(d[i], both(p.beta)), s = mul2(tb, g[i]);
        b[i] = mul2(b[i], both(r1));          // y
        dp[i] = fma2(s, b[i], dp[i]);
        g[i] = mul2(tb, mul2(b[i], w[i]));    // of the gate
        s1 = add2(s1, g[i]);
        d[i] = mul2(s, w[i]);                 // z
        s0 = fma2(d[i], b[i], s0);
      }
      if (gated) lanes.template put_row<T>(OUT_DGATE, t, g);
      float sums[2] = {s0.x + s0.y, s1.x + s1.y};
      if (post || (p.dgate && !gated)) team.sum(sums);
      if (p.dgate && !gated && team.warp == 0 && team.lane == 0) static_cast<float*>(p.dgate)[t] = sums[1];
      if (post) {
        const float2 minus = both(-sums[0] * inv_dim);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = mul2(fma2(b[i], minus, d[i]), both(r1));
      }
      lanes.template put_row<T>(OUT_DBRANCH, t, d);
    }
    lanes.taken();
    if (!WORDS && p.places == 1) {
      __syncwarp();
      fetch(t + stride);
    }
  }
  if (!p.partial) return;
  // the block's teams, in order; the rings are done with
  nsptx::cp_async_wait<0>();
  __syncthreads();
  float* const joined = reinterpret_cast<float*>(rows_smem);  // [teams][2][dim]
  const int dim = static_cast<int>(p.dim);
  lanes.join(joined + team.id * 2 * dim, dp, dw);
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * dim; c += blockDim.x) {
    float sum = 0.0f;
    for (int k = 0; k < p.teams; ++k) sum += joined[k * 2 * dim + c];
    p.partial[static_cast<long long>(blockIdx.x) * 2 * dim + c] = sum;
  }
}

// ------------------------------------------------------------- rows of any kind

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
// sums: rows of any width, stride and alignment, for those that registers do not
// hold (4096 rows of 16384 bf16 forward 540 us, backward 1514: 0.15 and 0.08 of the
// measured copy).
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
      if (dp && dn) dw[d] = fmaf(dnv, m, dw[d]);
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
// columns a block, whose warps split the partial sums.
__global__ void __launch_bounds__(32 * BN_SUM_WARPS) ns_block_norm_sum_kernel(const __grid_constant__ BlockNormSumParams p) {
  __shared__ float part[BN_SUM_WARPS][32];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + lane;
  float sum = 0.0f;
  if (col < 2 * p.dim) {
#pragma unroll 8
    for (int b = warp; b < p.blocks; b += BN_SUM_WARPS) sum += p.partial[b * 2 * p.dim + col];
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp || col >= 2 * p.dim) return;
  for (int w = 1; w < BN_SUM_WARPS; ++w) sum += part[w][lane];
  float* out = p.out[col >= p.dim];
  if (out) out[col >= p.dim ? col - p.dim : col] = sum;
}

// NV values a lane; false if the copies of a team's rows do not fit an SM (two of whole words, one value by value), or
// steps an int. Two rows of whole words and the fp32 weights no longer fit backward above 6656 columns of a 16-bit block
// with an fp32 residual (6144 with a gate for each value, 7680 without a branch), 5632 of an fp32 one (4608; 6656), 7680 of
// a 16-bit one with a gate for each value, and forward above 6656 of fp32 with such a gate: those rows are taken value by
// value with nothing on its way (8192 rows of 7168 bf16 with an fp32 residual 346 us, of 6144 172; fp32 rows of 6144 340,
// of 5632 205), fp32 gradients with a gate for each value above 7680 as rows of any kind.
template <typename T, typename R, int NV, bool WORDS>
bool launch_rows(bool grad, BlockNormParams p, int nsm, int* blocks, cudaStream_t st, cudaError_t* e) {
  using L = Lanes<T, R, NV, true, false>;
  using S = Singles<T, R, NV, true>;
  constexpr int BLOCKS[2] = {bn_blocks(false, NV), bn_blocks(true, NV)};
  p.warps = static_cast<int>((p.dim + 32 * NV - 1) / (32 * NV));
  // few rows are spread over the SMs, many share a block
  p.teams = static_cast<int>(std::clamp<long long>((p.tokens + nsm - 1) / nsm, 1, BN_WARPS / p.warps));
  struct {
    const void* at;
    long long ld;
    bool wide;
  } const in[2][INPUTS] = {{{p.branch, p.branch_ld, false}, {p.x, p.x_ld, true}, {}, {}, {p.gate, p.gate_ld, false}},
                           {{p.dn, p.dn_ld, false}, {p.x, p.x_ld, true}, {p.dh, p.dh_ld, true}, {p.branch, p.branch_ld, false}, {p.gate, p.gate_ld, false}}};
  struct {
    void* at;
    long long ld;
    bool wide;
  } const out[2][OUTPUTS] = {{{p.n, p.n_ld, false}, {p.h, p.h_ld, true}, {}},
                             {{p.dbranch, p.dbranch_ld, false}, {p.dx, p.dx_ld, true}, {p.dgate, p.dgate_ld, false}}};
  const bool value = p.gate_kind == VALUE_GATE;
  auto step = [&](long long ld, bool wide, int* bytes) {
    const long long b = p.tokens > 1 ? ld * static_cast<long long>(wide ? sizeof(R) : sizeof(T)) : 0;
    *bytes = static_cast<int>(b);
    return b <= INT_MAX / 4;
  };
  for (int k = 0; k < INPUTS; ++k) {
    const auto& i = in[grad][k];
    p.src[k] = k == IN_GATE && !value ? nullptr : i.at;
    p.wide[k] = i.wide && L::RW == 2;
    p.place[k] = p.stage;
    if (p.src[k]) p.stage += WORDS ? 32 * L::U * (i.wide ? L::RW : 1) : i.wide ? S::template WORDS_OF<R> : S::template WORDS_OF<T>;
    if (p.src[k] && !step(i.ld, i.wide, &p.src_step[k])) return false;
  }
  for (int k = 0; k < OUTPUTS; ++k) {
    const auto& o = out[grad][k];
    p.dst[k] = k == OUT_DGATE && !value ? nullptr : o.at;
    if (p.dst[k] && !step(o.ld, o.wide, &p.dst_step[k])) return false;
  }
  if (p.tokens > INT_MAX / 4) return false;
  if (p.gate_kind == TOKEN_GATE) ++p.stage;
  // a block's rows, zeros, weights
  const size_t row = sizeof(uint4) * p.stage * p.warps * p.teams;
  const size_t more = (WORDS ? sizeof(uint4) * 32 * L::U * L::RW : 0) + sizeof(float) * 2 * 32 * NV * p.warps;
  const int per_sm = 2 * row + more <= BN_SMEM / BLOCKS[grad] ? BLOCKS[grad] : 1;
  p.places = WORDS || 2 * row + more <= BN_SMEM / per_sm ? 2 : 1;
  if (p.places * row + more > BN_SMEM / per_sm) return false;
  const size_t joined = p.partial ? sizeof(float) * 2 * p.dim * p.teams : 0, smem = std::max(p.places * row + more, joined);
  *blocks = static_cast<int>(std::min<long long>((p.tokens + p.teams - 1) / p.teams, std::min(nsm * per_sm, BN_MAX_BLOCKS)));
  void (*kernel)(BlockNormParams) = ns_block_norm_kernel<T, R, NV, WORDS>;
  if (grad) kernel = ns_block_norm_grad_kernel<T, R, NV, WORDS, false>;
  if constexpr (WORDS) {
    // the usual gradient, without a choice for each row
    if (grad && p.post && p.src[IN_DN] && p.src[IN_DH] && p.src[IN_GRAD_BRANCH] && !p.src[IN_GATE] && p.dst[OUT_DBRANCH] && p.dst[OUT_DX])
      kernel = ns_block_norm_grad_kernel<T, R, NV, WORDS, true>;
  }
  *e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(BN_SMEM));
  if (*e == cudaSuccess) *e = launch_pdl(kernel, dim3(*blocks), dim3(32 * p.warps * p.teams), smem, st, p);
  return true;
}

// Whether a matrix's rows are made of aligned 16-byte words.
bool words_ok(const void* base, long long ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 15) == 0 && (!base || ld * bytes % 16 == 0);
}

template <typename T, typename R>
cudaError_t launch_block_norm(bool grad, const BlockNormParams& p, int nsm, int* blocks, cudaStream_t st) {
  constexpr int X = sizeof(T), Y = sizeof(R);
  const bool value = p.gate_kind == VALUE_GATE, many = p.tokens > 1;  // the stride of one row reaches nothing
  auto ok = [&](const void* base, long long ld, int bytes) { return words_ok(base, many ? ld : 0, bytes); };
  const bool words = p.dim % (16 / X) == 0 && ok(p.branch, p.branch_ld, X) && ok(p.x, p.x_ld, Y) &&
                     ok(p.h, p.h_ld, Y) && ok(p.n, p.n_ld, X) && ok(p.dh, p.dh_ld, Y) && ok(p.dn, p.dn_ld, X) &&
                     ok(p.dbranch, p.dbranch_ld, X) && ok(p.dx, p.dx_ld, Y) && ok(p.branch_weight, 0, 1) && ok(p.weight, 0, 1) &&
                     (!value || (ok(p.gate, p.gate_ld, X) && ok(p.dgate, p.dgate_ld, X)));
  // 32 bytes of an fp32 residual are stored at once
  const bool wide = Y == X || ((reinterpret_cast<uintptr_t>(p.h) | reinterpret_cast<uintptr_t>(p.dx)) % 32 == 0 &&
                               (!many || (p.h_ld % 8 == 0 && p.dx_ld % 8 == 0)));
  if (p.dim <= 32 * BN_WARPS * 16) {
    const bool few = p.dim <= 32 * BN_WARPS * 8;
    cudaError_t e;
    if (words && wide && (few ? launch_rows<T, R, 8, true>(grad, p, nsm, blocks, st, &e) : launch_rows<T, R, 16, true>(grad, p, nsm, blocks, st, &e)))
      return e;
    if (few ? launch_rows<T, R, 8, false>(grad, p, nsm, blocks, st, &e) : launch_rows<T, R, 16, false>(grad, p, nsm, blocks, st, &e)) return e;
  }
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
    return nsk::launch_pdl(nsk::ns_block_norm_sum_kernel, dim3(static_cast<unsigned>((2 * dim + 31) / 32)), dim3(32 * nsk::BN_SUM_WARPS), 0, st, sp);
  });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

}  // extern "C"
