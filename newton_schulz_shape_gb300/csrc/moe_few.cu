// A whole mixture-of-experts layer for a few tokens: each token's experts, their
// gated products and the weighted sum, in two kernels.
//
//   h_s = silu(G_e x_t) * (U_e x_t)     for slot s = (t, j) with expert e
//   y_t = sum over j of w_tj D_e h_s
// with silu(a) = a / (1 + exp(-a)).
//
// The weights of the experts that are named, 3 dim ffn values each, are read
// once and are nearly all of the bytes, so the layer is bound by memory: n
// tokens of an expert make 2 n operations of each value. The products run on
// m16n8k16 tensor instructions on registers (16 rows of weights, 8 tokens),
// which keep pace up to some 30 tokens an expert, because the weights then go
// from global memory to their instruction without a stop in shared memory: the
// order of k within a product is free, so a lane takes 16 consecutive bytes of a
// row and the tokens' values in the same order. Blocks find the tokens of their
// expert among all slots themselves, which spares a kernel.
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int MF_WARPS = 4;                  // of a block, which split k
constexpr int MF_THREADS = 32 * MF_WARPS;
constexpr int MF_BLOCKS = 4;                 // of an SM
constexpr int MF_AHEAD = 16;                 // 16-byte words of weights that a lane has on their way
constexpr int MF_MAX_TOKENS = 256;
constexpr int MF_SUM_ROWS = 32;              // rows of y that are summed together
constexpr int MF_NT = 4;                     // groups of 8 tokens that a pass over the weights serves

struct MoeFewParams {
  const void *x, *gate_up, *down;
  void* y;
  const void* ids;
  int id_bytes, tokens, k, experts;
  long long x_ld, y_ld, dim, ffn;
  long long hidden_ld, part_ld;  // values of a slot's rows below
  const float* weights;
  void* hidden;        // [tokens * k][hidden_ld] of 4 bytes: h in fp32, or as two bf16 rows
  float* part;         // [tokens * k][part_ld]: D_e h
  unsigned int* arrived;  // [dim / MF_SUM_ROWS]: blocks whose part of these rows of y is there
  int groups;          // row tiles that a block takes, one after the other
  unsigned int* status;
};

// ------------------------------------------------------- tokens of an expert
// What a block knows of the slots: `expert` [slots] (-1: goes nowhere), and the
// slots of its own expert in `list`.
struct Slots {
  short* expert;
  short* list;
};

// The block's expert, the nth of those that are named, -1 if there are fewer.
// *named: how many; *count: slots of the expert, in order in s.list.
__device__ __forceinline__ int find_expert(const MoeFewParams& p, const Slots& s, int nth, int* named, int* count) {
  __shared__ unsigned int bits[32];
  __shared__ int found[3];
  const int lane = threadIdx.x & 31, slots = p.tokens * p.k;
  if (threadIdx.x < 32) bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += MF_THREADS) {
    long long e = load_index(p.ids, p.id_bytes, i);
    if (e >= p.experts) {
      atomicOr(p.status, NS_DEV_BAD_INDEX);
      e = -1;
    }
    if (e >= 0) atomicOr(&bits[e >> 5], 1u << (e & 31));
    s.expert[i] = static_cast<short>(e < 0 ? -1 : e);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const unsigned int word = bits[lane];
    int upto = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    const unsigned int over = __ballot_sync(0xffffffffu, upto > nth);
    int e = -1;
    if (over) {
      const int at = __ffs(over) - 1;
      const int before = __shfl_sync(0xffffffffu, upto - __popc(word), at);
      unsigned int w = __shfl_sync(0xffffffffu, word, at);
      for (int i = before; i < nth; ++i) w &= w - 1;
      e = at * 32 + __ffs(w) - 1;
    }
    int n = 0;
    if (e >= 0) {
      for (int i0 = 0; i0 < slots; i0 += 32) {
        const bool mine = i0 + lane < slots && s.expert[i0 + lane] == e;
        const unsigned int who = __ballot_sync(0xffffffffu, mine);
        if (mine) s.list[n + __popc(who & ((1u << lane) - 1))] = static_cast<short>(i0 + lane);
        n += __popc(who);
      }
    }
    if (lane == 0) {
      found[0] = e;
      found[1] = all;
      found[2] = n;
    }
  }
  __syncthreads();
  *named = found[1];
  *count = found[2];
  return found[0];
}

// ------------------------------------------------------------------ products
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_tf32_8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ void mma_16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x = *hi + *lo with *hi of tf32's 11 significant bits; the instruction drops
// the last bits of *lo, 2^-22 of x. An infinity stays in *hi alone.
__device__ __forceinline__ void split(float x, uint32_t* hi, uint32_t* lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(*hi) : "f"(x));
  const float h = __uint_as_float(*hi);
  *lo = __float_as_uint(x == h ? 0.0f : x - h);
}

// 16 bytes of consecutive values of a row from k on, zero from n on. VEC: rows
// are made of aligned 16-byte words.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_row(const T* row, int k, int n) {
  constexpr int V = 16 / sizeof(T);
  if constexpr (VEC) {
    return k < n ? load_stream(row + k) : make_uint4(0, 0, 0, 0);
  } else {
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = k + i < n ? to_float(row[k + i]) : 0.0f;
    const Vec<T, V> v = pack<T, V>(f);
    return *reinterpret_cast<const uint4*>(&v);
  }
}

// The tokens' side of a product, 16 bytes' worth of k: of x, or (HIDDEN) of h.
// bf16 and fp16 products of x are exact; an fp32 factor is split in two. h has
// more bits and a larger range than 16-bit types: it meets bf16 weights as two
// bf16 values (2^-18 off), and fp16 weights, which tf32 holds, as two tf32 values.
template <typename T, bool HIDDEN>
struct Side {
  static constexpr int V = 16 / sizeof(T);
  static constexpr bool PAIR = HIDDEN && std::is_same<T, __nv_bfloat16>::value;
  static constexpr bool WIDE = sizeof(T) == 4 || (HIDDEN && !PAIR);
  uint32_t hi[WIDE ? V : 4], lo[WIDE ? V : PAIR ? 4 : 1];

  template <bool VEC>
  __device__ __forceinline__ void load(const MoeFewParams& p, int slot, int k, int n) {
    if (HIDDEN) {
      if constexpr (PAIR) {
        const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(p.hidden) + slot * 2 * p.hidden_ld + k;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (slot >= 0 && k < n) {
          a = *reinterpret_cast<const uint4*>(h);
          b = *reinterpret_cast<const uint4*>(h + p.hidden_ld);
        }
        hi[0] = a.x, hi[1] = a.y, hi[2] = a.z, hi[3] = a.w;
        lo[0] = b.x, lo[1] = b.y, lo[2] = b.z, lo[3] = b.w;
      } else {
        const float* h = static_cast<const float*>(p.hidden) + slot * p.hidden_ld + k;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 f = slot >= 0 && k < n ? *reinterpret_cast<const float4*>(h + i) : make_float4(0, 0, 0, 0);
          split(f.x, &hi[i], &lo[i]);
          split(f.y, &hi[i + 1], &lo[i + 1]);
          split(f.z, &hi[i + 2], &lo[i + 2]);
          split(f.w, &hi[i + 3], &lo[i + 3]);
        }
      }
    } else {
      uint4 a = make_uint4(0, 0, 0, 0);
      if (slot >= 0) {
        const T* x = static_cast<const T*>(p.x) + (slot / p.k) * p.x_ld;
        if constexpr (VEC) {
          if (k < n) a = *reinterpret_cast<const uint4*>(x + k);
        } else {
          a = load_row<T, false>(x, k, n);
        }
      }
      if constexpr (WIDE) {
        split(__uint_as_float(a.x), &hi[0], &lo[0]);
        split(__uint_as_float(a.y), &hi[1], &lo[1]);
        split(__uint_as_float(a.z), &hi[2], &lo[2]);
        split(__uint_as_float(a.w), &hi[3], &lo[3]);
      } else {
        hi[0] = a.x, hi[1] = a.y, hi[2] = a.z, hi[3] = a.w;
      }
    }
  }
};

// The weights' side: rows r and r + 8 of a tile.
template <typename T, bool HIDDEN>
struct Rows {
  using S = Side<T, HIDDEN>;
  static constexpr int V = S::V;
  uint32_t hi[2][S::WIDE ? V : 4], lo[2][sizeof(T) == 4 ? V : 1];
  __device__ __forceinline__ Rows(const uint4& r, const uint4& r8) {
    const uint32_t w[2][4] = {{r.x, r.y, r.z, r.w}, {r8.x, r8.y, r8.z, r8.w}};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          split(__uint_as_float(w[j][i]), &hi[j][i], &lo[j][i]);
        } else if constexpr (S::WIDE) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j][i]));
          hi[j][2 * i] = __float_as_uint(f.x);
          hi[j][2 * i + 1] = __float_as_uint(f.y);
        } else {
          hi[j][i] = w[j][i];
        }
      }
    }
  }
  __device__ __forceinline__ void times(float (&c)[4], const S& b) const {
    if constexpr (S::WIDE) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        mma_tf32_8(c, hi[0][i], hi[1][i], hi[0][i + 1], hi[1][i + 1], b.hi[i], b.hi[i + 1]);
        mma_tf32_8(c, hi[0][i], hi[1][i], hi[0][i + 1], hi[1][i + 1], b.lo[i], b.lo[i + 1]);
        if constexpr (sizeof(T) == 4)
          mma_tf32_8(c, lo[0][i], lo[1][i], lo[0][i + 1], lo[1][i + 1], b.hi[i], b.hi[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        mma_16<T>(c, hi[0][i], hi[1][i], hi[0][i + 1], hi[1][i + 1], b.hi[i], b.hi[i + 1]);
        if constexpr (S::PAIR) mma_16<T>(c, hi[0][i], hi[1][i], hi[0][i + 1], hi[1][i + 1], b.lo[i], b.lo[i + 1]);
      }
    }
  }
};

// A warp's share of the products of one tile of 16 rows with 8 * NT tokens: the
// 16-byte steps of k that fall to it. `top` and `low` are the lane's rows r and
// r + 8 (null: past the last).
template <typename T, bool HIDDEN, bool VEC, int NT>
__device__ __forceinline__ void tile_product(const MoeFewParams& p, const T* top, const T* low, int n, const int (&slot)[NT],
                                             float (&acc)[NT][4]) {
  constexpr int V = 16 / sizeof(T), U = MF_AHEAD / 2, STEP = 4 * V * MF_WARPS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int k = (warp * 4 + (lane & 3)) * V;
  uint4 a[U], b[U];
  auto fetch = [&](int u, int at) {
    a[u] = top ? load_row<T, VEC>(top, at, n) : make_uint4(0, 0, 0, 0);
    b[u] = low ? load_row<T, VEC>(low, at, n) : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(u, k + u * STEP);
  // as many steps for every lane: the tensor instructions are the warp's
  const int steps = (n - warp * 4 * V + STEP - 1) / STEP;
  for (int s = 0; s < steps; s += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u < steps) {
        const Rows<T, HIDDEN> rows(a[u], b[u]);
        fetch(u, k + U * STEP);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          Side<T, HIDDEN> side;
          side.template load<VEC>(p, slot[t], k, n);
          rows.times(acc[t], side);
        }
        k += STEP;
      }
    }
  }
}

// The products of a tile with 8 * NT tokens of the list from `first` on, summed
// over the block's warps in a fixed order: use(j, slot, v) gets v[0] and v[1],
// the sums of rows j and j + 8 of the tile for a slot.
template <typename T, bool HIDDEN, bool VEC, int NT, typename F>
__device__ __forceinline__ void tile_of_tokens(const MoeFewParams& p, const T* top, const T* low, int n, const Slots& s,
                                               int first, int count, float (*sums)[32], F&& use) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int slot[NT];
  float acc[NT][4] = {};
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int i = first + 8 * t + lane / 4;
    slot[t] = i < count ? s.list[i] : -1;
  }
  tile_product<T, HIDDEN, VEC, NT>(p, top, low, n, slot, acc);
  __syncthreads();  // the last tile's sums are read
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[(warp * NT + t) * 4 + i][lane] = acc[t][i];
  __syncthreads();
  // a lane holds columns 2 (lane % 4) and the next, rows lane / 4 (values 0, 1) and 8 more (2, 3)
  for (int i = threadIdx.x; i < NT * 2 * 32; i += MF_THREADS) {
    const int at = i & 31, c = (i >> 5) & 1, t = i >> 6, j = first + 8 * t + 2 * (at & 3) + c;
    if (j >= count) continue;
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < MF_WARPS; ++w) {
      v[0] += sums[(w * NT + t) * 4 + c][at];
      v[1] += sums[(w * NT + t) * 4 + c + 2][at];
    }
    use(at >> 2, s.list[j], v);
  }
}

// The same for all tokens of the list, 32 in a pass over the weights.
template <typename T, bool HIDDEN, bool VEC, typename F>
__device__ __forceinline__ void tile_of_list(const MoeFewParams& p, const T* top, const T* low, int n, const Slots& s,
                                             int count, float (*sums)[32], F&& use) {
  for (int first = 0; first < count; first += 8 * MF_NT) {
    const int left = count - first;
    if (left <= 8)
      tile_of_tokens<T, HIDDEN, VEC, 1>(p, top, low, n, s, first, count, sums, use);
    else if (left <= 16)
      tile_of_tokens<T, HIDDEN, VEC, 2>(p, top, low, n, s, first, count, sums, use);
    else
      tile_of_tokens<T, HIDDEN, VEC, MF_NT>(p, top, low, n, s, first, count, sums, use);
  }
}

__device__ __forceinline__ Slots slots_of(const MoeFewParams& p, void* smem) {
  short* const at = static_cast<short*>(smem);
  return {at, at + p.tokens * p.k};
}

// h of an expert's slots: a tile's rows are 8 gate rows and the 8 up rows that
// go with them.
template <typename T, bool VEC>
__global__ void __launch_bounds__(MF_THREADS, MF_BLOCKS) ns_moe_few_hidden_kernel(const __grid_constant__ MoeFewParams p) {
  __shared__ float sums[MF_WARPS * MF_NT * 4][32];
  extern __shared__ short few_smem[];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  // the other kernel's counts, which no earlier kernel still uses
  if (blockIdx.y == 0)
    for (long long i = blockIdx.x * MF_THREADS + threadIdx.x; i * MF_SUM_ROWS < p.dim; i += gridDim.x * MF_THREADS)
      p.arrived[i] = 0;
  const Slots s = slots_of(p, few_smem);
  int named, count;
  const int e = find_expert(p, s, blockIdx.y, &named, &count);
  if (e < 0) return;
  const T* const gate = static_cast<const T*>(p.gate_up) + 2 * e * p.ffn * p.dim;
  for (int g = 0; g < p.groups; ++g) {
    const long long f0 = 8 * (static_cast<long long>(blockIdx.x) * p.groups + g), f = f0 + lane / 4;
    if (f0 >= p.ffn) break;
    const T* const top = f < p.ffn ? gate + f * p.dim : nullptr;
    const T* const low = f < p.ffn ? top + p.ffn * p.dim : nullptr;
    tile_of_list<T, false, VEC>(p, top, low, static_cast<int>(p.dim), s, count, sums, [&](int j, int slot, const float (&v)[2]) {
      // zero up to the end of the last tile: the rows' last words are read whole
      const float h = f0 + j < p.ffn ? v[0] / (1.0f + expf(-v[0])) * v[1] : 0.0f;
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        __nv_bfloat16* const to = static_cast<__nv_bfloat16*>(p.hidden) + slot * 2 * p.hidden_ld + f0 + j;
        const __nv_bfloat16 hi = from_float<__nv_bfloat16>(h);
        const float rounded = to_float(hi);
        to[0] = hi;
        to[p.hidden_ld] = from_float<__nv_bfloat16>(rounded - rounded == 0.0f ? h - rounded : 0.0f);
      } else {
        static_cast<float*>(p.hidden)[slot * p.hidden_ld + f0 + j] = h;
      }
    });
  }
}

// D_e h of an expert's slots, and, in the block that comes last to its rows of y,
// their sums over each token's slots, in the slots' order.
template <typename T, bool VEC>
__global__ void __launch_bounds__(MF_THREADS, MF_BLOCKS) ns_moe_few_sum_kernel(const __grid_constant__ MoeFewParams p) {
  __shared__ float sums[MF_WARPS * MF_NT * 4][32];
  __shared__ bool last;
  extern __shared__ short few_smem[];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const Slots s = slots_of(p, few_smem);
  int named, count;
  const int e = find_expert(p, s, blockIdx.y, &named, &count);
  if (e < 0 && (named > 0 || blockIdx.y > 0)) return;
  const long long first_row = static_cast<long long>(blockIdx.x) * MF_SUM_ROWS;
  if (e >= 0) {
    const T* const down = static_cast<const T*>(p.down) + e * p.dim * p.ffn;
    for (int g = 0; g < MF_SUM_ROWS / 16; ++g) {
      const long long d0 = first_row + 16 * g, d = d0 + lane / 4;
      if (d0 >= p.dim) break;
      const T* const top = d < p.dim ? down + d * p.ffn : nullptr;
      const T* const low = d + 8 < p.dim ? down + (d + 8) * p.ffn : nullptr;
      tile_of_list<T, true, VEC>(p, top, low, static_cast<int>(p.ffn), s, count, sums, [&](int j, int slot, const float (&v)[2]) {
        float* const to = p.part + slot * p.part_ld + d0 + j;  // part_ld is a multiple of MF_SUM_ROWS
        to[0] = v[0];
        to[8] = v[1];
      });
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&p.arrived[blockIdx.x], 1u) == static_cast<unsigned int>(named - 1);
    __syncthreads();
    if (!last) return;
    __threadfence();
  }
  for (int i = threadIdx.x; i < p.tokens * (MF_SUM_ROWS / 4); i += MF_THREADS) {
    const int t = i / (MF_SUM_ROWS / 4);
    const long long d = first_row + i % (MF_SUM_ROWS / 4) * 4;
    float y[4] = {};
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
      const int slot = t * p.k + j;
      if (s.expert[slot] < 0) continue;
      const float w = p.weights ? p.weights[slot] : 1.0f;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part + slot * p.part_ld + d));
      y[0] = fmaf(w, v.x, y[0]);
      y[1] = fmaf(w, v.y, y[1]);
      y[2] = fmaf(w, v.z, y[2]);
      y[3] = fmaf(w, v.w, y[3]);
    }
    T* const to = static_cast<T*>(p.y) + t * p.y_ld + d;
    for (int j = 0; j < 4; ++j)
      if (d + j < p.dim) to[j] = from_float<T>(y[j]);
  }
}

template <typename T, bool VEC>
int launch_few(MoeFewParams p, int nsm, cudaStream_t st) {
  const int experts = std::min(p.experts, p.tokens * p.k);
  const size_t smem = 2 * sizeof(short) * static_cast<size_t>(p.tokens) * p.k;
  const long long tiles = (p.ffn + 7) / 8;
  p.groups = 1;
  cudaError_t e = nsorch::counted(nsorch::K_MOE, st, [&] {
    return launch_pdl(ns_moe_few_hidden_kernel<T, VEC>, dim3(static_cast<unsigned>((tiles + p.groups - 1) / p.groups), experts),
                      dim3(MF_THREADS), smem, st, p);
  });
  if (e != cudaSuccess) return NS_ERR_CUDA;
  e = nsorch::counted(nsorch::K_MOE, st, [&] {
    return launch_pdl(ns_moe_few_sum_kernel<T, VEC>, dim3(static_cast<unsigned>((p.dim + MF_SUM_ROWS - 1) / MF_SUM_ROWS), experts),
                      dim3(MF_THREADS), smem, st, p);
  });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

template <typename T>
int launch_few(const MoeFewParams& p, int nsm, cudaStream_t st) {
  const auto words = [](const void* q, long long ld) {
    return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld * sizeof(T) % 16 == 0;
  };
  const bool vec = words(p.x, p.tokens > 1 ? p.x_ld : 0) && words(p.gate_up, p.dim) && words(p.down, p.ffn);
  return vec ? launch_few<T, true>(p, nsm, st) : launch_few<T, false>(p, nsm, st);
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

// The workspace's parts: hidden values, products, counts.
struct FewParts {
  int64_t hidden_ld, part_ld;
  uint64_t part, arrived, bytes;
  FewParts(int64_t tokens, int k, int64_t dim, int64_t ffn) {
    const uint64_t slots = static_cast<uint64_t>(tokens) * k;
    hidden_ld = (ffn + 7) / 8 * 8;
    part_ld = (dim + nsk::MF_SUM_ROWS - 1) / nsk::MF_SUM_ROWS * nsk::MF_SUM_ROWS;
    part = (4 * slots * hidden_ld + 255) / 256 * 256;
    arrived = part + 4 * slots * part_ld;
    bytes = arrived + 4 * (part_ld / nsk::MF_SUM_ROWS);
  }
};

}  // namespace

extern "C" {

int ns_moe_few_tokens_workspace_bytes(int64_t tokens, int k, int64_t dim, int64_t ffn, uint64_t* bytes) {
  if (!bytes) return NS_ERR_ARG;
  const int rc = check_few(tokens, k, dim, ffn);
  if (rc == NS_OK) *bytes = FewParts(tokens, k, dim, ffn).bytes;
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
  const FewParts parts(tokens, k, dim, ffn);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < parts.bytes) return NS_ERR_WORKSPACE;
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
  p.hidden_ld = parts.hidden_ld;
  p.part_ld = parts.part_ld;
  p.weights = weights;
  p.hidden = workspace;
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + parts.part);
  p.arrived = reinterpret_cast<unsigned int*>(static_cast<char*>(workspace) + parts.arrived);
  int dev, nsm;
  if ((rc = device_setup(&dev, &p.status, &nsm)) != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == NS_DT_BF16) return nsk::launch_few<__nv_bfloat16>(p, nsm, st);
  if (dtype == NS_DT_FP16) return nsk::launch_few<__half>(p, nsm, st);
  return nsk::launch_few<float>(p, nsm, st);
}

}  // extern "C"
