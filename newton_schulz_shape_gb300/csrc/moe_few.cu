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
// experts among all slots themselves, which spares a kernel.
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int MF_WARPS = 8;                  // of a block
constexpr int MF_THREADS = 32 * MF_WARPS;
constexpr int MF_BLOCKS = 2;                 // of an SM
constexpr int MF_MAX_TOKENS = 256;
constexpr int MF_ROWS = 32;                  // of a tile: two of the tensor instruction's
constexpr int MF_NT = 4;                     // groups of 8 tokens that a pass over an expert's weights serves at most

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
  unsigned int* arrived;  // [dim / MF_ROWS]: passes whose part of these rows of y is there
  int team;            // warps that split k of a tile
  int entries;         // at most: passes over an expert
  unsigned int* status;
};

// ------------------------------------------------------- tokens of an expert
// A pass over an expert's weights: those of its slots that it serves.
struct Pass {
  int expert, first, count;  // slots sorted[first .. first + count)
};

// What a block knows of the routing, in shared memory.
struct Routing {
  Pass* passes;
  int* counts;    // [experts] slots, then where the next one goes
  short* expert;  // [slots], -1: goes nowhere
  short* sorted;  // the slots by expert
  __device__ __forceinline__ Routing(const MoeFewParams& p, void* smem)
      : passes(static_cast<Pass*>(smem)), counts(reinterpret_cast<int*>(passes + p.entries)),
        expert(reinterpret_cast<short*>(counts + p.experts)), sorted(expert + p.tokens * p.k) {}
};
constexpr size_t routing_bytes(int entries, int experts, int slots) {
  return sizeof(Pass) * entries + sizeof(int) * experts + 2 * sizeof(short) * static_cast<size_t>(slots);
}

// Reads the ids, sorts the slots by expert and lists the passes; their number, and
// the largest pass's slots. The order of the slots of a pass reaches no result:
// every column of a product is its own. So atomics may decide it, unless an
// expert takes several passes, which have to be the same ones in every block.
__device__ __forceinline__ int2 find_passes(const MoeFewParams& p, const Routing& r) {
  __shared__ int2 found;
  const int lane = threadIdx.x & 31, slots = p.tokens * p.k;
  for (int i = threadIdx.x; i < p.experts; i += MF_THREADS) r.counts[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += MF_THREADS) {
    long long e = load_index(p.ids, p.id_bytes, i);
    if (e >= p.experts) {
      atomicOr(p.status, NS_DEV_BAD_INDEX);
      e = -1;
    }
    if (e >= 0) atomicAdd(&r.counts[e], 1);
    r.expert[i] = static_cast<short>(e < 0 ? -1 : e);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int passes = 0, sum = 0, most = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane, n = e < p.experts ? r.counts[e] : 0, mine = (n + 8 * MF_NT - 1) / (8 * MF_NT);
      int upto = n + (mine << 16);  // slots (at most 8192) and passes up to this lane
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const int first = sum + (upto & 0xffff) - n, at = passes + (upto >> 16) - mine;
      if (e < p.experts) r.counts[e] = first;
      for (int i = 0; i < mine; ++i) r.passes[at + i] = {e, first + i * 8 * MF_NT, min(n - i * 8 * MF_NT, 8 * MF_NT)};
      most = max(most, n);
      upto = __shfl_sync(0xffffffffu, upto, 31);
      sum += upto & 0xffff;
      passes += upto >> 16;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) found = make_int2(passes, most);
  }
  __syncthreads();
  if (found.y <= 8 * MF_NT) {
    for (int i = threadIdx.x; i < slots; i += MF_THREADS)
      if (r.expert[i] >= 0) r.sorted[atomicAdd(&r.counts[r.expert[i]], 1)] = static_cast<short>(i);
  } else if (threadIdx.x < 32) {
    for (int i0 = 0; i0 < slots; i0 += 32) {
      const int e = i0 + lane < slots ? r.expert[i0 + lane] : -1;
      const unsigned int same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1)), first = e >= 0 ? r.counts[e] : 0;
      __syncwarp();
      if (e >= 0) r.sorted[first + before] = static_cast<short>(i0 + lane);
      if (e >= 0 && before == 0) r.counts[e] = first + __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  return found;
}

// ------------------------------------------------------------------ products
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

// 16 bytes of consecutive values of a row from k on, value by value, zero from n on.
template <typename T>
__device__ __forceinline__ uint4 load_values(const T* row, int k, int n) {
  constexpr int V = 16 / sizeof(T);
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = k + i < n ? to_float(row[k + i]) : 0.0f;
  const Vec<T, V> v = pack<T, V>(f);
  return *reinterpret_cast<const uint4*>(&v);
}

__device__ __forceinline__ uint4 load_words(const void* p) {
  uint4 v;  // volatile: stays in order with the products, so that it holds no registers for long
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The tokens' side of a product, 16 bytes' worth of k: of x, or (HIDDEN) of h.
// bf16 and fp16 products of x are exact; an fp32 factor is split in two. h has
// more bits and a larger range than 16-bit types: it meets bf16 weights as two
// bf16 values (2^-18 off), and fp16 weights, which tf32 holds, as two tf32 values.
template <typename T, bool HIDDEN>
struct Side {
  static constexpr bool PAIR = HIDDEN && std::is_same<T, __nv_bfloat16>::value;
  static constexpr bool WIDE = sizeof(T) == 4 || (HIDDEN && !PAIR);
  static constexpr int Q = HIDDEN && sizeof(T) == 2 ? 2 : 1;  // 16-byte words
  uint4 q[Q];  // PAIR: the upper parts, then the lower
  __device__ __forceinline__ uint32_t w(int i) const { return reinterpret_cast<const uint32_t*>(q)[i]; }

  // A slot's row, null for none.
  static __device__ __forceinline__ const char* row(const MoeFewParams& p, int slot) {
    if (slot < 0) return nullptr;
    if constexpr (HIDDEN)
      return static_cast<const char*>(p.hidden) + 4 * slot * p.hidden_ld;
    else
      return static_cast<const char*>(p.x) + sizeof(T) * (slot / p.k) * p.x_ld;
  }
  // Word i of the values from k on.
  static __device__ __forceinline__ const char* word(const MoeFewParams& p, const char* row, int i, int k) {
    if constexpr (PAIR) return row + 2 * (k + i * p.hidden_ld);
    if constexpr (HIDDEN) return row + 4 * (k + 4 * i);
    return row + sizeof(T) * k;
  }
  template <bool VEC>
  __device__ __forceinline__ void load(const MoeFewParams& p, const char* row, int k, int n) {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      q[i] = make_uint4(0, 0, 0, 0);
      if constexpr (HIDDEN || VEC) {
        if (row && k < n) q[i] = load_words(word(p, row, i, k));
      } else {
        if (row) q[i] = load_values(reinterpret_cast<const T*>(row), k, n);
      }
    }
  }
  // The same on its way to shared memory, words 32 apart.
  template <bool VEC>
  static __device__ __forceinline__ void fetch(const MoeFewParams& p, const char* row, int k, int n, uint4* to) {
    const bool there = row && k < n;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if constexpr (HIDDEN || VEC)
        nsptx::cp_async16_shared(to + 32 * i, there ? word(p, row, i, k) : static_cast<const char*>(p.hidden), there ? 16 : 0);
      else
        to[32 * i] = there ? load_values(reinterpret_cast<const T*>(row), k, n) : make_uint4(0, 0, 0, 0);
    }
  }
};

// The weights' side, rows r and r + 8 of a tile, times that.
template <typename T, bool HIDDEN>
__device__ __forceinline__ void times(float (&c)[4], const uint4& r, const uint4& r8, const Side<T, HIDDEN>& side) {
  using S = Side<T, HIDDEN>;
  const uint32_t a[2][4] = {{r.x, r.y, r.z, r.w}, {r8.x, r8.y, r8.z, r8.w}};
  if constexpr (!S::WIDE) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      mma_16<T>(c, a[0][i], a[1][i], a[0][i + 1], a[1][i + 1], side.w(i), side.w(i + 1));
      if constexpr (S::PAIR) mma_16<T>(c, a[0][i], a[1][i], a[0][i + 1], a[1][i + 1], side.w(4 + i), side.w(5 + i));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); i += 2) {
      uint32_t hi[2], lo[2], w[2][2], rest[2][2];  // [k][row]
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        split(__uint_as_float(side.w(i + j)), &hi[j], &lo[j]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if constexpr (sizeof(T) == 4) {
            split(__uint_as_float(a[q][i + j]), &w[j][q], &rest[j][q]);
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[q][i / 2]));
            w[j][q] = __float_as_uint(j ? f.y : f.x);
          }
        }
      }
      mma_tf32_8(c, w[0][0], w[0][1], w[1][0], w[1][1], hi[0], hi[1]);
      mma_tf32_8(c, w[0][0], w[0][1], w[1][0], w[1][1], lo[0], lo[1]);
      if constexpr (sizeof(T) == 4) mma_tf32_8(c, rest[0][0], rest[0][1], rest[1][0], rest[1][1], hi[0], hi[1]);
    }
  }
}

// A warp's ring of shared memory holds the words of its next steps. Up to 16
// slots bring their side of the products along; more are read when they are
// used, from L1 as a rule.
constexpr int MF_RING = 768;  // 16-byte words of a warp
template <typename T, bool HIDDEN, int NT>
struct Ring {
  static constexpr bool SIDE = NT <= 2;
  static constexpr int STAGE = 32 * (4 + (SIDE ? NT * Side<T, HIDDEN>::Q : 0));  // words of a step
  static constexpr int AHEAD = MF_RING / STAGE - 1;                              // steps on their way, beside the one in use
};

// A team of warps goes through the tiles of a block that fall to it, all passes in
// a row: `Stream` copies the weights of a warp's next steps to its ring, into the
// next tile and the next pass. (Held in registers they were waited for in the
// wrong order: a warp has six counters for the loads that it waits for.)
template <typename T, bool HIDDEN, bool VEC, int NT>
struct Stream {
  using S = Side<T, HIDDEN>;
  using R = Ring<T, HIDDEN, NT>;
  static constexpr int V = 16 / sizeof(T);
  const MoeFewParams& p;
  const Routing& r;
  int tiles, end, stride;  // tiles of a pass; items (tiles of all passes) of the block; of a team
  int n, step, steps;      // values of a row, from a warp's step to its next, steps of a tile
  int k0;                  // the lane's first value
  uint4* ring;
  int fill, take;
  int item, pass, s;       // of the next copy
  const T* at[4];          // the lane's rows there: r and r + 8 of each half of the tile
  int values[4];           // of the rows that are there
  const char* token[NT];   // the rows of the lane's columns there

  __device__ __forceinline__ Stream(const MoeFewParams& params, const Routing& routing, uint4* warp_ring, int first, int last,
                                    int team, int teams, int warp, int tiles_of_pass)
      : p(params), r(routing), tiles(tiles_of_pass), end(last), stride(teams), ring(warp_ring + (threadIdx.x & 31)), fill(0),
        take(0), item(first + team), pass(-1), s(0) {
    n = static_cast<int>(HIDDEN ? p.ffn : p.dim);
    step = 4 * V * p.team;
    steps = max(0, (n - warp * 4 * V + step - 1) / step);
    k0 = (warp * 4 + (threadIdx.x & 3)) * V;
    rows();
#pragma unroll
    for (int i = 0; i < R::AHEAD; ++i) fetch();
  }
  // The rows of the lane's columns in a pass.
  __device__ __forceinline__ void tokens_of(const Pass& of, const char* (&row)[NT]) const {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = 8 * t + (threadIdx.x & 31) / 4;
      row[t] = S::row(p, i < of.count ? r.sorted[of.first + i] : -1);
    }
  }
  __device__ __forceinline__ void rows() {
    if (item >= end) return;
    const int in = item / tiles, lane = (threadIdx.x & 31) / 4;
    if (R::SIDE && in != pass) tokens_of(r.passes[in], token);
    pass = in;
    const long long e = r.passes[in].expert, j = item - in * tiles;
    if (HIDDEN) {  // 32 rows of D
      const T* base = static_cast<const T*>(p.down) + e * p.dim * p.ffn;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long d = j * MF_ROWS + 8 * i + lane;
        values[i] = d < p.dim ? n : 0;
        at[i] = d < p.dim ? base + d * p.ffn : base;
      }
    } else {       // 16 rows of G and the rows of U that go with them
      const T* base = static_cast<const T*>(p.gate_up) + 2 * e * p.ffn * p.dim;
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const long long f = j * (MF_ROWS / 2) + 4 * i + lane;
        values[i] = values[i + 1] = f < p.ffn ? n : 0;
        at[i] = f < p.ffn ? base + f * p.dim : base;
        at[i + 1] = at[i] + p.ffn * p.dim;
      }
    }
  }
  __device__ __forceinline__ void fetch() {
    if (item < end && steps > 0) {
      const int k = k0 + s * step;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (VEC) {
          const bool there = k < values[i];
          nsptx::cp_async16_upto(ring + fill + 32 * i, at[i] + (there ? k : 0), there ? 16 : 0);
        } else {
          ring[fill + 32 * i] = load_values(at[i], k, values[i]);
        }
      }
      if constexpr (R::SIDE) {
#pragma unroll
        for (int t = 0; t < NT; ++t) S::template fetch<VEC>(p, token[t], k, n, ring + fill + 32 * (4 + t * S::Q));
      }
      if (++s == steps) {
        s = 0;
        item += stride;
        rows();
      }
    }
    nsptx::cp_async_commit();
    fill = fill == R::AHEAD * R::STAGE ? 0 : fill + R::STAGE;
  }

  // The products of the next tile with 8 * NT slots, whose rows are `row` (where the ring does not hold them).
  __device__ __forceinline__ void tile(const char* const (&row)[NT], float (&acc)[2][NT][4]) {
    for (int i = 0; i < steps; ++i) {
      nsptx::cp_async_wait<R::AHEAD - 1>();
      uint4 a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = ring[take + 32 * j];
      S side[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (R::SIDE) {
#pragma unroll
          for (int j = 0; j < S::Q; ++j) side[t].q[j] = ring[take + 32 * (4 + t * S::Q + j)];
        } else {
          side[t].template load<VEC>(p, row[t], k0 + i * step, n);
        }
      }
      take = take == R::AHEAD * R::STAGE ? 0 : take + R::STAGE;
      fetch();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        times(acc[0][t], a[0], a[1], side[t]);
        times(acc[1][t], a[2], a[3], side[t]);
      }
    }
  }
};

// A barrier of the team's warps, each of them together.
__device__ __forceinline__ void team_sync(int team, int warps) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * warps) : "memory");
}

// A block's share of all passes' tiles, each by a team of warps that split k:
// use(tile, half, slot, a, b) gets the sums, a of row lane / 4 of a half of the
// tile and b of the row 8 further, for a slot; done(tile) follows a tile's last.
// Both in one warp of the team.
template <typename T, bool HIDDEN, bool VEC, int NT, typename F, typename G>
__device__ __forceinline__ void all_tiles(const MoeFewParams& p, const Routing& r, uint4* smem, int passes, int tiles, F&& use, G&& done) {
  const long long items = static_cast<long long>(passes) * tiles;
  const int first = static_cast<int>(items * blockIdx.x / gridDim.x), last = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);
  const int lane = threadIdx.x & 31, warps = p.team, team = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) & (warps - 1);
  const int teams = MF_WARPS / warps;
  Stream<T, HIDDEN, VEC, NT> stream(p, r, smem + (threadIdx.x >> 5) * MF_RING, first, last, team, teams, warp, tiles);
  float* const sums = reinterpret_cast<float*>(smem + MF_WARPS * MF_RING) + team * warps * 8 * 32 + lane;
  const char* row[NT] = {};
  int held = -1;
  for (int item = first + team; item < last; item += teams) {
    const int pass = item / tiles, tile = item - pass * tiles;
    const Pass& of = r.passes[pass];
    if (!Ring<T, HIDDEN, NT>::SIDE && pass != held) stream.tokens_of(of, row);
    held = pass;
    float acc[2][NT][4] = {};
    stream.tile(row, acc);
    if (warps > 1) {  // summed by the team's first warp, in a fixed order, 8 slots at a time
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        team_sync(team, warps);  // the last ones are read
        if (warp > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sums[(warp * 8 + i) * 32] = acc[i / 4][t][i % 4];
        }
        team_sync(team, warps);
        if (warp > 0) continue;
        for (int w = 1; w < warps; ++w)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i / 4][t][i % 4] += sums[(w * 8 + i) * 32];
      }
      if (warp > 0) continue;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = 8 * t + 2 * (lane & 3) + c;
        if (j >= of.count) continue;
        const int slot = r.sorted[of.first + j];
        use(tile, 0, slot, acc[0][t][c], acc[0][t][c + 2]);
        use(tile, 1, slot, acc[1][t][c], acc[1][t][c + 2]);
      }
    }
    done(tile);
  }
}

// The same for passes of up to `most` slots.
template <typename T, bool HIDDEN, bool VEC, typename F, typename G>
__device__ __forceinline__ void all_tiles(const MoeFewParams& p, const Routing& r, uint4* smem, int2 found, int tiles, F&& use, G&& done) {
  if (found.y <= 8)
    all_tiles<T, HIDDEN, VEC, 1>(p, r, smem, found.x, tiles, use, done);
  else if (found.y <= 16)
    all_tiles<T, HIDDEN, VEC, 2>(p, r, smem, found.x, tiles, use, done);
  else
    all_tiles<T, HIDDEN, VEC, MF_NT>(p, r, smem, found.x, tiles, use, done);
}

// Shared memory: the rings, the parts of split sums, the routing.
constexpr int MF_SMEM_WORDS = MF_WARPS * MF_RING;
__host__ __device__ constexpr int sums_words(int team) { return team > 1 ? MF_WARPS * 8 * 8 : 0; }
__device__ __forceinline__ Routing routing_of(const MoeFewParams& p, uint4* smem) {
  return Routing(p, smem + MF_SMEM_WORDS + sums_words(p.team));
}

// h of all slots.
template <typename T, bool VEC>
__global__ void __launch_bounds__(MF_THREADS, MF_BLOCKS) ns_moe_few_hidden_kernel(const __grid_constant__ MoeFewParams p) {
  extern __shared__ uint4 few_smem[];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  // the other kernel's counts, which no earlier kernel still uses
  for (int i = blockIdx.x * MF_THREADS + threadIdx.x; i * MF_ROWS < p.dim; i += gridDim.x * MF_THREADS) p.arrived[i] = 0;
  const Routing r = routing_of(p, few_smem);
  const int2 found = find_passes(p, r);
  const int row = (threadIdx.x & 31) / 4;
  all_tiles<T, false, VEC>(
      p, r, few_smem, found, static_cast<int>((p.ffn + MF_ROWS / 2 - 1) / (MF_ROWS / 2)),
      [&](int tile, int half, int slot, float a, float b) {
        const long long f = tile * (MF_ROWS / 2) + 8 * half + row;
        if (f >= p.hidden_ld) return;
        // zero up to the row's end: its last words are read whole
        const float h = f < p.ffn ? a / (1.0f + expf(-a)) * b : 0.0f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          __nv_bfloat16* const to = static_cast<__nv_bfloat16*>(p.hidden) + slot * 2 * p.hidden_ld + f;
          const __nv_bfloat16 hi = from_float<__nv_bfloat16>(h);
          const float rounded = to_float(hi);
          to[0] = hi;
          to[p.hidden_ld] = from_float<__nv_bfloat16>(rounded - rounded == 0.0f ? h - rounded : 0.0f);
        } else {
          static_cast<float*>(p.hidden)[slot * p.hidden_ld + f] = h;
        }
      },
      [](int) {});
}

// The rows of y of a tile: the sums over each token's slots, in the slots' order. A lane takes 4 rows of every
// fourth token.
template <typename T>
__device__ __forceinline__ void sum_tile(const MoeFewParams& p, const Routing& r, int tile) {
  const int lane = threadIdx.x & 31;
  const long long d = tile * MF_ROWS + (lane & 7) * 4;
  for (int t = lane / 8; t < p.tokens; t += 4) {
    float y[4] = {};
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      float4 v[8];
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int slot = t * p.k + j0 + i;
        const bool there = j0 + i < p.k && r.expert[slot] >= 0;
        v[i] = there ? __ldcg(reinterpret_cast<const float4*>(p.part + slot * p.part_ld + d)) : make_float4(0, 0, 0, 0);
        w[i] = there ? (p.weights ? p.weights[slot] : 1.0f) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[0] = fmaf(w[i], v[i].x, y[0]);
        y[1] = fmaf(w[i], v[i].y, y[1]);
        y[2] = fmaf(w[i], v[i].z, y[2]);
        y[3] = fmaf(w[i], v[i].w, y[3]);
      }
    }
    T* const to = static_cast<T*>(p.y) + t * p.y_ld + d;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < p.dim) to[i] = from_float<T>(y[i]);
  }
}

// D_e h of all slots, and, by the warp that comes last to a tile of y, its sums.
template <typename T, bool VEC>
__global__ void __launch_bounds__(MF_THREADS, MF_BLOCKS) ns_moe_few_sum_kernel(const __grid_constant__ MoeFewParams p) {
  extern __shared__ uint4 few_smem[];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const Routing r = routing_of(p, few_smem);
  const int2 found = find_passes(p, r);
  const int passes = found.x, lane = threadIdx.x & 31, tiles = static_cast<int>((p.dim + MF_ROWS - 1) / MF_ROWS);
  if (passes == 0) {  // no slot goes anywhere
    for (int i = blockIdx.x * MF_WARPS + threadIdx.x / 32; i < tiles; i += gridDim.x * MF_WARPS) sum_tile<T>(p, r, i);
    return;
  }
  all_tiles<T, true, VEC>(
      p, r, few_smem, found, tiles,
      [&](int tile, int half, int slot, float a, float b) {
        // part_ld is a multiple of MF_ROWS
        float* const to = p.part + slot * p.part_ld + tile * MF_ROWS + 16 * half + lane / 4;
        to[0] = a;
        to[8] = b;
      },
      [&](int tile) {
        __threadfence();
        __syncwarp();
        unsigned int before = 0;
        if (lane == 0) before = atomicAdd(&p.arrived[tile], 1u);
        if (__shfl_sync(0xffffffffu, before, 0) != static_cast<unsigned int>(passes - 1)) return;
        __threadfence();
        sum_tile<T>(p, r, tile);
      });
}

// Warps that split a tile's k: as many as keep all of the card's warps busy, with 4 steps for each at least.
int team_of(long long tiles, long long steps, int nsm) {
  int team = 1;
  while (team < MF_WARPS && tiles * 2 * team <= static_cast<long long>(nsm) * MF_BLOCKS * MF_WARPS && steps >= 8 * team) team *= 2;
  return team;
}

template <typename T, bool VEC>
int launch_few(MoeFewParams p, int nsm, cudaStream_t st) {
  constexpr int VALUES = 64 / sizeof(T);  // of a step
  const int slots = p.tokens * p.k, named = std::min(p.experts, slots);
  p.entries = named + slots / (8 * MF_NT);
  // every call sets the same limit
  constexpr size_t MOST = sizeof(uint4) * (MF_SMEM_WORDS + sums_words(2)) + routing_bytes(1024 + MF_MAX_TOKENS * 32 / (8 * MF_NT), 1024, MF_MAX_TOKENS * 32);
  auto launch = [&](void (*kernel)(MoeFewParams), long long tiles, long long n) {
    p.team = team_of(tiles * named, (n + VALUES - 1) / VALUES, nsm);
    const long long teams = (tiles * p.entries * p.team + MF_WARPS - 1) / MF_WARPS;
    const int blocks = static_cast<int>(std::min<long long>(nsm * MF_BLOCKS, teams));
    const size_t smem = sizeof(uint4) * (MF_SMEM_WORDS + sums_words(p.team)) + routing_bytes(p.entries, p.experts, slots);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(MOST));
    if (e != cudaSuccess) return e;
    return nsorch::counted(nsorch::K_MOE, st, [&] { return launch_pdl(kernel, dim3(blocks), dim3(MF_THREADS), smem, st, p); });
  };
  if (launch(ns_moe_few_hidden_kernel<T, VEC>, (p.ffn + MF_ROWS / 2 - 1) / (MF_ROWS / 2), p.dim) != cudaSuccess) return NS_ERR_CUDA;
  return launch(ns_moe_few_sum_kernel<T, VEC>, (p.dim + MF_ROWS - 1) / MF_ROWS, p.ffn) == cudaSuccess ? NS_OK : NS_ERR_CUDA;
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
    part_ld = (dim + nsk::MF_ROWS - 1) / nsk::MF_ROWS * nsk::MF_ROWS;
    part = (4 * slots * hidden_ld + 255) / 256 * 256;
    arrived = part + 4 * slots * part_ld;
    bytes = arrived + 4 * (part_ld / nsk::MF_ROWS);
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
