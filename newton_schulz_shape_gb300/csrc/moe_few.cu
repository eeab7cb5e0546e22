// A whole mixture-of-experts layer for a few tokens: each token's experts, their
// gated products and the weighted sum, in two kernels and a short third.
//
//   h_s = silu(G_e x_t) * (U_e x_t)     for slot s = (t, j) with expert e
//   y_t = sum over j of w_tj D_e h_s
// with silu(a) = a / (1 + exp(-a)).
//
// The matrices of the experts that are named, 3 dim ffn values each, are nearly
// all of the bytes, so the layer is bound by memory: n tokens of an expert make
// 2 n operations of each value. Up to 16 of an expert's slots share a pass over its
// matrices, which are read once for each pass (128 tokens by 8 of 64 experts make
// 1.5 readings and 352 us, 64 by 2 of 8 as many and 58 us); a pass's tiles (32 rows)
// all blocks deal among them, and the 16 warps of a block split k of a tile. Each
// lane copies the 16-byte words of its rows ahead to its own places of shared
// memory and hands them to tensor instructions as they are (x by G and U, 16-bit
// types) or widened to tf32: the order of k within a product is free, so its words
// and the tokens' are taken in the same order, and nothing is exchanged between
// lanes. (The 5th-generation instruction takes 128 rows, whose tiles are too few
// for the card where few experts are named: 8 of 1408 rows make 176. It was not
// tried for many.)
// Blocks find the tokens of their experts among all slots themselves, which
// spares a kernel.
//
// 64 experts of 1408 x 2048 bf16 by one slot each take 194-201 us (5.6 TB/s with
// the three launches; 0.83 of the measured copy), by 8 each 208-212 and by 16 each
// 237; one token of 8 experts 36-37 us (3.7 TB/s: three kernels of 3 us each with
// nothing to do, and 4.6 tiles a block).
#include <algorithm>
#include <climits>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int MF_WARPS = 16;                 // of a block, which has an SM to itself
constexpr int MF_THREADS = 32 * MF_WARPS;
constexpr int MF_SUM_THREADS = 128;
constexpr int MF_MAX_TOKENS = 256;
constexpr int MF_ROWS = 32;                  // of a tile: two of the tensor instruction's
constexpr int MF_NT = 2;                     // groups of 8 slots that a pass over an expert's weights serves at most

struct MoeFewParams {
  const void *x, *gate_up, *down;
  void* y;
  const void* ids;
  int id_bytes, tokens, k, experts;
  long long x_ld, y_ld, dim, ffn;
  long long hidden_ld, part_ld;  // values of a slot's rows below
  const float* weights;
  float* hidden;       // [tokens * k][hidden_ld]: h
  float* part;         // [tokens * k][part_ld]: D_e h
  int team;            // warps that split k of a tile
  int entries;         // at most: passes over an expert
  int held;            // words of the tokens' side that a lane holds in shared memory
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

// Reads the ids, sorts the slots by expert and lists the passes; their number.
// The order of the slots of a pass reaches no result: every column of a product
// is its own. So atomics may decide it, unless an expert takes several passes,
// which have to be the same ones in every block.
__device__ __forceinline__ int find_passes(const MoeFewParams& p, const Routing& r) {
  __shared__ int2 found;
  const int lane = threadIdx.x & 31, slots = p.tokens * p.k;
  if (slots <= 32) {  // by one warp, without counts
    if (threadIdx.x < 32) {
      long long id = lane < slots ? load_index(p.ids, p.id_bytes, lane) : -1;
      if (id >= p.experts) {
        atomicOr(p.status, NS_DEV_BAD_INDEX);
        id = -1;
      }
      const int e = id < 0 ? -1 : static_cast<int>(id);
      const unsigned int same = __match_any_sync(0xffffffffu, e), before = (1u << lane) - 1;
      const bool first = e >= 0 && !(same & before);
      const unsigned int firsts = __ballot_sync(0xffffffffu, first);
      int upto = first ? __popc(same) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const int start = __shfl_sync(0xffffffffu, upto - __popc(same), __ffs(same) - 1);  // of the expert's slots
      const int rank = __popc(same & before);
      if (e >= 0) r.sorted[start + rank] = static_cast<short>(lane);
      // 32 slots make two passes of an expert at most, the second of which follows those before it
      const unsigned int doubles = __ballot_sync(0xffffffffu, first && __popc(same) > 8 * MF_NT);
      if (first) {
        const int at = __popc(firsts & before) + __popc(doubles & before), n = __popc(same);
        r.passes[at] = {e, start, min(n, 8 * MF_NT)};
        if (n > 8 * MF_NT) r.passes[at + 1] = {e, start + 8 * MF_NT, n - 8 * MF_NT};
      }
      if (lane == 0) found.x = __popc(firsts) + __popc(doubles);
    }
    __syncthreads();
    return found.x;
  }
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
  return found.x;
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
// Two values of a 16-bit type, which tf32 holds.
__device__ __forceinline__ float2 wide2(__nv_bfloat16, uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 wide2(__half, uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

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

// The tokens' side of a product, 16 bytes' worth of the weights' k: of x, or
// (HIDDEN) of h. bf16 and fp16 products of x are exact. h, in fp32, has more bits
// and a larger range than 16-bit types: it is split in two tf32 values, which
// meet the weights as tf32, and so are both factors of fp32 layers (without the
// product of their lower parts, 2^-24). D_e h is then 1.9e-7 of its size off, as
// with products in fp32 (1.5e-7). With bf16 weights and h as two bf16 values it was
// 2.5e-6 and 64 tokens through 64 experts took 220 us, now 232; with three bf16
// values 1e-7 and 249.
template <typename T, bool HIDDEN>
struct Side {
  static constexpr bool WIDE = sizeof(T) == 4 || HIDDEN;      // products of tf32
  // the weights have to be converted, or split as well
  static constexpr bool LONG = sizeof(T) == 4 || (HIDDEN && std::is_same<T, __half>::value);
  static constexpr int Q = HIDDEN && sizeof(T) == 2 ? 2 : 1;  // 16-byte words
  uint4 q[Q];
  __device__ __forceinline__ uint32_t w(int i) const { return reinterpret_cast<const uint32_t*>(q)[i]; }

  // A slot's row.
  static __device__ __forceinline__ const char* row(const MoeFewParams& p, int slot) {
    if constexpr (HIDDEN)
      return reinterpret_cast<const char*>(p.hidden + slot * p.hidden_ld);
    else
      return static_cast<const char*>(p.x) + sizeof(T) * (slot / p.k) * p.x_ld;
  }
  // Its values from k on, zero from n on.
  template <bool VEC>
  __device__ __forceinline__ void load(const char* row, int k, int n) {
#pragma unroll
    for (int i = 0; i < Q; ++i) q[i] = make_uint4(0, 0, 0, 0);
    if constexpr (HIDDEN || VEC) {
      if (k < n) {
        constexpr int BYTES = HIDDEN ? 4 : sizeof(T);
#pragma unroll
        for (int i = 0; i < Q; ++i) q[i] = load_words(row + BYTES * k + 16 * i);
      }
    } else {
      q[0] = load_values(reinterpret_cast<const T*>(row), k, n);
    }
  }
};

// The weights' side, rows r and r + 8 of a tile, times that. The instruction cuts
// what it adds at the sum's last place, always towards zero, which shows over long
// rows (1e-6 of the result): a step's products make a sum of their own, the small
// ones first, and that is added to the rest as usual.
template <typename T, bool HIDDEN>
__device__ __forceinline__ void times(float (&c)[4], const uint4& r, const uint4& r8, const Side<T, HIDDEN>& side) {
  using S = Side<T, HIDDEN>;
  const uint32_t a[2][4] = {{r.x, r.y, r.z, r.w}, {r8.x, r8.y, r8.z, r8.w}};
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (!S::WIDE) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) mma_16<T>(sum, a[0][i], a[1][i], a[0][i + 1], a[1][i + 1], side.w(i), side.w(i + 1));
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
            const float2 f = wide2(T(), a[q][i / 2]);
            w[j][q] = __float_as_uint(j ? f.y : f.x);
          }
        }
      }
      mma_tf32_8(sum, w[0][0], w[0][1], w[1][0], w[1][1], lo[0], lo[1]);
      if constexpr (sizeof(T) == 4) mma_tf32_8(sum, rest[0][0], rest[0][1], rest[1][0], rest[1][1], hi[0], hi[1]);
      mma_tf32_8(sum, w[0][0], w[0][1], w[1][0], w[1][1], hi[0], hi[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += sum[i];
}

// Steps of a warp whose words are on their way, and places for them in the warp's
// ring of shared memory. A lane copies into its own words there, once the products
// that took the step before from them are issued. Where those take long, one step
// more has its place and is copied before them (17 tokens by 4 of 60 experts of
// 2112 x 960 fp32 168 us, without 186; 64 tokens by 6 of 64 experts of 1408 x 2048
// fp16 233 us, without 239, and bf16 236, without 232). h is then twice its size or
// the ring wider, and takes the memory of one.
__host__ __device__ constexpr int ahead(bool hidden, bool vec, bool slow) { return slow && (hidden || !vec) ? 2 : 3; }
// 16-byte words of a step: four rows of 16 bytes a lane. Rows that are not made of aligned 16-byte words are copied in
// aligned 4-byte words, five of which cover the values of a 16-bit type.
__host__ __device__ constexpr int stage_words(bool vec) { return vec ? 4 * 32 : 5 * 32; }
template <typename S, bool HIDDEN, bool VEC>
constexpr int RING_WORDS = (ahead(HIDDEN, VEC, S::LONG) + S::LONG) * stage_words(VEC);

// A team of warps goes through the tiles of a block that fall to it, all passes in
// a row: `Stream` copies the weights of a warp's next steps to its ring, into the
// next tile and the next pass. (Held in registers they were waited for in the
// wrong order: a warp has six counters for the loads that it waits for.) L2 gives
// the weights up first, so that what the kernels leave for one another stays
// there (64 experts by 8 slots each 220 -> 208 us). Rows past the last, and
// columns of a pass without a slot, are computed from others and go nowhere.
template <typename T, bool HIDDEN, bool VEC>
struct Stream {
  using S = Side<T, HIDDEN>;
  static constexpr int V = 16 / sizeof(T), AHEAD = ahead(HIDDEN, VEC, S::LONG), STAGE = stage_words(VEC), RING = RING_WORDS<S, HIDDEN, VEC>;
  // 4-byte words of a row, where there are no 16-byte ones
  static constexpr int PLANES = sizeof(T) == 4 ? 4 : 5;
  static_assert(32 * 4 * PLANES <= 4 * stage_words(false), "a stage");
  const MoeFewParams& p;
  const Routing& r;
  int tiles, rows;             // tiles of a pass, rows of a matrix
  int end, stride;             // items (tiles of all passes): the block's last, from a team's to its next
  int n, step, steps;          // values of a row, from a warp's step to its next, steps of a tile
  int most_steps;              // of any of the team's warps
  int k0;                      // the lane's first value
  uint4* ring;
  int fill, take;
  int item, pass, tile, k, s;  // of the next copy
  const T* at[4];              // the lane's rows there: r and r + 8 of each half of the tile
  uint64_t policy;

  __device__ __forceinline__ Stream(const MoeFewParams& params, const Routing& routing, uint4* warp_ring, int first, int last,
                                    int team, int teams, int warp, int tiles_of_pass)
      : p(params), r(routing), tiles(tiles_of_pass), end(last), stride(teams), ring(warp_ring), fill(0),
        take(0), item(first + team), pass(item / tiles), tile(item - pass * tiles), policy(nsptx::evict_first_policy()) {
    n = static_cast<int>(HIDDEN ? p.ffn : p.dim);
    rows = static_cast<int>(HIDDEN ? p.dim : p.ffn);
    step = 4 * V * p.team;
    most_steps = (n + step - 1) / step;
    steps = max(0, (n - warp * 4 * V + step - 1) / step);
    k0 = (warp * 4 + (threadIdx.x & 3)) * V;
    if (steps == 0) item = end;
    find_rows();
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch();
  }
  static __device__ __forceinline__ const T* base(const MoeFewParams& p) { return static_cast<const T*>(HIDDEN ? p.down : p.gate_up); }
  // The lane's row i (r and r + 8 of each half) of a tile in a pass's matrix: 32 rows of D; or 16 rows of G, each
  // followed by the row of U that goes with it.
  __device__ __forceinline__ const T* row_of(int in, int of, int i) const {
    const int lane = (threadIdx.x & 31) / 4;
    const T* const matrix = base(p) + static_cast<long long>(r.passes[in].expert * (HIDDEN ? 1 : 2)) * rows * n;
    const int row = HIDDEN ? of * MF_ROWS + 8 * i + lane : of * (MF_ROWS / 2) + 8 * (i / 2) + lane;
    return matrix + static_cast<long long>(min(row, rows - 1) + (HIDDEN ? 0 : (i & 1) * rows)) * n;
  }
  __device__ __forceinline__ void find_rows() {
    s = 0;
    k = k0;
    if (item >= end) return;
    while (tile >= tiles) {
      tile -= tiles;
      ++pass;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = row_of(pass, tile, i);
  }
  __device__ __forceinline__ void fetch() {
    if (item < end) {
      const int lane = threadIdx.x & 31;
      if constexpr (VEC) {
        const int bytes = k < n ? 16 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) nsptx::cp_async16_upto(ring + fill + 32 * i + lane, at[i] + k, bytes, policy);
      } else {
        const T* const last = base(p) + (HIDDEN ? p.experts * p.dim : p.experts * 2 * p.ffn) * n;  // past the matrices
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch_words(reinterpret_cast<uint32_t*>(ring + fill) + i * PLANES * 32 + lane, at[i], last);
      }
      k += step;
      if (++s == steps) {
        item += stride;
        tile += stride;
        find_rows();
      }
    }
    nsptx::cp_async_commit();
    fill = fill + STAGE == RING ? 0 : fill + STAGE;
  }
  // The aligned 4-byte words, 32 apart, that cover what is left of 16 bytes from k on. One that begins before the
  // matrices or ends behind them is put together from its values.
  __device__ __forceinline__ void fetch_words(uint32_t* to, const T* row, const T* last) const {
    const uintptr_t from = reinterpret_cast<uintptr_t>(row + k), word = from & ~uintptr_t{3};
    const int bytes = static_cast<int>(from - word) + min(n - k, V) * static_cast<int>(sizeof(T));
#pragma unroll
    for (int w = 0; w < PLANES; ++w) {
      if (4 * w >= bytes || k >= n) break;
      const uintptr_t q = word + 4 * w;
      if (sizeof(T) == 4 || (q >= reinterpret_cast<uintptr_t>(base(p)) && q + 4 <= reinterpret_cast<uintptr_t>(last))) {
        nsptx::cp_async4(to + 32 * w, reinterpret_cast<const void*>(q));
      } else {
        uint32_t v = 0;
        if (q >= reinterpret_cast<uintptr_t>(base(p))) v = *reinterpret_cast<const unsigned short*>(q);
        if (q + 4 <= reinterpret_cast<uintptr_t>(last)) v |= static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(q + 2)) << 16;
        to[32 * w] = v;
      }
    }
  }
  // 16 bytes of a row from those words, `odd`: from the middle of the first on; `left` values, zeros behind.
  static __device__ __forceinline__ uint4 from_words(const uint32_t* words, bool odd, int left) {
    uint32_t w[PLANES], v[4];
#pragma unroll
    for (int i = 0; i < PLANES; ++i) w[i] = words[32 * i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = sizeof(T) == 2 && odd ? __funnelshift_r(w[i], w[PLANES - 1 < i + 1 ? i : i + 1], 16) : w[i];
      constexpr int PER = 4 / sizeof(T);
      if (left <= PER * i)
        v[i] = 0;
      else if (PER == 2 && left == 2 * i + 1)
        v[i] &= 0xffffu;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }

  // Puts the lane's words of 8 * NT slots, whose rows are `row`, for all of the warp's steps at `held`.
  template <int NT>
  __device__ __forceinline__ void hold(const char* const (&row)[NT], uint4* held) const {
    for (int i = 0; i < steps; ++i) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        S side;
        side.template load<VEC>(row[t], k0 + i * step, n);
#pragma unroll
        for (int j = 0; j < S::Q; ++j) held[((i * NT + t) * S::Q + j) * 32] = side.q[j];
      }
    }
  }
  // Words that are not held are loaded a step ahead (`now`, at first those of step 0), while registers last.
  template <int NT, bool HELD>
  static constexpr bool EARLY = !HELD && NT * S::Q <= 4;
  template <int NT>
  __device__ __forceinline__ void load(const char* const (&row)[NT], S (&side)[NT], int i) const {
#pragma unroll
    for (int t = 0; t < NT; ++t) side[t].template load<VEC>(row[t], k0 + i * step, n);
  }
  // The products of the next tile, `of` of pass `in`, with those slots.
  template <int NT, bool HELD>
  __device__ __forceinline__ void products(int in, int of, const char* const (&row)[NT], const uint4* held, S (&now)[NT], float (&acc)[2][NT][4]) {
    const int lane = threadIdx.x & 31;
    bool odd[4] = {};
    if constexpr (!VEC && sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) odd[i] = reinterpret_cast<uintptr_t>(row_of(in, of, i)) & 2;
    }
    for (int i = 0; i < steps; ++i) {
      S side[NT];
      if constexpr (HELD) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < S::Q; ++j) side[t].q[j] = held[((i * NT + t) * S::Q + j) * 32];
      } else if constexpr (EARLY<NT, HELD>) {
#pragma unroll
        for (int t = 0; t < NT; ++t) side[t] = now[t];
        load<NT>(row, now, i + 1 < steps ? i + 1 : 0);
      } else {
        load<NT>(row, side, i);
      }
      nsptx::cp_async_wait<AHEAD - 1>();
      uint4 a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (VEC)
          a[j] = ring[take + 32 * j + lane];
        else
          a[j] = from_words(reinterpret_cast<const uint32_t*>(ring + take) + j * PLANES * 32 + lane, odd[j], n - k0 - i * step);
      }
      take = take + STAGE == RING ? 0 : take + STAGE;
      if constexpr (S::LONG) fetch();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        times(acc[0][t], a[0], a[1], side[t]);
        times(acc[1][t], a[2], a[3], side[t]);
      }
      if constexpr (!S::LONG) fetch();
    }
  }
};

// A barrier of the team's warps, each of them together.
__device__ __forceinline__ void team_sync(int team, int warps) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * warps) : "memory");
}

// What a team of warps, which split k of its tiles, has at hand.
struct Team {
  int warps, warp, id;   // of the team; this one's; the team's number
  uint4* held;           // the lane's words
  float* sums;           // [MF_NT][warps][8][32]
};

// A team's tiles of one pass, from `item` on: use(tile, row, slot, a, b) gets the
// sums of rows `row` and `row` + 8 of a tile for a slot, row < 8 or 16 <= row < 24.
template <int NT, bool HELD, typename S, typename F>
__device__ __forceinline__ void tiles_of_pass(S& stream, const Team& team, int& item, int to, int pass, F&& use) {
  const MoeFewParams& p = stream.p;
  const Routing& r = stream.r;
  const Pass of = r.passes[pass];
  const int lane = threadIdx.x & 31;
  const char* row[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int i = 8 * t + lane / 4;
    row[t] = S::S::row(p, r.sorted[of.first + (i < of.count ? i : 0)]);
  }
  typename S::S now[NT];
  if constexpr (HELD) stream.template hold<NT>(row, team.held);
  if constexpr (S::template EARLY<NT, HELD>) stream.template load<NT>(row, now, 0);
  for (; item < to; item += stream.stride) {
    const int tile = item - pass * stream.tiles;
    float acc[2][NT][4] = {};
    stream.template products<NT, HELD>(pass, tile, row, team.held, now, acc);
    // a lane's sums: of rows lane / 4 and 8 more of each half of the tile, columns 2 (lane % 4) and the next
    auto give = [&](int t, int half, int c, int at, float a, float b) {
      const int j = 8 * t + 2 * (at & 3) + c;
      if (j < of.count) use(tile, 16 * half + at / 4, static_cast<int>(r.sorted[of.first + j]), a, b);
    };
    if (team.warps == 1) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) give(t, q >> 1, q & 1, lane, acc[q >> 1][t][q & 1], acc[q >> 1][t][(q & 1) + 2]);
      continue;
    }
    team_sync(team.id, team.warps);  // the last sums are read
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) team.sums[((t * team.warps + team.warp) * 8 + i) * 32 + lane] = acc[i / 4][t][i % 4];
    team_sync(team.id, team.warps);
    // Of all slots at once (64 experts by 12 slots each took 222 us then, 8 by 8 of them 236).
    // By four warps for 8 slots, in a fixed order of all, while the others go on with the next tile. (By two of them in
    // wider words 64 experts by 8 slots each take 228 us, by all 225, so 208.)
    for (int q = team.warp; q < 4 * NT; q += team.warps) {
      const int t = q >> 2, half = (q >> 1) & 1, c = q & 1;
      float a = 0.0f, b = 0.0f;
      const float* from = team.sums + (t * team.warps * 8 + half * 4 + c) * 32 + lane;
      for (int w = 0; w < team.warps; ++w, from += 8 * 32) {
        a += from[0];
        b += from[2 * 32];
      }
      give(t, half, c, lane, a, b);
    }
  }
}

// A block's share of all passes' tiles.
template <typename T, bool HIDDEN, bool VEC, typename F>
__device__ __forceinline__ void all_tiles(const MoeFewParams& p, const Routing& r, uint4* smem, int passes, int tiles, F&& use) {
  using S = Side<T, HIDDEN>;
  const long long items = static_cast<long long>(passes) * tiles;
  const int first = static_cast<int>(items * blockIdx.x / gridDim.x), last = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int RING = RING_WORDS<S, HIDDEN, VEC>;
  uint4* const held = smem + MF_WARPS * RING;
  float* const sums = reinterpret_cast<float*>(held + MF_WARPS * p.held * 32);
  const Team team = {p.team, warp & (p.team - 1), warp / p.team, held + warp * p.held * 32 + lane, sums + warp / p.team * p.team * MF_NT * 8 * 32};
  Stream<T, HIDDEN, VEC> stream(p, r, smem + warp * RING, first, last, team.id, MF_WARPS / p.team, team.warp, tiles);
  for (int item = first + team.id, pass = item / tiles; item < last; ++pass) {
    const int to = min(last, (pass + 1) * tiles), count = r.passes[pass].count;
    const int words = S::Q * stream.most_steps;
    if (count <= 8 && words <= p.held)
      tiles_of_pass<1, true>(stream, team, item, to, pass, use);
    else if (count <= 8)
      tiles_of_pass<1, false>(stream, team, item, to, pass, use);
    else if (2 * words <= p.held)
      tiles_of_pass<2, true>(stream, team, item, to, pass, use);
    else
      tiles_of_pass<2, false>(stream, team, item, to, pass, use);
  }
}

// Shared memory: the rings, what is held of the tokens, the parts of split sums, the routing.
template <typename T, bool HIDDEN, bool VEC>
constexpr int FIXED_WORDS = MF_WARPS * (RING_WORDS<Side<T, HIDDEN>, HIDDEN, VEC> + 8 * 8 * MF_NT);
constexpr int MF_HELD_WORDS = MF_WARPS * 32;
constexpr size_t MF_SMEM = 226 * 1024;
template <typename T, bool HIDDEN, bool VEC>
__device__ __forceinline__ Routing routing_of(const MoeFewParams& p, uint4* smem) {
  return Routing(p, smem + FIXED_WORDS<T, HIDDEN, VEC> + p.held * MF_HELD_WORDS);
}

// h of all slots.
template <typename T, bool VEC>
__global__ void __launch_bounds__(MF_THREADS, 1) ns_moe_few_hidden_kernel(const __grid_constant__ MoeFewParams p) {
  extern __shared__ uint4 few_smem[];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const Routing r = routing_of<T, false, VEC>(p, few_smem);
  const int passes = find_passes(p, r);
  all_tiles<T, false, VEC>(
      p, r, few_smem, passes, static_cast<int>((p.ffn + MF_ROWS / 2 - 1) / (MF_ROWS / 2)),
      [&](int tile, int row, int slot, float a, float b) {
        const long long f = tile * (MF_ROWS / 2) + (row & 7) + row / 16 * 8;
        if (f >= p.hidden_ld) return;
        // zero up to the row's end: its last words are read whole
        p.hidden[slot * p.hidden_ld + f] = f < p.ffn ? a / (1.0f + expf(-a)) * b : 0.0f;
      });
}

// D_e h of all slots.
template <typename T, bool VEC>
__global__ void __launch_bounds__(MF_THREADS, 1) ns_moe_few_down_kernel(const __grid_constant__ MoeFewParams p) {
  extern __shared__ uint4 few_smem[];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const Routing r = routing_of<T, true, VEC>(p, few_smem);
  const int passes = find_passes(p, r);
  all_tiles<T, true, VEC>(p, r, few_smem, passes, static_cast<int>((p.dim + MF_ROWS - 1) / MF_ROWS),
                          [&](int tile, int row, int slot, float a, float b) {
                            // part_ld is a multiple of MF_ROWS
                            float* const to = p.part + slot * p.part_ld + tile * MF_ROWS + row;
                            to[0] = a;
                            to[8] = b;
                          });
}

// y: the sums over each token's slots, in the slots' order, 4 values a thread.
// (Summed by the warp that brought a token's last part, the layer took one kernel
// less and 64 experts by one slot each 237 us instead of 202: a team waits for its
// warp's fence, count and loads.)
template <typename T>
__global__ void __launch_bounds__(MF_SUM_THREADS) ns_moe_few_sum_kernel(const __grid_constant__ MoeFewParams p) {
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int t = blockIdx.y;
  const long long d = (static_cast<long long>(blockIdx.x) * MF_SUM_THREADS + threadIdx.x) * 4;
  if (d >= p.dim) return;
  float y[4] = {};
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    float4 v[8];
    float w[8];
    bool there[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int slot = t * p.k + min(j0 + i, p.k - 1);
      const long long e = load_index(p.ids, p.id_bytes, slot);
      there[i] = j0 + i < p.k && e >= 0 && e < p.experts;
      w[i] = p.weights ? p.weights[slot] : 1.0f;
      v[i] = *reinterpret_cast<const float4*>(p.part + slot * p.part_ld + d);  // before it is known whether it is used
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!there[i]) continue;
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

// Warps that split a tile's k: as many as have some 4 steps each. A block's tiles are then few and small, so that all
// blocks have as many, and it reads long pieces of rows. (A warp a tile: some warps have three tiles where others have
// two.) Where there are too few tiles for the card's warps, a step or two each.
int team_of(long long tiles, long long steps, int nsm) {
  int team = 1;
  while (team < MF_WARPS && (steps >= 6 * team || (steps >= 2 * team && 2 * team * tiles <= nsm * MF_WARPS))) team *= 2;
  return team;
}

template <typename T, bool VEC>
int launch_few(MoeFewParams p, int nsm, cudaStream_t st) {
  constexpr int VALUES = 64 / sizeof(T);  // of a step
  const int slots = p.tokens * p.k, named = std::min(p.experts, slots);
  p.entries = named + slots / (8 * MF_NT);
  const size_t routing = routing_bytes(p.entries, p.experts, slots);
  static_assert(sizeof(uint4) * std::max(FIXED_WORDS<T, false, VEC>, FIXED_WORDS<T, true, VEC>) + routing_bytes(1024 + MF_MAX_TOKENS * 32 / (8 * MF_NT), 1024, MF_MAX_TOKENS * 32) <= MF_SMEM,
                "shared memory of a block");
  auto launch = [&](void (*kernel)(MoeFewParams), int fixed_words, long long tiles, long long n, int words) {
    const long long steps = (n + VALUES - 1) / VALUES;
    p.team = team_of(tiles * named, steps, nsm);
    const size_t fixed = sizeof(uint4) * fixed_words + routing;
    // of 8 or 16 slots; what is not held stays with L1
    const long long room = (MF_SMEM - fixed) / (sizeof(uint4) * MF_HELD_WORDS);
    const long long most = (steps + p.team - 1) / p.team * words;
    p.held = static_cast<int>(p.tokens > 8 && 2 * most <= room ? 2 * most : most <= room ? most : 0);
    const size_t smem = fixed + p.held * sizeof(uint4) * MF_HELD_WORDS;
    const long long teams = (tiles * p.entries * p.team + MF_WARPS - 1) / MF_WARPS;
    const int blocks = static_cast<int>(std::min<long long>(nsm, teams));
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(MF_SMEM));
    if (e != cudaSuccess) return e;
    return nsorch::counted(nsorch::K_MOE, st, [&] { return launch_pdl(kernel, dim3(blocks), dim3(MF_THREADS), smem, st, p); });
  };
  cudaError_t e = launch(ns_moe_few_hidden_kernel<T, VEC>, FIXED_WORDS<T, false, VEC>, (p.ffn + MF_ROWS / 2 - 1) / (MF_ROWS / 2), p.dim, Side<T, false>::Q);
  if (e == cudaSuccess) e = launch(ns_moe_few_down_kernel<T, VEC>, FIXED_WORDS<T, true, VEC>, (p.dim + MF_ROWS - 1) / MF_ROWS, p.ffn, Side<T, true>::Q);
  if (e != cudaSuccess) return NS_ERR_CUDA;
  e = nsorch::counted(nsorch::K_MOE, st, [&] {
    const unsigned int wide = static_cast<unsigned int>((p.dim + 4 * MF_SUM_THREADS - 1) / (4 * MF_SUM_THREADS));
    return launch_pdl(ns_moe_few_sum_kernel<T>, dim3(wide, p.tokens), dim3(MF_SUM_THREADS), 0, st, p);
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

// The workspace's parts: hidden values, products.
struct FewParts {
  int64_t hidden_ld, part_ld;
  uint64_t part, bytes;
  FewParts(int64_t tokens, int k, int64_t dim, int64_t ffn) {
    const uint64_t slots = static_cast<uint64_t>(tokens) * k;
    hidden_ld = (ffn + 7) / 8 * 8;
    part_ld = (dim + nsk::MF_ROWS - 1) / nsk::MF_ROWS * nsk::MF_ROWS;
    part = (4 * slots * hidden_ld + 255) / 256 * 256;
    bytes = part + 4 * slots * part_ld;
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
  p.hidden = static_cast<float*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + parts.part);
  int dev, nsm;
  if ((rc = device_setup(&dev, &p.status, &nsm)) != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == NS_DT_BF16) return nsk::launch_few<__nv_bfloat16>(p, nsm, st);
  if (dtype == NS_DT_FP16) return nsk::launch_few<__half>(p, nsm, st);
  return nsk::launch_few<float>(p, nsm, st);
}

}  // extern "C"
