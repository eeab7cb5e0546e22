// Tokens sorted by expert and back: the routing between a mixture-of-experts
// layer's tokens and its experts' rows, forward and backward.
//
// Slot s = t * k + j is token t's j-th choice. With e_s its expert,
//   rank_s   = number of slots s' < s with e_s' = e_s
//   kept     : 0 <= e_s < E and rank_s < capacity
//   row_s    = offset[e_s] + rank_s, offset the exclusive sum of the kept
//              counts, each rounded up to a multiple of `align`
// and then
//   dispatch       xs[row_s]  = x[t]             (0 in rows without a slot)
//   its gradient   dx[t]      = sum_j dxs[row(t, j)]
//   combine        y[t]       = sum_j w[t, j] ys[row(t, j)]
//   its gradient   dys[row_s] = w_s dy[t], dw[t, j] = <dy[t], ys[row(t, j)]>
// Sums over j are in fp32 in the order of j, dot products in a fixed order:
// the same call gives the same bits.
//
// The sort is bound by latency: 32 x 8 slots take one launch of 2.7 us,
// 32768 x 6 two, 7.8 us a pass: the ids are counted, then placed.
// The rest moves whole rows and is bound by memory: 8192 x 6 rows of 2048 bf16
// are dispatched (padded to 128 rows an expert) in 43 us, 6.3 TB/s, combined in
// 37 us, 6.3 TB/s, and the gradient of combining them takes 69 us, 6.3 TB/s,
// against 6.7 TB/s of the measured copy.
#include <algorithm>
#include <climits>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_K = 32;
constexpr long long MAX_SLOTS = 1 << 30;  // and rows: indexes and their steps fit an int
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_HELD = 4;  // rounds of 32 slots that a warp keeps in registers
constexpr int SORT_MAX_BLOCKS = 256;
constexpr int ROW_THREADS = 128;
constexpr int MANY_WARPS = 16;  // of a block where many share a token
// Rows that a warp clears; twice as many where they are short (28351 x 2 rows of 128
// dispatched in 10.5 us against 12.5).
constexpr int CLEAR_ROWS = 4;

// Counts of a block, a whole number of 16-byte words.
__host__ __device__ inline int count_stride(int experts) { return (experts + 3) / 4 * 4; }

struct SortParams {
  const void* ids;
  int id_bytes;
  int slots, experts, align, capacity, rows;
  int chunk;   // slots per block, a multiple of SORT_THREADS
  int blocks;
  int* row_of_slot;
  int* slot_of_row;
  int* counts;
  int* offsets;
  int* block_counts;  // [blocks][count_stride]
  unsigned int* status;
};

// Expert of a slot; -1 for a slot that goes nowhere (a negative id, or one
// past the last expert, which is refused).
__device__ __forceinline__ int slot_expert(const SortParams& p, int s, bool* refused) {
  const long long e = load_index(p.ids, p.id_bytes, s);
  if (e >= p.experts) *refused = true;
  return e >= 0 && e < p.experts ? static_cast<int>(e) : -1;
}

// Counts of one chunk's experts.
__global__ void __launch_bounds__(SORT_THREADS) ns_moe_count_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int sm[];
  for (int e = threadIdx.x; e < p.experts; e += SORT_THREADS) sm[e] = 0;
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  __syncthreads();
  const int s0 = blockIdx.x * p.chunk, s1 = min(p.slots, s0 + p.chunk);
  bool refused = false;
  for (int s = s0 + threadIdx.x; s < s1; s += SORT_THREADS) {
    const int e = slot_expert(p, s, &refused);
    if (e >= 0) atomicAdd(&sm[e], 1);
  }
  __syncthreads();
  const int stride = count_stride(p.experts);
  for (int e = threadIdx.x; e < stride; e += SORT_THREADS)
    p.block_counts[blockIdx.x * stride + e] = e < p.experts ? sm[e] : 0;
}

// Places one chunk's slots. Warp w owns a contiguous part of the chunk, 32
// slots a round; the rank of a slot is (slots of its expert in earlier chunks)
// + (in earlier warps) + (in earlier rounds of this warp) + (in lower lanes).
// HELD: the warp's slots fit SORT_HELD rounds, whose experts and ranks stay in
// registers; else they are read and ranked once more when they are placed.
template <bool HELD>
__global__ void __launch_bounds__(SORT_THREADS) ns_moe_place_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int sm[];
  __shared__ int warp_rows[SORT_WARPS];
  const int E = p.experts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* next = sm;                       // [warps][E]: count, then the next rank
  int* before = sm + SORT_WARPS * E;    // [E]: slots in earlier chunks
  int* total = before + E;              // [E]
  int* offset = total + E;              // [E + 1]
  for (int i = threadIdx.x; i < (SORT_WARPS + 2) * E; i += SORT_THREADS) sm[i] = 0;
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();

  const int per_warp = p.chunk / SORT_WARPS;
  const int w0 = min(p.slots, static_cast<int>(blockIdx.x) * p.chunk + warp * per_warp);
  const int w1 = min(p.slots, w0 + per_warp);
  bool refused = false;
  int held[SORT_HELD], rank[SORT_HELD];
  if (HELD) {
#pragma unroll
    for (int i = 0; i < SORT_HELD; ++i) {
      const int s = w0 + i * 32 + lane;
      held[i] = s < w1 ? slot_expert(p, s, &refused) : -1;
    }
  }
  __syncthreads();
  // rank of a slot among this warp's of its expert so far, counted on top of
  // what `next` holds
  auto take = [&](int e) {
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    int r = 0;
    if (e >= 0) r = next[warp * E + e] + __popc(peers & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && (peers >> lane) == 1u) next[warp * E + e] = r + 1;  // the highest lane of its peers
    __syncwarp();
    return r;
  };
  if (HELD) {
#pragma unroll
    for (int i = 0; i < SORT_HELD; ++i)
      if (w0 + i * 32 < w1) rank[i] = take(held[i]);
  } else {
    for (int s = w0 + lane; s < w1; s += 32) {
      const int e = slot_expert(p, s, &refused);
      if (e >= 0) atomicAdd(&next[warp * E + e], 1);
    }
  }
  if (refused) atomicOr(p.status, NS_DEV_BAD_INDEX);
  if (p.blocks > 1) {
    // four experts a thread; the threads that share them split the blocks
    const int lanes = count_stride(E) / 4, group = threadIdx.x / lanes, groups = SORT_THREADS / lanes;
    const int e = (threadIdx.x - group * lanes) * 4;
    int all[4] = {0, 0, 0, 0}, early[4] = {0, 0, 0, 0};
    if (group < groups) {
#pragma unroll 8
      for (int b = group; b < p.blocks; b += groups) {
        const int4 c = *reinterpret_cast<const int4*>(p.block_counts + b * count_stride(E) + e);
        const int v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          all[i] += v[i];
          if (b < static_cast<int>(blockIdx.x)) early[i] += v[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < E) {
          atomicAdd(&total[e + i], all[i]);
          atomicAdd(&before[e + i], early[i]);
        }
    }
  }
  __syncthreads();
  // per expert: the warps' first ranks, and the rows of its segment; then the
  // exclusive sum of those, SORT_THREADS experts at a time
  int rows_before = 0;
  for (int e0 = 0; e0 < E; e0 += SORT_THREADS) {
    const int e = e0 + threadIdx.x;
    int rows = 0;
    if (e < E) {
      int run = before[e];
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) {
        const int c = next[w * E + e];
        next[w * E + e] = run;
        run += c;
      }
      if (p.blocks == 1) total[e] = run;
      const unsigned kept = min(total[e], p.capacity), align = p.align;
      rows = static_cast<int>(align == 1 ? kept : (kept + align - 1) / align * align);
    }
    int upto = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) warp_rows[warp] = upto;
    __syncthreads();
    int start = rows_before + upto - rows;
#pragma unroll
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int v = warp_rows[w];
      if (w < warp) start += v;
      rows_before += v;
    }
    if (e < E) {
      offset[e] = start;
      if (blockIdx.x == 0) {
        p.counts[e] = min(total[e], p.capacity);
        p.offsets[e] = start;
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    offset[E] = rows_before;
    if (blockIdx.x == 0) p.offsets[E] = rows_before;
  }

  auto place = [&](int s, int e, int r) {
    int row = -1;
    if (e >= 0 && r < p.capacity) {
      row = offset[e] + r;
      p.slot_of_row[row] = s;
    }
    p.row_of_slot[s] = row;
  };
  if (HELD) {
#pragma unroll
    for (int i = 0; i < SORT_HELD; ++i) {
      const int s = w0 + i * 32 + lane;
      if (s < w1) place(s, held[i], held[i] >= 0 ? next[warp * E + held[i]] + rank[i] : 0);
    }
  } else {
    for (int i = w0; i < w1; i += 32) {
      const int s = i + lane;
      const int e = s < w1 ? slot_expert(p, s, &refused) : -1;
      const int r = take(e);
      if (s < w1) place(s, e, r);
    }
  }
  // rows without a slot: the ends of the segments, and what follows the last
  __syncthreads();
  for (int e = blockIdx.x * SORT_WARPS + warp; e < E; e += p.blocks * SORT_WARPS)
    for (int r = offset[e] + min(total[e], p.capacity) + lane; r < offset[e + 1]; r += 32) p.slot_of_row[r] = -1;
  for (int r = rows_before + blockIdx.x * SORT_THREADS + threadIdx.x; r < p.rows; r += p.blocks * SORT_THREADS)
    p.slot_of_row[r] = -1;
}

// --------------------------------------------------------- rows of tokens
struct RowParams {
  const void* src;          // dispatch: x; dispatch gradient, combine: rows; combine gradient: dy
  const void* rows_in;      // combine gradient: ys
  void* dst;
  long long src_ld, rows_ld, dst_ld;  // elements between rows
  const int* row_of_slot;
  const int* slot_of_row;
  const float* weights;     // null: 1
  float* grad_weights;
  long long tokens, rows, dim;
  int k;
  int parts;                // warps that share one token
  int clear;                // rows that a warp clears, where they hold no slot
  long long token_warps;    // warps before the ones that clear rows without a slot
  unsigned int* status;
};

// Row of token t's slot `lane`, -1 where there is none; a row outside the
// buffer is refused.
__device__ __forceinline__ int lane_row(const RowParams& p, long long t, int lane) {
  int r = -1;
  if (lane < p.k) r = p.row_of_slot[t * p.k + lane];
  if (r >= p.rows) {
    atomicOr(p.status, NS_DEV_BAD_INDEX);
    r = -1;
  }
  return r;
}

// Clears those of p.clear rows that hold no slot. Few rows a warp: they come
// in runs (the ends of segments), and a warp with 32 of them to clear would end
// long after the others.
template <typename T, int V>
__device__ __forceinline__ void clear_rows(const RowParams& p, long long group, int lane) {
  const long long r = group * p.clear + lane;
  unsigned todo = __ballot_sync(0xffffffffu, lane < p.clear && r < p.rows && p.slot_of_row[r] < 0);
  while (todo) {
    const int i = __ffs(todo) - 1;
    todo &= todo - 1;
    T* row = static_cast<T*>(p.dst) + (group * p.clear + i) * p.dst_ld;
    if (V == 1 && p.dim >= 512) {
      // zeros need no words of the row's own: 16 bytes at a time between its ends (8192 x 6 rows of 2047 bf16
      // among their padding dispatched in 47 us, element by element 53; 4-byte words lose by it, and short rows)
      constexpr int W = 16 / sizeof(T);
      const long long head = head_of(row, p.dim), words = (p.dim - head) / W, ends = p.dim - words * W;
      for (long long c = lane; c < words; c += 32) store_vec<T, W>(row + head + c * W, zero_vec<T, W>());
      for (long long c = lane; c < ends; c += 32) row[c < head ? c : words * W + c] = from_float<T>(0.0f);
    } else {
      for (long long c = lane * V; c < p.dim; c += 32 * V) store_vec<T, V>(row + c, zero_vec<T, V>());
    }
  }
}

// dispatch: a warp holds up to 32 * V * U elements of a token's row and stores
// them to each of its rows, so x is read once. (Bulk copies through shared
// memory measured no faster: a row's stores are what takes the time.)
template <typename T, int V, int U>
__global__ void __launch_bounds__(ROW_THREADS) ns_moe_dispatch_kernel(const __grid_constant__ RowParams p) {
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * (ROW_THREADS / 32) + (threadIdx.x >> 5);
  if (w >= p.token_warps) {
    clear_rows<T, V>(p, w - p.token_warps, lane);
    return;
  }
  const long long t = w / p.parts;
  const int start = static_cast<int>(w - t * p.parts) * (32 * V * U), c0 = start + lane * V;
  const int dim = static_cast<int>(p.dim);
  const T* src = static_cast<const T*>(p.src) + t * p.src_ld + c0;
  const int mine = lane_row(p, t, lane);
  // `whole`: the piece ends inside the row, and needs no check of its columns
  auto piece = [&](auto whole) {
    Vec<T, V> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (decltype(whole)::value || c0 + u * 32 * V < dim) x[u] = load_vec<T, V>(src + u * 32 * V);
    for (int j = 0; j < p.k; ++j) {
      const int r = __shfl_sync(0xffffffffu, mine, j);
      if (r < 0) continue;
      T* dst = static_cast<T*>(p.dst) + r * p.dst_ld + c0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (decltype(whole)::value || c0 + u * 32 * V < dim) store_vec<T, V>(dst + u * 32 * V, x[u]);
    }
  };
  if (start + 32 * V * U <= dim)
    piece(std::true_type());
  else
    piece(std::false_type());
}

// combine and the gradient of dispatch: a warp sums 32 * V * U elements of a
// token's rows, with those of J rows on their way at once.
template <typename T, int V, int U, int J>
__global__ void __launch_bounds__(ROW_THREADS) ns_moe_gather_kernel(const __grid_constant__ RowParams p) {
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * (ROW_THREADS / 32) + (threadIdx.x >> 5);
  if (w >= p.token_warps) return;
  const long long t = w / p.parts;
  const int start = static_cast<int>(w - t * p.parts) * (32 * V * U), c0 = start + lane * V;
  const int dim = static_cast<int>(p.dim);
  const int mine = lane_row(p, t, lane);
  const float my_weight = p.weights && lane < p.k ? p.weights[t * p.k + lane] : 1.0f;
  auto piece = [&](auto whole) {
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[u][i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += J) {
      Vec<T, V> x[J][U];
      float wt[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int r = j0 + j < MAX_K ? __shfl_sync(0xffffffffu, mine, j0 + j) : -1;  // -1 past the last slot too
        wt[j] = __shfl_sync(0xffffffffu, my_weight, j0 + j);
        const T* src = static_cast<const T*>(p.src) + r * p.src_ld + c0;
        if (r >= 0) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            x[j][u] =
                decltype(whole)::value || c0 + u * 32 * V < dim ? load_vec<T, V>(src + u * 32 * V) : zero_vec<T, V>();
        } else {
          wt[j] = 0.0f;
#pragma unroll
          for (int u = 0; u < U; ++u) x[j][u] = zero_vec<T, V>();
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[u][i] = fmaf(wt[j], get(x[j][u], i), acc[u][i]);
    }
    T* dst = static_cast<T*>(p.dst) + t * p.dst_ld + c0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (decltype(whole)::value || c0 + u * 32 * V < dim) store_vec<T, V>(dst + u * 32 * V, pack<T, V>(acc[u]));
  };
  if (start + 32 * V * U <= dim)
    piece(std::true_type());
  else
    piece(std::false_type());
}

// combine's gradient: `parts` warps of one block share a token; each walks its
// pieces of the row, writes w dy and sums dy ys, slot j's sum in lane j, with
// the pieces of J rows on their way at once.
template <typename T, int V, int U, int J, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) ns_moe_combine_grad_kernel(const __grid_constant__ RowParams p) {
  __shared__ float part_sum[WARPS][MAX_K];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long w = static_cast<long long>(blockIdx.x) * WARPS + warp;
  const bool on = w < p.token_warps;
  const long long t = w / p.parts;
  const int part = static_cast<int>(w - t * p.parts), dim = static_cast<int>(p.dim);
  float sum = 0.0f;
  if (on) {
    const T* dy = static_cast<const T*>(p.src) + t * p.src_ld;
    const int mine = lane_row(p, t, lane);
    const float my_weight = lane < p.k ? p.weights[t * p.k + lane] : 0.0f;
    auto piece = [&](int c0, auto whole) {
      float g[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Vec<T, V> x =
            decltype(whole)::value || c0 + u * 32 * V < dim ? load_vec<T, V>(dy + c0 + u * 32 * V) : zero_vec<T, V>();
#pragma unroll
        for (int i = 0; i < V; ++i) g[u][i] = get(x, i);
      }
      for (int j0 = 0; j0 < p.k; j0 += J) {
        int r[J];
        Vec<T, V> y[J][U];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          r[j] = j0 + j < MAX_K ? __shfl_sync(0xffffffffu, mine, j0 + j) : -1;  // -1 past the last slot too
          const T* ys = static_cast<const T*>(p.rows_in) + r[j] * p.rows_ld + c0;
          if (r[j] >= 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (decltype(whole)::value || c0 + u * 32 * V < dim) y[j][u] = load_vec<T, V>(ys + u * 32 * V);
          }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (r[j] < 0) continue;
          const float wt = __shfl_sync(0xffffffffu, my_weight, j0 + j);
          T* out = static_cast<T*>(p.dst) + r[j] * p.dst_ld + c0;
          float dot = 0.0f;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (decltype(whole)::value || c0 + u * 32 * V < dim) {
              float o[V];
#pragma unroll
              for (int i = 0; i < V; ++i) {
                dot = fmaf(g[u][i], get(y[j][u], i), dot);
                o[i] = wt * g[u][i];
              }
              store_vec<T, V>(out + u * 32 * V, pack<T, V>(o));
            }
          dot = warp_sum(dot);
          if (lane == j0 + j) sum += dot;
        }
      }
    };
    for (int start = part * (32 * V * U); start < dim; start += p.parts * (32 * V * U)) {
      if (start + 32 * V * U <= dim)
        piece(start + lane * V, std::true_type());
      else
        piece(start + lane * V, std::false_type());
    }
    if (p.parts == 1 && lane < p.k) p.grad_weights[t * p.k + lane] = sum;
  } else {
    clear_rows<T, V>(p, w - p.token_warps, lane);
  }
  if (p.parts == 1) return;
  part_sum[warp][lane] = sum;
  __syncthreads();
  if (on && part == 0 && lane < p.k) {
    for (int q = 1; q < p.parts; ++q) sum += part_sum[warp + q][lane];
    p.grad_weights[t * p.k + lane] = sum;
  }
}

}  // namespace
}  // namespace nsk

using namespace nsorch;

namespace {

using nsk::dtype_ok;
using nsk::elem_bytes;
using nsk::element_aligned;

bool all_aligned(int bytes, std::initializer_list<const void*> ps) {
  return std::all_of(ps.begin(), ps.end(), [&](const void* p) { return element_aligned(p, bytes); });
}
// Whether rows at p, `ld` elements apart, and their width are whole words.
bool in_words(const void* p, long long ld, long long dim, int elem, int word) {
  return reinterpret_cast<uintptr_t>(p) % word == 0 && ld * elem % word == 0 && dim * elem % word == 0;
}
// The widest word that all rows are made of: 16 bytes, 4, or an element.
int common_word(int elem, long long dim, std::initializer_list<std::pair<const void*, long long>> rows) {
  for (int word : {16, 4}) {
    bool all = true;
    for (const auto& r : rows) all = all && in_words(r.first, r.second, dim, elem, word);
    if (all) return word;
  }
  return elem;
}

// Slots per block and blocks of a sort: one block for as many slots as its warps
// hold in registers, then blocks of that size (with the counts first, a second
// launch), then larger ones.
void sort_split(long long slots, int* chunk, int* blocks) {
  constexpr int held = nsk::SORT_THREADS * nsk::SORT_HELD;
  long long c = slots;
  if (slots > held) c = std::max<long long>(held, (slots + nsk::SORT_MAX_BLOCKS - 1) / nsk::SORT_MAX_BLOCKS);
  c = std::max<long long>(1, (c + nsk::SORT_THREADS - 1) / nsk::SORT_THREADS) * nsk::SORT_THREADS;
  *chunk = static_cast<int>(c);
  *blocks = static_cast<int>(std::max<long long>(1, (slots + c - 1) / c));
}

int sort_args(int64_t tokens, int k, int experts) {
  if (tokens < 0 || k < 1 || experts < 1) return NS_ERR_ARG;
  if (k > nsk::MAX_K || experts > nsk::MAX_EXPERTS) return NS_ERR_UNSUPPORTED;
  if (tokens > nsk::MAX_SLOTS / k) return NS_ERR_SHAPE;
  return NS_OK;
}

// Dynamic shared memory of ns_moe_place_kernel.
constexpr size_t place_smem(int experts) {
  return (static_cast<size_t>(nsk::SORT_WARPS + 3) * experts + 1) * sizeof(int);
}

// Checks shared by the four row operators.
int row_args(int dtype, int64_t tokens, int k, int64_t dim, int64_t rows) {
  if (!dtype_ok(dtype) || tokens < 0 || k < 1 || dim < 0 || rows < 0) return NS_ERR_ARG;
  if (k > nsk::MAX_K) return NS_ERR_UNSUPPORTED;
  if (tokens > nsk::MAX_SLOTS / k || rows > nsk::MAX_SLOTS || dim > INT_MAX / 4) return NS_ERR_SHAPE;
  return NS_OK;
}

enum RowOp { DISPATCH, GATHER, COMBINE_GRAD };

// J: rows on their way at once, see the kernels. WARPS of a block.
template <RowOp OP, typename T, int V, int U, int J, int WARPS = nsk::ROW_THREADS / 32>
cudaError_t launch_rows(nsk::RowParams& p, int nsm, cudaStream_t st) {
  using namespace nsk;
  const long long pieces = (p.dim + 32 * V * U - 1) / (32 * V * U);
  if (OP == COMBINE_GRAD) {
    // a token's warps sit in one block; few tokens are shared by more warps
    p.parts = 1;
    while (p.parts < WARPS && p.parts < pieces && p.tokens * p.parts < nsm * 16) p.parts *= 2;
  } else {
    p.parts = static_cast<int>(pieces);
  }
  p.token_warps = p.tokens * p.parts;
  p.clear = p.dim * sizeof(T) <= 512 ? 2 * CLEAR_ROWS : CLEAR_ROWS;
  const long long all = p.token_warps + (OP == GATHER ? 0 : (p.rows + p.clear - 1) / p.clear);
  const long long blocks = (all + WARPS - 1) / WARPS;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * WARPS);
  if constexpr (OP == DISPATCH) return launch_pdl(ns_moe_dispatch_kernel<T, V, U>, grid, block, 0, st, p);
  if constexpr (OP == GATHER) return launch_pdl(ns_moe_gather_kernel<T, V, U, J>, grid, block, 0, st, p);
  if constexpr (OP == COMBINE_GRAD) return launch_pdl(ns_moe_combine_grad_kernel<T, V, U, J, WARPS>, grid, block, 0, st, p);
}

// Words of 16 bytes where rows allow it, else of 4 (16-bit rows of an even
// width), else single elements: 8192 x 6 bf16 rows of 2048, 2046 and 2047 are
// summed in 37.7, 38.7 and 53.0 us (6.3, 6.1 and 4.4 TB/s), backward in 70, 85
// and 100 us. U, the words of a row that a lane takes at once, is what a short
// row has for it, so that more warps fit (28351 x 2 rows of 256 bf16 backward
// 21 us with one word, 34 with the four of long rows; of 512, 31 with two against
// 41; of 70, 13 against 19). J, the rows in flight: 3 for the sums; backward 2, or 1
// of 32 or 64 bytes a lane (3 of those need 163 registers and take 136 us where 1
// takes 124).
template <RowOp OP, typename T>
cudaError_t launch_words(int word, nsk::RowParams& p, int nsm, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  // whether a row has more than u words of v elements for a lane
  const auto longer = [&](int v, int u) { return p.dim > 32LL * v * u; };
  if constexpr (OP == GATHER) {
    // few slots: more of each row at a time instead of more rows (16384 tokens of 1, 2 and 4 rows of 2048 bf16
    // in 24.6, 34.1 and 52.7 us against 34.5, 39.8 and 57.0; of 2047 columns, 1 and 2 rows in 37 and 44 against
    // 54 and 60, but three fp32 rows of 1001 in 10.0 against 9.5), where the row reaches the last of a lane's
    // words (8192 tokens of 2 rows of 512 take 5.9 us against 5.3, of 255 columns 5.3 against 4.5) and, for the
    // wide words, where the tokens fill the GPU (1216 tokens of 4 rows of 2048 take 4.9 us against 4.6, 2432
    // tokens 10.3 against 11.6)
    if (word == 16) {
      if (p.k <= 4 && longer(V, 3) && p.tokens >= 16 * nsm) return launch_rows<OP, T, V, 4, 1>(p, nsm, st);
      if (longer(V, 1)) return launch_rows<OP, T, V, 2, 3>(p, nsm, st);
      return launch_rows<OP, T, V, 1, 3>(p, nsm, st);
    }
    const auto narrow = [&](auto v) {
      constexpr int W = decltype(v)::value;
      if (p.k <= 2 && longer(W, 15)) return launch_rows<OP, T, W, 16, 2>(p, nsm, st);
      if (longer(W, 4)) return launch_rows<OP, T, W, 8, 3>(p, nsm, st);
      return launch_rows<OP, T, W, 4, 3>(p, nsm, st);
    };
    if constexpr (sizeof(T) == 2)
      if (word == 4) return narrow(std::integral_constant<int, 2>());
    return narrow(std::integral_constant<int, 1>());
  } else if constexpr (OP == COMBINE_GRAD) {
    // few tokens of long rows: more than the 4 warps of a block for each (13 x 8 rows of 3761 fp16 take 6.1 us
    // against 12.3, 7 x 8 of 6399 fp32 9.2 against 19; blocks this large cost 8 % where the tokens are many)
    const bool few = p.tokens < 4 * nsm;
    if (word == 16) {
      if (few && longer(V, 16)) return launch_rows<OP, T, V, 4, 1, nsk::MANY_WARPS>(p, nsm, st);
      if (longer(V, 2)) return launch_rows<OP, T, V, 4, 1>(p, nsm, st);
      if (longer(V, 1)) return launch_rows<OP, T, V, 2, 1>(p, nsm, st);
      return launch_rows<OP, T, V, 1, 2>(p, nsm, st);
    }
    const auto narrow = [&](auto v) {
      constexpr int W = decltype(v)::value;
      if (few && longer(W, 32)) return launch_rows<OP, T, W, 8, 2, nsk::MANY_WARPS>(p, nsm, st);
      // one or two slots leave registers for more of the row: 6000 x 1 rows of 5527 bf16 in 48 us against 70, x 2 in 74
      // against 91; of 5526 38 against 47, x 2 in 60 against 63
      if (p.k <= 2 && longer(W, 15)) return launch_rows<OP, T, W, 16, 1>(p, nsm, st);
      if (longer(W, 4)) return launch_rows<OP, T, W, 8, 2>(p, nsm, st);
      if (longer(W, 2)) return launch_rows<OP, T, W, 4, 2>(p, nsm, st);
      return launch_rows<OP, T, W, 2, 2>(p, nsm, st);
    };
    if constexpr (sizeof(T) == 2)
      if (word == 4) return narrow(std::integral_constant<int, 2>());
    return narrow(std::integral_constant<int, 1>());
  } else {
    if (word == 16) return launch_rows<OP, T, V, 4, 1>(p, nsm, st);
    if constexpr (sizeof(T) == 2)
      if (word == 4) return launch_rows<OP, T, 2, 8, 1>(p, nsm, st);
    return launch_rows<OP, T, 1, 8, 1>(p, nsm, st);
  }
}

template <RowOp OP>
cudaError_t launch_type(int dtype, int word, nsk::RowParams& p, int nsm, cudaStream_t st) {
  if (dtype == NS_DT_BF16) return launch_words<OP, __nv_bfloat16>(word, p, nsm, st);
  if (dtype == NS_DT_FP16) return launch_words<OP, __half>(word, p, nsm, st);
  return launch_words<OP, float>(word, p, nsm, st);
}

template <RowOp OP>
int run_rows(int dtype, nsk::RowParams& p, int word, void* stream) {
  int dev, nsm;
  const int rc = device_setup(&dev, &p.status, &nsm);
  if (rc != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = counted(K_MOE, st, [&] { return launch_type<OP>(dtype, word, p, nsm, st); });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

}  // namespace

extern "C" {

int ns_moe_rows(int64_t tokens, int k, int experts, int align, int64_t capacity, int64_t* rows_out) {
  if (!rows_out || align < 1 || capacity < 0) return NS_ERR_ARG;
  const int rc = sort_args(tokens, k, experts);
  if (rc != NS_OK) return rc;
  const int64_t slots = tokens * k;
  int64_t rows = slots + std::min<int64_t>(experts, slots) * (align - 1);
  if (capacity > 0) {
    const int64_t cap = std::min(capacity, slots);
    rows = std::min(rows, experts * ((cap + align - 1) / align * align));
  }
  if (rows > nsk::MAX_SLOTS) return NS_ERR_SHAPE;
  *rows_out = rows;
  return NS_OK;
}

int ns_moe_sort_workspace_bytes(int64_t tokens, int k, int experts, uint64_t* bytes) {
  if (!bytes) return NS_ERR_ARG;
  const int rc = sort_args(tokens, k, experts);
  if (rc != NS_OK) return rc;
  int chunk, blocks;
  sort_split(tokens * k, &chunk, &blocks);
  *bytes = blocks > 1 ? static_cast<uint64_t>(blocks) * nsk::count_stride(experts) * sizeof(int) : 0;
  return NS_OK;
}

int ns_moe_sort(const void* expert_ids, int id_bytes, int64_t tokens, int k, int experts, int align,
                int64_t capacity, int64_t rows, int32_t* row_of_slot, int32_t* slot_of_row, int32_t* counts,
                int32_t* offsets, void* workspace, uint64_t workspace_bytes, void* stream) {
  int64_t need_rows = 0;
  int rc = ns_moe_rows(tokens, k, experts, align, capacity, &need_rows);
  if (rc != NS_OK) return rc;
  if (id_bytes != 4 && id_bytes != 8) return NS_ERR_ARG;
  if (rows < need_rows || rows > nsk::MAX_SLOTS) return NS_ERR_SHAPE;
  if (!counts || !offsets || (tokens > 0 && (!expert_ids || !row_of_slot)) || (rows > 0 && !slot_of_row))
    return NS_ERR_ARG;
  if (!element_aligned(expert_ids, id_bytes) || !all_aligned(4, {row_of_slot, slot_of_row, counts, offsets}))
    return NS_ERR_ARG;
  nsk::SortParams p = {};
  p.ids = expert_ids;
  p.id_bytes = id_bytes;
  p.slots = static_cast<int>(tokens * k);
  p.experts = experts;
  p.align = align;
  p.capacity = capacity > 0 && capacity < INT_MAX ? static_cast<int>(capacity) : INT_MAX;
  p.rows = static_cast<int>(rows);
  sort_split(p.slots, &p.chunk, &p.blocks);
  const uint64_t need = p.blocks > 1 ? static_cast<uint64_t>(p.blocks) * nsk::count_stride(experts) * sizeof(int) : 0;
  if (need && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return NS_ERR_WORKSPACE;
  p.row_of_slot = row_of_slot;
  p.slot_of_row = slot_of_row;
  p.counts = counts;
  p.offsets = offsets;
  p.block_counts = static_cast<int*>(workspace);
  int dev, nsm;
  rc = device_setup(&dev, &p.status, &nsm);
  if (rc != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.blocks > 1) {
    const cudaError_t e = counted(K_MOE, st, [&] {
      return nsk::launch_pdl(nsk::ns_moe_count_kernel, dim3(p.blocks), dim3(nsk::SORT_THREADS),
                             experts * sizeof(int), st, p);
    });
    if (e != cudaSuccess) return NS_ERR_CUDA;
  }
  const size_t smem = place_smem(experts);
  void (*const place)(nsk::SortParams) = p.chunk <= nsk::SORT_THREADS * nsk::SORT_HELD ? nsk::ns_moe_place_kernel<true>
                                                                                      : nsk::ns_moe_place_kernel<false>;
  // the same limit in every call: a smaller one that another thread sets before this launch would refuse it
  if (smem > nsk::SMEM_WITHOUT_ASKING &&
      cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(place_smem(nsk::MAX_EXPERTS))) != cudaSuccess)
    return NS_ERR_CUDA;
  const cudaError_t e = counted(K_MOE, st, [&] {
    return nsk::launch_pdl(place, dim3(p.blocks), dim3(nsk::SORT_THREADS), smem, st, p);
  });
  return e == cudaSuccess ? NS_OK : NS_ERR_CUDA;
}

int ns_moe_dispatch(const void* x, int64_t x_stride, int dtype, int64_t tokens, int k, int64_t dim,
                    const int32_t* row_of_slot, const int32_t* slot_of_row, int64_t rows, void* out,
                    int64_t out_stride, void* stream) {
  const int rc = row_args(dtype, tokens, k, dim, rows);
  if (rc != NS_OK) return rc;
  if (x_stride < dim || out_stride < dim) return NS_ERR_SHAPE;
  if (rows == 0 || dim == 0) return NS_OK;
  if (!out || !slot_of_row || (tokens > 0 && (!x || !row_of_slot))) return NS_ERR_ARG;
  if (!all_aligned(elem_bytes(dtype), {x, out}) || !all_aligned(4, {row_of_slot, slot_of_row})) return NS_ERR_ARG;
  nsk::RowParams p = {};
  p.src = x;
  p.src_ld = x_stride;
  p.dst = out;
  p.dst_ld = out_stride;
  p.row_of_slot = row_of_slot;
  p.slot_of_row = slot_of_row;
  p.tokens = tokens;
  p.rows = rows;
  p.dim = dim;
  p.k = k;
  const int b = elem_bytes(dtype);
  return run_rows<DISPATCH>(dtype, p, common_word(b, dim, {{x, x_stride}, {out, out_stride}}), stream);
}

int ns_moe_combine(const void* expert_rows, int64_t rows_stride, int dtype, int64_t tokens, int k, int64_t dim,
                   const int32_t* row_of_slot, const float* weights, int64_t rows, void* y, int64_t y_stride,
                   void* stream) {
  const int rc = row_args(dtype, tokens, k, dim, rows);
  if (rc != NS_OK) return rc;
  if (rows_stride < dim || y_stride < dim) return NS_ERR_SHAPE;
  if (tokens == 0 || dim == 0) return NS_OK;
  if (!y || !row_of_slot || (rows > 0 && !expert_rows)) return NS_ERR_ARG;
  if (!all_aligned(elem_bytes(dtype), {expert_rows, y}) || !all_aligned(4, {row_of_slot, weights})) return NS_ERR_ARG;
  nsk::RowParams p = {};
  p.src = expert_rows;
  p.src_ld = rows_stride;
  p.dst = y;
  p.dst_ld = y_stride;
  p.row_of_slot = row_of_slot;
  p.weights = weights;
  p.tokens = tokens;
  p.rows = rows;
  p.dim = dim;
  p.k = k;
  const int b = elem_bytes(dtype);
  return run_rows<GATHER>(dtype, p, common_word(b, dim, {{expert_rows, rows_stride}, {y, y_stride}}), stream);
}

int ns_moe_dispatch_grad(const void* grad_rows, int64_t rows_stride, int dtype, int64_t tokens, int k, int64_t dim,
                         const int32_t* row_of_slot, int64_t rows, void* grad_x, int64_t grad_x_stride,
                         void* stream) {
  return ns_moe_combine(grad_rows, rows_stride, dtype, tokens, k, dim, row_of_slot, nullptr, rows, grad_x,
                        grad_x_stride, stream);
}

int ns_moe_combine_grad(const void* grad_y, int64_t grad_y_stride, const void* expert_rows, int64_t rows_stride,
                        int dtype, int64_t tokens, int k, int64_t dim, const int32_t* row_of_slot,
                        const int32_t* slot_of_row, const float* weights, int64_t rows, void* grad_rows,
                        int64_t grad_rows_stride, float* grad_weights, void* stream) {
  const int rc = row_args(dtype, tokens, k, dim, rows);
  if (rc != NS_OK) return rc;
  if (grad_y_stride < dim || rows_stride < dim || grad_rows_stride < dim) return NS_ERR_SHAPE;
  if (tokens == 0 && rows == 0) return NS_OK;
  if (tokens > 0 && (!row_of_slot || !weights || !grad_weights || (dim > 0 && !grad_y))) return NS_ERR_ARG;
  if (rows > 0 && (!slot_of_row || (dim > 0 && (!expert_rows || !grad_rows)))) return NS_ERR_ARG;
  if (!all_aligned(elem_bytes(dtype), {grad_y, expert_rows, grad_rows}) ||
      !all_aligned(4, {row_of_slot, slot_of_row, weights, grad_weights}))
    return NS_ERR_ARG;
  nsk::RowParams p = {};
  p.src = grad_y;
  p.src_ld = grad_y_stride;
  p.rows_in = expert_rows;
  p.rows_ld = rows_stride;
  p.dst = grad_rows;
  p.dst_ld = grad_rows_stride;
  p.row_of_slot = row_of_slot;
  p.slot_of_row = slot_of_row;
  p.weights = weights;
  p.grad_weights = grad_weights;
  p.tokens = tokens;
  p.rows = rows;
  p.dim = dim;
  p.k = k;
  const int b = elem_bytes(dtype);
  const int word = common_word(b, dim, {{grad_y, grad_y_stride}, {expert_rows, rows_stride}, {grad_rows, grad_rows_stride}});
  return run_rows<COMBINE_GRAD>(dtype, p, word, stream);
}

}  // extern "C"
