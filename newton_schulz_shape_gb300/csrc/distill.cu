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
// or that has no entry left has loss 0, lse 0 (as -0) and a zero gradient, whatever
// its logits hold (NaN included); those of a weight of 0 need not be read.
// The maximum, the sums and the logarithm are in fp32; a gradient value is
// rounded once, when it is stored. The maximum m of the logits is kept as it is
// and subtracted before anything is scaled: exp(s / tau - lse) is
// 2^((s - m) c - l) with c = log2(e) / tau and l the log2 of the sum of
// 2^((s - m) c), and the loss is taken from the largest logit s0 at the entries:
// sum_j p_j (log p_j + (s0 - s_{i_j}) / tau) + P ((m - s0) / tau + l ln 2).
// So finite logits of any size, the type's lowest among them, and rows far from
// zero lose nothing.
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
constexpr int FEW = 4;  // entries a lane of one warp that are held in registers
constexpr int DISTILL_MAX_CLUSTER = 8;  // the portable limit
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
  float tau, inv_tau;
  float* loss;          // null: the log-sum-exp is given
  float* lse;
  int places;           // of the hash table of the teacher's ids
  int cluster;          // blocks that share a token
  int slice_words;      // most words of 16 bytes of a block
  int eager;            // few blocks: a row is read before its weight is known
  unsigned int* status;
};

// Powers below the smallest normal number become 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Maximum and sum of exp2((x - max) c) of what was seen so far.
struct Online {
  float m = -INFINITY, s = 0.0f;
  __device__ __forceinline__ void join(float m2, float s2, float c) {
    const float n = fmaxf(m, m2);
    if (n == -INFINITY) {
      s += s2;  // 0, or NaN
      return;
    }
    s = s * exp2_fast((m - n) * c) + s2 * exp2_fast((m2 - n) * c);
    m = n;
  }
};

// What a logit x is compared with: exp(x / tau - lse) = exp2((x - m) c - l).
struct RowSum {
  float m, l;
  __device__ __forceinline__ float power(float x, float c) const { return exp2_fast(fmaf(x - m, c, -l)); }
};
// A token that the loss leaves out gets lse -0: equal to 0, but no log-sum-exp
// that was computed, so that a gradient with another weight can tell.
constexpr unsigned LEFT_OUT = 0x80000000u;
// From a log-sum-exp that was given; NaN for a token that had none.
__device__ __forceinline__ RowSum given_sum(const DistillParams& p, long long t) {
  const float lse = p.lse[t];
  return {__float_as_uint(lse) == LEFT_OUT ? __uint_as_float(0x7fc00000u) : lse * p.tau, 0.0f};
}

// Places of the hash table of `top` ids: a power of two, four times the ids or
// more, which keeps searches at one or two places, and twice that where it is
// small.
__host__ __device__ inline int table_size(int top) {
  int n = 4;
  while (n < (top <= 128 ? 8 : 4) * top) n *= 2;
  return n;
}

// The teacher's entries of a token, in shared memory.
struct Teacher {
  int* table;  // hash table of the ids; bit 31 marks one that is named more than once
  float* p;    // [top] probability
  float* s;    // [top] the student's logit at the entry
  int* id;     // [top] the entry, -1 if left out
  float* sums; // [3] sum of the probabilities, sum of p (log p - (s - s0) / tau), s0
  int* any;    // whether an entry is left
  __device__ __forceinline__ Teacher(void* at, int top, int places)
      : table(static_cast<int*>(at)), p(reinterpret_cast<float*>(table + places)), s(p + top),
        id(reinterpret_cast<int*>(s + top)), sums(reinterpret_cast<float*>(id + top)), any(reinterpret_cast<int*>(sums + 3)) {}
};
size_t teacher_bytes(int top) { return sizeof(float) * (3 * static_cast<size_t>(top) + table_size(top) + 4); }

constexpr int NO_ID = 0x7fffffff;  // an empty place; ids are below it

// The upper bits of a multiple of the golden ratio, mixed and multiplied once
// more: a single multiple puts ids whose distance is near a Fibonacci number in
// each other's way (64 ids 377 apart: 18 us a call where 5.3 are usual).
__device__ __forceinline__ int table_place(int id, int mask) {
  unsigned h = static_cast<unsigned>(id) * 2654435761u;
  h = (h ^ (h >> 15)) * 2654435761u;
  return static_cast<int>(h >> __clz(mask));
}

// Entry i of all tokens' as it was given.
__device__ __forceinline__ void entry_of(const DistillParams& p, long long i, long long* id, float* z) {
  *id = load_index(p.ids, p.id_bytes, i);
  *z = p.teacher_dtype == NS_DT_FP32   ? static_cast<const float*>(p.teacher)[i]
       : p.teacher_dtype == NS_DT_BF16 ? to_float(static_cast<const __nv_bfloat16*>(p.teacher)[i])
                                       : to_float(static_cast<const __half*>(p.teacher)[i]);
}

// Loads the entries with `n` threads, 4 at a time each so that their latencies
// overlap; whether this thread left any in. In the gradient alone in place of the
// logits, another block may have written its slice by then: of the logits read
// there only those of the block's own slice are used.
template <typename T>
__device__ __forceinline__ bool load_teacher(const DistillParams& p, const Teacher& te, long long t, const T* row,
                                             float weight, int first, int n) {
  constexpr int B = 4;
  bool refused = false, some = false;
  for (int j0 = first; j0 < p.top; j0 += B * n) {
    long long id[B];
    float z[B], s[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int j = j0 + b * n;
      id[b] = -1;
      z[b] = -INFINITY;
      if (j < p.top && weight != 0.0f) entry_of(p, t * p.top + j, &id[b], &z[b]);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      refused |= id[b] >= p.vocab;
      // NaN stays in: it shows in the outputs
      if (id[b] < 0 || id[b] >= p.vocab || z[b] == -INFINITY) id[b] = -1;
      some |= id[b] >= 0;
      s[b] = id[b] >= 0 ? to_float(row[id[b]]) : 0.0f;
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int j = j0 + b * n;
      if (j < p.top) {
        te.id[j] = static_cast<int>(id[b]);
        te.p[j] = id[b] >= 0 ? z[b] : -INFINITY;
        te.s[j] = s[b];
      }
    }
  }
  if (refused) atomicOr(p.status, NS_DEV_BAD_INDEX);
  return some;
}

// Enters the ids in the hash table, by one warp, whose lanes stay together: a
// loop that each leaves by itself, on what its exchange returned, would leave
// them apart to the block's barriers, where the first to arrive counted for
// all.
__device__ __forceinline__ void mark_repeated(const Teacher& te, int top, int mask, int lane) {
  for (int i = lane; i <= mask / 4; i += 32) reinterpret_cast<int4*>(te.table)[i] = make_int4(NO_ID, NO_ID, NO_ID, NO_ID);
  __syncwarp();
  for (int j0 = 0; j0 < top; j0 += 32) {
    const int id = j0 + lane < top ? te.id[j0 + lane] : -1;
    int h = table_place(id, mask);
    bool open = id >= 0;
    while (__any_sync(0xffffffffu, open)) {  // ends: most places stay empty
      if (open) {
        const int old = atomicCAS(&te.table[h], NO_ID, id);
        const bool again = old != NO_ID && (old & 0x7fffffff) == id;
        if (again) atomicOr(&te.table[h], 0x80000000);
        open = old != NO_ID && !again;
        h = (h + 1) & mask;
      }
      __syncwarp();
    }
  }
  __syncwarp();
}

// What the student's logits at the entries are measured from: the largest of
// all lanes' s0, or 0 where none is finite.
__device__ __forceinline__ float origin(float s0) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(s0));
  return m > -INFINITY ? m : 0.0f;
}

// Probabilities and their sums, by one warp; visible to the block after its
// next barrier.
__device__ __forceinline__ void teacher_probabilities(const DistillParams& p, const Teacher& te, long long t, int lane) {
  // log-sum-exp of the entries left, relative to their maximum so that values
  // near the type's lowest stay finite, unless the teacher's own is given
  float z0 = 0.0f, zlog;
  if (p.teacher_lse) {
    zlog = p.teacher_lse[t];
  } else {
    z0 = -INFINITY;
    for (int j = lane; j < p.top; j += 32) z0 = fmaxf(z0, te.p[j]);
    z0 = warp_max(z0);
    float sum = 0.0f;
    for (int j = lane; j < p.top; j += 32) sum += te.id[j] >= 0 ? expf((te.p[j] - z0) * p.inv_tau) : 0.0f;
    zlog = logf(warp_sum(sum));
  }
  float mass = 0.0f, part = 0.0f, s0 = -INFINITY;
  for (int j = lane; j < p.top; j += 32) {
    const float logp = (te.p[j] - z0) * p.inv_tau - zlog;
    const float pr = te.id[j] >= 0 ? expf(logp) : 0.0f;
    if (pr != 0.0f) {
      part += pr * logp;
      s0 = fmaxf(s0, te.s[j]);
    }
    mass += pr;
    te.p[j] = pr;
  }
  s0 = origin(s0);
  float apart = 0.0f;
  for (int j = lane; j < p.top; j += 32)
    if (te.p[j] != 0.0f) apart += te.p[j] * (s0 - te.s[j]);
  mass = warp_sum(mass);
  part = warp_sum(fmaf(apart, p.inv_tau, part));
  if (lane == 0) {
    te.sums[0] = mass;
    te.sums[1] = part;
    te.sums[2] = s0;
  }
}

// Both for up to 4 entries a lane, held in registers: the student's logits are
// on their way while the probabilities are computed. Whether an entry is left.
template <typename T>
__device__ __forceinline__ bool few_entries(const DistillParams& p, const Teacher& te, long long t, const T* row,
                                            float weight, int lane) {
  long long id[FEW];
  float z[FEW], s[FEW], pr[FEW];
  const float given = p.teacher_lse ? p.teacher_lse[t] : 0.0f;
#pragma unroll
  for (int b = 0; b < FEW; ++b) {
    const int j = lane + 32 * b;
    id[b] = -1;
    z[b] = -INFINITY;
    if (j < p.top) entry_of(p, t * p.top + j, &id[b], &z[b]);  // whatever the weight: it is on its way too
  }
  float z0 = -INFINITY;
  bool refused = false;
#pragma unroll
  for (int b = 0; b < FEW; ++b) {
    if (weight == 0.0f) id[b] = -1;
    refused |= id[b] >= p.vocab;
    if (id[b] < 0 || id[b] >= p.vocab || z[b] == -INFINITY) id[b] = -1;
    s[b] = id[b] >= 0 ? to_float(row[id[b]]) : 0.0f;
    if (id[b] >= 0) z0 = fmaxf(z0, z[b]);
  }
  if (refused) atomicOr(p.status, NS_DEV_BAD_INDEX);
  const bool any = __any_sync(0xffffffffu, id[0] >= 0 || id[1] >= 0 || id[2] >= 0 || id[3] >= 0);
  if (!any) return false;
  float sum = 0.0f;
  z0 = p.teacher_lse ? 0.0f : warp_max(z0);
#pragma unroll
  for (int b = 0; b < FEW; ++b) {
    z[b] = (z[b] - z0) * p.inv_tau - given;
    pr[b] = id[b] >= 0 ? expf(z[b]) : 0.0f;
    sum += pr[b];
  }
  sum = warp_sum(sum);
  const float inv = p.teacher_lse ? 1.0f : 1.0f / sum, zlog = p.teacher_lse ? 0.0f : logf(sum);
  float mass = 0.0f, part = 0.0f, s0 = -INFINITY;
#pragma unroll
  for (int b = 0; b < FEW; ++b) {
    pr[b] *= inv;
    if (pr[b] != 0.0f) s0 = fmaxf(s0, s[b]);
  }
  s0 = origin(s0);
#pragma unroll
  for (int b = 0; b < FEW; ++b) {
    const int j = lane + 32 * b;
    if (pr[b] != 0.0f) part += pr[b] * fmaf(s0 - s[b], p.inv_tau, z[b] - zlog);
    mass += pr[b];
    if (j < p.top) {
      te.id[j] = static_cast<int>(id[b]);
      te.p[j] = pr[b];
      te.s[j] = s[b];
    }
  }
  mass = warp_sum(mass);
  part = warp_sum(part);
  if (lane == 0) {
    te.sums[0] = mass;
    te.sums[1] = part;
    te.sums[2] = s0;
  }
  return true;
}

// The loss of a token and its log-sum-exp.
__device__ __forceinline__ void write_loss(const DistillParams& p, const Teacher& te, long long t, float weight,
                                           const RowSum& r) {
  const float log_sum = r.l * LN2;
  p.loss[t] = weight * (te.sums[1] + te.sums[0] * fmaf(r.m - te.sums[2], p.inv_tau, log_sum));
  p.lse[t] = fmaf(r.m, p.inv_tau, log_sum) + 0.0f;  // never -0
}

// The elements of a row that a block writes: its words, and for one block those
// before and after all words.
struct Slice {
  long long first, last;     // this block's words
  long long body, body_end;  // all blocks' words
  bool edges;
  __device__ __forceinline__ bool has(long long v) const {
    return (v >= first && v < last) || (edges && (v < body || v >= body_end));
  }
};

// Gradient of the teacher's entries in the slice, each with every probability
// that names it; once the rest of the slice is written.
template <typename T>
__device__ __forceinline__ void write_entries(const DistillParams& p, const Teacher& te, const Slice& slice, T* grad,
                                              float c, const RowSum& r, float scale, int start, int n) {
  const int mask = p.places - 1;
  for (int j = start; j < p.top; j += n) {
    const int id = te.id[j];
    if (id < 0 || !slice.has(id)) continue;
    int h = table_place(id, mask);
    for (int i = 0; i < mask && (te.table[h] & 0x7fffffff) != id; ++i) h = (h + 1) & mask;
    float sum = te.p[j];
    if (te.table[h] < 0) {
      sum = 0.0f;
      for (int i = 0; i < p.top; ++i) sum += te.id[i] == id ? te.p[i] : 0.0f;
    }
    grad[id] = from_float<T>(scale * te.sums[0] * r.power(te.s[j], c) - scale * sum);
  }
}

// The maximum and sum of a warp's threads, in all of them.
__device__ __forceinline__ Online join_warp(Online o, float c) {
  // one rescaling to the warp's maximum, then plain sums
  const float m = warp_max(o.m);
  o.s = m == -INFINITY ? o.s : o.s * exp2_fast((o.m - m) * c);
  o.m = m;
  o.s = warp_sum(o.s);
  return o;
}

// The sum over all parts of a token, in every lane.
template <int WARPS>
__device__ __forceinline__ RowSum join_parts(const float2* parts, int C, int lane, float c) {
  Online o;
  for (int i = lane; i < C * WARPS; i += 32) o.join(parts[i].x, parts[i].y, c);
  o = join_warp(o, c);
  return {o.m, log2f(o.s)};
}

// A cluster of blocks takes one token. NT threads of a block copy its logits to
// shared memory, each the words that it will use itself, and use them twice
// there, for the log-sum-exp and for the gradient, so that each is read once;
// one more warp sees to the teacher's entries meanwhile. Every warp writes its
// maximum and sum to all blocks of the cluster through distributed shared
// memory, so that one barrier joins them. The copies of a block are all in
// flight at once, and the blocks that share an SM overlap their phases: with
// slices of 64 KB there are three of them.
// Bound by memory: 4096 rows of 131072 bf16, loss and gradient, 342 us, 6.3 TB/s
// (0.94 of the measured copy); the loss alone 198 us, 5.4 TB/s, bound by its
// instructions. Two passes of one block a row took 564 us (the
// second read came from L2, but the phases of a row did not overlap), slices
// kept in registers 453 us (two blocks an SM at 56 registers). 8 such rows take
// 5.4 us, 2.5 of them the launch: 64 blocks, whose chain of loads is a token's
// weight, its entries' ids and the logits at those.
template <typename T, int NT>
__global__ void __launch_bounds__(NT + 32) ns_distill_kernel(const __grid_constant__ DistillParams p) {
  constexpr int V = 16 / sizeof(T), WARPS = NT / 32, B = 4;  // B words at a time
  extern __shared__ uint4 slice_smem[];
  const Teacher te(slice_smem + p.slice_words, p.top, p.places);
  __shared__ float2 parts[DISTILL_MAX_CLUSTER * WARPS];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.cluster, rank = C > 1 ? static_cast<int>(nsptx::cluster_ctarank()) : 0;
  const bool joins = C > 1 && p.loss;  // blocks that write each other's shared memory: all have to run by then
  if (joins) nsptx::cluster_arrive_relaxed();
  const long long t = blockIdx.x / C;
  const T* row = static_cast<const T*>(p.logits) + t * p.logits_ld;
  T* grad = static_cast<T*>(p.grad) + t * p.grad_ld;
  const float weight = p.weights ? p.weights[t] : 1.0f;
  const float c = p.inv_tau * LOG2E;  // logits to powers of two
  const int vocab = static_cast<int>(p.vocab);
  const int head = static_cast<int>(head_of(row, p.vocab)), words = (vocab - head) / V, tail = head + words * V;
  const int per = (words + C - 1) / C, w0 = min(words, rank * per), n = min(words, w0 + per) - w0;
  const int edge = tid < head ? tid : tail + tid - head;  // the elements around the words, rank 0's
  const bool has_edge = rank == 0 && edge < vocab && (tid < head || edge >= tail);

  if (warp == WARPS) {
    bool any;
    if (p.top <= 32 * FEW) {
      any = few_entries(p, te, t, row, weight, lane);
    } else {
      any = __any_sync(0xffffffffu, load_teacher(p, te, t, row, weight, lane, 32));
      __syncwarp();
      if (any) teacher_probabilities(p, te, t, lane);
    }
    if (lane == 0) *te.any = any;
    __syncwarp();
    if (joins) {
      nsptx::cluster_wait();
      nsptx::cluster_sync_all();
    } else {
      __syncthreads();
    }
    if (!any) {
      if (p.loss && rank == 0 && lane == 0) {
        p.loss[t] = 0.0f;
        p.lse[t] = __uint_as_float(LEFT_OUT);
      }
      return;
    }
    RowSum r;
    if (p.loss) {
      r = join_parts<WARPS>(parts, C, lane, c);
      if (rank == 0 && lane == 0) write_loss(p, te, t, weight, r);
    } else {
      r = given_sum(p, t);
    }
    if (!p.grad) return;
    mark_repeated(te, p.top, p.places - 1, lane);
    __syncthreads();  // the plain part of the gradient is written
    const int first = head + w0 * V;
    const Slice slice = {first, first + n * V, head, tail, rank == 0};
    write_entries<T>(p, te, slice, grad, c, r, weight * p.inv_tau, lane, 32);
    return;
  }

  float ex = -INFINITY;
  const T* body = row + head + static_cast<long long>(w0) * V;
  uint4* mine = slice_smem + tid;
  const int rounds = (n + NT - 1) / NT, quarter = (rounds + 4 * B - 1) / (4 * B) * B;  // words a thread; in a copy group
  if (weight != 0.0f || p.eager) {
    for (int g = 0; g < 4; ++g) {
      for (int u = g * quarter; u < min(rounds, (g + 1) * quarter); ++u)
        if (u * NT + tid < n) nsptx::cp_async16(mine + u * NT, body + (u * NT + tid) * V);
      nsptx::cp_async_commit();
    }
    if (has_edge) ex = to_float(row[edge]);
  }
  // B rounds of words from round u on; `whole`: all of them are inside the slice
  const int full = n / NT;
  auto words_at = [&](int u, Vec<T, V>(&x)[B], auto whole) {
#pragma unroll
    for (int i = 0; i < B; ++i)
      x[i] = decltype(whole)::value || (u + i) * NT + tid < n ? *reinterpret_cast<const Vec<T, V>*>(mine + (u + i) * NT)
                                                              : fill_vec<T, V>(-INFINITY);
  };
  const float2 c2 = make_float2(c, c);
  RowSum r;
  if (p.loss) {
    Online o;
    if (weight != 0.0f) {
      o.m = ex;
      o.s = ex == -INFINITY ? 0.0f : exp2_fast(ex - ex);  // 1, or NaN
      for (int g = 0; g < 4; ++g) {
        if (g == 0) nsptx::cp_async_wait<3>();
        if (g == 1) nsptx::cp_async_wait<2>();
        if (g == 2) nsptx::cp_async_wait<1>();
        if (g == 3) nsptx::cp_async_wait<0>();
        auto take = [&](int u, auto whole) {
          Vec<T, V> x[B];
          words_at(u, x, whole);
          const float m = max_of(max_vec(max_vec(x[0], x[1]), max_vec(x[2], x[3])));
          const float top = fmaxf(o.m, m), base = top == -INFINITY ? 0.0f : top;
          const float2 b2 = make_float2(-base, -base);
          float2 sum = make_float2(o.s * exp2_fast((o.m - base) * c), 0.0f);
#pragma unroll
          for (int i = 0; i < B; ++i)
#pragma unroll
            for (int k = 0; k < V; k += 2) {
              const float2 a = mul2(add2(make_float2(get(x[i], k), get(x[i], k + 1)), b2), c2);
              sum = add2(sum, make_float2(exp2_fast(a.x), exp2_fast(a.y)));
            }
          o.m = top;
          o.s = sum.x + sum.y;
        };
        const int end = min(rounds, (g + 1) * quarter);
        int u = g * quarter;
        for (; u + B <= min(end, full); u += B) take(u, std::true_type());
        for (; u < end; u += B) take(u, std::false_type());
      }
    } else {
      nsptx::cp_async_wait<0>();  // a row that was read before its weight was known
    }
    o = join_warp(o, c);
    if (joins) nsptx::cluster_wait();
    if (C == 1) {
      if (lane == 0) parts[warp] = make_float2(o.m, o.s);
    } else if (lane < C) {
      const uint32_t to = nsptx::map_to_rank(&parts[rank * WARPS + warp], lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(o.m), "f"(o.s) : "memory");
    }
    if (joins)
      nsptx::cluster_sync_all();
    else
      __syncthreads();
    r = join_parts<WARPS>(parts, C, lane, c);
  } else {
    nsptx::cp_async_wait<0>();
    __syncthreads();
    r = given_sum(p, t);
  }
  if (!p.grad) return;

  const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(grad)) & 15) == 0;
  T* out = grad + head + static_cast<long long>(w0) * V + tid * V;
  if (!*te.any) {
    // nothing to learn from: zeros, whatever the logits hold
    for (int u = 0; u < rounds; ++u) {
      if (u * NT + tid >= n) break;
      if (same) {
        store_once(out + u * NT * V, zero_vec<T, V>());
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) out[u * NT * V + k] = from_float<T>(0.0f);
      }
    }
    if (has_edge) grad[edge] = from_float<T>(0.0f);
    return;
  }
  const float mass = weight * p.inv_tau * te.sums[0];
  const float2 b2 = make_float2(-r.m, -r.m), l2 = make_float2(-r.l, -r.l), m2 = make_float2(mass, mass);
  auto give = [&](int u, auto whole) {
    Vec<T, V> x[B];
    words_at(u, x, whole);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (!decltype(whole)::value && (u + i) * NT + tid >= n) break;
      float y[V];
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float2 a = fma2(add2(make_float2(get(x[i], k), get(x[i], k + 1)), b2), c2, l2);
        const float2 b = mul2(m2, make_float2(exp2_fast(a.x), exp2_fast(a.y)));
        y[k] = b.x;
        y[k + 1] = b.y;
      }
      if (same) {
        store_once(out + (u + i) * NT * V, pack<T, V>(y));
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) out[(u + i) * NT * V + k] = from_float<T>(y[k]);
      }
    }
  };
  int u = 0;
  for (; u + B <= full; u += B) give(u, std::true_type());
  for (; u < rounds; u += B) give(u, std::false_type());
  if (has_edge) grad[edge] = from_float<T>(mass * r.power(ex, c));
  __syncwarp();  // lanes leave the last round of words one by one
  __syncthreads();
}

// Rows too long for the shared memory of a cluster: one block takes one token in
// two passes over its logits.
template <typename T>
__global__ void __launch_bounds__(DISTILL_THREADS) ns_distill_long_kernel(const __grid_constant__ DistillParams p) {
  constexpr int V = 16 / sizeof(T);
  extern __shared__ uint4 slice_smem[];
  const Teacher te(slice_smem, p.top, p.places);
  __shared__ float2 parts[DISTILL_WARPS];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const long long t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(p.logits) + t * p.logits_ld;
  T* grad = static_cast<T*>(p.grad) + t * p.grad_ld;
  const float weight = p.weights ? p.weights[t] : 1.0f;
  const float c = p.inv_tau * LOG2E;
  if (!__syncthreads_or(load_teacher(p, te, t, row, weight, tid, DISTILL_THREADS))) {
    if (p.loss && tid == 0) {
      p.loss[t] = 0.0f;
      p.lse[t] = __uint_as_float(LEFT_OUT);
    }
    if (p.grad) {
      const long long head = head_of(grad, p.vocab), words = (p.vocab - head) / V;
      for (long long i = tid; i < words; i += DISTILL_THREADS) store_once(grad + head + i * V, zero_vec<T, V>());
      for (long long i = tid; i < p.vocab - words * V; i += DISTILL_THREADS)
        grad[i < head ? i : words * V + i] = from_float<T>(0.0f);
    }
    return;
  }
  if (warp == 0) {
    teacher_probabilities(p, te, t, lane);
    mark_repeated(te, p.top, p.places - 1, lane);
  }

  const long long head = head_of(row, p.vocab), words = (p.vocab - head) / V, edges = p.vocab - words * V;
  RowSum r;
  if (p.loss) {
    Online o;
    for (long long i = tid; i < words; i += DISTILL_THREADS) {
      const Vec<T, V> x = load_vec<T, V>(row + head + i * V);
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) m = fmaxf(m, get(x, k));
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int k = 0; k < V; ++k) s += exp2_fast((get(x, k) - base) * c);
      o.join(m, s, c);
    }
    for (long long i = tid; i < edges; i += DISTILL_THREADS) {
      const float v = to_float(row[i < head ? i : words * V + i]);
      o.join(v, v == -INFINITY ? 0.0f : exp2_fast(v - v), c);
    }
    o = join_warp(o, c);
    if (lane == 0) parts[warp] = make_float2(o.m, o.s);
    __syncthreads();
    r = join_parts<DISTILL_WARPS>(parts, 1, lane, c);
    if (tid == 0) write_loss(p, te, t, weight, r);
  } else {
    r = given_sum(p, t);
    __syncthreads();
  }
  if (!p.grad) return;

  const float scale = weight * p.inv_tau, mass = scale * te.sums[0];
  if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(grad)) & 15) == 0) {
    for (long long i = tid; i < words; i += DISTILL_THREADS) {
      const Vec<T, V> x = load_vec<T, V>(row + head + i * V);
      float y[V];
#pragma unroll
      for (int k = 0; k < V; ++k) y[k] = mass * r.power(get(x, k), c);
      store_vec<T, V>(grad + head + i * V, pack<T, V>(y));
    }
    for (long long i = tid; i < edges; i += DISTILL_THREADS) {
      const long long v = i < head ? i : words * V + i;
      grad[v] = from_float<T>(mass * r.power(to_float(row[v]), c));
    }
  } else {
    for (long long v = tid; v < p.vocab; v += DISTILL_THREADS)
      grad[v] = from_float<T>(mass * r.power(to_float(row[v]), c));
  }
  __syncthreads();
  const Slice slice = {0, p.vocab, 0, p.vocab, false};
  write_entries<T>(p, te, slice, grad, c, r, scale, tid, DISTILL_THREADS);
}

constexpr int DISTILL_MAX_SMEM = 200 * 1024;

template <typename T, int NT>
cudaError_t launch_slices(const DistillParams& p, long long tokens, size_t smem, cudaStream_t st) {
  if (smem > SMEM_WITHOUT_ASKING) {
    const cudaError_t e = cudaFuncSetAttribute(ns_distill_kernel<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               DISTILL_MAX_SMEM);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl_cluster(ns_distill_kernel<T, NT>, dim3(static_cast<unsigned>(tokens * p.cluster)), dim3(NT + 32),
                            smem, p.cluster, st, p);
}

template <typename T>
cudaError_t launch_distill(DistillParams& p, long long tokens, int nsm, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const long long words = (p.vocab + V - 1) / V;
  // slices of 64 KB; of 32 KB where the blocks of a row need not meet (the gradient alone: 88 us against 91
  // for 1531 rows of 50001 fp32)
  const int most = p.loss ? 4096 : 2048, nt = words <= 64 * 8 ? 64 : words <= 128 * 8 || !p.loss ? 128 : 256;
  // (64 threads for the shortest rows: more rows an SM, 967 x 2092 bf16 in 7.1 us against 8.1)
  int C = 1;
  while (C < DISTILL_MAX_CLUSTER && (words + C - 1) / C > most) C *= 2;
  // few rows: split further, down to a word a thread
  while (C < DISTILL_MAX_CLUSTER && tokens * C < nsm && words / C > nt) C *= 2;
  p.cluster = C;
  p.slice_words = static_cast<int>((words + C - 1) / C);
  p.places = table_size(p.top);
  p.eager = tokens * C <= 2 * nsm;
  const size_t smem = 16 * static_cast<size_t>(p.slice_words) + teacher_bytes(p.top);
  if (smem > DISTILL_MAX_SMEM || tokens * C > INT_MAX)
    return launch_pdl(ns_distill_long_kernel<T>, dim3(static_cast<unsigned>(tokens)), dim3(DISTILL_THREADS),
                      teacher_bytes(p.top), st, p);
  if (nt == 64) return launch_slices<T, 64>(p, tokens, smem, st);
  return nt == 128 ? launch_slices<T, 128>(p, tokens, smem, st) : launch_slices<T, 256>(p, tokens, smem, st);
}

}  // namespace
}  // namespace nsk

using namespace nsorch;

namespace {

using nsk::dtype_ok;
using nsk::elem_bytes;
using nsk::element_aligned;

int run_distill(const void* logits, int64_t logits_stride, int dtype, int64_t tokens, int64_t vocab,
                const void* teacher_values, int teacher_dtype, const void* teacher_ids, int id_bytes, int top,
                const float* weights, const float* teacher_lse, float temperature, float* loss, float* lse,
                void* grad_logits, int64_t grad_stride, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype) || (id_bytes != 4 && id_bytes != 8)) return NS_ERR_ARG;
  if (tokens < 0 || vocab < 1 || top < 1 || !(temperature >= 1.0e-30f) || temperature > 1.0e30f) return NS_ERR_ARG;
  if (top > nsk::DISTILL_MAX_TOP) return NS_ERR_UNSUPPORTED;
  if (vocab > INT_MAX || tokens > INT_MAX || logits_stride < vocab || (grad_logits && grad_stride < vocab))
    return NS_ERR_SHAPE;
  if (tokens == 0) return NS_OK;
  if (!logits || !teacher_values || !teacher_ids || !lse) return NS_ERR_ARG;
  if (grad_logits == logits && grad_stride != logits_stride) return NS_ERR_ARG;
  if (!element_aligned(logits, elem_bytes(dtype)) || !element_aligned(grad_logits, elem_bytes(dtype)) ||
      !element_aligned(teacher_values, elem_bytes(teacher_dtype)) || !element_aligned(teacher_ids, id_bytes))
    return NS_ERR_ARG;
  for (const void* p : {static_cast<const void*>(weights), static_cast<const void*>(teacher_lse),
                        static_cast<const void*>(loss), static_cast<const void*>(lse)})
    if (!element_aligned(p, 4)) return NS_ERR_ARG;
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
  p.tau = temperature;
  p.inv_tau = 1.0f / temperature;
  p.loss = loss;
  p.lse = lse;
  int dev, nsm;
  const int rc = device_setup(&dev, &p.status, &nsm);
  if (rc != NS_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = counted(K_DISTILL, st, [&] {
    if (dtype == NS_DT_BF16) return nsk::launch_distill<__nv_bfloat16>(p, tokens, nsm, st);
    if (dtype == NS_DT_FP16) return nsk::launch_distill<__half>(p, tokens, nsm, st);
    return nsk::launch_distill<float>(p, tokens, nsm, st);
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
