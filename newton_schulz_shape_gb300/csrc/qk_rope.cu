// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradient.
//
// For one head x of D values at position pos, with weight g and the rotation
// R over the first `rot_dim` of them:
//   r = (mean(x^2) + eps)^(-1/2),  y = R_pos (x r g)
// and backward, with u = R_pos^T dy and h = u g:
//   dx = r (h - n mean(h n)), n = x r,  dg = sum over tokens and heads of u n.
// The rotation turns pairs (a, b) -> (a c - b s, b c + a s); the pairs are
// (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved.
//
// Every value is read and written once, so large calls are bound by memory:
// 16384 tokens of 32/8 heads of 128 bf16 take 60 us forward (5.7 TB/s) and 89 us
// backward (5.8 TB/s, 0.86 of the measured copy; the rest is the instructions of
// two reductions and a rotation for every 16 bytes). 16 tokens take 2.6 us.
#include <algorithm>
#include <climits>
#include <cstdlib>

#include "elem.cuh"
#include "launch.cuh"
#include "orchestrate.h"
#include "ptx.cuh"
#include "status.h"

namespace nsk {
namespace {

constexpr int QK_THREADS = 128;
constexpr int QK_WARPS = QK_THREADS / 32;
// What is rotated: whole words (or nothing); interleaved pairs that end inside a
// word; pairs (i, i + rot_dim / 2) that are not made of whole words.
enum QkTurn { WHOLE, PARTIAL, SPREAD };
// Blocks that share an SM, by the registers that their angles and sums take.
constexpr int qk_blocks(bool grad, QkTurn mode) { return 5 - (grad ? 1 : 0) - (mode == SPREAD ? 1 : 0); }
constexpr int QK_AHEAD = 3;  // rounds whose words are on their way
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
  // (token, head) strides of x, dy and out in bytes, where they fit
  int token_bytes[3], head_bytes[3];
};

// A pair (token, head) of one side, in token order; steps go by a number of
// pairs split into tokens and heads.
struct Place {
  int t, h;
};
__host__ __device__ __forceinline__ Place place_of(int pair, int heads) {
  const int t = pair / heads;
  return {t, pair - t * heads};
}

struct QkParams {
  QkSide side[2];     // queries, keys
  long long tokens;
  int dim, rot_dim, interleaved, weight_fp32;
  float eps;
  const float* table; // [table_rows][rot_dim]: cosines, then sines
  long long table_rows;
  const void* positions;  // null: the token's index
  int position_bytes;
  int lanes;          // of a head's group
  int chunk;          // rounds of 32 / lanes heads that a warp takes at a time
  int chunks[2];      // of the queries and of the keys
  Place within[2], between[2];  // steps of a warp from round to round: in a chunk, to its next chunk
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

// Sum over the lanes of a group, in all of them. G lanes, a power of two, or
// (G = 0) n, this one the i-th of them.
template <int G>
__device__ __forceinline__ float group_sum(float x, int n, int i) {
  if constexpr (G > 0) {
#pragma unroll
    for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  } else {
    for (int o = 1; o < n; o <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, x, o);
      if (i + o < n) x += y;
    }
    return __shfl_sync(0xffffffffu, x, (threadIdx.x & 31) - i);
  }
}

// A lane holds two words of 16 bytes of every head, a and b. Where the pairs
// (i, i + rot_dim / 2) are rotated, b lies rot_dim / 2 values after a, so that
// both values of each pair are in the lane and the two words share their
// angles; a head then takes dim / V / 2 lanes (8 for 128 bf16 values).
template <typename T>
struct Lane {
  static constexpr int V = 16 / sizeof(T);
  int a, b;            // first values of the words
  bool on_a, on_b;     // inside the head
  bool turn_a, turn_b; // rotated
};

// SPREAD: places of a warp's heads, at most 64 words and 32 heads.
__host__ __device__ constexpr int spread_places(int V) { return 64 * V + 64; }

// Lane i of a head's group. Where the pairs (i, i + rot_dim / 2) are not made of
// whole words the words are taken in order, as they are for interleaved pairs.
template <typename T, QkTurn MODE>
__device__ __forceinline__ Lane<T> lane_of(const QkParams& p, int i) {
  constexpr int V = Lane<T>::V;
  Lane<T> l;
  const int words = p.dim / V, turned = (p.rot_dim + V - 1) / V;
  if (MODE != WHOLE || p.interleaved) {
    const int a = i, b = i + (words + 1) / 2;
    l.on_a = a < (words + 1) / 2;
    l.on_b = l.on_a && b < words;
    l.turn_a = l.on_a && a < turned;
    l.turn_b = l.on_b && b < turned;
    l.a = a * V;
    l.b = b * V;
  } else if (i < turned / 2) {
    l.on_a = l.on_b = l.turn_a = l.turn_b = true;
    l.a = i * V;
    l.b = l.a + p.rot_dim / 2;
  } else {
    const int rest = words - turned, a = i - turned / 2, b = a + (rest + 1) / 2;
    l.on_a = a < (rest + 1) / 2;
    l.on_b = l.on_a && b < rest;
    l.turn_a = l.turn_b = false;
    l.a = (turned + a) * V;
    l.b = (turned + b) * V;
  }
  return l;
}

// The two words as pairs of fp32 values.
template <typename T>
struct Two {
  static constexpr int N = Lane<T>::V / 2;
  float2 a[N], b[N];
};

template <typename T>
__device__ __forceinline__ Two<T> unpack(const uint4* from) {
  constexpr int V = Lane<T>::V;
  const Vec<T, V> a = *reinterpret_cast<const Vec<T, V>*>(from), b = *reinterpret_cast<const Vec<T, V>*>(from + 32);
  Two<T> x;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    x.a[i] = make_float2(get(a, 2 * i), get(a, 2 * i + 1));
    x.b[i] = make_float2(get(b, 2 * i), get(b, 2 * i + 1));
  }
  return x;
}

template <typename T>
__device__ __forceinline__ void store_words(char* a, int to_b, const Lane<T>& l, const Two<T>& y) {
  constexpr int V = Lane<T>::V;
  float fa[V], fb[V];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    fa[2 * i] = y.a[i].x;
    fa[2 * i + 1] = y.a[i].y;
    fb[2 * i] = y.b[i].x;
    fb[2 * i + 1] = y.b[i].y;
  }
  if (l.on_a) store_vec<T, V>(reinterpret_cast<T*>(a), pack<T, V>(fa));
  if (l.on_b) store_vec<T, V>(reinterpret_cast<T*>(a + to_b), pack<T, V>(fb));
}

// Cosines and sines of the lane's V pairs at one table row: the pairs of both
// words, or (interleaved) those of word a and then those of word b.
template <typename T>
struct Angles {
  float2 c[Two<T>::N], s[Two<T>::N];
};

template <typename T, QkTurn MODE>
__device__ __forceinline__ void load_angles(const QkParams& p, const Lane<T>& l, const float* row, Angles<T>& g) {
  constexpr int N = Two<T>::N;
  const int half = p.rot_dim / 2;
  if constexpr (MODE == PARTIAL) {
    // interleaved pairs up to the middle of a word, whose others stay as they are; no row of the table need
    // start at a vector's boundary
    auto some = [&](float2* c, float2* s, int first) {
      float* const cf = reinterpret_cast<float*>(c);
      float* const sf = reinterpret_cast<float*>(s);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (first + i < half) {
          cf[i] = row[first + i];
          sf[i] = row[half + first + i];
        }
      }
    };
    if (l.turn_a) some(g.c, g.s, l.a / 2);
    if (l.turn_b) some(g.c + N / 2, g.s + N / 2, l.b / 2);
    return;
  }
  const int a = p.interleaved ? l.a / 2 : l.a, b = p.interleaved ? l.b / 2 : l.a + N;
  auto load = [&](float2* to, const float* from) {
    if constexpr (N == 4) {
      const float4 f = *reinterpret_cast<const float4*>(from);
      to[0] = make_float2(f.x, f.y);
      to[1] = make_float2(f.z, f.w);
    } else {
      to[0] = *reinterpret_cast<const float2*>(from);
    }
  };
  if (l.turn_a) {
    load(g.c, row + a);
    load(g.s, row + half + a);
  }
  if (l.turn_b) {
    load(g.c + N / 2, row + b);
    load(g.s + N / 2, row + half + b);
  }
}

// Rotates the lane's pairs, forward (sign 1) or back (sign -1).
template <typename T, QkTurn MODE>
__device__ __forceinline__ void turn(const QkParams& p, const Lane<T>& l, const Angles<T>& g, Two<T>& x, float sign) {
  constexpr int N = Two<T>::N;
  if (MODE == PARTIAL || p.interleaved) {
    // pair i of a word: cosine and sine i of the word's N
    auto one = [&](float2& v, float c, float s) { v = make_float2(v.x * c - v.y * s, v.y * c + v.x * s); };
    auto word = [&](float2* v, const float2* c, const float2* s, int pairs) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const int k = i / 2;
        if (i < pairs) one(v[i], c[k].x, sign * s[k].x);
        if (i + 1 < pairs) one(v[i + 1], c[k].y, sign * s[k].y);
      }
    };
    const int half = p.rot_dim / 2;
    if (MODE == PARTIAL) {
      if (l.turn_a) word(x.a, g.c, g.s, half - l.a / 2);
      if (l.turn_b) word(x.b, g.c + N / 2, g.s + N / 2, half - l.b / 2);
    } else {
      if (l.turn_a) word(x.a, g.c, g.s, N);
      if (l.turn_b) word(x.b, g.c + N / 2, g.s + N / 2, N);
    }
  } else if (l.turn_a) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 a = x.a[i], b = x.b[i], minus = mul2(g.s[i], make_float2(-1.0f, -1.0f));
      x.a[i] = fma2(a, g.c[i], mul2(b, sign > 0 ? minus : g.s[i]));
      x.b[i] = fma2(b, g.c[i], mul2(a, sign > 0 ? g.s[i] : minus));
    }
  }
}

// The same for pairs that are not made of whole words. Every value has its own
// angle, with the sine's sign of its place in the pair. The other value of value
// d's pair is the (d + rot_dim / 2)-th modulo rot_dim: the lanes put their words
// in the head's order in `head`, the group's part of shared memory, the first
// value once more behind the last, so that the others of two neighbours lie side
// by side, at even places (all are moved by one where rot_dim / 2 is odd). Read in
// pairs: 16384 tokens of 32/8 heads of 72, all rotated, 159 us backward value by
// value, 125 so.
template <typename T>
struct SpreadAngles {
  float2 ca[Two<T>::N], sa[Two<T>::N], cb[Two<T>::N], sb[Two<T>::N];
};

// The sines with `sign`: 1 forward, -1 back.
template <typename T>
__device__ __forceinline__ void load_spread(const QkParams& p, const Lane<T>& l, const float* row, SpreadAngles<T>& g,
                                            float sign) {
  const int half = p.rot_dim / 2;
  auto word = [&](float2* c, float2* s, int first) {
#pragma unroll
    for (int i = 0; i < Two<T>::N; ++i) {
      const int d = first + 2 * i;
      if (d >= p.rot_dim) continue;
      const int a = d < half ? d : d - half, b = d + 1 < half ? d + 1 : d + 1 - half;
      c[i] = make_float2(row[a], row[b]);
      s[i] = make_float2(d < half ? -sign * row[half + a] : sign * row[half + a],
                         d + 1 < half ? -sign * row[half + b] : sign * row[half + b]);
    }
  };
  word(g.ca, g.sa, l.a);
  word(g.cb, g.sb, l.b);
}

template <typename T>
__device__ __forceinline__ void turn_spread(const QkParams& p, const Lane<T>& l, const SpreadAngles<T>& g, Two<T>& x,
                                            float* head) {
  const int half = p.rot_dim / 2, odd = half & 1;
  auto put = [&](const float2* v, int first, bool on) {
#pragma unroll
    for (int i = 0; i < Two<T>::N; ++i) {
      float* const to = head + odd + first + 2 * i;
      if (!on || first + 2 * i >= p.rot_dim) continue;
      if (odd) {
        to[0] = v[i].x;
        to[1] = v[i].y;
      } else {
        *reinterpret_cast<float2*>(to) = v[i];
      }
    }
  };
  auto get = [&](float2* v, const float2* c, const float2* s, int first, bool on) {
#pragma unroll
    for (int i = 0; i < Two<T>::N; ++i) {
      const int d = first + 2 * i, o = d + half < p.rot_dim ? d + half : d - half;
      if (on && d < p.rot_dim) v[i] = fma2(v[i], c[i], mul2(*reinterpret_cast<const float2*>(head + odd + o), s[i]));
    }
  };
  __syncwarp();
  put(x.a, l.a, l.on_a);
  put(x.b, l.b, l.on_b);
  if (l.on_a && l.a == 0) head[odd + p.rot_dim] = x.a[0].x;
  __syncwarp();
  get(x.a, g.ca, g.sa, l.a, l.on_a);
  get(x.b, g.cb, g.sb, l.b, l.on_b);
}

// The weights of one of the lane's words.
template <typename T>
__device__ __forceinline__ void weights_of(const QkParams& p, const void* w, int first, bool on, float2 (&g)[Two<T>::N]) {
  constexpr int V = Lane<T>::V, N = Two<T>::N;
  if (!w || !on) {
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = make_float2(1.0f, 1.0f);
  } else if (p.weight_fp32) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + first + 2 * i));
      g[i] = make_float2(f.x, f.y);
      g[i + 1] = make_float2(f.z, f.w);
    }
  } else {
    Vec<T, V> x;
    *reinterpret_cast<uint4*>(&x) = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w) + first));
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = make_float2(get(x, 2 * i), get(x, 2 * i + 1));
  }
}

template <typename T>
__device__ __forceinline__ Two<T> lane_weights(const QkParams& p, const QkSide& side, const Lane<T>& l) {
  Two<T> g;
  weights_of<T>(p, side.weight, l.a, l.on_a, g.a);
  weights_of<T>(p, side.weight, l.b, l.on_b, g.b);
  return g;
}

// The heads that a lane's group goes through: p.chunk rounds in a row, then
// those of the warp's next chunk.
struct Walk {
  int t, h, left;
  __device__ __forceinline__ void step(const QkParams& p, int which, int heads) {
    const bool jump = --left == 0;
    if (jump) left = p.chunk;
    t += jump ? p.between[which].t : p.within[which].t;
    h += jump ? p.between[which].h : p.within[which].h;
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  }
};

// The norm, its rotation and (GRAD) its gradient: G (or, 0, p.lanes) lanes hold
// one head, a warp as many consecutive heads a round as fit 32 lanes. The warps
// of a grid that fits the card deal the queries and then the keys among them,
// p.chunk rounds at a time, so that together they walk through memory in order;
// a warp copies the words of its next QK_AHEAD rounds to shared memory while it
// computes one. For the gradient a lane keeps the sums of its columns of dg,
// which a block joins in a fixed order.
template <typename T, int G, bool GRAD, QkTurn MODE>
__global__ void __launch_bounds__(QK_THREADS, qk_blocks(GRAD, MODE)) ns_qk_kernel(const __grid_constant__ QkParams p) {
  constexpr int N = Two<T>::N, STAGES = QK_AHEAD + 1, STAGE = GRAD ? 128 : 64;
  extern __shared__ uint4 ring_smem[];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4* ring = ring_smem + warp * (STAGES * STAGE) + lane;
  const int group_size = G ? G : p.lanes, H = 32 / group_size;
  const int group = lane / group_size, i_lane = lane - group * group_size;
  const bool takes = group < H;  // a lane left over takes no head
  Lane<T> l = lane_of<T, MODE>(p, i_lane);
  if (!takes) l.on_a = l.on_b = l.turn_a = l.turn_b = false;
  // SPREAD: the group's head, of dim + 2 places
  float* head = reinterpret_cast<float*>(ring_smem + QK_WARPS * STAGES * STAGE) + warp * spread_places(Lane<T>::V) +
                min(group, H - 1) * (p.dim + 2);
  const float inv_dim = 1.0f / p.dim;
  const int warps = gridDim.x * QK_WARPS, me = blockIdx.x * QK_WARPS + warp;
  int chunk = me;  // this warp's next, in those of the queries and then of the keys
  for (int which = 0; which < 2; ++which) {
    const QkSide& side = p.side[which];
    const int first = chunk - (which ? p.chunks[0] : 0), todo = p.chunks[which] - first;
    const int mine = todo > 0 ? (todo + warps - 1) / warps : 0, n = mine * p.chunk;
    chunk += mine * warps;
    Two<T> dg;
    if (GRAD) {
#pragma unroll
      for (int i = 0; i < N; ++i) dg.a[i] = dg.b[i] = make_float2(0.0f, 0.0f);
    }
    if (n > 0) {
      // words outside the head are zero for the whole side (the sums of the other side lay in the ring)
      for (int i = 0; i < STAGES * STAGE; i += 64) {
        if (!l.on_a) ring[i] = make_uint4(0, 0, 0, 0);
        if (!l.on_b) ring[i + 32] = make_uint4(0, 0, 0, 0);
      }
      const Two<T> g = lane_weights<T>(p, side, l);
      const Place start = place_of(first * p.chunk * H + min(group, H - 1), side.heads);
      Walk ahead = {start.t, start.h, p.chunk}, at = ahead;  // of the copies, and of the rounds
      // tensor k's address of the lane's first word of a head: two wide multiply-adds
      auto offset = [&](const Walk& w, int k) {
        return static_cast<long long>(w.t) * side.token_bytes[k] + static_cast<long long>(w.h) * side.head_bytes[k];
      };
      const char* const x_base = static_cast<const char*>(side.x) + sizeof(T) * l.a;
      const char* const dy_base = static_cast<const char*>(side.dy) + sizeof(T) * l.a;
      char* const out_base = static_cast<char*>(side.out) + sizeof(T) * l.a;
      const int to_b = static_cast<int>(sizeof(T)) * (l.b - l.a);
      int fill = 0, take = 0;
      auto copy = [&](bool more) {
        if (more && takes && ahead.t < p.tokens) {
          const char* x_at = x_base + offset(ahead, 0);
          if (l.on_a) nsptx::cp_async16(ring + fill, x_at);
          if (l.on_b) nsptx::cp_async16(ring + fill + 32, x_at + to_b);
          if (GRAD) {
            const char* dy_at = dy_base + offset(ahead, 1);
            if (l.on_a) nsptx::cp_async16(ring + fill + 64, dy_at);
            if (l.on_b) nsptx::cp_async16(ring + fill + 96, dy_at + to_b);
          }
        }
        nsptx::cp_async_commit();
        ahead.step(p, which, side.heads);
        fill = fill + STAGE == STAGES * STAGE ? 0 : fill + STAGE;
      };
      for (int r = 0; r < QK_AHEAD; ++r) copy(r < n);
      int angles_of = -1;
      const float* row = nullptr;
      Angles<T> angles;
      SpreadAngles<T> spread;
      for (int r = 0; r < n; ++r) {
        copy(r + QK_AHEAD < n);
        nsptx::cp_async_wait<QK_AHEAD>();
        bool live = takes && at.t < p.tokens;  // of a whole group of lanes; the others' values go nowhere
        Two<T> xf = unpack<T>(ring + take);
        Two<T> u;
        if (GRAD) u = unpack<T>(ring + take + 64);
        take = take + STAGE == STAGES * STAGE ? 0 : take + STAGE;
        if (p.rot_dim && live && at.t != angles_of) {
          row = table_row(p, at.t);
          if (row && MODE == SPREAD) load_spread<T>(p, l, row, spread, GRAD ? -1.0f : 1.0f);
          if (row && MODE != SPREAD) load_angles<T, MODE>(p, l, row, angles);
          angles_of = at.t;
        }
        if (p.rot_dim && !row) live = false;
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          s2 = fma2(xf.a[i], xf.a[i], s2);
          s2 = fma2(xf.b[i], xf.b[i], s2);
        }
        const float r_norm = rsqrtf(fmaf(group_sum<G>(s2.x + s2.y, group_size, i_lane), inv_dim, p.eps));
        const float2 r2 = make_float2(r_norm, r_norm);
        if (!GRAD) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            u.a[i] = mul2(mul2(xf.a[i], r2), g.a[i]);
            u.b[i] = mul2(mul2(xf.b[i], r2), g.b[i]);
          }
          if (MODE == SPREAD)
            turn_spread<T>(p, l, spread, u, head);
          else
            turn<T, MODE>(p, l, angles, u, 1.0f);
        } else {
          if (MODE == SPREAD)
            turn_spread<T>(p, l, spread, u, head);
          else
            turn<T, MODE>(p, l, angles, u, -1.0f);
          // from here on x stands for n = x r: r^2 and r^3 leave fp32's range long before the results do
#pragma unroll
          for (int i = 0; i < N; ++i) {
            xf.a[i] = mul2(xf.a[i], r2);
            xf.b[i] = mul2(xf.b[i], r2);
          }
          if (live) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              dg.a[i] = fma2(u.a[i], xf.a[i], dg.a[i]);
              dg.b[i] = fma2(u.b[i], xf.b[i], dg.b[i]);
            }
          }
          float2 d2 = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            u.a[i] = mul2(u.a[i], g.a[i]);
            u.b[i] = mul2(u.b[i], g.b[i]);
            d2 = fma2(u.a[i], xf.a[i], d2);
            d2 = fma2(u.b[i], xf.b[i], d2);
          }
          const float m = -r_norm * (group_sum<G>(d2.x + d2.y, group_size, i_lane) * inv_dim);
          const float2 m2 = make_float2(m, m);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            u.a[i] = fma2(u.a[i], r2, mul2(xf.a[i], m2));
            u.b[i] = fma2(u.b[i], r2, mul2(xf.b[i], m2));
          }
        }
        if (live) store_words<T>(out_base + offset(at, 2), to_b, l, u);
        at.step(p, which, side.heads);
      }
      nsptx::cp_async_wait<0>();
    }
    if (GRAD && p.partial) {
      float* joined = reinterpret_cast<float*>(ring_smem);  // [warps][H][dim]; the rings are done with
      __syncthreads();
      if (group < H) {
        float* mine = joined + (warp * H + group) * p.dim;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (l.on_a) *reinterpret_cast<float2*>(mine + l.a + 2 * i) = dg.a[i];
          if (l.on_b) *reinterpret_cast<float2*>(mine + l.b + 2 * i) = dg.b[i];
        }
      }
      __syncthreads();
      for (int d = threadIdx.x; d < p.dim; d += QK_THREADS) {
        float sum = 0.0f;
#pragma unroll 4
        for (int k = 0; k < QK_WARPS * H; ++k) sum += joined[k * p.dim + d];
        p.partial[(static_cast<long long>(blockIdx.x) * 2 + which) * p.dim + d] = sum;
      }
      __syncthreads();
    }
  }
}

// Heads that are not made of aligned 16-byte words, or of more than 64 of them:
// a warp takes one head through shared memory, value by value, in the formulas'
// order. Bound by its 2- and 4-byte accesses, at about 0.5 TB/s.
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
      const Place at = place_of(static_cast<int>(pair), side.heads);
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
          const float n = xs[d] * r;
          xs[d] = n;
          dot = fmaf(u * weight_at<T>(p, side.weight, d), n, dot);
          dg[d] = fmaf(u, n, dg[d]);
        }
        const float m = warp_sum(dot) / D;
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

// dg: sums of the blocks' partial sums, in a fixed order: 32 columns a block,
// whose 32 warps split the partial sums.
__global__ void __launch_bounds__(1024) ns_qk_sum_kernel(const __grid_constant__ QkSumParams p) {
  __shared__ float part[32][33];
  nsptx::griddep_wait();
  nsptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < 2 * p.dim) {
#pragma unroll 8
    for (int b = warp; b < p.blocks; b += 32) sum += p.partial[static_cast<long long>(b) * 2 * p.dim + col];
  }
  part[warp][lane] = sum;
  __syncthreads();
  // warp w sums column w's parts
  sum = warp_sum(part[lane][warp]);
  const int c = blockIdx.x * 32 + warp;
  if (lane || c >= 2 * p.dim) return;
  float* out = p.out[c >= p.dim];
  if (out) out[c >= p.dim ? c - p.dim : c] = sum;
}

template <typename T, int G, QkTurn MODE>
cudaError_t launch_lanes(bool grad, QkParams& p, int nsm, int* blocks, cudaStream_t st) {
  const int H = 32 / p.lanes;
  const int most = std::min(nsm * qk_blocks(grad, MODE), QK_MAX_BLOCKS);
  // a warp's rounds in equal chunks of at most 8: long ones, since a token's angles serve all of its rounds
  // (16384 tokens of 32/8 heads take 131, 107, 97 and 93 us backward in chunks of 1, 2, 4 and 8)
  const int rounds = static_cast<int>((p.tokens * (p.side[0].heads + p.side[1].heads) + H - 1) / H);
  const int each = (rounds + most * QK_WARPS - 1) / (most * QK_WARPS), parts = (each + 7) / 8;
  p.chunk = std::max(1, (each + parts - 1) / std::max(1, parts));
  for (int i = 0; i < 2; ++i)
    p.chunks[i] = static_cast<int>((p.tokens * p.side[i].heads + H * p.chunk - 1) / (H * p.chunk));
  *blocks = std::min((p.chunks[0] + p.chunks[1] + QK_WARPS - 1) / QK_WARPS, most);
  for (int i = 0; i < 2; ++i) {
    if (!p.side[i].heads) continue;
    p.within[i] = place_of(H, p.side[i].heads);
    p.between[i] = place_of(H + (*blocks * QK_WARPS - 1) * p.chunk * H, p.side[i].heads);
  }
  const size_t smem = sizeof(uint4) * QK_WARPS * (QK_AHEAD + 1) * (grad ? 128 : 64) +
                      (MODE == SPREAD ? sizeof(float) * QK_WARPS * spread_places(Lane<T>::V) : 0);
  if (!grad) return launch_pdl(ns_qk_kernel<T, G, false, MODE>, dim3(*blocks), dim3(QK_THREADS), smem, st, p);
  const cudaError_t e = cudaFuncSetAttribute(ns_qk_kernel<T, G, true, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(ns_qk_kernel<T, G, true, MODE>, dim3(*blocks), dim3(QK_THREADS), smem, st, p);
}

template <typename T>
cudaError_t launch_qk(bool grad, bool lanes, QkParams& p, int nsm, int* blocks, cudaStream_t st) {
  constexpr int V = Lane<T>::V;
  if (lanes) {
    p.lanes = (p.dim / V + 1) / 2;
    if (p.interleaved && p.rot_dim % V) return launch_lanes<T, 0, PARTIAL>(grad, p, nsm, blocks, st);
    if (!p.interleaved && p.rot_dim % (2 * V)) return launch_lanes<T, 0, SPREAD>(grad, p, nsm, blocks, st);
    // sums over a known number of lanes, unrolled: heads of 128 bf16 60 us forward and 89 backward against 63 and 98,
    // of 256 57 and 87 against 61 and 100; other groups (heads of 64 in 16 bits have 4 lanes) take the general form,
    // which fp32 heads of 64 would be better served by backward (144 us against 153)
    if (p.lanes == 8) return launch_lanes<T, 8, WHOLE>(grad, p, nsm, blocks, st);
    if (p.lanes == 16) return launch_lanes<T, 16, WHOLE>(grad, p, nsm, blocks, st);
    return launch_lanes<T, 0, WHOLE>(grad, p, nsm, blocks, st);
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
  if (!nsk::dtype_ok(dtype)) return NS_ERR_ARG;
  if (weight_dtype != dtype && weight_dtype != NS_DT_FP32) return NS_ERR_ARG;
  if (tokens < 0 || heads[0] < 0 || heads[1] < 0 || head_dim < 1 || rot_dim < 0 || table_rows < 0) return NS_ERR_ARG;
  if (!(eps >= 0.0f) || !strides) return NS_ERR_ARG;
  if (rot_dim > head_dim || rot_dim % 2) return NS_ERR_SHAPE;
  if (head_dim > nsk::QK_MAX_DIM) return NS_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return NS_ERR_ARG;
  if (rot_dim > 0 && !table) return NS_ERR_ARG;
  if (positions && position_bytes != 4 && position_bytes != 8) return NS_ERR_ARG;
  const int most = std::max(heads[0], heads[1]);
  const int64_t both = static_cast<int64_t>(heads[0]) + heads[1];
  if (both > 0 && tokens > INT_MAX / 2 / both) return NS_ERR_SHAPE;
  const bool sums = grad && (grad_weight[0] || grad_weight[1]);
  for (int i = 0; i < 2; ++i) {
    if (grad && !nsk::element_aligned(grad_weight[i], 4)) return NS_ERR_ARG;  // written without tokens too
    if (tokens == 0 || heads[i] == 0) continue;
    if (!x[i] || !out[i] || (grad && !dy[i])) return NS_ERR_ARG;
    const int b = nsk::elem_bytes(dtype);
    if (!nsk::element_aligned(x[i], b) || !nsk::element_aligned(out[i], b) || (grad && !nsk::element_aligned(dy[i], b)))
      return NS_ERR_ARG;
    if (!nsk::element_aligned(weight[i], nsk::elem_bytes(weight_dtype))) return NS_ERR_ARG;
  }
  if (!nsk::element_aligned(table, 4) || (positions && !nsk::element_aligned(positions, position_bytes))) return NS_ERR_ARG;
  if (sums && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
               workspace_bytes < sizeof(float) * 2 * nsk::QK_MAX_BLOCKS * static_cast<uint64_t>(head_dim)))
    return NS_ERR_WORKSPACE;
  if ((tokens == 0 || most == 0) && !sums) return NS_OK;
  nsk::QkParams p = {};
  const int b = nsk::elem_bytes(dtype), V = 16 / b;
  bool lanes = head_dim % V == 0 && head_dim / V <= 64 && (reinterpret_cast<uintptr_t>(table) & 15) == 0;
  // strides: (token, head) of x, of out and, for the gradient, of dy; queries then keys of each
  for (int i = 0; i < 2; ++i) {
    nsk::QkSide& s = p.side[i];
    s.x = x[i];
    s.out = out[i];
    s.dy = grad ? dy[i] : nullptr;
    s.weight = weight[i];
    s.heads = heads[i];
    // the stride of one token, or of one head, reaches nothing
    auto token_stride = [&](int k) { return tokens > 1 ? strides[k] : 0; };
    auto head_stride = [&](int k) { return heads[i] > 1 ? strides[k] : 0; };
    s.x_token = token_stride(2 * i);
    s.x_head = head_stride(2 * i + 1);
    s.out_token = token_stride(4 + 2 * i);
    s.out_head = head_stride(5 + 2 * i);
    if (grad) {
      s.dy_token = token_stride(8 + 2 * i);
      s.dy_head = head_stride(9 + 2 * i);
    }
    const int64_t token[3] = {s.x_token, s.dy_token, s.out_token}, head[3] = {s.x_head, s.dy_head, s.out_head};
    for (int k = 0; k < 3; ++k) {
      const bool fits = std::llabs(token[k]) <= INT_MAX / 4 && std::llabs(head[k]) <= INT_MAX / 4;
      lanes = lanes && fits;
      s.token_bytes[k] = fits ? static_cast<int>(token[k]) * b : 0;
      s.head_bytes[k] = fits ? static_cast<int>(head[k]) * b : 0;
    }
    if (heads[i] == 0) continue;
    lanes = lanes && (reinterpret_cast<uintptr_t>(s.weight) & 15) == 0 && words_ok(s.x, s.x_token, s.x_head, b) &&
            words_ok(s.out, s.out_token, s.out_head, b) && (!grad || words_ok(s.dy, s.dy_token, s.dy_head, b));
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
    return nsk::launch_pdl(nsk::ns_qk_sum_kernel, dim3((2 * head_dim + 31) / 32), dim3(1024), 0, st, sp);
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
