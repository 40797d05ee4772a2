// What the kernels of attention over a cache share: the arguments, the rows and keys of a
// work unit, and how the work is divided.
//
// A sequence b has n = lengths[b] committed tokens in its cache and cnt <= T drafted ones
// behind them, drafted node j at cache row n + j and, by its depth in the tree, at
// position n + depth(j). Node t sees a committed token u < n when u lies in its window
// (u > n + depth(t) - window) or among the sinks (u < sinks), and of the drafted nodes
// itself and its ancestors under the same rule on their positions.
//
// A unit is (b, kv head, group of query rows); the query rows of a kv head are numbered
// t * rep + (head of the GQA group), so the rows of dead nodes come last. Its keys are
// visited in steps of `step` cache rows: the steps that hold sinks, then the steps from
// the lowest window start to the last drafted node. The steps of all units form one
// sequence that is divided evenly among the CTAs of a launch (each unit's steps start at a
// multiple of `quad` steps), whatever the lengths are: a CTA's share may end one unit and
// begin the next. CTA c's part of unit u goes to partial slot c + u, which is unique
// because every boundary raises one of the two.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mx_format.cuh"
#include "ringattn_internal.h"

namespace ringattn {
namespace tree {

constexpr int kMaxNodes = 64;

struct Params {
  CacheView c;
  const uint16_t* q;             // bf16, (b, h, t) strides in elements, unit head-dim stride
  int64_t qs_b, qs_h, qs_t;
  uint16_t* out;                 // [B, Hq, T, D] bf16
  float* lse;                    // [B, Hq, T]
  const int32_t* lengths;        // [B]
  const int32_t* parents;        // [B, T] or null (a chain)
  const int32_t* counts;         // [B] or null (T)
  int Hq, T, rep;
  int window, sinks;             // window 0: every committed token
  int groups;                    // row groups per kv head
  int rows_per_group;
  int step, quad;                // keys per step, steps per unit of division
  int ctas;                      // CTAs that share the steps
  int min_quads;                 // least share of a CTA
  float scale_log2;
  float* o_parts;                // [ctas + units][rows_per_group][D]
  float* lse_parts;              // [ctas + units][rows_per_group], base 2
  int* status;
  uint64_t watchdog_ns;
};

// The keys of one sequence's units.
struct Keys {
  int n, cnt;       // committed and drafted rows (0, 0 for a sequence that is refused)
  int sink_steps;   // steps [0, sink_steps) hold the sinks
  int first;        // the first step behind them
  int steps;        // steps in all
};

__device__ __forceinline__ bool bad_sequence(const Params& p, int b, int& n, int& cnt) {
  n = p.lengths[b];
  cnt = p.counts ? p.counts[b] : p.T;
  return n < 0 || cnt < 0 || cnt > p.T || (int64_t)n + cnt > p.c.capacity;
}

__device__ __forceinline__ Keys sequence_keys(const Params& p, int b) {
  Keys k;
  if (bad_sequence(p, b, k.n, k.cnt)) k.n = k.cnt = 0;
  k.sink_steps = 0;
  k.first = 0;
  k.steps = 0;
  if (k.cnt == 0) return k;  // no query row
  const int end = (int)(((int64_t)k.n + k.cnt + p.step - 1) / p.step);
  if (p.window > 0) {
    const int lo = k.n - p.window + 1;  // the lowest position that a root's window holds
    const int w0 = lo > 0 ? lo / p.step : 0;
    const int s = p.sinks < k.n ? p.sinks : k.n;
    const int s_steps = (int)(((int64_t)s + p.step - 1) / p.step);
    if (w0 > s_steps) {
      k.sink_steps = s_steps;
      k.first = w0;
    }
  }
  k.steps = k.sink_steps + end - k.first;
  return k;
}

__device__ __forceinline__ int step_key(const Params& p, const Keys& k, int i) {
  return (i < k.sink_steps ? i : k.first + i - k.sink_steps) * p.step;
}

// Cache row u can be seen by some query row of the sequence. Rows that none sees (behind
// the last node, or fallen out of the window) are never read: they may hold anything.
__device__ __forceinline__ bool key_live(const Params& p, const Keys& k, int u) {
  return u < k.n + k.cnt && (p.window <= 0 || u < p.sinks || u > k.n - p.window);
}

__device__ __forceinline__ int64_t sequence_quads(const Params& p, int b) {
  const Keys k = sequence_keys(p, b);
  return (int64_t)((k.steps + p.quad - 1) / p.quad) * p.c.Hkv * p.groups;
}

// One warp: the quads of all units, and the quads of the sequences before `b_stop`.
__device__ __forceinline__ void warp_totals(const Params& p, int b_stop, int64_t& total, int64_t& before) {
  const int lane = threadIdx.x % 32;
  int64_t t = 0, f = 0;
  for (int b = lane; b < p.c.B; b += 32) {
    const int64_t x = sequence_quads(p, b);
    t += x;
    if (b < b_stop) f += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t += __shfl_xor_sync(0xffffffffu, t, o);
    f += __shfl_xor_sync(0xffffffffu, f, o);
  }
  total = t;
  before = f;
}

// CTAs that get a share: none gets less than min_quads (except where there is less in all).
__device__ __forceinline__ int64_t active_ctas(const Params& p, int64_t total) {
  const int64_t most = (total + p.min_quads - 1) / p.min_quads;
  return most < p.ctas ? most : p.ctas;
}
__device__ __forceinline__ int64_t share_begin(int64_t total, int64_t ctas, int64_t c) { return total * c / ctas; }
// The CTA whose share holds quad x: the largest c with share_begin(c) <= x.
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t ctas, int64_t x) {
  return ((x + 1) * ctas - 1) / total;
}

// One warp: the sequence that holds quad x, and the quads before it.
__device__ __forceinline__ int warp_find_sequence(const Params& p, int64_t x, int64_t& before) {
  const int lane = threadIdx.x % 32;
  before = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    const int b = b0 + lane;
    const int64_t mine = b < p.c.B ? sequence_quads(p, b) : 0;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + incl > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      before += __shfl_sync(0xffffffffu, incl - mine, l);
      return b0 + l;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return p.c.B;
}

// Ancestors of the drafted nodes of sequence b as bit sets (bit t of anc[t] is the node
// itself), reduced to those that the window and the sinks let node t see, and the nodes'
// depths. All threads of the CTA call it; anc, vis, depth and jump hold kMaxNodes entries.
// A parent outside [-1, t) reads as -1 (and is reported by the status word).
__device__ __forceinline__ void tree_masks(const Params& p, int b, const Keys& k, uint64_t* anc, uint64_t* vis,
                                           int* depth, int* jump) {
  const int t = threadIdx.x;
  const bool mine = t < k.cnt;
  if (p.parents == nullptr) {
    if (mine) {
      anc[t] = t == 63 ? ~0ull : (1ull << (t + 1)) - 1;
      jump[t] = t - 1;
    }
    __syncthreads();
  } else {
    if (mine) {
      const int par = p.parents[(int64_t)b * p.T + t];
      anc[t] = 1ull << t;
      jump[t] = par >= -1 && par < t ? par : -1;
    }
    __syncthreads();
    // pointer doubling: after round i a node's set holds its first 2^i ancestors
    for (int r = 1; r < k.cnt; r <<= 1) {
      uint64_t add = 0;
      int next = -1;
      if (mine && jump[t] >= 0) {
        add = anc[jump[t]];
        next = jump[jump[t]];
      }
      __syncthreads();
      if (mine) {
        anc[t] |= add;
        jump[t] = next;
      }
      __syncthreads();
    }
  }
  if (mine) depth[t] = __popcll(anc[t]) - 1;
  __syncthreads();
  if (mine) {
    uint64_t v = anc[t];
    if (p.window > 0 && p.window <= depth[t]) {
      for (int j = 0; j < t; ++j)
        if ((v >> j & 1) && depth[j] <= depth[t] - p.window && (int64_t)k.n + depth[j] >= p.sinks) v &= ~(1ull << j);
    }
    vis[t] = v;
  }
  __syncthreads();
}

// Row of out and lse ([B, Hq, T]) of unit row r (t * rep + head of the group).
__device__ __forceinline__ int64_t out_row(const Params& p, int b, int kvh, int r) {
  return ((int64_t)b * p.Hq + kvh * p.rep + r % p.rep) * p.T + r / p.rep;
}

}  // namespace tree
}  // namespace ringattn
