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
//
// All of this is 32-bit arithmetic with power-of-two steps, and the parts that run once per
// unit are functions of their own: these kernels are short, and the instructions that a
// launch has to fetch first are a good part of its time (with 64-bit divisions inlined the
// merge alone was 45 KB of code and took 12 us).
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mx_format.cuh"
#include "ringattn_internal.h"

namespace ringattn {
namespace tree {

// Functions that run once per unit: calls, except in kernels that move registers between
// warpgroups (setmaxnreg), which cannot call functions.
#ifdef TREE_INLINE
#define TREE_ONCE __device__ __forceinline__
#else
#define TREE_ONCE __device__ __noinline__
#endif

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
  int step, step_log2;           // keys per step
  int quad_log2;                 // steps per quad, the grain of division
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
  // (capacity <= 2^30 and cnt <= 64: the sum cannot pass 2^31 once n is in range)
  return n < 0 || cnt < 0 || cnt > p.T || n > (int)p.c.capacity || n + cnt > (int)p.c.capacity;
}

__device__ __forceinline__ Keys sequence_keys(const Params& p, int b) {
  Keys k;
  if (bad_sequence(p, b, k.n, k.cnt)) k.n = k.cnt = 0;
  k.sink_steps = 0;
  k.first = 0;
  k.steps = 0;
  if (k.cnt == 0) return k;  // no query row
  const int end = (k.n + k.cnt + p.step - 1) >> p.step_log2;
  if (p.window > 0) {
    const int lo = k.n - p.window + 1;  // the lowest position that a root's window holds
    const int w0 = lo > 0 ? lo >> p.step_log2 : 0;
    const int s = p.sinks < k.n ? p.sinks : k.n;
    const int s_steps = (s + p.step - 1) >> p.step_log2;
    if (w0 > s_steps) {
      k.sink_steps = s_steps;
      k.first = w0;
    }
  }
  k.steps = k.sink_steps + end - k.first;
  return k;
}

__device__ __forceinline__ int step_key(const Params& p, const Keys& k, int i) {
  return (i < k.sink_steps ? i : k.first + i - k.sink_steps) << p.step_log2;
}

// Cache row u can be seen by some query row of the sequence. Rows that none sees (behind
// the last node, or fallen out of the window) are never read: they may hold anything.
__device__ __forceinline__ bool key_live(const Params& p, const Keys& k, int u) {
  return u < k.n + k.cnt && (p.window <= 0 || u < p.sinks || u > k.n - p.window);
}

__device__ __forceinline__ uint32_t unit_quads(const Params& p, const Keys& k) {
  return (uint32_t)(k.steps + (1 << p.quad_log2) - 1) >> p.quad_log2;
}
__device__ __forceinline__ uint32_t sequence_quads(const Params& p, int b) {
  return unit_quads(p, sequence_keys(p, b)) * (uint32_t)(p.c.Hkv * p.groups);
}

// How the quads are shared: the first `more` of `ctas` CTAs take base + 1, the others base.
// None gets less than min_quads (except where there is less in all).
struct Shares {
  uint32_t ctas, base, more;
};
__device__ __forceinline__ Shares shares_of(const Params& p, uint32_t total) {
  const uint32_t most = (total + p.min_quads - 1) / p.min_quads;
  Shares s;
  s.ctas = most < (uint32_t)p.ctas ? most : (uint32_t)p.ctas;
  s.base = s.ctas ? total / s.ctas : 0;
  s.more = total - s.base * s.ctas;
  return s;
}
__device__ __forceinline__ uint32_t share_begin(const Shares& s, uint32_t c) {
  return c >= s.ctas ? s.base * s.ctas + s.more : c * s.base + (c < s.more ? c : s.more);
}
// The CTA whose share holds quad x.
__device__ __forceinline__ uint32_t share_of(const Shares& s, uint32_t x) {
  const uint32_t wide = s.more * (s.base + 1);
  return x < wide ? x / (s.base + 1) : s.more + (x - wide) / s.base;
}

// One warp: the quads of all units, and the quads of the sequences before `b_stop`.
__device__ __forceinline__ void warp_totals(const Params& p, int b_stop, uint32_t& total, uint32_t& before) {
  const int lane = threadIdx.x % 32;
  uint32_t t = 0, f = 0;
#pragma unroll 1
  for (int b = lane; b < p.c.B; b += 32) {
    const uint32_t x = sequence_quads(p, b);
    t += x;
    if (b < b_stop) f += x;
  }
  total = __reduce_add_sync(0xffffffffu, t);
  before = __reduce_add_sync(0xffffffffu, f);
}

// One warp: the sequence that holds quad x, and the quads before it.
__device__ __forceinline__ int warp_find_sequence(const Params& p, uint32_t x, uint32_t& before) {
  const int lane = threadIdx.x % 32;
  before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    const int b = b0 + lane;
    const uint32_t mine = b < p.c.B ? sequence_quads(p, b) : 0;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
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

// The drafted nodes of a sequence, held by one warp: lane l has nodes l and l + 32. seen: the
// node itself and its ancestors as bits, reduced to those that the window and the sinks let
// it see. A parent outside [-1, t) reads as -1 (and is reported by the status word).
static_assert(kTreeMaxNodes == 64, "two nodes per lane, and their sets in 64 bits");
struct Nodes {
  uint64_t seen[2];
  int depth[2];
};

TREE_ONCE Nodes warp_nodes(const Params& p, int b, const Keys& k) {
  const int lane = threadIdx.x % 32;
  Nodes x;
  int jump[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t = lane + 32 * s;
    const bool mine = t < k.cnt;
    jump[s] = -1;
    if (p.parents == nullptr) {
      x.seen[s] = !mine ? 0 : (t == 63 ? ~0ull : (1ull << (t + 1)) - 1);
    } else {
      x.seen[s] = mine ? 1ull << t : 0;
      const int par = mine ? p.parents[(int64_t)b * p.T + t] : -1;
      if (par >= 0 && par < t) jump[s] = par;
    }
  }
  if (p.parents != nullptr) {
    // pointer doubling: after round i a node's set holds its first 2^i ancestors
#pragma unroll 1
    for (int r = 1; r < k.cnt; r <<= 1) {
      uint64_t add[2];
      int next[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int from = jump[s] & 31;
        const uint64_t a0 = __shfl_sync(0xffffffffu, x.seen[0], from), a1 = __shfl_sync(0xffffffffu, x.seen[1], from);
        const int j0 = __shfl_sync(0xffffffffu, jump[0], from), j1 = __shfl_sync(0xffffffffu, jump[1], from);
        add[s] = jump[s] < 0 ? 0 : (jump[s] < 32 ? a0 : a1);
        next[s] = jump[s] < 0 ? -1 : (jump[s] < 32 ? j0 : j1);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        x.seen[s] |= add[s];
        jump[s] = next[s];
      }
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) x.depth[s] = __popcll(x.seen[s]) - 1;
  // ancestors that fell out of a window shorter than the tree is deep
  if (__any_sync(0xffffffffu, p.window > 0 && (p.window <= x.depth[0] || p.window <= x.depth[1]))) {
    const uint64_t anc[2] = {x.seen[0], x.seen[1]};
#pragma unroll 1
    for (int j = 0; j < k.cnt; ++j) {
      const int d0 = __shfl_sync(0xffffffffu, x.depth[0], j & 31), d1 = __shfl_sync(0xffffffffu, x.depth[1], j & 31);
      const int dj = j < 32 ? d0 : d1;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if ((anc[s] >> j & 1) && dj <= x.depth[s] - p.window && k.n + dj >= p.sinks)
          x.seen[s] &= ~(1ull << j);
    }
  }
  return x;
}

// Node t's set and depth (all lanes call it, each with its own t).
__device__ __forceinline__ void node_of(const Nodes& x, int t, uint64_t& seen, int& depth) {
  const uint64_t a0 = __shfl_sync(0xffffffffu, x.seen[0], t & 31), a1 = __shfl_sync(0xffffffffu, x.seen[1], t & 31);
  const int d0 = __shfl_sync(0xffffffffu, x.depth[0], t & 31), d1 = __shfl_sync(0xffffffffu, x.depth[1], t & 31);
  seen = t < 32 ? a0 : a1;
  depth = t < 32 ? d0 : d1;
}

// A CTA's walk over the parts of its share: `part` is set to the next one while there is one.
struct Part {
  int b, kvh, grp;
  Keys ks;
  int q0, q1;        // quads of the unit
  bool alone;        // the whole unit
  int unit;
  int64_t head_row;  // first cache row of (b, kv head)
};
struct Walk {
  uint32_t x, x_end, before;  // next quad, end of the share, quads before sequence b
  int b;
};

// Called by one warp; `out` (shared memory) then holds the walk for every thread of the CTA.
TREE_ONCE void warp_begin_walk(const Params& p, Walk* out) {
  uint32_t total, before = 0, none;
  warp_totals(p, 0, total, none);
  const Shares sh = shares_of(p, total);
  const uint32_t x0 = share_begin(sh, blockIdx.x), x1 = share_begin(sh, blockIdx.x + 1);
  const int b = x0 < x1 ? warp_find_sequence(p, x0, before) : p.c.B;
  if (threadIdx.x % 32 == 0) {
    out->x = x0;
    out->x_end = x1;
    out->before = before;
    out->b = b;
  }
}

TREE_ONCE bool next_part(const Params& p, Walk& w, Part& part) {
  while (w.x < w.x_end) {
    part.ks = sequence_keys(p, w.b);
    const uint32_t per = unit_quads(p, part.ks);
    const uint32_t here = per * (uint32_t)(p.c.Hkv * p.groups);
    if (w.x >= w.before + here) {
      w.before += here;
      ++w.b;
      continue;
    }
    const uint32_t local = w.x - w.before;
    const uint32_t u = local / per;
    part.b = w.b;
    part.kvh = (int)(u / (uint32_t)p.groups);
    part.grp = (int)u - part.kvh * p.groups;
    part.q0 = (int)(local - u * per);
    part.q1 = (int)(per - part.q0 < w.x_end - w.x ? per : part.q0 + (w.x_end - w.x));
    part.alone = part.q0 == 0 && part.q1 == (int)per;
    part.unit = w.b * p.c.Hkv * p.groups + (int)u;
    part.head_row = ((int64_t)w.b * p.c.Hkv + part.kvh) * p.c.capacity;
    w.x += part.q1 - part.q0;
    return true;
  }
  return false;
}

// Where a unit's partial results are: those of CTAs first .. first + count - 1, in slots
// first + unit and following. count 1: the unit was done by one CTA, which wrote the result.
struct Parts {
  uint32_t first, count;
};
__device__ __forceinline__ Parts warp_parts(const Params& p, int b, uint32_t u_local, uint32_t per) {
  uint32_t total, before;
  warp_totals(p, b, total, before);
  const Shares sh = shares_of(p, total);
  const uint32_t x = before + u_local * per;
  Parts r;
  r.first = share_of(sh, x);
  r.count = share_of(sh, x + per - 1) - r.first + 1;
  return r;
}

// Row of out and lse ([B, Hq, T]) of unit row r (t * rep + head of the group).
__device__ __forceinline__ int64_t out_row(const Params& p, int b, int kvh, int r) {
  return ((int64_t)b * p.Hq + kvh * p.rep + r % p.rep) * p.T + r / p.rep;
}

// The launches of tree_tiles.cu and of the merge (tree_rows.cu).
int launch_tiles(const Params& p, cudaStream_t stream);

}  // namespace tree
}  // namespace ringattn
