// Causal attention with a sliding window and sinks: which tiles meet, host and device.
//
// Token t sees key u when u <= t and (u > t - window or u < sinks). In tiles of TK keys
// (or rows), a block of query rows meets the sink tiles and then the tiles from the
// window of its first row to its last row's diagonal; the two runs are disjoint.
#pragma once

#include <stdint.h>

#include "ring_schedule.h"

namespace ringattn {

struct WinGeom {
  int B, Hq, Hkv, D;
  int64_t S;
  int64_t window;  // >= 1, at most S
  int64_t sinks;   // >= 0, at most S
};

struct WinTiles {
  int ns;      // tiles [0, ns): sinks
  int w0, w1;  // tiles [w0, w1): window, w0 >= ns
};

// Tiles that query rows [r0, r1] meet (none when r0 >= S).
RA_HD WinTiles win_tiles(const WinGeom& g, int64_t r0, int64_t r1, int TK) {
  WinTiles t;
  if (r0 >= g.S) {
    t.ns = t.w0 = t.w1 = 0;
    return t;
  }
  if (r1 > g.S - 1) r1 = g.S - 1;
  const int64_t lo = r0 - g.window + 1;
  t.w0 = lo > 0 ? (int)(lo / TK) : 0;
  t.w1 = (int)(r1 / TK) + 1;
  const int n = (int)((g.sinks + TK - 1) / TK);
  t.ns = n < t.w0 ? n : t.w0;
  return t;
}

RA_HD int win_count(const WinTiles& t) { return t.ns + t.w1 - t.w0; }
RA_HD int win_tile(const WinTiles& t, int n) { return n < t.ns ? n : t.w0 + n - t.ns; }
RA_HD bool win_has(const WinTiles& t, int tile) { return tile < t.ns || (tile >= t.w0 && tile < t.w1); }

// Columns of the tile that starts at key k0 that query row a sees: c < hi and (c >= lo or
// c < sk), all in [0, N].
struct WinCut {
  int lo, hi, sk;
};
RA_HD int win_clip(int64_t x, int N) { return x <= 0 ? 0 : (x >= N ? N : (int)x); }
RA_HD WinCut win_cut(const WinGeom& g, int64_t a, int64_t k0, int N) {
  WinCut c;
  c.hi = win_clip((a < g.S ? a + 1 : g.S) - k0, N);
  c.lo = win_clip(a - g.window + 1 - k0, N);
  c.sk = win_clip(g.sinks - k0, N);
  return c;
}

}  // namespace ringattn
