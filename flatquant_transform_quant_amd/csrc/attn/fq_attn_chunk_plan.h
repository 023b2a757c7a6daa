// The plan of attention of new tokens (fq_attn_chunk.h): which row tiles and key tiles each workgroup has, from cu_q and lengths
// on the device.  A wave works it out by itself; wave_scan (fq_attn_dev.h) and the operations between lanes are the includer's.
#pragma once

#include "fq_attn.h"

namespace fq {
namespace {

constexpr int kKeys = 64;  // keys of a tile
constexpr int kStart = 2;  // tiles that a segment's beginning and end count as when the work is dealt

struct Seq {
  int q0, lq, lk, off;  // its first row and rows (tokens), its keys, keys ahead of the first row
  int tiles, places;    // row tiles, and what one head's count for
};

// Places of a sequence's row tiles before tile j, in key tiles: the sums of spans in tokens, over 64, rounded down.  A
// tile's span: kStart + 1 tiles, the whole tiles of the first tokens, and the keys up to behind its last token (at most
// behind the last key) or what a window of all its tokens can touch.  (So that it has a place for each of its key tiles.)
// With a workgroup a segment it is one place.
__device__ __forceinline__ int places_before(const ChunkArgs& a, int off, int lk, int j) {
  if (a.single) return j;
  const int64_t a0 = max(off, 0), R = a.tokens;
  int64_t cap = lk + R, more = (kStart + 1) * kKeys;
  if (a.window > 0) {
    cap = min(cap, static_cast<int64_t>(a.window) + R + 126);
    more += (a.sinks + kKeys - 1) / kKeys * static_cast<int64_t>(kKeys);
  }
  const int64_t n = cap > a0 ? min(static_cast<int64_t>(j), static_cast<int64_t>(static_cast<uint32_t>(cap - a0) / static_cast<uint32_t>(a.tokens))) : 0;
  return static_cast<int>((n * a0 + R * (n * (n + 1) / 2) + (j - n) * cap + j * more) >> 6);
}

__device__ __forceinline__ Seq seq_of(const ChunkArgs& a, int b) {
  Seq s{0, 0, 0, 0, 0, 0};
  if (b < a.B) {
    s.q0 = max(0, min(a.cu_q[b], a.Tq));
    s.lq = max(0, max(0, min(a.cu_q[b + 1], a.Tq)) - s.q0);  // (a difference of numbers that are not negative)
    s.lk = max(0, min(a.lengths[b], a.reach));
    s.off = s.lk - s.lq;
    s.tiles = (s.lq + a.tokens - 1) / a.tokens;
    s.places = places_before(a, s.off, s.lk, s.tiles);
  }
  return s;
}
__device__ __forceinline__ Seq lane_seq(const Seq& s, int w) {  // a lane's, for the whole wave
  return Seq{__builtin_amdgcn_readlane(s.q0, w),  __builtin_amdgcn_readlane(s.lq, w),    __builtin_amdgcn_readlane(s.lk, w),
             __builtin_amdgcn_readlane(s.off, w), __builtin_amdgcn_readlane(s.tiles, w), __builtin_amdgcn_readlane(s.places, w)};
}

// Run i of `runs` (at most `most`) has the places from start(i) up to start(i + 1).
struct Deal {
  uint32_t total, runs, q, r;
  __device__ Deal(uint32_t places, uint32_t most) : total(places), runs(min(places, most)) {
    q = runs ? total / runs : 0u;
    r = total - q * runs;
  }
  __device__ int start(uint32_t i) const { return static_cast<int>(i * q + i * r / runs); }
};

// All places (wave by wave, no barrier).
__device__ __forceinline__ int all_places(const ChunkArgs& a) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) total += __builtin_amdgcn_readlane(wave_scan(seq_of(a, b0 + lane).places), 63) * a.heads;
  return total;
}

// A segment: a row tile of one (sequence, cache head and heads' tile), and the first of its places.
struct Segment {
  Seq s;
  int b, head, tile, at;
};

// The segment that holds place x (below all of them; without row tiles if there is none, as sequences that lie over each other may
// have more places than an int counts).
__device__ __forceinline__ Segment segment_at(const ChunkArgs& a, int x) {
  const int lane = threadIdx.x & 63;
  Segment g;
  int before = 0;
  for (int b0 = 0;; b0 += 64) {
    const Seq s = seq_of(a, b0 + lane);
    const int incl = wave_scan(s.places) * a.heads;
    const uint64_t holds = __ballot(before + incl > x);
    if (holds == 0 && b0 + 64 < a.B) {
      before += __builtin_amdgcn_readlane(incl, 63);
      continue;
    }
    const int w = __builtin_ctzll(holds | (uint64_t(1) << 63));
    g.s = lane_seq(s, w);
    g.b = b0 + w;
    g.at = before + __builtin_amdgcn_readlane(incl - s.places * a.heads, w);
    break;
  }
  const int p = max(1, g.s.places);
  g.head = max(0, min((x - g.at) / p, a.heads - 1));
  g.at += g.head * p;
  int lo = 0, hi = max(1, g.s.tiles);  // the tile's first place is at or before x, that of tile hi behind it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.at + places_before(a, g.s.off, g.s.lk, mid) <= x) lo = mid; else hi = mid;
  }
  g.tile = lo;
  g.at += places_before(a, g.s.off, g.s.lk, lo);
  return g;
}

// The key tiles that a row tile walks: the first `sinks` ones, then those from `lo` on; n in all.
struct Walk {
  int row0, row1;  // its first and last token
  int n, sinks, lo;
  __device__ int tile(int u) const { return u < sinks ? u : lo + u - sinks; }
};
__device__ __forceinline__ Walk walk_of(const ChunkArgs& a, const Seq& s, int tile) {
  Walk w;
  w.row0 = tile * a.tokens;
  w.row1 = min(w.row0 + a.tokens, s.lq) - 1;
  const int last = s.off + w.row1;  // the last key that is seen
  w.sinks = w.lo = 0;
  w.n = 0;
  if (last < 0) return w;
  if (a.window > 0) {
    w.sinks = (min(a.sinks, last + 1) + kKeys - 1) / kKeys;
    w.lo = max(w.sinks, max(0, s.off + w.row0 - a.window + 1) / kKeys);
  }
  w.n = w.sinks + last / kKeys + 1 - w.lo;
  return w;
}

// The workgroup's run of places.
struct Run {
  int i, first, last;  // last <= first: none
};
__device__ __forceinline__ Run run_of(const ChunkArgs& a) {
  // (neighbouring runs, which share keys, on one XCD's L2)
  const Deal deal(all_places(a), a.single ? ~0u : a.runs);
  const int per_xcd = (deal.runs + 7) / 8, i = static_cast<int>(blockIdx.x & 7) * per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= per_xcd || i >= static_cast<int>(deal.runs)) return Run{0, 0, 0};
  return Run{i, deal.start(i), deal.start(i + 1)};
}
// What of a segment's walk is this run's: tiles u0 .. u1 - 1; whole: all of it (an empty walk is its first place's run's).
struct Share {
  int u0, u1;
  bool whole;
};
__device__ __forceinline__ Share share_of(const ChunkArgs& a, const Run& r, const Segment& sg, const Walk& wk) {
  const int base = sg.at + kStart;  // the place of the first tile
  Share s;
  s.u0 = a.single ? 0 : min(wk.n, max(0, r.first - base));
  s.u1 = a.single ? wk.n : max(s.u0, min(wk.n, r.last - base));
  s.whole = wk.n == 0 ? sg.at >= r.first && sg.at < r.last : s.u0 == 0 && s.u1 == wk.n;
  return s;
}
// The segment behind sg; false: it is not this run's.
__device__ __forceinline__ bool next_segment(const ChunkArgs& a, const Run& r, Segment& sg) {
  sg.at += places_before(a, sg.s.off, sg.s.lk, sg.tile + 1) - places_before(a, sg.s.off, sg.s.lk, sg.tile);
  if (sg.at >= r.last) return false;
  if (++sg.tile == sg.s.tiles) {
    sg.tile = 0;
    if (++sg.head == a.heads) {
      sg.head = 0;
      do sg.s = seq_of(a, ++sg.b); while (sg.s.tiles == 0 && sg.b < a.B);
      sg.s = lane_seq(sg.s, 0);
      return sg.s.tiles != 0;
    }
  }
  return true;
}

// The segment that begins in run `run` and goes on behind it, and how many runs behind that one have a part of it (0: there is none).
struct Shared {
  Segment sg;
  Walk wk;
  int parts;
};
__device__ __forceinline__ Shared shared_from(const ChunkArgs& a, int run) {
  Shared h{};
  const Deal deal(all_places(a), a.runs);
  if (run + 1 >= static_cast<int>(deal.runs)) return h;
  const int end = deal.start(run + 1);
  h.sg = segment_at(a, end - 1);
  if (h.sg.s.tiles == 0) return h;
  h.wk = walk_of(a, h.sg.s, h.sg.tile);
  const int base = h.sg.at + kStart;
  if (deal.start(run) > base || end <= base || end - base >= h.wk.n) return h;  // its first tile is not here, or its last one is
  h.parts = 1;
  while (run + h.parts + 1 < static_cast<int>(deal.runs) && deal.start(run + h.parts + 1) - base < h.wk.n) ++h.parts;
  return h;
}
// The place in the workspace of the part that a run has from a segment's tile u0 on.
__device__ __forceinline__ int part_at(int run, int u0) { return 2 * run + (u0 == 0 ? 1 : 0); }

}  // namespace
}  // namespace fq
