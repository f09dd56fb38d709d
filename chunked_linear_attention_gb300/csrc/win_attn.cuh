// What the kernels of the window attention share: which keys a query sees.
//
// Queries are taken in tiles of the token axis, whatever sequences lie in them.  A
// query at token i of a sequence that begins at token t0, with P tokens before the
// call, sees of the call's own keys
//     max(t0, i - window + 1) <= j <= i,   and   t0 <= j < t0 + sinks - P,
// and of the cache's places those of its sequence that hold a sink or a position
// within the window.  A tile's keys are a list of key tiles of three kinds: call's keys
// that are sinks of the sequence its first query lies in, call's keys of the window, and
// places of the caches of the sequences that lie in it.
#pragma once

#include "mixers.cuh"
#include "mixers.h"

namespace ttt {

struct WinParams {
  const void* q;
  const void* k;
  const void* v;
  const void* cache_k;
  const void* cache_v;
  const int* slots;
  const int* past;      // NULL: no sequence has a past
  const int* starts;
  void* out;
  int* status;
  int n_slots, n_seq, B, Hq, Hk, N, d, window, sinks;
  float scale;          // of the scores, times log2(e)
  window_attention_layout lay;
  unsigned long long wait_ns;
  int withhold;         // test hook, see ttt_selftest_withhold_window
};

// Slot and past of a sequence: no past without a slot of the pool.
__device__ __forceinline__ void seq_past(const WinParams& p, int seq, int& slot, int& past) {
  slot = -1;
  past = 0;
  if (!p.past) return;
  slot = p.slots ? p.slots[seq] : seq;
  if (slot < 0 || slot >= p.n_slots) {
    slot = -1;
    return;
  }
  past = max(p.past[seq], 0);
}

// What a query sees.
struct WinRow {
  int i;        // its token, for none -1
  int seq;
  int t0;       // first token of its sequence
  int lo;       // first key of the window among the call's
  int sink1;    // behind the last sink among the call's
  int wlo;      // positions from here on are in the window
};

__device__ __forceinline__ WinRow win_row(const WinParams& p, int b, int i) {
  WinRow r;
  r.i = r.seq = -1;
  r.t0 = r.lo = 0x7fffffff;
  r.sink1 = 0;
  r.wlo = 0;
  if (i >= p.N) return r;
  const TokenSeq s = token_seq(p.starts, p.n_seq, b, p.N, i);
  if (s.seq < 0) return r;
  int slot, past;
  seq_past(p, s.seq, slot, past);
  r.i = i;
  r.seq = s.seq;
  r.t0 = s.t0;
  r.lo = max(s.t0, i - p.window + 1);   // i >= 0 and window <= 2^30
  r.sink1 = s.t0 + max(0, p.sinks - past);   // t0 < 2^31 - 1 - N at most; sinks <= 2^30
  if (r.sink1 < s.t0) r.sink1 = 0x7fffffff;
  r.wlo = past + (i - s.t0) - p.window + 1;
  return r;
}

// Key j of the call (its own sequence's, of this tile's columns below `end`).
__device__ __forceinline__ bool sees_new(const WinRow& r, int j, int end) {
  return j <= r.i && j < end && (j >= r.lo || (j >= r.t0 && j < r.sink1));
}

// A sequence's cache as its queries in a tile see it: `count` places from the first
// on, of which those behind the sinks are a ring whose newest lap ends before `head`.
struct WinCache {
  int seq, slot, count, past, head;
  int i0, i1;   // the sequence's queries in the tile
};

__device__ __forceinline__ bool sees_cache(const WinRow& r, const WinCache& c, int place, int sinks,
                                           int window) {
  if (r.seq != c.seq || place >= c.count) return false;
  if (place < sinks) return true;
  const int ring = place - sinks;
  return c.past - c.head + ring - (ring >= c.head ? window : 0) >= r.wlo;
}

// The key tiles of the queries i0 .. i1 - 1 of batch b, KT keys each.  Every thread
// that walks the list does so by itself, with the same results.
struct WinTile {
  int base;    // first key (of the call) or place (of a cache); may be negative for a key
  int end;     // columns from here on do not count
  int seq;     // -1: the call's keys
  WinCache c;  // for a cache
};

template <int KT>
struct WinList {
  int sink0, sink1;   // the call's sinks in front of the window tiles
  int at, end;        // the window tiles
  int seq, seq1, place;
  int fresh, old;     // places that the first query of c sees: sinks, the newest lap's from
                      // `fresh` to the head, the last lap's from `old` on
  int i0, i1, b;
  WinCache c;
};

template <int KT>
__device__ __forceinline__ WinList<KT> win_list(const WinParams& p, int b, int i0, int i1) {
  WinList<KT> w;
  i1 = min(i1, p.N);
  w.i0 = i0;
  w.i1 = i1;
  w.b = b;
  const WinRow r = win_row(p, b, i0);
  const int lo = r.i >= 0 ? r.lo : max(0, i0 - p.window + 1);
  w.at = i0 - (int)((unsigned)(i0 - lo + KT - 1) / KT * KT);
  w.end = i1;
  w.sink0 = r.i >= 0 ? r.t0 : 0;
  w.sink1 = r.i >= 0 ? min(r.sink1, w.at) : 0;
  // the sequences in the tile, for their caches
  w.seq = 0;
  w.seq1 = -1;
  w.place = 0;
  w.fresh = w.old = 0x7fffffff;
  w.c.count = w.c.head = 0;
  if (p.past) {
    if (!p.starts) {
      w.seq = w.seq1 = b;
    } else {
      int s0 = 0, s1 = p.n_seq;   // last sequence that begins at or before i0
      while (s1 - s0 > 1) {
        const int m = (s0 + s1) >> 1;
        if (p.starts[m] <= i0) s0 = m;
        else s1 = m;
      }
      w.seq = s0;
      s1 = p.n_seq;               // and before i1
      while (s1 - s0 > 1) {
        const int m = (s0 + s1) >> 1;
        if (p.starts[m] < i1) s0 = m;
        else s1 = m;
      }
      w.seq1 = s0;
    }
    w.seq -= 1;   // next() goes on to the first
  }
  return w;
}

template <int KT>
__device__ __forceinline__ bool win_next(const WinParams& p, WinList<KT>& w, WinTile& t) {
  t.seq = -1;
  if (w.sink0 < w.sink1) {
    t.base = w.sink0;
    t.end = w.sink1;
    w.sink0 += KT;
    return true;
  }
  if (w.at < w.end) {
    t.base = w.at;
    t.end = w.end;
    w.at += KT;
    return true;
  }
  while (true) {
    const int sinks = min(w.c.count, p.sinks), head = p.sinks + w.c.head;
    while (w.place < w.c.count) {
      const int base = w.place;
      w.place += KT;
      // tiles that no query sees are left out (24 sequences of 20011 tokens, three quarters of
      // them with a past, and a window of 1000: 219 us, all tiles of a seen ring 231)
      if (base < sinks || (base < head && base + KT > w.fresh) || base + KT > w.old) {
        t.seq = w.c.seq;
        t.base = base;
        t.end = w.c.count;
        t.c = w.c;
        return true;
      }
    }
    if (w.seq >= w.seq1) return false;
    w.seq += 1;
    w.place = 0;
    w.c.count = 0;
    // the part of the sequence that lies in the tile; bad bounds hold no token
    int t0 = 0, t1 = p.N;
    if (p.starts) {
      t0 = p.starts[w.seq];
      t1 = p.starts[w.seq + 1];
      if (t0 < 0 || t1 > p.N) continue;
    }
    const int a = max(t0, w.i0), e = min(t1, w.i1);
    if (a >= e) continue;
    seq_past(p, w.seq, w.c.slot, w.c.past);
    if (w.c.past <= 0) continue;
    w.c.seq = w.seq;
    w.c.i0 = a;
    w.c.i1 = e;
    const int ring = w.c.past - p.sinks;   // tokens that went into the ring
    w.c.head = ring > 0 ? ring % p.window : 0;
    w.c.count = min(w.c.past, p.sinks);
    // the first query in the tile sees the newest `seen` of them
    const int seen = min(p.window - 1 - (a - t0), ring);
    w.fresh = w.old = 0x7fffffff;
    if (seen > 0) {
      w.c.count += min(ring, p.window);
      w.fresh = p.sinks + max(w.c.head - seen, 0);
      if (seen > w.c.head) w.old = p.sinks + p.window - (seen - w.c.head);
    }
  }
}

WinParams win_params(const WindowArgs& a);

}  // namespace ttt
