// Shared parts of the paged-cache calls: the cache's addressing, the tokens of
// a chunk, and how attention work is laid out and divided.
#pragma once

#include "common.cuh"

namespace medusa {
namespace paged {

struct Cache {
  const int32_t* page_table;  // [B][max_pages]
  int n_pages, page_size, max_pages;
  // Rows a sequence can hold (host-checked: < 2^31 - 2^16).
  __host__ __device__ int rows() const { return max_pages * page_size; }
};

// Pool row (within one layer) of row r of sequence b, or -1 for a page outside
// the pool.  0 <= r < rows().
__device__ __forceinline__ int pool_row(const Cache& c, int b, int r) {
  const int pg = r / c.page_size;
  const int id = c.page_table[(size_t)b * c.max_pages + pg];
  return id >= 0 && id < c.n_pages ? id * c.page_size + (r - pg * c.page_size) : -1;
}

// Where sequence j ends, or -1 when its starts decrease or leave [0, T].  Starts that decrease can
// bring a later sequence back among the tokens of earlier ones: one that begins before the largest
// of their ends is as bad as the one whose own starts decrease, so that a token is one sequence's.
__device__ __forceinline__ int end_of(const int32_t* q_start, int T, int j) {
  const int a = q_start[j], e = q_start[j + 1];
  return a >= 0 && a <= e && e <= T ? e : -1;
}

// ------------------------------------------------------------------ attention work
//
// An item is (layer, head group, sequence, block of `ctok` tokens); its cost is
// its number of KT-key tiles.  All items' tiles are laid end to end, layer and
// head group outermost (CTAs that run together then read the same head's rows),
// and CTA c of C takes tiles [c Q, (c + 1) Q), Q = ceil(U / C).
// Each CTA has at most two items that it shares with others: the one its range
// starts inside (partial slot 0) and the one its range ends inside (slot 1).
struct Work {
  const int32_t* q_start;     // [B + 1], or NULL: N tokens each (tree)
  const int32_t* prefix_len;  // [B]
  int B, T, N;                // N: tree nodes, 0 for a causal chunk
  int nl, nh, cap;            // nh: head groups per layer; cap: rows a sequence can hold
  int ctok, KT;               // tokens per block and keys per tile
  int ctok_log2, KT_log2;     // both are powers of two
  int ctas;
  unsigned long long ctas_inv;  // 2^64 / ctas, rounded up
};

struct Seq {
  int q0, len, L;  // first token, tokens, rows before them
  bool ok;
};

__device__ __forceinline__ Seq seq_of(const Work& w, int b) {
  Seq s;
  s.L = w.prefix_len[b];
  if (w.q_start) {
    const int a = w.q_start[b], e = w.q_start[b + 1];
    s.q0 = a;
    s.ok = a >= 0 && e >= a && e <= w.T && (e == a || (s.L >= 0 && s.L <= w.cap - (e - a)));
    s.len = s.ok ? e - a : 0;
  } else {
    s.q0 = b * w.N;
    s.ok = s.L >= 0 && s.L <= w.cap;
    s.len = s.ok ? w.N : 0;
  }
  return s;
}

__device__ __forceinline__ int n_blocks(const Work& w, const Seq& s) { return (s.len + w.ctok - 1) >> w.ctok_log2; }

// Key tiles of block i of a sequence.  Causal: the rows up to the block's last
// token.  Tree: the prefix tiles, then the tree tiles.
__device__ __forceinline__ int block_tiles(const Work& w, const Seq& s, int i) {
  if (w.N) return ((s.L + w.KT - 1) >> w.KT_log2) + ((w.N + w.KT - 1) >> w.KT_log2);
  const int last = min(s.len, (i + 1) * w.ctok);
  return (s.L + last + w.KT - 1) >> w.KT_log2;
}

// Tiles of the sequence's first i blocks, i <= n_blocks, in closed form.  With
// L = a KT + r, a block's count is a + ceil((r + k ctok) / KT), k = 1, 2, ...:
// when ctok is m tiles, ceil(r / KT) + m k; when a tile is m blocks,
// ceil((ceil(r / ctok) + k) / m), summed by h(n) = sum_{j <= n} ceil(j / m).
__device__ __forceinline__ long long tiles_before(const Work& w, const Seq& s, int i) {
  if (i == 0) return 0;
  if (w.N) return (long long)i * block_tiles(w, s, 0);
  const int nb = n_blocks(w, s);
  const bool all = i == nb;  // the last block may be short: added on its own
  const long long n = all ? i - 1 : i;
  const int r = s.L & (w.KT - 1);
  long long t = n * (s.L >> w.KT_log2);
  if (w.ctok >= w.KT) {
    t += n * (r > 0) + ((n * (n + 1) / 2) << (w.ctok_log2 - w.KT_log2));
  } else {
    const int m = w.KT_log2 - w.ctok_log2;
    const long long r1 = (r + w.ctok - 1) >> w.ctok_log2;
    auto h = [m](long long x) {
      const long long q = x >> m, e = x & ((1ll << m) - 1);
      return ((q * (q + 1) / 2) << m) + e * (q + 1);
    };
    t += h(r1 + n) - h(r1);
  }
  return all ? t + block_tiles(w, s, nb - 1) : t;
}

__device__ __forceinline__ long long seq_tiles(const Work& w, const Seq& s) {
  return s.len > 0 ? tiles_before(w, s, n_blocks(w, s)) : 0;
}

// The item that holds a tile: block i of sequence b for layer-head lg, the
// global index of its first tile and its tile count.
struct Item {
  int lg, b, i, tiles;
  long long first;
  Seq s;
  int top;  // the largest end of the sequences so far
};

// Block-wide set-up: every thread of the CTA calls plan_find() once.  It sums the
// tiles per layer-head over the sequences and finds the item that holds tile
// Q `cta`; false when that tile does not exist.  sh: 70 long longs of shared
// memory.  Up to blockDim sequences take one round of loads and two barriers.
// Kept small, without 64-bit divisions: it runs once, so its instructions are
// fetched cold.
struct Plan {
  long long per, U, Q;  // tiles per layer-head, in all, per CTA
  bool odd;             // some sequence is bad
};

__device__ __forceinline__ bool plan_find(const Work& w, Plan& pl, Item& it, long long* sh, int cta) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, wp = tid >> 5, nw = nt >> 5;
  const int rounds = (w.B + nt - 1) / nt;
  Seq s{};
  long long v = 0, inc = 0, before = 0, total = 0;
  pl.odd = false;
  int top = -1;  // the largest end in the rounds before, where some sequence is bad
  // This thread's sequence of a round, and the tiles of the round's sequences up to it and in all.
  // A bad one makes its warp's sum -1 and the total negative.
  auto round = [&](int k) {
    const int b = k * nt + tid;
    s = b < w.B ? seq_of(w, b) : Seq{0, 0, 0, true};
    if (pl.odd && w.q_start) {
      int mine = top;
      const int last = min(w.B, (k + 1) * nt);
#pragma unroll 1
      for (int j = k * nt; j < last; ++j) {
        const int e = end_of(w.q_start, w.T, j);
        if (j < b) mine = max(mine, e);
        top = max(top, e);
      }
      if (s.q0 < mine) s.len = 0;
    }
    v = inc = seq_tiles(w, s);
#pragma unroll 1
    for (int o = 1; o < 32 && o < w.B; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const bool bad = __any_sync(0xffffffffu, !s.ok) && !pl.odd;
    __syncthreads();  // the round before is read
    if (lane == min(31, w.B - 1)) sh[wp] = bad ? -1 : inc;  // fewer than 32 sequences: lanes behind them hold no sums
    __syncthreads();
    before = total = 0;
    const int busy = min(nw, (w.B - k * nt + 31) >> 5);  // warps that have sequences
#pragma unroll 1
    for (int j = 0; j < busy; ++j) {
      const long long y = sh[j];
      if (y < 0) total = y;
      if (total < 0) break;
      if (j < wp) before += y;
      total += y;
    }
  };
  // First the sums of all rounds, then, the last round first being the one in hand, the search.
  long long per = 0, u = -1, off = 0, base = 0;
  int lg = 0;
  bool found = false;
#pragma unroll 1
  for (int k = 0; k < 2 * rounds && !found; ++k) {
    if (k == rounds) top = -1;
    if (k < rounds || rounds > 1) round(k < rounds ? k : k - rounds);
    if (total < 0) {  // the first bad sequence: the round is made again, without those that begin too early
      pl.odd = true;
      if (k > 0 && w.q_start) top = w.q_start[k * nt];  // none was bad before
      --k;
      continue;
    }
    if (k < rounds) {
      per += total;
      if (k + 1 < rounds) continue;
      pl.per = per;
      pl.U = per * ((long long)w.nl * w.nh);
      pl.Q = (long long)__umul64hi((unsigned long long)(pl.U + w.ctas - 1), w.ctas_inv);
      u = pl.Q * cta;
      if (u >= pl.U) return false;
      lg = (int)((float)u / (float)per);  // to within a few
#pragma unroll 1
      while (lg * per > u) --lg;
#pragma unroll 1
      while ((lg + 1ll) * per <= u) ++lg;
      off = u - lg * per;
      continue;
    }
    if (tid == 0) sh[63] = pl.odd;
    const long long lo = base + before + inc - v;
    if (v > 0 && off >= lo && off < lo + v) {  // one thread
      int i0 = 0, i1 = n_blocks(w, s);
#pragma unroll 1
      while (i1 - i0 > 1) {
        const int m = (i0 + i1) >> 1;
        if (tiles_before(w, s, m) <= off - lo) i0 = m;
        else i1 = m;
      }
      sh[64] = (k - rounds) * nt + tid;
      sh[65] = i0;
      sh[66] = lo + tiles_before(w, s, i0);
      sh[67] = s.q0;
      sh[68] = s.len;
      sh[69] = s.L;
    }
    base += total;
    found = base > off;  // the same in every thread
  }
  __syncthreads();
  it.lg = lg;
  it.b = (int)sh[64];
  it.i = (int)sh[65];
  it.s = Seq{(int)sh[67], (int)sh[68], (int)sh[69], true};
  it.top = it.s.q0 + it.s.len;
  it.first = lg * per + sh[66];
  it.tiles = block_tiles(w, it.s, it.i);
  return true;
}

// The next item in order (`odd`: the plan's); false behind the last one.  Whole warps.  Behind a few
// sequences without tokens, 32 at a time are passed over: other warps wait for the item meanwhile,
// and a million of them, one by one, took longer than a wait may.
__device__ __forceinline__ bool next_item(const Work& w, bool odd, Item& it) {
  it.first += it.tiles;
  ++it.i;
#pragma unroll 1
  for (int n = 0; it.s.len == 0 || it.i >= n_blocks(w, it.s); ++n) {
    it.i = 0;
    if (n >= 8 && !odd)
      while (it.b + 33 < w.B && !__any_sync(0xffffffffu, seq_of(w, it.b + 1 + (threadIdx.x & 31)).len)) it.b += 32;
    if (++it.b == w.B) {
      it.b = 0;
      if (++it.lg == w.nl * w.nh) return false;
    }
    it.s = seq_of(w, it.b);
    if (odd && w.q_start) {
      if (it.b == 0) it.top = -1;
      if (it.s.q0 < it.top) it.s.len = 0;
      it.top = max(it.top, end_of(w.q_start, w.T, it.b));
    }
  }
  it.tiles = block_tiles(w, it.s, it.i);
  return true;
}

}  // namespace paged
}  // namespace medusa
