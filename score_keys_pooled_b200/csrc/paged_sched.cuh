// How the paged attention's work is cut: items, units and the shares of the workers.
//
// An item is a tile of query rows of one KV head against one list of keys.
// Rows of a tile are ordered token-major: row r is token tok0 + r / G, query
// head kvh * G + r % G.  There are two lists of items:
//   prefix items   every token of the batch, tile after tile, against the
//                  shared prefix (the prefix is read once for all rows of a
//                  tile, whichever sequences they belong to);
//   own items      the new tokens of one sequence, tile after tile, against
//                  the sequence's own keys, causal; with `walk_prefix` the
//                  prefix keys come first in the same item (long chunks fill
//                  a tile by themselves, so nothing has to be joined later).
// A unit is one tile of kt keys of an item, and `fixed` more at the item's
// front stand for what an item costs whatever its length (2.2 us against 3.2 us
// of a unit in the decode kernel).  The U units, in the order prefix
// items (kvh, row tile), own items (sequence, kvh, row tile), are cut into n
// even shares: share c takes units [c U / n, (c + 1) U / n), so the split
// follows the actual lengths, which only the device knows, and every share
// reads the same number of key tiles (n is the kernel's number of workers, or
// U where that is less).  A share's part of an item is a piece; a piece that
// is not a whole item leaves its rows' (reference, sum, accumulator) in slot
// 2c (the item began in an earlier share) or 2c + 1 (it began here and goes
// on), at most one of each per share.
// With prefix items alone and few row tiles (npt <= n / 2) the workers form
// teams of npt: the members of a team take the same keys for different row
// tiles at about the same time, so HBM is read once and the others hit L2 (in
// the plain order every row tile would read the whole prefix from HBM again).
// A share is then a team's, and a member's slots are those of share * npt +
// member.
#pragma once

#include "rotary.cuh"

namespace s2o {

struct PagedGeom {
  const int32_t* table;         // [nseq, max_pages]
  const int32_t* prefix_pages;  // [ceil(prefix / page)]
  const int32_t* q_start;       // [nseq + 1]
  const int32_t* kv_len;        // [nseq]
  int Hq, Hkv, G, nseq, max_pages, num_pages, page_log2, Tq, max_q, prefix;
};

// What one kernel makes of it.
struct PagedCut {
  int tpt;          // tokens of a row tile
  int kt_log2;      // keys of a unit
  int prefix_items; // prefix items exist
  int own_items;    // own items exist
  int walk_prefix;  // own items start with the prefix's tiles
  int fixed;        // units of an item that are no keys
};

struct SeqInfo {
  int q0, qlen, len;  // first token, tokens, own keys (the tokens' included)
};

// A sequence's numbers, checked; qlen 0 where it has no tokens or they are
// out of range (then the error word is set).
__device__ __forceinline__ SeqInfo seq_info(const PagedGeom& g, int s) {
  SeqInfo i;
  i.q0 = g.q_start[s];
  const int q1 = g.q_start[s + 1];
  i.len = g.kv_len[s];
  i.qlen = (int)((int64_t)q1 - i.q0);
  if (!seq_fits(s, i.q0, q1, i.len, g.Tq, g.max_q, (int64_t)g.max_pages << g.page_log2)) {
    set_error(kErrBadCache);
    i.qlen = 0;
  }
  return i;
}

// tokens of the batch: rows behind the last sequence belong to nobody
__device__ __forceinline__ int batch_tokens(const PagedGeom& g) { return max(0, min(g.q_start[g.nseq], g.Tq)); }

// a / b, a >= 0, b > 0: the 64-bit division is a long subroutine, so numbers
// that fit take the 32-bit one (a piece's bookkeeping sits between two loads)
static __host__ __device__ __noinline__ int64_t quot_long(int64_t a, int64_t b) { return a / b; }
__host__ __device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return quot_long(a, b);
}

// sum over i < n of floor((a i + b) / m), n, a, b >= 0, m > 0: the well-known
// recursion of Euclid's algorithm (whole parts out, then the axes swapped)
static __host__ __device__ __noinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t r = 0;
  while (n > 0) {
    if (a >= m) {
      const int64_t q = quot(a, m);
      r += n * (n - 1) / 2 * q;
      a -= q * m;
    }
    if (b >= m) {
      const int64_t q = quot(b, m);
      r += n * q;
      b -= q * m;
    }
    const int64_t y = a * n + b;
    if (y < m) break;
    n = quot(y, m);
    b = y - n * m;
    const int64_t t = m; m = a; a = t;
  }
  return r;
}

struct OwnUnits {
  int nrt;       // row tiles
  int np;        // prefix tiles of each (walk_prefix)
  int len, off;  // own keys; own keys before the first new token
  int tpt, kt_log2, fixed;
  // units of the first rt row tiles: tile i < nrt - 1 sees off + (i + 1) tpt keys, the last one all
  __host__ __device__ int64_t before(int rt) const {
    if (rt <= 0) return 0;
    const int64_t kt = (int64_t)1 << kt_log2;
    if (nrt == 1) return fixed + np + ((len + kt - 1) >> kt_log2);
    int64_t u = (int64_t)rt * (fixed + np) + floor_sum(rt < nrt ? rt : rt - 1, kt, tpt, (int64_t)off + tpt + kt - 1);
    if (rt >= nrt) u += (len + kt - 1) >> kt_log2;
    return u;
  }
};

__host__ __device__ __forceinline__ OwnUnits own_units(int qlen, int len, int prefix, const PagedCut& c) {
  OwnUnits u;
  u.nrt = qlen <= c.tpt ? 1 : (qlen + c.tpt - 1) / c.tpt;
  u.np = c.walk_prefix ? (int)(((int64_t)prefix + (1 << c.kt_log2) - 1) >> c.kt_log2) : 0;
  u.len = len;
  u.off = len - qlen;
  u.tpt = c.tpt;
  u.kt_log2 = c.kt_log2;
  u.fixed = c.fixed;
  return u;
}

// units of a prefix item
__host__ __device__ __forceinline__ int64_t prefix_units(int prefix, const PagedCut& c) {
  return c.fixed + (((int64_t)prefix + (1 << c.kt_log2) - 1) >> c.kt_log2);
}

__host__ __device__ __forceinline__ int shares_of(int64_t U, int workers) { return U < workers ? (int)U : workers; }
__host__ __device__ __forceinline__ int64_t share_begin(int64_t U, int n, int c) { return quot(U * c, n); }
// the share that holds unit u
__host__ __device__ __forceinline__ int share_owner(int64_t U, int n, int64_t u) {
  return (int)quot((u + 1) * n - 1, U);
}

// A piece: the share's part of an item.
struct Piece {
  int kind;          // 0 prefix item, 1 own item, -1 no more
  int seq, kvh;
  int tok0, ntok;    // tokens of the row tile
  int off;           // own: key index of token tok0 (it sees own keys 0 .. off)
  int len;           // keys of the list the rows of the tile can reach (prefix: all of it)
  int np;            // leading tiles that are the prefix's
  int tile0, tile1;  // tiles of the item the piece covers
  int first, last;   // the piece begins, ends the item
  int share;         // number of the worker (its slots)
};

// Walks the pieces of a share.
struct Sched {
  int64_t U, u, end;      // units in all, next unit, end of the share
  int n, me;              // shares; this one
  // position of unit u
  int kind, seq, kvh, rt;
  int64_t item0, items;   // the item's first unit and its units
  int npt, ntok_all;      // prefix row tiles; tokens of the batch
  int team;               // members of a team (1: none)
  SeqInfo si;
};

__device__ __forceinline__ void sched_own_item(const PagedGeom& g, const PagedCut& c, Sched& s, int64_t seq0) {
  const OwnUnits ou = own_units(s.si.qlen, s.si.len, g.prefix, c);
  const int64_t b = ou.before(s.rt);
  s.item0 = seq0 + s.kvh * ou.before(ou.nrt) + b;
  s.items = ou.before(s.rt + 1) - b;
}

// the first own item of a sequence at or after `seq` that has tokens
__device__ __forceinline__ void sched_next_seq(const PagedGeom& g, const PagedCut& c, Sched& s, int seq, int64_t u) {
  for (; seq < g.nseq; ++seq) {
    s.si = seq_info(g, seq);
    if (s.si.qlen > 0) break;
  }
  s.kind = 1;
  s.seq = seq;
  s.kvh = s.rt = 0;
  if (seq < g.nseq) sched_own_item(g, c, s, u);
}

// members of a team of n workers
__device__ __forceinline__ int team_size(const PagedCut& c, int npt, int n) {
  return c.prefix_items && !c.own_items && npt > 0 && 2 * npt <= n ? npt : 1;
}

struct SchedFound {
  int seq;
  int64_t u;  // the sequence's first unit
};
// Units of all own items, and where this thread's run of sequences [s0, s1)
// stands among them.  Block-wide, blockDim.x a multiple of 32 up to 1024;
// `red` is a word of shared memory for each warp; `found` (`own` entries) is
// made ready for sched_begin on the way.
struct OwnRun {
  int s0, s1;
  int64_t begin, mine, total;
};
__device__ __forceinline__ OwnRun own_run(const PagedGeom& g, const PagedCut& c, int own, int64_t* red,
                                          SchedFound* found) {
  const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nth >> 5;
  const int per = (g.nseq + nth - 1) / nth;
  OwnRun r;
  r.s0 = min(g.nseq, tid * per);
  r.s1 = min(g.nseq, r.s0 + per);
  r.mine = 0;
  for (int q = r.s0; q < r.s1; ++q) {
    const SeqInfo si = seq_info(g, q);
    if (si.qlen > 0) {
      const OwnUnits ou = own_units(si.qlen, si.len, g.prefix, c);
      r.mine += g.Hkv * ou.before(ou.nrt);
    }
  }
  int64_t incl = r.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) red[warp] = incl;
  if (tid < own) found[tid].seq = g.nseq;
  __syncthreads();
  // every thread adds up the sums of the warps before its own
  int64_t v = 0, before = 0;
  for (int w = 0; w < nw; ++w) {
    if (w == warp) before = v;
    v += red[w];
  }
  r.total = v;
  r.begin = before + incl - r.mine;
  return r;
}

// Prefix items in the tile kernel and own items in the decode kernel run side
// by side: of `sms` SMs the decode kernel gets a share that makes both end
// together.  A prefix unit (256 rows, 128 keys) keeps an SM 2250 ns busy (1300
// with 128 rows); an own unit (64 keys, 32 KB) costs an SM of eight or four
// streams 520 or 1100 ns (64 sequences of up to 1023 keys behind 32K: 71.8,
// 69.4, 71.5, 74.9 us at 400, 480, 560, 700; 128 of 600 behind 8K: 59.4, 57.2,
// 60.1 at 420, 520, 620; 64 of 5 tokens and 500 keys behind 16K, four streams:
// 125, 117, 121 at 900, 1100, 1300).  Both kernels come to the same answer; the
// host's choice between the prefix's ways goes by the same prices of a tile.
constexpr float kTileNs = 2250.f, kHalfTileNs = 1300.f;
__device__ __forceinline__ int decode_sms(const PagedGeom& g, const PagedCut& tile, int ntok, int64_t own_units,
                                          float own_ns, int sms) {
  const int npt = (ntok + tile.tpt - 1) / tile.tpt;
  const int64_t np = prefix_units(g.prefix, tile);
  const float w1 = (float)((int64_t)npt * g.Hkv * np) * (2 * ntok <= tile.tpt ? kHalfTileNs : kTileNs);
  const float w2 = (float)own_units * own_ns;
  const int n = __float2int_rn((float)sms * w2 / (w1 + w2));
  return max(1, min(sms - 1, n));
}

// Total units and the item of the first unit of this thread's share.  A block
// is `own` workers (1 to 8), `ctas` of the grid's blocks work: worker w of
// block b is number w * ctas + b; the calling thread asks for worker `which`
// of its block.  `run`, `found`: own_run()'s.  Block-wide.
__device__ __forceinline__ Sched sched_begin(const PagedGeom& g, const PagedCut& c, int own, int which, int ctas,
                                             const OwnRun& run, SchedFound* found) {
  Sched s;
  const int workers = ctas * own, number = which * ctas + blockIdx.x;
  const bool works = blockIdx.x < ctas;
  s.ntok_all = batch_tokens(g);
  s.npt = c.prefix_items ? (s.ntok_all + c.tpt - 1) / c.tpt : 0;
  const int64_t np = prefix_units(g.prefix, c);
  s.team = team_size(c, s.npt, workers);
  if (s.team > 1) {
    s.U = g.Hkv * np;
    s.n = shares_of(s.U, workers / s.team);
    s.me = number / s.team;
    s.kind = works && s.me < s.n ? 0 : -1;
    s.seq = 0;
    if (s.kind < 0) return s;
    s.u = share_begin(s.U, s.n, s.me);
    s.end = share_begin(s.U, s.n, s.me + 1);
    s.kvh = (int)quot(s.u, np);
    s.rt = number - s.me * s.team;
    s.item0 = s.kvh * np;
    s.items = np;
    return s;
  }
  const int64_t PU = (int64_t)s.npt * g.Hkv * np;
  s.U = PU + (c.own_items ? run.total : 0);
  s.n = shares_of(s.U, workers);
  s.me = number;
  // the thread whose sequences hold a worker's first unit looks it up
  const int64_t begin = PU + run.begin;
  for (int w = 0; w < own && works && c.own_items && run.mine > 0; ++w) {
    const int me = w * ctas + blockIdx.x;
    if (me >= s.n) break;
    const int64_t u = share_begin(s.U, s.n, me);
    if (u < begin || u >= begin + run.mine) continue;
    int64_t at = begin;
    for (int q = run.s0; q < run.s1; ++q) {
      const SeqInfo si = seq_info(g, q);
      if (si.qlen == 0) continue;
      const OwnUnits ou = own_units(si.qlen, si.len, g.prefix, c);
      const int64_t n = g.Hkv * ou.before(ou.nrt);
      if (u < at + n) {
        found[w].seq = q;
        found[w].u = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  if (!works || s.me >= s.n) {
    s.kind = -1;
    return s;
  }
  s.u = share_begin(s.U, s.n, s.me);
  s.end = share_begin(s.U, s.n, s.me + 1);
  if (s.u < PU) {
    s.kind = 0;
    s.seq = 0;
    const int64_t item = quot(s.u, np);
    s.kvh = (int)quot(item, s.npt);
    s.rt = (int)(item - (int64_t)s.kvh * s.npt);
    s.item0 = item * np;
    s.items = np;
    return s;
  }
  if (found[which].seq >= g.nseq) {  // the arrays changed under the call
    s.kind = -1;
    return s;
  }
  s.kind = 1;
  s.seq = found[which].seq;
  s.si = seq_info(g, s.seq);
  if (s.si.qlen <= 0) {
    s.kind = -1;
    return s;
  }
  const OwnUnits ou = own_units(s.si.qlen, s.si.len, g.prefix, c);
  const int64_t per_kvh = ou.before(ou.nrt), x = s.u - found[which].u;
  s.kvh = (int)quot(x, per_kvh);
  const int64_t y = x - s.kvh * per_kvh;
  int lo = 0, hi = ou.nrt;  // before(lo) <= y < before(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ou.before(mid) <= y) lo = mid; else hi = mid;
  }
  s.rt = lo;
  sched_own_item(g, c, s, found[which].u);
  return s;
}

// An own item that begins in a share and goes on: what the join of split items
// reads, one of each worker (ntok 0: none).
struct SplitItem {
  int tok0, ntok, kvh, c1;
};
// the share that holds the last unit of the item a share ends in
__device__ __forceinline__ int split_end(const Sched& s) { return share_owner(s.U, s.n, s.item0 + s.items - 1); }

// The next piece of the share (kind -1: none), and the state behind it.
__device__ __forceinline__ Piece sched_next(const PagedGeom& g, const PagedCut& c, Sched& s) {
  Piece p;
  if (s.kind < 0 || s.u >= s.end) {
    p.kind = -1;
    return p;
  }
  p.kind = s.kind;
  p.share = s.team > 1 ? s.me * s.team + s.rt : s.me;
  p.seq = s.seq;
  p.kvh = s.kvh;
  p.tile0 = (int)max((int64_t)0, s.u - s.item0 - c.fixed);
  const int64_t stop = min(s.end, s.item0 + s.items);
  if (stop - s.item0 <= c.fixed) {  // the share ends before the item's first keys
    p.kind = s.kind = -1;
    return p;
  }
  p.tile1 = (int)(stop - s.item0 - c.fixed);
  p.first = p.tile0 == 0;
  p.last = stop == s.item0 + s.items;
  if (s.kind == 0) {
    p.tok0 = s.rt * c.tpt;
    p.ntok = min(c.tpt, s.ntok_all - p.tok0);
    p.off = 0;
    p.len = g.prefix;
    p.np = 0;
  } else {
    const int t = s.rt * c.tpt;
    p.tok0 = s.si.q0 + t;
    p.ntok = min(c.tpt, s.si.qlen - t);
    p.off = s.si.len - s.si.qlen + t;
    p.len = p.off + p.ntok;
    p.np = c.walk_prefix ? (int)(((int64_t)g.prefix + (1 << c.kt_log2) - 1) >> c.kt_log2) : 0;
  }
  s.u = stop;
  if (s.u < s.end) {  // the item is done: the next one
    const int64_t item_end = s.item0 + s.items;
    if (s.kind == 0) {
      if (s.team > 1) ++s.kvh;
      else if (++s.rt == s.npt) { s.rt = 0; ++s.kvh; }
      s.item0 = item_end;
      if (s.kvh == g.Hkv) sched_next_seq(g, c, s, 0, item_end);
    } else {
      const OwnUnits ou = own_units(s.si.qlen, s.si.len, g.prefix, c);
      if (++s.rt == ou.nrt) { s.rt = 0; ++s.kvh; }
      if (s.kvh == g.Hkv) {
        sched_next_seq(g, c, s, s.seq + 1, item_end);
      } else {
        s.item0 = item_end;
        s.items = ou.before(s.rt + 1) - ou.before(s.rt);
      }
    }
  }
  return p;
}

}  // namespace s2o
