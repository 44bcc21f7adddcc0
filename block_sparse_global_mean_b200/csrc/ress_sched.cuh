// Even shares of ragged work.  An operator over packed sequences has items
// (sequence, head, tile of rows), each a loop over chunks of columns (keys, or
// query rows in the key gradient).  The lengths live on the device, so no host
// can plan the split.  Instead all items stand on one line of work units: an
// item is item_cost units (its fixed work: first loads, epilogue) and a unit per
// column, in whole chunks.  Worker i (a CTA; a warp over the cache's short
// query ranges) owns units [i * share, (i + 1) * share), and chunk c of an item
// belongs to the worker that owns its unit item_cost + chunk * c.  Items cut by a
// share's end leave float32 partial results, which a second kernel joins in the
// order of the chunks, so results do not depend on timing.  Long items are split
// over many workers, short ones share one, and one rule serves one row against
// 140,800 keys and thousands of rows alike.
#pragma once

#include "ress_seq.cuh"

namespace ress {

constexpr int kChunk = 128;       // columns per chunk of the tensor-core walks
constexpr int kItemCost = 256;    // an item's fixed work there, in units of a column
constexpr int kMinShare = 512;    // smallest share worth a CTA

struct SchedParams {
  DeviceError* err;
  const int32_t* row_off;     // packed rows (NULL: one sequence)
  const int32_t* row_lens;
  const int32_t* col_off;     // packed columns
  const int32_t* col_lens;
  const int32_t* lengths;     // the cache: columns of a request (col_off unused)
  int rows, cols;             // rows and columns in all
  int row_detail, col_detail; // error details of bad offsets
  int seqs, heads;
  int row_mult;               // item rows per sequence row
  int tile_rows;              // item rows of a tile
  int mult;                   // passes over the columns (query heads of a key head)
  int step;                   // the cache's step mask (0: none); needs row_mult 1
  int chunk, item_cost, min_share;
  int grid;                   // workers
  long long max_len;          // largest valid entry of `lengths`
};

__device__ __forceinline__ SeqRange sched_rows(const SchedParams& p, int b) {
  return seq_range(p.row_off, p.row_lens, b, p.rows, p.err, p.row_detail);
}
__device__ __forceinline__ SeqRange sched_cols(const SchedParams& p, int b) {
  if (p.lengths == nullptr)
    return seq_range(p.col_off, p.col_lens, b, p.cols, p.err, p.col_detail);
  int len = p.lengths[b];
  if (len < 0 || len > p.max_len) {
    raise_device_error(p.err, RESS_ERR_BAD_INDEX, 94);
    len = len < 0 ? 0 : (int)p.max_len;
  }
  return SeqRange{0, len, len};
}

// Items of one sequence: tile t of any head costs base + slope * t units.  A
// step mask makes later tiles longer; its staircase is taken as a line, which
// moves the borders of the shares but not what is computed.
struct SeqCost {
  int tiles;
  long long base, slope;
  __device__ __forceinline__ long long before(long long t) const {
    return base * t + slope * (t * (t - 1) / 2);
  }
};
__device__ __forceinline__ SeqCost sched_cost(const SchedParams& p, const SeqRange& r,
                                              const SeqRange& c) {
  SeqCost s{(int)(((long long)r.rows * p.row_mult + p.tile_rows - 1) / p.tile_rows), 0, 0};
  if (p.step > 0 && p.step < r.rows) {
    s.base = p.item_cost + max(c.valid - r.rows, 0) + p.tile_rows;
    s.slope = p.tile_rows;
  } else {
    s.base = p.item_cost + (long long)((c.valid + p.chunk - 1) / p.chunk) * p.chunk * p.mult;
  }
  return s;
}

// Chunks whose unit lies before unit x of an item.
__device__ __forceinline__ long long sched_chunks_before(const SchedParams& p, long long x) {
  return x <= p.item_cost ? 0 : (x - p.item_cost + p.chunk - 1) / p.chunk;
}

struct SchedShared {
  long long warp_sum[32];
  long long total, start;   // all units; first unit of sequence b
  int b;
};

// Units in all (sh->total) and the sequence that holds unit `u` (sh->b, -1 if
// none; its first unit sh->start).  `u` may depend on the total: it is taken
// from `pick(total)`.  Called by all threads of the CTA; ends in a barrier.
template <typename Pick>
__device__ __forceinline__ void sched_find(const SchedParams& p, SchedShared* sh, Pick pick) {
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.seqs + threads - 1) / threads;
  const int b0 = min(p.seqs, (int)threadIdx.x * per), b1 = min(p.seqs, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqCost s = sched_cost(p, sched_rows(p, b), sched_cols(p, b));
    mine += s.before(s.tiles) * p.heads;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  if (threadIdx.x == 0) sh->b = -1;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) before += sh->warp_sum[w];
    total += sh->warp_sum[w];
  }
  if (threadIdx.x == 0) sh->total = total;
  const long long u = pick(total);
  if (u >= before && u < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const SeqCost s = sched_cost(p, sched_rows(p, b), sched_cols(p, b));
      const long long n = s.before(s.tiles) * p.heads;
      if (u < at + n) {
        sh->b = b;
        sh->start = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
}

// The same for workers that are warps: `before` (one entry per thread of the
// CTA) gets the units before each thread's sequences, and each warp then looks
// up its own unit.
__device__ __forceinline__ long long sched_prefix(const SchedParams& p, long long* warp_sum,
                                                  long long* before) {
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.seqs + threads - 1) / threads;
  const int b0 = min(p.seqs, (int)threadIdx.x * per), b1 = min(p.seqs, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqCost s = sched_cost(p, sched_rows(p, b), sched_cols(p, b));
    mine += s.before(s.tiles) * p.heads;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long base = 0, total = 0;
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  before[threadIdx.x] = base + incl - mine;
  __syncthreads();
  return total;
}
// Sequence of unit u (< total) and its first unit.
__device__ __forceinline__ void sched_locate(const SchedParams& p, const long long* before,
                                             long long u, int* b, long long* start) {
  const int threads = blockDim.x, lane = threadIdx.x & 31;
  int slot = -1;   // last entry <= u that is not followed by an equal one
  for (int i = 0; i < threads; i += 32)
    slot += __popc(__ballot_sync(0xffffffffu, before[i + lane] <= u));
  const int per = (p.seqs + threads - 1) / threads;
  long long at = before[slot];
  int s = slot * per;
  for (; s < p.seqs; ++s) {
    const SeqCost c = sched_cost(p, sched_rows(p, s), sched_cols(p, s));
    const long long n = c.before(c.tiles) * p.heads;
    if (u < at + n) break;
    at += n;
  }
  *b = s;
  *start = at;
}

__device__ __forceinline__ long long sched_share(const SchedParams& p, long long total) {
  const long long s = (total + p.grid - 1) / p.grid;
  return s < p.min_share ? p.min_share : s;
}

// The item at a unit of a sequence.
struct SchedItem {
  int b, head, tile;
  long long start, cost;   // first unit, units
};
__device__ __forceinline__ SchedItem sched_item(const SeqCost& s, int b, long long seq_start,
                                                long long u) {
  const long long per_head = s.before(s.tiles);
  const long long r = u - seq_start;
  SchedItem it;
  it.b = b;
  it.head = (int)(r / per_head);
  const long long x = r - it.head * per_head;
  long long t;
  if (s.slope == 0) {
    t = x / s.base;
  } else {   // last t with before(t) <= x
    long long lo = 0, hi = s.tiles - 1;
    while (lo < hi) {
      const long long mid = (lo + hi + 1) >> 1;
      if (s.before(mid) <= x) lo = mid;
      else hi = mid - 1;
    }
    t = lo;
  }
  it.tile = (int)t;
  it.start = seq_start + it.head * per_head + s.before(t);
  it.cost = s.base + s.slope * t;
  return it;
}

// What a worker does of one item.  kind 0: nothing is left; 1: all of it (the
// result goes to the outputs); 2: its end or middle (partial slot 0 of the
// worker); 3: its beginning (partial slot 1).
struct Segment {
  int kind;
  int b, head, tile;
  int row_start, rows, rows_valid;
  int col_start, cols_valid;
  int c0, c1;              // chunks
  int pad;
};

// Walks the items of units [ua, ub), one call per item (one thread).
struct SchedWalk {
  long long at, ub, seq_start;
  int b;
};
__device__ __forceinline__ Segment sched_next(const SchedParams& p, SchedWalk& w) {
  Segment g;
  g.kind = 0;
  if (w.at >= w.ub) return g;
  for (;;) {
    const SeqRange r = sched_rows(p, w.b), c = sched_cols(p, w.b);
    const SeqCost s = sched_cost(p, r, c);
    const long long n = s.before(s.tiles) * p.heads;
    if (w.at >= w.seq_start + n) {   // the sequence is done (or has no rows)
      w.seq_start += n;
      if (++w.b >= p.seqs) return g;
      continue;
    }
    const SchedItem it = sched_item(s, w.b, w.seq_start, w.at);
    const long long x0 = w.at - it.start;
    const long long x1 = min(w.ub - it.start, it.cost);
    long long chunks = (long long)((c.valid + p.chunk - 1) / p.chunk) * p.mult;
    if (p.step > 0) {
      const int last = min((it.tile + 1) * p.tile_rows, r.rows) - 1;
      chunks = (step_end(c.valid, r.rows, last, p.step) + p.chunk - 1) / p.chunk;
    }
    g.b = w.b;
    g.head = it.head;
    g.tile = it.tile;
    g.row_start = r.start;
    g.rows = r.rows;
    g.rows_valid = r.valid;
    g.col_start = c.start;
    g.cols_valid = c.valid;
    g.c0 = (int)min(sched_chunks_before(p, x0), chunks);
    g.c1 = x1 == it.cost ? (int)chunks : (int)min(sched_chunks_before(p, x1), chunks);
    g.kind = x0 > 0 ? 2 : x1 == it.cost ? 1 : 3;
    w.at = it.start + x1;
    return g;
  }
}

// The item that CTA `cta` begins and does not end (head < 0: none), with the
// last CTA that works on it.  All threads call it; the result is uniform.
struct SplitItem {
  int b, head, tile, last_cta;
};
__device__ __forceinline__ SplitItem sched_split_item(const SchedParams& p, SchedShared* sh,
                                                      int cta) {
  SplitItem r{0, -1, 0, 0};
  long long share = 0;
  sched_find(p, sh, [&](long long total) {
    share = sched_share(p, total);
    return (cta + 1) * share - 1 < total ? (cta + 1) * share - 1 : total - 1;
  });
  const int b = sh->b;
  if (b < 0) return r;
  const long long ua = cta * share, ub = min(ua + share, sh->total);
  if (ua >= sh->total) return r;
  const SeqCost s = sched_cost(p, sched_rows(p, b), sched_cols(p, b));
  const SchedItem it = sched_item(s, b, sh->start, ub - 1);
  if (it.start < ua || it.start + it.cost <= ub) return r;
  r.b = b;
  r.head = it.head;
  r.tile = it.tile;
  r.last_cta = (int)((it.start + it.cost - 1) / share);
  return r;
}

}  // namespace ress
