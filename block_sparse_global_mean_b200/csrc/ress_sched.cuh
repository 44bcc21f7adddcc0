// Even shares of ragged work.  An operator over packed sequences has items
// (sequence, head, tile of rows), each a loop over chunks of columns (keys, or
// query rows in the key gradient).  The lengths live on the device, so no host
// can plan the split; every CTA plans it for itself from the same numbers.  An
// item costs item_cost units (its fixed work: first loads, epilogue) and a unit
// per column, in whole chunks.  A worker is a CTA (a warp over the cache's short
// query ranges).
//
// Three ways, chosen from the items' number and costs:
//   rounds  All items cost the same: each is cut into ns equal pieces, and worker w
//           does pieces w, w + grid, ... of (piece 0 of every item, piece 1 of every
//           item, ...).  Workers then read the same columns of all heads and tiles
//           at the same time, so each column comes from memory once (one view
//           against 100 padded ones: 0.58 GB instead of 3.4 GB).
//   pieces  Few items (at most half the workers) of several costs and little work,
//           where latency counts: an item in as many pieces as its cost asks for,
//           a worker does one piece.
//   line    Otherwise: the items stand on one line of units, and worker i owns units
//           [i * share, (i + 1) * share): chunk c of an item belongs to the worker
//           that owns its unit item_cost + chunk * c.  Long items spread over many
//           workers, short ones share one.
//
// Items that several workers touch leave float32 partial results, which a second
// kernel joins in the order of the chunks, so results do not depend on timing.
#pragma once

#include "ress_seq.cuh"

namespace ress {

constexpr int kChunkLog2 = 7;
constexpr int kChunk = 1 << kChunkLog2;   // columns per chunk of the tensor-core walks
// An item's fixed work in the attention walk, in units of a column (a ragged batch
// of 176 items: 89 us at 128, 69 us at 256, 70 us at 640), and the smallest share
// worth a CTA.
constexpr int kItemCost = 256;
constexpr int kMinShare = 512;

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
  int twice_rows;             // sequences of fewer valid rows than this make each pass twice
  int step;                   // the cache's step mask (0: none); needs row_mult 1
  int chunk_log2;             // columns per chunk
  int item_cost, min_share;   // units
  int grid;                   // workers
  int items, ns;              // ns > 0: the host knew the lengths and planned rounds
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

// floor(a / b) for a >= 0, b > 0 and a quotient below 2^24, by an estimate in
// float32 and its correction: a fraction of the instructions of a 64-bit division,
// which matter in the first microsecond of a kernel, when none is cached.
__device__ __forceinline__ int div_small(long long a, long long b) {
  int q = __float2int_rz(__fdividef(__ll2float_rz(a), __ll2float_rz(b)));
  long long r = a - (long long)q * b;
  while (r < 0) --q, r += b;
  while (r >= b) ++q, r -= b;
  return q;
}
__device__ __forceinline__ int ceil_small(long long a, long long b) {
  return div_small(a + b - 1, b);
}

// Items of one sequence: tile t of any head costs base + slope * t units.  A
// step mask makes later tiles longer; its staircase is taken as a line, which
// moves the borders of the shares but not what is computed.
struct SeqCost {
  int tiles;
  long long base, slope;
  int twice;   // 1: each pass is made twice; a piece then takes two chunks at least
  __device__ __forceinline__ long long before(long long t) const {
    return base * t + (slope == 0 ? 0 : slope * (t * (t - 1) / 2));
  }
  __device__ __forceinline__ long long most() const { return base + slope * (tiles - 1); }
  __device__ __forceinline__ int pieces(long long share) const { return ceil_small(most(), share); }
};
// Chunks of `cols` columns.  (Unsigned: a cache row may hold up to 2^31 - 64 tokens,
// and rounding that up to a chunk passes 2^31.)
__device__ __forceinline__ int sched_round_up(const SchedParams& p, int cols) {
  return (int)(((unsigned)cols + (1u << p.chunk_log2) - 1u) >> p.chunk_log2);
}
__device__ __forceinline__ long long sched_chunks_of(const SchedParams& p, int cols,
                                                     int valid_rows) {
  return (long long)sched_round_up(p, cols) * p.mult << (valid_rows < p.twice_rows ? 1 : 0);
}
__device__ __forceinline__ SeqCost sched_cost(const SchedParams& p, const SeqRange& r,
                                              const SeqRange& c) {
  SeqCost s{ceil_small((long long)r.rows * p.row_mult, p.tile_rows), 0, 0,
            r.valid < p.twice_rows ? 1 : 0};
  if (p.step > 0 && p.step < r.rows) {
    s.base = (long long)p.item_cost + max(c.valid - r.rows, 0) + p.tile_rows;
    s.slope = p.tile_rows;
  } else {
    s.base = p.item_cost + (sched_chunks_of(p, c.valid, r.valid) << p.chunk_log2);
  }
  return s;
}
__device__ __forceinline__ SeqCost sched_cost(const SchedParams& p, int b) {
  return sched_cost(p, sched_rows(p, b), sched_cols(p, b));
}

// Chunks whose unit lies before unit x of an item.
__device__ __forceinline__ long long sched_chunks_before(const SchedParams& p, long long x) {
  return x <= p.item_cost ? 0 : (x - p.item_cost + (1 << p.chunk_log2) - 1) >> p.chunk_log2;
}

enum SchedMode { kLine, kPieces, kRounds };
struct SchedPlan {
  SchedMode mode;
  long long share;    // line, pieces: units of a worker, of a piece
  int items, ns;      // rounds
};

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A worker's way through its items, one call of sched_next per item.
struct SchedWalk {
  long long at, ub, seq_start;   // next unit (or piece), end, first one of sequence b
  int b, worker;
};

// Pieces of a sequence, or its units on the line.
__device__ __forceinline__ long long sched_count(const SchedParams& p, const SeqCost& cost,
                                                 SchedMode mode, long long share) {
  if (cost.tiles == 0) return 0;
  return mode == kLine ? cost.before(cost.tiles) * p.heads
                       : (long long)cost.tiles * p.heads * cost.pieces(share);
}

// Upper bound of total / parts, within a millionth of it.
__device__ __forceinline__ long long sched_even(long long total, int parts) {
  return __float2ll_ru(__ll2float_ru(total) * 1.000001f / (float)parts) + 1;
}

// The plan, and where `worker` begins (at == ub: nowhere).  Called by a warp.
__device__ __forceinline__ SchedPlan sched_begin(const SchedParams& p, int worker, SchedWalk* walk) {
  const int lane = threadIdx.x & 31;
  walk->worker = worker;
  if (p.ns > 0) {
    walk->at = worker;
    walk->ub = (long long)p.items * p.ns;
    return SchedPlan{kRounds, 0, p.items, p.ns};
  }
  const bool few = p.seqs <= 32;   // a sequence per lane: its cost stays in registers
  SeqCost cost{0, 0, 0, 0};
  long long units = 0;
  int items = 0;
  for (int b = lane; b < p.seqs; b += 32) {
    cost = sched_cost(p, b);
    items += cost.tiles * p.heads;
    units += cost.before(cost.tiles) * p.heads;
  }
  const bool none = items == 0;
  units = warp_sum(units);
  items = __reduce_add_sync(0xffffffffu, items);
  walk->at = walk->ub = 0;
  SchedPlan plan{kLine, max(sched_even(units, p.grid), (long long)p.min_share), items, 1};
  if (items == 0) return plan;
  const int one = __ffs((int)__ballot_sync(0xffffffffu, !none)) - 1;
  const long long base1 = __shfl_sync(0xffffffffu, cost.base, one);
  const int twice1 = p.twice_rows == 0 ? 0 : __shfl_sync(0xffffffffu, cost.twice, one);
  if (few && __all_sync(0xffffffffu, none || (cost.base == base1 && cost.slope == 0 &&
                                              cost.twice == twice1)) &&
      items < (1 << 20)) {
    // Equal items.  Each lane tries a number of pieces: 1 .. 30, and those that
    // fill one or two rounds.  More than two rounds only of whole items (a worker
    // has two partial slots).
    const int chunks = (int)min((base1 - p.item_cost) >> p.chunk_log2, 1ll << 20);
    int ns = lane < 30 ? lane + 1 : div_small((long long)(lane - 29) * p.grid, items);
    ns = max(1, min(ns, chunks >> twice1));
    const int rounds = ceil_small((long long)items * ns, p.grid);
    // Rounds times an item's fixed work and its chunks, both in chunks.
    long long t = (long long)rounds * (((p.item_cost - 1) >> p.chunk_log2) + 1 + ceil_small(chunks, ns));
    if (ns > 1 && rounds > 2) t = 0xfffffff;
    // The fewest pieces of the shortest.
    const unsigned key = (unsigned)min(t, 0xfffffffll);
    const unsigned best = __reduce_min_sync(0xffffffffu, key);
    const int least = (int)__reduce_min_sync(0xffffffffu, key == best ? (unsigned)ns : 0xffffffffu);
    // The line is fully even, but costs an item's fixed work more.
    if (((long long)best << p.chunk_log2) <= plan.share + (plan.share >> 4) + p.item_cost) {
      plan.ns = least;
      plan.mode = kRounds;
      walk->at = worker;
      walk->ub = (long long)items * least;
      return plan;
    }
  }
  if (2 * items <= p.grid && units <= ((long long)p.grid * 16 << p.chunk_log2)) {
    // Shares that grow until all pieces fit.  sum ceil(cost / share) <= sum cost /
    // share + items, so the last one is sure to.
    plan.mode = kPieces;
    for (int i = 0; i < 9; ++i) {
      int n = 0;
      long long cap = 0;
      for (int b = lane; b < p.seqs; b += 32) {
        if (!few) cost = sched_cost(p, b);
        n += (int)sched_count(p, cost, kPieces, plan.share);
        cap += (long long)cost.tiles * p.heads * cost.most();
      }
      if (__reduce_add_sync(0xffffffffu, n) <= p.grid) break;
      plan.share = i < 7 ? plan.share + (plan.share >> 4)
                         : max(plan.share, sched_even(warp_sum(cap), p.grid - items));
    }
  }
  const long long unit = plan.mode == kLine ? worker * plan.share : worker;
  long long base = 0;
  for (int b0 = 0; b0 < p.seqs; b0 += 32) {
    const int b = b0 + lane;
    if (!few && b < p.seqs) cost = sched_cost(p, b);
    const long long n = b < p.seqs ? sched_count(p, cost, plan.mode, plan.share) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned behind = __ballot_sync(0xffffffffu, base + incl > unit);
    if (behind != 0) {
      const int l = __ffs((int)behind) - 1;
      walk->b = b0 + l;
      walk->seq_start = base + __shfl_sync(0xffffffffu, incl - n, l);
      walk->at = unit;
      walk->ub = plan.mode == kLine ? min(unit + plan.share, units) : unit + 1;
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return plan;
}

// The same choice on the host, where one sequence of known length needs none on the
// device (five queries against 1374 states: 14.0 -> 11.8 us).
inline void sched_plan_on_host(SchedParams* p) {
  p->items = p->ns = 0;
  if (p->row_off || p->col_off || p->col_lens || p->lengths || p->step || p->seqs != 1) return;
  const long long chunk = 1ll << p->chunk_log2;
  if (p->row_lens && p->twice_rows > 0) return;
  const int twice = p->rows < p->twice_rows ? 1 : 0;
  const long long chunks = (p->cols + chunk - 1) / chunk * p->mult << twice;
  const long long items =
      ((long long)p->rows * p->row_mult + p->tile_rows - 1) / p->tile_rows * p->heads;
  if (items == 0 || items >= (1 << 20)) return;
  const long long fixed = (p->item_cost + chunk - 1) / chunk;
  const long long units = items * (p->item_cost + chunks * chunk);
  long long best = 1ll << 60, share = (units + p->grid - 1) / p->grid;
  int best_ns = 1;
  for (int i = 0; i < 32; ++i) {
    long long ns = i < 30 ? i + 1 : (i - 29) * (long long)p->grid / items;
    ns = ns > chunks >> twice ? chunks >> twice : ns;
    ns = ns < 1 ? 1 : ns;
    const long long rounds = (items * ns + p->grid - 1) / p->grid;
    if (ns > 1 && rounds > 2) continue;
    const long long t = rounds * (fixed + (chunks + ns - 1) / ns);
    if (t < best || (t == best && ns < best_ns)) best = t, best_ns = (int)ns;
  }
  share = share < p->min_share ? p->min_share : share;
  if (best * chunk > share + (share >> 4) + p->item_cost) return;
  p->items = (int)items;
  p->ns = best_ns;
}

// The item at a unit of a sequence on the line.
struct SchedItem {
  int head, tile;
  long long start, cost;   // first unit, units
};
__device__ __forceinline__ SchedItem sched_item(const SeqCost& s, long long seq_start,
                                                long long u) {
  const long long per_head = s.before(s.tiles);
  const long long r = u - seq_start;
  SchedItem it;
  it.head = div_small(r, per_head);
  const long long x = r - it.head * per_head;
  long long t;
  if (s.slope == 0) {
    t = div_small(x, s.base);
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
// result goes to the outputs); 2: a part, to the worker's partial slot `slot`.
struct Segment {
  int kind, slot;
  int b, head, tile;
  int row_start, rows, rows_valid;
  int col_start, cols_valid;
  int c0, c1;              // chunks
  int parts, stride;       // of an item's first part: its parts, and from one to the next
};

__device__ __forceinline__ long long sched_chunks(const SchedParams& p, const SeqRange& r,
                                                  const SeqRange& c, int tile) {
  if (p.step == 0) return sched_chunks_of(p, c.valid, r.valid);
  const int last = min((tile + 1) * p.tile_rows, r.rows) - 1;
  return sched_round_up(p, step_end(c.valid, r.rows, last, p.step));
}

// Piece `piece` of `ns` of an item's chunks.
__device__ __forceinline__ void sched_piece(Segment& g, long long chunks, int piece, int ns) {
  const int q = ns == 1 ? (int)chunks : div_small(chunks, ns), rest = (int)chunks - q * ns;
  g.c0 = q * piece + min(piece, rest);   // the first `rest` get one more
  g.c1 = g.c0 + q + (piece < rest ? 1 : 0);
  g.kind = ns == 1 ? 1 : 2;
  if (piece == 0 && ns > 1) g.parts = ns;
}

__device__ __forceinline__ Segment sched_next(const SchedParams& p, const SchedPlan& plan,
                                              SchedWalk& w) {
  Segment g;
  g.kind = g.slot = g.parts = 0;
  g.stride = 1;
  if (w.at >= w.ub) return g;
  int piece = 0, item = 0;
  if (plan.mode == kRounds) {   // the sequence of the item: they differ in their tiles alone
    piece = plan.ns == 1 ? 0 : div_small(w.at, plan.items);
    item = (int)w.at - piece * plan.items;
    g.slot = w.at >= p.grid ? 1 : 0;   // of whole items, where there may be more rounds, unused
    g.stride = plan.items;
    w.at += p.grid;
    w.b = 0;
    if (p.seqs > 1)
      for (;; ++w.b) {
        const int n = sched_cost(p, w.b).tiles * p.heads;
        if (item < n) break;
        item -= n;
      }
  }
  for (;;) {
    const SeqRange r = sched_rows(p, w.b), c = sched_cols(p, w.b);
    const SeqCost s = sched_cost(p, r, c);
    if (plan.mode != kLine) {
      int ns = plan.ns;
      if (plan.mode == kPieces) {
        ns = s.pieces(plan.share);
        const int at = (int)(w.at - w.seq_start);   // at most grid, as ns
        item = div_small(at, ns);
        piece = at - item * ns;
        w.at = w.ub;
      }
      g.head = div_small(item, s.tiles);
      g.tile = item - g.head * s.tiles;
      sched_piece(g, sched_chunks(p, r, c, g.tile), piece, ns);
    } else {
      const long long n = s.before(s.tiles) * p.heads;
      if (w.at >= w.seq_start + n) {   // the sequence is done (or has no rows)
        w.seq_start += n;
        if (++w.b >= p.seqs) return g;
        continue;
      }
      const SchedItem it = sched_item(s, w.seq_start, w.at);
      g.head = it.head;
      g.tile = it.tile;
      const long long x0 = w.at - it.start;
      const long long x1 = min(w.ub - it.start, it.cost);
      const long long chunks = sched_chunks(p, r, c, g.tile);
      g.c0 = (int)min(sched_chunks_before(p, x0), chunks);
      g.c1 = (int)(x1 == it.cost ? chunks : min(sched_chunks_before(p, x1), chunks));
      g.kind = x0 == 0 && x1 == it.cost ? 1 : 2;
      if (x0 == 0 && g.kind == 2) {   // an end or middle is a worker's first, a beginning its last
        g.slot = 1;
        g.parts = div_small(it.start + it.cost - 1, plan.share) - w.worker + 1;
      }
      w.at = it.start + x1;
    }
    g.b = w.b;
    g.row_start = r.start;
    g.rows = r.rows;
    g.rows_valid = r.valid;
    g.col_start = c.start;
    g.cols_valid = c.valid;
    return g;
  }
}

// What the second kernel joins: the item whose first part is worker i's (record
// i of the workspace), if it has others (head < 0: none).  Part k is at stop
// i + k * stride: worker stop % grid, slot stop / grid; on the line (stride 1) the
// first part is in slot `slot`.
struct SplitItem {
  int head, tile, slot, parts;
  int row_start, rows, stride, pad;
};
__device__ __forceinline__ SplitItem no_split() { return SplitItem{-1, 0, 0, 0, 0, 0, 0, 0}; }
__device__ __forceinline__ SplitItem split_of(const Segment& g) {
  return SplitItem{g.head, g.tile, g.slot, g.parts, g.row_start, g.rows, g.stride, 0};
}
__device__ __forceinline__ void store_split(SplitItem* at, const SplitItem& s) {
  reinterpret_cast<int4*>(at)[0] = make_int4(s.head, s.tile, s.slot, s.parts);
  reinterpret_cast<int4*>(at)[1] = make_int4(s.row_start, s.rows, s.stride, 0);
}
__device__ __forceinline__ SplitItem load_split(const SplitItem* at) {
  const int4 a = reinterpret_cast<const int4*>(at)[0], b = reinterpret_cast<const int4*>(at)[1];
  return SplitItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, 0};
}
// Partial slot (2 worker + slot) of part k.
__device__ __forceinline__ size_t part_slot(const SplitItem& it, int first, int grid, int k) {
  if (k == 0) return (size_t)first * 2 + it.slot;
  const int stop = first + k * it.stride;
  const int round = stop >= grid ? 1 : 0;   // at most two rounds, and none on the line
  return (size_t)(stop - round * grid) * 2 + round;
}

// Partial results of attention: per row a maximum (log2 domain) and a sum in
// part_ml, and 64 unnormalised outputs in part_o; rows of worker w's slot s start
// at (2 w + s) * tile_rows.
//
// Parts stripe, stripe + stripes, ... of one row, by 16 lanes
// with four dimensions each.  Four parts are loaded at once, before their weights
// are known.
struct JoinedRow {
  float m, l;
  float4 o;   // dimensions 4 (lane % 16) ..
};
__device__ __forceinline__ void add_part(JoinedRow& j, float f, float l, const float4& x) {
  j.l = fmaf(f, l, j.l);
  j.o.x = fmaf(f, x.x, j.o.x);
  j.o.y = fmaf(f, x.y, j.o.y);
  j.o.z = fmaf(f, x.z, j.o.z);
  j.o.w = fmaf(f, x.w, j.o.w);
}
__device__ __forceinline__ JoinedRow join_row(const SplitItem& it, int first, int grid,
                                              const float2* part_ml, const float* part_o,
                                              int tile_rows, int row,
                                              int stripe, int stripes) {
  const int lane = threadIdx.x & 15;
  JoinedRow j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int k0 = stripe; k0 < it.parts; k0 += 4 * stripes) {
    float2 ml[4];
    float4 x[4];
    float m = j.m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + i * stripes;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (k < it.parts) {
        const size_t part = part_slot(it, first, grid, k) * tile_rows + row;
        ml[i] = part_ml[part];
        x[i] = reinterpret_cast<const float4*>(part_o + part * 64)[lane];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, ml[i].x);
    if (m == -INFINITY) continue;
    const float a = fast_exp2(j.m - m);
    j.l *= a, j.o.x *= a, j.o.y *= a, j.o.z *= a, j.o.w *= a;
#pragma unroll
    for (int i = 0; i < 4; ++i)   // without a key of the row its outputs were not written
      if (ml[i].x != -INFINITY) add_part(j, fast_exp2(ml[i].x - m), ml[i].y, x[i]);
    j.m = m;
  }
  return j;
}

__device__ __forceinline__ void write_row(const JoinedRow& j, __nv_bfloat16* out, float* lse) {
  const int lane = threadIdx.x & 15;
  const bool empty = j.m == -INFINITY;
  const float inv = empty ? 0.f : 1.0f / j.l;
  reinterpret_cast<uint2*>(out)[lane] =
      make_uint2(pack_bf16x2(j.o.x * inv, j.o.y * inv), pack_bf16x2(j.o.z * inv, j.o.w * inv));
  if (lane == 0 && lse != nullptr)
    *lse = empty ? -INFINITY : (j.m + __log2f(j.l)) * 0.6931471805599453f;
}

// Rows [r0, n) of a split item, live where out_of(row) is not null, by a CTA of
// kTeams half warps.  Few rows: several half warps share a row's parts.
template <int kTeams, typename OutOf, typename LseOf>
__device__ __forceinline__ void join_item(const SplitItem& it, int first, int grid,
                                          const float2* part_ml, const float* part_o, int tile_rows, int r0, int n,
                                          OutOf out_of, LseOf lse_of) {
  __shared__ float4 s_o[kTeams][16];
  __shared__ float2 s_ml[kTeams];
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
  int stripes = 1;
  while (stripes < kTeams && (n - r0) * stripes * 2 <= kTeams && stripes * 4 < it.parts) stripes *= 2;
  const int stripe = team % stripes;
  for (; r0 < n; r0 += kTeams / stripes) {
    const int r = r0 + team / stripes;
    __nv_bfloat16* out = r < n ? out_of(r) : nullptr;
    JoinedRow j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (out != nullptr) j = join_row(it, first, grid, part_ml, part_o, tile_rows, r, stripe, stripes);
    if (stripes == 1) {
      if (out != nullptr) write_row(j, out, lse_of(r));
      continue;
    }
    __syncthreads();
    s_o[team][lane] = j.o;
    if (lane == 0) s_ml[team] = make_float2(j.m, j.l);
    __syncthreads();
    if (stripe == 0 && out != nullptr) {
      float m = -INFINITY;
      for (int i = 0; i < stripes; ++i) m = fmaxf(m, s_ml[team + i].x);
      JoinedRow t{m, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      if (m != -INFINITY)
        for (int i = 0; i < stripes; ++i)
          add_part(t, fast_exp2(s_ml[team + i].x - m), s_ml[team + i].y, s_o[team + i][lane]);
      write_row(t, out, lse_of(r));
    }
  }
}

}  // namespace ress
