// Even shares of ragged work.  An operator over packed sequences has items
// (sequence, head, tile of rows), each a loop over chunks of columns (keys, or
// query rows in the key gradient).  The lengths live on the device, so no host
// can plan the split; every CTA plans it for itself from the same numbers.  An
// item costs item_cost units (its fixed work: first loads, epilogue) and a unit
// per column, in whole chunks.  A worker is a CTA (a warp over the cache's short
// query ranges).
//
// Few items (at most half the workers), where latency counts: an item is cut
// into equal pieces, as many as its cost asks for, and a worker does one piece.
// More items: they stand on one line of units, and worker i owns units [i *
// share, (i + 1) * share): chunk c of an item belongs to the worker that owns
// its unit item_cost + chunk * c.  Long items spread over many workers, short
// ones share one.
//
// Items that several workers touch leave float32 partial results, which a second
// kernel joins in the order of the chunks, so results do not depend on timing.
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
  __device__ __forceinline__ long long most() const { return base + slope * (tiles - 1); }
  __device__ __forceinline__ int pieces(long long share) const;
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
__device__ __forceinline__ SeqCost sched_cost(const SchedParams& p, int b) {
  return sched_cost(p, sched_rows(p, b), sched_cols(p, b));
}

// Chunks whose unit lies before unit x of an item.
__device__ __forceinline__ long long sched_chunks_before(const SchedParams& p, long long x) {
  return x <= p.item_cost ? 0 : (x - p.item_cost + p.chunk - 1) / p.chunk;
}

// a / b for a >= 0, b > 0, in 32 bits where they fit (a third of the time).
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

__device__ __forceinline__ int SeqCost::pieces(long long share) const {
  return (int)div_pos(most() + share - 1, share);
}

struct SchedPlan {
  bool pieces;        // which of the two ways
  long long share;
};

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A worker's way through its items, one call of sched_next per item.
struct SchedWalk {
  long long at, ub, seq_start;   // next unit (or piece), end, first one of sequence b
  int b;
};

// The plan, and where `worker` begins (at == ub: nowhere).  Called by a warp.
__device__ __forceinline__ SchedPlan sched_begin(const SchedParams& p, int worker, SchedWalk* walk) {
  const int lane = threadIdx.x & 31;
  SeqCost cost{0, 0, 0};
  long long units = 0, items = 0, most = 0;
  for (int b = lane; b < p.seqs; b += 32) {
    cost = sched_cost(p, b);
    const long long n = (long long)cost.tiles * p.heads;
    items += n;
    most += n * cost.most();
    units += cost.before(cost.tiles) * p.heads;
  }
  items = warp_sum(items);
  SchedPlan plan;
  plan.pieces = 2 * items <= p.grid;
  // Pieces: every item in ceil(cost / share), at most grid in all.
  units = warp_sum(plan.pieces ? most : units);
  const long long workers = plan.pieces ? p.grid - items : p.grid;
  plan.share = max(div_pos(units + workers - 1, workers), (long long)p.min_share);
  walk->at = plan.pieces ? worker : worker * plan.share;
  walk->ub = walk->at;
  long long base = 0;
  for (int b0 = 0; b0 < p.seqs; b0 += 32) {
    const int b = b0 + lane;
    if (p.seqs > 32 && b < p.seqs) cost = sched_cost(p, b);
    long long n = 0;
    if (b < p.seqs && cost.tiles > 0)
      n = plan.pieces ? (long long)cost.tiles * p.heads * cost.pieces(plan.share)
                      : cost.before(cost.tiles) * p.heads;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned behind = __ballot_sync(0xffffffffu, base + incl > walk->at);
    if (behind != 0) {
      const int l = __ffs((int)behind) - 1;
      walk->b = b0 + l;
      walk->seq_start = base + __shfl_sync(0xffffffffu, incl - n, l);
      // The walk ends with the work; without pieces it may go on behind this batch.
      walk->ub = plan.pieces ? walk->at + 1 : min(walk->at + plan.share, units);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return plan;
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
  it.head = (int)div_pos(r, per_head);
  const long long x = r - it.head * per_head;
  long long t;
  if (s.slope == 0) {
    t = div_pos(x, s.base);
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
// result goes to the outputs); 2: a piece, or an end or middle (partial slot 0
// of the worker); 3: a beginning on the line (partial slot 1).
struct Segment {
  int kind;
  int b, head, tile;
  int row_start, rows, rows_valid;
  int col_start, cols_valid;
  int c0, c1;              // chunks
  int last;                // of the worker with the item's first part: who has its last (else -1)
};

__device__ __forceinline__ long long sched_chunks(const SchedParams& p, const SeqRange& r,
                                                  const SeqRange& c, int tile) {
  if (p.step > 0) {
    const int last = min((tile + 1) * p.tile_rows, r.rows) - 1;
    return (step_end(c.valid, r.rows, last, p.step) + p.chunk - 1) / p.chunk;
  }
  return (long long)((c.valid + p.chunk - 1) / p.chunk) * p.mult;
}

__device__ __forceinline__ Segment sched_next(const SchedParams& p, const SchedPlan& plan,
                                              SchedWalk& w) {
  Segment g;
  g.kind = 0;
  if (w.at >= w.ub) return g;
  for (;;) {
    const SeqRange r = sched_rows(p, w.b), c = sched_cols(p, w.b);
    const SeqCost s = sched_cost(p, r, c);
    g.last = -1;
    if (plan.pieces) {
      const int ns = s.pieces(plan.share), at = (int)(w.at - w.seq_start);   // both at most grid
      const int item = at / ns, piece = at - item * ns;
      g.head = item / s.tiles;
      g.tile = item - g.head * s.tiles;
      const unsigned chunks = (unsigned)sched_chunks(p, r, c, g.tile), q = chunks / (unsigned)ns;
      const unsigned rest = chunks - q * (unsigned)ns;   // the first `rest` pieces get one more
      g.c0 = (int)(q * piece + min((unsigned)piece, rest));
      g.c1 = g.c0 + (int)(q + ((unsigned)piece < rest ? 1u : 0u));
      g.kind = ns == 1 ? 1 : 2;
      if (piece == 0 && ns > 1) g.last = (int)w.at + ns - 1;
      w.at = w.ub;
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
      g.kind = x0 > 0 ? 2 : x1 == it.cost ? 1 : 3;
      if (g.kind == 3) g.last = (int)div_pos(it.start + it.cost - 1, plan.share);
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
// i of the workspace), if other workers go on with it (head < 0: none).  Its parts
// are (i, slot), then (w, 0) up to w = last.
struct SplitItem {
  int head, tile, slot, last;
  int row_start, rows, pad0, pad1;
};
__device__ __forceinline__ SplitItem split_of(const Segment& g) {
  return SplitItem{g.head, g.tile, g.kind == 3 ? 1 : 0, g.last, g.row_start, g.rows, 0, 0};
}
__device__ __forceinline__ void store_split(SplitItem* at, const SplitItem& s) {
  reinterpret_cast<int4*>(at)[0] = make_int4(s.head, s.tile, s.slot, s.last);
  reinterpret_cast<int4*>(at)[1] = make_int4(s.row_start, s.rows, 0, 0);
}
__device__ __forceinline__ SplitItem load_split(const SplitItem* at) {
  const int4 a = reinterpret_cast<const int4*>(at)[0], b = reinterpret_cast<const int4*>(at)[1];
  return SplitItem{a.x, a.y, a.z, a.w, b.x, b.y, 0, 0};
}

// Partial results of attention: per row a maximum (log2 domain) and a sum in
// part_ml, and 64 unnormalised outputs in part_o; rows of worker w's slot s start
// at (2 w + s) * tile_rows.
struct JoinedRow {
  float m, l;
  float2 o;   // dimensions 2 lane, 2 lane + 1
};
// Parts first + stripe, first + stripe + stripes, ... of one row (a warp).  The
// outputs of eight parts are loaded at once, before the weights are known.
__device__ __forceinline__ JoinedRow join_row(const SplitItem& it, int first, const float2* part_ml,
                                              const float* part_o, int tile_rows, int row,
                                              int stripe, int stripes) {
  const int lane = threadIdx.x & 31;
  JoinedRow j{-INFINITY, 0.f, make_float2(0.f, 0.f)};
  for (int w0 = first + stripe; w0 <= it.last; w0 += 8 * stripes) {
    float2 ml[8], x[8];
    float m = j.m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int w = w0 + i * stripes;
      ml[i] = make_float2(-INFINITY, 0.f);
      x[i] = make_float2(0.f, 0.f);
      if (w <= it.last) {
        const size_t part = ((size_t)w * 2 + (w == first ? it.slot : 0)) * tile_rows + row;
        ml[i] = part_ml[part];
        x[i] = reinterpret_cast<const float2*>(part_o + part * 64)[lane];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, ml[i].x);
    if (m == -INFINITY) continue;
    const float a = fast_exp2(j.m - m);
    j.l *= a, j.o.x *= a, j.o.y *= a;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (ml[i].x != -INFINITY) {   // otherwise its outputs were not written
        const float f = fast_exp2(ml[i].x - m);
        j.l = fmaf(f, ml[i].y, j.l);
        j.o.x = fmaf(f, x[i].x, j.o.x);
        j.o.y = fmaf(f, x[i].y, j.o.y);
      }
    j.m = m;
  }
  return j;
}

__device__ __forceinline__ void write_row(const JoinedRow& j, __nv_bfloat16* out, float* lse) {
  const int lane = threadIdx.x & 31;
  const bool empty = j.m == -INFINITY;
  const float inv = empty ? 0.f : 1.0f / j.l;
  reinterpret_cast<uint32_t*>(out)[lane] = pack_bf16x2(j.o.x * inv, j.o.y * inv);
  if (lane == 0 && lse != nullptr)
    *lse = empty ? -INFINITY : (j.m + __log2f(j.l)) * 0.6931471805599453f;
}

// The rows [0, n) of a split item, live where `out_of(row)` is not null, by all
// warps of a CTA.  Few rows: several warps share a row's parts.
template <int kWarps, typename OutOf, typename LseOf>
__device__ __forceinline__ void join_item(const SplitItem& it, int first, const float2* part_ml,
                                          const float* part_o, int tile_rows, int n, OutOf out_of,
                                          LseOf lse_of) {
  __shared__ float2 s_o[kWarps][32];
  __shared__ float2 s_ml[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = it.last - first + 1;
  int stripes = 1;
  while (stripes < kWarps && n * stripes * 2 <= kWarps && stripes * 8 < parts) stripes *= 2;
  const int rows_at_once = kWarps / stripes;
  const int stripe = warp % stripes;
  for (int r0 = 0; r0 < n; r0 += rows_at_once) {
    const int r = r0 + warp / stripes;
    __nv_bfloat16* out = r < n ? out_of(r) : nullptr;
    JoinedRow j{-INFINITY, 0.f, make_float2(0.f, 0.f)};
    if (out != nullptr) j = join_row(it, first, part_ml, part_o, tile_rows, r, stripe, stripes);
    if (stripes == 1) {
      if (out != nullptr) write_row(j, out, lse_of(r));
      continue;
    }
    __syncthreads();
    s_o[warp][lane] = j.o;
    if (lane == 0) s_ml[warp] = make_float2(j.m, j.l);
    __syncthreads();
    if (stripe == 0 && out != nullptr) {
      float m = -INFINITY;
      for (int i = 0; i < stripes; ++i) m = fmaxf(m, s_ml[warp + i].x);
      JoinedRow t{m, 0.f, make_float2(0.f, 0.f)};
      if (m != -INFINITY)
        for (int i = 0; i < stripes; ++i) {
          const float f = fast_exp2(s_ml[warp + i].x - m);
          t.l = fmaf(f, s_ml[warp + i].y, t.l);
          t.o.x = fmaf(f, s_o[warp + i][lane].x, t.o.x);
          t.o.y = fmaf(f, s_o[warp + i][lane].y, t.o.y);
        }
      write_row(t, out, lse_of(r));
    }
  }
}

// Programmatic dependent launch: the second kernel of an operator is launched
// while the first still runs, plans its work, and waits here for the first
// one's results.
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void allow_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename Kernel, typename... Args>
cudaError_t launch_dependent(Kernel kernel, dim3 grid, dim3 block, cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace ress
