// Packed sequences on the device: the rows of a sequence, and the (sequence,
// tile) that a CTA of a ragged grid works on.  Offsets and lengths live in
// device memory, so every kernel checks them as it reads them.
#pragma once

#include "ress_common.cuh"

namespace ress {

// Rows start .. start + rows - 1 of a packed tensor; the first `valid` carry data.
struct SeqRange {
  int start;
  int rows;
  int valid;
};

// Sequence b of `off` (NULL: one sequence of all n rows).  Offsets out of
// 0..n or descending make the sequence empty (error `detail`), a length
// outside it is clamped (error `detail` + 2).
__device__ __forceinline__ SeqRange seq_range(const int32_t* off, const int32_t* lens, int b,
                                              int n, DeviceError* err, int detail) {
  SeqRange s{0, n, n};
  if (off != nullptr) {
    const int o0 = off[b], o1 = off[b + 1];
    if (o0 < 0 || o1 < o0 || o1 > n) {
      raise_device_error(err, RESS_ERR_BAD_INDEX, detail);
      return SeqRange{0, 0, 0};
    }
    s.start = o0;
    s.rows = s.valid = o1 - o0;
  }
  if (lens != nullptr) {
    const int l = lens[b];
    if (l < 0 || l > s.rows) raise_device_error(err, RESS_ERR_BAD_INDEX, detail + 2);
    s.valid = min(max(l, 0), s.rows);
  }
  return s;
}

// Shared scratch of find_tile.
struct TileFind {
  long long warp_sum[32];   // 64 bits: descending offsets can claim any number of rows
  int b, tile;
};

// The sequence and the tile within it of flat tile `target`, where sequence b
// owns ceil(rows_b / tile_rows) tiles; false (for the whole CTA) behind the
// last one.  The grid has the upper bound n / tile_rows + seqs tiles, because
// the host does not know the lengths.  Called by all threads of the CTA.
__device__ __forceinline__ bool find_tile(const int32_t* off, int seqs, int n, int tile_rows,
                                          int target, TileFind* sh, int* b, int* tile,
                                          DeviceError* err, int detail) {
  if (off == nullptr) {
    *b = 0;
    *tile = target;
    return target < (n + tile_rows - 1) / tile_rows;
  }
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (seqs + threads - 1) / threads;
  const int b0 = threadIdx.x * per, b1 = min(seqs, b0 + per);
  long long mine = 0;
  for (int i = b0; i < b1; ++i)
    mine += (seq_range(off, nullptr, i, n, err, detail).rows + tile_rows - 1) / tile_rows;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  if (threadIdx.x == 0) sh->b = -1;
  __syncthreads();
  long long before = incl - mine;
  for (int w = 0; w < warp; ++w) before += sh->warp_sum[w];
  if (target >= before && target < before + mine) {
    long long at = before;
    for (int i = b0; i < b1; ++i) {
      const int t = (seq_range(off, nullptr, i, n, err, detail).rows + tile_rows - 1) / tile_rows;
      if (target < at + t) {
        sh->b = i;
        sh->tile = (int)(target - at);
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  *b = sh->b;
  *tile = sh->tile;
  return sh->b >= 0;
}

// First key that row `i` of `n` query rows of a request with `len` tokens no
// longer sees (see ress_cache_attn).
__device__ __forceinline__ int step_end(int len, int n, int i, int step) {
  if (step == 0) return len;
  const int pos = len - n + i;
  if (pos < 0) return 0;
  const long long end = ((long long)(pos / step) + 1) * step;
  return end < len ? (int)end : len;
}

}  // namespace ress
