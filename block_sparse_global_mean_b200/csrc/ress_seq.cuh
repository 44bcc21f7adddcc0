// Packed sequences on the device.  Offsets and lengths live in device memory,
// so every kernel checks them as it reads them.
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
