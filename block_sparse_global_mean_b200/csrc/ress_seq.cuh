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

// Scales of cache pages: powers of two from 2^-100 to 2^119, so that both ways to take
// a code to code * scale are exact, or zero (a page that was never written).
__device__ __forceinline__ bool scale_ok(float scale) {
  const uint32_t b = __float_as_uint(scale);
  return b == 0u || ((b & 0x7fffffu) == 0u && b - (27u << 23) <= (219u << 23));
}

// Programmatic dependent launch: a kernel is launched while the one before it on
// the stream still runs, sets itself up, and waits here for its results.  What it
// reads may be written while it lives, so it reads global memory with plain loads,
// not with those of the read-only path.
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

// The first kernel of an operator, behind whatever the stream holds (calls in a row:
// two requests decoded 14.4 -> 12.2 us, 64 tokens appended 6.2 -> 3.8 us).  A graph
// keeps plain edges here.
template <typename Kernel, typename... Args>
cudaError_t launch_behind(Kernel kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                          Args... args) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaError_t e = cudaStreamIsCapturing(st, &capture)) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = capture == cudaStreamCaptureStatusNone ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace ress
