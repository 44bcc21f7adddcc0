// Gradients of the attention over keys of another length: one thread per row,
// partners in shared memory (first, plain version).
#include "ress_common.cuh"
#include "ress_internal.h"
#include "ress_kv.h"
#include "ress_seq.cuh"

namespace ress {

namespace {

constexpr int kRowsPerCta = 128;
constexpr int kKeys = 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void load_row(const __nv_bfloat16* src, float (&r)[64]) {
#pragma unroll
  for (int d = 0; d < 64; ++d) r[d] = __bfloat162float(src[d]);
}

// delta and dQ: one thread per query row.
__global__ void __launch_bounds__(kRowsPerCta) cross_dq_kernel(const CrossBwdParams p) {
  __shared__ float sk[kKeys][64], sv[kKeys][64];
  __shared__ TileFind find;
  int b, tile;
  if (!find_tile(p.q_off, p.seqs, p.nq, kRowsPerCta, blockIdx.x, &find, &b, &tile, p.err, 90))
    return;
  const int h = blockIdx.y, hk = h / p.group;
  const SeqRange qs = seq_range(p.q_off, p.q_lens, b, p.nq, p.err, 90);
  const SeqRange ks = seq_range(p.k_off, p.k_lens, b, p.nk, p.err, 91);
  const int i = tile * kRowsPerCta + threadIdx.x;
  const bool real = i < qs.valid;
  const int row = qs.start + i;
  float q[64], g[64], dq[64], delta = 0.f, lse = -INFINITY;
#pragma unroll
  for (int d = 0; d < 64; ++d) q[d] = g[d] = dq[d] = 0.f;
  if (real) {
    load_row(p.q + (size_t)row * p.q_stride + h * 64, q);
    load_row(p.dout + ((size_t)row * p.heads + h) * 64, g);
    const __nv_bfloat16* o = p.out + ((size_t)row * p.heads + h) * 64;
#pragma unroll
    for (int d = 0; d < 64; ++d) delta = fmaf(g[d], __bfloat162float(o[d]), delta);
    lse = p.lse[(size_t)h * p.nq + row];
    p.delta[(size_t)h * p.nq + row] = delta;
  }
  const bool live = real && lse != -INFINITY;
  for (int k0 = 0; k0 < ks.valid; k0 += kKeys) {
    __syncthreads();
    const int n = min(kKeys, ks.valid - k0);
    for (int e = threadIdx.x; e < n * 64; e += kRowsPerCta) {
      const int t = e >> 6, d = e & 63;
      sk[t][d] = __bfloat162float(p.k[(size_t)(ks.start + k0 + t) * p.k_stride + hk * 64 + d]);
      sv[t][d] = __bfloat162float(p.v[(size_t)(ks.start + k0 + t) * p.v_stride + hk * 64 + d]);
    }
    __syncthreads();
    if (!live) continue;
    for (int t = 0; t < n; ++t) {
      float s = 0.f, dp = 0.f;
#pragma unroll
      for (int d = 0; d < 64; ++d) {
        s = fmaf(q[d], sk[t][d], s);
        dp = fmaf(g[d], sv[t][d], dp);
      }
      const float ds = exp2f((s * 0.125f - lse) * kLog2e) * (dp - delta);
#pragma unroll
      for (int d = 0; d < 64; ++d) dq[d] = fmaf(ds, sk[t][d], dq[d]);
    }
  }
  if (i >= qs.rows) return;
  __nv_bfloat16* dst = p.dq + ((size_t)row * p.heads + h) * 64;
#pragma unroll
  for (int d = 0; d < 64; ++d) dst[d] = __float2bfloat16(dq[d] * 0.125f);
}

// dK and dV: one thread per key row, over the query heads that share it.
__global__ void __launch_bounds__(kRowsPerCta) cross_dkv_kernel(const CrossBwdParams p) {
  __shared__ float sq[kKeys][64], sg[kKeys][64], s_lse[kKeys], s_delta[kKeys];
  __shared__ TileFind find;
  int b, tile;
  if (!find_tile(p.k_off, p.seqs, p.nk, kRowsPerCta, blockIdx.x, &find, &b, &tile, p.err, 91))
    return;
  const int hk = blockIdx.y;
  const SeqRange qs = seq_range(p.q_off, p.q_lens, b, p.nq, p.err, 90);
  const SeqRange ks = seq_range(p.k_off, p.k_lens, b, p.nk, p.err, 91);
  const int i = tile * kRowsPerCta + threadIdx.x;
  const bool real = i < ks.valid;
  const int row = ks.start + i;
  float k[64], v[64], dk[64], dv[64];
#pragma unroll
  for (int d = 0; d < 64; ++d) k[d] = v[d] = dk[d] = dv[d] = 0.f;
  if (real) {
    load_row(p.k + (size_t)row * p.k_stride + hk * 64, k);
    load_row(p.v + (size_t)row * p.v_stride + hk * 64, v);
  }
  for (int h = hk * p.group; h < (hk + 1) * p.group; ++h)
    for (int q0 = 0; q0 < qs.valid; q0 += kKeys) {
      __syncthreads();
      const int n = min(kKeys, qs.valid - q0);
      for (int e = threadIdx.x; e < n * 64; e += kRowsPerCta) {
        const int t = e >> 6, d = e & 63;
        const size_t r = qs.start + q0 + t;
        sq[t][d] = __bfloat162float(p.q[r * p.q_stride + h * 64 + d]);
        sg[t][d] = __bfloat162float(p.dout[(r * p.heads + h) * 64 + d]);
        if (d == 0) {
          s_lse[t] = p.lse[(size_t)h * p.nq + r];
          s_delta[t] = p.delta[(size_t)h * p.nq + r];
        }
      }
      __syncthreads();
      if (!real) continue;
      for (int t = 0; t < n; ++t) {
        if (s_lse[t] == -INFINITY) continue;
        float s = 0.f, dp = 0.f;
#pragma unroll
        for (int d = 0; d < 64; ++d) {
          s = fmaf(k[d], sq[t][d], s);
          dp = fmaf(v[d], sg[t][d], dp);
        }
        const float pt = exp2f((s * 0.125f - s_lse[t]) * kLog2e);
        const float ds = pt * (dp - s_delta[t]);
#pragma unroll
        for (int d = 0; d < 64; ++d) {
          dk[d] = fmaf(ds, sq[t][d], dk[d]);
          dv[d] = fmaf(pt, sg[t][d], dv[d]);
        }
      }
    }
  if (i >= ks.rows) return;
  const size_t at = ((size_t)row * p.kv_heads + hk) * 64;
#pragma unroll
  for (int d = 0; d < 64; ++d) {
    p.dk[at + d] = __float2bfloat16(dk[d] * 0.125f);
    p.dv[at + d] = __float2bfloat16(dv[d]);
  }
}

unsigned tiles_of(int n, int seqs, bool packed) {
  return packed ? (unsigned)(n / kRowsPerCta + seqs) : (unsigned)((n + kRowsPerCta - 1) / kRowsPerCta);
}

}  // namespace

size_t cross_bwd_workspace(const CrossGeometry& g) {
  return align256(sizeof(float) * (size_t)g.heads * g.nq);
}
ress_status launch_cross_bwd(const CrossGeometry& g, CrossBwdParams p, void* ws, cudaStream_t st) {
  p.delta = static_cast<float*>(ws);
  if (p.nq > 0) {
    const dim3 grid(tiles_of(p.nq, p.seqs, p.q_off != nullptr), g.heads);
    cross_dq_kernel<<<grid, kRowsPerCta, 0, st>>>(p);
    if (ress_status s = record_cuda(cudaGetLastError())) return s;
  }
  if (p.nk > 0) {
    const dim3 grid(tiles_of(p.nk, p.seqs, p.k_off != nullptr), g.kv_heads);
    cross_dkv_kernel<<<grid, kRowsPerCta, 0, st>>>(p);
  }
  return record_cuda(cudaGetLastError());
}

}  // namespace ress
