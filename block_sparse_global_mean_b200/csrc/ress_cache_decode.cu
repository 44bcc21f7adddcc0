// Attention of a few query tokens per request over the 8-bit cache: the step
// that adds one token to every scene.
//
// Bound by reading the pages once (128 bytes a token and head), so everything is
// laid out for loads: every warp is a worker of its own (ress_sched.cuh) with a
// private ring of three 32-token chunks, copied by the bulk engine; no warp waits
// for another.  A chunk's codes go from shared memory straight into the operand
// registers of m16n8k16 products: 16 rows (token, query head of the key head)
// against 32 keys.  At a few rows per key the tensor core's rate is not the
// bound, and the register form needs no tile in shared or tensor memory.
//
//   S = q K^T     codes as f16 (exact); q as f16 times a power of two per row
//                 that puts its largest value at 2^14, exact down to 2^-28 of it
//                 and within 2^-39 of it below; key scale and the power of two go
//                 into the float32 logits.
//   P             exp2 of the logits less the chunk's own row maximum, as f16:
//                 11 bits, and only what is 2^-24 below the chunk's maximum is lost.
//   O             the chunk's product P V on codes as f16 (exact), then
//                 O = a O + b (P V) in float32, where b holds the value scale and
//                 the step from the chunk's maximum to the running one.
//
// One token for each of six scenes of 1 to 140,800 tokens (275 MB): 60 us, 4.6 TB/s
// (ten of them start and join; three scenes of 281,600: 5.7 TB/s).  The steady part
// is bound by issue, 650 instructions per 64 keys and head.  Chunks of 64 keys, 8
// or 16 warps, and rings of two or four chunks were all slower or the same (57 to 67
// us cold against 54); so were key codes moved into f16 by shifts, which halve the
// conversions but not the time.
//
// Which key stands in which column, and which dimension in which slot of the
// contraction, is free as long as both operands agree.  A thread (g = lane / 4,
// t = lane % 4) takes 16 consecutive dimensions 16 t .. of a key in S, and 8
// consecutive dimensions 8 g .. of key pairs in P V, so its loads are wide and
// its outputs are 16 consecutive dimensions.
#include "ress_common.cuh"
#include "ress_internal.h"
#include "ress_kv.h"
#include "ress_sched.cuh"

#include <cuda_fp16.h>

namespace ress {

namespace {

constexpr int kSms = 148;
constexpr int kWarps = 12;
constexpr int kWorkers = kSms * kWarps;
constexpr int kKeysLog2 = 5;
constexpr int kKeys = 1 << kKeysLog2;            // keys per chunk
constexpr int kRows = 16;
constexpr int kStages = 3;
constexpr uint32_t kHalf = kKeys * 64;           // bytes of keys (values) of a chunk
constexpr float kScaleLog2 = 1.4426950408889634f * 0.125f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  SchedParams sched;
  DeviceError* err;
  int nq, heads, kv_heads, group;
  int group_inv;       // 65536 / group, rounded up
  long long q_stride;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;       // [workers][2][16][64]
  float2* part_ml;     // [workers][2][16]
  SplitItem* split;    // [workers]
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  int pages, page_log2, max_pages, step;
};

struct Smem {
  uint8_t ring[kWarps][kStages][2 * kHalf];
  uint64_t full[kWarps][kStages];
  int abort_flag;
};
constexpr size_t kSmem = sizeof(Smem) + 128;

// Four e4m3 codes as two pairs of f16.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nonzero if one of four codes is NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 values of a query row as f16 times 2^(14 - e), e the exponent of the row's
// largest; returns 2^(e - 14).  The four threads of a row agree by shuffles.
__device__ __forceinline__ float query_f16(uint4 a, uint4 b, uint32_t (&w)[8]) {
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, max((u[i] << 16) & 0x7f800000u, u[i] & 0x7f800000u));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // Any bf16 number: both powers of two below are normal ones from 2^-112 on, and rows
  // of smaller values only lose depth below their largest.
  const int e = min(max((int)(top >> 23) - 127, -112), 127);
  const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = pack_f16x2(__uint_as_float(u[i] << 16) * up, __uint_as_float(u[i] & 0xffff0000u) * up);
  return __uint_as_float((uint32_t)(e - 14 + 127) << 23);
}

__global__ void __launch_bounds__(kWarps * 32, 1)
    cache_decode_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  Smem* sm = reinterpret_cast<Smem*>(
      smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t bar = smem_addr(&sm->full[warp][0]);
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
    fence_mbarrier_init();
  }
  if (threadIdx.x == 0) sm->abort_flag = 0;
  wait_for_previous_kernel();
  allow_next_kernel();
  __syncthreads();
  const int worker = warp * kSms + (int)blockIdx.x;   // few workers: spread over the SMs
  SchedWalk walk{0, 0, 0, 0, 0};
  const SchedPlan plan = sched_begin(p.sched, worker, &walk);
  SplitItem split = no_split();

  const int pos_mask = (1 << p.page_log2) - 1;
  uint8_t* ring = &sm->ring[warp][0][0];
  int issued = 0, used = 0;   // copies started and waited for
  bool ok = true;
  // Column n of S product j holds key 8 j + k_row(n): neighbours in a pair
  // and the four pairs differ in parity, so that neither the key loads nor the
  // value loads meet in the same banks more than twice.
  const int k_row = (g & ~1) + (((g >> 1) ^ g) & 1);
  const int v_row0 = 2 * t + (t & 1), v_row1 = 2 * t + 1 - (t & 1);

  for (;;) {
    const Segment seg = sched_next(p.sched, plan, walk);
    if (seg.kind == 0) break;
    if (seg.parts > 0) split = split_of(seg);
    const int rows = seg.rows * p.group;          // item rows of the request
    const int r0 = seg.tile * kRows + g, r1 = r0 + 8;
    const bool live0 = r0 < rows, live1 = r1 < rows;
    const bool upper = seg.tile * kRows + 8 < rows;   // rows 8..15 exist (warp-uniform)
    // Token and query head of a row: the tile's first, and from there less than
    // group + 16 rows on, where a 16-bit reciprocal divides exactly.
    const int tok_a = seg.tile == 0 ? 0 : div_small((long long)seg.tile * kRows, p.group);
    const int rest = seg.tile * kRows - tok_a * p.group + g;
    const int step0 = (rest * p.group_inv) >> 16, step1 = ((rest + 8) * p.group_inv) >> 16;
    const int tok0 = tok_a + step0, tok1 = tok_a + step1;
    const int head0 = seg.head * p.group + rest - step0 * p.group;
    const int head1 = seg.head * p.group + rest + 8 - step1 * p.group;
    const size_t row0 = (size_t)(seg.row_start + tok0), row1 = (size_t)(seg.row_start + tok1);
    uint32_t q0[8], q1[8];
    float qs0 = 0.f, qs1 = 0.f;
    const int end0 = live0 ? step_end(seg.cols_valid, seg.rows, tok0, p.step) : seg.cols_valid;
    const int end1 = live1 ? step_end(seg.cols_valid, seg.rows, tok1, p.step) : seg.cols_valid;
    float o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    // Pages and scales of 32 chunks at a time, one per lane.
    for (int base = seg.c0; base < seg.c1 && ok; base += 32) {
      const int n = min(32, seg.c1 - base);
      int id = -1;
      float ks = 0.f, vs = 0.f;
      if (lane < n) {
        id = p.table[(size_t)seg.b * p.max_pages + (((base + lane) * kKeys) >> p.page_log2)];
        if (id < 0 || id >= p.pages) {
          raise_device_error(p.err, RESS_ERR_BAD_INDEX, 95);
          id = -1;
        } else {
          ks = p.k_scale[(size_t)id * p.kv_heads + seg.head];
          vs = p.v_scale[(size_t)id * p.kv_heads + seg.head];
        }
      }
      // Chunks of the pool; the others are left out.
      const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
      unsigned to_load = have, to_use = have;
      auto load_next = [&]() {
        if (to_load == 0) return;
        const int c = __ffs((int)to_load) - 1;
        to_load &= to_load - 1u;
        const int page = __shfl_sync(0xffffffffu, id, c);
        const size_t at = (((size_t)page * p.kv_heads + seg.head) << p.page_log2) +
                          (size_t)(((base + c) * kKeys) & pos_mask);
        const int s = issued % kStages;
        if (elect_one()) {
          const uint32_t dst = smem_addr(ring + s * 2 * kHalf);
          mbar_arrive_expect_tx(bar + 8 * s, 2 * kHalf);
          bulk_load(dst, p.k_cache + at * kHeadDim, kHalf, bar + 8 * s);
          bulk_load(dst + kHalf, p.v_cache + at * kHeadDim, kHalf, bar + 8 * s);
        }
        __syncwarp();
        ++issued;
      };
#pragma unroll
      for (int s = 0; s < kStages; ++s) load_next();
      if (base == seg.c0) {   // behind the first copies, which need two loads before them
        const __nv_bfloat16* src0 = p.q + row0 * p.q_stride + head0 * kHeadDim + 16 * t;
        const __nv_bfloat16* src1 = p.q + row1 * p.q_stride + head1 * kHeadDim + 16 * t;
        uint4 a0 = make_uint4(0u, 0u, 0u, 0u), b0 = a0, a1 = a0, b1 = a0;
        if (live0) {
          a0 = reinterpret_cast<const uint4*>(src0)[0];
          b0 = reinterpret_cast<const uint4*>(src0)[1];
        }
        if (live1) {
          a1 = reinterpret_cast<const uint4*>(src1)[0];
          b1 = reinterpret_cast<const uint4*>(src1)[1];
        }
        qs0 = query_f16(a0, b0, q0);
        qs1 = query_f16(a1, b1, q1);
      }
      // Pages of a wrong scale are masked: their copies are on the way (the scales
      // looked at before them cost 1 us of every call).
      if (!scale_ok(ks) || !scale_ok(vs)) {
        raise_device_error(p.err, RESS_ERR_INVALID_ARG, 96);
        ks = -1.f;
        vs = 0.f;
      }
      while (to_use != 0) {
        const int c = __ffs((int)to_use) - 1;
        to_use &= to_use - 1u;
        const int s = used % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * s, (used / kStages) & 1, &sm->abort_flag,
                                               p.err, 180))) {
          ok = false;
          break;
        }
        ++used;
        const uint8_t* sk = ring + s * 2 * kHalf;
        const uint8_t* sv = sk + kHalf;
        const float kscale = __shfl_sync(0xffffffffu, ks, c) * kScaleLog2;
        const float vscale = __shfl_sync(0xffffffffu, vs, c);

        const int pos = (base + c) * kKeys;
        float x[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
          const uint4 w = *reinterpret_cast<const uint4*>(sk + (8 * j + k_row) * 64 + 16 * t);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            uint32_t b0, b1;
            codes_f16(u[d], b0, b1);
            const uint32_t a[4] = {q0[2 * d], q1[2 * d], q0[2 * d + 1], q1[2 * d + 1]};
            mma_f16(x[j], a, b0, b1);
          }
        }
        int lim0 = end0 - pos, lim1 = end1 - pos;
        const int left = seg.cols_valid - pos;
        if (__any_sync(0xffffffffu, lim0 < kKeys || lim1 < kKeys || kscale < 0.f)) {
          if (kscale < 0.f) lim0 = lim1 = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (8 * j + v_row0 >= lim0) x[j][0] = -INFINITY;
            if (8 * j + v_row1 >= lim0) x[j][1] = -INFINITY;
            if (8 * j + v_row0 >= lim1) x[j][2] = -INFINITY;
            if (8 * j + v_row1 >= lim1) x[j][3] = -INFINITY;
          }
          // Where one row sees keys that another does not, a NaN value would reach both
          // (0 * NaN): it leaves the value and goes into the logits of the rows that see
          // its token.
          const int most = min(left, kKeys);
          if (__any_sync(0xffffffffu, lim0 < most || lim1 < most)) {
            uint4* row = reinterpret_cast<uint4*>(ring + s * 2 * kHalf + kHalf + lane * 64);
            uint32_t nan = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint4 w = row[u];
              nan |= nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w);
            }
            const unsigned bad = __ballot_sync(0xffffffffu, nan != 0);
            if (bad != 0) {
              if (nan != 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) row[u] = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();   // the next copy into this place comes after it
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int k0 = 8 * j + v_row0, k1 = 8 * j + v_row1;
                if ((bad >> k0 & 1u) && k0 < lim0) x[j][0] = __int_as_float(0x7fffffff);
                if ((bad >> k1 & 1u) && k1 < lim0) x[j][1] = __int_as_float(0x7fffffff);
                if ((bad >> k0 & 1u) && k0 < lim1) x[j][2] = __int_as_float(0x7fffffff);
                if ((bad >> k1 & 1u) && k1 < lim1) x[j][3] = __int_as_float(0x7fffffff);
              }
            }
          }
        }
        // Chunk maximum, probabilities, sums.
        float c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c0 = fmax3(c0, x[j][0], x[j][1]);
          c1 = fmax3(c1, x[j][2], x[j][3]);
        }
        c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, 1));
        c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, 2));
        // Never zero: a masked logit (-inf) stays one.
        const float f0 = fmaxf(kscale * qs0, 1.2e-38f), f1 = fmaxf(kscale * qs1, 1.2e-38f);
        c0 *= f0;
        const bool any0 = c0 > -INFINITY;
        const float n0 = fmaxf(m0, c0);
        const float u0 = any0 ? -c0 : 0.f;
        float s0 = 0.f, s1 = 0.f;
        uint32_t pk[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pa = fast_exp2(fmaf(x[j][0], f0, u0)), pb = fast_exp2(fmaf(x[j][1], f0, u0));
          s0 += pa + pb;
          pk[j][0] = pack_f16x2(pa, pb);
          pk[j][1] = 0u;
        }
        const float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0);
        const float b0 = any0 ? fast_exp2(c0 - n0) : 0.f;
        m0 = n0;
        l0 = fmaf(b0, s0, a0 * l0);
        float a1 = 0.f, b1 = 0.f;
        if (upper) {
          c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, 1));
          c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, 2));
          c1 *= f1;
          const bool any1 = c1 > -INFINITY;
          const float n1 = fmaxf(m1, c1);
          const float u1 = any1 ? -c1 : 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float pa = fast_exp2(fmaf(x[j][2], f1, u1)), pb = fast_exp2(fmaf(x[j][3], f1, u1));
            s1 += pa + pb;
            pk[j][1] = pack_f16x2(pa, pb);
          }
          a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
          b1 = any1 ? fast_exp2(c1 - n1) : 0.f;
          m1 = n1;
          l1 = fmaf(b1, s1, a1 * l1);
        }
        // O = a O + b scale (P V).
        const bool tail = left < kKeys;
        float y[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j][0] = y[j][1] = y[j][2] = y[j][3] = 0.f;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const uint32_t a[4] = {pk[2 * kb][0], pk[2 * kb][1], pk[2 * kb + 1][0], pk[2 * kb + 1][1]};
          uint2 w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 16 * kb + (e >> 1) * 8 + ((e & 1) ? v_row1 : v_row0);
            w[e] = *reinterpret_cast<const uint2*>(sv + key * 64 + 8 * g);
            if (tail && key >= left) w[e] = make_uint2(0u, 0u);   // may hold NaN
          }
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const uint32_t e0 = d ? w[0].y : w[0].x, e1 = d ? w[1].y : w[1].x;
            const uint32_t e2 = d ? w[2].y : w[2].x, e3 = d ? w[3].y : w[3].x;
            uint32_t v0[4], v1[4];
            codes_f16(__byte_perm(e0, e1, 0x5140), v0[0], v0[1]);
            codes_f16(__byte_perm(e0, e1, 0x7362), v0[2], v0[3]);
            codes_f16(__byte_perm(e2, e3, 0x5140), v1[0], v1[1]);
            codes_f16(__byte_perm(e2, e3, 0x7362), v1[2], v1[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_f16(y[4 * d + j], a, v0[j], v1[j]);
          }
        }
        __syncwarp();   // every lane has read the chunk: its place may be filled again
        load_next();
        const float bv0 = b0 * vscale, bv1 = b1 * vscale;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][0] = fmaf(bv0, y[j][0], a0 * o[j][0]);
          o[j][1] = fmaf(bv0, y[j][1], a0 * o[j][1]);
        }
        if (upper) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j][2] = fmaf(bv1, y[j][2], a1 * o[j][2]);
            o[j][3] = fmaf(bv1, y[j][3], a1 * o[j][3]);
          }
        }
      }
    }
    if (!ok) break;

    // Column n of the value products is dimension 8 n + j: a thread's columns
    // 2 t and 2 t + 1 are dimensions 16 t .. 16 t + 15.
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // A NaN value has reached its own dimension: it goes to the row's sum, and so to
    // all of the row, as a NaN key does.
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      bool nan = false;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        nan |= isnan(o[j][2 * half]) || isnan(o[j][2 * half + 1]);
      const unsigned who = __ballot_sync(0xffffffffu, nan);
      if (who >> (lane & 28) & 15u) (half ? l1 : l0) = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const bool live = half ? live1 : live0;
      if (!live) continue;
      const float l = half ? l1 : l0;
      float m = half ? m1 : m0;
      if (m == -INFINITY && l != l) m = 0.f;   // NaN logits move no maximum, but reach the sum
      const bool empty = m == -INFINITY;
      if (seg.kind == 1) {
        const float inv = empty ? 0.f : 1.0f / l;
        const size_t row = half ? row1 : row0;
        const int head = half ? head1 : head0;
        uint4* dst = reinterpret_cast<uint4*>(p.out + (row * p.heads + head) * kHeadDim + 16 * t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = pack_bf16x2(o[2 * j][2 * half + e] * inv, o[2 * j + 1][2 * half + e] * inv);
          dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (t == 0 && p.lse != nullptr)
          p.lse[(size_t)head * p.nq + row] = empty ? -INFINITY : (m + __log2f(l)) * kLn2;
      } else {
        const size_t part = ((size_t)worker * 2 + seg.slot) * kRows + g + 8 * half;
        float4* dst = reinterpret_cast<float4*>(p.part_o + part * kHeadDim + 16 * t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          dst[2 * e] = make_float4(o[0][2 * half + e], o[1][2 * half + e], o[2][2 * half + e],
                                   o[3][2 * half + e]);
          dst[2 * e + 1] = make_float4(o[4][2 * half + e], o[5][2 * half + e], o[6][2 * half + e],
                                       o[7][2 * half + e]);
        }
        if (t == 0) p.part_ml[part] = make_float2(m, l);
      }
    }
  }
  if (lane == 0) store_split(p.split + worker, split);
  // Copies still in flight (after a timeout) land before the warp leaves.
  for (; used < issued; ++used)
    mbar_wait_drain(bar + 8 * (used % kStages), (used / kStages) & 1, p.err, 181);
}

// Joins the parts of the item that worker blockIdx.x began and did not end.
__global__ void __launch_bounds__(256)
    cache_decode_combine_kernel(const __grid_constant__ DecodeParams p) {
  wait_for_previous_kernel();
  allow_next_kernel();
  const SplitItem it = load_split(p.split + blockIdx.x);
  if (it.head < 0) return;
  auto token_of = [&](int r) { return (size_t)(it.row_start + (it.tile * kRows + r) / p.group); };
  auto head_of = [&](int r) { return it.head * p.group + (it.tile * kRows + r) % p.group; };
  join_item<16>(
      it, (int)blockIdx.x, p.sched.grid, p.part_ml, p.part_o, kRows, 0, min(kRows, it.rows * p.group - it.tile * kRows),
      [&](int r) -> __nv_bfloat16* {
        return p.out + (token_of(r) * p.heads + head_of(r)) * kHeadDim;
      },
      [&](int r) -> float* {
        return p.lse ? p.lse + (size_t)head_of(r) * p.nq + token_of(r) : nullptr;
      });
}

}  // namespace

size_t cache_decode_workspace() {
  return align256((size_t)kWorkers * (2 * kRows * (kHeadDim * sizeof(float) + sizeof(float2)) +
                                      sizeof(SplitItem)));
}

ress_status launch_cache_decode(const CrossParams& c, void* ws, cudaStream_t st) {
  DecodeParams p{};
  p.err = c.err;
  p.nq = c.nq;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.group = c.group;
  p.group_inv = (65535 + c.group) / c.group;
  p.q_stride = c.q_stride;
  p.q = c.q;
  p.out = c.out;
  p.lse = c.lse;
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)kWorkers * 2 * kRows * kHeadDim);
  p.split = reinterpret_cast<SplitItem*>(p.part_ml + (size_t)kWorkers * 2 * kRows);
  p.k_cache = c.k_cache;
  p.v_cache = c.v_cache;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.table = c.table;
  p.pages = c.pages;
  p.page_log2 = c.page == 64 ? 6 : 7;
  p.max_pages = c.max_pages;
  p.step = c.step;
  p.sched.err = c.err;
  p.sched.row_off = c.q_off;
  p.sched.rows = c.nq;
  p.sched.row_detail = 90;
  p.sched.lengths = c.lengths;
  p.sched.max_len = (long long)c.max_pages * c.page;
  p.sched.seqs = c.seqs;
  p.sched.heads = c.kv_heads;
  p.sched.row_mult = c.group;
  p.sched.tile_rows = kRows;
  p.sched.mult = 1;
  p.sched.chunk_log2 = kKeysLog2;
  p.sched.item_cost = 64;
  p.sched.min_share = 128;
  p.sched.grid = kWorkers;
  static std::atomic<uint64_t> allowed{0};
  if (ress_status s =
          allow_smem(reinterpret_cast<const void*>(cache_decode_kernel), kSmem, &allowed))
    return s;
  if (ress_status s = record_cuda(
          launch_behind(cache_decode_kernel, dim3(kSms), dim3(kWarps * 32), kSmem, st, p)))
    return s;
  return record_cuda(
      launch_dependent(cache_decode_combine_kernel, dim3(kWorkers), dim3(256), st, p));
}

}  // namespace ress
