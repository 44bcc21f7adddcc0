// Gradients of ress_cross_attn on tcgen05.
//
// With P = exp(S - lse), S = Q K^T / sqrt(d), delta = dout . out per row and
// dS = P (dout V^T - delta):
//   dV = P^T dout,  dK = dS^T Q / sqrt(d),  dQ = dS K / sqrt(d).
// dK and dV are sums over the query rows, dQ over the keys.  Sums that many
// CTAs add to in the order of their arrival would differ from run to run, so
// two walks are made, each with the accumulators of its own rows in TMEM: the
// key walk (kDQ = false: tiles of 128 keys against chunks of 128 query rows) and
// the query walk (kDQ = true: tiles of 128 query rows, the heads of a key head
// together, against chunks of 128 keys).  S and dout V^T are computed in both, and
// the query walk multiplies dS twice (below): eight products for the formula's five,
// and the exponentials twice; no atomics.
//
// In both walks the resident tile gives the rows of the products, so P and dS
// leave the registers as rows and go back to TMEM as the left operand of the
// accumulating products; nothing is transposed:
//   X = A1 B1^T   (key walk: K Q^T; query walk: Q K^T)
//   Y = A2 B2^T   (key walk: V dout^T; query walk: dout V^T)
//   P = exp2(X log2(e) / 8 - lse log2(e)),  dS = P (Y - delta)
//   key walk: dV += P B2, dK += dS B1;  query walk: dQ += dS B1.
//
// P and dS enter as bf16.  A row of dS sums to zero over its keys, so what keys
// have in common (their mean) cancels in dQ, but roundings of dS do not sum to
// zero: with keys whose mean is twice their spread a single bf16 dS left 0.41 %
// in dQ against 0.17 % of the output's own rounding.  The query walk therefore
// multiplies dS as two bf16 numbers, its rounding and the rest (16 bits of it).
// dK and dV have no such sum; over many keys they are off by 0.24 %, by the output's
// rounding and that of P or dS.  Over few keys a key's probabilities may all stand
// where bf16's steps are widest, and 0.35 % was met (one head, 100 queries, 33 keys).
// So over up to a tile of keys the key walk makes every chunk twice, with the
// roundings and with the rests: 0.17 %, as much as the output's own rounding.  It
// costs 1,374 queries against 128 keys 48 us for 39, 140,800 against 5 keys 1.51 ms
// for 1.08 (16 heads).
//
// TMEM (512 columns): X of the two softmax groups (2 x 128; P, or the rest of dS,
// and dS as bf16 over it once it is in registers), one Y (128, free again when it
// has been read), two accumulators (64 each).
//
// Warp roles: 0 TMA, 1 TMEM and MMA issue, 2 the next item, 3 (key walk) lse and
// delta of the chunk's rows, 4-11 two groups of four warps that take the even
// and the odd chunks, one row per thread.
//
// Bound by the groups' waits for one another's products (a task of 2,500 to 2,850
// cycles holds 1,024 of tensor work and 1,024 of exponentials) and, at full size,
// by the power limit, which holds the clock at 1.7 GHz.
//
// Both walks are one launch (blockIdx.y), so the second fills the SMs as the
// first one's CTAs end.
#define RESS_WAIT_FN __forceinline__
#include "ress_common.cuh"
#include "ress_internal.h"
#include "ress_kv.h"
#include "ress_sched.cuh"

#include <type_traits>

namespace ress {

namespace {

constexpr int kSms = 148;
constexpr int kThreads = 384;
constexpr int kStages = 5;
constexpr uint32_t kTileBytes = 128 * 128;
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColY = 256, kColA1 = 384, kColA2 = 448;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTwiceKeys = 129;   // fewer keys than this: every chunk twice

struct BwdParams {
  SchedParams sched[2];      // key walk, query walk
  DeviceError* err;
  int nq, heads, kv_heads, group, tps;
  const float* nl;           // [heads][nq]: -lse log2(e)
  const float* nd;           // [heads][nq]: -delta
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* part[2];            // [grid][2][128 rows][128 (key walk) or 64]
  SplitItem* split;          // [2 walks][grid]
};

struct __align__(16) Ctl {
  float nl[kStages][128];    // key walk: of the chunk's query rows
  float nd[kStages][128];
  uint64_t a_full;
  uint64_t b_full[kStages];
  uint64_t b_empty[kStages];
  uint64_t x_full[2];
  uint64_t y_full[2];
  uint64_t y_free[2];
  uint64_t p_full[2];
  uint64_t acc_full;
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  Segment seg[2];
};
constexpr size_t kSmem = 1024 + 2 * kTileBytes + kStages * kStageBytes + sizeof(Ctl);
static_assert(kSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          DeviceError* err, int detail) {
  const bool ok = mbar_wait(bar, parity, abort_flag, err, detail);
  return __all_sync(0xffffffffu, ok);
}

// delta and lse of every row, negated and in the units the walks use: eight
// lanes per row, 16 bytes each.  A row without a key (lse -inf) gets
// nl = -inf, which makes its P zero.  Bound by reading out and dout once.
__global__ void __launch_bounds__(256)
    cross_delta_kernel(const __nv_bfloat16* out, const __nv_bfloat16* dout, const float* lse,
                       float* nl, float* nd, int nq, int heads) {
  const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) >> 3;
  const long long rows = (long long)nq * heads;
  const int sub = threadIdx.x & 7;
  float d = 0.f;
  wait_for_previous_kernel();
  if (at < rows) {
    const uint4 a = *(reinterpret_cast<const uint4*>(out + at * kHeadDim) + sub);
    const uint4 b = *(reinterpret_cast<const uint4*>(dout + at * kHeadDim) + sub);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      d = fmaf(__uint_as_float(x[u] << 16), __uint_as_float(y[u] << 16), d);
      d = fmaf(__uint_as_float(x[u] & 0xffff0000u), __uint_as_float(y[u] & 0xffff0000u), d);
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (at < rows && sub == 0) {
    const int row = (int)(at / heads), h = (int)(at % heads);
    const float l = lse[(size_t)h * nq + row];
    nl[(size_t)h * nq + row] = l == -INFINITY ? l : -l * kLog2e;
    nd[(size_t)h * nq + row] = -d;
  }
}

// x less its bf16 rounding (the pair `hi`), as bf16.
__device__ __forceinline__ uint32_t rest_bf16x2(float2 x, uint32_t hi) {
  const float2 r = fadd2(x, make_float2(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xffff0000u)));
  return pack_bf16x2(r.x, r.y);
}

template <bool kDQ>
__device__ __forceinline__ void bwd_walk(const CUtensorMap* tm_a1, const CUtensorMap* tm_a2,
                                         const CUtensorMap* tm_b1, const CUtensorMap* tm_b2,
                                         const BwdParams& p, uint8_t* smem) {
  const SchedParams& sp = p.sched[kDQ ? 1 : 0];
  uint8_t* sA = smem;
  uint8_t* sB = smem + 2 * kTileBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(sB + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t bar_a = smem_addr(&ctl->a_full);
  const uint32_t bar_bf = smem_addr(&ctl->b_full[0]);
  const uint32_t bar_be = smem_addr(&ctl->b_empty[0]);
  const uint32_t bar_x = smem_addr(&ctl->x_full[0]);
  const uint32_t bar_y = smem_addr(&ctl->y_full[0]);
  const uint32_t bar_yf = smem_addr(&ctl->y_free[0]);
  const uint32_t bar_p = smem_addr(&ctl->p_full[0]);
  const uint32_t bar_acc = smem_addr(&ctl->acc_full);
  const uint32_t bar_done = smem_addr(&ctl->mma_done);
  volatile int* abortf = &ctl->abort_flag;

  if (threadIdx.x == 0) {
    mbar_init(bar_a, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_bf + 8 * s, kDQ ? 1 : 33);   // the copies, and warp 3's lanes
      mbar_init(bar_be + 8 * s, 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar_x + 8 * g, 1);
      mbar_init(bar_y + 8 * g, 1);
      mbar_init(bar_yf + 8 * g, 128);
      mbar_init(bar_p + 8 * g, 128);
    }
    mbar_init(bar_acc, 1);
    mbar_init(bar_done, 1);
    ctl->abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&ctl->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 96) {
    tma_prefetch_desc(tm_a1);
    tma_prefetch_desc(tm_a2);
    tma_prefetch_desc(tm_b1);
    tma_prefetch_desc(tm_b2);
  }
  wait_for_previous_kernel();   // delta, and what came before it
  allow_next_kernel();
  SchedWalk walk{0, 0, 0, 0, 0};
  SchedPlan plan;
  if (warp == 2) {
    plan = sched_begin(sp, (int)blockIdx.x, &walk);
    if (lane == 0) ctl->seg[0] = sched_next(sp, plan, walk);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  auto end_of_item = [&]() -> bool {
    tc_fence_before();
    named_bar_sync(1, kThreads);
    tc_fence_after();
    return *abortf == 0;
  };
  // Few keys: every chunk twice, first with P and dS rounded to bf16, then with what
  // that left (1: shift of the item's chunks).
  auto twice = [&](const Segment& g) { return !kDQ && g.rows_valid < kTwiceKeys ? 1 : 0; };
  // Chunk c of an item: its column rows (and, in the key walk, its query head).
  auto chunk_at = [&](const Segment& g, int c, int& col, int& head) {
    if (kDQ) {
      col = c * kChunk;
      head = g.head;
    } else {
      const int per = (g.cols_valid + kChunk - 1) / kChunk;
      c >>= twice(g);
      const int h = c / per;
      col = (c - h * per) * kChunk;
      head = g.head * p.group + h;
    }
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------- TMA ----------------
      int kc = 0, n_a = 0;
      for (int s = 0;; ++s) {
        const Segment g = ctl->seg[s & 1];
        if (g.kind == 0) break;
        if (g.c1 > g.c0) {
          if (elect_one()) {
            const int row = g.row_start + g.tile * sp.tile_rows;
            const uint32_t bytes = kDQ ? (uint32_t)(p.tps * p.group) * 128u : kTileBytes;
            mbar_arrive_expect_tx(bar_a, 2 * bytes);
            const int head = kDQ ? g.head * p.group : g.head;
            tma_load_3d(smem_addr(sA), tm_a1, bar_a, 0, head, row);
            tma_load_3d(smem_addr(sA) + kTileBytes, tm_a2, bar_a, 0, head, row);
          }
          __syncwarp();
          ++n_a;
          for (int c = g.c0; c < g.c1; ++c, ++kc) {
            const int st = kc % kStages;
            if (kc >= kStages &&
                !warp_wait(bar_be + 8 * st, ((kc / kStages) - 1) & 1, abortf, p.err, 150))
              break;
            int col, head;
            chunk_at(g, c, col, head);
            const uint32_t dst = smem_addr(sB) + (uint32_t)st * kStageBytes;
            const uint32_t bar = bar_bf + 8 * st;
            if (elect_one()) {
              mbar_arrive_expect_tx(bar, kStageBytes);
              tma_load_3d(dst, tm_b1, bar, 0, head, g.col_start + col);
              tma_load_3d(dst + kTileBytes, tm_b2, bar, 0, head, g.col_start + col);
            }
            __syncwarp();
          }
        }
        if (!end_of_item()) break;
      }
      // Copies still in flight (after a timeout) land before the CTA exits.
      for (int c = kc > kStages ? kc - kStages : 0; c < kc; ++c)
        mbar_wait_drain(bar_bf + 8 * (c % kStages), (c / kStages) & 1, p.err, 151);
      if (n_a > 0) mbar_wait_drain(bar_a, (n_a - 1) & 1, p.err, 152);
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- MMA issue ----------------
      constexpr uint32_t idX = idesc_bf16_f32(128, 128, false);
      constexpr uint32_t idA = idesc_bf16_f32(128, 64, true);
      const uint64_t da1 = smem_desc_sw128(smem_addr(sA), 16, 1024);
      const uint64_t db1 = smem_desc_sw128(smem_addr(sB), 16, 1024);
      const uint64_t dt1 = smem_desc_sw128(smem_addr(sB), 16384, 1024);   // N-major view
      constexpr uint64_t kStageDesc = kStageBytes >> 4, kTileDesc = kTileBytes >> 4;
      int kc0 = 0, n_a = 0, cnt0 = 0, cnt1 = 0;   // chunks, items, tasks of each group before
      bool any = false;
      for (int s = 0;; ++s) {
        const Segment& g = ctl->seg[s & 1];
        if (g.kind == 0) break;
        const int n = g.c1 - g.c0;
        if (n > 0) {
          bool ok = warp_wait(bar_a, n_a & 1, abortf, p.err, 160);
          any = true;
          auto issue_x = [&](int i) -> bool {
            const int kc = kc0 + i, st = kc % kStages;
            if (!warp_wait(bar_bf + 8 * st, (kc / kStages) & 1, abortf, p.err, 161)) return false;
            tc_fence_after();
            const uint64_t b = db1 + (uint64_t)st * kStageDesc;
            const uint32_t d = tmem + 128u * (uint32_t)(i & 1);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss(d, da1 + (uint64_t)(kk * 2), b + (uint64_t)(kk * 2), idX, kk > 0 ? 1u : 0u);
              mma_commit(bar_x + 8u * (uint32_t)(i & 1));
            }
            __syncwarp();
            return true;
          };
          auto issue_y = [&](int i) {
            const int st = (kc0 + i) % kStages;
            const uint64_t b = db1 + (uint64_t)st * kStageDesc + kTileDesc;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss(tmem + kColY, da1 + kTileDesc + (uint64_t)(kk * 2), b + (uint64_t)(kk * 2),
                       idX, kk > 0 ? 1u : 0u);
              mma_commit(bar_y + 8u * (uint32_t)(i & 1));
            }
            __syncwarp();
          };
          ok = ok && issue_x(0);
          if (ok) issue_y(0);
          if (ok && n > 1) ok = issue_x(1);
          for (int i = 0; ok && i < n; ++i) {
            const int gr = i & 1;
            const uint32_t ph = (uint32_t)((gr ? cnt1 : cnt0) + (i >> 1)) & 1u;
            if (i + 1 < n) {   // Y(i) is read: the next one may take its place
              if (!warp_wait(bar_yf + 8u * (uint32_t)gr, ph, abortf, p.err, 162)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_y(i + 1);
            }
            if (!warp_wait(bar_p + 8u * (uint32_t)gr, ph, abortf, p.err, 163)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const int st = (kc0 + i) % kStages;
            const uint64_t t1 = dt1 + (uint64_t)st * kStageDesc, t2 = t1 + kTileDesc;
            const uint32_t tP = tmem + 128u * (uint32_t)gr;
            if (elect_one()) {
              if (!kDQ) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_ts(tmem + kColA1, tP + kk * 8, t2 + (uint64_t)(kk * 128), idA,
                         (kk > 0 || i > 0) ? 1u : 0u);
              }
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_ts(tmem + kColA2, tP + 64 + kk * 8, t1 + (uint64_t)(kk * 128), idA,
                       (kk > 0 || i > 0) ? 1u : 0u);
              if (kDQ) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_ts(tmem + kColA2, tP + kk * 8, t1 + (uint64_t)(kk * 128), idA, 1u);
              }
              mma_commit(bar_be + 8 * st);
            }
            __syncwarp();
            if (i + 2 < n) ok = issue_x(i + 2);   // over P(i), dS(i): in issue order
          }
          if (ok && elect_one()) mma_commit(bar_acc);
          __syncwarp();
          kc0 += n;
          cnt0 += (n + 1) >> 1;
          cnt1 += n >> 1;
          ++n_a;
        }
        if (!end_of_item()) break;
      }
      if (any) {
        if (elect_one()) mma_commit(bar_done);
        __syncwarp();
        mbar_wait_drain(bar_done, 0, p.err, 164);
      }
      __syncwarp();
    } else {
      // ---------------- the next item (warp 2); lse and delta of a chunk (warp 3) ----------------
      int kc = 0;
      SplitItem split = no_split();
      for (int s = 0;; ++s) {
        const Segment& g = ctl->seg[s & 1];
        if (g.kind == 0) break;
        if (threadIdx.x == 64) {
          if (g.parts > 0) split = split_of(g);
          ctl->seg[(s + 1) & 1] = sched_next(sp, plan, walk);
        }
        if (!kDQ && warp == 3) {
          for (int c = g.c0; c < g.c1; ++c, ++kc) {
            const int st = kc % kStages;
            int col, head;
            chunk_at(g, c, col, head);
            float a[4], b[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = col + lane + 32 * u;
              const bool in = i < g.cols_valid;
              const size_t at = (size_t)head * p.nq + g.col_start + i;
              a[u] = in ? p.nl[at] : -INFINITY;
              b[u] = in ? p.nd[at] : 0.f;
            }
            if (kc >= kStages &&
                !warp_wait(bar_be + 8 * st, ((kc / kStages) - 1) & 1, abortf, p.err, 153))
              break;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              ctl->nl[st][lane + 32 * u] = a[u];
              ctl->nd[st][lane + 32 * u] = b[u];
            }
            mbar_arrive(bar_bf + 8 * st);
          }
        }
        __syncwarp();
        if (!end_of_item()) break;
      }
      if (threadIdx.x == 64) store_split(p.split + (kDQ ? kSms : 0) + blockIdx.x, split);
    }
  } else {
    // ---------------- P, dS and the epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int quad = warp & 3;
    const int par = (warp - 4) >> 2;
    const int rr = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tX = tmem + lane_off + 128u * (uint32_t)par;
    const uint32_t tY = tmem + lane_off + kColY;
    const float2 scale2 = make_float2(kLog2e * 0.125f, kLog2e * 0.125f);
    const int tok_in_tile = kDQ ? rr / p.group : rr;
    const int head_in_group = kDQ ? rr % p.group : 0;
    const bool in_tile = !kDQ || rr < p.tps * p.group;
    int kc0 = 0, cnt = 0, n_acc = 0;
    for (int s = 0;; ++s) {
      const Segment& g = ctl->seg[s & 1];
      if (g.kind == 0) break;
      const int kind = g.kind, c0 = g.c0, n = g.c1 - g.c0, cols = g.cols_valid;
      const int per = (cols + kChunk - 1) / kChunk, tw = twice(g);
      const int tok = g.tile * sp.tile_rows + tok_in_tile;
      const bool live = in_tile && tok < g.rows;
      const bool real = in_tile && tok < g.rows_valid;
      const size_t row = (size_t)(g.row_start + tok);
      const int head = kDQ ? g.head * p.group + head_in_group : g.head;
      float nl_row = -INFINITY, nd_row = 0.f;
      if (kDQ && real) {
        nl_row = p.nl[(size_t)head * p.nq + row];
        nd_row = p.nd[(size_t)head * p.nq + row];
      }
      bool ok = true;
      for (int i = par; i < n; i += 2, ++cnt) {
        const uint32_t ph = (uint32_t)cnt & 1u;
        const int kc = kc0 + i, st = kc % kStages;
        const int left = cols - (kDQ ? c0 + i : ((c0 + i) >> tw) % per) * kChunk;
        if (!warp_wait(bar_x + 8u * (uint32_t)par, ph, abortf, p.err, 170)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[4][32];
        tmem_ld32(tX, r[0]);
        // Own view of the chunk (already complete: X needed it).
        if ((!kDQ || left < kChunk) &&
            !warp_wait(bar_bf + 8 * st, (kc / kStages) & 1, abortf, p.err, 171)) {
          ok = false;
          break;
        }
        // Each piece of X (and below of Y) is on its way while the one before it
        // is worked on.
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_ld_wait_regs(r[q]);
          if (q < 3) tmem_ld32(tX + 32 * (q + 1), r[q + 1]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 nl4 = make_float4(nl_row, nl_row, nl_row, nl_row);
            if (!kDQ) nl4 = reinterpret_cast<const float4*>(ctl->nl[st])[8 * q + e];
            const float2 x0 = ffma2(make_float2(__uint_as_float(r[q][4 * e]),
                                                __uint_as_float(r[q][4 * e + 1])),
                                    scale2, make_float2(nl4.x, nl4.y));
            const float2 x1 = ffma2(make_float2(__uint_as_float(r[q][4 * e + 2]),
                                                __uint_as_float(r[q][4 * e + 3])),
                                    scale2, make_float2(nl4.z, nl4.w));
            r[q][4 * e] = __float_as_uint(fast_exp2(x0.x));
            r[q][4 * e + 1] = __float_as_uint(fast_exp2(x0.y));
            r[q][4 * e + 2] = __float_as_uint(fast_exp2(x1.x));
            r[q][4 * e + 3] = __float_as_uint(fast_exp2(x1.y));
          }
        }
        if (!warp_wait(bar_y + 8u * (uint32_t)par, ph, abortf, p.err, 172)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (left < kChunk) {
          // Columns behind the sequence: P and dS are zero, and what the chunk
          // holds there (it may be NaN) becomes zero before it is an operand.
#pragma unroll
          for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (32 * q + u >= left) r[q][u] = 0u;
          }
          if (rr >= left) {
            uint8_t* base = sB + st * kStageBytes + rr * 128;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              reinterpret_cast<uint4*>(base)[u] = make_uint4(0u, 0u, 0u, 0u);
              if (!kDQ) reinterpret_cast<uint4*>(base + kTileBytes)[u] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
        }
        auto operands = [&](auto rest_c) {
          constexpr bool kRest = decltype(rest_c)::value;
          uint32_t y[2][16];
          tmem_ld16(tY, y[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16], dk[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // 16 columns of Y
              tmem_ld_wait_regs16(y[h]);
              if (2 * q + h < 7) {
                tmem_ld16(tY + 16 * (2 * q + h + 1), y[h ^ 1]);
              } else {
                tc_fence_before();
                mbar_arrive(bar_yf + 8u * (uint32_t)par);
              }
              if (left < kChunk) {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                  if (32 * q + 16 * h + u >= left) y[h][u] = 0u;
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float4 nd4 = make_float4(nd_row, nd_row, nd_row, nd_row);
                if (!kDQ) nd4 = reinterpret_cast<const float4*>(ctl->nd[st])[8 * q + 4 * h + e];
                const uint32_t* pr = &r[q][16 * h + 4 * e];
                const float2 p0 = make_float2(__uint_as_float(pr[0]), __uint_as_float(pr[1]));
                const float2 p1 = make_float2(__uint_as_float(pr[2]), __uint_as_float(pr[3]));
                const float2 d0 = fmul2(p0, fadd2(make_float2(__uint_as_float(y[h][4 * e]),
                                                              __uint_as_float(y[h][4 * e + 1])),
                                                  make_float2(nd4.x, nd4.y)));
                const float2 d1 = fmul2(p1, fadd2(make_float2(__uint_as_float(y[h][4 * e + 2]),
                                                              __uint_as_float(y[h][4 * e + 3])),
                                                  make_float2(nd4.z, nd4.w)));
                const int at = 8 * h + 2 * e;
                dk[at] = pack_bf16x2(d0.x, d0.y);
                dk[at + 1] = pack_bf16x2(d1.x, d1.y);
                if (kDQ) {   // what the rounding leaves
                  pk[at] = rest_bf16x2(d0, dk[at]);
                  pk[at + 1] = rest_bf16x2(d1, dk[at + 1]);
                } else {
                  pk[at] = pack_bf16x2(p0.x, p0.y);
                  pk[at + 1] = pack_bf16x2(p1.x, p1.y);
                }
                if (kRest) {
                  dk[at] = rest_bf16x2(d0, dk[at]);
                  dk[at + 1] = rest_bf16x2(d1, dk[at + 1]);
                  pk[at] = rest_bf16x2(p0, pk[at]);
                  pk[at + 1] = rest_bf16x2(p1, pk[at + 1]);
                }
              }
            }
            tmem_st16(tX + 16 * q, pk);
            tmem_st16(tX + 64 + 16 * q, dk);
          }
        };
        if (!kDQ && (tw & (c0 + i)) != 0) operands(std::true_type{});
        else operands(std::false_type{});
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_p + 8u * (uint32_t)par);
      }
      if (ok && n > 0) ok = warp_wait(bar_acc, n_acc & 1, abortf, p.err, 173);
      if (ok) {
        tc_fence_after();
        // Key walk: the even group writes dV, the odd one dK; query walk: each
        // group half of dQ.
        constexpr int kHalves = kDQ ? 1 : 2;
        const bool scaled = kDQ || par == 1;
        const size_t part = ((size_t)blockIdx.x * 2 + g.slot) * 128 + rr;
        const uint32_t tAcc = tmem + lane_off + (kDQ ? kColA2 + 32u * (uint32_t)par
                                                     : par == 0 ? kColA1 : kColA2);
#pragma unroll
        for (int hc = 0; hc < kHalves; ++hc) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(tAcc + 32 * hc, o);
            tmem_ld_wait_regs(o);
          }
          const bool zero = n == 0 || !real;
          const int col = kDQ ? 32 * par : 32 * hc;
          if (kind != 1) {
            float4* dst = reinterpret_cast<float4*>(
                p.part[kDQ ? 1 : 0] + part * (kDQ ? 64 : 128) + (kDQ ? 0 : 64 * par) + col);
#pragma unroll
            for (int u = 0; u < 8; ++u)
              dst[u] = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]),
                                          __uint_as_float(o[4 * u + 2]), __uint_as_float(o[4 * u + 3]));
          } else if (live) {
            const float f = scaled ? 0.125f : 1.0f;
            __nv_bfloat16* t = kDQ ? p.dq : par == 0 ? p.dv : p.dk;
            uint4* dst = reinterpret_cast<uint4*>(
                t + (row * (kDQ ? p.heads : p.kv_heads) + head) * kHeadDim + col);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = zero ? 0u
                            : pack_bf16x2(__uint_as_float(o[8 * u + 2 * j]) * f,
                                          __uint_as_float(o[8 * u + 2 * j + 1]) * f);
              dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      if (n > 0) ++n_acc;
      kc0 += n;
      if (!end_of_item()) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    cross_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_qg,
                     const __grid_constant__ CUtensorMap tm_dog,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024_shared(smem_raw);
  if (blockIdx.y == 0) bwd_walk<false>(&tm_k, &tm_v, &tm_q, &tm_do, p, smem);
  else bwd_walk<true>(&tm_qg, &tm_dog, &tm_k, &tm_v, p, smem);
}

// Adds the parts of the items that were cut (see ress_sched.cuh) in the order
// of their chunks: blockIdx.y the walk, one warp per row at a time.
__global__ void __launch_bounds__(256)
    cross_bwd_combine_kernel(const __grid_constant__ BwdParams p) {
  const bool dq = blockIdx.y == 1;
  const SchedParams& sp = p.sched[dq ? 1 : 0];
  const int first = (int)blockIdx.x;
  wait_for_previous_kernel();
  allow_next_kernel();
  const SplitItem it = load_split(p.split + (dq ? kSms : 0) + first);
  if (it.head < 0) return;
  const int lane = threadIdx.x & 31;
  const int width = dq ? 64 : 128;
  for (int rr = (int)blockIdx.z * 32 + (threadIdx.x >> 5); rr < (int)blockIdx.z * 32 + 32; rr += 8) {
    const int tok = it.tile * sp.tile_rows + (dq ? rr / p.group : rr);
    if ((dq && rr >= p.tps * p.group) || tok >= it.rows) continue;
    float2 a = make_float2(0.f, 0.f), b = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < it.parts; ++k) {
      const size_t part = part_slot(it, first, sp.grid, k) * 128 + rr;
      const float2* src = reinterpret_cast<const float2*>(p.part[dq ? 1 : 0] + part * width);
      a = fadd2(a, src[lane]);
      if (!dq) b = fadd2(b, src[32 + lane]);
    }
    const size_t row = (size_t)(it.row_start + tok);
    if (dq) {
      const int head = it.head * p.group + rr % p.group;
      reinterpret_cast<uint32_t*>(p.dq + (row * p.heads + head) * kHeadDim)[lane] =
          pack_bf16x2(a.x * 0.125f, a.y * 0.125f);
    } else {
      const size_t at = (row * p.kv_heads + it.head) * kHeadDim;
      reinterpret_cast<uint32_t*>(p.dv + at)[lane] = pack_bf16x2(a.x, a.y);
      reinterpret_cast<uint32_t*>(p.dk + at)[lane] = pack_bf16x2(b.x * 0.125f, b.y * 0.125f);
    }
  }
}

struct BwdLayout {
  size_t nl, nd, part_k, part_q, split, total;
};
BwdLayout bwd_layout(const CrossGeometry& g) {
  BwdLayout l{};
  const size_t rows = align256(sizeof(float) * (size_t)g.heads * g.nq);
  const size_t part = sizeof(float) * (size_t)kSms * 2 * 128;
  l.nd = rows;
  l.part_k = 2 * rows;
  l.part_q = l.part_k + part * 128;
  l.split = l.part_q + part * 64;
  l.total = align256(l.split + 2 * kSms * sizeof(SplitItem));
  return l;
}

}  // namespace

size_t cross_bwd_workspace(const CrossGeometry& g) {
  return g.nq == 0 && g.nk == 0 ? 0 : bwd_layout(g).total;
}

ress_status launch_cross_bwd(const CrossGeometry& g, CrossBwdParams c, void* ws, cudaStream_t st) {
  const BwdLayout lay = bwd_layout(g);
  uint8_t* base = static_cast<uint8_t*>(ws);
  BwdParams p{};
  p.err = c.err;
  p.nq = g.nq;
  p.heads = g.heads;
  p.kv_heads = g.kv_heads;
  p.group = g.group;
  p.tps = 128 / g.group;
  float* nl = reinterpret_cast<float*>(base + lay.nl);
  float* nd = reinterpret_cast<float*>(base + lay.nd);
  p.nl = nl;
  p.nd = nd;
  p.dq = c.dq;
  p.dk = c.dk;
  p.dv = c.dv;
  p.part[0] = reinterpret_cast<float*>(base + lay.part_k);
  p.part[1] = reinterpret_cast<float*>(base + lay.part_q);
  p.split = reinterpret_cast<SplitItem*>(base + lay.split);
  for (int w = 0; w < 2; ++w) {
    SchedParams& s = p.sched[w];
    const bool dq = w == 1;
    s.err = c.err;
    s.row_off = dq ? c.q_off : c.k_off;
    s.row_lens = dq ? c.q_lens : c.k_lens;
    s.col_off = dq ? c.k_off : c.q_off;
    s.col_lens = dq ? c.k_lens : c.q_lens;
    s.rows = dq ? g.nq : g.nk;
    s.cols = dq ? g.nk : g.nq;
    s.row_detail = dq ? 90 : 91;
    s.col_detail = dq ? 91 : 90;
    s.seqs = g.seqs;
    s.heads = g.kv_heads;
    s.tile_rows = dq ? p.tps : 128;
    s.mult = dq ? 1 : g.group;
    s.twice_rows = dq ? 0 : kTwiceKeys;
    s.row_mult = 1;
    s.chunk_log2 = kChunkLog2;
    s.item_cost = 5 * kChunk;   // a ragged batch: 165 us at 2 chunks, 151 us at 5
    s.min_share = kMinShare;
    s.grid = kSms;
    sched_plan_on_host(&s);
  }
  CUtensorMap tq, tdo, tqg, tdog, tk, tv;
  const int64_t dense = (int64_t)g.heads * kHeadDim;
  if (g.nq > 0) {
    if (!make_rows_map(&tq, c.q, g.heads, g.nq, g.q_stride, 1, 128) ||
        !make_rows_map(&tdo, c.dout, g.heads, g.nq, dense, 1, 128) ||
        !make_rows_map(&tqg, c.q, g.heads, g.nq, g.q_stride, g.group, p.tps) ||
        !make_rows_map(&tdog, c.dout, g.heads, g.nq, dense, g.group, p.tps))
      return RESS_ERR_CUDA;
    const long long threads = (long long)g.nq * g.heads * 8;
    if (ress_status e = record_cuda(
            launch_behind(cross_delta_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0,
                          st, c.out, c.dout, c.lse, nl, nd, g.nq, g.heads)))
      return e;
  }
  if (g.nk > 0 && (!make_rows_map(&tk, c.k, g.kv_heads, g.nk, g.k_stride, 1, 128) ||
                   !make_rows_map(&tv, c.v, g.kv_heads, g.nk, g.v_stride, 1, 128)))
    return RESS_ERR_CUDA;
  // Without rows on one side no item has a chunk, and its maps are not used.
  if (g.nq == 0) tq = tdo = tqg = tdog = tk;
  if (g.nk == 0) tk = tv = tq;
  static std::atomic<uint64_t> allowed{0};
  if (ress_status e =
          allow_smem(reinterpret_cast<const void*>(cross_bwd_kernel), kSmem, &allowed))
    return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kSms, 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = g.nq > 0 ? 1 : 0;   // behind cross_delta_kernel
  if (ress_status e = record_cuda(
          cudaLaunchKernelEx(&cfg, cross_bwd_kernel, tq, tdo, tqg, tdog, tk, tv, p)))
    return e;
  if (p.sched[0].ns == 1 && p.sched[1].ns == 1) return RESS_OK;   // no item is cut
  return record_cuda(launch_dependent(cross_bwd_combine_kernel, dim3(kSms, 2, 4), dim3(256), st, p));
}

}  // namespace ress
