// Attention of packed query rows over packed keys (ress_cross_attn) and over
// the pages of the 8-bit cache (ress_cache_attn, long query ranges), on tcgen05.
//
// The query heads that share a key head stand in one tile: row r of a 128-row
// tile is (token r / group, query head r % group), so a key is read once for
// all of them and a few tokens fill a tile.  A CTA walks its share of the
// items (see ress_sched.cuh): per item it loads the query tile once and streams
// chunks of 128 keys through a ring.
//
//   kPair: 256 rows, one 128-row tile per softmax group; the groups take turns
//          on the tensor core and share each chunk of keys.
//   split: 128 rows, the two groups take the even and the odd chunks, each with
//          its own maximum, sum and accumulator; joined in the epilogue.  Used
//          where the second tile of a pair would be empty too often.
// Either way the tensor core sees one line of tasks i = 0, 1, ...: S of task i
// in TMEM buffer i % 3, its group i % 2.
//
// Warp roles:
//   0      TMA: query tiles, and keys and values of a packed batch
//   1      TMEM and MMA issue: S = Q K^T (128 x 128 x 64), O += P V (128 x 64 x 128)
//   2      the next item, while this one runs
//   4-11   softmax, one row per thread (online, log2 domain, lazy rescale when the
//          maximum grows by more than 2^8), epilogue
//   12-15  cache only: pages to bf16.  An e4m3 code is moved into the bits of a
//          bf16 number 2^-120 times its value and multiplied by 2^120 * scale,
//          which is exact for the cache's power-of-two scales, so the tensor
//          core sees code * scale without a rounding.  NaN codes are looked for
//          on the way (2,748 rows over 45,342 tokens and two smaller requests:
//          880 us without, 903 us with).
//
// Keys outside a row's range get -inf before the maximum; values of such keys
// are zeroed in shared memory (0 * NaN would reach the sums).
//
// Bound by the exponentials at d = 64 (1,024 cycles of MUFU for a chunk of a tile,
// 512 of tensor work) and by how well the groups' phases overlap: a tile's chunk
// takes about 1,260 cycles, over the cache 1,520 to 1,800, since the conversion
// competes for issue slots.  One view against 100 padded ones (16 heads): 1.02 ms,
// 775 TFLOP/s, 65 % of the exponentials' rate; 9,472 rows against 14,080: 888
// TFLOP/s.  Measured and left out: S and P in buffers of their own, so that S never
// waits for P V (one MMA warp 1.14 ms, one per group 1.17 ms against 1.06); 16
// softmax warps with half a row each (1.16 ms); a quarter or an eighth of the
// exponentials as polynomials on the FMA pipe (1 % either way, and they hide NaN).
#define RESS_WAIT_FN __forceinline__
#include "ress_common.cuh"
#include "ress_internal.h"
#include "ress_kv.h"
#include "ress_sched.cuh"

namespace ress {

namespace {

constexpr int kSms = 148;
constexpr uint32_t kTileBytes = 128 * 128;       // 128 rows of 64 bf16
constexpr uint32_t kStageBytes = 2 * kTileBytes; // keys, values
constexpr int kSBufs = 3;
constexpr int kMaxStages = 6;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 384;                  // S buffers at 0, 128, 256; O of group g at 384 + 64 g
constexpr float kScaleLog2 = 1.4426950408889634f * 0.125f;   // log2(e) / sqrt(64)
constexpr float kLn2 = 0.6931471805599453f;

template <bool kPair, bool kCache>
struct Cfg {
  static constexpr int threads = kCache ? 512 : 384;
  static constexpr int rows = kPair ? 256 : 128;
  static constexpr int stages = kPair ? 5 : 6;
  static constexpr uint32_t q_bytes = kPair ? 2 * kTileBytes : kTileBytes;
};

struct SeqAttnParams {
  SchedParams sched;
  DeviceError* err;
  int nq, heads, kv_heads, group, tps;   // tps: tokens of a 128-row tile
  __nv_bfloat16* out;
  float* lse;
  float* part_o;     // [grid][2][rows][64]
  float2* part_ml;   // [grid][2][rows]: maximum (log2 domain), sum
  SplitItem* split;  // [grid]
  // The cache.
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  int pages, page_log2, max_pages;
};

struct __align__(8) Ctl {
  uint64_t q_full;
  uint64_t kv_full[kMaxStages];
  uint64_t kv_empty[kMaxStages];
  uint64_t s_full[kSBufs];
  uint64_t p_full[kSBufs];
  uint64_t o_done[2];
  uint64_t o_full;
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int page_ok[kMaxStages][2];   // cache: a 64-key half of a stage comes from a page that counts
  Segment seg[2];
  float odd_m[128];
  float odd_l[128];
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          DeviceError* err, int detail) {
  const bool ok = mbar_wait(bar, parity, abort_flag, err, detail);
  return __all_sync(0xffffffffu, ok);
}

// Two e4m3 codes in the high bytes of each half: exponent and mantissa below bf16's
// sign, and the sign to bit 15, so that a half reads as 2^-120 times the code.
constexpr uint32_t kNanPair = 0x07f0u;   // the magnitude of a NaN code
__device__ __forceinline__ uint32_t code_magnitudes(uint32_t h) { return (h >> 4) & 0x07f007f0u; }
__device__ __forceinline__ uint32_t code_pair(uint32_t h, uint32_t mag, __nv_bfloat162 m) {
  uint32_t x = (h & 0x80008000u) | mag;
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x), m);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One row of 64 codes times `scale` into a 128-byte swizzled row of bf16.  Returns the
// largest magnitudes of the codes and `top`, in two halves.
__device__ __forceinline__ uint32_t store_codes(uint8_t* tile, int row, const uint4 (&w)[4],
                                                float scale, uint32_t top) {
  // 2^120 * scale passes bf16's range above scale 2^7: the rest is a second factor.
  const float lo = fminf(scale, 128.0f);
  const __nv_bfloat162 m = __float2bfloat162_rn(lo * 1.329227995784916e36f);   // 2^120
  const bool big = scale > 128.0f;
  const __nv_bfloat162 m2 = __float2bfloat162_rn(big ? scale * 0.0078125f : 1.0f);
  uint8_t* dst = tile + row * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t c[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
    uint32_t o[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t h0 = __byte_perm(c[u], 0, 0x1404), h1 = __byte_perm(c[u], 0, 0x3424);
      const uint32_t m0 = code_magnitudes(h0), m1 = code_magnitudes(h1);
      top = __vimax3_u16x2(top, m0, m1);
      o[2 * u] = code_pair(h0, m0, m);
      o[2 * u + 1] = code_pair(h1, m1, m);
    }
    if (big) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&o[u]), m2);
        o[u] = *reinterpret_cast<const uint32_t*>(&r);
      }
    }
    *reinterpret_cast<uint4*>(dst + (((2 * j) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(dst + (((2 * j + 1) ^ (row & 7)) << 4)) =
        make_uint4(o[4], o[5], o[6], o[7]);
  }
  return top;
}

__device__ __forceinline__ void store_bf16_half_row(__nv_bfloat16* dst, const float (&o)[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint4 v;
    v.x = pack_bf16x2(o[8 * u + 0], o[8 * u + 1]);
    v.y = pack_bf16x2(o[8 * u + 2], o[8 * u + 3]);
    v.z = pack_bf16x2(o[8 * u + 4], o[8 * u + 5]);
    v.w = pack_bf16x2(o[8 * u + 6], o[8 * u + 7]);
    reinterpret_cast<uint4*>(dst)[u] = v;
  }
}

// Registers per thread of the control, softmax and conversion warps.  Their sum
// over the warps is at most what the launch gives (512 * 128 or 384 * 168).
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <bool kPair, bool kCache>
__global__ void __launch_bounds__((Cfg<kPair, kCache>::threads), 1)
    seq_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const SeqAttnParams p) {
  using C = Cfg<kPair, kCache>;
  constexpr int kStages = C::stages;
  constexpr int kItemsPerChunk = kPair ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024_shared(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::q_bytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(sKV + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t bar_q = smem_addr(&ctl->q_full);
  const uint32_t bar_kvf = smem_addr(&ctl->kv_full[0]);
  const uint32_t bar_kve = smem_addr(&ctl->kv_empty[0]);
  const uint32_t bar_s = smem_addr(&ctl->s_full[0]);
  const uint32_t bar_p = smem_addr(&ctl->p_full[0]);
  const uint32_t bar_od = smem_addr(&ctl->o_done[0]);
  const uint32_t bar_o = smem_addr(&ctl->o_full);
  const uint32_t bar_done = smem_addr(&ctl->mma_done);
  volatile int* abortf = &ctl->abort_flag;

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_kvf + 8 * s, kCache ? 128 : 1);
      mbar_init(bar_kve + 8 * s, 1);
    }
    for (int b = 0; b < kSBufs; ++b) {
      mbar_init(bar_s + 8 * b, 1);
      mbar_init(bar_p + 8 * b, 128);
    }
    mbar_init(bar_od, 1);
    mbar_init(bar_od + 8, 1);
    mbar_init(bar_o, 1);
    mbar_init(bar_done, 1);
    ctl->abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&ctl->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 96) {
    tma_prefetch_desc(&tm_q);
    if (!kCache) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  wait_for_previous_kernel();
  allow_next_kernel();
  SchedWalk walk{0, 0, 0, 0, 0};
  SchedPlan plan;
  if (warp == 2) {
    plan = sched_begin(p.sched, (int)blockIdx.x, &walk);
    if (lane == 0) ctl->seg[0] = sched_next(p.sched, plan, walk);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  // Every role walks the same items; all of them meet at the end of each.
  auto end_of_item = [&]() -> bool {
    tc_fence_before();
    named_bar_sync(1, C::threads);
    tc_fence_after();
    return *abortf == 0;
  };

  if (warp < 4) {
    regs_dec<56>();
    if (warp == 0) {
      // ---------------- TMA ----------------
      int kc = 0, n_q = 0;   // chunks and query tiles loaded so far
      for (int s = 0;; ++s) {
        const Segment& g = ctl->seg[s & 1];
        if (g.kind == 0) break;
        const int c0 = g.c0, n = g.c1 - c0, head = g.head, col0 = g.col_start;
        if (n > 0) {
          if (elect_one()) {
            const int tok = g.row_start + g.tile * p.sched.tile_rows;
            const uint32_t bytes = (uint32_t)(p.tps * p.group) * 128u;
            mbar_arrive_expect_tx(bar_q, kPair ? 2 * bytes : bytes);
            tma_load_3d(smem_addr(sQ), &tm_q, bar_q, 0, head * p.group, tok);
            if (kPair)
              tma_load_3d(smem_addr(sQ) + kTileBytes, &tm_q, bar_q, 0, head * p.group, tok + p.tps);
          }
          __syncwarp();
          ++n_q;
          if (!kCache) {
            for (int c = 0; c < n; ++c, ++kc) {
              const int st = kc % kStages;
              if (kc >= kStages &&
                  !warp_wait(bar_kve + 8 * st, ((kc / kStages) - 1) & 1, abortf, p.err, 110))
                break;
              const uint32_t dst = smem_addr(sKV) + (uint32_t)st * kStageBytes;
              const uint32_t bar = bar_kvf + 8 * st;
              const int row = col0 + (c0 + c) * kChunk;
              if (elect_one()) {
                mbar_arrive_expect_tx(bar, kStageBytes);
                tma_load_3d(dst, &tm_k, bar, 0, head, row);
                tma_load_3d(dst + kTileBytes, &tm_v, bar, 0, head, row);
              }
              __syncwarp();
            }
          }
        }
        if (!end_of_item()) break;
      }
      // Copies still in flight (after a timeout) land before the CTA exits.
      if (!kCache)
        for (int c = kc > kStages ? kc - kStages : 0; c < kc; ++c)
          mbar_wait_drain(bar_kvf + 8 * (c % kStages), (c / kStages) & 1, p.err, 111);
      if (n_q > 0) mbar_wait_drain(bar_q, (n_q - 1) & 1, p.err, 112);
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- MMA issue ----------------
      // The softmax groups wait for this warp's next S, so its path from P(i) to
      // S(i + 3) is kept short: the stage's copies are awaited before P(i), and PV
      // and S are issued in one go.
      constexpr uint32_t idS = idesc_bf16_f32(128, 128, false);
      constexpr uint32_t idPV = idesc_bf16_f32(128, 64, true);
      const uint32_t dq = smem_desc_lo(smem_addr(sQ), 16);
      const uint32_t dk0 = smem_desc_lo(smem_addr(sKV), 16);
      const uint32_t dv0 = smem_desc_lo(smem_addr(sKV) + kTileBytes, 16384);
      constexpr uint32_t kStageDesc = kStageBytes >> 4, kTileDesc = kTileBytes >> 4;
      int kc0 = 0, it0 = 0, n_q = 0;
      bool any = false;
      for (int s = 0;; ++s) {
        const Segment& g = ctl->seg[s & 1];
        if (g.kind == 0) break;
        const int n = (g.c1 - g.c0) * kItemsPerChunk;
        if (n > 0) {
          bool ok = warp_wait(bar_q, n_q & 1, abortf, p.err, 120);
          any = true;
          auto wait_keys = [&](int i) -> bool {
            const int kc = kc0 + i / kItemsPerChunk;
            return warp_wait(bar_kvf + 8 * (kc % kStages), (kc / kStages) & 1, abortf, p.err, 121);
          };
          auto issue_s = [&](int i, int b) {   // one thread
            const uint32_t a = kPair ? dq + (uint32_t)(i & 1) * kTileDesc : dq;
            const uint32_t dk = dk0 + (uint32_t)((kc0 + i / kItemsPerChunk) % kStages) * kStageDesc;
            const uint32_t d = tmem + 128u * (uint32_t)b;
            mma_ss_lo<false>(d, a, dk, idS);
            mma_ss_lo<true>(d, a + 2, dk + 2, idS);
            mma_ss_lo<true>(d, a + 4, dk + 4, idS);
            mma_ss_lo<true>(d, a + 6, dk + 6, idS);
            mma_commit(bar_s + 8u * (uint32_t)b);
          };
          for (int i = 0; ok && i < n && i < kSBufs; ++i) {
            ok = wait_keys(i);
            tc_fence_after();
            if (ok && elect_one()) issue_s(i, (it0 + i) % kSBufs);
            __syncwarp();
          }
          for (int i = 0; ok && i < n; ++i) {
            const bool more = i + kSBufs < n;
            const int b = (it0 + i) % kSBufs;
            const int st = (kc0 + i / kItemsPerChunk) % kStages;
            const uint32_t dv = dv0 + (uint32_t)st * kStageDesc;
            const uint32_t tP = tmem + 128u * (uint32_t)b;
            const uint32_t tO = tmem + kColO + 64u * (uint32_t)(i & 1);
            if ((more && !wait_keys(i + kSBufs)) ||
                !warp_wait(bar_p + 8u * (uint32_t)b, ((it0 + i) / kSBufs) & 1, abortf, p.err, 122)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              mma_ts_lo(tO, tP, dv, idPV, i > 1 ? 1u : 0u);
#pragma unroll
              for (int kk = 1; kk < 8; ++kk)
                mma_ts_lo(tO, tP + kk * 8, dv + kk * 128, idPV, 1u);
              mma_commit(bar_od + 8u * (uint32_t)(i & 1));
              // S(i + 3) takes the buffer of P(i): the tensor core works in issue order.
              if (more) issue_s(i + kSBufs, b);
              if (!kPair || (i & 1)) mma_commit(bar_kve + 8 * st);
            }
            __syncwarp();
          }
          if (ok && elect_one()) mma_commit(bar_o);
          __syncwarp();
          kc0 += n / kItemsPerChunk;
          it0 += n;
          ++n_q;
        }
        if (!end_of_item()) break;
      }
      if (any) {
        if (elect_one()) mma_commit(bar_done);
        __syncwarp();
        mbar_wait_drain(bar_done, 0, p.err, 123);
      }
      __syncwarp();
    } else {
      // ---------------- the next item ----------------
      SplitItem split = no_split();
      for (int s = 0;; ++s) {
        const Segment& g = ctl->seg[s & 1];
        if (g.kind == 0) break;
        if (threadIdx.x == 64) {
          if (g.parts > 0) split = split_of(g);
          ctl->seg[(s + 1) & 1] = sched_next(p.sched, plan, walk);
        }
        if (!end_of_item()) break;
      }
      if (threadIdx.x == 64) store_split(p.split + blockIdx.x, split);
    }
  } else if (warp < 12) {
    // ---------------- softmax and epilogue ----------------
    regs_inc<kCache ? 184 : 224>();
    const int quad = warp & 3;
    const int par = (warp - 4) >> 2;
    const int rr = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tmem + kColO + lane_off + 64u * (uint32_t)par;
    const int tok_in_tile = rr / p.group + (kPair ? par * p.tps : 0);
    const int head_in_group = rr % p.group;
    const bool in_tile = rr < p.tps * p.group;
    const float2 scale2 = make_float2(kScaleLog2, kScaleLog2);
    int kc0 = 0, it0 = 0, pv = 0, n_o = 0;   // chunks, tasks, this group's PVs, items so far
    for (int s = 0;; ++s) {
      const Segment& g = ctl->seg[s & 1];
      if (g.kind == 0) break;
      const int kind = g.kind, n_ch = g.c1 - g.c0, c0 = g.c0, cols = g.cols_valid;
      const int tok = g.tile * p.sched.tile_rows + tok_in_tile;   // within the sequence
      const bool live = in_tile && tok < g.rows;
      const bool real = in_tile && tok < g.rows_valid;
      const int end = real ? (kCache ? step_end(cols, g.rows, tok, p.sched.step) : cols) : cols;
      const size_t row = (size_t)(g.row_start + tok);
      const int head = g.head * p.group + head_in_group;
      const bool warp_live = __any_sync(0xffffffffu, real);
      float m_ref = -INFINITY;
      float2 sum_a = make_float2(0.f, 0.f), sum_b = make_float2(0.f, 0.f);
      bool ok = true;
      const int n = n_ch * kItemsPerChunk;
      for (int i = par; i < n; i += 2) {
        const int lc = i / kItemsPerChunk;
        const int b = (it0 + i) % kSBufs;
        const uint32_t tS = tmem + lane_off + 128u * (uint32_t)b;
        const uint32_t bp = bar_p + 8u * (uint32_t)b;
        const int kc = kc0 + lc, st = kc % kStages;
        if (!warp_wait(bar_s + 8u * (uint32_t)b, ((it0 + i) / kSBufs) & 1, abortf, p.err, 130)) {
          ok = false;
          break;
        }
        const int left = cols - (c0 + lc) * kChunk;   // keys of the sequence from this chunk on
        bool hole0 = false, hole1 = false;
        if (kCache || left < kChunk) {
          // Own view of the stage's contents (already complete: S needed them).
          if (!warp_wait(bar_kvf + 8 * st, (kc / kStages) & 1, abortf, p.err, 131)) {
            ok = false;
            break;
          }
          if (kCache) {
            hole0 = ctl->page_ok[st][0] == 0;
            hole1 = ctl->page_ok[st][1] == 0;
          } else if (rr >= left && (!kPair || par == 0)) {
            // Values behind the sequence may be anything.  In a pair the even
            // group's P comes first, so its zeros are there for both.
            uint4* dst = reinterpret_cast<uint4*>(sKV + st * kStageBytes + kTileBytes + rr * 128);
#pragma unroll
            for (int u = 0; u < 8; ++u) dst[u] = make_uint4(0u, 0u, 0u, 0u);
          }
          if (!kCache) fence_proxy_async_smem();
        }
        tc_fence_after();
        if (!warp_live) {   // no query row in this warp: P is not looked at
          tc_fence_before();
          mbar_arrive(bp);
          ++pv;
          continue;
        }
        uint32_t r[4][32];
        tmem_ld32(tS, r[0]);
        tmem_ld32(tS + 32, r[1]);
        tmem_ld32(tS + 64, r[2]);
        tmem_ld32(tS + 96, r[3]);
        tmem_ld_wait_regs(r[0]);
        tmem_tie_regs(r[1]);
        tmem_tie_regs(r[2]);
        tmem_tie_regs(r[3]);
        const int lim = end - (c0 + lc) * kChunk;
        const bool masked = hole0 || hole1 || __any_sync(0xffffffffu, lim < kChunk);
        if (masked) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bool hole = q < 2 ? hole0 : hole1;
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (hole || 32 * q + u >= lim) r[q][u] = 0xFF800000u;
          }
        }
        float mxa[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) mxa[q] = -INFINITY;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mxa[2 * q] = fmax3(mxa[2 * q], __uint_as_float(r[q][4 * u]), __uint_as_float(r[q][4 * u + 1]));
            mxa[2 * q + 1] =
                fmax3(mxa[2 * q + 1], __uint_as_float(r[q][4 * u + 2]), __uint_as_float(r[q][4 * u + 3]));
          }
        }
        const float mx = fmaxf(fmaxf(fmax3(mxa[0], mxa[1], mxa[2]), fmax3(mxa[3], mxa[4], mxa[5])),
                               fmaxf(mxa[6], mxa[7]));
        const float m_new = mx * kScaleLog2;
        const bool grow = m_new > m_ref + 8.0f;
        const bool rescale_o = __any_sync(0xffffffffu, grow) && i > 1;
        float alpha = 1.0f;
        if (grow) {
          alpha = fast_exp2(m_ref - m_new);   // 0 on the row's first key
          sum_a.x *= alpha, sum_a.y *= alpha;
          sum_b.x *= alpha, sum_b.y *= alpha;
          m_ref = m_new;
        }
        // A row without a key yet has the reference -inf; its logits are -inf
        // too and must become 0, not NaN.
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        const float2 neg_m2 = make_float2(-m_use, -m_use);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 sv = make_float2(__uint_as_float(r[q][2 * e]), __uint_as_float(r[q][2 * e + 1]));
            const float2 x = ffma2(sv, scale2, neg_m2);
            const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            if (e & 1) sum_b = fadd2(sum_b, pe);
            else sum_a = fadd2(sum_a, pe);
            pk[e] = pack_bf16x2(pe.x, pe.y);
          }
          tmem_st16(tS + 16 * q, pk);
        }
        if (rescale_o) {
          // The group's previous PV (task i - 2) is done before O is touched;
          // its PV before that was done before S(i), so the parity is unambiguous.
          if (!warp_wait(bar_od + 8u * (uint32_t)par, (pv - 1) & 1, abortf, p.err, 132)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t o[32];
#pragma unroll
          for (int hc = 0; hc < 2; ++hc) {
            tmem_ld32(tO + 32 * hc, o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
            tmem_st32(tO + 32 * hc, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bp);
        ++pv;
      }
      float l = (sum_a.x + sum_a.y) + (sum_b.x + sum_b.y);
      float m = m_ref, a0 = 1.f, a1 = 0.f;
      const bool two = !kPair && n_ch > 1;
      if (!kPair) {
        if (par == 1) {
          ctl->odd_m[rr] = m_ref;
          ctl->odd_l[rr] = l;
        }
        named_bar_sync(2, 256);
        if (par == 0 && two) {
          const float m1 = ctl->odd_m[rr];
          m = fmaxf(m_ref, m1);
          const float mu = m == -INFINITY ? 0.f : m;
          a0 = fast_exp2(m_ref - mu);
          a1 = fast_exp2(m1 - mu);
          l = fmaf(a1, ctl->odd_l[rr], a0 * l);
        }
      }
      const bool writes = kPair || par == 0;   // warp-uniform
      if (ok && n_ch > 0) ok = warp_wait(bar_o, n_o & 1, abortf, p.err, 133);
      if (ok && writes) {
        tc_fence_after();
        // Logits that are NaN move no maximum, but reach the sum.
        if (m == -INFINITY && l != l) m = 0.f;
        const bool empty = !real || m == -INFINITY;
        const float inv = kind != 1 ? 1.f : empty ? 0.f : 1.0f / l;
        const size_t part = ((size_t)blockIdx.x * 2 + g.slot) * C::rows +
                            (kPair ? par * 128 : 0) + rr;
        if (kind != 1) p.part_ml[part] = empty ? make_float2(-INFINITY, 0.f) : make_float2(m, l);
        else if (live && p.lse != nullptr)
          p.lse[(size_t)head * p.nq + row] = empty ? -INFINITY : (m + __log2f(l)) * kLn2;
#pragma unroll
        for (int hc = 0; hc < 2; ++hc) {
          float o[32];
          if (n_ch > 0 && warp_live) {
            uint32_t oa[32], ob[32];
            tmem_ld32(tO + 32 * hc, oa);
            if (two) tmem_ld32(tO + 64 + 32 * hc, ob);
            tmem_ld_wait_regs(oa);
            tmem_tie_regs(ob);
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              o[u] = a0 * __uint_as_float(oa[u]);
              if (two) o[u] = fmaf(a1, __uint_as_float(ob[u]), o[u]);
              o[u] = empty ? 0.f : o[u] * inv;
            }
          } else {
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = 0.f;
          }
          if (kind == 1) {
            if (live) store_bf16_half_row(p.out + (row * p.heads + head) * kHeadDim + 32 * hc, o);
          } else if (!empty) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + part * kHeadDim + 32 * hc);
#pragma unroll
            for (int u = 0; u < 8; ++u)
              dst[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
          }
        }
      }
      if (n_ch > 0) ++n_o;
      kc0 += n_ch;
      it0 += n;
      if (!end_of_item()) break;
    }
  } else if (kCache) {
    // ---------------- pages to bf16 (one key row per thread) ----------------
    regs_dec<88>();
    const int row = threadIdx.x - 384;
    const int mask = (1 << p.page_log2) - 1;
    int kc = 0;
    for (int s = 0;; ++s) {
      const Segment& g = ctl->seg[s & 1];
      if (g.kind == 0) break;
      const int n = g.c1 - g.c0, cols = g.cols_valid, hk = g.head;
      const int32_t* tab = p.table + (size_t)g.b * p.max_pages;
      int pos = g.c0 * kChunk + row;
      uint4 kw[4], vw[4];
      float ks = 0.f, vs = 0.f;
      bool have = false, hole = false;
      // The row at `at`: codes and scales, if its page is one of the pool.
      auto fetch = [&](int id, int at) {
        have = at < cols && id >= 0 && id < p.pages;
        hole = at < cols && !have;
        if (have) {
          const size_t ph = (size_t)id * p.kv_heads + hk;
          const size_t off = ((ph << p.page_log2) + (size_t)(at & mask)) * kHeadDim;
          ks = p.k_scale[ph];
          vs = p.v_scale[ph];
          const uint4* ksrc = reinterpret_cast<const uint4*>(p.k_cache + off);
          const uint4* vsrc = reinterpret_cast<const uint4*>(p.v_cache + off);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            kw[u] = ksrc[u];
            vw[u] = vsrc[u];
          }
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
          ks = vs = 0.f;
        }
      };
      auto page_of = [&](int at) { return at < cols ? tab[at >> p.page_log2] : -1; };
      int id_next = n > 1 ? page_of(pos + kChunk) : -1;
      if (n > 0) fetch(page_of(pos), pos);
      for (int c = 0; c < n; ++c, ++kc, pos += kChunk) {
        const int st = kc % kStages;
        if (hole) raise_device_error(p.err, RESS_ERR_BAD_INDEX, 95);
        uint4 kcur[4], vcur[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) kcur[u] = kw[u], vcur[u] = vw[u];
        float kscale = ks, vscale = vs;
        bool hole_now = hole;
        if (!scale_ok(kscale) || !scale_ok(vscale)) {   // left out, like a page of no pool
          raise_device_error(p.err, RESS_ERR_INVALID_ARG, 96);
          kscale = vscale = 0.f;
          hole_now = true;
        }
        // The next chunk's codes, and the page of the one behind it, are on
        // their way while this one is converted.
        if (c + 1 < n) fetch(id_next, pos + kChunk);
        if (c + 2 < n) id_next = page_of(pos + 2 * kChunk);
        if (kc >= kStages &&
            !warp_wait(bar_kve + 8 * st, ((kc / kStages) - 1) & 1, abortf, p.err, 140))
          break;
        uint8_t* tile = sKV + st * kStageBytes;
        uint32_t top = store_codes(tile, row, kcur, kscale, 0u);
        top = store_codes(tile + kTileBytes, row, vcur, vscale, top);
        // A NaN code counts as 480 here, and a NaN value would also reach rows that do
        // not see it (0 * NaN).  So a token that holds one gets a key of NaN: its logits
        // are NaN for the rows that see it and masked for the others.
        if ((top & 0xffffu) == kNanPair || top >> 16 == kNanPair) {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(tile + row * 128 + 16 * u) =
                make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        }
        if ((row & 63) == 0) ctl->page_ok[st][row >> 6] = hole_now ? 0 : 1;
        fence_proxy_async_smem();
        mbar_arrive(bar_kvf + 8 * st);
      }
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

// Joins the parts of the item that CTA blockIdx.x of the kernel above began
// and did not end.
template <bool kPair>
__global__ void __launch_bounds__(256) seq_combine_kernel(const __grid_constant__ SeqAttnParams p) {
  constexpr int kRows = kPair ? 256 : 128;
  wait_for_previous_kernel();
  allow_next_kernel();
  const SplitItem it = load_split(p.split + blockIdx.x);
  if (it.head < 0) return;
  auto token_of = [&](int r) { return it.tile * p.sched.tile_rows + (r >> 7) * p.tps + (r & 127) / p.group; };
  auto head_of = [&](int r) { return it.head * p.group + (r & 127) % p.group; };
  const int left = it.rows - it.tile * p.sched.tile_rows;   // tokens of the tile and behind it
  const int n = left >= p.sched.tile_rows ? kRows
                : left > p.tps                ? 128 + (left - p.tps) * p.group
                                              : left * p.group;
  const int r0 = (int)blockIdx.y * 32;
  join_item<16>(
      it, (int)blockIdx.x, p.sched.grid, p.part_ml, p.part_o, kRows, r0, min(n, r0 + 32),
      [&](int r) -> __nv_bfloat16* {
        if ((r & 127) >= p.tps * p.group) return nullptr;
        return p.out + ((size_t)(it.row_start + token_of(r)) * p.heads + head_of(r)) * kHeadDim;
      },
      [&](int r) -> float* {
        return p.lse ? p.lse + (size_t)head_of(r) * p.nq + it.row_start + token_of(r) : nullptr;
      });
}

// Pairs share each chunk of keys between two tiles, which makes a tile's chunk
// 1.18 times as fast (1,024 rows against 40,000 keys, 16 heads: 212 us, split 250
// us), but pad a sequence to 256 rows (320 rows: 124 us, split 92 us; 192 rows: 71
// us, split 78 us; 64 rows: 59 us, split 47 us).  So: by the tiles either way of a
// sequence of the average length.
bool use_pair(int nq, int group, int seqs) {
  const long long rows = ((long long)nq * group + seqs - 1) / seqs;
  return (rows + 255) / 256 * 2 * 100 <= (rows + 127) / 128 * 118;
}

template <bool kPair, bool kCache>
ress_status launch_seq_typed(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             SeqAttnParams p, void* ws, cudaStream_t st) {
  using C = Cfg<kPair, kCache>;
  constexpr size_t smem = 1024 + C::q_bytes + C::stages * kStageBytes + sizeof(Ctl);
  static_assert(smem <= 227 * 1024, "shared memory");
  p.sched.tile_rows = p.tps * (kPair ? 2 : 1);
  sched_plan_on_host(&p.sched);
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)kSms * 2 * C::rows * kHeadDim);
  p.split = reinterpret_cast<SplitItem*>(p.part_ml + (size_t)kSms * 2 * C::rows);
  static std::atomic<uint64_t> allowed{0};
  if (ress_status s =
          allow_smem(reinterpret_cast<const void*>(seq_attn_kernel<kPair, kCache>), smem, &allowed))
    return s;
  if (ress_status s = record_cuda(launch_behind(seq_attn_kernel<kPair, kCache>, dim3(kSms),
                                                dim3(C::threads), smem, st, tq, tk, tv, p)))
    return s;
  if (p.sched.ns == 1) return RESS_OK;   // no item is cut
  return record_cuda(launch_dependent(seq_combine_kernel<kPair>, dim3(kSms, C::rows / 32),
                                      dim3(256), st, p));
}

size_t parts_bytes(bool pair) {
  return align256((size_t)kSms * 2 * (pair ? 256 : 128) * (kHeadDim * sizeof(float) + sizeof(float2)) +
                  kSms * sizeof(SplitItem));
}

}  // namespace

size_t cross_workspace(const CrossGeometry& g) {
  return g.nq == 0 ? 0 : parts_bytes(use_pair(g.nq, g.group, g.seqs));
}
// Up to 64 rows per request and key head on average, the step that adds a token
// or a few to every request, go to the register form of ress_cache_decode.cu.  64
// requests of 2,000 tokens, 4 key heads, both ways: 4 rows 30 and 69 us, 32 rows 40
// and 73 us, 64 rows 66 and 77 us, 128 rows 115 and 81 us.  The lengths are on the
// device, so the average decides for the whole call, and a batch that mixes the kinds
// pays for it: 2,048 rows of one request beside 47 single ones (2,000 tokens, 16 heads)
// take 213 us, in two calls 56 and 49 us.
static bool use_decode(int tokens, int group, int requests) {
  return (long long)tokens * group <= 64ll * requests;
}
size_t cache_attn_workspace(const ress_cache_shape& s, int heads, int tokens) {
  const int group = heads / s.kv_heads;
  if (tokens == 0) return 0;
  return use_decode(tokens, group, s.requests) ? cache_decode_workspace()
                                               : parts_bytes(use_pair(tokens, group, s.requests));
}

static ress_status launch_seq(const CrossParams& c, bool cache, void* ws, cudaStream_t st) {
  SeqAttnParams p{};
  p.err = c.err;
  p.nq = c.nq;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.group = c.group;
  p.tps = 128 / c.group;
  p.out = c.out;
  p.lse = c.lse;
  p.sched.err = c.err;
  p.sched.row_off = c.q_off;
  p.sched.row_lens = c.q_lens;
  p.sched.col_off = c.k_off;
  p.sched.col_lens = c.k_lens;
  p.sched.rows = c.nq;
  p.sched.cols = c.nk;
  p.sched.row_detail = 90;
  p.sched.col_detail = 91;
  p.sched.seqs = c.seqs;
  p.sched.heads = c.kv_heads;
  p.sched.mult = 1;
  p.sched.row_mult = 1;
  p.sched.chunk_log2 = kChunkLog2;
  p.sched.item_cost = kItemCost;
  p.sched.min_share = kMinShare;
  p.sched.grid = kSms;
  CUtensorMap tq, tk, tv;
  if (!make_rows_map(&tq, c.q, c.heads, c.nq, c.q_stride, c.group, p.tps)) return RESS_ERR_CUDA;
  tk = tv = tq;   // not used over the cache, nor without keys
  if (cache) {
    p.sched.lengths = c.lengths;
    p.sched.max_len = (long long)c.max_pages * c.page;
    p.sched.step = c.step;
    p.k_cache = c.k_cache;
    p.v_cache = c.v_cache;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.table = c.table;
    p.pages = c.pages;
    p.page_log2 = c.page == 64 ? 6 : 7;
    p.max_pages = c.max_pages;
  } else if (c.nk > 0 && (!make_rows_map(&tk, c.k, c.kv_heads, c.nk, c.k_stride, 1, 128) ||
                          !make_rows_map(&tv, c.v, c.kv_heads, c.nk, c.v_stride, 1, 128))) {
    return RESS_ERR_CUDA;
  }
  const bool pair = use_pair(c.nq, c.group, c.seqs);
  if (cache)
    return pair ? launch_seq_typed<true, true>(tq, tk, tv, p, ws, st)
                : launch_seq_typed<false, true>(tq, tk, tv, p, ws, st);
  return pair ? launch_seq_typed<true, false>(tq, tk, tv, p, ws, st)
              : launch_seq_typed<false, false>(tq, tk, tv, p, ws, st);
}

ress_status launch_cross(CrossParams p, void* ws, cudaStream_t st) {
  return launch_seq(p, false, ws, st);
}

ress_status launch_cache_attn(CrossParams p, void* ws, cudaStream_t st) {
  if (use_decode(p.nq, p.group, p.seqs)) return launch_cache_decode(p, ws, st);
  return launch_seq(p, true, ws, st);
}

}  // namespace ress
