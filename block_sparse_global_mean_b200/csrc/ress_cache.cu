// Paged 8-bit key/value cache: block tables and slot maps (plan) and the
// writer (append).
#include "ress_common.cuh"
#include "ress_internal.h"
#include "ress_kv.h"
#include "ress_seq.cuh"

namespace ress {

namespace {

// ---------------------------------------------------------------------------
// Plan.  Two exclusive sums over the requests (pages needed, tokens added),
// then independent lookups: every CTA takes the sums of all requests into its
// own shared memory and does its share of the table entries and slots, so one
// launch is enough and no CTA waits for another.
//
// Bound by latency: a decoding step moves a few hundred bytes, and even 512
// requests that add whole views (360,000 slots, 1.4 MB) are a microsecond of
// bandwidth next to the two dependent loads, the scan and the search: 3.2 us for 16
// requests of a token, 7.2 us for 512 of up to 1,408.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;

struct PlanParams {
  DeviceError* err;
  const int32_t* added;
  const int32_t* lengths;
  int32_t* table;
  const int32_t* free_pages;
  const int32_t* cursor;
  int32_t* offsets;
  int32_t* slots;
  int32_t* new_lengths;
  int32_t* new_cursor;
  int requests, max_pages, page, page_log2, pages, n_free, tokens;
};

// Tokens and new pages of one request.  A request whose numbers are wrong or
// whose row is too short adds no tokens to the cache and takes no pages (its
// tokens still stand in the packed order when the count itself is valid).
struct Ask {
  int len, add, old_pages, need;
  bool row_ok;
};
__device__ __forceinline__ Ask plan_ask(const PlanParams& p, int r) {
  Ask a;
  a.len = p.lengths[r];
  a.add = p.added[r];
  const bool numbers = a.len >= 0 && a.add >= 0;
  a.add = max(a.add, 0);
  const long long total = (long long)a.len + a.add;
  const int mask = p.page - 1;
  a.row_ok = numbers && total <= ((long long)p.max_pages << p.page_log2);
  a.old_pages = a.row_ok ? (a.len + mask) >> p.page_log2 : 0;
  a.need = a.row_ok ? (int)((total + mask) >> p.page_log2) - a.old_pages : 0;
  return a;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  int32_t* s_off = plan_smem;                       // [requests + 1] first packed token
  int32_t* s_first = s_off + p.requests + 1;        // [requests + 1] first new page (of all)
  int32_t* s_state = s_first + p.requests + 1;      // [requests] length, or -1 when it fails
  __shared__ longlong2 s_warp[kPlanThreads / 32];
  __shared__ int s_taken;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool lead = blockIdx.x == 0;
  wait_for_previous_kernel();
  const int cursor = p.cursor[0];
  const bool cursor_ok = cursor >= 0 && cursor <= p.n_free;
  if (threadIdx.x == 0) s_taken = 0;

  // Both sums run in 64 bits: no counts that int32 arrays can hold overflow them.
  long long page_sum = 0, token_sum = 0;
  for (int r0 = 0; r0 < p.requests; r0 += kPlanThreads) {
    const int r = r0 + threadIdx.x;
    Ask a{0, 0, 0, 0, false};
    if (r < p.requests) a = plan_ask(p, r);
    long long pages = a.need, toks = a.add;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, pages, o);
      const long long z = __shfl_up_sync(0xffffffffu, toks, o);
      if (lane >= o) pages += y, toks += z;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = make_longlong2(pages, toks);
    __syncthreads();
    long long first = page_sum + pages - a.need, tok = token_sum + toks - a.add;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const longlong2 sum = s_warp[w];
      if (w < warp) first += sum.x, tok += sum.y;
      page_sum += sum.x, token_sum += sum.y;
    }
    if (r < p.requests) {
      const bool tok_ok = tok + a.add <= p.tokens;
      const bool list_ok = a.need == 0 || (cursor_ok && cursor + first + a.need <= p.n_free);
      const bool ok = a.row_ok && tok_ok && list_ok;
      if (lead && !ok)
        raise_device_error(p.err, RESS_ERR_BAD_INDEX, !a.row_ok ? 100 : !tok_ok ? 102 : 101);
      s_off[r] = (int)min(tok, 0x7fffffffll);
      s_first[r] = (int)min(first, 0x7fffffffll);
      s_state[r] = ok ? a.len : -1;
      if (ok && lead && a.need > 0) atomicMax(&s_taken, (int)first + a.need);
    }
  }
  if (threadIdx.x == 0) {
    s_off[p.requests] = (int)min(token_sum, 0x7fffffffll);
    s_first[p.requests] = (int)min(page_sum, 0x7fffffffll);
  }
  __syncthreads();

  // Request r of a flat position: the last one whose first entry is <= i.
  auto owner = [&](const int32_t* first, int i) {
    int lo = 0, hi = p.requests - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  // (64 bits: a position within a stride of 2^31 would wrap past the end.)
  const long long stride = gridDim.x * kPlanThreads;
  const int at = blockIdx.x * kPlanThreads + threadIdx.x;
  const int mask = p.page - 1;

  for (long long r = at; r <= p.requests; r += stride) {
    p.offsets[r] = s_off[r];
    if (r < p.requests) {
      const int len = p.lengths[r];
      p.new_lengths[r] = s_state[r] >= 0 ? len + p.added[r] : len;
    }
  }
  if (at == 0) p.new_cursor[0] = cursor + s_taken;

  // New table entries.  Positions run over the pages asked for; those of a
  // request that failed are passed over.
  const int new_pages = min(s_first[p.requests], p.n_free);
  for (long long next = at; next < new_pages; next += stride) {
    const int i = (int)next, r = owner(s_first, i);
    if (s_state[r] < 0) continue;
    const int old_pages = (s_state[r] + mask) >> p.page_log2;
    const int32_t id = p.free_pages[cursor + i];
    if (id < 0 || id >= p.pages) raise_device_error(p.err, RESS_ERR_BAD_INDEX, 103);
    p.table[(size_t)r * p.max_pages + old_pages + (i - s_first[r])] = id;
  }

  // Slots.  The page of a token is an old table entry or the free-list entry
  // that the table gets, so nothing written above is read here.
  for (long long next = at; next < p.tokens; next += stride) {
    const int t = (int)next;
    int slot = -1;
    if (t < s_off[p.requests]) {
      const int r = owner(s_off, t);
      if (s_state[r] >= 0) {
        const int pos = s_state[r] + (t - s_off[r]);
        const int j = pos >> p.page_log2;
        const int old_pages = (s_state[r] + mask) >> p.page_log2;
        const int32_t id = j < old_pages ? p.table[(size_t)r * p.max_pages + j]
                                         : p.free_pages[cursor + s_first[r] + (j - old_pages)];
        if (id >= 0 && id < p.pages) slot = id * p.page + (pos & mask);
        else raise_device_error(p.err, RESS_ERR_BAD_INDEX, 103);
      }
    }
    p.slots[t] = slot;
  }
}

// ---------------------------------------------------------------------------
// Append.
// ---------------------------------------------------------------------------
struct AppendParams {
  DeviceError* err;
  const void* x[2];            // new keys, values
  long long stride[2];         // elements between their token rows
  const int32_t* slots;
  uint8_t* cache[2];           // [pages][kv_heads][page][64] codes
  float* scale[2];             // [pages][kv_heads]
  int tokens, kv_heads, page, pages;
};

// Exponent e of the smallest power of two with amax <= 448 * 2^e, at least
// -100: 448 = 1.75 * 2^8, so the mantissa of amax decides between two values.
// At most 119: a code up to 256 stands in a page of scale 2^120, which would be
// an infinity.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -100), 119);
}
constexpr uint32_t kMostBits = 0x7f600000u;   // 448 * 2^119: what a cell can hold
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two float32 values as e4m3 codes (nearest, ties to even, saturating); a is the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Eight consecutive values of a token row, as they stand in memory and in float32.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* src) {
    w = *reinterpret_cast<const uint4*>(src);
  }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  // Largest magnitudes so far, as the bits of two bf16.
  __device__ __forceinline__ uint32_t most(uint32_t top) const {
    top = __vmaxu2(top, w.x & 0x7fff7fffu);
    top = __vmaxu2(top, w.y & 0x7fff7fffu);
    top = __vmaxu2(top, w.z & 0x7fff7fffu);
    return __vmaxu2(top, w.w & 0x7fff7fffu);
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t top) {
    return max(top & 0xffff0000u, top << 16);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* src) {
    a = *reinterpret_cast<const float4*>(src);
    b = *(reinterpret_cast<const float4*>(src) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  // Largest magnitude so far, as bits.
  __device__ __forceinline__ uint32_t most(uint32_t top) const {
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
    return top;
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t top) { return top; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// A CTA per (window of `window` tokens, head, tensor), a thread per token of a
// page.  It finds the runs that start in its window (a run: consecutive slots
// within one page) from two bit masks, and each run passes through registers
// once: every warp loads 32 of its tokens, eight loads per lane in flight; the
// largest magnitude gives the page's scale; the codes go out 256 bytes per
// warp and store.
// The launch bound asks for the occupancy that measured best: 1,152 threads per SM
// for bf16 (56 registers; 49.8 us at 704 threads, 46.9 us so), 704 for float32,
// whose run is twice the registers (75.5 us without, 69.2 us so).
template <typename T, int kPage>
__global__ void __launch_bounds__(kPage, (sizeof(T) == 2 ? 1152 : 704) / kPage)
    cache_append_kernel(const AppendParams p, int window) {
  constexpr int kWarps = kPage / 32;
  __shared__ uint32_t s_cont[2 * kWarps + 1];   // token goes on with the run of the one before
  __shared__ uint32_t s_start[kWarps];          // token of the window that starts a run
  __shared__ uint32_t s_top[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = (int)(blockIdx.x & 1u);
  const int head = (int)((blockIdx.x >> 1) % (unsigned)p.kv_heads);
  const long long t0 = (long long)((blockIdx.x >> 1) / (unsigned)p.kv_heads) * window;
  constexpr int mask = kPage - 1;
  wait_for_previous_kernel();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const long long pos = t0 + u * kPage + threadIdx.x;
    bool cont = false, start = false;
    if (pos < p.tokens) {
      const int s = p.slots[pos];
      const int prev = pos > 0 ? p.slots[pos - 1] : -1;
      cont = s >= 0 && prev >= 0 && prev + 1 == s && (s & mask) != 0;
      start = u == 0 && s >= 0 && !cont && (int)threadIdx.x < window;
    }
    const unsigned c = __ballot_sync(0xffffffffu, cont), b = __ballot_sync(0xffffffffu, start);
    if (lane == 0) {
      s_cont[u * kWarps + warp] = c;
      if (u == 0) s_start[warp] = b;
    }
  }
  if (threadIdx.x == 0) s_cont[2 * kWarps] = 0u;
  __syncthreads();
  // Choices, not indexes: an indexed parameter would be copied to local memory.
  const T* x = static_cast<const T*>(which ? p.x[1] : p.x[0]) + (size_t)head * 64;
  const long long stride = which ? p.stride[1] : p.stride[0];
  uint8_t* const cache = which ? p.cache[1] : p.cache[0];
  float* const scales = which ? p.scale[1] : p.scale[0];
  const int col = (lane & 7) * 8;
  const int row0 = warp * 32 + (lane >> 3);   // of the run; then every fourth
  for (int word = 0; word < kWarps; ++word) {
    for (uint32_t todo = s_start[word]; todo != 0; todo &= todo - 1u) {
      const int bit = word * 32 + __ffs((int)todo) - 1;
      const long long first = t0 + bit;
      const int slot = p.slots[first];
      const int page = slot / kPage, c = slot & mask;
      if (page >= p.pages) {
        if (threadIdx.x == 0) raise_device_error(p.err, RESS_ERR_BAD_INDEX, 104);
        continue;
      }
      int n = 1;
      for (int i = bit + 1;;) {   // the tokens that go on with it (never past the page's end)
        const uint32_t off = ~(s_cont[i >> 5] >> (i & 31));
        const int room = 32 - (i & 31), ones = off == 0u ? 32 : __ffs((int)off) - 1;
        n += min(ones, room);
        if (ones < room || (i = (i | 31) + 1) >= 2 * kPage) break;
      }
      Eight<T> v[8];
      float* scale_at = scales + (size_t)page * p.kv_heads + head;
      const float old = c > 0 ? *scale_at : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (row0 + 4 * k < n) v[k].load(x + (first + row0 + 4 * k) * stride + col);
        else v[k].zero();
      }
      // Largest magnitude as bits, which order as the values do, with infinities
      // and NaN on top; the scale is that of the finite ones.  What no cell can
      // hold is flagged: those two, and values beyond 448 * 2^119.
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = v[k].most(top);
      top = __reduce_max_sync(0xffffffffu, Eight<T>::bits(top));
      if (top > kMostBits) {
        if (lane == 0) raise_device_error(p.err, RESS_ERR_INVALID_ARG, 105);
        top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float f[8];
          v[k].get(f);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint32_t b = __float_as_uint(f[u]) & 0x7fffffffu;
            top = max(top, b >= 0x7f800000u ? 0u : b);
          }
        }
        top = __reduce_max_sync(0xffffffffu, top);
      }
      if (lane == 0) s_top[warp] = top;
      __syncthreads();   // (and every thread has read the old scale)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = max(top, s_top[w]);
      const float amax = __uint_as_float(top);
      const float now = fmaxf(pow2(scale_exponent(amax)), old);
      const float inv = 1.0f / now;   // exact: a power of two
      uint8_t* dst = cache + ((size_t)page * p.kv_heads + head) * kPage * 64;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (row0 + 4 * k < n) {
          float f[8];
          v[k].get(f);
          uint2 o;
          o.x = e4m3x2(f[0] * inv, f[1] * inv) | e4m3x2(f[2] * inv, f[3] * inv) << 16;
          o.y = e4m3x2(f[4] * inv, f[5] * inv) | e4m3x2(f[6] * inv, f[7] * inv) << 16;
          *reinterpret_cast<uint2*>(dst + (c + row0 + 4 * k) * 64 + col) = o;
        }
      }
      if (now != old) {
        if (threadIdx.x == 0) *scale_at = now;
        const float ratio = old * inv;
        for (int i = threadIdx.x; i < c * 16; i += kPage) {   // older codes, four at a time
          uint32_t* at = reinterpret_cast<uint32_t*>(dst) + i;
          const uint32_t codes = *at;
          const float2 a = from_e4m3x2(codes & 0xffffu), b = from_e4m3x2(codes >> 16);
          *at = e4m3x2(a.x * ratio, a.y * ratio) | e4m3x2(b.x * ratio, b.y * ratio) << 16;
        }
      }
      __syncthreads();   // s_top is free again
    }
  }
}

template <typename T>
cudaError_t launch_append_typed(const AppendParams& p, cudaStream_t st) {
  // Runs that start in one window are written one after another.  Whole views
  // start one run per page of tokens, so a window is a page; short calls (a few
  // tokens each for many requests) start one per token or few (64 requests of one
  // token: 3.7 us; in one window their 64 runs would follow one another).  Windows of
  // 1, 8 and a page (64) tokens, 16 heads: 64 runs of 128 tokens 137, 20 and 12 us; 300
  // of 20 tokens 101, 20 and 15 us; 512 of 8 tokens 70 and 20 us (1, 8); 8,192 requests
  // of one token 264, 212 and 228 us, so a total above 4,096 of single tokens loses 7 %.
  const int window = p.tokens <= 1024 ? 1 : p.tokens <= 4096 ? 8 : p.page;
  const unsigned blocks = (unsigned)(((long long)p.tokens + window - 1) / window * p.kv_heads * 2);
  return p.page == 64
             ? launch_behind(cache_append_kernel<T, 64>, dim3(blocks), dim3(64), 0, st, p, window)
             : launch_behind(cache_append_kernel<T, 128>, dim3(blocks), dim3(128), 0, st, p, window);
}

}  // namespace

ress_status launch_cache_plan(const ress_cache_shape& s, const int32_t* added,
                              const int32_t* lengths, int32_t* table, const int32_t* free_pages,
                              int32_t n_free, const int32_t* cursor, int32_t tokens,
                              int32_t* offsets, int32_t* slots, int32_t* new_lengths,
                              int32_t* new_cursor, cudaStream_t st) {
  PlanParams p{};
  p.err = device_error_ptr();
  if (p.err == nullptr) return RESS_ERR_CUDA;
  p.added = added;
  p.lengths = lengths;
  p.table = table;
  p.free_pages = free_pages;
  p.cursor = cursor;
  p.offsets = offsets;
  p.slots = slots;
  p.new_lengths = new_lengths;
  p.new_cursor = new_cursor;
  p.requests = s.requests;
  p.max_pages = s.max_pages;
  p.page = s.page;
  p.page_log2 = s.page == 64 ? 6 : 7;
  p.pages = s.pages;
  p.n_free = n_free;
  p.tokens = tokens;
  auto smem_of = [](int requests) { return sizeof(int32_t) * (3 * (size_t)requests + 2); };
  const size_t smem = smem_of(s.requests);
  // Once and for the most requests that a call may have: set to each call's own size,
  // another thread's call could lower it before this one's launch.
  static std::atomic<uint64_t> allowed{0};
  if (smem > 48 * 1024)
    if (ress_status e = allow_smem(reinterpret_cast<const void*>(cache_plan_kernel),
                                   smem_of(kMaxSeqs), &allowed))
      return e;
  const long long items = (long long)tokens + s.requests;
  const long long blocks = (items + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  return record_cuda(launch_behind(cache_plan_kernel,
                                   dim3((unsigned)(blocks < 1 ? 1 : blocks > 148 ? 148 : blocks)),
                                   dim3(kPlanThreads), smem, st, p));
}

ress_status launch_cache_append(const ress_cache_shape& s, const void* k, const void* v, bool f32,
                                int64_t k_stride, int64_t v_stride, const int32_t* slots,
                                int32_t tokens, void* k_cache, void* v_cache, float* k_scale,
                                float* v_scale, cudaStream_t st) {
  AppendParams p{};
  p.err = device_error_ptr();
  if (p.err == nullptr) return RESS_ERR_CUDA;
  p.x[0] = k;
  p.x[1] = v;
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.slots = slots;
  p.cache[0] = static_cast<uint8_t*>(k_cache);
  p.cache[1] = static_cast<uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.tokens = tokens;
  p.kv_heads = s.kv_heads;
  p.page = s.page;
  p.pages = s.pages;
  return record_cuda(f32 ? launch_append_typed<float>(p, st)
                         : launch_append_typed<__nv_bfloat16>(p, st));
}

}  // namespace ress
