// Paged 8-bit key/value cache: the plan of a step (block tables, packed row
// offsets, slot numbers) and the store of its keys and values.
#pragma once
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace prism {
namespace cache {

constexpr int kDevErrCache = -13;  // == PRISM_ERR_CACHE

// ---------------------------------------------------------------------------
// plan: integer work on the request lengths, bound by latency (a decode step
// reads and writes about 25 bytes a request).  One launch and no wait between
// CTAs: every CTA scans all requests itself (at most 4096, so 8 a thread; a
// second launch or a grid-wide wait would cost more than the scan), then
// writes the slots and table entries of its own rows, found by a binary search
// in the scanned row offsets.  lens, starts and the state are written by every
// CTA for its part of the requests; only where they share memory with the
// inputs (a step in place) does the last CTA to finish its reads (a ticket)
// write them.  Measured (calls in one graph): 64 requests of one token 4.0 us,
// 1000 prompts with 250K rows 9.7 us, of which CTA 0's look at every page taken,
// four bytes a thread and four in flight, is the end.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxRequests = 4096;
constexpr int kPlanPerThread = kPlanMaxRequests / kPlanThreads;
constexpr int kPlanRowsPerThread = 2;
constexpr int kPlanRows = kPlanThreads * kPlanRowsPerThread;
constexpr int kPlanMaxGrid = 1024;  // the ticket word counts CTAs in its low 16 bits

struct PlanParams {
  const int32_t *held, *add;
  int32_t* ring;
  const int32_t* state;
  int32_t *table, *lens, *starts, *slots, *state_out;
  int n, page_shift, num_pages, max_pages, tokens;
  int apart;  // no output shares memory with an input
};

struct Sum3 {
  long long a, b, c;
};
__device__ __forceinline__ Sum3 shfl_up3(Sum3 v, int d) {
  return {__shfl_up_sync(0xffffffffu, v.a, d), __shfl_up_sync(0xffffffffu, v.b, d),
          __shfl_up_sync(0xffffffffu, v.c, d)};
}

// Largest i with first[i] <= x (first ascends, first[0] <= x); of equal ones
// the last, so a request without rows owns none.
__device__ __forceinline__ int owner_of(const int32_t* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams P) {
  extern __shared__ int32_t s_first[];  // [4][n]: first row, first opened page, first returned page, tokens of each request
  __shared__ Sum3 s_warp[kPlanThreads / 32];
  __shared__ int s_late, s_last;
  int32_t* first_row = s_first;
  int32_t* first_new = s_first + P.n;
  int32_t* first_back = s_first + 2 * P.n;
  int32_t* s_held = s_first + 3 * P.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << P.page_shift;
  const long long room = (long long)P.max_pages << P.page_shift;
  if (tid == 0) s_late = 0;

  // rows, opened pages and returned pages of this thread's requests
  const int per = (P.n + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(tid * per, P.n), i1 = min(i0 + per, P.n);
  int32_t held_[kPlanPerThread], add_[kPlanPerThread];
#pragma unroll
  for (int x = 0; x < kPlanPerThread; ++x)
    if (i0 + x < i1) {
      held_[x] = P.held[i0 + x];
      add_[x] = P.add[i0 + x];
    }
  const int head = P.state[0], count = P.state[1];
  auto request = [&](int x) -> Sum3 {
    const long long held = held_[x], add = add_[x], have = (held + page - 1) >> P.page_shift;
    if (add < 0) return {0, 0, have};
    return {add, ((held + add + page - 1) >> P.page_shift) - have, 0};
  };
  bool bad = false;
  Sum3 mine = {0, 0, 0};
#pragma unroll
  for (int x = 0; x < kPlanPerThread; ++x)
    if (i0 + x < i1) {
      const long long held = held_[x], add = add_[x];
      if (held < 0 || held > room || add < -1 || (add > 0 && held + add > room)) {
        bad = true;
        continue;
      }
      if (add > 0 && (held & (page - 1))) {  // its begun page has to be one of the cache's
        const int32_t e = P.table[(size_t)(i0 + x) * P.max_pages + (size_t)(held >> P.page_shift)];
        bad |= e < 0 || e >= P.num_pages;
      }
      const Sum3 r = request(x);
      mine.a += r.a;
      mine.b += r.b;
      mine.c += r.c;
    }
  Sum3 inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sum3 up = shfl_up3(inc, d);
    if (lane >= d) {
      inc.a += up.a;
      inc.b += up.b;
      inc.c += up.c;
    }
  }
  if (lane == 31) s_warp[warp] = inc;
  bad = __syncthreads_or(bad) != 0;
  Sum3 base = {0, 0, 0}, total = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const Sum3 t = s_warp[w];
    if (w < warp) {
      base.a += t.a;
      base.b += t.b;
      base.c += t.c;
    }
    total.a += t.a;
    total.b += t.b;
    total.c += t.c;
  }
  // all or nothing: a step that does not fit changes nothing
  const bool fits = !(bad || head < 0 || head >= P.num_pages || count < 0 || count > P.num_pages || total.a > P.tokens ||
                      total.b > count || count + total.c > P.num_pages);
  if (fits) {
    Sum3 at = {base.a + inc.a - mine.a, base.b + inc.b - mine.b, base.c + inc.c - mine.c};
#pragma unroll
    for (int x = 0; x < kPlanPerThread; ++x)
      if (i0 + x < i1) {
        const int i = i0 + x;
        const Sum3 r = request(x);
        first_row[i] = (int32_t)at.a;
        first_new[i] = (int32_t)at.b;
        first_back[i] = (int32_t)at.c;
        s_held[i] = held_[x];
        at.a += r.a;
        at.b += r.b;
        at.c += r.c;
      }
  }
  __syncthreads();
  auto ring_at = [&](long long k) {  // (head < num_pages, k <= num_pages)
    const long long x = head + k;
    return (size_t)(x >= P.num_pages ? x - P.num_pages : x);
  };

  // slots of this CTA's rows, and the table entries of the pages they open
  for (long long r0 = (long long)blockIdx.x * kPlanRows; r0 < P.tokens; r0 += (long long)gridDim.x * kPlanRows)
#pragma unroll
    for (int x = 0; x < kPlanRowsPerThread; ++x) {
      const long long t = r0 + x * kPlanThreads + tid;
      if (t >= P.tokens) continue;
      int32_t slot = -1;
      if (fits && t < total.a) {
        const int i = owner_of(first_row, P.n, (int)t);
        const long long held = s_held[i], pos = held + (t - first_row[i]);
        const long long have = (held + page - 1) >> P.page_shift, j = pos >> P.page_shift;
        const int off = (int)(pos & (page - 1));
        int32_t* entry = P.table + (size_t)i * P.max_pages + (size_t)j;
        int32_t pg;
        if (j >= have) {
          pg = P.ring[ring_at(first_new[i] + (j - have))];
          if (pg < 0 || pg >= P.num_pages) {  // not a page: no slot, reported below
            pg = -1;
            s_late = 1;
          }
          if (off == 0) *entry = pg;
        } else {
          pg = *entry;
        }
        if (pg >= 0) slot = (pg << P.page_shift) + off;
      }
      P.slots[t] = slot;
    }
  // pages of ended requests go behind the ring's last free page (places that
  // no page is taken from in this call: count + returned <= num_pages)
  if (fits) {
    bool none = false;
    for (long long k = (long long)blockIdx.x * kPlanThreads + tid; k < total.c;
         k += (long long)gridDim.x * kPlanThreads) {
      const int i = owner_of(first_back, P.n, (int)k);
      const int32_t pg = P.table[(size_t)i * P.max_pages + (size_t)(k - first_back[i])];
      none |= pg < 0 || pg >= P.num_pages;
      P.ring[ring_at(count + k)] = pg;
    }
    if (none) set_device_error(kDevErrCache);
  }
  auto write = [&](int i) {
    const int32_t held = P.held[i], add = P.add[i];
    P.lens[i] = !fits ? held : add < 0 ? 0 : held + add;
    P.starts[i] = fits ? first_row[i] : 0;
  };
  auto write_state = [&](bool late) {
    P.starts[P.n] = fits ? (int32_t)total.a : 0;
    P.state_out[0] = fits ? (int32_t)ring_at(total.b) : head;
    P.state_out[1] = fits ? (int32_t)(count - total.b + total.c) : count;
    P.state_out[2] = 0;
    const int status = fits && !late ? 0 : kDevErrCache;
    P.state_out[3] = status;
    if (status) set_device_error(status);
  };
  if (gridDim.x > 1 && P.apart) {
    // every CTA writes its part; CTA 0 sees for itself whether each page taken is one
    for (int i = blockIdx.x * kPlanThreads + tid; i < P.n; i += gridDim.x * kPlanThreads) write(i);
    if (blockIdx.x != 0) return;
    bool late = false;
    if (fits)
#pragma unroll 4
      for (long long k = tid; k < total.b; k += kPlanThreads) {
        const int32_t pg = P.ring[ring_at(k)];
        late |= pg < 0 || pg >= P.num_pages;
      }
    late = __syncthreads_or(late) != 0;
    if (tid == 0) write_state(late);
    return;
  }
  __syncthreads();
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      const unsigned was = atomicAdd(reinterpret_cast<unsigned*>(P.state_out) + 2, 1u + ((unsigned)s_late << 16));
      s_last = (was & 0xffffu) == gridDim.x - 1;
      s_late |= (int)(was >> 16);
      __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
  }
  for (int i = tid; i < P.n; i += kPlanThreads) write(i);
  __syncthreads();  // (a thread's held and state are read before another's lens and state are written)
  if (tid == 0) write_state(s_late != 0);
}

// ---------------------------------------------------------------------------
// store: bf16 rows -> e4m3 codes with one scale for each (page, KV head).
//
// s = 2^ceil(log2(amax / 448)), the smallest power of two that brings the
// page's largest value into e4m3's range (448 = 1.75 2^8), from the bits of
// amax.  A power of two costs a floating-point code nothing in relative
// precision, makes x / s exact (one rounding, to the code), and lets a page
// that grows under single-token appends be moved to a larger scale exactly
// (only codes that become subnormal round again).
//
// Bound by HBM: 4 bytes read and 2 written for each K/V element pair.  A team
// of page / 16 warps holds a page's rows in registers (8 x 16 bytes a lane, 16
// rows a warp), so each value is read once for both its maximum and its code.
// Measured (calls in one graph): 131072 tokens of 8 heads 149 us, 5.4 TB/s (83 %
// of a copy's rate) at four CTAs an SM (152 to 160 us call by call, into other
// caches each time); 159 us at five, 155 at three, 175 with the rows read before
// the slots; 64 single tokens 4.5 us.
// ---------------------------------------------------------------------------
constexpr int kStoreThreads = 256;
constexpr int kMinScaleExp = -64;

struct StoreParams {
  const __nv_bfloat16 *k, *v;
  const int32_t* slots;
  uint8_t *kc, *vc;
  float *ks, *vs;
  long long k_tok, k_head, v_tok, v_head;  // elements between rows and between heads
  long long page_stride;                   // bytes between pages
  int tokens, hkv, page_shift, num_pages, window;
};

// Exponent of the page scale for a finite amax >= 0.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // mantissa over 1.75
  return max(e, kMinScaleExp);  // (zero and subnormal amax have e < the minimum)
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two fp32 -> two e4m3 codes (low byte = lo), to nearest even.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_from_f16x2(uint32_t halves) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(halves));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return h;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  uint32_t h = f16x2_from_e4m3x2(codes);
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// bf16 pair -> codes at 1 / s.  x 0 is NaN for an infinite x and adds nothing
// to a finite one, so infinities become NaN codes instead of the largest value.
__device__ __forceinline__ uint32_t encode2(uint32_t w, float inv) {
  const float a = bf16lo(w), b = bf16hi(w);
  return to_e4m3x2(fmaf(a, inv, a * 0.f), fmaf(b, inv, b * 0.f));
}
__device__ __forceinline__ float finite_abs(float x) {
  x = fabsf(x);
  return x < INFINITY ? x : 0.f;
}

__device__ __forceinline__ void team_sync(int team, int team_warps) {
  if (team_warps == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(team_warps * 32) : "memory");
}

__global__ void __launch_bounds__(kStoreThreads) store_kernel(const StoreParams P) {
  __shared__ float s_max[kStoreThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int page = 1 << P.page_shift;
  const int team_warps = page >> 4, team = warp / team_warps, tw = warp - team * team_warps;
  const int teams = (kStoreThreads / 32) / team_warps;
  const int head = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const __nv_bfloat16* src = is_v ? P.v + head * P.v_head : P.k + head * P.k_head;
  const long long tok_stride = is_v ? P.v_tok : P.k_tok;
  uint8_t* codes = is_v ? P.vc : P.kc;
  float* scales = is_v ? P.vs : P.ks;
  const int slot_end = P.num_pages << P.page_shift;

  const long long w0 = ((long long)blockIdx.x * teams + team) * P.window;
  const int t_end = (int)min(w0 + P.window, (long long)P.tokens);
  for (long long t0 = w0; t0 < t_end; t0 += 32) {
    // rows of the window at which a run of rows of one page begins
    const int t = (int)t0 + lane;
    int32_t here = -1, before = -1;
    if (t < t_end) {
      here = P.slots[t];
      if (t > 0) before = P.slots[t - 1];
    }
    if (here >= slot_end || here < -1) {
      here = -1;
      if (t < t_end) set_device_error(kDevErrCache);
    }
    const bool begins = here >= 0 && (before < 0 || (before >> P.page_shift) != (here >> P.page_shift));
    uint32_t starts = __ballot_sync(0xffffffffu, begins);
    while (starts) {
      const int b = __ffs(starts) - 1;
      starts &= starts - 1u;
      const int first = (int)t0 + b;
      const int slot0 = __shfl_sync(0xffffffffu, here, b);
      const int pg = slot0 >> P.page_shift, off0 = slot0 & (page - 1);
      // this warp's rows of the run: first + 16 tw + (0 .. 15)
      const int row0 = first + 16 * tw;
      const int past = first + page - off0;  // (slots that ascend leave the page here)
      if (tw == 0 && past < P.tokens && P.slots[past] >= 0 && (P.slots[past] >> P.page_shift) == pg)
        set_device_error(kDevErrCache);
      int32_t own = -1;
      if (lane < 16 && 16 * tw + lane < page - off0 && row0 + lane < P.tokens) own = P.slots[row0 + lane];
      if (own < 0 || (own >> P.page_shift) != pg) own = -1;
      uint4 x[8];
      uint32_t top2 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 2 * i + (lane >> 4);
        const bool live = __shfl_sync(0xffffffffu, own, r) >= 0;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (live) x[i] = ldg_nc_v4(src + (long long)(row0 + r) * tok_stride + (lane & 15) * 8);
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = w[e] & 0x7fff7fffu;
          __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&top2),
                                     *reinterpret_cast<const __nv_bfloat162*>(&a));  // (a NaN is left out)
          top2 = *reinterpret_cast<uint32_t*>(&m);
        }
      }
      top = fmaxf(bf16lo(top2), bf16hi(top2));
      if (!(top < INFINITY)) {  // an infinity among the values: the finite ones alone
        top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(finite_abs(bf16lo(w[e])), finite_abs(bf16hi(w[e]))));
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const size_t sc = (size_t)pg * P.hkv + head;
      const float old = off0 > 0 ? scales[sc] : 0.f;
      if (lane == 0) s_max[warp] = top;
      team_sync(team, team_warps);
      for (int w = 0; w < team_warps; ++w) top = fmaxf(top, s_max[team * team_warps + w]);
      team_sync(team, team_warps);  // every thread has read s_max and the old scale
      const float fresh = exp2_int(scale_exp(top));
      const float s = fmaxf(fresh, old);
      const float inv = 1.0f / s;
      uint8_t* base = codes + (size_t)pg * (size_t)P.page_stride + (size_t)head * (size_t)page * 128;
      if (tw == 0 && lane == 0 && s != old) scales[sc] = s;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 2 * i + (lane >> 4);
        const int slot = __shfl_sync(0xffffffffu, own, r);
        if (slot < 0) continue;
        uint2 c;
        c.x = encode2(x[i].x, inv) | (encode2(x[i].y, inv) << 16);
        c.y = encode2(x[i].z, inv) | (encode2(x[i].w, inv) << 16);
        *reinterpret_cast<uint2*>(base + (size_t)(slot & (page - 1)) * 128 + (lane & 15) * 8) = c;
      }
      // older rows of a page that was begun before, at the larger scale
      if (off0 > 0 && old < s) {
        const float ratio = old * inv;
        for (int r = 4 * tw + (lane >> 3); r < off0; r += 4 * team_warps) {
          uint4* cell = reinterpret_cast<uint4*>(base + (size_t)r * 128 + (lane & 7) * 16);
          uint4 c = *cell;
          uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 lo = from_e4m3x2(w[e] & 0xffffu), hi = from_e4m3x2(w[e] >> 16);
            w[e] = to_e4m3x2(lo.x * ratio, lo.y * ratio) | (to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
          }
          *cell = c;
        }
      }
    }
  }
}

}  // namespace cache
}  // namespace prism
