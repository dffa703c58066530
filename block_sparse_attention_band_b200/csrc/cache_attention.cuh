// Causal attention of packed query rows over a paged e4m3 cache: what the kernel
// for few rows a request (cache_rows.cuh) and the one for many (cache_tiles.cuh)
// share.
#pragma once
#include "cache.cuh"

namespace prism {
namespace cache {

struct AttnParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int32_t *table, *lens, *starts;
  const uint32_t* mask;        // [n, hq, words] or null: every block kept
  const int* counts;           // [n, hkv] or null: blocks that some head of a KV head's group keeps
  long long q_tok, q_head;     // elements between rows and between heads of q
  long long page_stride;       // bytes between pages
  int n, tokens, hq, hkv, page_shift, num_pages, max_pages, words;
  int least, most;             // this kernel's requests: least <= rows x group <= most
  int choose;                  // both kernels are launched (see few_rows_will_do)
  float scale_log2;
};

// Rows of request i: [row0, row0 + rows), its tokens; clamped to the buffers.
struct Request {
  int row0, rows, len;
};
__device__ __forceinline__ Request request_of(const AttnParams& P, int i) {
  Request r;
  r.row0 = min(max(P.starts[i], 0), P.tokens);
  r.rows = min(max(P.starts[i + 1], r.row0), P.tokens) - r.row0;
  r.len = (int)min(max((long long)P.lens[i], 0ll), (long long)P.max_pages << P.page_shift);
  return r;
}

// Is request i as request_of takes it, with nothing clamped?
__device__ __forceinline__ bool inside(const AttnParams& P, int i) {
  const int a = P.starts[i], b = P.starts[i + 1], len = P.lens[i];
  return a >= 0 && b >= a && b <= P.tokens && len >= 0 && len <= (long long)P.max_pages << P.page_shift;
}

// One unit's run of steps within a CTA's share.
struct Segment {
  Request r;
  int i, h;        // request, KV head
  int first, live; // the unit's rows: [first, first + live) of the request's rows x group
  int limit;       // tokens that some row of it sees
  int low;         // tokens that every row of it sees
  int h0, h1;      // heads of the group among its rows
  int j0, j1, nt;  // steps of this segment, steps of the unit (with counts: kept ones)
  int none;        // with counts: no step is kept
  long long unit, step0;  // the unit's first place in the flat order, its first step's
};

// Walks a CTA's share [at, end) of the flat order: request, row tile, head, step.
// A request's rows are numbered token x group + head, or (kHeadMajor) head x
// tokens + token.  A unit counts kUnitCost steps more than it has, for its
// beginning and end: a share of many short units is as long as one of few long
// ones.  With counts, a unit's steps are its kept ones: a block mask leaves a
// share as many as any other.
template <int R, bool kHeadMajor, int kUnitCost>
struct Walk {
  long long at, end, unit;
  int i, rt, h, nt, tiles, kept;
  Request r;
  int g, least, most;

  __device__ __forceinline__ void init(const AttnParams& P) {
    g = P.hq / P.hkv;
    least = P.least;
    most = P.most;
  }
  __device__ __forceinline__ int token_of(const Request& q, int row) const {
    return kHeadMajor ? row % q.rows : row / g;
  }
  __device__ __forceinline__ int head_of(const Request& q, int row) const {
    return kHeadMajor ? row / q.rows : row % g;
  }
  __device__ __forceinline__ int row_tiles(const Request& q) const {
    const long long rows = (long long)q.rows * g;
    return rows < least || rows > most ? 0 : (int)((rows + R - 1) / R);
  }
  // tokens that a row of the request sees
  __device__ __forceinline__ int seen(const Request& q, int row) const { return seen_by(q, token_of(q, row)); }
  __device__ __forceinline__ int seen_by(const Request& q, int token) const {
    return min(max(q.len - q.rows + token + 1, 0), q.len);
  }
  // the most and the fewest that a row of rows [a, b] sees
  __device__ __forceinline__ int most_seen(const Request& q, int a, int b) const {
    return kHeadMajor && a / q.rows != b / q.rows ? seen_by(q, q.rows - 1) : seen(q, b);
  }
  __device__ __forceinline__ int least_seen(const Request& q, int a, int b) const {
    return kHeadMajor && a / q.rows != b / q.rows ? seen_by(q, 0) : seen(q, a);
  }
  __device__ __forceinline__ int steps_for(int tokens_seen) const { return max((tokens_seen + 127) >> 7, 1); }
  __device__ __forceinline__ int steps(const Request& q, int tile) const {
    const int last = min((long long)(tile + 1) * R, (long long)q.rows * g) - 1;
    return steps_for(most_seen(q, tile * R, last));
  }
  // steps of a request's tiles one after the other, by additions (a prompt has
  // hundreds of tiles, which one thread adds up)
  struct Tiles {
    int at, left;  // head-major: token of the tile's first row; rows left
  };
  __device__ __forceinline__ Tiles first_tile(const Request& q) const { return {0, q.rows * g}; }
  __device__ __forceinline__ int next_tile(const Request& q, Tiles& t, int tile) const {
    if (!kHeadMajor) return steps(q, tile);
    const int n = min(R, t.left), last = t.at + n - 1;
    t.left -= n;
    t.at += n;
    if (t.at >= q.rows) t.at = t.at < 2 * q.rows ? t.at - q.rows : t.at % q.rows;
    return steps_for(seen_by(q, min(last, q.rows - 1)));
  }
  __device__ __forceinline__ long long cost(const AttnParams& P, int req) const {
    const Request q = request_of(P, req);
    long long c = 0;
    const int n = row_tiles(q);
    if (n == 0) return 0;
    if (P.counts) return n * kept_cost(P, req);
    Tiles t = first_tile(q);
    for (int x = 0; x < n; ++x) c += next_tile(q, t, x) + kUnitCost;
    return c * P.hkv;
  }
  // of one row tile, all heads
  __device__ __forceinline__ long long kept_cost(const AttnParams& P, int req) const {
    long long c = 0;
    for (int x = 0; x < P.hkv; ++x) c += max(P.counts[(size_t)req * P.hkv + x], 1) + kUnitCost;
    return c;
  }
  __device__ __forceinline__ void begin(const AttnParams& P, long long lo, long long hi, int req, long long base) {
    at = lo;
    end = hi;
    i = req;
    if (at >= end) return;
    r = request_of(P, i);
    tiles = row_tiles(r);
    rt = 0;
    if (P.counts) {
      const long long all = kept_cost(P, i);
      rt = (int)((at - base) / all);
      unit = base + rt * all;
      h = 0;
      set_steps(P);
      while (at >= unit + nt + kUnitCost) {
        unit += nt + kUnitCost;
        ++h;
        set_steps(P);
      }
      return;
    }
    Tiles t = first_tile(r);
    nt = next_tile(r, t, 0);
    while (at >= base + (long long)P.hkv * (nt + kUnitCost)) {
      base += (long long)P.hkv * (nt + kUnitCost);
      nt = next_tile(r, t, ++rt);
    }
    h = (int)((at - base) / (nt + kUnitCost));
    unit = base + (long long)h * (nt + kUnitCost);
  }
  __device__ __forceinline__ void set_steps(const AttnParams& P) {
    kept = P.counts ? P.counts[(size_t)i * P.hkv + h] : 1;
    nt = P.counts ? max(kept, 1) : steps(r, rt);
  }
  __device__ __forceinline__ bool next(const AttnParams& P, Segment& s) {
    for (;;) {
      if (at >= end) return false;
      if (at >= unit + nt + kUnitCost) {  // on to the next unit
        unit += nt + kUnitCost;
        if (++h == P.hkv) {
          h = 0;
          if (++rt == tiles) {
            rt = 0;
            do {
              r = request_of(P, ++i);
              tiles = row_tiles(r);
            } while (tiles == 0);
          }
          if (!P.counts) set_steps(P);
        }
        if (P.counts) set_steps(P);
      }
      // step j of the unit is place kUnitCost + j of its
      s.step0 = unit + kUnitCost;
      s.j0 = (int)max(at - s.step0, 0ll);
      s.j1 = (int)min((long long)nt, end - s.step0);
      at = s.step0 + nt;
      if (s.j1 > s.j0) break;
    }
    s.r = r;
    s.i = i;
    s.h = h;
    s.first = rt * R;
    s.live = min(R, r.rows * g - rt * R);
    s.limit = most_seen(r, s.first, s.first + s.live - 1);
    s.low = least_seen(r, s.first, s.first + s.live - 1);
    s.h0 = head_of(r, s.first);
    s.h1 = kHeadMajor ? head_of(r, s.first + s.live - 1) : g - 1;
    if (!kHeadMajor) s.h0 = 0;
    s.nt = nt;
    s.none = P.counts && kept == 0;
    s.unit = unit;
    return true;
  }
};

// This CTA's share [lo, hi) of all steps and (in *s, after the next barrier)
// the request in which it begins; contains a barrier.
struct Share {
  int req;
  long long base, total, warp_sum[16];
};
template <int kThreads, class W>
__device__ __forceinline__ void find_share(const AttnParams& A, const W& walk, Share* s, long long& lo, long long& hi,
                                           long long& ctas) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (A.n + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, A.n), i1 = min(i0 + per, A.n);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) mine += walk.cost(A, i);
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  if (lane == 31) s->warp_sum[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s->warp_sum[w];
    total += s->warp_sum[w];
  }
  ctas = min((long long)gridDim.x, total);
  lo = hi = 0;
  if ((long long)blockIdx.x < ctas) {
    lo = total * blockIdx.x / ctas;
    hi = total * (blockIdx.x + 1) / ctas;
  }
  long long at = before + inc - mine;
  if (lo < hi && lo >= at && lo < at + mine)
    for (int i = i0; i < i1; ++i) {
      const long long c = walk.cost(A, i);
      if (lo < at + c) {
        s->req = i;
        s->base = at;
        break;
      }
      at += c;
    }
  if (tid == 0) s->total = total;
}

// A call whose requests may bring many rows launches both kernels, and each
// request's rows decide which of them takes it.  Where all requests of many rows
// together are little work, the few-row kernel takes them as well: 32 rows a
// unit, on twice the CTAs and with less to set up.  Both kernels decide alike,
// from the lengths: the few-row kernel's places in the flat order that those
// requests would take, at most kLittleWork of them (about 14 a CTA).  Measured,
// few-row against tile kernel, 4 heads a group, in us (a call from Python): 2176
// places (1 request, 128 new tokens over 1000) 47 against 62, 2624 (64 over 4000)
// 50 against 88, 3264 (4 requests, 48 over 1000) 52 against 58, 4000 (4, 40 over
// 2000) 61 against 61, 4800 (8, 24 over 2000) 68 against 61, 6144 (8, 64 over
// 300) 59 against 56; 8 heads a group within 3 us of these, but for one long
// request (24 over 32000, 6216 places), 75 against 127.
constexpr int kLittleWork = 4000;
constexpr int kFewUnitRows = 32, kFewUnitCost = 9;
template <int kThreads>
__device__ __forceinline__ bool few_rows_will_do(const AttnParams& A, int few_most, Share* s) {
  const int tid = threadIdx.x, lane = tid & 31;
  long long sum = 0;
  for (int i = tid; i < A.n; i += kThreads) {
    const Request r = request_of(A, i);
    const long long rows = (long long)r.rows * (A.hq / A.hkv);
    if (rows > few_most)
      sum += (rows + kFewUnitRows - 1) / kFewUnitRows * (max((r.len + 127) >> 7, 1) + kFewUnitCost) * A.hkv;
  }
  int mine = (int)min(sum, (long long)kLittleWork + 1);
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) s->warp_sum[tid >> 5] = mine;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += s->warp_sum[w];
  __syncthreads();  // (find_share uses the same words)
  return total <= kLittleWork;
}

// The steps of a segment that some head of its rows keeps (warp-collective;
// lane x holds the mask words of heads x and x + 32 of the group).
struct Kept {
  const uint32_t* base;
  int words, h0, h1, w;
  uint32_t own0, own1, any;
  __device__ __forceinline__ void begin(const AttnParams& P, const Segment& s) {
    h0 = s.h0;
    h1 = s.h1;
    words = P.words;
    base = P.mask ? P.mask + ((size_t)s.i * P.hq + (size_t)s.h * (P.hq / P.hkv)) * words : nullptr;
    w = -1;
    own0 = own1 = any = ~0u;
  }
  __device__ __forceinline__ int next(int j, int j1) {
    if (!base) return j;
    while (j < j1) {
      if (w != (j >> 5)) {
        w = j >> 5;
        const int lane = threadIdx.x & 31;
        own0 = lane >= h0 && lane <= h1 ? __ldg(base + (size_t)lane * words + w) : 0u;
        own1 = lane + 32 >= h0 && lane + 32 <= h1 ? __ldg(base + (size_t)(lane + 32) * words + w) : 0u;
        any = __reduce_or_sync(0xffffffffu, own0 | own1);
      }
      const uint32_t rest = any >> (j & 31);
      if (rest) return min(j + __ffs(rest) - 1, j1);
      j = (j | 31) + 1;
    }
    return j1;
  }
  // The k-th kept step (there are more than k): 32 words at a time.
  __device__ __forceinline__ int seek(int k) {
    if (!base) return k;
    const int lane = threadIdx.x & 31;
    for (int w0 = 0; w0 < words; w0 += 32) {
      uint32_t x = 0u;
      if (w0 + lane < words)
#pragma unroll 4
        for (int head = h0; head <= h1; ++head) x |= __ldg(base + (size_t)head * words + w0 + lane);
      int upto = __popc(x);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, upto > k);
      if (past) {
        const int at = __ffs(past) - 1;
        uint32_t bits = __shfl_sync(0xffffffffu, x, at);
        for (int before = __shfl_sync(0xffffffffu, upto, at) - __popc(bits); before < k; ++before) bits &= bits - 1u;
        return next((w0 + at) * 32 + __ffs(bits) - 1, words * 32);
      }
      k -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return 0;
  }
  __device__ __forceinline__ bool all(uint64_t heads) const {
    const uint64_t want = ((h1 >= 63 ? 0ull : 1ull << (h1 + 1)) - 1ull) & ~((1ull << h0) - 1ull);
    return (heads & want) == want;
  }
  // bit x: head x of the group keeps step j (the last one next() returned)
  __device__ __forceinline__ uint64_t heads(int j) const {
    if (!base) return ~0ull;
    const uint32_t lo = __ballot_sync(0xffffffffu, (own0 >> (j & 31)) & 1u);
    const uint32_t hi = __ballot_sync(0xffffffffu, (own1 >> (j & 31)) & 1u);
    return (uint64_t)hi << 32 | lo;
  }
};

// What the producer tells the other roles of a step.
struct PageWindow;
struct Step {
  float4 group[8];   // of 16 tokens: scale of K, log2 and inverse of V's, 0 if there is no such page
  uint32_t nan[4];   // tokens with a NaN among their values (tile kernel)
  uint64_t heads;    // heads that keep the step's block
  int j;             // the unit's step
  int last;          // the segment's last one
  int full;          // every row sees every token
  int there;         // every token is there (few-row kernel)
  __device__ __forceinline__ void set_page(int x, int npg, const PageWindow& w);  // page x of npg
};
// 32 entries of a request's table, one a lane, and the scales of their pages for
// one head; pg = -1: behind the request's last page, kNoPage: no page of the
// cache (an error only where a step reads it: a dropped block may have none).
struct PageWindow {
  static constexpr int kNoPage = -2;
  int pg = -1;
  float ks = 1.f, vs = 0.f;
  __device__ __forceinline__ void load(const AttnParams& A, const int32_t* entries, int pages, int w, int h) {
    pg = -1;
    const int p = 32 * w + (threadIdx.x & 31);
    if (p >= pages) return;
    pg = __ldg(entries + p);
    if (pg < 0 || pg >= A.num_pages) {
      pg = kNoPage;
    } else {
      ks = __ldg(A.ks + (size_t)pg * A.hkv + h);
      vs = __ldg(A.vs + (size_t)pg * A.hkv + h);
    }
  }
};
__device__ __forceinline__ void Step::set_page(int x, int npg, const PageWindow& w) {
  float4 f = make_float4(1.f, 0.f, 0.f, 0.f);
  if (w.pg >= 0) {
    const float vs = fmaxf(w.vs, exp2_int(kMinScaleExp));
    f = make_float4(w.ks, __log2f(vs), __fdividef(1.0f, vs), 1.f);  // (exact for powers of two)
  }
  for (int e = x * 8 / npg; e < (x + 1) * 8 / npg; ++e) group[e] = f;
}

// Factor of S: K's scale and the row's.  Above 0, so that it keeps a masked
// score at minus infinity.
__device__ __forceinline__ float score_scale(float ks, float c) { return fmaxf(ks * c, 1.2e-38f); }
// (volatile: read where it is used, so that no group's values wait in registers)
__device__ __forceinline__ float4 lds_v4(const float4* p) {
  float4 f;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(smem_u32(p)));
  return f;
}

__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
// Byte offset of row `row`, byte `b` in a 128-byte-swizzled tile of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int row, int b) {
  return (uint32_t)(row * 128 + ((((b >> 4) ^ (row & 7)) << 4) | (b & 15)));
}

// 16 dims of a row of Q, 8 threads a row: two e4m3 terms of Q / 2^ex; returns ex.
__device__ __forceinline__ int split_q(const float (&x)[16], uint32_t (&w0)[4], uint32_t (&w1)[4]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = fmaxf(top, finite_abs(x[e]));
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const int ex = scale_exp(top);
  const float inv = exp2_int(-ex);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w0[e] = w1[e] = 0;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const float a = x[4 * e + 2 * f], b = x[4 * e + 2 * f + 1];
      const float ya = fmaf(a, inv, a * 0.f), yb = fmaf(b, inv, b * 0.f);  // (infinite: NaN)
      const uint32_t t0 = to_e4m3x2(ya, yb);
      const float2 back = from_e4m3x2(t0);
      w0[e] |= t0 << (16 * f);
      w1[e] |= to_e4m3x2(ya - back.x, yb - back.y) << (16 * f);
    }
  }
  return ex;
}

// Clears the counters (CTA 0), reports lengths and row offsets that request_of
// clamps and, for a block mask, counts the kept blocks of each request and KV
// head: a warp each, which looks at its request by the way.  (The next kernel
// waits for the counts: CTA 0 looking at all requests made masked calls 1 us
// longer.)
constexpr int kPrepareThreads = 256;
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(const AttnParams P, unsigned* counters, int n, int* counts) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0)
    for (int x = threadIdx.x; x < n; x += kPrepareThreads) counters[x] = 0u;
  const int lane = threadIdx.x & 31, g = P.hq / P.hkv;
  const long long unit = (long long)blockIdx.x * (kPrepareThreads / 32) + (threadIdx.x >> 5);
  if (!P.mask)
    for (int i = threadIdx.x; i < P.n; i += kPrepareThreads)
      if (!inside(P, i)) set_device_error(kDevErrCache);
  if (!P.mask || unit >= (long long)P.n * P.hkv) return;
  const int req = (int)(unit / P.hkv);
  const bool good = inside(P, req);
  const int blocks = (request_of(P, req).len + 127) >> 7;
  const uint32_t* base = P.mask + (size_t)unit * g * P.words;  // (hq = hkv x group)
  int kept = 0;
  for (int w = lane; w * 32 < blocks; w += 32) {
    uint32_t x = 0u;
#pragma unroll 4
    for (int head = 0; head < g; ++head) x |= __ldg(base + (size_t)head * P.words + w);
    if (blocks - w * 32 < 32) x &= (1u << (blocks - w * 32)) - 1u;
    kept += __popc(x);
  }
  kept = __reduce_add_sync(0xffffffffu, kept);
  if (lane == 0) counts[unit] = kept;
  if (lane == 0 && !good) set_device_error(kDevErrCache);
}

}  // namespace cache
}  // namespace prism
