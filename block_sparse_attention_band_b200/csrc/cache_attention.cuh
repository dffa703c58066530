// Causal attention of packed query rows over a paged e4m3 cache.
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
  long long q_tok, q_head;     // elements between rows and between heads of q
  long long page_stride;       // bytes between pages
  int n, tokens, hq, hkv, page_shift, num_pages, max_pages, words;
  int least, most;             // this kernel's requests: least <= rows x group <= most
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

// ---------------------------------------------------------------------------
// Few rows a KV head (single tokens, drafts): tokens as the tensor cores' M.
//
// A work unit is up to R rows (row = token x head of the group) of one request
// and KV head; a step covers 128 tokens of its cache:
//   S^T [128 tokens, R]  = K Q^T          A = K (e4m3 as stored), B = Q
//   O^T [128 dims, 3 R] += V^T [P_0 P_1 P_2]   A = V (as stored, read dim-major)
// so K and V go from HBM to the tensor cores as they lie in the cache, by TMA
// and without a conversion, and the softmax threads (thread = token) only
// touch the rows that exist.
//
// What 8-bit operands cost in precision is bought back by more terms:
//   Q / s = q_0 + q_1, e4m3 each, s the row's power of two with max|Q| / s in
//     (224, 448]: 4 + 4 bits hold a bf16 value's 8 exactly, down to 2^-10 s;
//     both products add into the same S.
//   P = 2^-6 (p_0 + 2^-4 p_1 + 2^-8 p_2): each term leaves at most 2^-4 of
//     what it rounds, so 12 bits are kept down to 2^-24 of the largest P.
//     (Two terms would keep 8 bits but only down to 2^-20: a token that takes
//     most of the weight would cost the many small ones their precision.)
//   The three terms are separate columns of one product, added at the end.
// The scales of the pages are powers of two: K's multiplies S, V's is added to
// the exponent, P' = 2^(x + log2 vs - m), and taken out again in the row sum.
//
// Bound by HBM: 32 KB a step against 4 to 32 KB of row data a unit.  All CTAs
// (two an SM) take equal shares of the steps of all units, counted in one flat
// order that every CTA derives from the lengths itself, so a batch of any
// lengths is balanced to one step.  A unit that is cut by a share's end leaves
// (O, m, l) partials in the workspace, and the last of its CTAs to finish adds
// them in order (a counter a unit; the order of arrival changes no result).
//
// 192 threads: warps 0-3 softmax, warp 4 producer (page lookups 32 at a time,
// TMA), warp 5 tensor cores.
// ---------------------------------------------------------------------------
constexpr int kRowsThreads = 192;
constexpr uint32_t kStepBytes = 128 * 128;  // K or V of one step
constexpr int kRowsMaxCtas = 512;
constexpr float kGrow = 2.0f;       // the reference maximum moves when a value exceeds it by more (log2)
constexpr float kPScale = 6.0f;     // log2: P <= 2^kGrow -> first term <= 2^8
static_assert(kGrow + kPScale == 8.0f, "the first term's largest value is 256 (e4m3: 448)");

template <int R>
struct RowsCfg {
  static constexpr int kStages = R <= 16 ? 3 : 2;
  static constexpr uint32_t kQBytes = 2 * R * 128;  // two terms
  static constexpr uint32_t kPBytes = 3 * R * 128;  // three terms
  static constexpr uint32_t kOffQ = kStages * 2 * kStepBytes;
  static constexpr uint32_t kOffP = kOffQ + kQBytes;
  static constexpr uint32_t kSmem = kOffP + kPBytes + 1024;  // + slack for 1024-byte alignment
  static constexpr uint32_t kColS = 0;                       // two S buffers, then O
  static constexpr uint32_t kColO = 2 * R;
  static constexpr uint32_t kCols = R <= 16 ? 128 : 256;
  static_assert(5 * R <= (int)kCols, "tensor memory columns");
  static constexpr size_t kSlotFloats = (size_t)R * 130;  // O [R][128], m [R], l [R]
};

struct RowsParams {
  AttnParams A;
  float* partial;       // [2 * CTAs] slots
  unsigned* counters;   // [CTAs], zero
};

// One unit's run of steps within a CTA's share.
struct Segment {
  Request r;
  int i, h;        // request, KV head
  int first, live; // the unit's rows: [first, first + live) of the request's rows x group
  int limit;       // tokens that some row of it sees
  int low;         // tokens that every row of it sees
  int h0, h1;      // heads of the group among its rows
  int j0, j1, nt;  // steps of this segment, steps of the unit
  long long unit;  // flat index of the unit's first step
};

// Walks a CTA's share [at, end) of the flat order: request, row tile, head, step.
// A request's rows are numbered token x group + head, or (kHeadMajor) head x
// tokens + token.
template <int R, bool kHeadMajor>
struct Walk {
  long long at, end, unit;
  int i, rt, h, nt, tiles;
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
  __device__ __forceinline__ long long cost(const Request& q, int hkv) const {
    long long c = 0;
    const int n = row_tiles(q);
    if (n == 0) return 0;
    Tiles t = first_tile(q);
    for (int x = 0; x < n; ++x) c += next_tile(q, t, x);
    return c * hkv;
  }
  __device__ __forceinline__ void begin(const AttnParams& P, long long lo, long long hi, int req, long long base) {
    at = lo;
    end = hi;
    i = req;
    if (at >= end) return;
    r = request_of(P, i);
    tiles = row_tiles(r);
    rt = 0;
    Tiles t = first_tile(r);
    nt = next_tile(r, t, 0);
    while (at >= base + (long long)P.hkv * nt) {
      base += (long long)P.hkv * nt;
      nt = next_tile(r, t, ++rt);
    }
    h = (int)((at - base) / nt);
    unit = base + (long long)h * nt;
  }
  __device__ __forceinline__ bool next(const AttnParams& P, Segment& s) {
    if (at >= end) return false;
    if (at >= unit + nt) {  // on to the next unit
      unit += nt;
      if (++h == P.hkv) {
        h = 0;
        if (++rt == tiles) {
          rt = 0;
          do {
            r = request_of(P, ++i);
            tiles = row_tiles(r);
          } while (tiles == 0);
        }
        nt = steps(r, rt);
      }
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
    s.unit = unit;
    s.j0 = (int)(at - unit);
    s.j1 = (int)min((long long)nt, end - unit);
    at = unit + s.j1;
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
  for (int i = i0; i < i1; ++i) mine += walk.cost(request_of(A, i), A.hkv);
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
      const long long c = walk.cost(request_of(A, i), A.hkv);
      if (lo < at + c) {
        s->req = i;
        s->base = at;
        break;
      }
      at += c;
    }
  if (tid == 0) s->total = total;
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

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
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

__global__ void __launch_bounds__(32) zero_counters_kernel(unsigned* counters, int n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int x = threadIdx.x; x < n; x += 32) counters[x] = 0u;
}

template <int R>
__global__ void __launch_bounds__(kRowsThreads, 2)
attn_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const RowsParams P) {
  using C = RowsCfg<R>;
  constexpr int kStages = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bars[2 * kStages + 2 + 1 + 2 + 1 + 1];
  __shared__ float s_ks[kStages][8], s_vs[kStages][8];  // scales of a stage's pages; ks < 0: no such page
  __shared__ float s_c[R], s_thr[R], s_off[R], s_alpha[R], s_wmax[4][R], s_sum[4][R];
  __shared__ int s_see[R], s_head[R];
  __shared__ uint32_t s_nan[R][4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_any_nan, s_last;
  __shared__ volatile int s_fail;
  __shared__ Share s_share;

  const AttnParams& A = P.A;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sgen = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = A.hq / A.hkv;
  auto bar = [&](int x) { return smem_u32(&s_bars[x]); };
  const int kFull = 0, kEmpty = kStages, kSFull = 2 * kStages, kPFull = kSFull + 2, kODone = kPFull + 1,
            kQFull = kODone + 2, kDone = kQFull + 1;

  if (tid == 0) {
    for (int x = 0; x < kStages; ++x) {
      mbar_init(bar(kFull + x), 1);
      mbar_init(bar(kEmpty + x), 1);
    }
    mbar_init(bar(kSFull), 1);
    mbar_init(bar(kSFull + 1), 1);
    mbar_init(bar(kPFull), 128);
    mbar_init(bar(kODone), 1);
    mbar_init(bar(kODone + 1), 1);
    mbar_init(bar(kQFull), 128);
    mbar_init(bar(kDone), 128);
    fence_mbar_init();
    s_any_nan = 0;
    s_fail = 0;
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&s_tmem), C::kCols);
    tmem_relinquish();
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  // this CTA's share of all steps, and the request in which it begins
  Walk<R, false> walk;
  walk.init(A);
  long long lo, hi, ctas;
  find_share<kRowsThreads>(A, walk, &s_share, lo, hi, ctas);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  walk.begin(A, lo, hi, s_share.req, s_share.base);
  Segment sg;
  int gt = 0;  // steps done by this role

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int npg = 128 >> A.page_shift;  // pages a step
    const uint32_t pbytes = 128u << A.page_shift;
    bool ok = true;
    while (ok && walk.next(A, sg)) {
      const int32_t* entries = A.table + (size_t)sg.i * A.max_pages;
      const int pages = (sg.limit + (1 << A.page_shift) - 1) >> A.page_shift;  // of the unit
      struct Win {
        int pg;
        float ks, vs;
      };
      // 32 pages at a time: lane x holds page 32 w + x
      auto window = [&](int w) {
        Win v = {-1, -1.f, 0.f};
        const int p = 32 * w + lane;
        if (p < pages) {
          v.pg = __ldg(entries + p);
          if (v.pg < 0 || v.pg >= A.num_pages) {
            v.pg = -1;
            set_device_error(kDevErrCache);
          } else {
            v.ks = __ldg(A.ks + (size_t)v.pg * A.hkv + sg.h);
            v.vs = __ldg(A.vs + (size_t)v.pg * A.hkv + sg.h);
          }
        }
        return v;
      };
      Kept kept;
      kept.begin(A, sg);
      int j = kept.next(sg.j0, sg.j1);
      int w = j * npg >> 5;
      Win cur = {-1, -1.f, 0.f}, nxt = cur;
      if (j < sg.j1) {
        cur = window(w);
        nxt = window(w + 1);
      }
      for (; j < sg.j1; j = kept.next(j + 1, sg.j1)) {
        const int p0 = j * npg;
        if (p0 >> 5 != w) {
          if (p0 >> 5 == w + 1) cur = nxt;
          else cur = window(p0 >> 5);
          w = p0 >> 5;
          nxt = window(w + 1);
        }
        const int s = gt % kStages, x = lane - (p0 & 31);  // this lane's page of the step
        const bool mine = x >= 0 && x < npg;
        if (gt >= kStages && !(ok = __all_sync(0xffffffffu, mbar_wait(bar(kEmpty + s), (gt / kStages - 1) & 1)))) break;
        if (mine) {
          s_ks[s][x] = cur.ks;
          s_vs[s][x] = cur.vs;
        }
        const bool there = mine && cur.pg >= 0;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, there));
        if (lane == 0) mbar_arrive_expect_tx(bar(kFull + s), n * 2 * pbytes);
        __syncwarp();
        if (there) {
          const uint32_t dst = sbase + s * 2 * kStepBytes + x * pbytes;
          tma_load_4d(dst, &tmK, 0, 0, sg.h, cur.pg, bar(kFull + s));
          tma_load_4d(dst + kStepBytes, &tmV, 0, 0, sg.h, cur.pg, bar(kFull + s));
        }
        ++gt;
      }
    }
    if (!ok)  // given up: the copies in flight land before the CTA leaves
      for (int x = max(gt - kStages, 0); x < gt; ++x) mbar_wait(bar(kFull + x % kStages), (x / kStages) & 1);
    // what this kernel was launched beside is complete when it is
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else if (warp == 5) {
    // ------------------------------------------------------------ tensor cores
    constexpr uint32_t idS = idesc_e4m3_f32(128, R, 0, 0), idO = idesc_e4m3_f32(128, 3 * R, 1, 0);
    const uint64_t dQ = smem_desc_sw128(sbase + C::kOffQ, 16, 1024), dP = smem_desc_sw128(sbase + C::kOffP, 16, 1024);
    bool ok = true;
    auto qk = [&](int t) {
      const uint64_t dK = smem_desc_sw128(sbase + (t % kStages) * 2 * kStepBytes, 16, 1024);
#pragma unroll
      for (int x = 0; x < 8; ++x)  // four steps of 32 dims, first then second term of Q
        mma_f8_ss(tmem + C::kColS + (t & 1) * R, dK + (x & 3) * 2, dQ + (x >> 2) * (R * 128 / 16) + (x & 3) * 2, idS,
                  x > 0);
      mma_commit(bar(kSFull + (t & 1)));
    };
    int seg = 0;
    while (ok && walk.next(A, sg)) {
      Kept kept;
      kept.begin(A, sg);
      int j = kept.next(sg.j0, sg.j1);
      if (j >= sg.j1) continue;  // nothing kept
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kQFull), seg & 1)))) break;
      ++seg;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kFull + gt % kStages), (gt / kStages) & 1)))) break;
      tc_fence_after();
      if (lane == 0) qk(gt);
      for (bool first = true; j < sg.j1; first = false) {
        j = kept.next(j + 1, sg.j1);
        if (j < sg.j1) {
          const int t = gt + 1;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kFull + t % kStages), (t / kStages) & 1)))) break;
          tc_fence_after();
          if (lane == 0) qk(t);
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kPFull), gt & 1)))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dV =
              smem_desc_sw128(sbase + (gt % kStages) * 2 * kStepBytes + kStepBytes, kStepBytes, 1024);
#pragma unroll
          for (int x = 0; x < 4; ++x)  // 32 tokens a step
            mma_f8_ss(tmem + C::kColO, dV + x * (4096 / 16), dP + x * 2, idO, !first || x > 0);
          mma_commit(bar(kODone + (gt & 1)));
          mma_commit(bar(kEmpty + gt % kStages));
        }
        __syncwarp();
        ++gt;
      }
    }
    __syncwarp();
    mbar_wait(bar(kDone), 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    bool ok = true;
    // A wait that is given up is noted; the warps leave together at the next
    // barrier, none is left at one.
    auto waited = [&](uint32_t b, uint32_t parity) {
      const bool got = __all_sync(0xffffffffu, mbar_wait(b, parity));
      if (!got) s_fail = 1;
      return got;
    };
    while (ok && walk.next(A, sg)) {
      // Q of the unit's rows in two terms: 8 threads a row, 16 dims each
#pragma unroll
      for (int r0 = 0; r0 < R; r0 += 16) {
        const int r = r0 + (tid >> 3), c = tid & 7;
        const int row = (sg.first + r) / g, head = (sg.first + r) % g;
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.f;
        if (r < sg.live) {
          const __nv_bfloat16* src = A.q + (long long)(sg.r.row0 + row) * A.q_tok +
                                     (long long)(sg.h * g + head) * A.q_head + c * 16;
          const uint4 v[2] = {ldg_nc_v4(src), ldg_nc_v4(src + 8)};
          const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[2 * e] = bf16lo(w[e]);
            x[2 * e + 1] = bf16hi(w[e]);
          }
        }
        uint32_t w0[4], w1[4];
        const int ex = split_q(x, w0, w1);
        unsigned char* q0 = sgen + C::kOffQ + sw128(r, 16 * c);
        *reinterpret_cast<uint4*>(q0) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        *reinterpret_cast<uint4*>(q0 + R * 128) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        if (c == 0) {
          s_c[r] = exp2_int(ex) * A.scale_log2;
          s_thr[r] = r < sg.live ? -INFINITY : INFINITY;
          s_off[r] = kPScale;
          s_see[r] = r < sg.live ? walk.seen(sg.r, sg.first + r) : 0;
          s_head[r] = head;
          s_nan[r][0] = s_nan[r][1] = s_nan[r][2] = s_nan[r][3] = 0u;
        }
      }
      Kept kept;
      kept.begin(A, sg);
      int j = kept.next(sg.j0, sg.j1);
      fence_proxy_async_smem();
      softmax_sync();
      if (s_fail) break;
      if (j < sg.j1) mbar_arrive(bar(kQFull));
      float l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.f;
      bool first = true;
      for (; j < sg.j1; j = kept.next(j + 1, sg.j1), ++gt, first = false) {
        const int s = gt % kStages;
        const uint64_t heads = kept.heads(j);
        const bool got = waited(bar(kSFull + (gt & 1)), (gt >> 1) & 1) && waited(bar(kFull + s), (gt / kStages) & 1);
        tc_fence_after();
        uint32_t sv[R];
        if constexpr (R == 16) {
          tmem_ld16(tmem + C::kColS + (gt & 1) * R + lanes, sv);
          tmem_wait_ld_dep16(sv);
        } else {
          tmem_ld32(tmem + C::kColS + (gt & 1) * R + lanes, sv);
          tmem_wait_ld_dep(sv);
        }
        const int pos = j * 128 + tid, pg = tid >> A.page_shift;
        const float ks = s_ks[s][pg], vs = s_vs[s][pg];
        const bool there = pos < sg.limit && ks >= 0.f;
        const float lv = there ? fmaxf(__log2f(vs), (float)kMinScaleExp) : 0.f;
        const float inv_vs = there ? 1.0f / fmaxf(vs, exp2_int(kMinScaleExp)) : 0.f;
        // every row sees all 128 tokens?
        const bool full = (j + 1) * 128 <= sg.low && kept.all(heads);
        bool grow = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if ((r & 3) == 0 && r >= sg.live) break;
          float x = fmaf(__uint_as_float(sv[r]), ks * s_c[r], lv);
          if (!there || (!full && (pos >= s_see[r] || !((heads >> s_head[r]) & 1ull)))) x = -INFINITY;
          sv[r] = __float_as_uint(x);
          grow |= x > s_thr[r];
        }
        if (softmax_any(grow || !got)) {
          if (s_fail) {
            ok = false;
            break;
          }
          // some value exceeds its row's reference: move the references to the maxima so far
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if ((r & 3) == 0 && r >= sg.live) break;
            const float mx = warp_max(__uint_as_float(sv[r]));
            if (lane == 0) s_wmax[warp][r] = mx;
          }
          softmax_sync();
          if (tid < sg.live) {
            const float m = s_thr[tid] - kGrow;
            const float mx = fmaxf(fmaxf(s_wmax[0][tid], s_wmax[1][tid]), fmaxf(s_wmax[2][tid], s_wmax[3][tid]));
            const bool up = mx > m + kGrow;
            s_alpha[tid] = up ? fast_exp2(m - mx) : 1.f;
            if (up) {
              s_thr[tid] = mx + kGrow;
              s_off[tid] = kPScale - mx;
            }
          }
          softmax_sync();
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if ((r & 3) == 0 && r >= sg.live) break;
            l[r] *= s_alpha[r];
          }
          if (!first) {
            waited(bar(kODone + ((gt - 1) & 1)), ((gt - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 3 * R; c += 16) {
              if ((c & (R - 1)) >= sg.live) continue;
              uint32_t v[16];
              tmem_ld16(tmem + C::kColO + c + lanes, v);
              tmem_wait_ld_dep16(v);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((c & (R - 1)) + e < sg.live)
                  v[e] = __float_as_uint(__uint_as_float(v[e]) * s_alpha[(c & (R - 1)) + e]);
              tmem_st16(tmem + C::kColO + c + lanes, v);
            }
            tmem_wait_st();
          }
        }
        // places without a token hold anything: their V must not meet a P of 0.
        // A NaN in V is kept from the rows that do not see its token.
        if (!full || (j + 1) * 128 > sg.limit || __any_sync(0xffffffffu, !there)) {
          unsigned char* vrow = sgen + s * 2 * kStepBytes + kStepBytes + tid * 128;
          uint32_t nan[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
          for (int x = 0; x < 8; ++x) {
            const int c = (x + lane) & 7;  // (all banks)
            uint4* cell = reinterpret_cast<uint4*>(vrow + (((c ^ (tid & 7)) << 4)));
            if (!there) {
              *cell = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            uint4 v = *cell;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
            bool found = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t hit = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (hit) {
                found = true;
                for (int b = 0; b < 4; ++b)
                  if (hit >> (8 * b + 7) & 1u) {
                    nan[c >> 1] |= 1u << ((c & 1) * 16 + e * 4 + b);
                    w[e] &= ~(0xffu << (8 * b));
                  }
              }
            }
            if (found) *cell = v;
          }
          if (nan[0] | nan[1] | nan[2] | nan[3]) {
            s_any_nan = 1;
            for (int r = 0; r < sg.live; ++r)
              if (pos < s_see[r] && ((heads >> s_head[r]) & 1ull))
                for (int e = 0; e < 4; ++e) atomicOr(&s_nan[r][e], nan[e]);
          }
        }
        // P of this step overwrites the last one's
        if (!first) waited(bar(kODone + ((gt - 1) & 1)), ((gt - 1) >> 1) & 1);
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          if ((r & 3) == 0 && r >= sg.live) break;
          const float a = fast_exp2(__uint_as_float(sv[r]) + s_off[r]);
          const float b = fast_exp2(__uint_as_float(sv[r + 1]) + s_off[r + 1]);
          l[r] = fmaf(a, inv_vs, l[r]);
          l[r + 1] = fmaf(b, inv_vs, l[r + 1]);
          const uint32_t p0 = to_e4m3x2(a, b);
          const float2 b0 = from_e4m3x2(p0);
          const float a1 = (a - b0.x) * 16.f, c1 = (b - b0.y) * 16.f;
          const uint32_t p1 = to_e4m3x2(a1, c1);
          const float2 b1 = from_e4m3x2(p1);
          const uint32_t p2 = to_e4m3x2((a1 - b1.x) * 16.f, (c1 - b1.y) * 16.f);
          unsigned char* at = sgen + C::kOffP;
          at[sw128(r, tid)] = (unsigned char)p0;
          at[sw128(r + 1, tid)] = (unsigned char)(p0 >> 8);
          at[sw128(R + r, tid)] = (unsigned char)p1;
          at[sw128(R + r + 1, tid)] = (unsigned char)(p1 >> 8);
          at[sw128(2 * R + r, tid)] = (unsigned char)p2;
          at[sw128(2 * R + r + 1, tid)] = (unsigned char)(p2 >> 8);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kPFull));
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if ((r & 3) == 0 && r >= sg.live) break;
        const float t = warp_sum(l[r]);
        if (lane == 0) s_sum[warp][r] = t;
      }
      softmax_sync();
      const bool none = first;  // no kept step: O stays 0
      if (!none) {
        waited(bar(kODone + ((gt - 1) & 1)), ((gt - 1) >> 1) & 1);
        tc_fence_after();
      }
      const bool whole = sg.j0 == 0 && sg.j1 == sg.nt;
      const long long begin = sg.unit + sg.j0;
      float* slot = P.partial + C::kSlotFloats * (2 * (size_t)blockIdx.x + (begin == lo ? 0 : 1));
      const bool nans = s_any_nan != 0;
#pragma unroll 1
      for (int r0 = 0; r0 < sg.live; r0 += 16) {
        uint32_t v[3][16];
        if (!none) {
#pragma unroll
          for (int k = 0; k < 3; ++k) tmem_ld16(tmem + C::kColO + k * R + r0 + lanes, v[k]);
#pragma unroll
          for (int k = 0; k < 3; ++k) tmem_wait_ld_dep16(v[k]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = r0 + e;
          if (r >= sg.live) break;
          float o = 0.f;
          if (!none)
            o = fmaf(fmaf(__uint_as_float(v[2][e]), 0.0625f, __uint_as_float(v[1][e])), 0.0625f,
                     __uint_as_float(v[0][e]));
          if (nans && (s_nan[r][tid >> 5] >> lane & 1u)) o = NAN;
          const float sum = (s_sum[0][r] + s_sum[1][r]) + (s_sum[2][r] + s_sum[3][r]);
          if (whole) {
            const int row = sg.r.row0 + (sg.first + r) / g, head = sg.h * g + (sg.first + r) % g;
            // sum is 0 only where no token was seen; it is NaN where a score was
            A.o[((size_t)row * A.hq + head) * 128 + tid] = __float2bfloat16(sum == 0.f ? 0.f : o / sum);
          } else {
            __stcg(slot + r * 128 + tid, o);
            if (tid == 0) {
              __stcg(slot + R * 128 + r, s_thr[r] - kGrow);
              __stcg(slot + R * 129 + r, sum);
            }
          }
        }
      }
      if (!whole) {
        // count this part; the CTA that counts the last one adds them all
        const long long last = sg.unit + sg.nt - 1, total = s_share.total;
        const int c0 = (int)(((sg.unit + 1) * ctas - 1) / total), c1 = (int)(((last + 1) * ctas - 1) / total);
        __threadfence();
        softmax_sync();
        if (tid == 0) {
          asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zero
          const unsigned was = atomicAdd(P.counters + c0, 1u);
          s_last = was == (unsigned)(c1 - c0);
          __threadfence();
        }
        softmax_sync();
        if (s_last) {
          // warp = row, lane = 4 dims
          for (int r = warp; r < sg.live; r += 4) {
            auto slot_of = [&](int c) -> const float* {
              // slot 0 holds the segment with which a CTA begins, slot 1 the one with which it ends
              const long long b = total * c / ctas;
              return P.partial + C::kSlotFloats * (2 * (size_t)c + (b >= sg.unit ? 0 : 1));
            };
            float m = -INFINITY;
            for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, __ldcg(slot_of(c) + R * 128 + r));
            m = warp_max(m);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
              const float* p = slot_of(c);
              const float mc = __ldcg(p + R * 128 + r), lc = __ldcg(p + R * 129 + r);
              const float4 o = __ldcg(reinterpret_cast<const float4*>(p + r * 128) + lane);
              const float wt = mc == -INFINITY ? (lc == 0.f ? 0.f : 1.f) : fast_exp2(mc - m);
              acc.x = fmaf(o.x, wt, acc.x);
              acc.y = fmaf(o.y, wt, acc.y);
              acc.z = fmaf(o.z, wt, acc.z);
              acc.w = fmaf(o.w, wt, acc.w);
              sum = fmaf(lc, wt, sum);
            }
            const int row = sg.r.row0 + (sg.first + r) / g, head = sg.h * g + (sg.first + r) % g;
            const float f = sum == 0.f ? 0.f : 1.0f / sum;
            uint2 out;
            out.x = pack_bf16x2(acc.x * f, acc.y * f);
            out.y = pack_bf16x2(acc.z * f, acc.w * f);
            *reinterpret_cast<uint2*>(A.o + ((size_t)row * A.hq + head) * 128 + lane * 4) = out;
          }
        }
      }
      softmax_sync();  // s_sum, s_nan and the rows' arrays are free for the next unit
      if (tid == 0) s_any_nan = 0;
    }
    tc_fence_before();
    mbar_arrive(bar(kDone));
  }
}

}  // namespace cache
}  // namespace prism
