// Causal attention of many query rows a request (pieces of prompts) over a
// paged e4m3 cache.
//
// A work unit is 256 rows of one request and KV head, two tiles of 128; a step
// covers 128 tokens of its cache:
//   S [128 rows, 128 tokens] = (Q_0 + Q_1) K^T   e4m3, K as it lies in the cache
//   O [128 rows, 128 dims]  += P V               fp16, P from tensor memory
// Q / s = q_0 + q_1 holds bf16's 8 bits in two e4m3 terms (the few-row kernel's
// split), at twice fp16's rate: the same tensor time as one fp16 product, but K
// needs no conversion.  P needs 11 bits (2^-11 a value, one rounding), which
// four e4m3 terms would give for twice fp16's tensor time; V is converted
// instead, exactly (an e4m3 code is an fp16 number), by two warps at 64 codes a
// clock while the other warps compute: 256 of the 2048 clocks that a step's
// products take.  The scales of pages are powers of two and enter S and the
// exponent of P, where they are taken out of the row sum again.
//
// Rows are numbered head x tokens + token, so that the rows of a unit are one
// head's wherever a piece has 256 tokens: they share its block mask.
//
// A step's products take 2080 clocks, its shared memory traffic 2180 (192 KB of
// operands and 80 KB moved, at 128 B a clock), its exponentials 1800 (16 a
// clock; an eighth are polynomials).  Measured: 3900 clocks a step; two pieces
// of 1800-2048 tokens over 20-33K, 32 query / 8 KV heads, call after call: 1.80 to
// 1.85 ms, 960 to 935 TFLOP/s, 58 % of the measured bf16 rate (67 % of its rate in
// a long run, under the power cap).  A tile's softmax (about 2900 clocks beside
// the other tile's) and the round trip of its products (1000) follow one
// another, since S, P and O of two tiles fill tensor memory.
//
// 384 threads:
//   warp 0      producer: page lookups 32 at a time, TMA of K (3 stages) and V
//               (2 stages), the scales of each step's pages
//   warp 1      tensor cores: PV_A(t), QK_A(t+1), PV_B(t), QK_B(t+1), so one
//               tile's softmax runs beside the other's products
//   warps 2-3   V from e4m3 to fp16 (2 stages)
//   warps 4-11  softmax, thread = row; P is published in two parts
// The steps of all units are split evenly over the CTAs (one an SM) as in the
// few-row kernel.
#pragma once
#include <type_traits>

#include "cache_attention.cuh"

namespace prism {
namespace cache {
namespace tiles {

constexpr int kThreads = 384;
constexpr int kRows = 256;
constexpr int kUnitCost = 6;  // beginning and end of a unit, in steps
constexpr int kMaxCtas = 160;  // (B200: 148 SMs)
constexpr uint32_t kRegsLow = 72, kRegsHigh = 216;
constexpr int kMinLaunchRegs = (128 * kRegsLow + 256 * kRegsHigh + 383) / 384;
static_assert(kMinLaunchRegs <= 168, "register split exceeds what a 384-thread CTA can be given");
constexpr int kKStages = 3, kVStages = 2, kScales = 4;
constexpr uint32_t kCodeBytes = 128 * 128;           // K or V of a step
constexpr uint32_t kHalfBytes = 128 * 64 * 2;        // 64 dims of it in fp16
constexpr uint32_t kOffQ = 0;                        // tile A: two terms, tile B: two terms
constexpr uint32_t kOffK = kOffQ + 4 * kCodeBytes;
constexpr uint32_t kOffRaw = kOffK + kKStages * kCodeBytes;
constexpr uint32_t kOffV = kOffRaw + kVStages * kCodeBytes;
constexpr uint32_t kSmem = kOffV + 2 * 2 * kHalfBytes + 1024;  // + slack for 1024-byte alignment
constexpr uint32_t kTmemCols = 512;                  // S_A, S_B, O_A, O_B
constexpr float kGrow = 8.0f;      // the reference maximum moves when a value exceeds it by more (log2)
constexpr float kPScale = 7.0f;    // log2: P <= 2^(kGrow + kPScale) = 2^15 < 65504
// Beyond this maximum (log2) the reference is taken off the rounded score: the
// sum of a reference and an offset of 7, and one rounding of both with the score,
// are off by half a last place of the maximum, which P has no room for (2^24: 1).
constexpr float kFarMax = 1048576.0f;
constexpr int kPFirst = 6;         // P of keys [0, 16 kPFirst) is published first
constexpr int kByArithmetic = 1;   // of 8 pairs, whose exponentials are polynomials (at cooler clocks, 0: 1.73 ms, 1: 1.65, 2: 1.70, 3: 1.84)
constexpr size_t kSlotFloats = (size_t)kRows * 130;  // O [256][128], (m, l) [256]

enum : int {
  kKFull = 0,
  kKEmpty = kKFull + kKStages,
  kRawFull = kKEmpty + kKStages,
  kRawEmpty = kRawFull + kVStages,
  kVFull = kRawEmpty + kVStages,
  kVEmpty = kVFull + 2,
  kSFull = kVEmpty + 2,
  kPHalf = kSFull + 2,
  kPFull = kPHalf + 2,
  kODone = kPFull + 2,
  kQFull = kODone + 2,
  kDone = kQFull + 1,
  kNumBars = kDone + 1
};

struct Params {
  AttnParams A;
  float* partial;      // [2 * CTAs] slots
  unsigned* counters;  // [CTAs], zero
};

// S = (Q_0 + Q_1) K^T: four steps of 32 dims, first then second term of Q.
__device__ __forceinline__ void mma_qk(uint32_t leader, uint32_t d_tmem, uint32_t q_lo, uint32_t k_lo, uint32_t hi) {
  constexpr uint32_t idesc = idesc_e4m3_f32(128, 128, 0, 0);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    mma_f8_ss_lead(leader, d_tmem, q_lo + (e >> 2) * (kCodeBytes / 16) + (e & 3) * 2, k_lo + (e & 3) * 2, hi, idesc, e > 0);
}
// O += P V of tokens [16 K0, 16 K1).
template <int K0, int K1>
__device__ __forceinline__ void mma_pv(uint32_t leader, uint32_t o_tmem, uint32_t p_tmem, uint32_t v_lo, uint32_t hi, bool more) {
  constexpr uint32_t idesc = idesc_f16_f32(128, 128, 0, 1);
#pragma unroll
  for (int e = K0; e < K1; ++e)
    mma_f16_ts_lead(leader, o_tmem, p_tmem + e * 8, v_lo + e * (2048 / 16), hi, idesc, more || e > 0 ? 1u : 0u);
}

__device__ constexpr float kExp2[6] = {1.000000119e+00f, 6.931471825e-01f, 2.402210683e-01f, 5.550356954e-02f, 9.676031768e-03f, 1.339086331e-03f};
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// 2^x of a pair by arithmetic: the special function unit's 16 a clock are as much
// in demand as the tensor cores.  x = n + f, n the nearest integer (read off the
// low bits of x + 1.5 2^23), 2^f on [-1/2, 1/2] by the polynomial that meets it
// at the Chebyshev points (relative error 2^-22), times 2^n put together from
// its exponent.  Below 2^-126 it stays there: nothing, in fp16, and in a row sum
// too, beside a token that the row sees: its largest P is 2^kPScale or more, and
// V's scales lie within 2^80 of each other.  A row that sees none has only such
// rests: it is told by its maximum.  NaN stays NaN.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x2) {
  float x0, x1, t0, t1;
  f2_unpack(x2, x0, x1);
  x2 = f2_pack(max_nan(x0, -126.f), max_nan(x1, -126.f));
  const uint64_t big = f2_pack(12582912.f, 12582912.f), t2 = f2_add(x2, big);
  const uint64_t n2 = f2_add(t2, f2_pack(-12582912.f, -12582912.f));
  const uint64_t f2 = f2_fma(n2, f2_pack(-1.f, -1.f), x2);
  auto both = [](float c) { return f2_pack(c, c); };
  uint64_t p = f2_fma(f2, both(kExp2[5]), both(kExp2[4]));
  p = f2_fma(f2, p, both(kExp2[3]));
  p = f2_fma(f2, p, both(kExp2[2]));
  p = f2_fma(f2, p, both(kExp2[1]));
  p = f2_fma(f2, p, both(kExp2[0]));
  f2_unpack(t2, t0, t1);
  return f2_mul(p, f2_pack(__uint_as_float((__float_as_uint(t0) << 23) + 0x3f800000u),
                           __uint_as_float((__float_as_uint(t1) << 23) + 0x3f800000u)));
}

// P = 2^(a S + off) of the 16 tokens of group gi, two fp16 a word, and their
// weight in the row sum.
__device__ __forceinline__ void p_group(const uint32_t (&sv)[128], int gi, float a, float off, float inv,
                                        uint64_t (&acc)[4], uint32_t* pk) {
  const uint64_t a2 = f2_pack(a, a), o2 = f2_pack(off, off), i2 = f2_pack(inv, inv);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = gi * 16 + 2 * e;
    const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), a2, o2);
    float p0, p1;
    uint64_t p2;
    if (e % 8 < kByArithmetic) {
      p2 = exp2_pair(x2);
      f2_unpack(p2, p0, p1);
    } else {
      f2_unpack(x2, p0, p1);
      p0 = fast_exp2(p0);
      p1 = fast_exp2(p1);
      p2 = f2_pack(p0, p1);
    }
    acc[e & 3] = f2_fma(p2, i2, acc[e & 3]);
    pk[e] = pack_f16x2(p0, p1);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
attn_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params P) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bars[kNumBars];
  __shared__ Step s_sc[kScales];
  __shared__ float s_c[kRows];
  __shared__ int s_see[kRows], s_head[kRows];
  __shared__ float s_sum[2][kRows];
  __shared__ __align__(16) uint32_t s_nan[kRows][4];  // dims of a row that saw a NaN in V
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ Share s_share;
  __shared__ Walk<kRows, true, kUnitCost> s_walk[5];
  __shared__ Segment s_seg[5];
  __shared__ int s_more, s_steps;

  const AttnParams& A = P.A;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sgen = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int x) { return smem_u32(&s_bars[x]); };

  if (few_rows_will_do<kThreads>(A, A.least - 1, &s_share)) {  // nothing here
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (complete only when what it was launched beside is)
    return;
  }
  if (tid == 0) {
    for (int x = 0; x < kNumBars; ++x) {
      const bool conv = (x >= kRawEmpty && x < kRawEmpty + kVStages) || x == kVFull || x == kVFull + 1;
      const bool rows = x >= kPHalf && x < kODone;
      mbar_init(bar(x), conv ? 64 : rows ? 128 : x == kQFull || x == kDone ? 256 : 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    tmem_relinquish();
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  Walk<kRows, true, kUnitCost> walk;
  walk.init(A);
  long long lo, hi, ctas;
  find_share<kThreads>(A, walk, &s_share, lo, hi, ctas);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const long long total = s_share.total;
  // Each role walks the segments by itself (one thread of it, in shared memory:
  // the roles' registers are for their tiles).
  if (tid < 5) {
    walk.begin(A, lo, hi, s_share.req, s_share.base);
    s_walk[tid] = walk;
  }
  __syncthreads();
  const int role = min(warp, 4);
  const Segment& sg = s_seg[role];
  auto next_segment = [&]() -> bool {  // of a warp's role
    __syncwarp();
    bool more = false;
    if (lane == 0) more = s_walk[role].next(A, s_seg[role]);
    return __any_sync(0xffffffffu, more);
  };
  auto nothing_kept = [&]() -> bool {
    Kept kept;
    kept.begin(A, sg);
    return kept.next(sg.j0, sg.j1) >= sg.j1;
  };
  int gt = 0;  // steps done by this role

  // Each warpgroup sets its register budget first and then runs its own roles.
  if (warp < 4) {
    regs_dec<kRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      const int npg = 128 >> A.page_shift;  // pages a step
      const uint32_t pbytes = 128u << A.page_shift;
      bool ok = true;
      while (ok && next_segment()) {
        const int32_t* entries = A.table + (size_t)sg.i * A.max_pages;
        const int pages = (sg.limit + (1 << A.page_shift) - 1) >> A.page_shift;  // of the unit
        PageWindow cur, nxt;
        Kept kept;
        kept.begin(A, sg);
        int j = kept.next(sg.j0, sg.j1);
        int w = j * npg >> 5;
        if (j < sg.j1) {
          cur.load(A, entries, pages, w, sg.h);
          nxt.load(A, entries, pages, w + 1, sg.h);
        }
        for (int jn; j < sg.j1; j = jn) {
          const uint64_t heads = kept.heads(j);
          const bool all_heads = kept.all(heads);
          jn = kept.next(j + 1, sg.j1);
          const int p0 = j * npg;
          if (p0 >> 5 != w) {
            if (p0 >> 5 == w + 1) cur = nxt;
            else cur.load(A, entries, pages, p0 >> 5, sg.h);
            w = p0 >> 5;
            nxt.load(A, entries, pages, w + 1, sg.h);
          }
          const int s = gt % kKStages, v = gt & 1, x = lane - (p0 & 31);  // this lane's page of the step
          const bool mine = x >= 0 && x < npg, there = mine && cur.pg >= 0;
          if (mine && cur.pg == PageWindow::kNoPage) set_device_error(kDevErrCache);
          const uint32_t n = __popc(__ballot_sync(0xffffffffu, there));
          // K's stage is free once both tiles' S of step gt - 3 are done, which
          // is after the softmax of step gt - 4: its scales' place is free too
          if (gt >= kKStages &&
              !(ok = __all_sync(0xffffffffu, mbar_wait(bar(kKEmpty + s), (gt / kKStages - 1) & 1))))
            break;
          Step& sc = s_sc[gt & (kScales - 1)];
          if (mine) sc.set_page(x, npg, cur);
          if (lane < 4) sc.nan[lane] = 0u;
          if (lane == 0) {
            sc.heads = heads;
            sc.j = j;
            sc.last = jn >= sg.j1;
            sc.full = n == (uint32_t)npg && (j + 1) * 128 <= sg.low && all_heads;
          }
          __syncwarp();  // the step is described before K or V of it can be there
          if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + s), n * pbytes);
          __syncwarp();
          const uint32_t at = x * pbytes;
          if (there) tma_load_4d(sbase + kOffK + s * kCodeBytes + at, &tmK, 0, 0, sg.h, cur.pg, bar(kKFull + s));
          if (gt >= kVStages &&
              !(ok = __all_sync(0xffffffffu, mbar_wait(bar(kRawEmpty + v), (gt / kVStages - 1) & 1)))) {
            ++gt;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kRawFull + v), n * pbytes);
          __syncwarp();
          if (there) tma_load_4d(sbase + kOffRaw + v * kCodeBytes + at, &tmV, 0, 0, sg.h, cur.pg, bar(kRawFull + v));
          ++gt;
        }
      }
      if (!ok) {  // given up: the copies in flight land before the CTA leaves
        for (int x = max(gt - kKStages, 0); x < gt; ++x) mbar_wait(bar(kKFull + x % kKStages), (x / kKStages) & 1);
        for (int x = max(gt - kVStages - 1, 0); x < gt - 1; ++x)
          mbar_wait(bar(kRawFull + x % kVStages), (x / kVStages) & 1);
      }
      // the counters' clearing, and what came before it, are complete when this kernel is
      asm volatile("griddepcontrol.wait;" ::: "memory");
    } else if (warp == 1) {
      // ---------------------------------------------------------- tensor cores
      // the whole warp takes the role, one lane of it issues: descriptors stay in
      // uniform registers
      const uint32_t leader = elect_one();
      const uint64_t dQ = smem_desc_sw128(sbase + kOffQ, 16, 1024);
      const uint32_t hi = (uint32_t)(dQ >> 32), q_lo = (uint32_t)dQ, k_lo = q_lo + (kOffK - kOffQ) / 16;
      const uint32_t v_lo = (uint32_t)smem_desc_sw128(sbase + kOffV, kHalfBytes, 1024);
      bool ok = true;
      auto wait = [&](int b, int parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1));
        tc_fence_after();
        return ok;
      };
      auto next_stage = [](int s) { return s + 1 == kKStages ? 0 : s + 1; };
      int seg = 0, u[2] = {0, 0}, ks = 0, kphase = 0;  // K's stage and its phase
      while (ok && next_segment()) {
        if (nothing_kept()) continue;
        {
          const bool two = __any_sync(0xffffffffu, sg.live > 128);
          if (wait(kQFull, seg) && wait(kKFull + ks, kphase)) {
            mma_qk(leader, tmem, q_lo, k_lo + ks * (kCodeBytes / 16), hi);
            mma_commit_lead(leader, bar(kSFull));
            if (two) {
              mma_qk(leader, tmem + 128, q_lo + 2 * (kCodeBytes / 16), k_lo + ks * (kCodeBytes / 16), hi);
              mma_commit_lead(leader, bar(kSFull + 1));
            }
            mma_commit_lead(leader, bar(kKEmpty + ks));
          }
          for (bool first = true, more = true; ok && more; first = false) {
            if (!wait(kVFull + (gt & 1), gt >> 1)) break;
            more = !__any_sync(0xffffffffu, s_sc[gt & (kScales - 1)].last);
            const uint32_t v = v_lo + (gt & 1) * (2 * kHalfBytes / 16);
            ks = next_stage(ks);
            if (ks == 0) kphase ^= 1;
            if (!wait(kPHalf, u[0])) break;
            mma_pv<0, kPFirst>(leader, tmem + 256, tmem, v, hi, !first);
            if (!wait(kPFull, u[0])) break;
            mma_pv<kPFirst, 8>(leader, tmem + 256, tmem, v, hi, true);
            ++u[0];
            if (more) {
              if (!wait(kKFull + ks, kphase)) break;
              mma_qk(leader, tmem, q_lo, k_lo + ks * (kCodeBytes / 16), hi);
              mma_commit_lead(leader, bar(kSFull));
            } else {
              mma_commit_lead(leader, bar(kODone));
            }
            if (two) {
              if (!wait(kPHalf + 1, u[1])) break;
              mma_pv<0, kPFirst>(leader, tmem + 384, tmem + 128, v, hi, !first);
              if (!wait(kPFull + 1, u[1])) break;
              mma_pv<kPFirst, 8>(leader, tmem + 384, tmem + 128, v, hi, true);
              ++u[1];
              if (more) {
                mma_qk(leader, tmem + 128, q_lo + 2 * (kCodeBytes / 16), k_lo + ks * (kCodeBytes / 16), hi);
                mma_commit_lead(leader, bar(kSFull + 1));
              } else {
                mma_commit_lead(leader, bar(kODone + 1));
              }
            }
            mma_commit_lead(leader, bar(kVEmpty + (gt & 1)));
            if (more) mma_commit_lead(leader, bar(kKEmpty + ks));
            ++gt;
          }
        }
        ++seg;
      }
      __syncwarp();
      mbar_wait(bar(kDone), 0);
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    } else {
      // ---------------------------------------------------------- V to fp16
      bool ok = true;
      const int cw = warp - 2, c = lane & 7, flip = c >> 2;  // warp, 16 dims of a token, 64-dim half
      auto wait = [&](int b, int parity) {
        return ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1));
      };
      while (ok && next_segment()) {
        if (nothing_kept()) continue;
        for (bool last = false; !last; ++gt) {
          const int v = gt & 1;
          Step& sc = s_sc[gt & (kScales - 1)];
          if (!wait(kRawFull + v, gt >> 1) || (gt >= 2 && !wait(kVEmpty + v, (gt >> 1) - 1))) break;
          last = sc.last;
          const unsigned char* src = sgen + kOffRaw + v * kCodeBytes;
          unsigned char* dst = sgen + kOffV + v * 2 * kHalfBytes + flip * kHalfBytes;
          const bool plain = sc.full;
          const int limit = sg.limit - sc.j * 128;
#pragma unroll 4
          for (int it = 0; it < 16; ++it) {
            const int row = (2 * it + cw) * 4 + (lane >> 3);
            uint4 w = *reinterpret_cast<const uint4*>(src + row * 128 + ((c ^ (row & 7)) << 4));
            if (!plain) {
              // places without a token hold anything, and a NaN must reach only
              // the rows that see its token: neither meets a P of 0
              const bool there = row < limit && sc.group[row >> 4].w != 0.f;
              uint32_t* e = reinterpret_cast<uint32_t*>(&w);
              bool found = false;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (!there) e[k] = 0u;
                const uint32_t hit = ((e[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                found |= hit != 0u;
                e[k] &= ~((hit >> 7) * 0xffu);
              }
              if (found) atomicOr(&sc.nan[row >> 5], 1u << (row & 31));
            }
            uint32_t h[8];
            const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[2 * k] = f16x2_from_e4m3x2(e[k] & 0xffffu);
              h[2 * k + 1] = f16x2_from_e4m3x2(e[k] >> 16);
            }
            // the two 16-byte pieces in the order that gives a row's eight lanes
            // all banks
            unsigned char* at = dst + row * 128;
            const int p0 = 2 * (c & 3) + flip, p1 = p0 ^ 1;
            const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
            *reinterpret_cast<uint4*>(at + ((p0 ^ (row & 7)) << 4)) = flip ? b : a;
            *reinterpret_cast<uint4*>(at + ((p1 ^ (row & 7)) << 4)) = flip ? a : b;
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(kRawEmpty + v));
          mbar_arrive(bar(kVFull + v));
        }
      }
    }
    return;
  }
  regs_inc<kRegsHigh>();
  // ------------------------------------------------------------ softmax
  const int x = (warp - 4) >> 2;    // tile
  const int r = tid - 128;          // row of the unit: tile x, tensor memory lane r % 128
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t tS = tmem + 128 * x + lanes, tO = tmem + 256 + 128 * x + lanes;
  bool ok = true;
  // A wait that is given up is recorded; what follows runs on without further
  // waits (its results are void), so that no warp is left at a barrier.
  const Walk<kRows, true, kUnitCost>& rows = s_walk[role];
  auto wait = [&](int b, int parity) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1));
    tc_fence_after();
  };
  int u = 0, segs = 0;  // steps and segments of this tile
  for (;;) {
    if (r == 0) s_more = s_walk[role].next(A, s_seg[role]);
    rows_sync();
    if (!s_more) break;
    // Q of the unit's rows in two terms: 8 threads a row, 16 dims each, 32 rows a
    // round, the next three rounds' loads in flight (a short loop: code that a
    // unit runs once is fetched once, at a memory's latency)
    {
      const int c = r & 7;
      int rr = r >> 3, head = rows.head_of(sg.r, sg.first + rr), token = sg.first + rr - head * sg.r.rows;
      struct Round {
        uint4 lo, hi;
      };
      auto load = [&](int row, int h, int t) {
        Round v = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (row < sg.live) {
          const __nv_bfloat16* src =
              A.q + (long long)(sg.r.row0 + t) * A.q_tok + (long long)(sg.h * rows.g + h) * A.q_head + c * 16;
          v.lo = ldg_nc_v4(src);
          v.hi = ldg_nc_v4(src + 8);
        }
        return v;
      };
      // 32 rows on: a division only where heads are shorter than that
      auto advance = [&](int& h, int& t) {
        t += 32;
        if (t >= sg.r.rows) {
          const int more = t < 2 * sg.r.rows ? 1 : t / sg.r.rows;
          h += more;
          t -= more * sg.r.rows;
        }
      };
      int ahead_h = head, ahead_t = token;
      Round v0 = load(rr, ahead_h, ahead_t);
      advance(ahead_h, ahead_t);
      Round v1 = load(rr + 32, ahead_h, ahead_t);
      advance(ahead_h, ahead_t);
      Round v2 = load(rr + 64, ahead_h, ahead_t);
      const int end = sg.live > 128 ? 256 : 128;
#pragma unroll 1
      for (; rr < end; rr += 32) {
        advance(ahead_h, ahead_t);
        const Round v3 = load(rr + 96, ahead_h, ahead_t);
        __syncwarp();
        const uint32_t w[8] = {v0.lo.x, v0.lo.y, v0.lo.z, v0.lo.w, v0.hi.x, v0.hi.y, v0.hi.z, v0.hi.w};
        float f[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[2 * e] = bf16lo(w[e]);
          f[2 * e + 1] = bf16hi(w[e]);
        }
        uint32_t w0[4], w1[4];
        const int ex = split_q(f, w0, w1);
        unsigned char* q0 = sgen + kOffQ + (rr >> 7) * 2 * kCodeBytes + sw128(rr & 127, 16 * c);
        *reinterpret_cast<uint4*>(q0) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        *reinterpret_cast<uint4*>(q0 + kCodeBytes) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        if (c == 0) {
          s_c[rr] = exp2_int(ex) * A.scale_log2;
          s_see[rr] = rr < sg.live ? rows.seen_by(sg.r, token) : 0;
          s_head[rr] = rr < sg.live ? head : 0;
        }
        advance(head, token);
        v0 = v1;
        v1 = v2;
        v2 = v3;
      }
    }
    *reinterpret_cast<uint4*>(s_nan[r]) = make_uint4(0u, 0u, 0u, 0u);
    const bool none = nothing_kept();  // O stays 0
    fence_proxy_async_smem();
    tc_fence_before();
    rows_sync();
    if (!none) mbar_arrive(bar(kQFull));
    const bool tile_live = x * 128 < sg.live;
    const float c = s_c[r];
    float m = -INFINITY, l = 0.f;
    bool first = true, far = false;
    for (bool last = none || !tile_live; !last; ++gt) {
      const Step& sc = s_sc[gt & (kScales - 1)];
      // S is there, and PV of the last step, issued before it, is done
      wait(kSFull + x, u);
      last = sc.last || !ok;
      uint32_t sv[128];
#pragma unroll
      for (int e = 0; e < 4; ++e) tmem_ld32(tS + 32 * e, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * e));
#pragma unroll
      for (int e = 0; e < 4; ++e) tmem_wait_ld_dep(*reinterpret_cast<uint32_t(*)[32]>(sv + 32 * e));
      if (__builtin_expect(!sc.full, 0)) {
        const int bound = (sc.heads >> s_head[r]) & 1ull ? s_see[r] - sc.j * 128 : 0;
#pragma unroll
        for (int gi = 0; gi < 8; ++gi) {
          const int n = sc.group[gi].w != 0.f ? bound - 16 * gi : 0;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (e >= n) sv[16 * gi + e] = __float_as_uint(-INFINITY);
        }
        // a NaN among the values of a token that this row sees
        wait(kVFull + (gt & 1), gt >> 1);
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          uint32_t bits = sc.nan[w];
#pragma unroll 1
          while (bits) {
            const int tok = 32 * w + __ffs(bits) - 1;
            bits &= bits - 1u;
            if (tok >= bound) continue;
            const int pos = sc.j * 128 + tok;
            const int pg = __ldg(A.table + (size_t)sg.i * A.max_pages + (pos >> A.page_shift));
            const uint8_t* v = A.vc + (size_t)pg * (size_t)A.page_stride +
                               (((size_t)sg.h << A.page_shift) + (pos & ((1 << A.page_shift) - 1))) * 128;
#pragma unroll 1
            for (int e = 0; e < 128; ++e)
              if ((__ldg(v + e) & 0x7f) == 0x7f) s_nan[r][e >> 5] |= 1u << (e & 31);
          }
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int gi = 0; gi < 8; ++gi) {
        float t0 = __uint_as_float(sv[16 * gi]), t1 = __uint_as_float(sv[16 * gi + 1]);
#pragma unroll
        for (int e = 2; e < 14; e += 4) {
          t0 = max3f(t0, __uint_as_float(sv[16 * gi + e]), __uint_as_float(sv[16 * gi + e + 1]));
          t1 = max3f(t1, __uint_as_float(sv[16 * gi + e + 2]), __uint_as_float(sv[16 * gi + e + 3]));
        }
        t0 = max3f(t0, __uint_as_float(sv[16 * gi + 14]), __uint_as_float(sv[16 * gi + 15]));
        const float2 f = *reinterpret_cast<const float2*>(&sc.group[gi]);
        mx = fmaxf(mx, fmaf(fmaxf(t0, t1), score_scale(f.x, c), f.y));
      }
      // the reference maximum moves only when it is exceeded by 2^kGrow
      const bool grow = mx - m > kGrow;
      const float m_new = grow ? mx : m;
      if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
        far = __any_sync(0xffffffffu, m_new != -INFINITY && fabsf(m_new) > kFarMax);
        if (!first) {
          const float alpha = grow ? fast_exp2(m - m_new) : 1.0f;
#pragma unroll 1
          for (int e = 0; e < 8; ++e) {
            uint32_t v[16];
            tmem_ld16(tO + e * 16, v);
            tmem_wait_ld_dep16(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
            tmem_st16(tO + e * 16, v);
          }
          l *= alpha;
        }
      }
      m = m_new;
      const float ref = m == -INFINITY ? 0.f : m;
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
      static_assert(kPFirst == 6, "the store shapes below assume 96 + 32 tokens");
      const float base = kPScale - ref;
      if (__builtin_expect(far, 0)) {
        // S becomes score - reference (0 and exact for the maximum), which the
        // groups below take by a factor of 1 and an offset of kPScale alone
#pragma unroll
        for (int gi = 0; gi < 8; ++gi) {
          const float2 f = *reinterpret_cast<const float2*>(&sc.group[gi]);
          const float a = score_scale(f.x, c);
#pragma unroll
          for (int e = 16 * gi; e < 16 * gi + 16; ++e)
            sv[e] = __float_as_uint(fmaf(__uint_as_float(sv[e]), a, f.y) - ref);
        }
      }
      auto publish = [&](auto far_c) {
        constexpr bool kFar = decltype(far_c)::value;
        float4 next = lds_v4(&sc.group[0]);
        auto group = [&](int gi, uint32_t* pk) {
          const float4 f = next;
          if (gi < 7) next = lds_v4(&sc.group[gi + 1]);
          p_group(sv, gi, kFar ? 1.f : score_scale(f.x, c), kFar ? kPScale : f.y + base, f.z, acc, pk);
        };
        {
          uint32_t pk[48];
#pragma unroll
          for (int gi = 0; gi < 6; ++gi) group(gi, pk + 8 * gi);
          tmem_st32(tS, *reinterpret_cast<const uint32_t(*)[32]>(pk));
          tmem_st16(tS + 32, *reinterpret_cast<const uint32_t(*)[16]>(pk + 32));
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kPHalf + x));
        }
        {
          uint32_t pk[16];
          group(6, pk);
          group(7, pk + 8);
          tmem_st16(tS + 48, pk);
        }
      };
      if (__builtin_expect(far, 0)) publish(std::true_type());
      else publish(std::false_type());
      float a0, a1;
      f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
      l += a0 + a1;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(kPFull + x));
      ++u;
      first = false;
    }
    // ---------------------------------------------------------- epilogue
    const bool whole = sg.j0 == 0 && sg.j1 == sg.nt;
    float* slot = P.partial + kSlotFloats * (2 * (size_t)blockIdx.x + (lo >= sg.unit ? 0 : 1));
    const bool live = r < sg.live;
    auto out_row = [&](int row) {
      return A.o + ((size_t)(sg.r.row0 + rows.token_of(sg.r, sg.first + row)) * A.hq + sg.h * rows.g +
                    rows.head_of(sg.r, sg.first + row)) * 128;
    };
    if (tile_live) {
      if (!first) wait(kODone + x, segs++);
      // no maximum: nothing was seen (l holds what masked scores leave), or NaN
      // scores alone (l is NaN)
      const float f = !whole ? 1.f : m == -INFINITY && l == l ? 0.f : 1.0f / l;
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        uint32_t v[32];
        if (!first) {
          tmem_ld32(tO + e * 32, v);
          tmem_wait_ld_dep(v);
        }
        const uint32_t nan = s_nan[r][e];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float y = first ? 0.f : __uint_as_float(v[k]) * f;
          if (nan >> k & 1u) y = NAN;
          v[k] = __float_as_uint(y);
        }
        if (live && whole) {
          uint4* dst = reinterpret_cast<uint4*>(out_row(r)) + e * 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            auto two = [&](int n) { return pack_bf16x2(__uint_as_float(v[8 * k + n]), __uint_as_float(v[8 * k + n + 1])); };
            dst[k] = make_uint4(two(0), two(2), two(4), two(6));
          }
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(slot + r * 128 + e * 32);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            __stcg(dst + k, make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                        __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3])));
        }
      }
      if (live && !whole) __stcg(reinterpret_cast<float2*>(slot + kRows * 128) + r, make_float2(m, l));
    }
    tc_fence_before();
    if (!whole) {
      // count this part; the CTA that counts the last one adds them all, in order
      const long long last = sg.step0 + sg.nt - 1;
      const int c0 = (int)(((sg.step0 + 1) * ctas - 1) / total), c1 = (int)(((last + 1) * ctas - 1) / total);
      rows_sync();
      if (r == 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zero
        s_last = count_acq_rel(P.counters + c0) == (unsigned)(c1 - c0);
      }
      rows_sync();
      if (s_last) {
        const int slot0 = total * c0 / ctas >= sg.unit ? 0 : 1;
        auto slot_of = [&](int k) -> const float* {
          // slot 0 holds the segment with which a CTA begins, slot 1 the one with which it ends
          return P.partial + kSlotFloats * (2 * (size_t)k + (k == c0 ? slot0 : 0));
        };
        // thread = row: its maximum and sum (a part without a maximum saw
        // nothing, or NaN scores alone)
        auto weight = [](float mk, float lk, float mm) {
          return mk == -INFINITY ? (lk == lk ? 0.f : 1.f) : fast_exp2(mk - mm);
        };
        float mm = -INFINITY, sum = 0.f;
#pragma unroll 4
        for (int k = c0; k <= c1; ++k) mm = fmaxf(mm, ldcg_v2(slot_of(k) + kRows * 128 + 2 * r).x);
#pragma unroll 4
        for (int k = c0; k <= c1; ++k) {
          const float2 ml = ldcg_v2(slot_of(k) + kRows * 128 + 2 * r);
          sum = fmaf(ml.y, weight(ml.x, ml.y, mm), sum);
        }
        s_sum[0][r] = mm;
        s_sum[1][r] = sum == 0.f ? 0.f : 1.0f / sum;
        rows_sync();
        // then warp = eight rows at a time, lane = 4 dims
#pragma unroll 1
        for (int row0 = (warp - 4) * 8; row0 < sg.live; row0 += 64) {
          float4 a[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) a[n] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int k0 = c0; k0 <= c1; k0 += 2) {
            float2 ml[2][8];
            float4 o[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float* p = slot_of(min(k0 + k, c1));
#pragma unroll
              for (int n = 0; n < 8; ++n) {  // (rows behind the unit's last are in the slot, and dropped below)
                ml[k][n] = ldcg_v2(p + kRows * 128 + 2 * (row0 + n));
                o[k][n] = ldcg_v4(p + (row0 + n) * 128 + 4 * lane);
              }
            }
            __syncwarp();  // (no load sinks to its use: they are all in flight here)
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float mm = s_sum[0][row0 + n];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if (k0 + k > c1) break;
                const float wt = weight(ml[k][n].x, ml[k][n].y, mm);
                a[n].x = fmaf(o[k][n].x, wt, a[n].x);
                a[n].y = fmaf(o[k][n].y, wt, a[n].y);
                a[n].z = fmaf(o[k][n].z, wt, a[n].z);
                a[n].w = fmaf(o[k][n].w, wt, a[n].w);
              }
            }
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int row = row0 + n;
            if (row >= sg.live) break;
            const float f = s_sum[1][row];
            *reinterpret_cast<uint2*>(out_row(row) + lane * 4) =
                make_uint2(pack_bf16x2(a[n].x * f, a[n].y * f), pack_bf16x2(a[n].z * f, a[n].w * f));
          }
        }
      }
    }
    if (r == 0) s_steps = gt;
    rows_sync();  // the rows' arrays are free for the next unit
    gt = s_steps;  // (the warps of a tile without rows took no step)
  }
  tc_fence_before();
  mbar_arrive(bar(kDone));
}

}  // namespace tiles
}  // namespace cache
}  // namespace prism
