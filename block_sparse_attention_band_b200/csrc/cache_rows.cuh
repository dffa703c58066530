// Causal attention of few query rows a request (single tokens, drafts) over a
// paged e4m3 cache: tokens as the tensor cores' M.
//
// A work unit is up to R rows (row = token x head of the group) of one request
// and KV head; a step covers 128 tokens of its cache:
//   S^T [128 tokens, R]  = K Q^T          A = K (e4m3 as stored), B = Q
//   O^T [128 dims, 4 R] += V^T [P_0 .. P_3]    A = V (as stored, read dim-major)
// so K and V go from HBM to the tensor cores as they lie in the cache, by TMA
// and without a conversion, and the softmax threads (thread = token) only
// touch the rows that exist.
//
// What 8-bit operands cost in precision is bought back by more terms:
//   Q / s = q_0 + q_1, e4m3 each, s the row's power of two with max|Q| / s in
//     (224, 448]: 4 + 4 bits hold a bf16 value's 8 exactly, down to 2^-10 s;
//     both products add into the same S.
//   P = 2^-4 (p_0 + 2^-5 p_1 + 2^-10 p_2 + 2^-15 p_3) of a P rounded to fp16
//     (2^-11 a value): a term of at most 2^8 leaves at most half a step of 2^4,
//     2^3, so 32 times the rest is at most 2^8 again, and the last term's
//     smallest step, 2^-9 2^-15, is fp16's: the four hold every fp16 P exactly,
//     its smallest step 2^-28 of the largest P.  (Three end at 2^-23: a token
//     that takes all but 0.002 of the weight took the rest, spread over 32K
//     tokens, with it.)
//   The terms are separate columns of one product, added at the end.
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
// 256 threads: warps 0-3 softmax, warp 4 producer (page lookups 32 at a time,
// TMA), warp 5 tensor cores, warps 6-7 clean V where some row does not see some
// token, beside the softmax, which they would hold up.  A token's P of 16 rows
// is one 16-byte store a term (B of the second product is read row-major, its
// rows' bytes side by side); the loop over the rows is compiled for the rows a
// unit has.  (20 of 32 drafts of 5 tokens: 80 us, 88 by the loop for 24.  Loops
// for 12 and 28 as well cost 4 % at 36 to 64 rows: code is fetched as it is run.)
//
// Measured (32 query / 8 KV heads, copy rate 6.54 TB/s, calls in one graph; call
// by call 1 to 3 % more): six single tokens over 60-131K tokens 174 us, 6.5 TB/s;
// 64 over 1-16K 160 us, 6.3 TB/s; one over 131K 55 us, of which 40 are the read
// and the rest the way in and out; one over 777 13.3 us, all latency (launches,
// lengths, table, first K, the count and the sum of the parts); 32 x 5 drafted
// tokens over 0.1-8K 80 us (23 steps a unit cannot hide its beginning and end);
// eight over 30-131K under an 18 % mask 52 us.
#pragma once
#include "cache_attention.cuh"

namespace prism {
namespace cache {
namespace rows {

constexpr int kThreads = 256;
// register split: the softmax warpgroup takes what the other roles leave
constexpr uint32_t kRegsLow = 64, kRegsHigh = 192;
constexpr int kMinLaunchRegs = (kRegsLow + kRegsHigh) / 2;
constexpr uint32_t kStepBytes = 128 * 128;  // K or V of one step
constexpr int kMaxCtas = 512;
constexpr float kGrow = 4.0f;    // the reference maximum moves when a value exceeds it by more (log2)
constexpr float kPScale = 4.0f;  // log2: P <= 2^(kGrow + kPScale)
static_assert(kGrow + kPScale == 8.0f, "the first term's largest value is 256 (e4m3: 448)");
constexpr float kNoMax = 1e30f;  // offset of a row that has seen nothing: every score exceeds its reference

template <int R>
struct Cfg {
  // beginning and end of a unit, in steps (measured, with three terms of P: 16 rows:
  // 64 mixed requests 159 us at 4, 161 at 12; 32 rows: 32 drafts 86 us at 4, 80 at
  // 9, 81 at 12)
  static constexpr int kUnitCost = R <= 16 ? 5 : kFewUnitCost;
  static_assert(R <= 16 || R == kFewUnitRows, "rows a unit");
  // K is free again once S is, a step before V: fewer stages keep as much in
  // flight (3 of K and 2 of V, or V copied by a producer of its own pace: no faster)
  static constexpr int kKStages = 2, kVStages = R <= 16 ? 3 : 2, kSteps = 4;
  static constexpr uint32_t kQBytes = 2 * R * 128;            // two terms
  static constexpr uint32_t kPPitch = 4 * R;                  // bytes of a token: four terms of R rows
  static constexpr uint32_t kPBytes = 128 * kPPitch;
  static constexpr uint32_t kOffV = kKStages * kStepBytes;
  static constexpr uint32_t kOffP = kOffV + kVStages * kStepBytes;  // two buffers
  static constexpr uint32_t kOffQ = kOffP + 2 * kPBytes;
  static constexpr uint32_t kSmem = kOffQ + kQBytes + 1024;   // + slack for 1024-byte alignment
  static constexpr uint32_t kColO = 2 * R;                    // after two S buffers
  static constexpr uint32_t kCols = R <= 16 ? 128 : 256;
  static_assert(6 * R <= (int)kCols, "tensor memory columns");
  static constexpr size_t kSlotFloats = (size_t)R * 130;      // O [R][128], (m, l) [R]
};

struct Params {
  AttnParams A;
  float* partial;       // [2 * CTAs] slots
  unsigned* counters;   // [CTAs], zero
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

// Byte offset of piece c (16 bytes) of token t in P's operand tile: 64-byte rows
// with 64-byte swizzle, or 128-byte rows with 128-byte swizzle.
template <int R>
__device__ __forceinline__ uint32_t p_piece(int t, int c) {
  return R <= 16 ? (uint32_t)(t * 64 + ((c ^ ((t >> 1) & 3)) << 4)) : (uint32_t)(t * 128 + ((c ^ (t & 7)) << 4));
}

// P of four rows of a token in its four terms, a byte a row.
__device__ __forceinline__ void split_p(float p0, float p1, float p2, float p3, uint32_t& w0, uint32_t& w1,
                                        uint32_t& w2, uint32_t& w3) {
  const __half2 f = __float2half2_rn(32.f);
  auto half2 = [](uint32_t x) { return *reinterpret_cast<__half2*>(&x); };
  auto bits = [](__half2 x) { return *reinterpret_cast<uint32_t*>(&x); };
  __half2 a = half2(pack_f16x2(p0, p1)), b = half2(pack_f16x2(p2, p3));
  uint32_t ta = e4m3x2_from_f16x2(bits(a)), tb = e4m3x2_from_f16x2(bits(b));
  w0 = __byte_perm(ta, tb, 0x5410);
  a = __hmul2(__hsub2(a, half2(f16x2_from_e4m3x2(ta))), f);  // (exact: the bits below the term's)
  b = __hmul2(__hsub2(b, half2(f16x2_from_e4m3x2(tb))), f);
  ta = e4m3x2_from_f16x2(bits(a));
  tb = e4m3x2_from_f16x2(bits(b));
  w1 = __byte_perm(ta, tb, 0x5410);
  a = __hmul2(__hsub2(a, half2(f16x2_from_e4m3x2(ta))), f);
  b = __hmul2(__hsub2(b, half2(f16x2_from_e4m3x2(tb))), f);
  ta = e4m3x2_from_f16x2(bits(a));
  tb = e4m3x2_from_f16x2(bits(b));
  w2 = __byte_perm(ta, tb, 0x5410);
  a = __hmul2(__hsub2(a, half2(f16x2_from_e4m3x2(ta))), f);
  b = __hmul2(__hsub2(b, half2(f16x2_from_e4m3x2(tb))), f);
  w3 = __byte_perm(e4m3x2_from_f16x2(bits(a)), e4m3x2_from_f16x2(bits(b)), 0x5410);
}

template <int R>
__global__ void __launch_bounds__(kThreads, 2)
attn_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params P) {
  using C = Cfg<R>;
  constexpr int kKStages = C::kKStages, kVStages = C::kVStages, kSteps = C::kSteps;
  constexpr int kKFull = 0, kKEmpty = kKFull + kKStages, kVFull = kKEmpty + kKStages, kVEmpty = kVFull + kVStages,
                kVClean = kVEmpty + kVStages, kSFull = kVClean + kVStages, kPFull = kSFull + 2, kODone = kPFull + 2, kQFull = kODone + 2,
                kDone = kQFull + 1;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bars[kDone + 1];
  __shared__ Step s_step[kSteps];
  __shared__ float4 s_row[R / 2];  // of two rows: factors of S, offsets (kPScale - reference)
  __shared__ __align__(16) float s_alpha[R], s_wmax[4][R], s_sum[4][R];
  __shared__ int s_see[R], s_head[R];
  __shared__ long long s_out[R];  // elements of O before a row
  __shared__ uint32_t s_nan[R][4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_any_nan, s_last, s_more;
  __shared__ volatile int s_fail;
  __shared__ Share s_share;
  __shared__ Walk<R, false, C::kUnitCost> s_walk[5];
  __shared__ Segment s_seg[5];

  const AttnParams& A = P.A;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sgen = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = A.hq / A.hkv;
  auto bar = [&](int x) { return smem_u32(&s_bars[x]); };
  // the tile kernel of the call may start on SMs that this one leaves
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (A.counts) asm volatile("griddepcontrol.wait;" ::: "memory");  // they are written
  if (tid == 0) {
    for (int x = 0; x <= kDone; ++x)
      mbar_init(bar(x), x >= kVClean && x < kSFull ? 64 : x == kPFull || x == kPFull + 1 || x == kQFull || x == kDone ? 128 : 1);
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
  Walk<R, false, C::kUnitCost> walk;
  walk.init(A);
  if (A.choose && few_rows_will_do<kThreads>(A, A.most, &s_share)) walk.most = 0x7fffffff;
  long long lo, hi, ctas;
  find_share<kThreads>(A, walk, &s_share, lo, hi, ctas);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // each role walks the segments by itself (one thread of it, in shared memory)
  const int role = max(warp - 3, 0);
  if (tid == 0 || (warp >= 4 && lane == 0)) {
    walk.begin(A, lo, hi, s_share.req, s_share.base);
    s_walk[role] = walk;
  }
  const Segment& sg = s_seg[role];
  auto next_segment = [&]() -> bool {  // of a warp's role
    __syncwarp();
    bool more = false;
    if (lane == 0) more = s_walk[role].next(A, s_seg[role]);
    return __any_sync(0xffffffffu, more);
  };
  auto nothing_kept = [&]() -> bool { return sg.none != 0; };
  int gt = 0;  // steps done by this role

  // Each warpgroup sets its register budget first and then runs its own roles.
  if (warp >= 4) {
  regs_dec<kRegsLow>();
  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int npg = 128 >> A.page_shift;  // pages a step
    const uint32_t pbytes = 128u << A.page_shift;
    bool ok = true, k_only = false;
    auto wait = [&](int b, int parity) {
      return ok = __all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1));
    };
    int kst = 0, vst = 0;
    while (ok && next_segment()) {
      const int32_t* entries = A.table + (size_t)sg.i * A.max_pages;
      const int pages = (sg.limit + (1 << A.page_shift) - 1) >> A.page_shift;  // of the unit
      PageWindow cur, nxt;
      Kept kept;
      kept.begin(A, sg);
      if (sg.none) continue;
      int j = kept.seek(sg.j0), left = sg.j1 - sg.j0;
      int w = j * npg >> 5;
      cur.load(A, entries, pages, w, sg.h);
      nxt.load(A, entries, pages, w + 1, sg.h);
      for (int jn; left > 0; j = jn) {
        const uint64_t heads = kept.heads(j);
        const bool all_heads = kept.all(heads);
        jn = --left > 0 ? kept.next(j + 1, A.words * 32) : j;
        const int p0 = j * npg;
        if (p0 >> 5 != w) {
          if (p0 >> 5 == w + 1) cur = nxt;
          else cur.load(A, entries, pages, p0 >> 5, sg.h);
          w = p0 >> 5;
          nxt.load(A, entries, pages, w + 1, sg.h);
        }
        const int x = lane - (p0 & 31);  // this lane's page of the step
        const bool mine = x >= 0 && x < npg, there = mine && cur.pg >= 0;
        if (mine && cur.pg == PageWindow::kNoPage) set_device_error(kDevErrCache);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, there)) * pbytes;
        // K's stage is free once S of step gt - 2 is done, which is after the
        // softmax of step gt - 4: the place of its description is free too
        if (gt >= kKStages && !wait(kKEmpty + kst, (gt / kKStages) - 1)) break;
        // the copies first (the barrier's phase ends with the arrival below), the
        // pages' scales may still be on their way
        if (there) tma_load_4d(sbase + kst * kStepBytes + x * pbytes, &tmK, 0, 0, sg.h, cur.pg, bar(kKFull + kst));
        const bool v_free = gt < kVStages || mbar_test_wait(bar(kVEmpty + vst), (gt / kVStages - 1) & 1);
        const bool early = __all_sync(0xffffffffu, v_free);
        auto load_v = [&]() {
          if (there)
            tma_load_4d(sbase + C::kOffV + vst * kStepBytes + x * pbytes, &tmV, 0, 0, sg.h, cur.pg, bar(kVFull + vst));
        };
        if (early) load_v();
        Step& st = s_step[gt & (kSteps - 1)];
        if (mine) st.set_page(x, npg, cur);
        if (lane == 0) {
          st.heads = heads;
          st.j = j;
          st.last = left == 0;
          st.there = bytes == kStepBytes && (j + 1) * 128 <= sg.limit;
          st.full = bytes == kStepBytes && (j + 1) * 128 <= sg.low && all_heads;
        }
        __syncwarp();  // the step is described before K or V of it can be there
        if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + kst), bytes);
        if (!early) {
          if (!wait(kVEmpty + vst, gt / kVStages - 1)) {
            k_only = true;
            break;
          }
          load_v();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(bar(kVFull + vst), bytes);
        ++gt;
        kst = kst + 1 == kKStages ? 0 : kst + 1;
        vst = vst + 1 == kVStages ? 0 : vst + 1;
      }
    }
    if (!ok) {  // given up: the copies in flight land before the CTA leaves
      const int nk = gt + (k_only ? 1 : 0);
      for (int x = max(nk - kKStages, 0); x < nk; ++x) mbar_wait(bar(kKFull + x % kKStages), (x / kKStages) & 1);
      for (int x = max(gt - kVStages, 0); x < gt; ++x) mbar_wait(bar(kVFull + x % kVStages), (x / kVStages) & 1);
    }
    // what this kernel was launched beside is complete when it is
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else if (warp == 5) {
    // ------------------------------------------------------------ tensor cores
    // the whole warp takes the role, one lane of it issues: descriptors stay in
    // uniform registers
    const uint32_t leader = elect_one();
    const uint64_t dK = smem_desc_sw128(sbase, 16, 1024);
    const uint64_t dP = R <= 16 ? smem_desc_sw64(sbase + C::kOffP, 16, 512) : smem_desc_sw128(sbase + C::kOffP, 16, 1024);
    const uint32_t hi_k = (uint32_t)(dK >> 32), hi_p = (uint32_t)(dP >> 32), k_lo = (uint32_t)dK,
                   q_lo = k_lo + C::kOffQ / 16, p_lo = (uint32_t)dP;
    const uint64_t dV = smem_desc_sw128(sbase + C::kOffV, kStepBytes, 1024);
    const uint32_t hi_v = (uint32_t)(dV >> 32), v_lo = (uint32_t)dV;
    bool ok = true;
    auto wait = [&](int b, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1));
      tc_fence_after();
      return ok;
    };
    int ks = 0, kphase = 0, vs = 0, vphase = 0;  // stages of the next K and V, their phases
    auto qk = [&](int t) {
      const uint32_t a = k_lo + ks * (kStepBytes / 16);
#pragma unroll
      for (int x = 0; x < 8; ++x)  // four steps of 32 dims, first then second term of Q
        mma_f8_ss_lead(leader, tmem + (t & 1) * R, a + (x & 3) * 2, q_lo + (x >> 2) * (R * 128 / 16) + (x & 3) * 2, hi_k,
                       idesc_e4m3_f32(128, R, 0, 0), x > 0);
      mma_commit_lead(leader, bar(kSFull + (t & 1)));
      mma_commit_lead(leader, bar(kKEmpty + ks));
      if (++ks == kKStages) {
        ks = 0;
        kphase ^= 1;
      }
    };
    int seg = 0;
    while (ok && next_segment()) {
      if (nothing_kept()) continue;
      if (!wait(kQFull, seg) || !wait(kKFull + ks, kphase)) break;
      ++seg;
      qk(gt);
      for (bool first = true, more = true; more; first = false) {
        more = !__any_sync(0xffffffffu, s_step[gt & (kSteps - 1)].last);
        if (more) {
          if (!wait(kKFull + ks, kphase)) break;
          qk(gt + 1);
        }
        if (!wait(kVClean + vs, vphase) || !wait(kPFull + (gt & 1), gt >> 1)) break;
        const uint32_t a = v_lo + vs * (kStepBytes / 16), p = p_lo + (gt & 1) * (C::kPBytes / 16);
#pragma unroll
        for (int x = 0; x < 4; ++x)  // 32 tokens a step
          mma_f8_ss_lead2(leader, tmem + C::kColO, a + x * (4096 / 16), hi_v, p + x * (32 * C::kPPitch / 16), hi_p,
                          idesc_e4m3_f32(128, 4 * R, 1, 1), !first || x > 0);
        mma_commit_lead(leader, bar(kODone + (gt & 1)));
        mma_commit_lead(leader, bar(kVEmpty + vs));
        if (++vs == kVStages) {
          vs = 0;
          vphase ^= 1;
        }
        ++gt;
      }
    }
    __syncwarp();
    mbar_wait(bar(kDone), 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  } else {
    // ------------------------------------------------------------ V
    bool ok = true;
    auto wait = [&](int b, int parity) {
      return ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1));
    };
    int vs = 0, vphase = 0, seg = 0;
    while (ok && next_segment()) {
      if (nothing_kept()) continue;
      for (bool last = false; !last; ++gt) {
        if (!wait(kVFull + vs, vphase)) break;
        const Step& st = s_step[gt & (kSteps - 1)];
        last = st.last;
        if (__builtin_expect(!st.full, 0)) {
          // Places without a token hold anything: their V must not meet a P of 0.
          // A NaN in V is kept from the rows that do not see its token.  A step
          // that is all there is read once; NaN is what a prompt hardly has.
          unsigned char* tile = sgen + C::kOffV + vs * kStepBytes;
          const int row0 = (warp & 1) * 4 + (lane >> 3), c = lane & 7;  // rows row0 + 8 it; row0 mod 8 = row mod 8
          auto cell_of = [&](int it) {
            return reinterpret_cast<uint4*>(tile + (row0 + 8 * it) * 128 + ((c ^ (row0 & 7)) << 4));
          };
          auto nan_in = [](const uint4& v) {
            return (((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                    ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u;
          };
          uint32_t any = 1u;
          if (st.there) {
            any = 0u;
#pragma unroll
            for (int it = 0; it < 16; ++it) any |= nan_in(*cell_of(it));
          }
          if (__any_sync(0xffffffffu, any != 0u)) {
            const int limit = sg.limit - st.j * 128;
#pragma unroll 1
            for (int it = 0; it < 16; ++it) {
              const int row = row0 + 8 * it;
              const bool there = row < limit && st.group[row >> 4].w != 0.f;
              uint4* cell = cell_of(it);
              const uint4 v = *cell;
              if (!there) *cell = make_uint4(0u, 0u, 0u, 0u);
              else if (nan_in(v)) {
                mbar_wait(bar(kQFull), seg & 1);  // the segment's rows are described
                uint32_t w[4] = {v.x, v.y, v.z, v.w}, nan = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t h = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                  for (int b = 0; b < 4; ++b) nan |= (h >> (8 * b + 7) & 1u) << (4 * e + b);
                  w[e] &= ~((h >> 7) * 0xffu);
                }
                *cell = make_uint4(w[0], w[1], w[2], w[3]);
                s_any_nan = 1;
                for (int r = 0; r < sg.live; ++r)
                  if (st.j * 128 + row < s_see[r] && ((st.heads >> s_head[r]) & 1ull))
                    atomicOr(&s_nan[r][c >> 1], nan << ((c & 1) * 16));
              }
            }
          }
          fence_proxy_async_smem();
        }
        mbar_arrive(bar(kVClean + vs));
        if (++vs == kVStages) {
          vs = 0;
          vphase ^= 1;
        }
      }
      ++seg;
    }
  }
  return;
  }
  regs_inc<kRegsHigh>();
  {
    // ------------------------------------------------------------ softmax
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    bool ok = true;
    // A wait that is given up is noted; the warps leave together at the next
    // barrier, none is left at one.
    auto waited = [&](uint32_t b, uint32_t parity) {
      const bool got = __all_sync(0xffffffffu, mbar_wait(b, parity));
      if (!got) s_fail = 1;
      tc_fence_after();
      return got;
    };
    bool first;
    // The steps of a segment for L >= live rows, and the rows' sums.
    auto steps = [&](auto rows_c) {
      constexpr int L = decltype(rows_c)::value;
      uint64_t l2[L / 2];
#pragma unroll
      for (int r = 0; r < L / 2; ++r) l2[r] = 0ull;
      for (bool last = false; !last; ++gt, first = false) {
        // S is there, and so is an end to PV of the step before the last, issued
        // before it: P's buffer is free
        const bool got = waited(bar(kSFull + (gt & 1)), (gt >> 1) & 1);
        const Step& st = s_step[gt & (kSteps - 1)];
        uint32_t sv[L <= 16 ? 16 : 32];
        if constexpr (L <= 16) {
          tmem_ld16(tmem + (gt & 1) * R + lanes, sv);
          tmem_wait_ld_dep16(sv);
        } else {
          tmem_ld32(tmem + (gt & 1) * R + lanes, sv);
          tmem_wait_ld_dep(sv);
        }
        last = st.last;
        const float4 f = st.group[tid >> 4];
        // y = S x factor + log2 of V's scale + offset: P = 2^y
        const uint64_t ks2 = f2_pack(f.x, f.x), lv2 = f2_pack(f.y, f.y);
        uint64_t y2[L / 2];
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < L / 2; ++r) {
          const float4 c = s_row[r];
          y2[r] = f2_fma(f2_pack(__uint_as_float(sv[2 * r]), __uint_as_float(sv[2 * r + 1])),
                         f2_mul(ks2, f2_pack(c.x, c.y)), f2_add(lv2, f2_pack(c.z, c.w)));
        }
        const bool full = st.full;
        bool there = true;
        const int pos = st.j * 128 + tid;
        // y of the rows that do not see this thread's token
        auto masked = [&]() {
          const uint64_t heads = st.heads;
#pragma unroll
          for (int r = 0; r < L / 2; ++r) {
            float y0, y1;
            f2_unpack(y2[r], y0, y1);
            if (!there || pos >= s_see[2 * r] || !((heads >> s_head[2 * r]) & 1ull)) y0 = -INFINITY;
            if (!there || pos >= s_see[2 * r + 1] || !((heads >> s_head[2 * r + 1]) & 1ull)) y1 = -INFINITY;
            y2[r] = f2_pack(y0, y1);
          }
        };
        if (__builtin_expect(!full, 0)) {
          there = f.w != 0.f && pos < sg.limit;
          masked();
        }
#pragma unroll
        for (int r = 0; r < L / 2; ++r) {
          float y0, y1;
          f2_unpack(y2[r], y0, y1);
          top = max3f(top, y0, y1);
        }
        if (softmax_any(top > kGrow + kPScale || !got)) {
          if (s_fail) {
            ok = false;
            return;
          }
          // some value exceeds its row's reference: move the references to the
          // maxima so far, found without their offsets
#pragma unroll
          for (int r = 0; r < L / 2; ++r) {
            const float4 c = s_row[r];
            y2[r] = f2_fma(f2_pack(__uint_as_float(sv[2 * r]), __uint_as_float(sv[2 * r + 1])),
                           f2_mul(ks2, f2_pack(c.x, c.y)), lv2);
          }
          if (!full) masked();
#pragma unroll
          for (int r = 0; r < L / 2; ++r) {
            float x0, x1;
            f2_unpack(y2[r], x0, x1);
            x0 = redux_max(x0);
            x1 = redux_max(x1);
            if (lane == 0) *reinterpret_cast<float2*>(&s_wmax[warp][2 * r]) = make_float2(x0, x1);
          }
          softmax_sync();
          if (tid < L) {
            float* off = reinterpret_cast<float*>(&s_row[tid >> 1]) + 2 + (tid & 1);
            const float old = *off;
            const float mx = fmaxf(fmaxf(s_wmax[0][tid], s_wmax[1][tid]), fmaxf(s_wmax[2][tid], s_wmax[3][tid]));
            const bool up = mx + old > kGrow + kPScale;
            s_alpha[tid] = up ? fast_exp2(kPScale - mx - old) : 1.f;
            if (up) *off = kPScale - mx;
          }
          softmax_sync();
#pragma unroll
          for (int r = 0; r < L / 2; ++r) {
            const float4 c = s_row[r];
            y2[r] = f2_add(y2[r], f2_pack(c.z, c.w));
            float a0, a1;
            f2_unpack(l2[r], a0, a1);
            l2[r] = f2_pack(a0 * s_alpha[2 * r], a1 * s_alpha[2 * r + 1]);
          }
          if (!first) {
            waited(bar(kODone + ((gt - 1) & 1)), ((gt - 1) >> 1) & 1);
#pragma unroll 1
            for (int c = 0; c < 4 * R; c += 16) {
              if ((c & (R - 1)) >= L) continue;
              uint32_t v[16];
              tmem_ld16(tmem + C::kColO + c + lanes, v);
              tmem_wait_ld_dep16(v);
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 f4 = *reinterpret_cast<const float4*>(&s_alpha[(c & (R - 1)) + e]);
                v[e] = __float_as_uint(__uint_as_float(v[e]) * f4.x);
                v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) * f4.y);
                v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) * f4.z);
                v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) * f4.w);
              }
              tmem_st16(tmem + C::kColO + c + lanes, v);
            }
            tmem_wait_st();
          }
        }
        const uint64_t i2 = f2_pack(f.z, f.z);
        unsigned char* at = sgen + C::kOffP + (gt & 1) * C::kPBytes;
#pragma unroll
        for (int r0 = 0; r0 < L; r0 += 16) {
          uint32_t w[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = r0 + 4 * q;
            if (r < L) {
              float p[4];
              f2_unpack(y2[r / 2], p[0], p[1]);
              f2_unpack(y2[r / 2 + 1], p[2], p[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) p[e] = fast_exp2(p[e]);
              l2[r / 2] = f2_fma(f2_pack(p[0], p[1]), i2, l2[r / 2]);
              l2[r / 2 + 1] = f2_fma(f2_pack(p[2], p[3]), i2, l2[r / 2 + 1]);
              split_p(p[0], p[1], p[2], p[3], w[0][q], w[1][q], w[2][q], w[3][q]);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            unsigned char* to = at + p_piece<R>(tid, (k * R + r0) / 16);
            if (L - r0 >= 16) *reinterpret_cast<uint4*>(to) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
            else if (L - r0 == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[k][0], w[k][1]);
            else *reinterpret_cast<uint32_t*>(to) = w[k][0];
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kPFull + (gt & 1)));
      }
#pragma unroll
      for (int r = 0; r < L / 2; ++r) {
        float a, b;
        f2_unpack(l2[r], a, b);
        a = warp_sum(a);
        b = warp_sum(b);
        if (lane == 0) *reinterpret_cast<float2*>(&s_sum[warp][2 * r]) = make_float2(a, b);
      }
    };
    for (;;) {
      if (tid == 0) s_more = s_walk[0].next(A, s_seg[0]);
      softmax_sync();
      if (!s_more) break;
      // Q of the unit's rows in two terms: 8 threads a row, 16 dims each
      const int c = tid & 7;
      uint4 v[R / 16][2];
#pragma unroll
      for (int n = 0; n < R / 16; ++n) {
        const int r = 16 * n + (tid >> 3), row = (sg.first + r) / g, head = (sg.first + r) - row * g;
        v[n][0] = v[n][1] = make_uint4(0u, 0u, 0u, 0u);
        if (r < sg.live) {
          const __nv_bfloat16* src = A.q + (long long)(sg.r.row0 + row) * A.q_tok +
                                     (long long)(sg.h * g + head) * A.q_head + c * 16;
          v[n][0] = ldg_nc_v4(src);
          v[n][1] = ldg_nc_v4(src + 8);
        }
        if (c == 0) {
          s_out[r] = ((long long)(sg.r.row0 + row) * A.hq + sg.h * g + head) * 128;
          s_see[r] = r < sg.live ? walk.seen_by(sg.r, row) : 0;
          s_head[r] = head;
          s_nan[r][0] = s_nan[r][1] = s_nan[r][2] = s_nan[r][3] = 0u;
        }
      }
#pragma unroll 1
      for (int r = tid >> 3; r < R; r += 16) {
        const uint32_t w[8] = {v[0][0].x, v[0][0].y, v[0][0].z, v[0][0].w, v[0][1].x, v[0][1].y, v[0][1].z, v[0][1].w};
        if constexpr (R > 16) {
          v[0][0] = v[1][0];
          v[0][1] = v[1][1];
        }
        float x[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[2 * e] = bf16lo(w[e]);
          x[2 * e + 1] = bf16hi(w[e]);
        }
        uint32_t w0[4], w1[4];
        const int ex = split_q(x, w0, w1);
        unsigned char* q0 = sgen + C::kOffQ + sw128(r, 16 * c);
        *reinterpret_cast<uint4*>(q0) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        *reinterpret_cast<uint4*>(q0 + R * 128) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        if (c == 0) {
          float* f = reinterpret_cast<float*>(&s_row[r >> 1]) + (r & 1);
          f[0] = exp2_int(ex) * A.scale_log2;
          f[2] = r < sg.live ? kNoMax : 0.f;
        }
      }
      const bool none = nothing_kept();  // O stays 0
      first = true;
      fence_proxy_async_smem();
      softmax_sync();
      if (s_fail) break;
      if (none) {
        if (tid < R) s_sum[0][tid] = s_sum[1][tid] = s_sum[2][tid] = s_sum[3][tid] = 0.f;
      } else {
        mbar_arrive(bar(kQFull));
        if (sg.live <= 4) steps(std::integral_constant<int, 4>());
        else if (sg.live <= 8) steps(std::integral_constant<int, 8>());
        else if (R == 16 || sg.live <= 16) steps(std::integral_constant<int, 16>());
        else if constexpr (R > 16) {
          if (sg.live <= 20) steps(std::integral_constant<int, 20>());
          else if (sg.live <= 24) steps(std::integral_constant<int, 24>());
          else steps(std::integral_constant<int, 32>());
        }
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      softmax_sync();
      if (!none) waited(bar(kODone + ((gt - 1) & 1)), ((gt - 1) >> 1) & 1);
      const bool whole = sg.j0 == 0 && sg.j1 == sg.nt;
      float* slot = P.partial + C::kSlotFloats * (2 * (size_t)blockIdx.x + (lo >= sg.unit ? 0 : 1));
      const bool nans = s_any_nan != 0;
      // (short loops: code that a unit runs once is fetched once, at a memory's latency)
#pragma unroll 1
      for (int r0 = 0; r0 < sg.live; r0 += 4) {
        uint32_t v[4][4];
        if (!none) {
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld4(tmem + C::kColO + k * R + r0 + lanes, v[k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_wait_ld_dep4(v[k]);
        }
        const float4 s0 = *reinterpret_cast<const float4*>(&s_sum[0][r0]), s1 = *reinterpret_cast<const float4*>(&s_sum[1][r0]),
                     s2 = *reinterpret_cast<const float4*>(&s_sum[2][r0]), s3 = *reinterpret_cast<const float4*>(&s_sum[3][r0]);
        const float sums[4] = {(s0.x + s1.x) + (s2.x + s3.x), (s0.y + s1.y) + (s2.y + s3.y),
                               (s0.z + s1.z) + (s2.z + s3.z), (s0.w + s1.w) + (s2.w + s3.w)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + e;
          if (r >= sg.live) break;
          float o = 0.f;
          if (!none)
            o = fmaf(fmaf(fmaf(__uint_as_float(v[3][e]), 0.03125f, __uint_as_float(v[2][e])), 0.03125f,
                          __uint_as_float(v[1][e])), 0.03125f, __uint_as_float(v[0][e]));
          if (nans && (s_nan[r][tid >> 5] >> lane & 1u)) o = NAN;
          const float sum = sums[e];
          if (whole) {
            // sum is 0 only where no token was seen; it is NaN where a score was
            A.o[s_out[r] + tid] = __float2bfloat16(sum == 0.f ? 0.f : o / sum);
          } else {
            __stcg(slot + r * 128 + tid, o);
            if (tid == 0)
              __stcg(reinterpret_cast<float2*>(slot + R * 128) + r,
                     make_float2(kPScale - (reinterpret_cast<float*>(&s_row[r >> 1]))[2 + (r & 1)], sum));
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        // count this part; the CTA that counts the last one adds them all
        const long long last = sg.step0 + sg.nt - 1, total = s_share.total;
        const int c0 = (int)(((sg.step0 + 1) * ctas - 1) / total), c1 = (int)(((last + 1) * ctas - 1) / total);
        softmax_sync();
        if (tid == 0) {
          asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zero
          s_last = count_acq_rel(P.counters + c0) == (unsigned)(c1 - c0);
        }
        softmax_sync();
        if (s_last) {
          const int slot0 = total * c0 / ctas >= sg.unit ? 0 : 1;
          auto slot_of = [&](int c) -> const float* {
            // slot 0 holds the segment with which a CTA begins, slot 1 the one with which it ends
            return P.partial + C::kSlotFloats * (2 * (size_t)c + (c == c0 ? slot0 : 0));
          };
          // The parts of N rows r, r + 4, ... (r: warp = row mod 4, lane = 4 dims), a
          // chunk of parts in flight: few rows can have hundreds of parts, many
          // rows have few.
          auto add_parts = [&](auto rows_c, auto chunk_c, int r) {
            constexpr int N = decltype(rows_c)::value, kChunk = decltype(chunk_c)::value;
            float m[N], sum[N];
            float4 acc[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
              m[n] = -kNoMax;
              sum[n] = 0.f;
              acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll 1
            for (int k0 = c0; k0 <= c1; k0 += kChunk) {
              float2 ml[kChunk][N];
              float4 o[kChunk][N];
#pragma unroll
              for (int k = 0; k < kChunk; ++k) {
                const float* p = slot_of(min(k0 + k, c1));
#pragma unroll
                for (int n = 0; n < N; ++n) {  // (rows behind the unit's last are in the slot, and dropped below)
                  ml[k][n] = ldcg_v2(p + R * 128 + 2 * (r + 4 * n));
                  o[k][n] = ldcg_v4(p + (r + 4 * n) * 128 + 4 * lane);
                }
              }
              __syncwarp();  // (no load sinks to its use: they are all in flight here)
#pragma unroll
              for (int n = 0; n < N; ++n) {
                float mx = m[n];
#pragma unroll
                for (int k = 0; k < kChunk; ++k) mx = fmaxf(mx, ml[k][n].x);
                const float old = fast_exp2(m[n] - mx);
                m[n] = mx;
                acc[n] = make_float4(acc[n].x * old, acc[n].y * old, acc[n].z * old, acc[n].w * old);
                sum[n] *= old;
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                  if (k0 + k > c1) break;
                  const float wt = fast_exp2(ml[k][n].x - mx);
                  acc[n].x = fmaf(o[k][n].x, wt, acc[n].x);
                  acc[n].y = fmaf(o[k][n].y, wt, acc[n].y);
                  acc[n].z = fmaf(o[k][n].z, wt, acc[n].z);
                  acc[n].w = fmaf(o[k][n].w, wt, acc[n].w);
                  sum[n] = fmaf(ml[k][n].y, wt, sum[n]);
                }
              }
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
              const int rr = r + 4 * n;
              if (rr >= sg.live) break;
              const float f = sum[n] == 0.f ? 0.f : 1.0f / sum[n];
              *reinterpret_cast<uint2*>(A.o + s_out[rr] + lane * 4) =
                  make_uint2(pack_bf16x2(acc[n].x * f, acc[n].y * f), pack_bf16x2(acc[n].z * f, acc[n].w * f));
            }
          };
          if (sg.live <= 4) {
            if (warp < sg.live) add_parts(std::integral_constant<int, 1>(), std::integral_constant<int, 16>(), warp);
          } else if (R == 16 || sg.live <= 16) {
            add_parts(std::integral_constant<int, 4>(), std::integral_constant<int, 4>(), warp);
          } else {
            add_parts(std::integral_constant<int, R / 4>(), std::integral_constant<int, 2>(), warp);
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

}  // namespace rows
}  // namespace cache
}  // namespace prism
