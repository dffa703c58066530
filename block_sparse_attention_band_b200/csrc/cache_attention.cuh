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

// One CTA per (row, query head): thread = token for the scores of a 128-token
// tile, thread = dim for the products with V.
__global__ void __launch_bounds__(128) attn_simple_kernel(const AttnParams P) {
  __shared__ float s_q[128], s_p[128], s_red[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, h = blockIdx.y, hk = h / (P.hq / P.hkv);
  int lo = 0, hi = P.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.starts[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const Request R = request_of(P, lo);
  if (t < R.row0 || t >= R.row0 + R.rows) return;
  const int limit = min(R.len, R.len - R.rows + (t - R.row0) + 1);  // tokens that this row sees
  s_q[tid] = __bfloat162float(P.q[t * P.q_tok + h * P.q_head + tid]) * P.scale_log2;
  __syncthreads();
  const int page = 1 << P.page_shift;
  const uint32_t* mrow = P.mask ? P.mask + ((size_t)lo * P.hq + h) * P.words : nullptr;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int p0 = 0; p0 < limit; p0 += 128) {
    if (mrow && !((mrow[p0 >> 12] >> ((p0 >> 7) & 31)) & 1u)) continue;
    const int pos = p0 + tid;
    float s = -INFINITY;
    if (pos < limit) {
      const int pg = P.table[(size_t)lo * P.max_pages + (pos >> P.page_shift)];
      if (pg >= 0 && pg < P.num_pages) {
        const uint8_t* row = P.kc + (size_t)pg * P.page_stride + ((size_t)hk * page + (pos & (page - 1))) * 128;
        float d = 0.f;
        for (int c = 0; c < 128; c += 2) {
          const float2 k2 = from_e4m3x2(*reinterpret_cast<const uint16_t*>(row + c));
          d = fmaf(k2.x, s_q[c], fmaf(k2.y, s_q[c + 1], d));
        }
        s = d * P.ks[(size_t)pg * P.hkv + hk];
      } else {
        set_device_error(kDevErrCache);
      }
    }
    float mx = s;
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if (lane == 0) s_red[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) {  // (only pages that are not there)
      __syncthreads();
      continue;
    }
    const float alpha = exp2f(m - mn);
    m = mn;
    s_p[tid] = exp2f(s - m);
    __syncthreads();
    l *= alpha;
    acc *= alpha;
    for (int x = 0; x < 128 && p0 + x < limit; ++x) {
      const float p = s_p[x];
      l += p;
      const int pg = P.table[(size_t)lo * P.max_pages + ((p0 + x) >> P.page_shift)];
      if (pg < 0 || pg >= P.num_pages) continue;
      const uint8_t c = P.vc[(size_t)pg * P.page_stride + ((size_t)hk * page + ((p0 + x) & (page - 1))) * 128 + tid];
      acc = fmaf(p * P.vs[(size_t)pg * P.hkv + hk], from_e4m3x2(c).x, acc);
    }
    __syncthreads();
  }
  P.o[((size_t)t * P.hq + h) * 128 + tid] = __float2bfloat16(l > 0.f ? acc / l : 0.f);
}

}  // namespace cache
}  // namespace prism
