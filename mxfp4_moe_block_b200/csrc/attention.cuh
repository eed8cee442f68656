// attention.cuh -- attention of a drafted block over a paged key-value cache.
#pragma once
#include "common.cuh"

namespace moe {

struct AttnArgs {
  const uint16_t *q;             // [S, N, Hq, D]
  int S, N, Hq, Hkv;
  const uint16_t *k_cache, *v_cache;   // [num_pages, Hkv, page_size, D]
  int num_pages, page_size;
  const int32_t *block_table;    // [S, max_pages]
  int max_pages;
  const int32_t *kv_len;         // [S]
  float scale;
  int window;
  uint16_t *out;                 // [S, N, Hq, D]
};

constexpr int ATTN_ROW_WARPS = 4;

// One warp per row (sequence, token, query head); 32 keys at a time: lane j
// scores key j, then the warp adds the 32 weighted value rows.
template <int D>
__global__ void __launch_bounds__(32 * ATTN_ROW_WARPS) attn_rows_kernel(const AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long row = (long)blockIdx.x * ATTN_ROW_WARPS + w;
  if (row >= (long)a.S * a.N * a.Hq) return;
  const int h = (int)(row % a.Hq), t = (int)(row / a.Hq), s = t / a.N, i = t - s * a.N;
  const int kvh = h / (a.Hq / a.Hkv);
  int n = max(__ldg(a.kv_len + s), 0);
  if ((n + a.page_size - 1) / a.page_size > a.max_pages) {   // longer than its row of the table
    raise_status(MOE_DEV_BAD_INDEX);
    n = 0;
  }
  const int pos = n - a.N + i;
  __shared__ float sq[ATTN_ROW_WARPS][D];
  for (int d = lane; d < D; d += 32) sq[w][d] = bf16_lo(a.q[(size_t)row * D + d]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  const int j0 = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  for (int b = j0; b <= pos; b += 32) {
    const int j = b + lane;
    float z = -INFINITY;
    size_t off = 0;
    if (j <= pos) {
      const int lp = j / a.page_size;
      const int page = __ldg(a.block_table + (size_t)s * a.max_pages + lp);
      if (page < 0 || page >= a.num_pages) {
        raise_status(MOE_DEV_BAD_INDEX);
      } else {
        off = (((size_t)page * a.Hkv + kvh) * a.page_size + (j - lp * a.page_size)) * D;
        const uint32_t *k = reinterpret_cast<const uint32_t *>(a.k_cache + off);
        float acc = 0.f;
        for (int d = 0; d < D / 2; ++d) {
          const uint32_t kk = __ldg(k + d);
          acc += bf16_lo(kk) * sq[w][2 * d] + bf16_hi(kk) * sq[w][2 * d + 1];
        }
        z = acc * a.scale;
      }
    }
    float zm = z;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) zm = fmaxf(zm, __shfl_xor_sync(FULL, zm, x));
    const float mn = fmaxf(m, zm);
    if (mn == -INFINITY) continue;
    const float corr = expf(m - mn), p = expf(z - mn);
    l = l * corr + warp_sum(p);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] *= corr;
    m = mn;
    for (int k = 0; k < 32; ++k) {
      const float pk = __shfl_sync(FULL, p, k);
      const size_t ok = __shfl_sync(FULL, off, k);
      if (pk == 0.f) continue;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] += pk * bf16_lo(a.v_cache[ok + lane + 32 * e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    a.out[(size_t)row * D + lane + 32 * e] = f32_to_bf16_bits(o[e] * inv);
}

}  // namespace moe
