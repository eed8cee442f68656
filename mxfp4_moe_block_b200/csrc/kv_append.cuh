// kv_append.cuh -- a drafted block's queries, keys and values on their way
// from the packed projection to the attention: head norms, position rotation
// and the append to the paged cache, in one launch.
//
//   x^ = x / sqrt(mean_d x_d^2 + eps) * w        (queries and keys, per head)
//   (a, b) -> (a cos - b sin, a sin + b cos)     (the first `rot` dims)
//
// in float, rounded to bf16 once at the end; values are copied bit for bit.
// Pages name these as the "non-core" steps that dominate a verify step at
// microsecond scale (RMSNorm, RoPE, KV-cache write: "MiMo-v2.5-Pro-UltraSpeed
// - infra 架构解读"), hence one launch and no intermediate.
//
// Bound by memory (4 bytes moved per element, about 10 operations) and, for a
// few tokens, by the launch.  A group of D/8 lanes holds one head, 16 bytes a
// lane; the rotation's partner of a lane is a fixed lane of the group (rot is
// a multiple of 16, so rot/2 is a whole number of lanes), reached by a
// shuffle.  The heads are asked for before the token's place is looked up, and
// eight CTAs of 128 threads and 64 registers share an SM (the largest case below:
// 37.4 us, with four of 256 threads 39.0, with three 43).  Measured: one token of 80
// heads 2.4 us, 128 tokens of 56 heads 3.4 us (the launch), 4224 tokens of 80 heads
// of 128 37 us: 175 MB at 4.7 TB/s, 0.72 of a plain copy's rate (the shuffles, four a
// head for the norm and eight for the rotation of halves, fill the issue slots beside
// the loads; the eight are this layout's: a lane that held both units of a pair would
// need none).
#pragma once
#include "common.cuh"

namespace moe {

constexpr int APPEND_THREADS = 128;

struct AppendArgs {
  const uint16_t *qkv;           // [S*N, Hq + 2*Hkv, D]
  int N, Hq, Hkv;
  int norm;
  const uint16_t *q_weight, *k_weight;   // [D] or null (ones)
  float eps;
  const float *cos_sin;          // [max_pos, rot]: cosines, then sines
  int max_pos, rot, interleaved;
  const int32_t *kv_len, *block_table;
  int max_pages, num_pages, page_size;
  uint16_t *k_cache, *v_cache;   // [num_pages, Hkv, page_size, D]
  uint16_t *q_out;               // [S*N, Hq, D]
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// grid (S*N tokens, groups of HPT * 128/(D/8) heads).  Each lane group takes
// HPT heads of its token, so that the cosines and sines are read once for all.
template <int D, int HPT>
__global__ void __launch_bounds__(APPEND_THREADS, 8)
kv_append_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int LANES = D / 8;                     // lanes of one head: 8, 16 or 32
  constexpr int PER_PASS = APPEND_THREADS / LANES; // heads of one pass of the CTA
  const int t = blockIdx.x, s = t / a.N, i = t - s * a.N;
  const int l = threadIdx.x % LANES;
  const int h0 = blockIdx.y * (PER_PASS * HPT) + threadIdx.x / LANES;
  const int heads = a.Hq + 2 * a.Hkv;

  // the heads, on their way while the token's place is looked up
  uint4 raw[HPT];
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = h0 + j * PER_PASS;
    raw[j] = h < heads ? __ldcs(reinterpret_cast<const uint4 *>(a.qkv + ((size_t)t * heads + h) * D) + l)
                       : make_uint4(0, 0, 0, 0);
  }
  uint4 qw = make_uint4(0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80), kw = qw;   // ones
  if (a.norm && a.q_weight) qw = __ldg(reinterpret_cast<const uint4 *>(a.q_weight) + l);
  if (a.norm && a.k_weight) kw = __ldg(reinterpret_cast<const uint4 *>(a.k_weight) + l);

  // The token's place: its position is its distance from the end of the
  // cache.  A slot that is not in use (kv_len 0) and tokens before position 0
  // are left out; a position past the tables or a page id outside the pool is
  // reported and left out.
  const int pos = max(__ldg(a.kv_len + s), 0) - a.N + i;
  if (pos < 0) return;
  const int lp = pos / a.page_size;
  int page = -1;
  if (lp < a.max_pages) page = __ldg(a.block_table + (size_t)s * a.max_pages + lp);

  // this lane's cosines and sines: dims 8l..8l+7 turn with frequency
  // (dim mod rot/2), or with dim/2 where neighbours are pairs.  Pairs of halves:
  // x c + partner s, the sine's sign the half's.  Lanes past rot keep their dims (by
  // c = 1, s = 0 an infinity would become NaN).
  const int half = a.rot / 2;
  const bool turns = 8 * l < a.rot && pos < a.max_pos;
  const bool upper = 8 * l >= half;                // the pair's second element (halves)
  float c[8] = {}, sn[8] = {};
  if (turns) {
    const float *row = a.cos_sin + (size_t)pos * a.rot;
    if (a.interleaved) {
      const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + 4 * l));
      const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * l));
      c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
      sn[0] = s4.x; sn[1] = s4.y; sn[2] = s4.z; sn[3] = s4.w;
    } else {
      const int d = 8 * l - (upper ? half : 0);
      const float sign = upper ? 1.f : -1.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + d + 4 * j));
        const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + d + 4 * j));
        c[4 * j] = c4.x; c[4 * j + 1] = c4.y; c[4 * j + 2] = c4.z; c[4 * j + 3] = c4.w;
        sn[4 * j] = sign * s4.x; sn[4 * j + 1] = sign * s4.y;
        sn[4 * j + 2] = sign * s4.z; sn[4 * j + 3] = sign * s4.w;
      }
    }
  }
  if (page < 0 || page >= a.num_pages || (a.rot && pos >= a.max_pos)) {
    if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(MOE_DEV_BAD_INDEX);
    return;
  }
  const size_t row0 = (size_t)page * a.Hkv * a.page_size + (pos - lp * a.page_size);
  const int partner = 8 * l < a.rot ? (upper ? l - half / 8 : l + half / 8) : l;

#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = h0 + j * PER_PASS;
    const bool is_v = h >= a.Hq + a.Hkv;
    uint4 r = raw[j];
    // (the shuffles below are taken by every lane of the warp, or by none)
    if (__any_sync(FULL, h < a.Hq + a.Hkv)) {
      float x[8];
      unpack8(r, x);
      if (a.norm) {
        float ss = 0.f, w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
        const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        unpack8(h < a.Hq ? qw : kw, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv * w[e];
      }
      if (a.rot) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = x[2 * e], q = x[2 * e + 1];
            x[2 * e] = turns ? p * c[e] - q * sn[e] : p;
            x[2 * e + 1] = turns ? p * sn[e] + q * c[e] : q;
          }
        } else {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(FULL, x[e], partner, LANES);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = turns ? fmaf(y[e], sn[e], x[e] * c[e]) : x[e];
        }
      }
      if (!is_v)
        r = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                       pack_bf16(x[6], x[7]));
    }
    if (h >= heads) continue;
    uint16_t *dst;
    if (h < a.Hq) {
      dst = a.q_out + ((size_t)t * a.Hq + h) * D;
    } else {
      const int kvh = h - a.Hq - (is_v ? a.Hkv : 0);
      dst = (is_v ? a.v_cache : a.k_cache) + (row0 + (size_t)kvh * a.page_size) * D;
    }
    reinterpret_cast<uint4 *>(dst)[l] = r;
  }
}

// Heads per lane group: one where the tokens are few (one token of 80 heads: 2.4
// us with one, 4.1 with five), up to five, in equal shares, where each SM has four
// CTAs of tokens all the same (4224 tokens x 80 heads of 128: 69 us with one, 46
// with up to three, 37 with five).
template <int HPT>
inline cudaError_t launch_append_hpt(const AppendArgs &a, int T, int D, cudaStream_t s) {
  const int heads = a.Hq + 2 * a.Hkv;
  const int per = APPEND_THREADS / (D / 8) * HPT;
  const dim3 grid((unsigned)T, (unsigned)((heads + per - 1) / per));
  auto kern = D == 64    ? kv_append_kernel<64, HPT>
              : D == 128 ? kv_append_kernel<128, HPT>
                         : kv_append_kernel<256, HPT>;
  return launch_pdl(kern, grid, APPEND_THREADS, 0, s, a);
}

inline cudaError_t launch_append(const AppendArgs &a, int T, int D, int sms, cudaStream_t s) {
  const int per = APPEND_THREADS / (D / 8), passes = (a.Hq + 2 * a.Hkv + per - 1) / per;
  const int groups = (passes + 4) / 5;
  if ((long)T * groups < 4L * sms) return launch_append_hpt<1>(a, T, D, s);
  switch ((passes + groups - 1) / groups) {
    case 1: return launch_append_hpt<1>(a, T, D, s);
    case 2: return launch_append_hpt<2>(a, T, D, s);
    case 3: return launch_append_hpt<3>(a, T, D, s);
    case 4: return launch_append_hpt<4>(a, T, D, s);
    default: return launch_append_hpt<5>(a, T, D, s);
  }
}

}  // namespace moe
