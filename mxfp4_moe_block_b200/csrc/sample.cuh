// sample.cuh -- probabilities and tokens from logits under temperature,
// top-k, top-p and min-p.
//
// With z_v = (l_v - max l) / temperature the weight of token v is
// w_v = exp(z_v) and its mass the integer W_v = floor(w_v 2^40), both from
// double.  Tokens are ranked by logit, ties to the lowest index; every filter
// keeps a prefix of that ranking (top-k: the first k; top-p: the least prefix
// whose mass reaches top_p of the mass of the top-k prefix; min-p: W_v >=
// floor(min_p 2^40)), so that all together keep one, given by a threshold
// logit and, for the tokens equal to it, a last index.  The token drawn is the
// least v whose kept mass up to v exceeds floor(total U / 2^24): integer sums
// do not depend on the order of adding, so results are the same on every run.
//
// A thread-block cluster per row: each CTA brings its slice of the row into
// shared memory once and every later pass reads it there.  The threshold is
// found without sorting the row: a histogram of the distance to the maximum
// (counts, and exact masses where top-p needs them) over 1024 buckets names the
// bucket of the threshold; its few tokens -- and, for a small top-k, all
// tokens above -- go to the cluster's first CTA, which sorts them.  A bucket
// with more tokens than that list holds (many nearly equal logits) is split
// again by the bits of the logit, three times at most, and a group of equal
// logits is cut by a quotient and a count.
//
// The exponentials are the arithmetic: a double costs an SM 1/64 cycle an
// operation and one weight takes 14, ~4.5 weights per cycle and SM, against ~10
// logits per cycle that HBM delivers to an SM.  So each kept token's weight is
// computed once (twice for top-p over a whole row), the float of it stays in
// shared memory for the probabilities, and the draw recomputes 1/16 of one
// slice.
#pragma once
#include <cooperative_groups.h>
#include "common.cuh"

namespace moe {
namespace cg = cooperative_groups;

constexpr int SAMPLE_THREADS = 512;
constexpr int SAMPLE_WARPS = SAMPLE_THREADS / 32;
constexpr int SAMPLE_MAX_V = 393216;
constexpr int SAMPLE_BUCKETS = 1024;     // two per thread
constexpr int SAMPLE_LIST = 1024;        // tokens the first CTA sorts
constexpr int SAMPLE_MAX_CLUSTER = 8;
constexpr unsigned long long SAMPLE_ONE = 1ull << 40;

struct SampleArgs {
  const float *logits;           // [S*K, V]
  int K, V;
  const float *temperature;      // [S] or null
  const int32_t *top_k;
  const float *top_p, *min_p;
  const float *u;                // [S*K] or null
  int32_t *token;                // [S*K] or null
  float *probs;                  // [S*K, V] or null
  int slice;                     // tokens of a CTA, a multiple of 4
};

// In shared memory a logit is canonical: NaN becomes -infinity, -0 becomes 0,
// and places outside the row hold NaN.
__device__ __forceinline__ float canonical(float x) { return x == x ? x + 0.f : -INFINITY; }

// order-preserving key of a canonical logit
__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// w = 2^((x - top) c), c = log2(e) / temperature.  The exponent's integer part
// is split off by adding 1.5 2^52; 2^f on [-1/2, 1/2] is 1 + f p(f), p of degree
// 8 fitted to the least relative error at Chebyshev nodes: 2^-45.7.  Weights
// below 2^-1000 count as 0.
__device__ __forceinline__ double sample_weight(float x, float top, double c) {
  if (x == top) return 1.0;
  const double t = ((double)x - (double)top) * c;
  if (!(t > -1000.0)) return 0.0;
  const double shifted = t + 6755399441055744.0;
  const double f = t - (shifted - 6755399441055744.0);
  double p = 1.013516777919082e-07;
  p = fma(p, f, 1.3258416121625738e-06);
  p = fma(p, f, 1.525306990799785e-05);
  p = fma(p, f, 0.00015403440465134365);
  p = fma(p, f, 0.0013333557458737857);
  p = fma(p, f, 0.009618129181844376);
  p = fma(p, f, 0.05550410866978266);
  p = fma(p, f, 0.2402265069571947);
  p = fma(p, f, 0.6931471805598506);
  p = fma(p, f, 1.0);
  const long long bits = __double_as_longlong(p) +
                         ((long long)(int)(uint32_t)__double_as_longlong(shifted) << 52);
  return __longlong_as_double(bits);
}
// floor(w 2^40), w <= 1: added to 2^52 the integer part is the low bits
__device__ __forceinline__ unsigned long long sample_mass(double w) {
  return (unsigned long long)__double_as_longlong(__dadd_rd(w * 1099511627776.0, 4503599627370496.0)) &
         0xfffffffffffffull;
}

// A cluster's view of one row, and the block- and cluster-wide sums.
struct SampleRow {
  typedef unsigned long long u64;
  struct Found {               // what the first CTA tells the others
    int bucket, count;         // bucket of the threshold, its tokens
    u64 above, mass_above;     // tokens and mass of the buckets before it
    u64 upto;                  // tokens up to and with it
    u64 bar;                   // top-p's mass
    uint32_t thr;
    int cut;
  };
  struct Shared {
    u64 xch[8][SAMPLE_MAX_CLUSTER];
    double xchd[SAMPLE_MAX_CLUSTER];
    u64 red[SAMPLE_WARPS];
    double redd[SAMPLE_WARPS];
    u64 wsum[SAMPLE_WARPS];
    Found found;
    int list_n;
    int pos;
  };
};

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(FULL, v, o);
    v = w > v ? w : v;
  }
  return v;
}
// exclusive prefix of a value over the block's threads, and the block's total
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v,
                                                         unsigned long long *red,
                                                         unsigned long long &total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) red[w] = x;
  __syncthreads();
  unsigned long long before = 0;
  total = 0;
#pragma unroll
  for (int j = 0; j < SAMPLE_WARPS; ++j) {
    if (j < w) before += red[j];
    total += red[j];
  }
  return before + x - v;
}

// grid (cluster size, rows), cluster (cluster size, 1, 1)
__global__ void __launch_bounds__(SAMPLE_THREADS, 2) sample_kernel(const SampleArgs a) {
  typedef unsigned long long u64;
  pdl_wait();
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  cluster.barrier_arrive();       // (waited for before the first remote access)
  const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
  const int row = blockIdx.y, s = row / a.K, V = a.V;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  extern __shared__ __align__(16) uint8_t sample_smem[];
  __shared__ SampleRow::Shared sh;
  float *const val = reinterpret_cast<float *>(sample_smem);        // [slice + 4]
  uint32_t *const h_cnt = reinterpret_cast<uint32_t *>(val + a.slice + 4);   // filters only
  uint32_t *const h_lo = h_cnt + SAMPLE_BUCKETS, *const h_hi = h_lo + SAMPLE_BUCKETS;
  u64 *const list = reinterpret_cast<u64 *>(h_hi + SAMPLE_BUCKETS);

  // this CTA's tokens [c0, c1); val[i] is token c0 - shift + i, so that 16-byte
  // units of shared memory are 16-byte units of the row
  const int c0 = min(V, rank * a.slice), c1 = min(V, c0 + a.slice);
  const float *x = a.logits + (size_t)row * V;
  const int shift = (int)((reinterpret_cast<uintptr_t>(x + c0) >> 2) & 3);
  const int v0 = c0 - shift;                                        // token of val[0]
  const int units = c1 > c0 ? (c1 - v0 + 3) / 4 : 0;
  float4 *const val4 = reinterpret_cast<float4 *>(val);

  int use = 0;                    // exchange buffer: eight uses apart, barriers between
  auto exchange = [&](u64 v) -> const u64 * {                       // v: the same in every thread
    u64 *mine = sh.xch[use & 7];
    ++use;
    if (tid < C) *cluster.map_shared_rank(mine + rank, tid) = v;
    cluster.sync();
    return mine;
  };
  auto block_max = [&](u64 v) -> u64 {
    v = warp_max_u64(v);
    __syncthreads();
    if (lane == 0) sh.red[warp] = v;
    __syncthreads();
    v = sh.red[0];
#pragma unroll
    for (int j = 1; j < SAMPLE_WARPS; ++j) v = sh.red[j] > v ? sh.red[j] : v;
    return v;
  };
  auto cluster_max = [&](u64 v) -> u64 {
    const u64 *p = exchange(block_max(v));
    u64 m = p[0];
    for (int j = 1; j < C; ++j) m = p[j] > m ? p[j] : m;
    return m;
  };

  // ---- the slice into shared memory; the largest logit and its first index ----
  u64 best = 0;                                                     // key << 32 | ~index
  {
    constexpr int U = 4;
    for (int j = tid; j < units; j += U * SAMPLE_THREADS) {
      float4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int unit = j + i * SAMPLE_THREADS, v = v0 + 4 * unit;
        const float none = __int_as_float(0x7fffffff);
        if (unit >= units) break;
        if (v >= c0 && v + 3 < c1) {
          q[i] = __ldcs(reinterpret_cast<const float4 *>(x + v));
          q[i] = make_float4(canonical(q[i].x), canonical(q[i].y), canonical(q[i].z), canonical(q[i].w));
        } else {
          q[i].x = v >= c0 && v < c1 ? canonical(x[v]) : none;
          q[i].y = v + 1 >= c0 && v + 1 < c1 ? canonical(x[v + 1]) : none;
          q[i].z = v + 2 >= c0 && v + 2 < c1 ? canonical(x[v + 2]) : none;
          q[i].w = v + 3 >= c0 && v + 3 < c1 ? canonical(x[v + 3]) : none;
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int unit = j + i * SAMPLE_THREADS, v = v0 + 4 * unit;
        if (unit >= units) break;
        val4[unit] = q[i];
        const float e[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (e[k] == e[k]) {
            const u64 cand = ((u64)logit_key(e[k]) << 32) | (uint32_t)~(uint32_t)(v + k);
            best = cand > best ? cand : best;
          }
      }
    }
  }
  cluster.barrier_wait();
  best = cluster_max(best);
  const uint32_t top_key = (uint32_t)(best >> 32);
  const int top_token = (int)~(uint32_t)best;
  const float top = key_logit(top_key);

  // probabilities: 16-byte stores where the output's units are the input's
  float *const probs = a.probs ? a.probs + (size_t)row * V : nullptr;
  auto write_probs = [&](auto value) {                              // value(unit index) -> float4
    const bool same = ((reinterpret_cast<uintptr_t>(probs + c0) >> 2) & 3) == (uintptr_t)shift;
    for (int j = tid; j < units; j += SAMPLE_THREADS) {
      const int v = v0 + 4 * j;
      const float4 p = value(j);
      if (same && v >= c0 && v + 3 < c1) {
        __stcs(reinterpret_cast<float4 *>(probs + v), p);
      } else {
        const float e[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (v + k >= c0 && v + k < c1) probs[v + k] = e[k];
      }
    }
  };
  const double T = a.temperature ? (double)__ldg(a.temperature + s) : 1.0;
  const bool none = top == -INFINITY;
  if (none || !(T > 0.0)) {                       // no mass, or the first-ranked token alone
    if (rank == 0 && tid == 0) {
      if (none) raise_status(MOE_DEV_NO_MASS);
      if (a.token) a.token[row] = none ? -1 : top_token;
    }
    if (probs)
      write_probs([&](int j) {
        const int d = none ? -1 : top_token - (v0 + 4 * j);
        return make_float4(d == 0, d == 1, d == 2, d == 3);
      });
    return;                                       // (no remote access after the exchange)
  }
  const double c = 1.4426950408889634 / T;
  auto weight = [&](float l) { return sample_weight(l, top, c); };

  // ---- the threshold: kept are keys above thr, and at thr the tokens <= cut ----
  uint32_t thr = 0;
  int cut = 0x7fffffff;
  const int k = a.top_k ? __ldg(a.top_k + s) : 0;
  const double p = a.top_p ? (double)__ldg(a.top_p + s) : 1.0;
  const bool by_k = k > 0 && k < V, by_p = p < 1.0;
  const float mp = a.min_p ? __ldg(a.min_p + s) : 0.f;
  const u64 low = mp > 0.f ? (u64)((double)fminf(mp, 1.f) * (double)SAMPLE_ONE) : 0;

  if (by_k || by_p) {
    SampleRow::Found *const lead = cluster.map_shared_rank(&sh.found, 0);
    u64 *const lead_list = cluster.map_shared_rank(list, 0);
    int *const lead_n = cluster.map_shared_rank(&sh.list_n, 0);

    // every token of the slice that is still kept, with its key
    auto for_kept = [&](auto f) {
      for (int j = tid; j < units; j += SAMPLE_THREADS) {
        const float4 q = val4[j];
        const float e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!(e[i] == e[i])) continue;
          const uint32_t key = logit_key(e[i]);
          const int v = v0 + 4 * j + i;
          if (key > thr || (key == thr && v <= cut)) f(e[i], key, v);
        }
      }
    };
    // tokens to the first CTA's list
    auto push = [&](bool take, uint32_t key, int v) {
      if (take) {
        const int at = atomicAdd(lead_n, 1);
        if (at < SAMPLE_LIST) lead_list[at] = ((u64)key << 32) | (uint32_t)~(uint32_t)v;
      }
    };
    // the list, sorted by key and index (descending words), padded with zeros;
    // returns its length
    auto sort_list = [&]() -> int {
      const int n = min(sh.list_n, SAMPLE_LIST);
      int m = 32;
      while (m < n) m <<= 1;
      for (int i = n + tid; i < m; i += SAMPLE_THREADS) list[i] = 0;
      for (int size = 2; size <= m; size <<= 1)
        for (int d = size >> 1; d > 0; d >>= 1) {
          __syncthreads();
          for (int i = tid; i < m / 2; i += SAMPLE_THREADS) {
            const int lo = 2 * i - (i & (d - 1)), hi = lo + d;
            const u64 x0 = list[lo], x1 = list[hi];
            if ((x0 < x1) == ((lo & size) == 0)) {
              list[lo] = x1;
              list[hi] = x0;
            }
          }
        }
      __syncthreads();
      return n;
    };

    // One filter: the least prefix (of what is kept) with `want` tokens, or with
    // a mass of top_p times all.  `all`: where few enough, every token of the
    // prefix is listed and both filters are settled at once.
    auto select = [&](bool by_mass, u64 want) -> bool {
      const float scale =
          by_mass ? (float)(c * (SAMPLE_BUCKETS - 1) / 40.0) : (float)(SAMPLE_BUCKETS - 1) / 32.f;
      uint32_t khi = 0xffffffffu, klo = 0;       // keys in question
      int bits = -1;                             // bucket width, or the first level's scale
      u64 above = 0, mass_above = 0, bar = 0;
      for (;;) {
        auto bucket_of = [&](float l, uint32_t key) -> int {
          if (bits >= 0) return (int)((khi - key) >> bits);
          return l == top ? 0 : (int)fminf((top - l) * scale, (float)(SAMPLE_BUCKETS - 1));
        };
        for (int i = tid; i < SAMPLE_BUCKETS; i += SAMPLE_THREADS) h_cnt[i] = h_lo[i] = h_hi[i] = 0;
        if (tid == 0) sh.list_n = 0;
        __syncthreads();
        for_kept([&](float l, uint32_t key, int) {
          if (key < klo || key > khi) return;
          const int b = bucket_of(l, key);
          atomicAdd(h_cnt + b, 1u);
          if (by_mass) {
            const u64 m = sample_mass(weight(l));
            const uint32_t lo = (uint32_t)m, old = atomicAdd(h_lo + b, lo);
            const uint32_t hi = (uint32_t)(m >> 32) + (old + lo < old ? 1u : 0u);
            if (hi) atomicAdd(h_hi + b, hi);
          }
        });
        cluster.sync();
        if (rank == 0) {                         // add the CTAs' histograms, find the bucket
          u64 n[2] = {0, 0}, m[2] = {0, 0};
          for (int r = 0; r < C; ++r) {
            const uint32_t *rc = cluster.map_shared_rank(h_cnt, r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              n[i] += rc[2 * tid + i];
              if (by_mass)
                m[i] += ((u64)rc[2 * SAMPLE_BUCKETS + 2 * tid + i] << 32) + rc[SAMPLE_BUCKETS + 2 * tid + i];
            }
          }
          u64 tn, tm = 0, bm = 0;
          const u64 bn = block_scan(n[0] + n[1], sh.red, tn);
          if (by_mass) bm = block_scan(m[0] + m[1], sh.red, tm);
          if (by_mass && bits < 0) {             // (the first level sees every kept token)
            bar = p > 0.0 ? (u64)ceil(p * (double)tm) : 1;
            if (bar < 1) bar = 1;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const u64 pn = above + bn + (i ? n[0] : 0), pm = mass_above + bm + (i ? m[0] : 0);
            const bool here = by_mass ? pm < bar && bar <= pm + m[i] : pn < want && want <= pn + n[i];
            if (here)
              sh.found = SampleRow::Found{2 * tid + i, (int)n[i], pn, pm, pn + n[i], bar, 0, 0};
          }
        }
        cluster.sync();
        const SampleRow::Found f = *lead;
        bar = f.bar;
        const bool all = !by_mass && bits < 0 && f.upto <= SAMPLE_LIST;
        if (all || f.count <= SAMPLE_LIST) {
          for_kept([&](float l, uint32_t key, int v) {
            if (key < klo || key > khi) return;
            const int b = bucket_of(l, key);
            push(all ? b <= f.bucket : b == f.bucket, key, v);
          });
          cluster.sync();
          if (rank == 0) {
            const int n = sort_list();
            int last;                            // the list's last kept token
            if (!by_mass && !(all && by_p)) {
              last = (int)(want - (all ? 0 : f.above)) - 1;
            } else {
              // masses along the list: two tokens to a thread
              const int nk = by_mass ? n : min(n, (int)want);
              u64 m[2], total;
#pragma unroll
              for (int i = 0; i < 2; ++i)
                m[i] = 2 * tid + i < nk ? sample_mass(weight(key_logit((uint32_t)(list[2 * tid + i] >> 32)))) : 0;
              const u64 before = block_scan(m[0] + m[1], sh.red, total);
              u64 need = by_mass ? bar - f.mass_above
                                 : (p > 0.0 ? (u64)ceil(p * (double)total) : 1);
              if (need < 1) need = 1;
              if (tid == 0) sh.pos = nk - 1;
              __syncthreads();
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const u64 pm = before + (i ? m[0] : 0);
                if (pm < need && need <= pm + m[i]) sh.pos = 2 * tid + i;
              }
              __syncthreads();
              last = sh.pos;
            }
            if (tid == 0) {
              const u64 e = list[max(0, min(last, n - 1))];
              sh.found.thr = (uint32_t)(e >> 32);
              sh.found.cut = (int)~(uint32_t)e;
            }
          }
          cluster.sync();
          thr = lead->thr;
          cut = lead->cut;
          cluster.sync();                        // (found is free for the next filter)
          return all;
        }
        // more tokens than the list holds: the keys of this bucket
        above = f.above;
        mass_above = f.mass_above;
        if (bits < 0) {
          u64 hi = 0, lo = 0;
          for_kept([&](float l, uint32_t key, int) {
            if (bucket_of(l, key) != f.bucket) return;
            hi = key > hi ? key : hi;
            lo = (uint32_t)~key > lo ? (uint32_t)~key : lo;
          });
          khi = (uint32_t)cluster_max(hi);
          klo = ~(uint32_t)cluster_max(lo);
        } else {
          khi -= (uint32_t)f.bucket << bits;
          const uint32_t width = (1u << bits) - 1;
          klo = khi - klo > width ? khi - width : klo;
        }
        if (khi == klo) {                        // equal logits: cut by count
          const u64 one = by_mass ? sample_mass(weight(key_logit(khi))) : 1;
          const u64 take = by_mass ? (bar - mass_above + one - 1) / one : want - above;
          u64 mine = 0;
          for_kept([&](float, uint32_t key, int) { mine += key == khi; });
          u64 cnt;
          block_scan(mine, sh.red, cnt);
          const u64 *pc = exchange(cnt);
          u64 before = 0;
          for (int j = 0; j < rank; ++j) before += pc[j];
          // the CTA that holds the take-th of them finds its index
          u64 at = 0;
          if (before < take && take <= before + cnt) {
            u64 run = before;
            for (int b = 0; b < units && at == 0; b += SAMPLE_THREADS) {
              const int j = b + tid;
              const float4 q = j < units ? val4[j] : make_float4(NAN, NAN, NAN, NAN);
              const float e[4] = {q.x, q.y, q.z, q.w};
              u64 n = 0, sum;
              bool eq[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int v = v0 + 4 * j + i;
                eq[i] = e[i] == e[i] && logit_key(e[i]) == khi && (khi > thr || v <= cut);
                n += eq[i];
              }
              u64 r = run + block_scan(n, sh.red, sum);
              if (tid == 0) sh.pos = -1;
              __syncthreads();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (eq[i] && ++r == take) sh.pos = v0 + 4 * j + i;
              __syncthreads();
              if (sh.pos >= 0) at = (u64)sh.pos + 1;
              run += sum;
            }
          }
          const u64 *pa = exchange(at);
          u64 sum = 0;
          for (int j = 0; j < C; ++j) sum += pa[j];
          thr = khi;
          cut = (int)sum - 1;
          return false;
        }
        const int width = 32 - __clz(khi - klo);   // bits of the distance
        bits = width > 10 ? width - 10 : 0;
      }
    };

    bool settled = false;
    if (by_k) settled = select(false, (u64)k);
    if (by_p && !settled) select(true, 0);
  }

  // ---- sums over what is kept; warp w takes the w-th part of the slice ----
  const int wu = (units + SAMPLE_WARPS - 1) / SAMPLE_WARPS;         // units of a warp
  u64 mass = 0;
  double wsum = 0.0;
  {
    const int j1 = min(units, (warp + 1) * wu);
    const float below = (float)(-1000.0 / c);
    for (int j = warp * wu + lane; j < j1; j += 32) {
      const float4 q = val4[j];
      float e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float keep = 0.f;
        if (e[i] == e[i] && (e[i] == top || e[i] - top > below)) {
          const uint32_t key = logit_key(e[i]);
          if (key > thr || (key == thr && v0 + 4 * j + i <= cut)) {
            const double w = weight(e[i]);
            const u64 m = sample_mass(w);
            if (m >= low) {
              mass += m;
              wsum += w;
              keep = (float)w;
            }
          }
        }
        e[i] = keep;
      }
      if (probs) val4[j] = make_float4(e[0], e[1], e[2], e[3]);     // weights, for the probabilities
    }
  }
  mass = warp_sum_u64(mass);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(FULL, wsum, o);
  __syncthreads();
  if (lane == 0) {
    sh.wsum[warp] = mass;
    sh.redd[warp] = wsum;
  }
  __syncthreads();
  u64 cta_mass = 0;
  double cta_w = 0.0;
#pragma unroll
  for (int j = 0; j < SAMPLE_WARPS; ++j) {
    cta_mass += sh.wsum[j];
    cta_w += sh.redd[j];
  }
  if (tid < C) *cluster.map_shared_rank(&sh.xchd[rank], tid) = cta_w;
  const u64 *pm = exchange(cta_mass);
  u64 total = 0, before = 0;
  double sum = 0.0;
  for (int j = 0; j < C; ++j) {
    if (j < rank) before += pm[j];
    total += pm[j];
    sum += sh.xchd[j];
  }
  // no CTA leaves before every other has finished writing to it: the exchange
  // above was the last remote access
  if (probs) {
    const float inv = (float)(1.0 / sum);
    write_probs([&](int j) {
      const float4 q = val4[j];
      return make_float4(q.x * inv, q.y * inv, q.z * inv, q.w * inv);
    });
  }
  if (!a.token) return;

  // ---- the draw: the CTA, the warp's part, then a few tokens to a thread ----
  const u64 U = (u64)((double)__ldg(a.u + row) * 16777216.0);
  const u64 m = (__umul64hi(total, U) << 40) | ((total * U) >> 24);
  if (!(before <= m && m < before + cta_mass)) return;
  int part = 0;
  for (u64 w = sh.wsum[0]; before + w <= m; w = sh.wsum[part]) {
    before += w;
    ++part;
  }
  const int b0 = max(c0, v0 + 4 * part * wu), b1 = min(c1, v0 + 4 * min(units, (part + 1) * wu));
  const int each = (b1 - b0 + SAMPLE_THREADS - 1) / SAMPLE_THREADS;
  const int t0 = min(b1, b0 + tid * each), t1 = min(b1, t0 + each);
  auto mass_of = [&](int v) -> u64 {
    const float l = canonical(x[v]);
    const uint32_t key = logit_key(l);
    if (key < thr || (key == thr && v > cut)) return 0;
    const u64 mv = sample_mass(weight(l));
    return mv >= low ? mv : 0;
  };
  u64 mine = 0, all;
  for (int v = t0; v < t1; ++v) mine += mass_of(v);
  u64 run = before + block_scan(mine, sh.red, all);
  if (run <= m && m < run + mine)
    for (int v = t0; v < t1; ++v) {
      run += mass_of(v);
      if (run > m) {
        a.token[row] = v;
        break;
      }
    }
}

// CTAs of a row: slices of at most 18432 tokens (72 KB, two CTAs per SM) and,
// for few rows, enough CTAs for the machine with 2048 tokens each at least.
inline int sample_cluster(int rows, int V, int sms) {
  int c = 1;
  while (c < SAMPLE_MAX_CLUSTER &&
         ((V + c - 1) / c > 18432 || ((long)rows * c < sms && V / (2 * c) >= 2048)))
    c *= 2;
  return c;
}
inline int sample_slice(int V, int c) { return ((V + c - 1) / c + 3) / 4 * 4; }
inline size_t sample_smem_bytes(int slice, bool filters) {
  return (size_t)(slice + 4) * 4 + (filters ? SAMPLE_BUCKETS * 12 + SAMPLE_LIST * 8 : 0);
}

}  // namespace moe
