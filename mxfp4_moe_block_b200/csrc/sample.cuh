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
// (counts, or the exact masses where top-p needs them) over 1024 buckets names the
// bucket of the threshold, whose few tokens go to the cluster's first CTA; with
// four words (logit, ~index) to a thread it narrows them by histograms of its own
// and ranks the last 32 by comparing.  A bucket with more tokens than that list
// holds (many nearly equal logits) is split again by the bits of the logit, three
// times at most, and a group of equal logits is cut by a quotient and a count.  A
// small top-k needs no histogram over the cluster: the k first-ranked lie above
// the k-th largest of a CTA's 512 threads' own maxima, and the first CTA settles
// the row from the tokens there.
//
// Bounds.  The bytes: a row in and, where wanted, its probabilities out.  The
// exponentials: an SM does 64 double operations a cycle and a weight with its mass
// takes 10 (and two conversions, 16 a cycle), ~6 weights per cycle and SM, against
// ~6 logits per cycle that HBM delivers to an SM.  So a kept token's weight is
// computed once (top-p over a whole row: every weight, and the kept ones again);
// where few are kept they wait in a queue until a warp has 32 of them; the float of
// a weight stays in shared memory for the probabilities.  And the row's steps one
// after another: five to nine barriers of the cluster and the first CTA's search
// between them, 8 us for a row of 32000 without filters, 19 with top-p, hidden by
// other rows only as far as two CTAs fit an SM (issue slots 58 % busy, DRAM 16 %).  Two
// it is by registers (64 of 512 threads); the shared memory of a slice of 16000 tokens
// without filters would do for three.
// Measured, with probabilities: 128 rows of 152064, mixed filters, 122 us (24 us at
// HBM's rate); 1024 rows of 32000, temperature 109 us (40 us), top-k 50 133 us,
// top-p 0.9 261 us; one row of 32000 under every filter, token only, 13 us.
#pragma once
#include <cfloat>
#include <cooperative_groups.h>
#include <type_traits>
#include "common.cuh"

namespace moe {
namespace cg = cooperative_groups;

constexpr int SAMPLE_THREADS = 512;
constexpr int SAMPLE_WARPS = SAMPLE_THREADS / 32;
constexpr int SAMPLE_MAX_V = 393216;
constexpr int SAMPLE_BUCKETS = 1024;     // two per thread
constexpr int SAMPLE_LIST = 2048;        // tokens the first CTA looks through, four per thread
constexpr int SAMPLE_QUEUE = 160;        // a warp's kept tokens that wait for their weights
constexpr int SAMPLE_SMALL_K = 128;      // top-k that the first CTA settles alone
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

// order-preserving key of a logit, -0 as 0.  (NaN counts as no token at all; in
// shared memory it also fills the places outside the row.)
__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// 2^40 w = 2^(d c + 40), d = x - top <= 0, c = log2(e) / temperature, for
// d c > -1000 (the caller takes 0 for less).  The exponent's nearest integer
// comes from float (it need not be exact: the remainder f is), counted in 16ths.  Of
// 2^(n + j/16 + f) the middle factor is looked up (16 doubles, a shared memory bank
// pair each: no conflicts) and 2^f on [-1/32, 1/32] is 1 + f p(f), p of degree 5
// fitted to the least relative error at Chebyshev nodes: 2^-55.8.  With the rounding
// of what it takes 2^40 w comes within 2^-12 of its value, so a mass can differ from the
// definition's floor only where that lies as near to a whole number (5 of 10^5 masses
// above 2^39).  9 double operations and two conversions.
__constant__ double kSampleSteps[16] = {
    1.0, 1.0442737824274138, 1.0905077326652577, 1.1387886347566916,
    1.189207115002721, 1.241857812073484, 1.2968395546510096, 1.3542555469368927,
    1.4142135623730951, 1.4768261459394993, 1.5422108254079407, 1.6104903319492543,
    1.681792830507429, 1.7562521603732995, 1.8340080864093424, 1.9152065613971474};
struct SampleScale {
  double top, c, halving;         // halving: logits to a factor of two
  float ftop, fc, lowest;         // logits below `lowest` (d c < -1000) weigh 0
  const double *steps;            // 2^(j/16), in shared memory
  __device__ __forceinline__ SampleScale(float t, double temperature, const double *steps)
      : steps(steps), top((double)t), c(1.4426950408889634 / temperature),
        halving(temperature * 0.6931471805599453), ftop(t), fc((float)c) {
    const double least = fma(-1000.0, halving, top);
    lowest = fmaxf((float)least, -FLT_MAX);
    if ((double)lowest < least) lowest = key_logit(logit_key(lowest) + 1);   // (rounded down)
  }
  __device__ __forceinline__ bool positive(float x) const { return x >= lowest; }   // NaN: no
  __device__ __forceinline__ double weight(float x) const {
    const float magic = 786432.f + 40.f;                            // 1.5 2^19, and the 2^40
    const float shifted = fmaf(x - ftop, fc, magic);
    const int b = __float_as_int(shifted);
    const double f = fma((double)x - top, c, -(double)(shifted - magic));
    const double t = steps[b & 15];
    double p = 0.0001540372522169807;
    p = fma(p, f, 0.001333378300903704);
    p = fma(p, f, 0.00961812910691042);
    p = fma(p, f, 0.05550410865653406);
    p = fma(p, f, 0.24022650695910075);
    p = fma(p, f, 0.6931471805599457);
    p = fma(t * f, p, t);
    return __hiloint2double(__double2hiint(p) + ((b & ~15) << 16), __double2loint(p));
  }
};
// floor(2^40 w), 2^-960 < 2^40 w <= 2^40: added to 2^52 the integer part is the
// low 52 bits (the high 12 are left to the caller to mask: sums of masses below
// 2^52 stay apart from them)
constexpr unsigned long long SAMPLE_MASK = 0xfffffffffffffull;
__device__ __forceinline__ unsigned long long sample_mass_bits(double w40) {
  return (unsigned long long)__double_as_longlong(__dadd_rd(w40, 4503599627370496.0));
}
__device__ __forceinline__ unsigned long long sample_mass(double w40) {
  return sample_mass_bits(w40) & SAMPLE_MASK;
}

// A cluster's view of one row, and the block- and cluster-wide sums.
struct SampleRow {
  typedef unsigned long long u64;
  struct Found {               // what the first CTA tells the others
    int bucket, count;         // bucket of the threshold, its tokens (by count)
    u64 above, mass_above;     // tokens or mass of the buckets before it
    u64 bar;                   // top-p's mass
    uint32_t thr;
    int cut;
    float inv;                 // 2^-40 / sum of the kept weights, where the list settles a row
  };
  struct Shared {
    u64 xch[8][SAMPLE_MAX_CLUSTER];
    double xchd[SAMPLE_MAX_CLUSTER];
    u64 red[SAMPLE_WARPS];
    double redd[SAMPLE_WARPS];
    u64 wsum[SAMPLE_WARPS];
    alignas(16) uint32_t warp_max[2 * SAMPLE_WARPS];
    Found found;
    int list_n;                // tokens in this CTA's list
    int above_n;               // and of its slice above the threshold's bucket
    int pos;
    double steps[16];          // (SampleScale)
  };
};

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
__device__ __forceinline__ void sample_copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
// A thread's arrival at the cluster's barrier that publishes nothing of its own
// (an ordinary one first waits for the thread's own writes to be seen)
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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
  cluster_arrive_relaxed();       // (waited for before the first remote access)
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

  // One value of each CTA to all: warp 0 of a CTA gives it (in every lane) and
  // publishes it; nothing else is published.
  int use = 0;                    // exchange buffer: eight uses apart, barriers between
  auto exchange = [&](u64 v) -> const u64 * {
    u64 *mine = sh.xch[use & 7];
    ++use;
    if (tid < C) *cluster.map_shared_rank(mine + rank, tid) = v;
    __syncwarp();
    if (warp == 0) cluster.barrier_arrive();
    else cluster_arrive_relaxed();
    cluster.barrier_wait();
    return mine;
  };
  auto cluster_max = [&](uint32_t v) -> uint32_t {
    v = __reduce_max_sync(FULL, v);
    if (lane == 0) sh.warp_max[warp] = v;
    __syncthreads();
    const u64 *p = exchange(warp ? 0 : __reduce_max_sync(FULL, sh.warp_max[lane % SAMPLE_WARPS]));
    uint32_t m = (uint32_t)p[0];
    for (int j = 1; j < C; ++j) m = max(m, (uint32_t)p[j]);
    return m;
  };

  // ---- the slice into shared memory, all of it in flight at once; a
  // sequence's settings meanwhile ----
  for (int j = tid; j < units; j += SAMPLE_THREADS) {
    const int v = v0 + 4 * j;
    if (v >= c0 && v + 3 < c1) {
      sample_copy16(val4 + j, x + v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        val[4 * j + i] = v + i >= c0 && v + i < c1 ? x[v + i] : __int_as_float(0x7fffffff);
    }
  }
  if (tid < 16) sh.steps[tid] = kSampleSteps[tid];
  const double T = a.temperature ? (double)__ldg(a.temperature + s) : 1.0;
  const int k = a.top_k ? __ldg(a.top_k + s) : 0;
  const double p = a.top_p ? (double)__ldg(a.top_p + s) : 1.0;
  const float mp = a.min_p ? __ldg(a.min_p + s) : 0.f;
  const u64 U = a.token ? (u64)(fminf(__ldg(a.u + row), 0x0.ffffffp0f) * 16777216.f) : 0;   // < 2^24
  asm volatile("cp.async.wait_all;" ::: "memory");
  // (each thread reads back what it copied itself)
  float most = -INFINITY;
  for (int j = tid; j < units; j += SAMPLE_THREADS) {
    const float4 q = val4[j];
    most = fmaxf(most, fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)));    // (skips NaN)
  }
  cluster.barrier_wait();
  const uint32_t top_key = cluster_max(logit_key(most));
  float top = key_logit(top_key);
  // +infinity takes all mass: such a row counts as 0 there and -infinity elsewhere
  const bool inf_row = top == INFINITY;
  auto infinite = [&](float l) { return inf_row ? (l == INFINITY ? 0.f : l == l ? -INFINITY : l) : l; };
  if (inf_row) {
    for (int j = tid; j < units; j += SAMPLE_THREADS) {
      const float4 q = val4[j];
      val4[j] = make_float4(infinite(q.x), infinite(q.y), infinite(q.z), infinite(q.w));
    }
    top = 0.f;
    __syncthreads();
  }

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
  const bool none = top == -INFINITY;
  if (none || !(T > 0.0)) {                       // no mass, or the first-ranked token alone
    uint32_t first = 0;                           // ~index of the first largest logit
    if (!none) {
      for (int j = tid; j < units; j += SAMPLE_THREADS) {
        const float4 q = val4[j];
        const int i = q.x == top ? 0 : q.y == top ? 1 : q.z == top ? 2 : q.w == top ? 3 : 4;
        if (i < 4) {
          first = ~(uint32_t)(v0 + 4 * j + i);
          break;
        }
      }
      first = cluster_max(first);
    }
    const int top_token = (int)~first;
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
  // (limits that keep the scale, its reciprocal and its products finite in float)
  const SampleScale z(top, fmin(fmax(T, 1e-36), 1e30), sh.steps);
  auto mass_at = [&](float l) -> u64 { return z.positive(l) ? sample_mass(z.weight(l)) : 0; };

  // ---- the threshold: kept are logits above `at`, and at it the tokens <= last ----
  float at = -INFINITY;
  int last = 0x7fffffff;
  bool cutting = false;
  auto kept = [&](float l, int v) { return l > at || (l == at && v <= last); };      // (NaN: no)
  auto cut_to = [&](uint32_t key, int v) {
    at = key_logit(key);
    last = v;
    cutting = true;
  };
  const bool by_k = k > 0 && k < V, by_p = p < 1.0;
  const u64 low = mp > 0.f ? (u64)((double)fminf(mp, 1.f) * (double)SAMPLE_ONE) : 0;

  // Every kept token of a warp's part of the slice, weighed by f(place in val) with
  // full warps: few are kept as a rule, and they wait in the warp's queue (in the
  // list's place) until there is one for every lane.  `zero`: the others become 0.
  const int wu = (units + SAMPLE_WARPS - 1) / SAMPLE_WARPS;         // units of a warp
  // top-p keeps a third of the slice or more: then each weight where it stands, else
  // the queue (1024 rows of 32000, top-p 0.9: queue 261 us, in place 272; 0.99: 285
  // and 274; top-p 0.7 246 and 266)
  bool many = false;
  float least = -INFINITY;                       // no token below this logit is kept
  auto for_queued = [&](auto f, bool zero = false) {
    uint32_t *const queue = reinterpret_cast<uint32_t *>(list) + warp * SAMPLE_QUEUE;
    const int j1 = min(units, (warp + 1) * wu);
    const float from = fmaxf(fmaxf(at, z.lowest), least);
    const int upto = from == at ? last : 0x7fffffff;                // of the tokens at `from`
    int waiting = 0;
    auto serve = [&](int n) {                                       // the queue's last n
      waiting -= n;
      if (lane < n) f(queue[waiting + lane]);
      __syncwarp();
    };
    for (int j = warp * wu + lane; j - lane < j1; j += 32) {
      const float none = __int_as_float(0x7fffffff);
      const float4 q = j < j1 ? val4[j] : make_float4(none, none, none, none);
      float e[4] = {q.x, q.y, q.z, q.w};
      bool keep[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        keep[i] = e[i] > from || (e[i] == from && v0 + 4 * j + i <= upto);
      if (__any_sync(FULL, keep[0] || keep[1] || keep[2] || keep[3])) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned who = __ballot_sync(FULL, keep[i]);
          if (keep[i]) queue[waiting + __popc(who & lanemask_lt())] = (uint32_t)(4 * j + i);
          waiting += __popc(who);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = keep[i] ? e[i] : 0.f;
      if (zero && j < j1) val4[j] = make_float4(e[0], e[1], e[2], e[3]);
      __syncwarp();
      while (waiting >= 32) serve(32);
    }
    if (waiting) serve(waiting);
  };

  if (by_k || by_p) {
    SampleRow::Found *const lead = cluster.map_shared_rank(&sh.found, 0);

    // every token of the slice that is still kept
    auto for_kept = [&](auto f) {
      for (int j = tid; j < units; j += SAMPLE_THREADS) {
        const float4 q = val4[j];
        const float e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (kept(e[i], v0 + 4 * j + i)) f(e[i]);
      }
    };
    auto clear = [&]() {
      for (int i = tid; i < SAMPLE_BUCKETS; i += SAMPLE_THREADS) h_cnt[i] = h_lo[i] = h_hi[i] = 0;
      __syncthreads();
    };
    // The first CTA adds the CTAs' histograms and finds the bucket in which the
    // count (after `above` tokens) reaches `want`, or the mass (after
    // mass_above) reaches bar; a bar of 0 is set here, from the mass of all.
    // Every CTA gets what was found; bucket -1: fewer than wanted.
    auto find = [&](bool by_mass, u64 want, u64 above, u64 mass_above, u64 bar) -> SampleRow::Found {
      cluster.sync();
      if (rank == 0) {
        u64 n[2] = {0, 0};                       // tokens or mass of this thread's two buckets
#pragma unroll
        for (int r = 0; r < SAMPLE_MAX_CLUSTER; ++r) {
          if (r >= C) break;
          const uint32_t *rc = cluster.map_shared_rank(h_cnt, r);
          if (by_mass) {
            const uint2 lo = *reinterpret_cast<const uint2 *>(rc + SAMPLE_BUCKETS + 2 * tid);
            const uint2 hi = *reinterpret_cast<const uint2 *>(rc + 2 * SAMPLE_BUCKETS + 2 * tid);
            n[0] += ((u64)hi.x << 32) + lo.x;
            n[1] += ((u64)hi.y << 32) + lo.y;
          } else {
            const uint2 cnt = *reinterpret_cast<const uint2 *>(rc + 2 * tid);
            n[0] += cnt.x;
            n[1] += cnt.y;
          }
        }
        u64 all;
        u64 run = (by_mass ? mass_above : above) + block_scan(n[0] + n[1], sh.red, all);
        if (by_mass) {
          if (bar == 0) {
            bar = p > 0.0 ? (u64)ceil(p * (double)all) : 1;
            if (bar < 1) bar = 1;
          }
          want = bar;
        } else if (tid == 0 && above + all < want) {
          sh.found.bucket = -1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (run < want && want <= run + n[i])
            sh.found = SampleRow::Found{2 * tid + i, (int)n[i], run, run, bar, 0, 0, 0.f};
          run += n[i];
        }
      }
      cluster.sync();
      return *lead;
    };
    // kept tokens that pass a test (few do) to this CTA's list; the first CTA looks
    // through all CTAs' together
    auto collect = [&](auto test) {
      for (int j = tid; j < units; j += SAMPLE_THREADS) {
        const float4 q = val4[j];
        const float e[4] = {q.x, q.y, q.z, q.w};
        bool take[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) take[i] = test(e[i]);
        if (!(take[0] || take[1] || take[2] || take[3])) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (take[i] && kept(e[i], v0 + 4 * j + i)) {
            const int to = atomicAdd(&sh.list_n, 1);
            if (to < SAMPLE_LIST)
              list[to] = ((u64)logit_key(e[i]) << 32) | (uint32_t)~(uint32_t)(v0 + 4 * j + i);
          }
      }
    };
    auto list_total = [&]() {
      int n = 0;
      for (int r = 0; r < C; ++r) n += *cluster.map_shared_rank(&sh.list_n, r);
      return n;
    };
    // ---- the first CTA's part: the lists' words (key, ~index), four to a thread,
    // in registers; all are different, so a prefix of the ranking is the words at or
    // above one of them ----
    constexpr int PER = SAMPLE_LIST / SAMPLE_THREADS;
    auto take_lists = [&](int n, u64 (&v)[PER]) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        int i = tid + j * SAMPLE_THREADS, r = 0;
        v[j] = 0;
        if (i >= n) continue;
        int c = sh.list_n;
        while (i >= c) {
          i -= c;
          c = *cluster.map_shared_rank(&sh.list_n, ++r);
        }
        v[j] = cluster.map_shared_rank(list, r)[i];
      }
    };
    auto word_logit = [&](u64 v) { return key_logit((uint32_t)(v >> 32)); };
    // The word down to which the words (0: none) reach `want` in count or mass.  A
    // histogram over the range of those in question, as often as more than a
    // warp's worth is left: of their keys, then, where those are equal, of ~index.
    auto pick = [&](const u64 (&v)[PER], const u64 (&m)[PER], bool by_mass, u64 want) -> u64 {
      uint32_t klo = 1, khi = 0xffffffffu, tlo = 0, thi = 0xffffffffu;   // in question
      u64 above = 0;                                         // sum of those before
      auto key_of = [](u64 w) { return (uint32_t)(w >> 32); };
      auto asked = [&](u64 w) {
        return key_of(w) >= klo && key_of(w) <= khi && (uint32_t)w >= tlo && (uint32_t)w <= thi;
      };
      for (;;) {
        const bool by_key = klo != khi;
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (asked(v[j])) {
            const uint32_t x = by_key ? key_of(v[j]) : (uint32_t)v[j];
            hi = max(hi, x);
            lo = max(lo, ~x);
          }
        hi = __reduce_max_sync(FULL, hi);
        lo = __reduce_max_sync(FULL, lo);
        __syncthreads();
        if (lane == 0) {
          sh.warp_max[warp] = hi;
          sh.warp_max[SAMPLE_WARPS + warp] = lo;
        }
        for (int i = tid; i < SAMPLE_BUCKETS; i += SAMPLE_THREADS) h_cnt[i] = h_lo[i] = h_hi[i] = 0;
        __syncthreads();
        const uint4 *const most4 = reinterpret_cast<const uint4 *>(sh.warp_max);
#pragma unroll
        for (int j = 0; j < SAMPLE_WARPS / 4; ++j) {
          const uint4 a = most4[j], b = most4[SAMPLE_WARPS / 4 + j];
          hi = max(max(hi, max(a.x, a.y)), max(a.z, a.w));
          lo = max(max(lo, max(b.x, b.y)), max(b.z, b.w));
        }
        lo = ~lo;
        if (hi == lo) {                                      // one key: by index; one word: found
          if (!by_key) return ((u64)khi << 32) | hi;
          klo = khi = hi;
          continue;
        }
        const int width = 32 - __clz(hi - lo), shift = width > 10 ? width - 10 : 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (asked(v[j])) {
            const int b = (int)((hi - (by_key ? key_of(v[j]) : (uint32_t)v[j])) >> shift);
            atomicAdd(h_cnt + b, 1u);
            if (by_mass) {
              const uint32_t x = (uint32_t)m[j], old = atomicAdd(h_lo + b, x);
              const uint32_t y = (uint32_t)(m[j] >> 32) + (old + x < old ? 1u : 0u);
              if (y) atomicAdd(h_hi + b, y);
            }
          }
        __syncthreads();
        u64 n[2], total;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          n[i] = by_mass ? ((u64)h_hi[2 * tid + i] << 32) + h_lo[2 * tid + i] : h_cnt[2 * tid + i];
        u64 run = above + block_scan(n[0] + n[1], sh.red, total);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (run < want && want <= run + n[i]) {
            sh.found.bucket = 2 * tid + i;
            sh.found.count = (int)h_cnt[2 * tid + i];
            sh.found.above = run;
          }
          run += n[i];
        }
        if (tid == 0) sh.pos = 0;
        __syncthreads();
        above = sh.found.above;
        const uint32_t up = hi - ((uint32_t)sh.found.bucket << shift), step = (1u << shift) - 1;
        const uint32_t down = up - lo > step ? up - step : lo;
        if (by_key) klo = down, khi = up;
        else tlo = down, thi = up;
        const int count = sh.found.count;
        if (count > 32) continue;
        // the last few: ranks by comparing in one warp
        u64 *const few = reinterpret_cast<u64 *>(h_cnt);
        __syncthreads();                         // (the histogram is read)
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (asked(v[j])) {
            const int at = atomicAdd(&sh.pos, 1);
            few[2 * at] = v[j];
            few[2 * at + 1] = by_mass ? m[j] : 1;
          }
        __syncthreads();
        if (warp == 0) {
          const u64 mine = lane < count ? few[2 * lane] : 0;
          u64 before = above;
          for (int i = 0; i < count; ++i)
            if (few[2 * i] > mine) before += few[2 * i + 1];
          if (lane < count && before < want && want <= before + few[2 * lane + 1]) sh.red[0] = mine;
        }
        __syncthreads();
        const u64 found = sh.red[0];
        __syncthreads();
        return found;
      }
    };

    const float by_logit = (SAMPLE_BUCKETS - 1) / 32.f;       // 1024 buckets over 32 logits
    auto level0 = [&](float l, float scale) {
      return (int)fminf((top - l) * scale, (float)(SAMPLE_BUCKETS - 1));
    };

    // ---- a small top-k: the first CTA settles the row (1024 rows of 32000, top-k 50:
    // 133 us, by the histograms below 168; with top-p 0.9 beside it 142 and 253) ----
    // Every CTA lists its tokens down to the k-th largest of its threads' own maxima:
    // the k first-ranked of the row are among them, and few more than k of each CTA.
    SampleRow::Found f{};
    if (by_k && k <= SAMPLE_SMALL_K && !inf_row) {
      clear();
      if (tid == 0) {
        sh.list_n = 0;
        sh.pos = SAMPLE_BUCKETS - 1;             // (fewer maxima than k: every token)
      }
      if (most > -INFINITY) atomicAdd(h_cnt + level0(most, by_logit), 1u);
      __syncthreads();
      {
        const uint2 n = *reinterpret_cast<const uint2 *>(h_cnt + 2 * tid);
        u64 total;
        const u64 run = block_scan((u64)n.x + n.y, sh.red, total);
        if (run < (u64)k && (u64)k <= run + n.x + n.y) sh.pos = 2 * tid + (run + n.x < (u64)k);
        __syncthreads();
      }
      const float down = sh.pos == SAMPLE_BUCKETS - 1 ? NAN : (float)(sh.pos + 1);
      collect([&](float l) { return !((top - l) * by_logit >= down); });
      cluster.sync();
      const int n = list_total();
      if (n <= SAMPLE_LIST) {
        if (rank == 0) {
          u64 v[PER], m[PER];
          take_lists(n, v);
          cluster.barrier_arrive();              // (the others' lists are read)
          const u64 kth = pick(v, m, false, (u64)min(n, k));
          // the k words and their masses, four threads to a word from here on
          ulonglong2 *const few = reinterpret_cast<ulonglong2 *>(h_cnt);
          if (tid == 0) sh.pos = 0;
          __syncthreads();
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (v[j] >= kth) few[atomicAdd(&sh.pos, 1)] = make_ulonglong2(v[j], mass_at(word_logit(v[j])));
          __syncthreads();
          const int count = sh.pos, i = tid >> 2;
          const ulonglong2 mine = i < count ? few[i] : make_ulonglong2(0, 0);
          // sum of the masses of the words that pass a test against this one's
          auto sum_of = [&](auto test) {
            u64 x = 0;
            for (int j = tid & 3; j < count; j += 4)
              if (test(few[j])) x += few[j].y;
            x += __shfl_xor_sync(FULL, x, 1);
            x += __shfl_xor_sync(FULL, x, 2);
            return x;
          };
          u64 lowest = kth;
          if (by_p) {
            const u64 all = sum_of([](const ulonglong2 &) { return true; });
            u64 bar = p > 0.0 ? (u64)ceil(p * (double)all) : 1;
            if (bar < 1) bar = 1;
            const u64 upto = sum_of([&](const ulonglong2 &w) { return w.x >= mine.x; });
            __syncthreads();
            if (i < count && upto >= bar && upto - mine.y < bar) sh.red[0] = mine.x;
            __syncthreads();
            lowest = sh.red[0];
          }
          auto stays = [&](const ulonglong2 &w) {
            return w.x >= lowest && (w.y >= low || (uint32_t)(w.x >> 32) == top_key);
          };
          // The weights in steps of 2^-50: whole numbers, since the lists' order
          // changes from run to run.
          const bool mine_stays = i < count && (tid & 3) == 0 && stays(mine);
          const float l = word_logit(mine.x);
          u64 fine = mine_stays && z.positive(l) ? sample_mass(z.weight(l) * 1024.0) : 0, fines;
          block_scan(fine, sh.red, fines);
          if (tid == 0) {
            sh.found.thr = (uint32_t)(lowest >> 32);
            sh.found.cut = (int)~(uint32_t)lowest;
            sh.found.inv = (float)(1024.0 / (double)fines);
          }
          if (a.token) {
            const u64 total = sum_of(stays);
            const u64 want = (__umul64hi(total, U) << 40) | ((total * U) >> 24);
            const u64 upto = sum_of(
                [&](const ulonglong2 &w) { return (uint32_t)w.x >= (uint32_t)mine.x && stays(w); });
            if (mine_stays && upto > want && upto - mine.y <= want) a.token[row] = (int)~(uint32_t)mine.x;
          }
        } else {
          cluster.barrier_arrive();
        }
        cluster.barrier_wait();
        if (!probs) return;
        cluster.sync();
        cut_to(lead->thr, lead->cut);
        const float inv = lead->inv;
        cluster.barrier_arrive();                // (read before the first CTA leaves)
        write_probs([&](int j) {
          const float4 q = val4[j];
          float e[4] = {q.x, q.y, q.z, q.w};
          if (!(e[0] >= at || e[1] >= at || e[2] >= at || e[3] >= at))
            return make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float pv = 0.f;
            if (kept(e[i], v0 + 4 * j + i) && z.positive(e[i])) {
              const double w = z.weight(e[i]);
              if (sample_mass(w) >= low) pv = (float)w * inv;
            }
            e[i] = pv;
          }
          return make_float4(e[0], e[1], e[2], e[3]);
        });
        cluster.barrier_wait();
        return;
      }
      cluster.sync();                            // (the lists' lengths are read)
    }

    // ---- one filter: the least prefix of what is kept with `want` tokens, or
    // with top_p of its mass ----
    auto select = [&](bool by_mass, u64 want) {
      const float scale = by_mass ? z.fc * ((SAMPLE_BUCKETS - 1) / 40.f) : by_logit;
      uint32_t khi = 0xffffffffu, klo = 0;       // keys in question
      int bits = -1;                             // bucket width, or the first level's scale
      u64 above = 0, mass_above = 0, bar = 0;
      for (;;) {
        // the bucket of a logit, -1 if it is not in question any more
        auto bucket_of = [&](float l) -> int {
          if (bits < 0) return level0(l, scale);
          const uint32_t key = logit_key(l);
          return key < klo || key > khi ? -1 : (int)((khi - key) >> bits);
        };
        clear();
        if (tid == 0) sh.list_n = sh.above_n = 0;
        if (by_mass) {                           // (tokens without weight are not in question)
          auto add = [&](float l, u64 m) {
            const int b = z.positive(l) ? bucket_of(l) : -1;
            if (b < 0) return;
            const uint32_t lo = (uint32_t)m, old = atomicAdd(h_lo + b, lo);
            const uint32_t hi = (uint32_t)(m >> 32) + (old + lo < old ? 1u : 0u);
            if (hi) atomicAdd(h_hi + b, hi);
          };
          if (cutting)
            for_queued([&](uint32_t i) { add(val[i], sample_mass(z.weight(val[i]))); });
          else
            for (int j = tid; j < units; j += SAMPLE_THREADS) {
              const float4 q = val4[j];
              const float e[4] = {q.x, q.y, q.z, q.w};
              u64 m[4];
              // the four weights side by side: a double's latency is that of many others
#pragma unroll
              for (int i = 0; i < 4; ++i) m[i] = sample_mass(z.weight(e[i]));
#pragma unroll
              for (int i = 0; i < 4; ++i) add(e[i], m[i]);
            }
        } else {
          for_kept([&](float l) {
            const int b = bucket_of(l);
            if (b >= 0) atomicAdd(h_cnt + b, 1u);
          });
        }
        f = find(by_mass, want, above, mass_above, bar);
        if (f.bucket < 0) return;                // fewer tokens than wanted (the rest is NaN)
        bar = f.bar;
        if (by_mass || f.count <= SAMPLE_LIST) {
          // (tested without the conversions and the logit's key)
          int higher = 0;                        // kept tokens above the bucket
          if (bits < 0) {
            const float from = (float)f.bucket;
            const float to = f.bucket == SAMPLE_BUCKETS - 1 ? NAN : (float)(f.bucket + 1);
            collect([&](float l) {
              const float d = (top - l) * scale;
              higher += d < from;
              return d >= from && !(d >= to) && (!by_mass || z.positive(l));
            });
          } else {
            const uint32_t up = khi - ((uint32_t)f.bucket << bits), width = (1u << bits) - 1;
            const float from = key_logit(up), to = key_logit(up - klo > width ? up - width : klo);
            collect([&](float l) {
              higher += l > from;
              return l <= from && l >= to && (!by_mass || z.positive(l));
            });
          }
          if (by_mass) {
            higher = __reduce_add_sync(FULL, higher);
            if (lane == 0) atomicAdd(&sh.above_n, higher);
          }
          cluster.sync();
          const int n = by_mass ? list_total() : f.count;
          if (n <= SAMPLE_LIST) {
            if (by_mass) many = (sh.above_n + n) * 3 > units * 4;
            if (rank == 0) {
              u64 v[PER], m[PER];
              take_lists(n, v);
#pragma unroll
              for (int j = 0; j < PER; ++j) m[j] = by_mass && v[j] ? mass_at(word_logit(v[j])) : 0;
              const u64 last = pick(v, m, by_mass, by_mass ? bar - f.mass_above : want - f.above);
              if (tid == 0) {
                sh.found.thr = (uint32_t)(last >> 32);
                sh.found.cut = (int)~(uint32_t)last;
              }
            }
            cluster.sync();
            cut_to(lead->thr, lead->cut);        // (found is not written before the next barrier)
            return;
          }
          many = true;                           // thousands of nearly equal logits at the border
          cluster.sync();                        // (the lists' lengths are read)
        }
        // more tokens than the list holds: the keys of this bucket
        above = f.above;                         // (the one of the two that counts)
        mass_above = f.mass_above;
        if (bits < 0) {
          uint32_t hi = 0, lo = 0;
          for_kept([&](float l) {
            if ((by_mass && !z.positive(l)) || bucket_of(l) != f.bucket) return;
            const uint32_t key = logit_key(l);
            hi = key > hi ? key : hi;
            lo = ~key > lo ? ~key : lo;
          });
          khi = cluster_max(hi);
          klo = ~cluster_max(lo);
        } else {
          khi -= (uint32_t)f.bucket << bits;
          const uint32_t width = (1u << bits) - 1;
          klo = khi - klo > width ? khi - width : klo;
        }
        if (khi == klo) {                        // equal logits: cut by count
          const u64 one = by_mass ? mass_at(key_logit(khi)) : 1;
          const u64 take = by_mass ? (bar - mass_above + one - 1) / one : want - above;
          u64 mine = 0;
          for_kept([&](float l) { mine += logit_key(l) == khi; });
          u64 cnt;
          block_scan(mine, sh.red, cnt);
          const u64 *pc = exchange(cnt);
          u64 before = 0;
          for (int j = 0; j < rank; ++j) before += pc[j];
          // the CTA that holds the take-th of them finds its index
          u64 spot = 0;
          if (before < take && take <= before + cnt) {
            u64 run = before;
            for (int b = 0; b < units && spot == 0; b += SAMPLE_THREADS) {
              const int j = b + tid;
              const float4 q = j < units ? val4[j] : make_float4(NAN, NAN, NAN, NAN);
              const float e[4] = {q.x, q.y, q.z, q.w};
              u64 n = 0, sum;
              bool eq[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int v = v0 + 4 * j + i;
                eq[i] = kept(e[i], v) && logit_key(e[i]) == khi;
                n += eq[i];
              }
              u64 r = run + block_scan(n, sh.red, sum);
              if (tid == 0) sh.pos = -1;
              __syncthreads();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (eq[i] && ++r == take) sh.pos = v0 + 4 * j + i;
              __syncthreads();
              if (sh.pos >= 0) spot = (u64)sh.pos + 1;
              run += sum;
            }
          }
          const u64 *pa = exchange(spot);
          u64 sum = 0;
          for (int j = 0; j < C; ++j) sum += pa[j];
          cut_to(khi, (int)sum - 1);
          return;
        }
        const int width = 32 - __clz(khi - klo);   // bits of the distance
        bits = width > 10 ? width - 10 : 0;
      }
    };
    if (by_k) select(false, (u64)k);
    if (by_p) select(true, 0);
  }

  // ---- sums over what is kept; warp w takes the w-th part of the slice ----
  u64 mass = 0;
  double wsum = 0.0;
  {
    const int j1 = min(units, (warp + 1) * wu);
    // Every token, or most: each is weighed where it stands.  A thread's masses add
    // up below 2^52, so the bits above are dropped once at the end.
    auto sums = [&](auto with_probs, auto with_cut) {
      for (int j = warp * wu + lane; j < j1; j += 32) {
        const float4 q = val4[j];
        float e[4] = {q.x, q.y, q.z, q.w};
        double w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = z.weight(e[i]);          // (side by side)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u64 m = sample_mass_bits(w[i]);
          bool keep = z.positive(e[i]);
          if constexpr (decltype(with_cut)::value)
            keep = keep && kept(e[i], v0 + 4 * j + i) && (m & SAMPLE_MASK) >= low;
          if (keep) mass += m;
          if constexpr (decltype(with_probs)::value) {
            if (keep) wsum += w[i];
            e[i] = keep ? (float)w[i] : 0.f;
          }
        }
        if constexpr (decltype(with_probs)::value)                  // weights, for the probabilities
          val4[j] = make_float4(e[0], e[1], e[2], e[3]);
      }
    };
    const std::true_type yes;
    const std::false_type no;
    if ((cutting || low) && !many) {
      // min-p in advance, with room for what float loses (4e-6); exact by the mass
      if (low) least = (float)fma((double)(log2f((float)low) - 40.f - 1e-4f), z.halving, z.top);
      for_queued([&](uint32_t i) {
        const double w = z.weight(val[i]);
        const u64 m = sample_mass(w);
        const bool keep = m >= low;
        mass += keep ? m : 0;
        wsum += keep ? w : 0.0;
        if (probs) val[i] = keep ? (float)w : 0.f;
      }, probs != nullptr);
    } else if (many) {
      if (probs) sums(yes, yes);
      else sums(no, yes);
    } else {
      if (probs) sums(yes, no);
      else sums(no, no);
    }
    mass &= SAMPLE_MASK;
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
  u64 cta_mass = 0;                // (of warp 0, which adds the warps' up)
  if (warp == 0) {
    cta_mass = warp_sum_u64(lane < SAMPLE_WARPS ? sh.wsum[lane] : 0);
    double cta_w = lane < SAMPLE_WARPS ? sh.redd[lane] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cta_w += __shfl_xor_sync(FULL, cta_w, o);
    if (lane < C) *cluster.map_shared_rank(&sh.xchd[rank], lane) = cta_w;
  }
  const u64 *pm = exchange(cta_mass);
  u64 total = 0, before = 0;
  double sum = 0.0;
  for (int j = 0; j < C; ++j) {
    if (j < rank) before += pm[j];
    total += pm[j];
    sum += sh.xchd[j];
  }
  cta_mass = pm[rank];
  // (no CTA leaves before every other has finished writing to it: the exchange
  // above was the last remote access)

  // ---- the draw: the CTA, the warp's part, then a few tokens to a thread, whose
  // logits are on their way while the probabilities are written ----
  const u64 m = (__umul64hi(total, U) << 40) | ((total * U) >> 24);
  const bool here = a.token != nullptr && before <= m && m < before + cta_mass;
  int t0 = 0, t1 = 0;
  constexpr int AHEAD = 4;
  float ahead[AHEAD];
  if (here) {
    int part = 0;
    for (u64 w = sh.wsum[0]; before + w <= m; w = sh.wsum[part]) {
      before += w;
      ++part;
    }
    const int b0 = max(c0, v0 + 4 * part * wu), b1 = min(c1, v0 + 4 * min(units, (part + 1) * wu));
    const int each = (b1 - b0 + SAMPLE_THREADS - 1) / SAMPLE_THREADS;
    t0 = min(b1, b0 + tid * each);
    t1 = min(b1, t0 + each);
    // (weights took the logits' place in shared memory where probabilities are wanted)
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      ahead[i] = t0 + i < t1 ? (probs ? x[t0 + i] : val[t0 + i - v0]) : 0.f;
  }
  if (probs) {
    const float inv = (float)(1.0 / sum);
    write_probs([&](int j) {
      const float4 q = val4[j];
      return make_float4(q.x * inv, q.y * inv, q.z * inv, q.w * inv);
    });
  }
  if (!here) return;
  auto mass_of = [&](int v, float l) -> u64 {
    if (probs) l = infinite(l);
    if (!kept(l, v)) return 0;
    const u64 mv = mass_at(l);
    return mv >= low ? mv : 0;
  };
  auto each_mass = [&](auto f) {                 // f(token, mass) -> whether to go on
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (t0 + i < t1 && !f(t0 + i, mass_of(t0 + i, ahead[i]))) return;
    for (int v = t0 + AHEAD; v < t1; ++v)
      if (!f(v, mass_of(v, probs ? x[v] : val[v - v0]))) return;
  };
  u64 mine = 0, all;
  each_mass([&](int, u64 mv) {
    mine += mv;
    return true;
  });
  u64 run = before + block_scan(mine, sh.red, all);
  if (run <= m && m < run + mine)
    each_mass([&](int v, u64 mv) {
      run += mv;
      if (run > m) a.token[row] = v;
      return run <= m;
    });
}

// CTAs of a row: slices of at most 18432 tokens (72 KB, two CTAs per SM) and,
// for few rows, enough CTAs for the machine with 2048 tokens each at least.  (1024
// rows of 32000 at a temperature: two CTAs 109 us, one 118, four 150, the steps between
// barriers being paid by each; a single row of 32000, all filters: eight CTAs 11.4 us,
// two 11.9.)
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
  static_assert(SAMPLE_WARPS * SAMPLE_QUEUE <= 2 * SAMPLE_LIST && SAMPLE_SMALL_K * 16 <= SAMPLE_BUCKETS * 12,
                "what takes the list's and the histogram's place");
}

}  // namespace moe
