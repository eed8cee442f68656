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
#pragma once
#include "common.cuh"

namespace moe {

constexpr int SAMPLE_THREADS = 1024;
constexpr int SAMPLE_MAX_V = 1 << 20;
constexpr double SAMPLE_ONE = 1099511627776.0;     // 2^40

struct SampleArgs {
  const float *logits;           // [S*K, V]
  int K, V;
  const float *temperature;      // [S] or null
  const int32_t *top_k;
  const float *top_p, *min_p;
  const float *u;                // [S*K] or null
  int32_t *token;                // [S*K] or null
  float *probs;                  // [S*K, V] or null
};

// order-preserving key of a logit; -0 counts as 0, NaN as -infinity
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (!(x == x)) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

__device__ __forceinline__ double sample_weight(float x, float top, double inv_t) {
  if (x == top) return 1.0;
  return exp(((double)x - (double)top) * inv_t);
}

template <typename T>
__device__ __forceinline__ T block_sum(T v, T *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T t = 0;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += red[i];
  return t;
}

// One CTA per row.
__global__ void __launch_bounds__(SAMPLE_THREADS) sample_kernel(const SampleArgs a) {
  pdl_wait();
  pdl_trigger();
  typedef unsigned long long u64;
  __shared__ u64 red[32];
  __shared__ double redd[32];
  __shared__ float rv[32];
  __shared__ int ri[32];
  const int row = blockIdx.x, s = row / a.K, V = a.V;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, w = tid >> 5, nw = nt >> 5;
  const float *x = a.logits + (size_t)row * V;
  float *probs = a.probs ? a.probs + (size_t)row * V : nullptr;

  float bv = -INFINITY;
  int bi = -1;
  for (int v = tid; v < V; v += nt)
    if (x[v] > bv) { bv = x[v]; bi = v; }
  warp_argmax(bv, bi);
  if (lane == 0) { rv[w] = bv; ri[w] = bi; }
  __syncthreads();
  bv = rv[0]; bi = ri[0];
  for (int j = 1; j < nw; ++j)
    if (better(rv[j], ri[j], bv, bi)) { bv = rv[j]; bi = ri[j]; }
  if (bi < 0) {                               // nothing but -infinity (or NaN)
    if (tid == 0) {
      raise_status(MOE_DEV_NO_MASS);
      if (a.token) a.token[row] = -1;
    }
    if (probs) for (int v = tid; v < V; v += nt) probs[v] = 0.f;
    return;
  }
  const float top = bv;
  const double T = a.temperature ? (double)a.temperature[s] : 1.0;
  if (!(T > 0.0)) {
    if (tid == 0 && a.token) a.token[row] = bi;
    if (probs) for (int v = tid; v < V; v += nt) probs[v] = v == bi ? 1.f : 0.f;
    return;
  }
  const double inv_t = 1.0 / T;
  auto mass_of = [&](float l) { return (u64)(sample_weight(l, top, inv_t) * SAMPLE_ONE); };

  uint32_t thr = 0;                           // kept: key > thr, or equal with rank < ties
  u64 ties = ~0ull;
  const int k = a.top_k ? a.top_k[s] : 0;
  if (k > 0 && k < V) {
    for (int b = 31; b >= 0; --b) {
      const uint32_t cand = thr | (1u << b);
      u64 c = 0;
      for (int v = tid; v < V; v += nt) c += logit_key(x[v]) >= cand;
      if (block_sum(c, red) >= (u64)k) thr = cand;
    }
    u64 c = 0;
    for (int v = tid; v < V; v += nt) c += logit_key(x[v]) > thr;
    ties = k - block_sum(c, red);
  }
  const double p = a.top_p ? (double)a.top_p[s] : 1.0;
  if (p < 1.0) {
    u64 m = 0;
    for (int v = tid; v < V; v += nt) {
      const uint32_t key = logit_key(x[v]);
      if (key > thr || ties == ~0ull) m += mass_of(key_logit(key));
    }
    u64 total = block_sum(m, red);
    if (ties != ~0ull) total += ties * mass_of(key_logit(thr));
    u64 bar = p > 0.0 ? (u64)ceil(p * (double)total) : 1;
    if (bar < 1) bar = 1;
    uint32_t pt = 0;
    for (int b = 31; b >= 0; --b) {
      const uint32_t cand = pt | (1u << b);
      if (ties != ~0ull && cand <= thr) { pt = cand; continue; }
      u64 m = 0;
      for (int v = tid; v < V; v += nt) {
        const uint32_t key = logit_key(x[v]);
        if (key >= cand) m += mass_of(key_logit(key));
      }
      if (block_sum(m, red) >= bar) pt = cand;
    }
    m = 0;
    for (int v = tid; v < V; v += nt) {
      const uint32_t key = logit_key(x[v]);
      if (key > pt) m += mass_of(key_logit(key));
    }
    m = block_sum(m, red);
    const u64 one = mass_of(key_logit(pt));
    const u64 t = one ? (bar - m + one - 1) / one : 1;
    if (pt > thr || ties == ~0ull) { thr = pt; ties = t; }
    else ties = min(ties, t);
  }
  // the last index kept among the tokens equal to the threshold
  int cut = V;
  if (ties != ~0ull) {
    u64 run = 0;
    for (int b = 0; b < V && cut == V; b += nt) {
      const int v = b + tid;
      const bool eq = v < V && logit_key(x[v]) == thr;
      const unsigned bal = __ballot_sync(FULL, eq);
      __syncthreads();
      if (lane == 0) ri[w] = __popc(bal);
      if (tid == 0) red[0] = ~0ull;
      __syncthreads();
      u64 before = run, all = run;
      for (int j = 0; j < nw; ++j) { if (j < w) before += ri[j]; all += ri[j]; }
      before += __popc(bal & lanemask_lt());
      if (eq && before + 1 == ties) red[0] = (u64)v;
      __syncthreads();
      if (red[0] != ~0ull) cut = (int)red[0];
      run = all;
    }
  }
  const float mp = a.min_p ? a.min_p[s] : 0.f;
  const u64 low = mp > 0.f ? (u64)((double)fminf(mp, 1.f) * SAMPLE_ONE) : 0;
  auto kept = [&](float l, int v) -> double {       // the weight if kept, else -1
    const uint32_t key = logit_key(l);
    if (key < thr || (key == thr && v > cut)) return -1.0;
    const double wt = sample_weight(key_logit(key), top, inv_t);
    return (u64)(wt * SAMPLE_ONE) >= low ? wt : -1.0;
  };
  const int chunk = (V + nw - 1) / nw, c0 = min(V, w * chunk), c1 = min(V, c0 + chunk);
  u64 mine = 0;
  double ws = 0.0;
  for (int v = c0 + lane; v < c1; v += 32) {
    const double wt = kept(x[v], v);
    if (wt >= 0.0) { ws += wt; mine += (u64)(wt * SAMPLE_ONE); }
  }
  if (probs) {
    const double inv = 1.0 / block_sum(ws, redd);
    for (int v = tid; v < V; v += nt) {
      const double wt = kept(x[v], v);
      probs[v] = wt >= 0.0 ? (float)(wt * inv) : 0.f;
    }
  }
  if (!a.token) return;
  const u64 total = block_sum(mine, red);
  const u64 U = (u64)((double)a.u[row] * 16777216.0);
  const u64 lo = total * U, hi = __umul64hi(total, U);
  const u64 m = (hi << 40) | (lo >> 24);
  u64 run = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(FULL, mine, o);
  for (int j = 0; j < w; ++j) run += red[j];
  if (!(run <= m && m < run + mine)) return;
  for (int b = c0; b < c1; b += 32) {
    const int v = b + lane;
    const double wt = v < c1 ? kept(x[v], v) : -1.0;
    const u64 wv = wt >= 0.0 ? (u64)(wt * SAMPLE_ONE) : 0;
    u64 c = wv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(FULL, c, o);
      if (lane >= o) c += y;
    }
    const bool hit = wv > 0 && run + c > m && run + c - wv <= m;
    if (hit) a.token[row] = v;
    if (__any_sync(FULL, hit)) return;
    run += __shfl_sync(FULL, c, 31);
  }
}

}  // namespace moe
