// attention.cuh -- attention of a drafted block over a paged key-value cache.
//
//   out = sum_j softmax_j(scale q.k_j) v_j,  keys j <= position, inside the window
//
// The N tokens x (Hq/Hkv) query heads that share a key/value head are the rows
// of one matrix: S = Q K^T and O += P V run on tcgen05 with 128 rows (rows past
// the last are left as they are, and reach no output), keys in tiles of KT = 128
// (64 for D = 256, whose queries take twice the shared memory), S, P and O in
// tensor memory.  At these row counts the cache's bytes bound the call (2 flops
// per row and byte against ~250 flops per byte of the machine), so a padded
// 128-row MMA costs nothing: a 64 KB tile (128 keys, D = 128) takes the tensor
// pipe ~1000 cycles and an SM's share of HBM ~2700.  More rows than 128 are several
// row blocks, each of which reads the cache again (16 sequences of up to 30000 keys,
// 64/8 heads of 128: 16 tokens, 128 rows 194 us; 17 tokens, 136 rows 336 us; 33
// tokens, 264 rows 507 us).
//
// Softmax in one pass: every row keeps a maximum m and a sum l in float; O is
// rescaled only when a tile's maximum exceeds m by 8 (in powers of two), so
// weights reach 2^8 at most and the accumulator in tensor memory is rarely
// touched.  The weights go to the tensor cores as bf16, which its product with
// the bf16 values asks for (half a step, 2^-8 of a weight, like the keys and
// values); l sums them before rounding.  Values that are not finite would spoil
// the rows that do not see them (0 x NaN): see attn_row_alone.
//
// Split over the length: the tiles of all (sequence, key/value head, row block)
// items form one line, cut into G equal pieces, one per CTA (one CTA per SM),
// so uneven lengths and single long sequences fill the GPU alike.  An item that
// lies in one piece is written out directly; of the others each piece leaves
// its unnormalised O, m and l in the workspace and attn_join_kernel adds them
// in the order of the pieces (the same bits on every run).
//
// Warps: a warpgroup of softmax threads (a thread per row, tensor-memory lane =
// row; they also bring the queries), the MMA issuer, and the producers of the K
// and the V tiles of a shared ring in the 128-byte swizzle: by TMA page by page
// where pages are multiples of 8 rows, or row by row through cp.async, where rows
// outside the sequence or on a bad page are zero-filled and masked by a bit per
// key.  (By rows alone: 14 sequences of up to 30000 keys 241 us, by TMA 158.  With 16
// sequences pages of 16 to 256 rows take 172 to 181 us, of 8 226, of 30 and 100, by
// rows, 281 and 273.)
// Where pages do not fill a tile (24, 40, 48 ..) the tile is the whole pages that fit,
// and every score of it is tested for its key (pages of 24 179 us, of 32 174).  The
// ring's order is that of use, K0 K1 V0 K2 V1 .., each tile scored two ahead of
// its product with V.  For D = 64 a tile's bytes arrive in half the time, but its
// weights take as long: two warpgroups take every other tile, each with an O of
// its own (64 sequences of 5000 keys, 16 heads, 8 tokens: 278 us, with one 289).
//
// Few rows would leave most lanes, and so most softmax warps, without work: up
// to 32 rows (64) the queries stand in the 128 MMA rows four (two) times, lane
// group g weighs the g-th quarter (half) of each tile's keys, its other weights
// stay zero, and the groups' O, m and l are joined at the segment's end.  (64
// sequences, 16 heads of 64, window: 36 us, without groups 51, with two 41; a
// sequence of 131000 keys, 8 rows to a head: 58 us, without 62.)
//
// Measured (floor: the visible cache once at a plain copy's rate): 14 sequences of
// up to 30000 keys, 64/8 heads of 128, 8 tokens 155-158 us (132); 64 of up to 9000,
// 32/4 heads, 16 tokens 142-145 us (98); one of 131000, 32/4 heads, one token 58 us
// (41); one of 777 keys 14 us (0.5).  What is left: the start of a call (barriers,
// tensor memory, the pieces' places, the first tiles) 4-5 us, the join 4-6 us, the
// output of an item 1.3 us, in which its CTA's loads run on into the ring only.
// Every wait is bounded (MOE_DEV_TIMEOUT), as in the expert FFN.
#pragma once
#include "common.cuh"
#include "ffn_tc.cuh"
#include "kv_append.cuh"

namespace moe {

constexpr int ATTN_MAX_CTAS = 148;
constexpr int ATTN_ROWS = 128;
constexpr int ATTN_MASKS = 8;

struct AttnArgs {
  const uint16_t *q;                   // [S, N, Hq, D]
  int S, N, Hq, Hkv;
  const uint16_t *k_cache, *v_cache;   // [num_pages, Hkv, page_size, D]
  int num_pages, page_size;
  const int32_t *block_table;          // [S, max_pages]
  int max_pages;
  const int32_t *kv_len;               // [S]
  float scale_log2;                    // scale * log2(e), > 0
  int window;
  uint16_t *out;                       // [S, N, Hq, D]
  // workspace: unnormalised O [2G][rows_cap][D/4] float4, (m, l) [2G][rows_cap],
  // one AttnSplit per piece
  // keys of a tile, and what its first key is a multiple of: whole pages where
  // the pages go by TMA (use_tma), else KT and 1
  int tile_keys, align, use_tma;
  float4 *part_o;
  float2 *part_ml;
  struct AttnSplit *split;
  int rows_cap, rows, row_blocks;      // rows = N * Hq / Hkv
};

// An item cut by pieces: first piece and how many pieces it spans (0: none
// whose first cut is this piece's start).
struct AttnSplit {
  int s, kvh, rb, first, count;
};

template <int D, int KS>
struct AttnCfg {
  static constexpr int KT = D == 256 ? 64 : 128;      // keys per tile
  static constexpr int WGS = D == 64 ? 2 : 1;         // softmax warpgroups, a tile each in turn
  static constexpr int NC = KT / KS;                  // keys of a tile to one softmax thread
  static constexpr int RG = ATTN_ROWS / KS;           // rows of a lane group
  static constexpr int kSoftmax = 128 * WGS;          // softmax threads
  static constexpr int kThreads = kSoftmax + 96;      // and the MMA, K and V warps
  static constexpr int kSlot = KT * D * 2;            // one K or V tile
  static constexpr int kQ = ATTN_ROWS * D * 2;
  // 32 dims of O for the groups' sum: 8 columns of a float4 per softmax thread,
  // one apart more so that the quads of a row lie in different banks
  static constexpr int kPitch = kSoftmax + 1;
  static constexpr int kScratch = 8 * kPitch * 16;
  static constexpr int kMisc = 2048;
  static constexpr int kSlots = (232448 - kQ - kScratch - kMisc) / kSlot;
  static constexpr int kSmem = kQ + kSlots * kSlot + kScratch + kMisc;
  // Tensor memory columns: S and P (two bf16 to a column) of two tiles in flight,
  // O of each warpgroup.
  static constexpr uint32_t kS = 0, kP = 2 * KT, kO = 512 - WGS * D;
  static constexpr uint32_t kCols = 512;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kP + KT <= kO, "tensor memory");
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}

// The MMA warp runs its loop as a whole, one elected lane issuing: addresses and
// descriptors then stay in uniform registers (with a single lane in the loop every
// operand was moved there anew, ~50 ns an MMA, which bound the whole kernel).
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A from tensor memory: lane = row, two consecutive K elements to a column
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
// bf16 x bf16 -> float, M = 128; transpose_b: B is N-major in shared memory
constexpr uint32_t idesc_bf16(uint32_t n, uint32_t transpose_b) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (transpose_b << 16) | ((n >> 3) << 17) |
         ((128u >> 4) << 24);
}

__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bounded wait, inline: the softmax threads hold a tile of scores in
// registers, which a call would have to spill.
__device__ __forceinline__ bool attn_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  const uint64_t limit = *(volatile unsigned long long *)&g_wait_limit_ns;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_ns() - t0 >= limit) {
      raise_status(MOE_DEV_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}
// The same for the MMA warp and the producers, which also wait while rows are
// summed anew (attn_row_alone), for as long as their keys take: a beat counts that
// work, and the limit starts again when it has moved.
__device__ __noinline__ bool attn_wait_on(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          const volatile uint32_t *beat) {
  uint64_t t0 = global_ns();
  uint32_t seen = *beat;
  const uint64_t limit = *(volatile unsigned long long *)&g_wait_limit_ns;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_ns() - t0 >= limit) {
      if (*beat == seen) break;
      seen = *beat;
      t0 = global_ns();
    }
  }
  raise_status(MOE_DEV_TIMEOUT);
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool attn_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          const volatile uint32_t *beat) {
  return mbar_try_wait(bar, parity) || attn_wait_on(bar, parity, abort, beat);
}

// 16-byte unit u of row r in a tile of `rows` rows: blocks of 64 dims, swizzled
__device__ __forceinline__ uint32_t attn_place(int u, int r, int rows) {
  return (uint32_t)((u >> 3) * rows * 128 + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// Visible keys of a sequence: [lo, n), in tiles from `start` on; none for a
// slot not in use or (reported) a length past the table's row.
struct AttnSeq {
  int lo, start, n, tiles;
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs &a, int s) {
  const int n = __ldg(a.kv_len + s);
  if (n <= 0) return AttnSeq{0, 0, 0, 0};
  if (n > a.max_pages * a.page_size) {
    raise_status(MOE_DEV_BAD_INDEX);
    return AttnSeq{0, 0, 0, 0};
  }
  const int lo = a.window > 0 ? max(0, n - a.N - a.window + 1) : 0;
  const int start = lo - lo % a.align;
  return AttnSeq{lo, start, n, (n - start + a.tile_keys - 1) / a.tile_keys};
}

__device__ __forceinline__ unsigned long long attn_div(unsigned long long a, unsigned long long b) {
  return ((a | b) >> 32) == 0 ? (uint32_t)a / (uint32_t)b : a / b;
}

// A place in the ring and the parity of its barriers' phase.  K and V tiles share
// the ring in the order K0 K1 V0 K2 V1 K3 .. in which they are used.
template <int SLOTS>
struct AttnRing {
  uint32_t slot, phase;
  __device__ __forceinline__ explicit AttnRing(uint32_t first) : slot(first), phase(0) {}
  __device__ __forceinline__ void advance(uint32_t n) {
    slot += n;
    if (slot >= SLOTS) {
      slot -= SLOTS;
      phase ^= 1;
    }
  }
};

// What an item costs beside its tiles, in tiles (the walk below; 64 sequences of up
// to 9000 keys, 4 heads: 142 us with 3, 156 with 0; a single sequence is the same).
constexpr unsigned ATTN_ITEM_COST = 3;
__device__ __forceinline__ unsigned attn_cost(int tiles) {
  return tiles ? (unsigned)tiles + ATTN_ITEM_COST : 0;
}

// A CTA's piece of the line of tiles, item by item.  Every role walks it alone.
// An item counts ATTN_ITEM_COST tiles more than it has: what its start and end
// (queries, first tiles, O out) cost a CTA, so that CTAs with many short items
// end with the others.
struct AttnWalk {
  unsigned long long base, pos, end;   // first tile of sequence s, next tile, end of the piece
  AttnSeq q;
  int s;
  // the segment: tiles [t0, t1) of an item of q.tiles tiles that starts at item_at
  int kvh, rb, t0, t1;
  unsigned long long item_at;

  __device__ __forceinline__ bool next(const AttnArgs &a, unsigned units) {
    for (;;) {
      if (pos >= end) return false;
      while (pos >= base + (unsigned long long)attn_cost(q.tiles) * units) {
        base += (unsigned long long)attn_cost(q.tiles) * units;
        q = attn_seq(a, ++s);
      }
      const unsigned cost = attn_cost(q.tiles);
      const unsigned long long at = pos - base;
      const unsigned item = (unsigned)attn_div(at, cost);
      t0 = (int)(at - (unsigned long long)item * cost);
      t1 = (int)min((unsigned long long)q.tiles, t0 + (end - pos));
      kvh = (int)(item / (unsigned)a.row_blocks);
      rb = (int)(item - (unsigned)kvh * (unsigned)a.row_blocks);
      item_at = base + (unsigned long long)item * cost;
      const bool some = t0 < q.tiles;                  // (else in the item's extra cost)
      pos = t1 < q.tiles ? pos + (t1 - t0) : item_at + cost;
      if (some) return true;
    }
  }
};

// the bits [a, b) of a word whose bit 0 is key 32 w
__device__ __forceinline__ uint32_t bit_range(int a, int b, int w) {
  a = max(0, min(32, a - 32 * w));
  b = max(0, min(32, b - 32 * w));
  const uint32_t below_b = b == 32 ? 0xffffffffu : (1u << b) - 1u;
  const uint32_t below_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
  return below_b & ~below_a;
}

// true iff `v` holds on every softmax thread (named barrier 1), so that they
// decide together to stay or leave
template <int THREADS>
__device__ __forceinline__ bool softmax_all(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"((uint32_t)v), "n"(THREADS) : "memory");
  return r != 0;
}
template <int THREADS>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// One row's sum over the keys [k0, k1) of its sequence, for rows in whose product
// with V some key of a segment weighs 0 though not all values are finite: 0 x NaN
// or infinity would be NaN.
// A warp: lanes take a key each for the scores, then D/32 dims each for the sum.
// Every ATTN_BEAT keys of its rows (`done` so far, returned) it counts `beat` up: a
// segment may have more keys than fit the limit of the waits beside it (see attn_wait).
constexpr int ATTN_BEAT = 32768;
template <int D>
__device__ __noinline__ int attn_row_alone(const AttnArgs &a, int s, int tok, int head, int k0,
                                            int k1, float base, float f, uint16_t *out16,
                                            float *out32, int done, uint32_t *beat) {
  constexpr int W = D / 64;                              // words of two dims per lane
  const int lane = threadIdx.x & 31, kvh = head / (a.Hq / a.Hkv);
  const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (((size_t)s * a.N + tok) * a.Hq + head) * D);
  float o[2 * W];
#pragma unroll
  for (int e = 0; e < 2 * W; ++e) o[e] = 0.f;
  for (int b = k0; b < k1; b += 32) {
    done += 32;
    if (lane == 0 && done % ATTN_BEAT == 0) atomicAdd(beat, 1u);
    const int key = b + lane;
    long long at = -1;                                   // this lane's row of the cache
    float p = 0.f;
    if (key < k1) {
      const int lp = key / a.page_size;
      const int id = __ldg(a.block_table + (size_t)s * a.max_pages + lp);
      if (id >= 0 && id < a.num_pages)
        at = ((long long)id * a.Hkv + kvh) * a.page_size + (key - lp * a.page_size);
    }
    if (at >= 0) {
      const uint4 *k = reinterpret_cast<const uint4 *>(a.k_cache + at * D);
      float z = 0.f;
#pragma unroll 4
      for (int u = 0; u < D / 8; ++u) {
        float x[8], y[8];
        unpack8(__ldg(q + u), x);
        unpack8(__ldg(k + u), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) z = fmaf(x[e], y[e], z);
      }
      p = exp2_approx(fmaf(z, a.scale_log2, -base));
    }
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(FULL, p, j);
      const long long row = __shfl_sync(FULL, at, j);
      const uint32_t *v = reinterpret_cast<const uint32_t *>(a.v_cache + row * D) + lane * W;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const uint32_t x = row >= 0 ? __ldg(v + e) : 0u;
        o[2 * e] = fmaf(pj, bf16_lo(x), o[2 * e]);
        o[2 * e + 1] = fmaf(pj, bf16_hi(x), o[2 * e + 1]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < W; ++e) {
    if (out16 != nullptr)
      reinterpret_cast<uint32_t *>(out16)[lane * W + e] = pack_bf16(o[2 * e] * f, o[2 * e + 1] * f);
    else
      reinterpret_cast<float2 *>(out32)[lane * W + e] = make_float2(o[2 * e], o[2 * e + 1]);
  }
  return done;
}

template <int D, int KS>
__global__ void __launch_bounds__(AttnCfg<D, KS>::kThreads, 1)
attn_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
            const __grid_constant__ AttnArgs a) {
  typedef AttnCfg<D, KS> C;
  constexpr int KT = C::KT, WGS = C::WGS, THREADS = C::kThreads;
  constexpr int MMA_WARP = 4 * WGS, K_WARP = MMA_WARP + 1;
  typedef unsigned long long u64;
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  uint8_t *const s_q = attn_smem;
  uint8_t *const s_ring = attn_smem + C::kQ;
  float4 *const scratch = reinterpret_cast<float4 *>(s_ring + C::kSlots * C::kSlot);
  uint8_t *const misc = s_ring + C::kSlots * C::kSlot + C::kScratch;
  uint32_t *const masks = reinterpret_cast<uint32_t *>(misc);                  // [8][4]
  int *const row_at = reinterpret_cast<int *>(masks + ATTN_MASKS * 4);         // [128]
  uint64_t *const full = reinterpret_cast<uint64_t *>(row_at + ATTN_ROWS);     // [kSlots]
  uint64_t *const empty = full + C::kSlots;                                    // [kSlots]
  uint64_t *const s_full = empty + C::kSlots;                                  // [2] S written
  uint64_t *const s_free = s_full + 2;                                         // [2] S read
  uint64_t *const p_full = s_free + 2;                                         // [2] P written
  uint64_t *const pv_done = p_full + 2;                                        // [2] P read, O summed
  uint64_t *const q_full = pv_done + 2;
  uint64_t *const drain = q_full + 1;
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(drain + 1);
  uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(drain + 1) + 1;
  int *const s_start = reinterpret_cast<int *>(drain + 2);                     // first sequence
  uint32_t *const issued = reinterpret_cast<uint32_t *>(drain + 4);            // [2] K, V tiles
  u64 *const s_base = reinterpret_cast<u64 *>(drain + 3);
  uint32_t *const beat = reinterpret_cast<uint32_t *>(drain + 5);              // (attn_wait)
  u64 *const scan = reinterpret_cast<u64 *>(s_q);                              // before Q arrives

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(full + i, 33);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, 128);
      mbar_init(p_full + i, 128);
      mbar_init(pv_done + i, 1);
    }
    mbar_init(q_full, C::kSoftmax);
    mbar_init(drain, 1);
    *abort_flag = 0;
    issued[0] = issued[1] = *beat = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's piece: prefix sums of the sequences' tiles ----
  const unsigned units = (unsigned)a.Hkv * (unsigned)a.row_blocks;   // items per sequence
  const int per = (a.S + THREADS - 1) / THREADS;
  const int q0 = min(a.S, tid * per), q1 = min(a.S, q0 + per);
  u64 mine = 0;
  for (int s = q0; s < q1; ++s) mine += attn_cost(attn_seq(a, s).tiles);
  u64 upto = mine;                                 // inclusive prefix over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 v = __shfl_up_sync(FULL, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) scan[warp] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  u64 before = upto - mine, total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const u64 v = scan[i];
    if (i < warp) before += v;
    total += v;
  }
  total *= units;
  const u64 chunk = attn_div(total + gridDim.x - 1, gridDim.x);
  const u64 start = min(total, chunk * blockIdx.x), stop = min(total, start + chunk);
  if (start < stop && before * units <= start && start < (before + mine) * units) {
    int s = q0;
    u64 base = before * units;
    for (;;) {
      const u64 t = (u64)attn_cost(attn_seq(a, s).tiles) * units;
      if (start < base + t) break;
      base += t;
      ++s;
    }
    *s_start = s;
    *s_base = base;
  }
  __syncthreads();
  // What the softmax warps do beside: sequences without a key get zeros, and
  // the item that this piece's start cuts, if no earlier start does, is noted.
  auto beside = [&](const AttnWalk *w) {
    for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
      if (attn_seq(a, s).tiles) continue;
      uint4 *o = reinterpret_cast<uint4 *>(a.out + (size_t)s * a.N * a.Hq * D);
      for (int i = tid; i < a.N * a.Hq * (D / 8); i += C::kSoftmax) o[i] = make_uint4(0, 0, 0, 0);
    }
    if (tid == 0) {
      AttnSplit sp{0, 0, 0, 0, 0};
      if (w != nullptr && w->t0 > 0) {           // (w: the piece's first segment)
        const u64 from = w->item_at, to = from + (unsigned)w->q.tiles - 1;
        sp = AttnSplit{w->s, w->kvh, w->rb, (int)attn_div(from, chunk), 0};
        if (sp.first + 1 == (int)blockIdx.x) sp.count = (int)attn_div(to, chunk) - sp.first + 1;
      }
      a.split[blockIdx.x] = sp;
    }
  };

  if (start < stop) {
    AttnWalk w;
    w.base = *s_base;
    w.pos = start;
    w.end = stop;
    w.s = *s_start;
    w.q = attn_seq(a, w.s);
    // rows that a tile of whole pages leaves unused: their weights are 0, their
    // values must not be NaN
    if (a.tile_keys < KT)
      for (int i = tid; i < C::kSlots * C::kSlot / 16; i += THREADS)
        reinterpret_cast<uint4 *>(s_ring)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
    __syncthreads();       // (the scan's memory becomes Q)
    const int group = a.Hq / a.Hkv;

    if (warp >= K_WARP) {
      // ----------------------------------------------------- producers: K and V --
      // A page is a TMA box per 64 dims.  Rows outside [lo, n) may hold anything:
      // of K they come along (their scores are masked), of V, where a weight of 0
      // times NaN would spoil the sum, pages with such rows go row by row through
      // cp.async, which zero-fills them.  Pages that are no whole number of eight
      // rows (the swizzle's period) all go that way.  A slot's barrier gets an arrival
      // a lane, after its cp.asyncs, and one with the bytes that TMA brings.
      constexpr int UNITS = D / 8;                     // 16-byte units of a row
      constexpr int RPP = 32 / UNITS;                  // rows of one pass of the warp
      const bool is_k = warp == K_WARP;
      const int u = lane % UNITS, r0 = lane / UNITS;
      const uint16_t *const cache = is_k ? a.k_cache : a.v_cache;
      const CUtensorMap *const map = is_k ? &k_map : &v_map;
      const uint64_t policy = policy_evict_normal();
      const int boxes = a.use_tma ? max(1, a.tile_keys / a.page_size) : 0;   // pages of a tile
      const int box_rows = a.use_tma ? a.tile_keys / boxes : 0;
      // this lane's page of the tile whose first key is k0, -1 where no key is seen
      auto page_of = [&](const AttnWalk &g, int k0) -> int {
        const int first = k0 + lane * box_rows;
        if (lane >= boxes || first + box_rows <= g.q.lo || first >= g.q.n) return -1;
        return __ldg(a.block_table + (size_t)g.s * a.max_pages + first / a.page_size);
      };
      auto first_key = [&](const AttnWalk &g) { return g.q.start + g.t0 * a.tile_keys; };
      uint32_t t = 0;                                  // tile
      AttnRing<C::kSlots> rg(is_k ? 0 : 2);
      bool ok = true, more = w.next(a, units);
      int next_page = more && a.use_tma ? page_of(w, first_key(w)) : -1;
      while (ok && more) {
        AttnWalk ahead = w;
        more = ahead.next(a, units);
        for (int tile = w.t0; tile < w.t1; ++tile, rg.advance(is_k && t == 0 ? 1 : 2), ++t) {
          const int k0 = w.q.start + tile * a.tile_keys;
          const int page = next_page;
          if (a.use_tma) {
            if (tile + 1 < w.t1) next_page = page_of(w, k0 + a.tile_keys);
            else if (more) next_page = page_of(ahead, first_key(ahead));
          }
          uint64_t *const bar = full + rg.slot;
          uint8_t *const to = s_ring + rg.slot * C::kSlot;
          const uint32_t dst = smem_u32(to);
          ok = __all_sync(FULL, attn_wait(empty + rg.slot, rg.phase ^ 1, abort_flag, beat));
          if (!ok) break;
          // lane = page + boxes * column block of 64 dims (32 boxes at most)
          const int pg = lane % max(boxes, 1), c64 = lane / max(boxes, 1);
          auto box = [&](int id) {
            tma_load_2d(to + c64 * KT * 128 + pg * box_rows * 128, map, c64 * 64,
                        (id * a.Hkv + w.kvh) * a.page_size + k0 % a.page_size, bar, policy);
          };
          if (a.use_tma && k0 >= w.q.lo && k0 + a.tile_keys <= w.q.n &&
              __all_sync(FULL, lane >= boxes || (page >= 0 && page < a.num_pages))) {
            if (is_k && lane < KT / 32)
              masks[(t % ATTN_MASKS) * 4 + lane] = bit_range(0, a.tile_keys, lane);
            __syncwarp();
            if (lane == 0) mbar_expect_tx(bar, (uint32_t)a.tile_keys * D * 2);
            const int id = __shfl_sync(FULL, page, pg);
            if (c64 < D / 64) box(id);
            mbar_arrive(bar);
          } else if (a.use_tma) {
            // this lane's page: seen in part or whole, in the pool; brought by TMA
            const int first = k0 + lane * box_rows;
            const bool seen = lane < boxes && first + box_rows > w.q.lo && first < w.q.n;
            const bool good = seen && page >= 0 && page < a.num_pages;
            const bool whole = good && first >= w.q.lo && first + box_rows <= w.q.n;
            if (seen && !good) raise_status(MOE_DEV_BAD_INDEX);
            const unsigned tma = __ballot_sync(FULL, is_k ? good : whole);
            const unsigned goods = __ballot_sync(FULL, good), bad = __ballot_sync(FULL, seen && !good);
            if (is_k && lane < KT / 32) {              // masks: keys in [lo, n) on good pages
              uint32_t m = bit_range(w.q.lo - k0, min(w.q.n - k0, a.tile_keys), lane);
              for (unsigned b = bad; b; b &= b - 1) {
                const int row0 = (__ffs(b) - 1) * box_rows;
                m &= ~bit_range(row0, row0 + box_rows, lane);
              }
              masks[(t % ATTN_MASKS) * 4 + lane] = m;
            }
            __syncwarp();
            if (lane == 0) mbar_expect_tx(bar, (uint32_t)__popc(tma) * box_rows * D * 2);
            __syncwarp();
            const int id = __shfl_sync(FULL, page, pg);
            if (c64 < D / 64 && ((tma >> pg) & 1)) box(id);
            if (!is_k) {
              // the other pages' rows, or zeros, in the 16-row steps of the product
              const int hull0 = max(w.q.lo - k0, 0) & ~15;
              const int hull1 = (min(w.q.n - k0, a.tile_keys) + 15) & ~15;
              for (int pgv = hull0 / box_rows; pgv < boxes && pgv * box_rows < hull1; ++pgv) {
                if ((tma >> pgv) & 1) continue;
                const bool in = (goods >> pgv) & 1;
                const int idv = __shfl_sync(FULL, page, pgv), row0 = pgv * box_rows;
                const size_t base =
                    in ? ((size_t)idv * a.Hkv + w.kvh) * a.page_size + (k0 + row0) % a.page_size : 0;
#pragma unroll 4
                for (int r = r0; r < box_rows; r += RPP) {
                  const int key = k0 + row0 + r;
                  const bool live = in && key >= w.q.lo && key < w.q.n;
                  cp_async16_zfill(dst + attn_place(u, row0 + r, KT),
                                   cache + (live ? (base + r) * D : 0) + u * 8, live);
                }
              }
            }
            __syncwarp();
            cp_async_arrive_noinc(bar);
          } else {
            uint32_t idx[KT / 32];                     // rows lane + 32 c of the cache
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) {
              const int e = c * 32 + lane, key = k0 + e;
              idx[c] = 0xffffffffu;
              if (key >= w.q.lo && key < w.q.n) {
                const int lp = key / a.page_size;
                const int id = __ldg(a.block_table + (size_t)w.s * a.max_pages + lp);
                if (id >= 0 && id < a.num_pages)
                  idx[c] = (uint32_t)(((size_t)id * a.Hkv + w.kvh) * a.page_size + (key - lp * a.page_size));
                else
                  raise_status(MOE_DEV_BAD_INDEX);
              }
              const uint32_t m = __ballot_sync(FULL, idx[c] != 0xffffffffu);
              if (is_k && lane == 0) masks[(t % ATTN_MASKS) * 4 + c] = m;
            }
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) {
#pragma unroll 8
              for (int j = 0; j < 32 / RPP; ++j) {
                const int r = c * 32 + j * RPP + r0;
                const uint32_t row = __shfl_sync(FULL, idx[c], j * RPP + r0);
                const bool live = row != 0xffffffffu;
                cp_async16_zfill(dst + attn_place(u, r, KT), cache + (live ? (size_t)row * D : 0) + u * 8, live);
              }
            }
            __syncwarp();                              // (the masks are written)
            if (lane == 0) mbar_arrive(bar);
            cp_async_arrive_noinc(bar);
          }
        }
        w = ahead;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) issued[is_k ? 0 : 1] = t;
    } else if (warp == MMA_WARP) {
      // ---------------------------------------------------------------- MMA --
      const uint32_t ring = smem_u32(s_ring), q = smem_u32(s_q);
      const uint32_t tm = __shfl_sync(FULL, tmem, 0);    // (uniform for the compiler too)
      constexpr uint32_t kIdS = idesc_bf16(KT, 0), kIdO = idesc_bf16(D, 1);
      uint32_t t = 0, seg = 0;
      AttnRing<C::kSlots> kr(0), vr(2);
      bool ok = true;                                    // (lanes agree after a vote per tile)
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        ok = ok && attn_wait(bar, parity, abort_flag, beat);
      };
      // S[tt & 1] = Q K^T, its K tile waited for
      auto scores = [&](uint32_t tt) {
        const uint64_t qd = smem_desc(q, 16, 1024, kSwizzle128B);
        const uint64_t kd = smem_desc(ring + kr.slot * C::kSlot, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int c = 0; c < D / 16; ++c)                 // (descriptors count 16 bytes)
          mma_f16_ss(tm + C::kS + (tt & 1) * KT, qd + ((c >> 2) * ATTN_ROWS * 128 + (c & 3) * 32) / 16,
                     kd + ((c >> 2) * KT * 128 + (c & 3) * 32) / 16, kIdS, c > 0);
        mma_commit(empty + kr.slot);
        mma_commit(s_full + (tt & 1));
        kr.advance(tt ? 2 : 1);
      };
      while (ok && w.next(a, units)) {
        const uint32_t t_first = t, t_end = t + __shfl_sync(FULL, (uint32_t)(w.t1 - w.t0), 0);
        wait(q_full, seg & 1);
        // tile t is scored as soon as the softmax has read tile t - 2 from its
        // place, two tiles ahead of its product with V
        for (uint32_t tt = t; tt < t_end + 2; ++tt) {
          if (tt < t_end) {
            if (tt >= 2) wait(s_free + (tt & 1), ((tt - 2) >> 1) & 1);
            wait(full + kr.slot, kr.phase);
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            fence_proxy_async();                         // (cp.async: the generic proxy)
            tc_fence_after();
            scores(tt);
          }
          if (tt < t_first + 2) continue;
          wait(p_full + (t & 1), (t >> 1) & 1);
          wait(full + vr.slot, vr.phase);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
          fence_proxy_async();
          tc_fence_after();
          const uint64_t vd = smem_desc(ring + vr.slot * C::kSlot, KT * 128, 1024, kSwizzle128B);
          // the 16-key steps that hold a key of the sequence: the others weigh 0, and
          // their values were not brought
          auto product = [&](int c, bool first) {
            mma_f16_ts(tm + C::kO + (WGS == 2 ? (t & 1) * D : 0),
                       tm + C::kP + (t & 1) * (KT / 2) + c * 8, vd + c * 2048 / 16, kIdO,
                       t >= t_first + WGS || !first);
          };
          if (t == t_first || t + 1 == t_end) {
            const int k0 = w.q.start + (w.t0 + (int)(t - t_first)) * a.tile_keys;
            const int c0 = __shfl_sync(FULL, max(w.q.lo - k0, 0) / 16, 0);
            const int c1 = __shfl_sync(FULL, (min(w.q.n - k0, a.tile_keys) + 15) / 16, 0);
#pragma unroll 1
            for (int c = c0; c < c1; ++c) product(c, c == c0);
          } else {
#pragma unroll
            for (int c = 0; c < KT / 16; ++c) product(c, c == 0);
          }
          mma_commit(empty + vr.slot);
          mma_commit(pv_done + (t & 1));
          vr.advance(2);
          ++t;
        }
        ++seg;
      }
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
    } else {
      // ------------------------------------------------------------ softmax --
      constexpr int NC = C::NC, GROUPS = WGS * KS;
      constexpr int PART = WGS == 1 || NC < 64 ? NC : 64;   // scores held at a time
      const int wg = warp >> 2, lid = tid & 127;            // warpgroup, tensor-memory lane
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const int kq = lid / C::RG, r = lid % C::RG;          // lane group: keys [kq NC, +NC) of a tile
      if (KS > 1) {                                         // weights of the other groups' keys: 0
        uint32_t zero[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) zero[e] = 0;
        if (wg == 0) {
#pragma unroll
          for (int c = 0; c < KT / 32; ++c) tc_st32(lanes + C::kP + c * 32, zero);
          tc_wait_st();
        }
        tc_fence_before();
        softmax_sync<C::kSoftmax>();
        tc_fence_after();
      }
      uint32_t t = 0;
      // A segment's queries, each warp rows of its lanes (rows past the last are
      // left as they are: they reach no output).  Called once all score MMAs of
      // the segment before are complete.
      auto load_q = [&](const AttnWalk &g) {
        constexpr int UNITS = D / 8, RPP = 32 / UNITS;
        const int row = g.rb * ATTN_ROWS + r;
        if (row - lane < a.rows) {
          const uint16_t *src = a.q + (size_t)g.s * a.N * a.Hq * D;
          const int u = lane % UNITS, r0 = lane / UNITS, tok = row / group;
          const int at = row < a.rows ? (tok * a.Hq + g.kvh * group + row - tok * group) * D : -1;
          const uint32_t dst = smem_u32(s_q);
#pragma unroll 8
          for (int jj = 0; jj < 32 / RPP / WGS; ++jj) {
            const int rr = (jj * WGS + wg) * RPP + r0;
            const int from = __shfl_sync(FULL, at, rr);
            if (from >= 0)
              cp_async16_zfill(dst + attn_place(u, (warp & 3) * 32 + rr, ATTN_ROWS), src + from + u * 8,
                               true);
          }
        }
        cp_async_arrive_noinc(q_full);
      };
      // columns [c, c + PART) of S, keys that the row does not see at -infinity
      auto load_s = [&](uint32_t at, int c, const uint32_t *vis, bool all, uint32_t (&s)[PART]) {
        if constexpr (PART == 16) {
          tc_ld16_nowait(at, s);
        } else {
#pragma unroll
          for (int h = 0; h < PART / 32; ++h) tc_ld32(at + c + h * 32, s + h * 32);
        }
        tc_wait_ld();
        if (!all) {
#pragma unroll
          for (int e = 0; e < PART; ++e)
            if (!((vis[(c + e) / 32] >> (e & 31)) & 1)) s[e] = 0xff800000u;
        }
      };
      bool more = w.next(a, units);
      if (more) load_q(w);
      beside(more ? &w : nullptr);
      while (more) {
        const int row = w.rb * ATTN_ROWS + r;
        const bool warp_live = row - lane < a.rows;
        const int tok = row < a.rows ? row / group : 0;
        const int pos = w.q.n - a.N + tok;                  // this row sees keys (pos-window, pos]
        const int see_lo = a.window > 0 ? pos - a.window + 1 : 0;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        const uint32_t t_first = t, t_end = t + (uint32_t)(w.t1 - w.t0);
        for (; t < t_end; ++t) {
          if (WGS == 2 && (int)(t & 1) != wg) continue;     // the other warpgroup's tile
          ok = attn_wait(s_full + (t & 1), (t >> 1) & 1, abort_flag);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
          tc_fence_after();
          if (warp_live) {
            const int k0 = w.q.start + (w.t0 + (int)(t - t_first)) * a.tile_keys + kq * NC;
            const uint32_t at = lanes + C::kS + (t & 1) * KT + kq * NC;
            constexpr int WORDS = NC < 32 ? 1 : NC / 32;
            constexpr uint32_t FULL_WORD = NC < 32 ? (1u << (NC & 31)) - 1u : 0xffffffffu;
            uint32_t vis[WORDS];                            // this group's keys, a bit each
            bool all = k0 + NC - 1 <= w.q.n - a.N && (a.window == 0 || k0 > w.q.n - 1 - a.window);
#pragma unroll
            for (int c = 0; c < WORDS; ++c) {
              const int key = kq * NC + c * 32;
              vis[c] = (masks[(t % ATTN_MASKS) * 4 + key / 32] >> (key & 31)) & FULL_WORD;
              all = all && vis[c] == FULL_WORD;
            }
            if (!all) {
#pragma unroll
              for (int c = 0; c < WORDS; ++c) vis[c] &= bit_range(see_lo - k0, pos + 1 - k0, c);
            }
            uint32_t s[PART];
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < NC; c += PART) {
              load_s(at, c, vis, all, s);
#pragma unroll
              for (int e = 0; e < PART; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
            }
            const float top =
                fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            // raise the maximum only where a weight would pass 2^8
            const bool raise = top > m + 8.f || (m == -INFINITY && top > -INFINITY);
            if (__any_sync(FULL, raise)) {
              const float mn = raise ? top : m;
              const float f = raise ? exp2_approx(m - mn) : 1.f;     // m = -inf: 0
              if (t >= t_first + WGS) {
                ok = attn_wait(pv_done + ((t - WGS) & 1), ((t - WGS) >> 1) & 1, abort_flag);
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ot = lanes + C::kO + (uint32_t)wg * D;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t o[32];
                  tc_ld32(ot + c * 32, o);
                  tc_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tc_st32(ot + c * 32, o);
                }
              }
              l *= f;
              m = mn;
            }
            const float base = m == -INFINITY ? 0.f : m;
            if (t >= 2) {                         // P[t & 1] is free once PV(t-2) is done
              ok = attn_wait(pv_done + (t & 1), ((t - 2) >> 1) & 1, abort_flag);
              ok = __all_sync(FULL, ok);
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t pt = lanes + C::kP + (t & 1) * (KT / 2) + kq * (NC / 2);
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NC; c += PART) {
              if (NC > PART) load_s(at, c, vis, all, s);
              if (c + PART == NC) {                         // S is read: the next tile may come
                tc_fence_before();
                mbar_arrive(s_free + (t & 1));
              }
#pragma unroll
              for (int e = 0; e < PART; e += 2) {
                const float p0 = exp2_approx(fmaf(__uint_as_float(s[e]), a.scale_log2, -base));
                const float p1 = exp2_approx(fmaf(__uint_as_float(s[e + 1]), a.scale_log2, -base));
                sum[(e >> 1) & 3] += p0 + p1;
                s[e >> 1] = pack_bf16(p0, p1);
              }
              if constexpr (PART == 16) tc_st_x8(pt, reinterpret_cast<const uint32_t(&)[8]>(s));
              else if constexpr (PART == 32) tc_st16(pt, s);
              else {
#pragma unroll
                for (int h = 0; h < PART / 64; ++h) tc_st32(pt + c / 2 + h * 32, s + h * 32);
              }
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc_wait_st();
          } else {
            // A warp without rows must not run a phase ahead of the others either: S(t + 2)
            // may come as soon as S(t) is read, and a second arrival of this warp would
            // then complete P(t) in the place of a warp that still writes it.
            mbar_arrive(s_free + (t & 1));
            if (t >= 2) {
              ok = attn_wait(pv_done + (t & 1), ((t - 2) >> 1) & 1, abort_flag);
              ok = __all_sync(FULL, ok);
              if (!ok) break;
            }
          }
          tc_fence_before();
          mbar_arrive(p_full + (t & 1));
        }
        // ---- the segment's end: once all its score MMAs are complete, the next
        // segment's queries; then O / l to out, or O, m, l to the workspace ----
        AttnWalk ahead = w;
        more = ahead.next(a, units);
        t = t_end;
        if (ok && WGS == 2) ok = attn_wait(s_full + ((t - 1) & 1), ((t - 1) >> 1) & 1, abort_flag);
        ok = __all_sync(FULL, ok);
        if (ok && more) load_q(ahead);
        // this warpgroup's last tile: t - 1, or the one before; none in a segment
        // of the other's single tile
        const uint32_t mine = WGS == 1 || (int)((t - 1) & 1) == wg ? t - 1 : t - 2;
        const bool had = mine + 1 > t_first;                // (mine may be t_first - 1 = ~0)
        if (ok && had) {
          ok = attn_wait(pv_done + (mine & 1), (mine >> 1) & 1, abort_flag);
          ok = __all_sync(FULL, ok);
        }
        ok = softmax_all<C::kSoftmax>(ok);
        if (!ok) break;
        tc_fence_after();
        // The warpgroups' and lane groups' shares of a row meet in shared memory,
        // 32 dims at a time; 8 threads then add up and write a row's quads.
        const bool whole = w.t0 == 0 && w.t1 == w.q.tiles, live = row < a.rows;
        const int slot = 2 * (int)blockIdx.x + (w.t0 == 0 ? 1 : 0);
        float2 *const ml = reinterpret_cast<float2 *>(scratch);
        ml[tid] = make_float2(m, l);
        if (wg == 0 && kq == 0) row_at[r] = live ? (tok * a.Hq + row - tok * group) * D : -1;
        softmax_sync<C::kSoftmax>();
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, ml[g * C::RG + r].x);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const float2 x = ml[g * C::RG + r];
          sum += exp2_approx(x.x - base) * x.y;
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const float f = exp2_approx(m - base) * (whole ? inv : 1.f);
        if (!whole && live && wg == 0 && kq == 0)
          a.part_ml[(size_t)slot * a.rows_cap + r] = make_float2(top, sum);
        softmax_sync<C::kSoftmax>();
        uint16_t *const item = a.out + ((size_t)w.s * a.N * a.Hq + w.kvh * group) * D + (tid & 7) * 4;
        float4 *const piece = a.part_o + (size_t)slot * a.rows_cap * (D / 4) + (tid & 7);
        const int rows = min(C::RG, a.rows - w.rb * ATTN_ROWS);
        const uint32_t ot = lanes + C::kO + (uint32_t)wg * D;
        bool finite = true;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          if (warp_live) {
            uint32_t o[32];
            if (had) {
              tc_ld32(ot + c * 32, o);
              tc_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              scratch[e * C::kPitch + tid] =
                  had ? make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                    __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          softmax_sync<C::kSoftmax>();
          for (int rr = tid >> 3; rr < rows; rr += C::kSoftmax / 8) {
            const float4 *const from = scratch + (tid & 7) * C::kPitch + rr;
            float4 x = from[0];
#pragma unroll
            for (int g = 1; g < GROUPS; ++g) {
              const float4 y = from[g * C::RG];
              x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            }
            finite = finite && fmaf(x.x, 0.f, fmaf(x.y, 0.f, fmaf(x.z, 0.f, x.w * 0.f))) == 0.f;
            if (whole)
              *reinterpret_cast<uint2 *>(item + row_at[rr] + c * 32) =
                  make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
            else
              piece[(size_t)rr * (D / 4) + c * 8] = x;
          }
          if (c + 1 < D / 32) softmax_sync<C::kSoftmax>();
        }
        if (!softmax_all<C::kSoftmax>(finite)) {
          // values that are not finite: the rows in whose product some of the segment's
          // keys weigh 0 are summed anew over the keys that they see.  Those are the rows
          // that do not see all of them, and with lane groups every row (the other
          // groups' keys weigh 0, and an infinity would come out as NaN).
          if (wg == 0 && kq == 0) ml[r] = make_float2(base, inv);
          softmax_sync<C::kSoftmax>();
          const int ka = max(w.q.lo, w.q.start + w.t0 * a.tile_keys);
          const int kb = (int)min((long long)w.q.n, w.q.start + (long long)w.t1 * a.tile_keys);
          int done = 0;
          for (int rr = warp; rr < rows; rr += C::kSoftmax / 32) {
            const int at = w.rb * ATTN_ROWS + rr, i = at / group, p = w.q.n - a.N + i;
            const int k0 = max(ka, a.window > 0 ? p - a.window + 1 : 0), k1 = min(kb, p + 1);
            if (KS == 1 && k0 == ka && k1 == kb) continue;
            done = attn_row_alone<D>(
                a, w.s, i, w.kvh * group + at - i * group, k0, k1, ml[rr].x, ml[rr].y,
                whole ? item - (tid & 7) * 4 + row_at[rr] : nullptr,
                reinterpret_cast<float *>(piece - (tid & 7) + (size_t)rr * (D / 4)), done, beat);
          }
          softmax_sync<C::kSoftmax>();
        }
        tc_fence_before();
        w = ahead;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp < MMA_WARP) {
    beside(nullptr);
  }
  tc_fence_before();
  __syncthreads();
  // after a wait that ran out: the copies still in flight into this CTA's memory
  if (*abort_flag && tid < C::kSlots) {
    int last = -1;                                      // the last tile put into slot tid
    for (int t = 0; t < (int)issued[0]; ++t) {
      const int i = t ? 2 * t - 1 : 0;
      if (i % C::kSlots == tid) last = max(last, i);
    }
    for (int t = 0; t < (int)issued[1]; ++t)
      if ((2 * t + 2) % C::kSlots == tid) last = max(last, 2 * t + 2);
    if (last >= 0) mbar_wait_drain(full + tid, (uint32_t)(last / C::kSlots) & 1);
  }
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::kCols));
  }
}

// Adds the pieces of the cut items.  A CTA takes units of (item, a few of its
// rows); a thread owns four dims of a row and every G-th piece, and the G
// groups' sums meet in shared memory, always in the same order.  G grows with
// the pieces (148 of one item where a single sequence fills the GPU, two or
// three where many do), the rows of a unit shrink with it.
constexpr int JOIN_THREADS = 512;

template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) attn_join_kernel(const AttnArgs a, int pieces) {
  pdl_wait();
  pdl_trigger();
  constexpr int QUADS = D / 4;
  constexpr int MOST_ROWS = JOIN_THREADS / QUADS;        // G = 1
  // rows x pieces of a unit: 4 MOST_ROWS x 4, MOST_ROWS / 2 x 16 or / 8 x 148 at most
  __shared__ float wgt[MOST_ROWS / 8 * ATTN_MAX_CTAS];
  static_assert(16 <= ATTN_MAX_CTAS / 8, "weights of few pieces");
  __shared__ float4 acc[JOIN_THREADS];
  __shared__ AttnSplit items[ATTN_MAX_CTAS];
  __shared__ int first[ATTN_MAX_CTAS + 1];               // units before an item
  __shared__ int warp_sum[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.Hq / a.Hkv;
  // groups of pieces: a unit's weights (rows x pieces) fit `wgt` either way
  auto shift_of = [](int count) { return count > 16 ? 3 : count > 4 ? 1 : 0; };
  auto rows_per_unit = [&](int count) { return count > 4 ? MOST_ROWS >> shift_of(count) : 4 * MOST_ROWS; };
  auto rows_of = [&](const AttnSplit &sp) { return min(ATTN_ROWS, a.rows - sp.rb * ATTN_ROWS); };
  int mine = 0;
  if (tid < pieces) {
    const AttnSplit sp = a.split[tid];
    items[tid] = sp;
    const int rpu = rows_per_unit(sp.count);
    mine = sp.count ? (rows_of(sp) + rpu - 1) / rpu : 0;
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31 && warp < 8) warp_sum[warp] = upto;
  __syncthreads();
  for (int i = 0; i < min(warp, 8); ++i) upto += warp_sum[i];
  if (tid < pieces) first[tid + 1] = upto;
  if (tid == 0) first[0] = 0;
  __syncthreads();
  const int total = first[pieces];

  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int lo = 0, hi = pieces;                             // the item: first[lo] <= u < first[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= u) lo = mid;
      else hi = mid;
    }
    const AttnSplit sp = items[lo];
    const int G = 1 << shift_of(sp.count), rpu = rows_per_unit(sp.count);
    const int r0 = (u - first[lo]) * rpu, rows = min(rpu, rows_of(sp) - r0);
    auto slot = [&](int i) { return 2 * (size_t)(sp.first + i) + (i == 0 ? 1 : 0); };
    // the pieces' weights 2^(m_i - m) / l: a warp per row
    for (int rr = warp; rr < rows; rr += JOIN_THREADS / 32) {
      const float2 *ml = a.part_ml + r0 + rr;
      constexpr int MOST = (ATTN_MAX_CTAS + 31) / 32;
      float2 x[MOST];
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int j = 0; j < MOST; ++j)
        x[j] = lane + 32 * j < sp.count ? ml[slot(lane + 32 * j) * a.rows_cap] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < MOST; ++j) m = fmaxf(m, x[j].x);
      m = warp_max(m);
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int j = 0; j < MOST; ++j) {
        x[j].x = exp2_approx(x[j].x - base);
        l = fmaf(x[j].y, x[j].x, l);
      }
      l = moe::warp_sum(l);
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int j = 0; j < MOST; ++j)
        if (lane + 32 * j < sp.count) wgt[rr * sp.count + lane + 32 * j] = x[j].x * inv;
    }
    __syncthreads();
    const int d4 = tid % QUADS;
    auto add = [](float4 &o, const float4 &x, float f) {
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    };
    auto store = [&](int rr, const float4 &o) {
      const int row = sp.rb * ATTN_ROWS + r0 + rr, tok = row / group;
      uint16_t *dst = a.out +
                      (((size_t)sp.s * a.N + tok) * a.Hq + sp.kvh * group + (row - tok * group)) * D + d4 * 4;
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
    };
    const size_t step = (size_t)QUADS * a.rows_cap;
    if (sp.count <= 4) {                                 // four rows to a thread
      float4 o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= sp.count) break;
        const float4 *x = a.part_o + slot(i) * step + (size_t)r0 * QUADS + d4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = tid / QUADS + k * MOST_ROWS;
          if (rr < rows) add(o[k], x[(size_t)rr * QUADS], wgt[rr * sp.count + i]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rr = tid / QUADS + k * MOST_ROWS;
        if (rr < rows) store(rr, o[k]);
      }
    } else {
      const int rr = (tid / QUADS) % rpu, grp = tid / (rpu * QUADS);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows) {
        const float4 *x = a.part_o + (size_t)(r0 + rr) * QUADS + d4;
#pragma unroll 4
        for (int i = grp; i < sp.count; i += G) add(o, x[slot(i) * step], wgt[rr * sp.count + i]);
      }
      acc[tid] = o;
      __syncthreads();
      if (grp == 0 && rr < rows) {
        for (int g = 1; g < G; ++g) add(o, acc[tid + g * rpu * QUADS], 1.f);
        store(rr, o);
      }
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- host --

struct AttnWs {
  size_t ml, split, total;
};
inline int attn_rows_cap(int N, int Hq, int Hkv) {
  const long rows = (long)N * (Hq / Hkv);
  return (int)std::min<long>(ATTN_ROWS, (rows + 7) / 8 * 8);
}
inline AttnWs attn_ws(int N, int Hq, int Hkv, int D) {
  const size_t cap = (size_t)attn_rows_cap(N, Hq, Hkv), slots = 2 * ATTN_MAX_CTAS;
  AttnWs w;
  w.ml = slots * cap * D * sizeof(float);
  w.split = w.ml + slots * cap * sizeof(float2);
  w.total = (w.split + ATTN_MAX_CTAS * sizeof(AttnSplit) + 255) & ~size_t(255);
  return w;
}

template <int D, int KS>
inline int attn_launch(AttnArgs a, uint8_t *ws, int sms, cudaStream_t s) {
  typedef AttnCfg<D, KS> C;
  static std::mutex mu;
  static uint64_t done = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!((done >> dev) & 1ull)) {
      if (cudaFuncSetAttribute(attn_kernel<D, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::kSmem) != cudaSuccess ||
          // (the join runs between two attention kernels: the same split of an
          // SM's memory, which is changed on an idle SM only)
          cudaFuncSetAttribute(attn_join_kernel<D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
      }
      done |= 1ull << dev;
    }
  }
  const AttnWs w = attn_ws(a.N, a.Hq, a.Hkv, D);
  a.rows_cap = attn_rows_cap(a.N, a.Hq, a.Hkv);
  a.row_blocks = (a.rows + ATTN_ROWS - 1) / ATTN_ROWS;
  a.part_o = reinterpret_cast<float4 *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
  a.split = reinterpret_cast<AttnSplit *>(ws + w.split);
  const unsigned grid = (unsigned)std::min(sms, ATTN_MAX_CTAS);
  // Pages of 8 rows or a multiple go by TMA (the swizzle repeats every 8 rows),
  // as many whole ones to a tile as fit, or a tile's worth of a larger one.
  const int ps = a.page_size;
  CUtensorMap k_map{}, v_map{};
  a.tile_keys = C::KT;
  a.align = 1;
  a.use_tma = 0;
  if (ps % 8 == 0 && (ps <= C::KT || ps % C::KT == 0)) {
    a.tile_keys = ps <= C::KT ? C::KT / ps * ps : C::KT;
    a.align = std::min(ps, C::KT);
    a.use_tma = 1;
    const uint64_t rows = (uint64_t)a.num_pages * a.Hkv * ps;
    const uint32_t box = (uint32_t)a.align;
    if (rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (!make_map(&k_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.k_cache, D, rows, D * 2, 64, box) ||
        !make_map(&v_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.v_cache, D, rows, D * 2, 64, box))
      return MOE_ERR_CUDA;
  }
  cudaError_t e = launch_pdl(attn_kernel<D, KS>, grid, C::kThreads, C::kSmem, s, k_map, v_map, a);
  if (e == cudaSuccess)
    e = launch_pdl(attn_join_kernel<D>, grid, JOIN_THREADS, 0, s, a, (int)grid);
  if (e != cudaSuccess) {
    fprintf(stderr, "mxfp4_moe: launch failed: %s\n", cudaGetErrorString(e));
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// Lane groups by the rows to a key/value head (measured at the head of this file).
template <int D>
inline int attn_dispatch(AttnArgs a, uint8_t *ws, int sms, cudaStream_t s) {
  a.rows = a.N * (a.Hq / a.Hkv);
  return a.rows <= 32   ? attn_launch<D, 4>(a, ws, sms, s)
         : a.rows <= 64 ? attn_launch<D, 2>(a, ws, sms, s)
                        : attn_launch<D, 1>(a, ws, sms, s);
}

}  // namespace moe
