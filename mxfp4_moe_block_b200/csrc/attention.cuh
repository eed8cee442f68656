// attention.cuh -- attention of a drafted block over a paged key-value cache.
//
//   out = sum_j softmax_j(scale q.k_j) v_j,  keys j <= position, inside the window
//
// The N tokens x (Hq/Hkv) query heads that share a key/value head are the rows
// of one matrix: S = Q K^T and O += P V run on tcgen05 with 128 rows (rows past
// the last are zeros), keys in tiles of KT, S and O in tensor memory.  At
// these row counts the cache's bytes bound the call (2 flops per row and byte
// against ~250 flops per byte of the machine), so a padded 128-row MMA costs
// nothing: a 64 KB tile (128 keys, D = 128) takes the tensor pipe ~1000 cycles
// and an SM's share of HBM ~2700.
//
// Softmax in one pass: every row keeps a maximum m and a sum l in float; O is
// rescaled only when a tile's maximum exceeds m by 8 (in powers of two), so
// weights reach 2^8 at most and the accumulator in tensor memory is rarely
// touched.  The weights go to the tensor cores as bf16 (8 bits, half a step
// 2^-9 of a weight, like the keys and values); l sums them before rounding.
//
// Split over the length: the tiles of all (sequence, key/value head, row block)
// items form one line, cut into G equal pieces, one per CTA (one CTA per SM),
// so uneven lengths and single long sequences fill the GPU alike.  An item that
// lies in one piece is written out directly; of the others each piece leaves
// its unnormalised O, m and l in the workspace and attn_join_kernel adds them
// in the order of the pieces (the same bits on every run).
//
// Warps: 0-3 softmax (a thread per row, tensor-memory lane = row), 4 the MMA
// issuer, 5-8 producers: cp.async of 16-byte units, page by page, into a ring
// of K and V tiles in the 128-byte swizzle; rows outside the sequence or on a
// bad page are zero-filled and masked by a bit per key.
// Every wait is bounded (MOE_DEV_TIMEOUT), as in the expert FFN.
#pragma once
#include "common.cuh"
#include "ffn_tc.cuh"

namespace moe {

constexpr int ATTN_MAX_CTAS = 148;
constexpr int ATTN_ROWS = 128;
constexpr int ATTN_THREADS = 288;
constexpr int ATTN_PRODUCERS = 128;
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
  // workspace: unnormalised O [2G][D/4][rows_cap] float4, (m, l) [2G][rows_cap],
  // one AttnSplit per piece
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

template <int D>
struct AttnCfg {
  static constexpr int KT = D == 256 ? 64 : 128;      // keys per tile
  static constexpr int kSlot = KT * D * 2;            // one K or V tile
  static constexpr int kQ = ATTN_ROWS * D * 2;
  static constexpr int kSlots = D == 64 ? 12 : D == 128 ? 6 : 5;
  static constexpr int kMisc = 2048;
  static constexpr int kSmem = kQ + kSlots * kSlot + kMisc;
  // tensor memory columns: S x2, O, P x2 (two bf16 to a column)
  static constexpr uint32_t kS = 0, kO = D == 256 ? 256 : 2 * KT;
  static constexpr uint32_t kP = D == 256 ? 2 * KT : kO + D;
  static constexpr uint32_t kCols = 512;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kP + KT <= kCols && kO + D <= kCols, "tensor memory");
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A from tensor memory: lane = row, two consecutive K elements to a column
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
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

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
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

// Visible keys of a sequence: [lo, n), in tiles from lo on; none for a slot not
// in use or (reported) a length past the table's row.
struct AttnSeq {
  int lo, n, tiles;
};
template <int KT>
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs &a, int s) {
  const int n = __ldg(a.kv_len + s);
  if (n <= 0) return AttnSeq{0, 0, 0};
  if (n > a.max_pages * a.page_size) {
    raise_status(MOE_DEV_BAD_INDEX);
    return AttnSeq{0, 0, 0};
  }
  const int lo = a.window > 0 ? max(0, n - a.N - a.window + 1) : 0;
  return AttnSeq{lo, n, (n - lo + KT - 1) / KT};
}

// A CTA's piece of the line of tiles, item by item.  Every role walks it alone.
template <int KT>
struct AttnWalk {
  unsigned long long base, pos, end;   // first tile of sequence s, next tile, end of the piece
  AttnSeq q;
  int s;
  // the segment: tiles [t0, t1) of an item of q.tiles tiles
  int kvh, rb, t0, t1;

  __device__ __forceinline__ bool next(const AttnArgs &a, unsigned units) {
    if (pos >= end) return false;
    while (pos >= base + (unsigned long long)q.tiles * units) {
      base += (unsigned long long)q.tiles * units;
      q = attn_seq<KT>(a, ++s);
    }
    const unsigned long long at = pos - base;
    const unsigned item = (unsigned)(at / (unsigned)q.tiles);
    t0 = (int)(at - (unsigned long long)item * (unsigned)q.tiles);
    t1 = (int)min((unsigned long long)q.tiles, t0 + (end - pos));
    kvh = (int)(item / (unsigned)a.row_blocks);
    rb = (int)(item - (unsigned)kvh * (unsigned)a.row_blocks);
    pos += t1 - t0;
    return true;
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

// true iff `v` holds on every producer thread (named barrier 1)
__device__ __forceinline__ bool producers_all(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"((uint32_t)v) : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(ATTN_THREADS, 1) attn_kernel(const AttnArgs a) {
  typedef AttnCfg<D> C;
  constexpr int KT = C::KT;
  typedef unsigned long long u64;
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  uint8_t *const s_q = attn_smem;
  uint8_t *const s_ring = attn_smem + C::kQ;
  uint8_t *const misc = s_ring + C::kSlots * C::kSlot;
  uint32_t *const rowidx = reinterpret_cast<uint32_t *>(misc);                 // [2][128]
  uint32_t *const masks = rowidx + 2 * 128;                                    // [8][4]
  uint64_t *const full = reinterpret_cast<uint64_t *>(masks + ATTN_MASKS * 4); // [kSlots]
  uint64_t *const empty = full + C::kSlots;                                    // [kSlots]
  uint64_t *const s_full = empty + C::kSlots;                                  // [2]
  uint64_t *const p_full = s_full + 2;                                         // [2]
  uint64_t *const pv_done = p_full + 2;                                        // [2]
  uint64_t *const q_full = pv_done + 2;
  uint64_t *const q_empty = q_full + 1;
  uint64_t *const drain = q_empty + 1;
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(drain + 1);
  uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(drain + 1) + 1;
  int *const s_start = reinterpret_cast<int *>(drain + 2);                     // sequence, tiles
  u64 *const s_base = reinterpret_cast<u64 *>(drain + 3);
  u64 *const scan = reinterpret_cast<u64 *>(s_q);                              // before Q arrives

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(full + i, ATTN_PRODUCERS + 4);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(pv_done + i, 1);
    }
    mbar_init(q_full, ATTN_PRODUCERS + 4);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's piece: prefix sums of the sequences' tiles ----
  const unsigned units = (unsigned)a.Hkv * (unsigned)a.row_blocks;   // items per sequence
  const int per = (a.S + ATTN_THREADS - 1) / ATTN_THREADS;
  const int q0 = min(a.S, tid * per), q1 = min(a.S, q0 + per);
  u64 mine = 0;
  for (int s = q0; s < q1; ++s) mine += attn_seq<KT>(a, s).tiles;
  scan[tid] = mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  u64 before = 0, total = 0;
  for (int i = 0; i < ATTN_THREADS; ++i) {
    const u64 v = scan[i];
    if (i < tid) before += v;
    total += v;
  }
  total *= units;
  const u64 chunk = (total + gridDim.x - 1) / gridDim.x;
  const u64 start = min(total, chunk * blockIdx.x), stop = min(total, start + chunk);
  if (start < stop && before * units <= start && start < (before + mine) * units) {
    int s = q0;
    u64 base = before * units;
    for (;;) {
      const u64 t = (u64)attn_seq<KT>(a, s).tiles * units;
      if (start < base + t) break;
      base += t;
      ++s;
    }
    *s_start = s;
    *s_base = base;
    // the item that this piece's start cuts, if no earlier start does
    const unsigned T = (unsigned)attn_seq<KT>(a, s).tiles;
    const unsigned item = (unsigned)((start - base) / T);
    const u64 from = base + (u64)item * T;
    AttnSplit sp{s, (int)(item / (unsigned)a.row_blocks), (int)(item % (unsigned)a.row_blocks),
                 (int)(from / chunk), 0};
    if (from < start && sp.first + 1 == (int)blockIdx.x)
      sp.count = (int)((from + T - 1) / chunk) - sp.first + 1;
    a.split[blockIdx.x] = sp;
  }
  if (tid == 0 && start >= stop) a.split[blockIdx.x] = AttnSplit{0, 0, 0, 0, 0};
  // sequences without a key: zeros
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    if (attn_seq<KT>(a, s).tiles) continue;
    uint4 *o = reinterpret_cast<uint4 *>(a.out + (size_t)s * a.N * a.Hq * D);
    for (int i = tid; i < a.N * a.Hq * (D / 8); i += ATTN_THREADS) o[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();

  if (start < stop) {
    AttnWalk<KT> w;
    w.base = *s_base;
    w.pos = start;
    w.end = stop;
    w.s = *s_start;
    w.q = attn_seq<KT>(a, w.s);
    __syncthreads();       // (the scan's memory becomes Q)
    const int group = a.Hq / a.Hkv;

    if (warp >= 5) {
      // ---------------------------------------------------------- producers --
      constexpr int UNITS = D / 8;                     // 16-byte units of a row
      constexpr int RPP = ATTN_PRODUCERS / UNITS;      // rows of one pass
      const int p = tid - 160, u = p % UNITS, r0 = p / UNITS;
      const uint32_t ring = smem_u32(s_ring);
      // unit u of row r in a tile of `rows` rows: 64-dim column blocks, swizzled
      auto place = [&](int r, int rows) -> uint32_t {
        return (uint32_t)((u >> 3) * rows * 128 + r * 128 + (((u & 7) ^ (r & 7)) << 4));
      };
      uint32_t i = 0, t = 0, seg = 0;                  // ring index, tile, segment
      bool ok = true;
      auto slot_free = [&]() {
        return i < (uint32_t)C::kSlots ||
               attn_wait(empty + i % C::kSlots, (i / C::kSlots + 1) & 1, abort_flag);
      };
      auto load = [&](const uint16_t *cache, const uint32_t *rows) {
        const uint32_t dst = ring + (i % C::kSlots) * C::kSlot;
#pragma unroll
        for (int j = 0; j < KT / RPP; ++j) {
          const int r = r0 + j * RPP;
          const uint32_t row = rows[r];
          const bool live = row != 0xffffffffu;
          cp_async16_zfill(dst + place(r, KT), cache + (live ? (size_t)row * D : 0) + u * 8, live);
        }
        cp_async_arrive_noinc(full + i % C::kSlots);
        if (lane == 0) mbar_arrive(full + i % C::kSlots);
        ++i;
      };
      // (the producers leave together: a wait that ran out is carried to the
      // next tile's barrier)
      bool leave = false;
      while (!leave && w.next(a, units)) {
        const int32_t *table = a.block_table + (size_t)w.s * a.max_pages;
        for (int tile = w.t0; tile < w.t1; ++tile, ++t) {
          ok = slot_free() && ok;
          uint32_t *rows = rowidx + (t & 1) * 128;
          if (p < KT) {
            const int key = w.q.lo + tile * KT + p;
            uint32_t row = 0xffffffffu;
            if (key < w.q.n) {
              const int lp = key / a.page_size;
              const int page = __ldg(table + lp);
              if (page >= 0 && page < a.num_pages)
                row = (uint32_t)(((size_t)page * a.Hkv + w.kvh) * a.page_size + (key - lp * a.page_size));
              else
                raise_status(MOE_DEV_BAD_INDEX);
            }
            rows[p] = row;
            const uint32_t m = __ballot_sync(FULL, row != 0xffffffffu);
            if (lane == 0) masks[(t % ATTN_MASKS) * 4 + p / 32] = m;
          }
          ok = producers_all(ok);
          if (!ok) {
            leave = true;
            break;
          }
          load(a.k_cache, rows);
          if (tile == w.t0) {                          // the segment's queries
            if (seg) ok = attn_wait(q_empty, (seg + 1) & 1, abort_flag);
            if (ok) {
              const uint32_t dst = smem_u32(s_q);
#pragma unroll 4
              for (int r = r0; r < ATTN_ROWS; r += RPP) {
                const int row = w.rb * ATTN_ROWS + r;
                const bool live = row < a.rows;
                const int tok = live ? row / group : 0, h = live ? row - tok * group : 0;
                cp_async16_zfill(dst + place(r, ATTN_ROWS),
                                 a.q + (((size_t)w.s * a.N + tok) * a.Hq + w.kvh * group + h) * D + u * 8,
                                 live);
              }
              cp_async_arrive_noinc(q_full);
              if (lane == 0) mbar_arrive(q_full);
            }
            ++seg;
          }
          ok = ok && slot_free();
          if (ok) load(a.v_cache, rows);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 4) {
      // ---------------------------------------------------------------- MMA --
      if (lane == 0) {
        const uint32_t ring = smem_u32(s_ring), q = smem_u32(s_q);
        constexpr uint32_t kIdS = idesc_bf16(KT, 0), kIdO = idesc_bf16(D, 1);
        uint32_t i = 0, t = 0, seg = 0;
        bool ok = true;
        auto ready = [&]() {
          if (!attn_wait(full + i % C::kSlots, (i / C::kSlots) & 1, abort_flag)) return false;
          fence_proxy_async();         // cp.async wrote through the generic proxy
          tc_fence_after();
          return true;
        };
        // S[t] = Q K^T; K tiles sit at even ring indices 2t, V tiles at 2t + 1
        auto scores = [&](uint32_t tt) {
          i = 2 * tt;
          if (!ready()) return false;
          const uint32_t k = ring + (i % C::kSlots) * C::kSlot;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t ofs = (c & 3) * 32;
            mma_f16_ss(tmem + C::kS + (tt & 1) * KT,
                       smem_desc(q + (c >> 2) * ATTN_ROWS * 128 + ofs, 16, 1024, kSwizzle128B),
                       smem_desc(k + (c >> 2) * KT * 128 + ofs, 16, 1024, kSwizzle128B), kIdS, c > 0);
          }
          tc_commit(empty + i % C::kSlots);
          tc_commit(s_full + (tt & 1));
          return true;
        };
        while (ok && w.next(a, units)) {
          const uint32_t t_end = t + (uint32_t)(w.t1 - w.t0), t_first = t;
          ok = attn_wait(q_full, seg & 1, abort_flag) && scores(t);
          if (ok && t + 1 == t_end) tc_commit(q_empty);
          for (; ok && t < t_end; ++t) {
            if (t + 1 < t_end) {
              ok = scores(t + 1);
              if (ok && t + 2 == t_end) tc_commit(q_empty);
            }
            ok = ok && attn_wait(p_full + (t & 1), (t >> 1) & 1, abort_flag);
            if (!ok) break;
            i = 2 * t + 1;
            ok = ready();
            if (!ok) break;
            const uint32_t v = ring + (i % C::kSlots) * C::kSlot;
#pragma unroll
            for (int c = 0; c < KT / 16; ++c)
              mma_f16_ts(tmem + C::kO, tmem + C::kP + (t & 1) * (KT / 2) + c * 8,
                         smem_desc(v + c * 2048, KT * 128, 1024, kSwizzle128B), kIdO,
                         t > t_first || c > 0);
            tc_commit(empty + i % C::kSlots);
            tc_commit(pv_done + (t & 1));
          }
          ++seg;
        }
        tc_commit(drain);
        mbar_wait_drain(drain, 0);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ softmax --
      const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
      uint32_t t = 0;
      bool ok = true;
      while (ok && w.next(a, units)) {
        const int row = w.rb * ATTN_ROWS + tid;
        const bool warp_live = w.rb * ATTN_ROWS + warp * 32 < a.rows;
        const int tok = row < a.rows ? row / group : 0;
        const int pos = w.q.n - a.N + tok;                  // this row sees keys (pos-window, pos]
        const int see_lo = a.window > 0 ? pos - a.window + 1 : 0;
        float m = -INFINITY, l = 0.f;
        const uint32_t t_first = t, t_end = t + (uint32_t)(w.t1 - w.t0);
        for (; t < t_end; ++t) {
          ok = attn_wait(s_full + (t & 1), (t >> 1) & 1, abort_flag);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
          tc_fence_after();
          if (warp_live) {
            uint32_t s[KT];
#pragma unroll
            for (int c = 0; c < KT / 32; ++c)
              tc_ld32(lanes + C::kS + (t & 1) * KT + c * 32, s + c * 32);
            const int k0 = w.q.lo + (w.t0 + (int)(t - t_first)) * KT;
            uint32_t vis[KT / 32];
            bool all = k0 + KT - 1 <= w.q.n - a.N && (a.window == 0 || k0 > w.q.n - 1 - a.window);
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) {
              vis[c] = masks[(t % ATTN_MASKS) * 4 + c];
              all = all && vis[c] == 0xffffffffu;
            }
            tc_wait_ld();
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (!all) {
#pragma unroll
              for (int c = 0; c < KT / 32; ++c) {
                vis[c] &= bit_range(see_lo - k0, pos + 1 - k0, c);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((vis[c] >> e) & 1)) s[c * 32 + e] = 0xff800000u;      // -infinity
              }
            }
#pragma unroll
            for (int e = 0; e < KT; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
            const float top =
                fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            // raise the maximum only where a weight would pass 2^8
            const bool raise = top > m + 8.f || (m == -INFINITY && top > -INFINITY);
            if (__any_sync(FULL, raise)) {
              const float mn = raise ? top : m;
              const float f = raise ? exp2_approx(m - mn) : 1.f;     // m = -inf: 0
              if (t > t_first) {
                ok = attn_wait(pv_done + ((t - 1) & 1), ((t - 1) >> 1) & 1, abort_flag);
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t o[32];
                  tc_ld32(lanes + C::kO + c * 32, o);
                  tc_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tc_st32(lanes + C::kO + c * 32, o);
                }
              }
              l *= f;
              m = mn;
            }
            const float base = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < KT; e += 2) {
              const float p0 = exp2_approx(fmaf(__uint_as_float(s[e]), a.scale_log2, -base));
              const float p1 = exp2_approx(fmaf(__uint_as_float(s[e + 1]), a.scale_log2, -base));
              sum[(e >> 1) & 3] += p0 + p1;
              s[e >> 1] = cvt_bf16x2(p0, p1);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (t >= 2) {                         // P[t & 1] is free once PV(t-2) is done
              ok = attn_wait(pv_done + (t & 1), ((t - 2) >> 1) & 1, abort_flag);
              ok = __all_sync(FULL, ok);
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll
            for (int c = 0; c < KT / 64; ++c)
              tc_st32(lanes + C::kP + (t & 1) * (KT / 2) + c * 32, s + c * 32);
            tc_wait_st();
          }
          tc_fence_before();
          mbar_arrive(p_full + (t & 1));
        }
        if (!ok) break;
        // ---- the segment's end: O / l to out, or O, m, l to the workspace ----
        ok = attn_wait(pv_done + ((t - 1) & 1), ((t - 1) >> 1) & 1, abort_flag);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          const bool whole = w.t0 == 0 && w.t1 == w.q.tiles;
          const bool live = row < a.rows;
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const int slot = 2 * (int)blockIdx.x + (w.t0 == 0 ? 1 : 0);
          uint16_t *dst = a.out + (((size_t)w.s * a.N + tok) * a.Hq + w.kvh * group + (row - tok * group)) * D;
          float4 *part = a.part_o + ((size_t)slot * (D / 4)) * a.rows_cap + tid;
          if (!whole && live) a.part_ml[(size_t)slot * a.rows_cap + tid] = make_float2(m, l);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc_ld32(lanes + C::kO + c * 32, o);
            tc_wait_ld();
            if (!live) continue;
            if (whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  // l = 0: the row saw no key (its O is a sum of zeros)
                  const float lo = __uint_as_float(o[e + 2 * k]) * inv;
                  const float hi = __uint_as_float(o[e + 2 * k + 1]) * inv;
                  x[k] = cvt_bf16x2(lo, hi);
                }
                *reinterpret_cast<uint4 *>(dst + c * 32 + e) = make_uint4(x[0], x[1], x[2], x[3]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                part[(size_t)(c * 8 + e / 4) * a.rows_cap] =
                    make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            }
          }
        }
        tc_fence_before();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::kCols));
  }
}

// Adds the pieces of each cut item.  grid (pieces, row groups); a thread
// owns four dims of one row.
constexpr int JOIN_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) attn_join_kernel(const AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int RPB = JOIN_THREADS / (D / 4);            // rows of a CTA
  const AttnSplit sp = a.split[blockIdx.x];
  if (sp.count == 0) return;
  const int r = blockIdx.y * RPB + threadIdx.x % RPB, d4 = threadIdx.x / RPB;
  const int row = sp.rb * ATTN_ROWS + r;
  if (r >= a.rows_cap || row >= a.rows) return;
  auto slot = [&](int i) { return 2 * (size_t)(sp.first + i) + (i == 0 ? 1 : 0); };
  float m = -INFINITY;
  for (int i = 0; i < sp.count; ++i) m = fmaxf(m, a.part_ml[slot(i) * a.rows_cap + r].x);
  float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  if (m > -INFINITY) {
#pragma unroll 4
    for (int i = 0; i < sp.count; ++i) {
      const float2 ml = a.part_ml[slot(i) * a.rows_cap + r];
      const float4 x = a.part_o[(slot(i) * (D / 4) + d4) * a.rows_cap + r];
      const float f = exp2_approx(ml.x - m);
      l = fmaf(ml.y, f, l);
      o[0] = fmaf(x.x, f, o[0]);
      o[1] = fmaf(x.y, f, o[1]);
      o[2] = fmaf(x.z, f, o[2]);
      o[3] = fmaf(x.w, f, o[3]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int group = a.Hq / a.Hkv, tok = row / group;
  uint16_t *dst =
      a.out + (((size_t)sp.s * a.N + tok) * a.Hq + sp.kvh * group + (row - tok * group)) * D + d4 * 4;
  *reinterpret_cast<uint2 *>(dst) =
      make_uint2(cvt_bf16x2(o[0] * inv, o[1] * inv), cvt_bf16x2(o[2] * inv, o[3] * inv));
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

template <int D>
inline int attn_launch(AttnArgs a, uint8_t *ws, int sms, cudaStream_t s) {
  typedef AttnCfg<D> C;
  static std::mutex mu;
  static uint64_t done = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!((done >> dev) & 1ull)) {
      if (cudaFuncSetAttribute(attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::kSmem) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
      }
      done |= 1ull << dev;
    }
  }
  const AttnWs w = attn_ws(a.N, a.Hq, a.Hkv, D);
  a.rows = a.N * (a.Hq / a.Hkv);
  a.rows_cap = attn_rows_cap(a.N, a.Hq, a.Hkv);
  a.row_blocks = (a.rows + ATTN_ROWS - 1) / ATTN_ROWS;
  a.part_o = reinterpret_cast<float4 *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
  a.split = reinterpret_cast<AttnSplit *>(ws + w.split);
  const unsigned grid = (unsigned)std::min(sms, ATTN_MAX_CTAS);
  cudaError_t e = launch_pdl(attn_kernel<D>, grid, ATTN_THREADS, C::kSmem, s, a);
  if (e == cudaSuccess) {
    constexpr int RPB = JOIN_THREADS / (D / 4);
    e = launch_pdl(attn_join_kernel<D>, dim3(grid, (unsigned)((a.rows_cap + RPB - 1) / RPB)),
                   JOIN_THREADS, 0, s, a);
  }
  if (e != cudaSuccess) {
    fprintf(stderr, "mxfp4_moe: launch failed: %s\n", cudaGetErrorString(e));
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace moe
