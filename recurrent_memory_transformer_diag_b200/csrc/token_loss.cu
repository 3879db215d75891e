// Softmax cross entropy over a large vocabulary, straight from hidden states
// and head weights, with its gradients; the logits are never kept.
//
//   l[n][v] = scale * h_n . w_v        lse_n = log sum_v exp l[n][v]
//   loss_n  = lse_n - l[n][t_n]        (0 for a row without a target)
//   P[n][v] = g_n (exp(l[n][v] - lse_n) - [v = t_n])
//   dH = scale P W       dW = scale P^T H
//
// One tensor-core kernel computes every product, in three roles:
//   LSE   logits tile by tile; each tile leaves (max, sum of exponentials) of
//         its columns per row and the target's logit, joined by a small kernel
//   PROB  logits of one vocabulary piece again, turned into P (bf16: half a step
//         of bf16 a value, as an operand of the products.  Up to 64 rows, where
//         few roundings average out, two terms; fp32 operands three.  Errors of
//         the gradients of bf16 operands against 64 bits: 1.9e-3 to 2.3e-3, of
//         which the results' own rounding is 1.7e-3; a second term for all rows would
//         double the products of both gradients)
//   GRAD  both gradients of the piece from P in one launch: dW tiles contract
//         over the rows, dH tiles over the piece's columns
// A piece of the vocabulary is as wide as P of that piece stays within 256 MB (of
// 256 columns at least: more from 524288 bf16 rows on), so no logits or P of the
// whole vocabulary are kept.  What does grow with it: fp32 operands' head as
// three bf16 terms (6 bytes an element) and, of the loss, two numbers per row
// and 128 entries for 8192 rows at a time.
//
// Rows are put in order first: rows with a target in front, the others behind
// them as zeros (so what stands in a masked row cannot reach the head's
// gradient), and the products stop at the last row with a target.
//
// Accumulation: tcgen05 adds into fp32 accumulators with truncation, measured
// here as a relative error of about 2e-6 at K = 2048 growing with K.  Where
// the result is read in fp32 (all logits, P's as the loss's; everything of fp32
// operands) the accumulator therefore covers one to eight k-blocks only, where
// it is rounded to bf16 right away (the gradients of bf16 operands) 128, and the
// epilogue threads add these chunks in registers, rounded to nearest.
//
// fp32 operands: x = hi + mid + lo with three bf16 terms (24 bits).  A k-block
// is three stages, one for each term of both operands (lo first), and six
// products into one accumulator: every pair of terms but the three whose
// product is below 2^-24 of the result, the small ones first, so that only the
// last product truncates a sum of full size.  (Six copies of two tiles instead took 437 ns a product
// of a 256 x 256 tile, against 270 for the product itself.)
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "armt_internal.cuh"
#include "copies_in_flight.cuh"
#include "tcgen05_ptx.cuh"
#include "vec8.cuh"

namespace armt {

namespace {

using namespace tc;

constexpr int TILE = 256;              // rows and columns of a CTA pair's tile (each CTA: 128 rows)
constexpr int BK = 64;                 // 64 bf16 = 128 bytes = one swizzle row
constexpr int BOX_BYTES = 64 * BK * 2; // one copied box: 64 x 64 bf16
constexpr int STAGE_BYTES = 4 * BOX_BYTES;   // two boxes of A, two of B
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 128 + 32 * EPI_WARPS;   // a control warpgroup and two epilogue ones
// registers per thread: 384 threads start with 168 (64512 in all); the control
// warpgroup gives its to the epilogue, which holds 128 sums a thread
constexpr int CTRL_REGS = 40, EPI_REGS = 232;
static_assert(128 * CTRL_REGS + 32 * EPI_WARPS * EPI_REGS <= 168 * NUM_THREADS, "register split");
constexpr int SLOT_BYTES = 4096;       // 32 rows x 128 bytes of output; two per epilogue warp

enum Role { LSE = 0, PROB = 1, GRAD = 2 };

// Shared memory: LSE writes no tile and has all of it for stages in flight.
template <int ROLE>
struct Smem {
  static constexpr int STAGES = ROLE == LSE ? 7 : 5;
  static constexpr int SLOTS = STAGES * STAGE_BYTES;
  static constexpr int BARS = SLOTS + (ROLE == LSE ? 0 : 2 * EPI_WARPS * SLOT_BYTES);
  static constexpr int TOTAL = BARS + 256 + 1024;   // + alignment slack
  static_assert(TOTAL <= 227 * 1024, "shared memory per CTA");
};

constexpr int ROW_GROUP = 32;          // row tiles that share a vocabulary tile before the next one
constexpr int LSE_CHUNK = 8;           // k-blocks per accumulator of the logits of many rows (K = 512)
constexpr int GRAD_CHUNK = 128;        // ... of the gradients of bf16 operands (K = 8192: 1e-5 where the type rounds by
                                       // 2e-3; one over 262144 rows lost 3e-4.  K = 2048 took 1 to 2 % more time)
constexpr int F32_CHUNK = 1;           // ... of everything that fp32 operands give (six products of K = 64)
constexpr float LOG2E = 1.4426950408889634f;

struct LossParams {
  int n_rows, d, vocab;
  int two_terms;              // GRAD, few bf16 rows: the second terms of P stand as further rows, this far behind
  int planes;                 // 1: bf16 operands; 3: fp32 operands as three bf16 terms
  int v0, vc;                 // vocabulary piece
  int panels;                 // P is kept in panels of 64 columns: [term][panel][row][64], 4 to 8 KB a copy
  int chunk;                  // k-blocks per accumulator
  int tile_n;                 // LSE, PROB: columns of a tile, 256 or 128
  float scale;
  const int* n_valid;         // rows with a target (device)
  const int* perm;            // fp32 few rows, PROB: where an ordered row stands in hidden
  const int* target;          // per row in order
  // LSE
  float2* part; int part_pitch; float* target_logit;
  // PROB
  const float* lse; const float* g;
  bf16* p_out; int p_trans;   // few rows: P is kept transposed, each thread writing its entry: [term][entry][NT], or
                              // [entry][term][NT] beside bf16 operands
  // few rows, LSE: rows in their own order, targets as the caller gave them
  const void* ids; int id_bytes; unsigned* block_err;
  // GRAD
  int want_dw, want_dh, splits, k_split, dh_add, dw_bf16;
  int dw_splits, dw_k;        // dW's contraction in splits of dw_k rows, as partial sums where there are several
  const float* g_max;
  unsigned* err;
  int debug_no_loads;         // test hook: no copies are issued, so the first wait for a stage runs out
};

struct LossMaps {
  CUtensorMap a, b, c;        // operands: LSE/PROB hidden, head; GRAD P, head, hidden
  CUtensorMap out0, out1;     // PROB: P; GRAD: dW, dH partial sums
};

// Bounded waits (as in the header) that sleep in the hardware: a waiting warp is
// woken by the barrier or after the hint, instead of reading the clock all the
// while (the tensor cores are under the power cap here).
constexpr uint32_t SLEEP_NS = 20000;

template <bool CLUSTER>
__device__ __forceinline__ bool try_wait_sleeping(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(SLEEP_NS)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(SLEEP_NS)
        : "memory");
  return ok != 0;
}

// By a whole converged warp; the same answer in all lanes.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__any_sync(0xffffffffu, try_wait_sleeping<CLUSTER>(bar, parity))) return true;
  const unsigned long long t0 = global_ns();
  while (true) {
    if (__any_sync(0xffffffffu, try_wait_sleeping<CLUSTER>(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0 || global_ns() - t0 > WAIT_LIMIT_NS)) return false;
  }
}

// One tile of work: D[256 x 256] = A B^T over k-blocks kb = 0 .. kblocks-1.
struct Job {
  int m0, n0;        // first row / column in the operands' own coordinates
  int ka, kb;        // first k coordinate in A / B
  int kblocks;
  int n;             // columns computed: 256, or 128 (few tiles, or where the gradient's width ends there)
  bool dw;           // GRAD: a tile of dW (A is P transposed)
  int split;         // GRAD, dH: which partial sum
  int ntile;         // LSE: index of the vocabulary tile
};

template <int ROLE>
struct Jobs {
  int mt, nt, dt, total, n_dw, n_dh;
  bool dw_first;   // the longer contraction first, so that the shorter tiles fill the end
  __device__ Jobs(const LossParams& p, int nv) {
    mt = (nv + TILE - 1) / TILE;
    nt = ROLE == GRAD ? (p.vc + TILE - 1) / TILE : (p.vc + p.tile_n - 1) / p.tile_n;
    dt = (p.d + TILE - 1) / TILE;
    if (ROLE == GRAD) {
      n_dw = p.want_dw ? nt * dt * p.dw_splits : 0;
      n_dh = p.want_dh ? mt * dt * p.splits : 0;
      total = n_dw + n_dh;
      dw_first = min(nv, p.dw_k) >= p.k_split;
    } else {
      n_dw = n_dh = 0;
      dw_first = false;
      total = mt * nt;
    }
  }
  __device__ Job get(const LossParams& p, int nv, int t) const {
    Job j;
    j.dw = false;
    j.split = 0;
    j.ntile = 0;
    j.n = TILE;
    if (ROLE != GRAD) {
      // consecutive tiles share a vocabulary tile: the head is read from HBM
      // once per group of rows, the group's hidden rows stay in L2
      const int per = ROW_GROUP * nt;
      const int grp = t / per, r = t - grp * per;
      const int mg = min(ROW_GROUP, mt - grp * ROW_GROUP);
      j.ntile = r / mg;
      j.m0 = (grp * ROW_GROUP + r - j.ntile * mg) * TILE;
      j.n = p.tile_n;
      j.n0 = p.v0 + j.ntile * p.tile_n;
      j.ka = j.kb = 0;
      j.kblocks = (p.d + BK - 1) / BK;
    } else if (dw_first ? t < n_dw : t >= n_dh) {
      int r = dw_first ? t : t - n_dh;
      j.dw = true;
      j.n0 = (r % dt) * TILE;
      r /= dt;
      j.m0 = (r % nt) * TILE;
      j.split = r / nt;
      j.ka = j.kb = j.split * p.dw_k;
      j.kblocks = (max(min(nv - j.ka, p.dw_k), 0) + BK - 1) / BK;
    } else {
      int r = dw_first ? t - n_dw : t;
      j.n0 = (r % dt) * TILE;
      r /= dt;
      j.m0 = (r % mt) * TILE;
      j.split = r / mt;
      j.ka = j.split * p.k_split;
      j.kb = p.v0 + j.ka;
      j.kblocks = (min(p.vc - j.ka, p.k_split) + BK - 1) / BK;
    }
    if (ROLE == GRAD && p.d - j.n0 <= TILE / 2) j.n = TILE / 2;
    return j;
  }
};

// Shared-memory operand descriptors (128-byte swizzle).  A box is 64 rows of
// 128 bytes.  K-major: the rows are the tile's rows, 8-row groups 1024 bytes
// apart, 32 bytes per K = 16.  MN-major (the operand stored with k as rows):
// a row holds 64 of the tile's rows, the next 64 are the next box (leading
// offset), 8-k groups 1024 bytes apart, 2048 bytes per K = 16.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, bool mn) {
  uint64_t d = sw128_desc(saddr);
  if (mn) d += (uint64_t)((BOX_BYTES >> 4) - 1) << 16;   // LBO 1 -> one box
  return d;
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// 16-byte piece q of this lane's row in a slot (128-byte swizzle).
__device__ __forceinline__ uint4* slot_piece(uint8_t* slot, int lane, int q) {
  return reinterpret_cast<uint4*>(slot + lane * 128 + ((q ^ (lane & 7)) << 4));
}

// Output of a warp's 32 rows through its two slots: put() each 128 bytes a row,
// then send().  begin(): the slots may be written (their last stores have read
// them).
__device__ __forceinline__ void begin_out(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

// REST: v keeps what the written term leaves of the value.
template <bool REST>
__device__ __forceinline__ void put_bf16x64(uint8_t* slot, int lane, float2* v) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint4 pk;
    uint32_t* w = reinterpret_cast<uint32_t*>(&pk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b2 = __float22bfloat162_rn(v[q * 4 + i]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b2);
      if constexpr (REST) {
        v[q * 4 + i].x -= __uint_as_float(w[i] << 16);
        v[q * 4 + i].y -= __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    *slot_piece(slot, lane, q) = pk;
  }
}

__device__ __forceinline__ void put_f32x32(uint8_t* slot, int lane, const float2* v) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *slot_piece(slot, lane, q) = make_uint4(__float_as_uint(v[2 * q].x), __float_as_uint(v[2 * q].y),
                                            __float_as_uint(v[2 * q + 1].x), __float_as_uint(v[2 * q + 1].y));
}

// Slots 0 and (two) 1 to (c0, c1, c2) and dc0, dc2 further.
__device__ __forceinline__ void send_out(const CUtensorMap* map, uint8_t* slots, int lane, int c0, int c1, int c2,
                                         int dc0, int dc2, bool two, bool add) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add) {
      tma_add_3d(map, slots, c0, c1, c2);
      if (two) tma_add_3d(map, slots + SLOT_BYTES, c0 + dc0, c1, c2 + dc2);
    } else {
      tma_store_3d(map, slots, c0, c1, c2);
      if (two) tma_store_3d(map, slots + SLOT_BYTES, c0 + dc0, c1, c2 + dc2);
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What the epilogue needs of its row, loaded before it waits for the products.
struct RowData {
  int target;        // -1: none, or past the last row
  float g, lse;      // PROB
};

template <int ROLE>
__device__ __forceinline__ RowData load_row(const LossParams& p, int row, int nv) {
  RowData r = {-1, 0.f, 0.f};
  if (ROLE != GRAD && row < nv) {
    r.target = p.target[row];
    if (ROLE == PROB) {
      r.g = p.g[row];
      r.lse = p.lse[row];
    }
  }
  return r;
}

// Epilogue of one tile: sums holds this thread's row (TMEM lane) of 128
// columns, those of its half of the tile.
template <int ROLE>
__device__ __forceinline__ void finish_tile(const LossParams& p, const LossMaps& maps, const Job& j, int nv,
                                            const RowData& rd, float2 (&sums)[64], int row_in_tile, int half,
                                            int lane, uint8_t* slots) {
  const int row = j.m0 + row_in_tile;
  const int wrow0 = row - lane;
  const int col0 = j.n0 + half * 128;
  if (half * 128 >= j.n) return;   // a tile of 128 columns
  if constexpr (ROLE == LSE) {
    const float2 scale2 = make_float2(p.scale, p.scale);
#pragma unroll
    for (int i = 0; i < 64; ++i) sums[i] = __fmul2_rn(sums[i], scale2);
    if (col0 + 128 > p.vocab) {   // the last tile: columns past the vocabulary do not count
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        if (col0 + 2 * i >= p.vocab) sums[i].x = -INFINITY;
        if (col0 + 2 * i + 1 >= p.vocab) sums[i].y = -INFINITY;
      }
    }
    float mx[4] = {sums[0].x, sums[0].y, sums[1].x, sums[1].y};
#pragma unroll
    for (int i = 2; i < 64; ++i) {
      mx[2 * (i & 1)] = fmaxf(mx[2 * (i & 1)], sums[i].x);
      mx[2 * (i & 1) + 1] = fmaxf(mx[2 * (i & 1) + 1], sums[i].y);
    }
    const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    const float ms = m == -INFINITY ? 0.f : m;
    const float2 neg = make_float2(-ms, -ms), log2e = make_float2(LOG2E, LOG2E);
    float2 s2[2] = {};
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const float2 x = __fmul2_rn(__fadd2_rn(sums[i], neg), log2e);
      s2[i & 1] = __fadd2_rn(s2[i & 1], make_float2(ex2(x.x), ex2(x.y)));
    }
    s2[0] = __fadd2_rn(s2[0], s2[1]);
    if (row < nv) {
      p.part[(long long)(j.ntile * (j.n / 128) + half) * p.part_pitch + row] = make_float2(m, s2[0].x + s2[0].y);
      const unsigned at = (unsigned)(rd.target - col0);
      if (at < 128u) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          t = at == 2u * i ? sums[i].x : t;
          t = at == 2u * i + 1 ? sums[i].y : t;
        }
        p.target_logit[row] = t;
      }
    }
  } else if constexpr (ROLE == PROB) {
    const float g = rd.g, lse = rd.lse;
    const float2 scale2 = make_float2(p.scale, p.scale), neg = make_float2(-lse, -lse),
                 log2e = make_float2(LOG2E, LOG2E), g2 = make_float2(g, g);
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const float2 x = __fmul2_rn(__fadd2_rn(__fmul2_rn(sums[i], scale2), neg), log2e);
      sums[i] = __fmul2_rn(make_float2(ex2(x.x), ex2(x.y)), g2);
    }
    if (rd.target >= 0) {
      const unsigned at = (unsigned)(rd.target - col0);
      if (at < 128u) {
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          sums[i].x -= at == 2u * i ? g : 0.f;
          sums[i].y -= at == 2u * i + 1 ? g : 0.f;
        }
      }
    }
    if (g == 0.f) {   // rows without a target or weight: zero whatever their logits are
#pragma unroll
      for (int i = 0; i < 64; ++i) sums[i] = make_float2(0.f, 0.f);
    }
    if (col0 + 128 > p.vocab) {   // the last tile: columns past the vocabulary (logits of 0) may be infinite, and dH
                                  // contracts over the whole panel that they stand in
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        if (col0 + 2 * i >= p.vocab) sums[i].x = 0.f;
        if (col0 + 2 * i + 1 >= p.vocab) sums[i].y = 0.f;
      }
    }
    const int pc = col0 - p.v0;   // column in the piece
    if (wrow0 >= p.n_rows || pc >= p.vc) return;   // nothing of these panels is in P
    for (int t = 0; t + 1 < p.planes; ++t) {
      begin_out(lane);
      put_bf16x64<true>(slots, lane, sums);
      put_bf16x64<true>(slots + SLOT_BYTES, lane, sums + 32);
      send_out(&maps.out0, slots, lane, 0, wrow0, t * p.panels + pc / 64, 0, 1, pc + 64 < p.vc, false);
    }
    begin_out(lane);
    put_bf16x64<false>(slots, lane, sums);
    put_bf16x64<false>(slots + SLOT_BYTES, lane, sums + 32);
    send_out(&maps.out0, slots, lane, 0, wrow0, (p.planes - 1) * p.panels + pc / 64, 0, 1, pc + 64 < p.vc, false);
  } else {
    if (col0 >= p.d || wrow0 >= (j.dw ? p.vc : p.n_rows)) return;
    const bool parts = !j.dw || p.dw_splits > 1;   // partial sums, joined by a later kernel
    if (!parts) {
      const float f = *p.g_max * p.scale;
      const float2 f2 = make_float2(f, f);
#pragma unroll
      for (int i = 0; i < 64; ++i) sums[i] = __fmul2_rn(sums[i], f2);
      if (p.dw_bf16) {
        begin_out(lane);
        put_bf16x64<false>(slots, lane, sums);
        put_bf16x64<false>(slots + SLOT_BYTES, lane, sums + 32);
        send_out(&maps.out0, slots, lane, col0, p.v0 + wrow0, 0, 64, 0, col0 + 64 < p.d, false);
        return;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (col0 + 64 * h >= p.d) break;
      begin_out(lane);
      put_f32x32(slots, lane, sums + 32 * h);
      put_f32x32(slots + SLOT_BYTES, lane, sums + 32 * h + 16);
      send_out(j.dw ? &maps.out0 : &maps.out1, slots, lane, col0 + 64 * h, parts ? wrow0 : p.v0 + wrow0,
               parts ? j.split : 0, 32, 0, col0 + 64 * h + 32 < p.d, !j.dw && p.dh_add);
    }
  }
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Persistent, one CTA pair per two SMs (cluster of 2, tcgen05 cta_group::2):
//   warp 0      copies: this CTA's 128 rows of A and 128 of the tile's 256 B
//               rows per stage, counted on the even CTA's barrier
//   warp 1      (even CTA) issues the products, M = 256, N = 256, K = 16
//   warps 4..11 epilogue: thread = row, each warp half of the columns
// Two accumulators of 256 TMEM columns: the epilogue of one chunk runs beside
// the products of the next.  Every wait is bounded (about one second).
template <int ROLE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    token_loss_kernel(const __grid_constant__ LossMaps maps, const LossParams p) {
  using SM = Smem<ROLE>;
  constexpr int STAGES = SM::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::BARS);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* skip_word = tmem_slot + 2;
  uint32_t* sent = tmem_slot + 3;      // [rank]: the stages each CTA has issued copies to, in both CTAs
  uint32_t* narrow = tmem_slot + 5;    // of the odd CTA's, in the even one: those of 128 columns (three boxes, not four)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    // an earlier kernel of this call already gave up on a wait: skip the work
    // (the even CTA decides for both)
    *skip_word = *reinterpret_cast<volatile unsigned*>(p.err) & ERR_WAIT_TIMEOUT_MASK;
    sent[0] = sent[1] = *narrow = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const bool skip = ld_cluster_u32(mapa_shared(smem_u32(skip_word), 0)) != 0;

  const int nv = ROLE == GRAD && p.two_terms ? 2 * p.two_terms : *p.n_valid;
  const Jobs<ROLE> jobs(p, nv);
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
  if (skip) {
    // nothing to do
  } else if (warp == 0) {
    // ---------------- copies (both CTAs; whole warp, one elected lane issues) ----------------
    const bool issuer = elect_one();
    int stage = 0;
    uint32_t phase = 0, of_128 = 0;
    CopiesInFlight copies;
    bool ok = true;
    const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
    for (int t = cid; t < jobs.total && ok; t += ncl) {
      const Job j = jobs.get(p, nv, t);
      const bool a_mn = ROLE == GRAD && j.dw != (p.p_trans != 0), b_mn = ROLE == GRAD;
      const CUtensorMap* ma = &maps.a;
      const CUtensorMap* mb = ROLE == GRAD && j.dw ? &maps.c : &maps.b;
      const int am = j.m0 + (int)rank * 128, bn = j.n0 + (int)rank * (j.n / 2);
      for (int kb = 0, q = p.planes - 1; kb < j.kblocks;) {   // q: the term of both operands
        if (!wait_warp<true>(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
        uint8_t* sa = smem + stage * STAGE_BYTES;
        if (issuer && !p.debug_no_loads) {
          // both CTAs' copies
          if (leader) mbar_expect_tx(&full[stage], 2 * (2 * BOX_BYTES + j.n / 128 * BOX_BYTES));
          const uint32_t fb = full0 + (uint32_t)(stage * sizeof(uint64_t));
          const int ka = j.ka + kb * BK, kbb = j.kb + kb * BK;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = am + 64 * h;
            if (ROLE == GRAD && !p.p_trans)
              tma_load_3d_pair(ma, fb, sa + h * BOX_BYTES, 0, a_mn ? ka : row, q * p.panels + (a_mn ? row : ka) / BK);
            else
              tma_load_3d_pair(ma, fb, sa + h * BOX_BYTES, a_mn ? row : ka, a_mn ? ka : row, q);
            if (128 * h < j.n)
              tma_load_3d_pair(mb, fb, sa + (2 + h) * BOX_BYTES, b_mn ? bn + 64 * h : kbb, b_mn ? kbb : bn + 64 * h,
                               q);
          }
        }
        if (!p.debug_no_loads) copies.issued(stage, phase);
        of_128 = (of_128 & ~(1u << stage)) | (j.n == 128 ? 1u << stage : 0u);
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
        if (--q < 0) { q = p.planes - 1; ++kb; }
      }
    }
    if (!ok) {
      if (issuer) atomicOr(p.err, 1u);
      *abort_flag = 1;
    }
    if (issuer) {
      st_cluster_u32(mapa_shared(smem_u32(&sent[rank]), 0), copies.word());
      st_cluster_u32(mapa_shared(smem_u32(&sent[rank]), 1), copies.word());
      if (!leader) st_cluster_u32(mapa_shared(smem_u32(narrow), 0), of_128);
    }
    if (leader) {   // copies of both CTAs are counted on the even CTA's barriers
      const unsigned long long t0 = global_ns();
      copies.drain([&](int s, uint32_t par) { return mbar_try_wait_cluster(&full[s], par); },
                   [&] { return global_ns() - t0 > WAIT_LIMIT_NS; });
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- products (even CTA; whole warp, one elected lane issues) ----------------
      const bool issuer = elect_one();
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = cid; t < jobs.total && ok; t += ncl) {
        const Job j = jobs.get(p, nv, t);
        const bool a_mn = ROLE == GRAD && j.dw != (p.p_trans != 0), b_mn = ROLE == GRAD;
        const uint32_t idesc = idesc_f16(j.n, 1, TILE) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        const uint32_t step_a = a_mn ? 2048 : 32, step_b = b_mn ? 2048 : 32;
        for (int it = 0; it < j.kblocks && ok;) {
          if (!wait_warp<true>(&tempty[buf], acc_phase ^ 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(buf * TILE);
          const int end = min(j.kblocks, it + p.chunk);
          auto product = [&](int sa, int sb, bool add) {   // of the A tile of one stage and the B tile of another
            const uint32_t a = smem_u32(smem + sa * STAGE_BYTES), b = smem_u32(smem + sb * STAGE_BYTES) + 2 * BOX_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_f16_pair(d_tmem, operand_desc(a + kk * step_a, a_mn), operand_desc(b + kk * step_b, b_mn), idesc,
                           (add || kk > 0) ? 1u : 0u);
          };
          for (int first = it; it < end && ok; ++it) {
            int lo = stage, mid = stage;   // stages of the terms; the last one is hi's, or the only one
            for (int q = p.planes - 1; q >= 0; --q) {
              if (!wait_warp<true>(&full[stage], phase, abort_flag)) { ok = false; break; }
              if (q == 1) mid = stage;
              if (q == 0) {
                tc_fence_after();
                if (issuer) {
                  if (p.planes == 3) {
                    product(stage, lo, it > first);
                    product(lo, stage, true);
                    mma_commit_pair(&empty[lo], 0x3);
                    product(mid, mid, true);
                    product(stage, mid, true);
                    product(mid, stage, true);
                    mma_commit_pair(&empty[mid], 0x3);
                  }
                  product(stage, stage, p.planes == 3 || it > first);
                  mma_commit_pair(&empty[stage], 0x3);
                }
              }
              if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
          }
          if (!ok) break;
          if (issuer) mma_commit_pair(&tfull[buf], 0x3);
          if (++buf == 2) { buf = 0; acc_phase ^= 1; }
        }
      }
      if (!ok) {
        if (issuer) atomicOr(p.err, 2u);
        *abort_flag = 1;
      }
      if (issuer) mma_commit_pair(drain, 0x1);   // no product writes either CTA's TMEM after this arrives
      const unsigned long long t0 = global_ns();
      while (!mbar_try_wait(drain, 0)) {
        if (global_ns() - t0 > WAIT_LIMIT_NS) break;
      }
    }
  }   // warps 2 and 3: nothing to do
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    // ---------------- epilogue (warps 4..11, both CTAs) ----------------
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;
    const int row_in_tile = (int)rank * 128 + quarter * 32 + lane;
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    uint8_t* slots = smem + SM::SLOTS + (warp - 4) * 2 * SLOT_BYTES;
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = !skip;
    for (int t = cid; t < jobs.total && ok; t += ncl) {
      const Job j = jobs.get(p, nv, t);
      const RowData rd = load_row<ROLE>(p, j.m0 + row_in_tile, nv);
      float2 acc[64];   // this thread's row, 128 columns (pairs: two additions or products an instruction)
      if (j.kblocks == 0) {
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      }
      for (int it = 0; it < j.kblocks; it += p.chunk) {
        if (!wait_warp<true>(&tfull[buf], acc_phase, abort_flag)) {
          if (lane == 0) atomicOr(p.err, 4u);
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * TILE + half * 128);
        if (it == 0) {   // the first chunk straight into the sums
          uint32_t v[2][64];
          tmem_ld64_nowait(tbase, v[0]);
          tmem_ld64_nowait(tbase + 64, v[1]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 64; ++i)
            acc[i] = make_float2(__uint_as_float(v[i / 32][2 * (i % 32)]), __uint_as_float(v[i / 32][2 * (i % 32) + 1]));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld32(tbase + (uint32_t)(c * 32), v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[c * 16 + i] = __fadd2_rn(acc[c * 16 + i], make_float2(v[2 * i], v[2 * i + 1]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + (uint32_t)(buf * sizeof(uint64_t)));
        if (++buf == 2) { buf = 0; acc_phase ^= 1; }
      }
      if (ok) finish_tile<ROLE>(p, maps, j, nv, rd, acc, row_in_tile, half, lane, slots);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync_all();   // no product, copy or epilogue of either CTA still uses TMEM or shared memory
  tc_fence_after();
  if (sent[0] != sent[1]) {
    // a wait ran out: the odd CTA may have issued copies to stages that the even
    // one has not armed (where the even one is ahead, the odd one's have landed).
    // Those are armed for it here, and waited for (by an epilogue warp: the
    // control warps have given their registers away)
    if (leader && warp == 4) {
      const CopiesInFlight rest = CopiesInFlight::of(sent[1]).beyond(CopiesInFlight::of(sent[0]));
      auto landed = [&](int s, uint32_t par) { return mbar_try_wait_cluster(&full[s], par); };
      if (lane < STAGES && (rest.stages >> lane & 1u) && !landed(lane, rest.parity >> lane & 1u))
        mbar_expect_tx(&full[lane], (*narrow >> lane & 1u ? 3 : 4) * BOX_BYTES);
      __syncwarp();
      const unsigned long long t0 = global_ns();
      rest.drain(landed, [&] { return global_ns() - t0 > WAIT_LIMIT_NS; });
    }
    cluster_sync_all();
  }
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
}

// One more logit in a running (max, sum of exponentials); one exponential: that
// of the smaller relative to the larger.  (Equal infinities count as 1: where
// the maximum stays -inf the sum is not used.)
__device__ __forceinline__ void add_logit(float l, float& m, float& sum) {
  const float d = l == m ? 0.f : l - m;
  const float e = ex2(-fabsf(d) * LOG2E);
  sum = l > m ? fmaf(sum, e, 1.f) : sum + e;
  m = fmaxf(m, l);
}

// Two running (max, sum) as one.
__device__ __forceinline__ void merge(float& m, float& sum, float om, float os) {
  const float nm = fmaxf(m, om), base = nm == -INFINITY ? 0.f : nm;
  sum = sum * ex2((m - base) * LOG2E) + os * ex2((om - base) * LOG2E);
  m = nm;
}

// A row's target, -1 where it has none.
__device__ __forceinline__ int target_of(const void* ids, int id_bytes, int i, int vocab) {
  const long long t = load_id(ids, id_bytes, i);
  return t >= 0 && t < vocab ? (int)t : -1;
}

// ---------------------------------------------------------------------------
// LSE and PROB for few rows (at most NT): bound by reading the head once, so
// the head is the 128-row operand of one CTA and the hidden rows are the N =
// NT columns: the shared memory holds almost only head tiles in flight (NT =
// 64: 9 stages of 16 + 8 KB; NT = 16: 12 stages of 16 + 2 KB, against 96 KB
// of head per SM in the pair kernel), and the products cost next to nothing.
// Thread = vocabulary entry; LSE keeps a running (max, sum) per hidden row in
// registers over all tiles of the CTA and joins the 32 lanes at the end.  One
// row against 131072 x 2048: 98 us, 5.5 TB/s.  The loss against 50021 x 2048, in
// whole calls: 1 row 53 us, 16 rows 55 (66 and 68 with 64 columns), 17 to 64
// rows 60; the pair kernel takes 67 for 17 rows and the same 60 from 64 on (fp32
// operands, 17 rows: 312 here, 419 there).

// Entries per block of the few-rows kernel: one block per SM of the B200, in
// steps of 32 (tiles of 128 dealt round leave half of the SMs idle in the last
// round: 50021 entries are 2.6 tiles an SM).
__host__ __device__ inline int few_range(int v) { return ((v + 147) / 148 + 31) / 32 * 32; }

template <int NT>
struct Few {
  static constexpr int H_BYTES = NT * 128;
  static constexpr int STAGE = 2 * BOX_BYTES + H_BYTES;
  static constexpr int N_STAGES = NT == 16 ? 12 : 9;
  static constexpr int ROWS = N_STAGES * STAGE;           // lse, g, target of the rows
  static constexpr int BARS = ROWS + 3 * NT * 4;
  static constexpr int TOTAL = BARS + 512 + 1024;
  // accumulators: a chunk is one or two k-blocks (0.4 us of the head each), shorter
  // than the way from the products to the epilogue and back
  static constexpr int BUFS = NT == 16 ? 8 : 4;
  static constexpr int COLS = BUFS * NT;   // TMEM columns
  static_assert(TOTAL <= 227 * 1024, "shared memory per CTA");
};
constexpr int FEW_THREADS = 256;     // warp 0 copies, warp 1 products, warps 4..7 epilogue
constexpr int FEW_ROWS = 64;

template <int ROLE, int NT>
__global__ void __launch_bounds__(FEW_THREADS, 1)
    token_loss_few_kernel(const __grid_constant__ LossMaps maps, const LossParams p) {
  using SM = Few<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_lse = reinterpret_cast<float*>(smem + SM::ROWS);
  float* s_g = s_lse + NT;
  int* s_target = reinterpret_cast<int*>(s_g + NT);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::BARS);
  uint64_t* empty = full + SM::N_STAGES;
  uint64_t* tfull = empty + SM::N_STAGES;
  uint64_t* tempty = tfull + SM::BUFS;
  uint64_t* drain = tempty + SM::BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ unsigned skip_cta;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool own_order = ROLE == LSE && p.ids != nullptr;
  const int nv = own_order ? p.n_rows : *p.n_valid;
  __shared__ unsigned s_err;
  unsigned* const err = own_order ? &s_err : p.err;   // own_order: the first kernel of the call, nothing is cleared yet
  if (threadIdx.x == 0) {
    s_err = 0;
    skip_cta = own_order ? 0 : *reinterpret_cast<volatile unsigned*>(p.err) & ERR_WAIT_TIMEOUT_MASK;
    for (int s = 0; s < SM::N_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < SM::BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < NT) {
    const bool in = (int)threadIdx.x < nv;
    s_target[threadIdx.x] = !in ? -1 : (own_order ? target_of(p.ids, p.id_bytes, threadIdx.x, p.vocab) : p.target[threadIdx.x]);
    s_lse[threadIdx.x] = ROLE == PROB && in ? p.lse[threadIdx.x] : 0.f;
    s_g[threadIdx.x] = ROLE == PROB && in ? p.g[threadIdx.x] : 0.f;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(SM::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int kblocks = (p.d + BK - 1) / BK;
  // the CTA's entries: as even as 32 rows (a box) allow
  const int per = few_range(p.vc);
  const int v0 = min((int)blockIdx.x * per, p.vc);
  const int v1 = skip_cta || (ROLE == LSE && nv == 0) ? v0 : min(v0 + per, p.vc);   // PROB: P is read in any case

  if (warp == 0) {
    const bool issuer = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    CopiesInFlight copies;
    bool ok = true;
    for (int t = v0; t < v1 && ok; t += 128) {
      const int v = p.v0 + t, boxes = (min(v1 - t, 128) + 31) / 32;
      for (int kb = 0, q = p.planes - 1; kb < kblocks;) {
        if (!wait_warp<false>(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
        uint8_t* sa = smem + stage * SM::STAGE;
        if (issuer && !p.debug_no_loads) {
          mbar_expect_tx(&full[stage], boxes * (BOX_BYTES / 2) + SM::H_BYTES);
          for (int h = 0; h < boxes; ++h)
            tma_load_3d(&maps.b, &full[stage], sa + h * (BOX_BYTES / 2), kb * BK, v + 32 * h, q);
          tma_load_3d(&maps.a, &full[stage], sa + 2 * BOX_BYTES, kb * BK, 0, q);
        }
        if (!p.debug_no_loads) copies.issued(stage, phase);
        if (++stage == SM::N_STAGES) { stage = 0; phase ^= 1; }
        if (--q < 0) { q = p.planes - 1; ++kb; }
      }
    }
    if (!ok) {
      if (issuer) atomicOr(err, 1u);
      *abort_flag = 1;
    }
    {   // every issued copy lands before the CTA ends
      const unsigned long long t0 = global_ns();
      copies.drain([&](int s, uint32_t par) { return mbar_try_wait(&full[s], par); },
                   [&] { return global_ns() - t0 > WAIT_LIMIT_NS; });
    }
  } else if (warp == 1) {
    const bool issuer = elect_one();
    constexpr uint32_t IDESC = idesc_f16(NT, 1, 128);
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = v0; t < v1 && ok; t += 128) {
      for (int it = 0; it < kblocks && ok;) {
        if (!wait_warp<false>(&tempty[buf], acc_phase ^ 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * NT);
        const int end = min(kblocks, it + p.chunk);
        auto product = [&](int sa, int sb, bool add) {   // of the head tile of one stage and the rows of another
          const uint32_t a = smem_u32(smem + sa * SM::STAGE), b = smem_u32(smem + sb * SM::STAGE) + 2 * BOX_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_f16(d_tmem, sw128_desc(a + kk * 32), sw128_desc(b + kk * 32), IDESC, (add || kk > 0) ? 1u : 0u);
        };
        for (int first = it; it < end && ok; ++it) {
          int lo = stage, mid = stage;   // as in the pair kernel
          for (int q = p.planes - 1; q >= 0; --q) {
            if (!wait_warp<false>(&full[stage], phase, abort_flag)) { ok = false; break; }
            if (q == 1) mid = stage;
            if (q == 0) {
              tc_fence_after();
              if (issuer) {
                if (p.planes == 3) {
                  product(stage, lo, it > first);
                  product(lo, stage, true);
                  mma_commit(&empty[lo]);
                  product(mid, mid, true);
                  product(stage, mid, true);
                  product(mid, stage, true);
                  mma_commit(&empty[mid]);
                }
                product(stage, stage, p.planes == 3 || it > first);
                mma_commit(&empty[stage]);
              }
            }
            if (++stage == SM::N_STAGES) { stage = 0; phase ^= 1; }
          }
        }
        if (!ok) break;
        if (issuer) mma_commit(&tfull[buf]);
        if (++buf == SM::BUFS) { buf = 0; acc_phase ^= 1; }
      }
    }
    if (!ok) {
      if (issuer) atomicOr(err, 2u);
      *abort_flag = 1;
    }
    if (issuer) mma_commit(drain);   // no product still writes TMEM when it is freed
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(drain, 0)) {
      if (global_ns() - t0 > WAIT_LIMIT_NS) break;
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3;
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    float m[ROLE == LSE ? NT : 1], sum[ROLE == LSE ? NT : 1];
    if constexpr (ROLE == LSE) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        m[i] = -INFINITY;
        sum[i] = 0.f;
      }
    }
    for (int t = v0; t < v1 && ok; t += 128) {
      const int v = t + quarter * 32 + lane;   // in the piece
      float acc[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = 0.f;
      for (int it = 0; it < kblocks; it += p.chunk) {
        if (!wait_warp<false>(&tfull[buf], acc_phase, abort_flag)) {
          if (lane == 0) atomicOr(err, 4u);
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * NT);
#pragma unroll
        for (int c = 0; c < NT / 16; ++c) {
          float x[16];
          tmem_ld16(tbase + (uint32_t)(c * 16), x);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c * 16 + i] += x[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
        if (++buf == SM::BUFS) { buf = 0; acc_phase ^= 1; }
      }
      if (!ok) break;
      const bool in = v < v1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float l = acc[i] * p.scale;
        const bool hit = s_target[i] == p.v0 + v;
        if constexpr (ROLE == LSE) {
          if (in) add_logit(l, m[i], sum[i]);
          if (hit && in) p.target_logit[i] = l;
        } else {
          const float g = s_g[i];
          float x = g * ex2((l - s_lse[i]) * LOG2E);
          if (hit) x -= g;
          acc[i] = g == 0.f ? 0.f : x;
        }
      }
      if constexpr (ROLE == PROB) {
        // fp32 operands: a plane a term; bf16: two terms side by side
        const int terms = p.planes == 3 ? 3 : 2;
        for (int q = 0; q < terms; ++q) {
          bf16* dst = p.p_out + (p.planes == 3 ? ((long long)q * p.vc + v) * NT : ((long long)v * 2 + q) * NT);
#pragma unroll
          for (int i = 0; i < NT; i += 8) {
            Vec8<bf16> y;
            y.set(acc + i);
            if (in) y.store(dst + i);
            float hi[8];
            y.get(hi);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[i + k] -= hi[k];
          }
        }
      }
    }
    if constexpr (ROLE == LSE) {
      // over the lanes: at each step a lane keeps half of its rows (those whose
      // number has the lane's bit), so that NT rows take about NT merges, not 5 NT
      constexpr int W = NT < 32 ? NT : 32;
#pragma unroll
      for (int o = W / 2, n = NT; o; o >>= 1, n >>= 1) {
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
          if (i < n / 2) {
            const int at = i / o * 2 * o + i % o;
            const bool up = lane & o;
            const float om = __shfl_xor_sync(0xffffffffu, up ? m[at] : m[at + o], o);
            const float os = __shfl_xor_sync(0xffffffffu, up ? sum[at] : sum[at + o], o);
            m[i] = up ? m[at + o] : m[at];
            sum[i] = up ? sum[at + o] : sum[at];
            merge(m[i], sum[i], om, os);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NT / W; ++i) {   // row 32 i + lane (16 rows: lane mod 16)
#pragma unroll
        for (int o = 16; o >= W; o >>= 1)
          merge(m[i], sum[i], __shfl_xor_sync(0xffffffffu, m[i], o), __shfl_xor_sync(0xffffffffu, sum[i], o));
        const int row = i * W + lane;
        if (lane < W && row < p.part_pitch)
          p.part[(long long)(blockIdx.x * 4 + quarter) * p.part_pitch + row] = make_float2(m[i], sum[i]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (own_order && threadIdx.x == 0) p.block_err[blockIdx.x] = s_err;
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(SM::COLS) : "memory");
  }
}

// ---------------------------------------------------------------------------
// LSE and PROB of up to 16 fp32 rows: bound by reading the fp32 head once, which
// splitting it into bf16 terms would not allow.  Plain fp32 multiply-adds: the
// hidden rows in shared memory, a warp four vocabulary entries at a time so that
// every value read from there meets four head values; the 4 x NT sums are spread
// over the lanes while they are added up across the warp, and each lane keeps
// (max, sum) of one row.  The gradient's logits come from here too: they have to
// be the very numbers that the lse was made of, or the difference (1e-6 of a
// logit of 14) shows in P.
// The loss against 50021 x 2048 (410 MB: 64 us), in whole calls: 1 to 4 rows 104
// to 106 us, 5 to 16 rows 180 to 187 (shared memory: each head value meets NT
// rows); four rows through the form of 16 177, 1 to 16 rows through the three
// terms 297 to 300.
constexpr int F32_FEW_ROWS = 16;
constexpr int F32_FEW_SMEM = 200 * 1024;
constexpr int F32_FEW_THREADS = 384;   // 168 registers: all but 56 to 84 bytes of 16 rows' sums stay in them

// Sum over the lanes of N values each; lane l ends with values l, l + 32, ...
// (N a multiple of 32) in v[0 .. N/32-1].
template <int N>
__device__ __forceinline__ void spread_sum(float* v, int lane) {
#pragma unroll
  for (int o = 16, n = N; o; o >>= 1, n >>= 1) {
    // keep the half of the values whose index has the lane's bit o
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (i < n / 2) {
        // indices are blocks of 32: bit o of the index <-> bit o of the lane
        const int blk = i / o, in = i % o;
        const float a = v[blk * 2 * o + in], b = v[blk * 2 * o + in + o];
        const bool up = lane & o;
        const float mine = up ? b : a, other = up ? a : b;
        v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
      }
    }
  }
}

template <int ROLE, int NT>
__global__ void __launch_bounds__(F32_FEW_THREADS, 1) token_loss_f32_few_kernel(const LossParams p, const float* hidden,
                                                                               const float* head) {
  extern __shared__ __align__(16) float s_h[];   // [NT][d]
  constexpr int N = 4 * NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = p.d;
  for (int k = threadIdx.x * 4; k < NT * d; k += F32_FEW_THREADS * 4) {
    const int r = k / d, c = k - r * d;
    // a row without a target counts for nothing, whatever it holds
    const bool ok = ROLE == LSE ? r < p.n_rows && target_of(p.ids, p.id_bytes, r, p.vocab) >= 0 : r < *p.n_valid;
    *reinterpret_cast<float4*>(s_h + k) =
        ok ? *reinterpret_cast<const float4*>(hidden + (long long)(ROLE == LSE ? r : p.perm[r]) * d + c)
           : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  // value i = 32 u + lane of the sums: entry i / NT, row i % NT
  constexpr int U = N / 32 > 0 ? N / 32 : 1;
  const int row = lane % NT;
  const int target = row >= p.n_rows ? -1 : (ROLE == LSE ? target_of(p.ids, p.id_bytes, row, p.vocab) : p.target[row]);
  const float weight = ROLE == PROB && row < p.n_rows ? p.g[row] : 0.f, lse = ROLE == PROB && row < p.n_rows ? p.lse[row] : 0.f;
  float m = -INFINITY, sum = 0.f;
  const int groups = (p.vc + 3) / 4;
  const float* piece = head + (long long)p.v0 * d;
  for (int g = blockIdx.x * (F32_FEW_THREADS / 32) + warp; g < groups; g += gridDim.x * (F32_FEW_THREADS / 32)) {
    const float* w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = piece + (long long)min(4 * g + e, p.vc - 1) * d;
    float2 acc[4][NT];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[e][n] = make_float2(0.f, 0.f);
    float4 next[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      next[e] = lane * 4 < d ? __ldg(reinterpret_cast<const float4*>(w[e] + lane * 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = lane * 4; c < d; c += 128) {
      float4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = next[e];
        if (c + 128 < d) next[e] = __ldg(reinterpret_cast<const float4*>(w[e] + c + 128));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 h = *reinterpret_cast<const float4*>(s_h + n * d + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[e][n] = __ffma2_rn(make_float2(x[e].x, x[e].y), make_float2(h.x, h.y), acc[e][n]);
          acc[e][n] = __ffma2_rn(make_float2(x[e].z, x[e].w), make_float2(h.z, h.w), acc[e][n]);
        }
      }
    }
    float v[N < 32 ? 32 : N];
#pragma unroll
    for (int i = 0; i < (N < 32 ? 32 : N); ++i) v[i] = i < N ? acc[i / NT % 4][i % NT].x + acc[i / NT % 4][i % NT].y : 0.f;
    spread_sum<(N < 32 ? 32 : N)>(v, lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = 32 * u + lane, entry = 4 * g + i / NT;
      if (i < N && entry < p.vc) {
        const float l = v[u] * p.scale;
        if constexpr (ROLE == LSE) {
          add_logit(l, m, sum);
          if (entry == target) p.target_logit[row] = l;
        } else if (row < p.n_rows) {
          float x = weight * ex2((l - lse) * LOG2E);
          if (p.v0 + entry == target) x -= weight;
          if (weight == 0.f) x = 0.f;
#pragma unroll
          for (int q = 0; q < 3; ++q) {   // as the few-rows kernel leaves it: [term][entry][16]
            const bf16 y = __float2bfloat16_rn(x);
            p.p_out[((long long)q * p.vc + entry) * 16 + row] = y;
            x -= __bfloat162float(y);
          }
        }
      }
    }
  }
  if (ROLE != LSE) return;
  // lanes of the same row
#pragma unroll
  for (int o = 16; o >= NT; o >>= 1) {
    merge(m, sum, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, sum, o));
  }
  if (lane < NT && row < p.n_rows)
    p.part[(long long)(blockIdx.x * (F32_FEW_THREADS / 32) + warp) * p.part_pitch + row] = make_float2(m, sum);
  if (threadIdx.x == 0) p.block_err[blockIdx.x] = 0;
}

// ---------------------------------------------------------------------------
// Row order: rows with a target first, in their order; the others fill the
// end backwards.  Copies the hidden rows there as bf16 (fp32 rows as three
// terms); rows without a target are written as zeros.
struct RowParams {
  int n, d, vocab, rows_per_block;
  int clear_err;
  int twice;                  // few bf16 rows: rows 0 .. twice-1, zeros behind the last, and the same again
  const void* targets; int target_bytes;
  const void* hidden;
  bf16* rows; int pitch;      // [planes][n][pitch]
  int* perm; int* target; int* n_valid;
  const int2* counts;         // many rows: rows with a target and the largest |weight| (its bits) of every 1024 rows
  // gradient: weights divided by the largest magnitude (so that a weight that
  // is the same for all rows leaves P at exact multiples), lse gathered
  const float* d_loss; const float* lse_in; float* g; float* lse; float* g_max;
  // loss: outputs of rows without a target
  float* loss_out; float* lse_out;
  unsigned* err;
};

__device__ __forceinline__ void split3(float x, bf16& hi, bf16& mid, bf16& lo) {
  hi = __float2bfloat16_rz(x);   // toward zero: the largest fp32 numbers stay finite
  const float r = x - __bfloat162float(hi);
  mid = __float2bfloat16_rn(r);
  lo = __float2bfloat16_rn(r - __bfloat162float(mid));
  if (!isfinite(x)) mid = lo = __float2bfloat16_rn(0.f);   // inf - inf would be NaN
}

// The larger one; infinities and NaN do not count (the weight of one row must
// not scale the others').
__device__ __forceinline__ float max_finite(float a, float b) { return b > a && b < INFINITY ? b : a; }

// counts[k]: rows with a target among 1024 k .. 1024 k + 1023, and their largest
// |weight|.  Without it every block of order_rows looks through all rows, which
// is cheap for few of them only.
constexpr int COUNT_ROWS = 1024;
__global__ void __launch_bounds__(COUNT_ROWS) count_rows_kernel(const RowParams p, int2* counts) {
  __shared__ float s_max[32];
  const int i = blockIdx.x * COUNT_ROWS + threadIdx.x;
  const bool ok = i < p.n && target_of(p.targets, p.target_bytes, i, p.vocab) >= 0;
  float gm = ok && p.d_loss ? fabsf(p.d_loss[i]) : 0.f;
  const int count = __syncthreads_count(ok);
#pragma unroll
  for (int o = 16; o; o >>= 1) gm = max_finite(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = gm;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) gm = max_finite(gm, s_max[w]);
    counts[blockIdx.x] = make_int2(count, __float_as_int(gm));
  }
}

template <typename T>
__global__ void __launch_bounds__(256) order_rows_kernel(const RowParams p) {
  __shared__ int s_count[8];
  __shared__ float s_max[8];
  __shared__ int s_slot[64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * p.rows_per_block;
  const int rows = max(p.n, p.twice), nr = min(p.rows_per_block, rows - r0);
  auto valid = [&](int i) { return i < p.n && target_of(p.targets, p.target_bytes, i, p.vocab) >= 0; };
  int before = 0;
  float gm = 0.f;
  if (p.counts) {
    const int here = r0 / COUNT_ROWS;
    for (int k = threadIdx.x; k < (p.n + COUNT_ROWS - 1) / COUNT_ROWS; k += 256) {
      const int2 c = p.counts[k];
      if (k < here) before += c.x;
      gm = max_finite(gm, __int_as_float(c.y));
    }
    for (int i = here * COUNT_ROWS + threadIdx.x; i < r0; i += 256) before += valid(i);
  } else {
    const int scan = p.d_loss ? p.n : min(r0, p.n);
    for (int i0 = threadIdx.x; i0 < scan; i0 += 4 * 256) {   // four rows in flight
      bool ok[4];
      float g[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 256;
        ok[u] = i < scan && valid(i);
        g[u] = p.d_loss && i < scan ? fabsf(p.d_loss[i]) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        before += ok[u] && i0 + u * 256 < r0;
        if (ok[u]) gm = max_finite(gm, g[u]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    gm = max_finite(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  }
  if (lane == 0) { s_count[warp] = before; s_max[warp] = gm; }
  __syncthreads();
  before = 0;
  gm = 0.f;
  for (int w = 0; w < 8; ++w) {
    before += s_count[w];
    gm = max_finite(gm, s_max[w]);
  }
  if (threadIdx.x == 0 && blockIdx.x == 0) {
    if (p.clear_err) *p.err = 0;
    if (p.d_loss) *p.g_max = gm;
  }
  if (warp == 0) {
    int seen = before;
    for (int b = 0; b < nr; b += 32) {
      const int i = r0 + b + lane;
      const bool here = b + lane < nr;
      const bool ok = here && valid(i);
      const unsigned mask = __ballot_sync(0xffffffffu, ok);
      const int vb = seen + __popc(mask & ((1u << lane) - 1));   // rows with a target before row i
      if (here) {
        const int at = ok ? vb : (i < p.n ? p.n - 1 - (i - vb) : i);
        s_slot[b + lane] = ok ? at : ~at;
      }
      if (here && i < p.n) {
        const int at = ok ? vb : p.n - 1 - (i - vb);
        p.perm[at] = i;
        p.target[at] = ok ? (int)load_id(p.targets, p.target_bytes, i) : -1;
        if (p.d_loss) {
          p.g[at] = !ok ? 0.f : (gm != 0.f ? p.d_loss[i] / gm : p.d_loss[i] * 0.f);
          p.lse[at] = ok ? p.lse_in[i] : 0.f;
        }
        if (p.loss_out && !ok) {
          p.loss_out[i] = 0.f;
          p.lse_out[i] = 0.f;
        }
      }
      seen += __popc(mask);
    }
    if (r0 + nr == rows && lane == 0) *p.n_valid = seen;
  }
  __syncthreads();
  const int vecs = p.d / 8;   // 8 elements per step, four steps in flight
  const long long plane = (long long)p.n * p.pitch;
  const T* src = reinterpret_cast<const T*>(p.hidden) + (long long)r0 * p.d;
  for (int k0 = threadIdx.x; k0 < nr * vecs; k0 += 4 * 256) {
    Vec8<T> x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * 256;
      x[u].zero();
      if (k < nr * vecs && s_slot[k / vecs] >= 0) x[u].load(src + (long long)k * 8);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * 256;
      if (k >= nr * vecs) continue;
      const int r = k / vecs, c = (k - r * vecs) * 8;
      const int at = s_slot[r] >= 0 ? s_slot[r] : ~s_slot[r];
      bf16* dst = p.rows + (long long)at * p.pitch + c;
      if constexpr (sizeof(T) == 2) {
        x[u].store(dst);
        if (p.twice) x[u].store(dst + (long long)p.twice * p.pitch);
      } else {
        float f[8];
        x[u].get(f);
        __align__(16) bf16 t[3][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split3(f[i], t[0][i], t[1][i], t[2][i]);
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4*>(dst + q * plane) = *reinterpret_cast<uint4*>(t[q]);
      }
    }
  }
}

// fp32 head as three bf16 terms, out[3][rows][pitch]: n groups of 8 columns, vecs a row.
__global__ void __launch_bounds__(256) split_terms_kernel(const float* x, bf16* out, long long n, int vecs,
                                                          int pitch) {
  const long long plane = n / vecs * pitch;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = i / vecs;
    const int c = (int)(i - r * vecs) * 8;
    Vec8<float> v;
    v.load(x + i * 8);
    float f[8];
    v.get(f);
    __align__(16) bf16 t[3][8];
#pragma unroll
    for (int k = 0; k < 8; ++k) split3(f[k], t[0][k], t[1][k], t[2][k]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint4*>(out + q * plane + r * pitch + c) = *reinterpret_cast<uint4*>(t[q]);
  }
}

// Joins the (max, sum) of each row: rb rows per block, 1024 / rb threads share a
// row's parts and meet in shared memory.  The order of the sums is fixed.
// Ordered rows: n_valid of them, their places in perm.  Rows in their own order
// (ids): those with a target; the blocks' error words become the call's.
struct JoinParams {
  const float2* part; int part_pitch; int n_parts;
  const float* target_logit; const int* n_valid; const int* perm;
  int rb;
  float* loss; float* lse;
  unsigned* err;
  const void* ids; int id_bytes; int n, vocab; const unsigned* block_err; int blocks;
};

__global__ void __launch_bounds__(1024) join_lse_kernel(const JoinParams p) {
  __shared__ float2 s[1024];
  const int x = threadIdx.x % p.rb, y = threadIdx.x / p.rb, ny = 1024 / p.rb;
  const int row = blockIdx.x * p.rb + x;
  const bool in = p.ids ? row < p.n && target_of(p.ids, p.id_bytes, row, p.vocab) >= 0 : row < *p.n_valid;
  bool bad;
  if (p.ids) {
    const unsigned e = (int)threadIdx.x < p.blocks ? p.block_err[threadIdx.x] : 0;
    bad = __syncthreads_or(e != 0) != 0;
    if (threadIdx.x == 0 && blockIdx.x == 0) *p.err = bad;
  } else {
    bad = *p.err != 0;
  }
  float m = -INFINITY, sum = 0.f;
  if (in) {
    for (int i0 = y; i0 < p.n_parts; i0 += 8 * ny) {   // eight at a time: one running maximum for all
      float2 o[8];
      float nm = m;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * ny;
        o[u] = i < p.n_parts ? p.part[(long long)i * p.part_pitch + row] : make_float2(-INFINITY, 0.f);
        nm = fmaxf(nm, o[u].x);
      }
      const float base = nm == -INFINITY ? 0.f : nm;
      sum *= ex2((m - base) * LOG2E);
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += o[u].y * ex2((o[u].x - base) * LOG2E);
      m = nm;
    }
  }
  s[threadIdx.x] = make_float2(m, sum);
  __syncthreads();
  for (int h = ny / 2; h; h >>= 1) {
    if (y < h) {
      merge(m, sum, s[threadIdx.x + h * p.rb].x, s[threadIdx.x + h * p.rb].y);
      s[threadIdx.x] = make_float2(m, sum);
    }
    __syncthreads();
  }
  if (y != 0) return;
  if (in) {
    const float ls = logf(sum);
    const int at = p.ids ? row : p.perm[row];
    p.loss[at] = bad ? NAN : (m - p.target_logit[row]) + ls;
    p.lse[at] = bad ? NAN : m + ls;
  } else if (p.ids && row < p.n) {
    p.loss[row] = 0.f;
    p.lse[row] = 0.f;
  }
}

// Partial sums of a gradient, [splits][rows][d], added in order, times the
// weights' common factor.  Rows of dH go to their places (perm), those without
// a target become zero, and with two terms of P a row is the sum of two.  G
// groups of splits side by side, 1024 / G columns a block and step.  After a
// wait that ran out: NaN here and in all of `head`, where that is given.
struct JoinRows {
  const float* part; int splits, rows, pitch, two_terms, n, d;
  const int* perm; const int* n_valid;
  const float* g_max; float scale;
  const unsigned* err;
  void* out; void* head; long long head_n;
};

template <typename T, int G>
__global__ void __launch_bounds__(256) join_rows_kernel(const JoinRows p) {
  constexpr int X = 256 / G;
  __shared__ float4 s[G][X];
  const int x = threadIdx.x % X, y = threadIdx.x / X;
  const bool bad = *p.err != 0;
  if (bad && p.head) {
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < p.head_n; i += (long long)gridDim.x * 256)
      reinterpret_cast<T*>(p.head)[i] = (T)NAN;
  }
  if (!p.out) return;
  const int nv = p.perm ? *p.n_valid : p.n;
  const float f = *p.g_max * p.scale;
  const int vecs = p.d / 4, per = (p.splits + G - 1) / G;
  const long long total = (long long)p.n * vecs, plane = (long long)p.rows * p.pitch;
  for (long long k0 = (long long)blockIdx.x * X; k0 < total; k0 += (long long)gridDim.x * X) {
    const long long k = k0 + x;
    const int r = (int)(k / vecs), c = (int)(k - (long long)r * vecs) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float4 a) { v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w; };
    if (k < total && r < nv) {
#pragma unroll 4
      for (int i = y * per; i < min(p.splits, (y + 1) * per); ++i) {
        const float* at = p.part + i * plane + (long long)r * p.pitch + c;
        add(*reinterpret_cast<const float4*>(at));
        if (p.two_terms) add(*reinterpret_cast<const float4*>(at + (long long)p.two_terms * p.pitch));
      }
    }
    if constexpr (G > 1) {
      __syncthreads();
      s[y][x] = v;
      __syncthreads();
      if (y == 0)
        for (int g = 1; g < G; ++g) add(s[g][x]);
    }
    if (y == 0 && k < total) {
      v.x *= f; v.y *= f; v.z *= f; v.w *= f;
      if (r >= nv) v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (bad) v = make_float4(NAN, NAN, NAN, NAN);
      T* dst = reinterpret_cast<T*>(p.out) + (long long)(p.perm ? p.perm[r] : r) * p.d + c;
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        *reinterpret_cast<float4*>(dst) = v;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int COUNTED_FROM = 2048;                 // rows from which they are counted first (8192 rows: 19 + 4 us, 37 without)
constexpr int LOSS_ROWS = 8192;                    // rows per forward pass: bounds the (max, sum) workspace
constexpr long long P_BYTES = 256ll << 20;         // P of one vocabulary piece, where 256 columns fit

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
int round_up(int a, int b) { return (a + b - 1) / b * b; }
int div_up(int a, int b) { return (a + b - 1) / b; }

int few_blocks(int v) { return div_up(v, few_range(v)); }

// Whether the logits of fp32 rows run on plain multiply-adds (the rows have to
// fit the shared memory, up to 3200 columns for 16 of them).
int f32_few_rows(int n) { return n <= 4 ? 4 : F32_FEW_ROWS; }
bool f32_few(bool f32, int n, int d) {
  return f32 && n <= F32_FEW_ROWS && (size_t)f32_few_rows(n) * d * 4 <= F32_FEW_SMEM;
}

// Columns of the few-rows kernel's products.
int few_cols(int n) { return n <= 16 ? 16 : FEW_ROWS; }

// Columns of a tile of logits: 256; 128 where those would leave most of the
// device idle (the products' time is the tile's, its copies' less than halved).
int logit_tile(int n, int v) { return div_up(n, TILE) * div_up(v, TILE) * 2 <= 74 ? 128 : 256; }

// Workspace of one call, laid out in order.
struct Layout {
  int planes, dp, dq, rows, g_rows, two_terms, pieces, vc, splits, k_split, dw_splits, dw_k, n_parts;
  size_t block_err, counts, n_valid, g_max, rows_b, perm, target, g, lse, tlogit, part, head, p, dh, dw, total;
  Layout(int n, int v, int d, bool f32, bool grad) {
    planes = f32 ? 3 : 1;
    dp = round_up(d, 64);   // rows kept here start on 128-byte lines: a copied box row is one line, not two
    dq = round_up(d, 32);   // (834 rows, 96794 x 1032: 181 us off the lines, 156 on them)
    // P beside bf16 operands is one bf16 term; for few rows two (few roundings do
    // not average out, and the products are not what bounds the gradient): the
    // second terms stand as further rows of P, beside the same hidden rows again
    two_terms = grad && !f32 && n <= FEW_ROWS ? few_cols(n) : 0;
    g_rows = two_terms ? 2 * two_terms : n;
    const bool simt = f32_few(f32, n, d);
    rows = grad ? n : (n < LOSS_ROWS ? n : LOSS_ROWS);
    n_parts = simt ? 148 * (F32_FEW_THREADS / 32)
                   : (n <= FEW_ROWS ? 4 * few_blocks(v) : logit_tile(rows, v) / 128 * div_up(v, logit_tile(rows, v)));
    vc = v; pieces = 1; splits = k_split = dw_k = 0; dw_splits = 1;
    if (grad) {
      long long w = P_BYTES / ((long long)g_rows * 2 * planes) / TILE * TILE;
      if (w < TILE) w = TILE;
      if (w < v) {
        pieces = div_up(v, (int)w);
        vc = round_up(div_up(v, pieces), TILE);
        pieces = div_up(v, vc);
      }
      // dH tiles contract over the piece in splits, so that a launch has about four
      // tiles of equal work per CTA pair; of 256 to 8192 columns each
      const long long mt = div_up(g_rows, TILE), dt = div_up(d, TILE), nt = div_up(vc, TILE);
      const long long blocks = dt * (mt * div_up(vc, BK) + nt * div_up(g_rows, BK));
      const long long want = blocks / (4 * 74);
      const int ks = BK * (int)(want < 4 ? 4 : (want > 128 ? 128 : want));
      // dW likewise where its tiles alone would not fill the device
      if (nt * dt * 2 <= 74 && g_rows > 512) {
        const int most = div_up(g_rows, 256), fill = div_up(74, (int)(nt * dt));
        dw_splits = most < fill ? most : fill;
      }
      dw_k = round_up(div_up(g_rows, dw_splits), BK);
      dw_splits = div_up(g_rows, dw_k);
      splits = div_up(vc, ks);
      k_split = round_up(div_up(vc, splits), BK);
      splits = div_up(vc, k_split);
    }
    size_t o = 256;   // the error word
    auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
    block_err = take(148 * 4);
    counts = take(rows > COUNTED_FROM ? (size_t)div_up(rows, COUNT_ROWS) * 8 : 0);
    n_valid = take(4);
    g_max = take(4);
    rows_b = take((size_t)planes * (grad ? g_rows : rows) * dp * 2);
    perm = take((size_t)rows * 4);
    target = take((size_t)rows * 4);
    g = take(grad ? (size_t)rows * 4 : 0);
    lse = take(grad ? (size_t)rows * 4 : 0);
    tlogit = take(grad ? 0 : (size_t)rows * 4);
    part = take(grad ? 0 : (size_t)n_parts * rows * 8);
    head = take(f32 && (grad || !simt) ? (size_t)3 * v * dp * 2 : 0);
    p = take(grad ? (size_t)planes * (two_terms ? g_rows : (n <= FEW_ROWS ? few_cols(n) : n)) * round_up(vc, 64) * 2 : 0);
    dh = take(grad ? (size_t)splits * g_rows * dq * 4 : 0);
    dw = take(dw_splits > 1 ? (size_t)dw_splits * vc * dq * 4 : 0);
    total = o;
  }
};

// [outer][rows][inner] with rows `pitch` elements apart, box box_inner x box_rows, 128-byte swizzle.
cudaError_t make_map(CUtensorMap* map, const void* base, bool f32, int inner, long long pitch, int rows, int outer,
                     int box_inner, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = get_tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t esz = f32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[2] = {(cuuint64_t)pitch * esz, (cuuint64_t)pitch * rows * esz};
  cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t load_map(CUtensorMap* map, const void* base, int inner, long long pitch, int rows, int outer) {
  return make_map(map, base, false, inner, pitch, rows, outer, BK, 64);
}

// Pairs of CTAs the device runs at once, per device (set up on first use).
template <int ROLE>
cudaError_t pairs_on_device(int* out) {
  constexpr int MAX_DEVICES = 64;
  static std::mutex mu;
  static int known[MAX_DEVICES] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    e = cudaFuncSetAttribute(token_loss_kernel<ROLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<ROLE>::TOTAL);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(NUM_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Smem<ROLE>::TOTAL;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2; attr.val.clusterDim.y = 1; attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, token_loss_kernel<ROLE>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    known[dev] = n;
  }
  *out = known[dev];
  return cudaSuccess;
}

template <int ROLE, int NT>
cudaError_t launch_few(const LossMaps& maps, const LossParams& p, cudaStream_t st) {
  // an attribute of the function on this device; cheap, so set at every launch
  cudaError_t e = cudaFuncSetAttribute(token_loss_few_kernel<ROLE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Few<NT>::TOTAL);
  if (e != cudaSuccess) return e;
  token_loss_few_kernel<ROLE, NT><<<few_blocks(p.vc), FEW_THREADS, Few<NT>::TOTAL, st>>>(maps, p);
  return cudaGetLastError();
}

template <int ROLE, int NT>
cudaError_t launch_f32_few(const LossParams& p, const void* hidden, const void* head, cudaStream_t st) {
  const int smem = NT * p.d * 4;
  // always the most: other threads may launch other sizes between this and the launch
  cudaError_t e = cudaFuncSetAttribute(token_loss_f32_few_kernel<ROLE, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, F32_FEW_SMEM);
  if (e != cudaSuccess) return e;
  token_loss_f32_few_kernel<ROLE, NT><<<148, F32_FEW_THREADS, smem, st>>>(p, (const float*)hidden, (const float*)head);
  return cudaGetLastError();
}

// k-blocks per accumulator of the logits.  Few rows, K = 64 or 128: the truncation
// of longer ones shows: a row's loss is a small difference of two logits, and of
// one row nothing averages out (error of the loss of one row against 64 bits,
// 12 inputs: K = 64 2.4e-7 in 98 us, K = 128 2.8e-7 in 94, K = 256 7.2e-7 in
// 86; the plain fp32 form 2.0e-7).
// The same for the loss and the gradient, whose P is made of exp(l - lse): with
// the very logits that the lse is made of their errors cancel in 1 - p of a sure
// target, with others (one accumulator over the whole width) they do not.  Rows
// with 1 - p near 2e-4, error of their d_hidden: 4e-3 to 1e-2, against 0.44 (d =
// 2048) and 2.1 (d = 8192), for 1 to 2 % of the gradient's time.
int logit_chunk(int n, int planes) {
  if (planes == 3) return F32_CHUNK;
  return n <= 16 ? 1 : (n <= FEW_ROWS ? 2 : LSE_CHUNK);
}

// The head as the few-rows kernel reads it: boxes of 32 entries.
cudaError_t few_head_map(CUtensorMap* map, const void* head, int v, int d, int pitch, int planes) {
  return make_map(map, head, false, d, pitch, v, planes, BK, 32);
}

// Hidden rows as the few-rows kernel reads them: boxes of NT rows.
cudaError_t few_map(CUtensorMap* map, const void* rows, int n, int d, int pitch, int planes) {
  return make_map(map, rows, false, d, pitch, n, planes, BK, n <= 16 ? 16 : FEW_ROWS);
}

template <int ROLE>
cudaError_t launch_products(const LossMaps& maps, const LossParams& p, long long jobs, cudaStream_t st) {
  int pairs = 0;
  cudaError_t e = pairs_on_device<ROLE>(&pairs);
  if (e != cudaSuccess) return e;
  const int grid = (int)(jobs < pairs ? jobs : pairs);
  token_loss_kernel<ROLE><<<2 * grid, NUM_THREADS, Smem<ROLE>::TOTAL, st>>>(maps, p);
  return cudaGetLastError();
}

cudaError_t launch_join_rows(const JoinRows& jr, bool f32, cudaStream_t st) {
  const bool groups = jr.splits >= 8;
  const long long blocks = ((long long)jr.n * (jr.d / 4) + (groups ? 31 : 255)) / (groups ? 32 : 256);
  const int grid = (int)(blocks < 148 * 16 ? blocks : 148 * 16);
  if (f32 && groups) join_rows_kernel<float, 8><<<grid, 256, 0, st>>>(jr);
  else if (f32) join_rows_kernel<float, 1><<<grid, 256, 0, st>>>(jr);
  else if (groups) join_rows_kernel<bf16, 8><<<grid, 256, 0, st>>>(jr);
  else join_rows_kernel<bf16, 1><<<grid, 256, 0, st>>>(jr);
  return cudaGetLastError();
}

cudaError_t launch_order_rows(RowParams rp, bool f32, int2* counts, cudaStream_t st) {
  rp.rows_per_block = rp.n <= 2048 ? 4 : (rp.n <= 65536 ? 16 : 64);   // both divide COUNT_ROWS
  if (rp.n > COUNTED_FROM) {
    rp.counts = counts;
    count_rows_kernel<<<div_up(rp.n, COUNT_ROWS), COUNT_ROWS, 0, st>>>(rp, counts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int grid = div_up(rp.n > rp.twice ? rp.n : rp.twice, rp.rows_per_block);
  if (f32) order_rows_kernel<float><<<grid, 256, 0, st>>>(rp);
  else order_rows_kernel<bf16><<<grid, 256, 0, st>>>(rp);
  return cudaGetLastError();
}

// The head as the products read it: bf16 as it is, fp32 as three terms.
cudaError_t head_operand(const Layout& L, char* ws, const void* head, int v, int d, bool f32, const void** out,
                         cudaStream_t st) {
  *out = head;
  if (!f32) return cudaSuccess;
  const long long n = (long long)v * (d / 8), blocks = (n + 255) / 256;
  split_terms_kernel<<<(int)(blocks < 148 * 16 ? blocks : 148 * 16), 256, 0, st>>>((const float*)head,
                                                                                (bf16*)(ws + L.head), n, d / 8, L.dp);
  *out = ws + L.head;
  return cudaGetLastError();
}

}  // namespace

}  // namespace armt

using namespace armt;

extern "C" armt_status armt_token_loss_workspace(armt_dtype dtype, int n, int vocab, int d, int grad, size_t* bytes) {
  if (!bytes) return ARMT_ERR_INVALID_ARG;
  *bytes = 0;
  if (grad != 0 && grad != 1) return ARMT_ERR_INVALID_ARG;
  const armt_status s = check_sizes(dtype, n, vocab, d);
  if (s != ARMT_OK) return s;
  *bytes = Layout(n, vocab, d, dtype == ARMT_FP32, grad != 0).total;
  return ARMT_OK;
}

static armt_status token_loss(armt_dtype dtype, int n, int vocab, int d, const void* hidden, const void* head,
                              const void* targets, int target_bytes, float scale, float* loss, float* lse,
                              void* workspace, size_t workspace_bytes, void* stream, int debug_no_loads) {
  armt_status s = check_sizes(dtype, n, vocab, d);
  if (s != ARMT_OK) return s;
  if (!hidden || !head || !targets || !loss || !lse || !workspace || !std::isfinite(scale) ||
      (target_bytes != 4 && target_bytes != 8) || !aligned16(hidden) || !aligned16(head) || !aligned16(workspace) ||
      !aligned_to(targets, target_bytes) || !aligned_to(loss, 4) || !aligned_to(lse, 4))
    return ARMT_ERR_INVALID_ARG;
  const bool f32 = dtype == ARMT_FP32;
  const Layout L(n, vocab, d, f32, false);
  if (workspace_bytes < L.total) return ARMT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  char* ws = (char*)workspace;
  JoinParams jp{};
  jp.part = (const float2*)(ws + L.part); jp.n_parts = L.n_parts; jp.target_logit = (const float*)(ws + L.tlogit);
  jp.err = (unsigned*)ws; jp.vocab = vocab;
  LossParams p{};
  p.d = d; p.vocab = vocab; p.planes = L.planes; p.v0 = 0; p.vc = vocab; p.scale = scale;
  p.debug_no_loads = debug_no_loads;
  p.part = (float2*)(ws + L.part); p.target_logit = (float*)(ws + L.tlogit); p.err = (unsigned*)ws;
  auto join = [&](int rows, int r0) {
    jp.rb = 32;
    while (jp.rb > 1 && jp.rb / 2 >= rows) jp.rb /= 2;
    jp.part_pitch = rows;
    jp.n = rows;
    jp.loss = loss + r0;
    jp.lse = lse + r0;
    join_lse_kernel<<<div_up(rows, jp.rb), 1024, 0, st>>>(jp);
    return cudaGetLastError();
  };
  LossMaps maps{};
  const bool simt = f32_few(f32, n, d);
  if (simt || (!f32 && n <= FEW_ROWS)) {   // few rows, in their own order: two launches
    p.n_rows = p.part_pitch = n;
    p.ids = jp.ids = targets;
    p.id_bytes = jp.id_bytes = target_bytes;
    p.block_err = (unsigned*)(ws + L.block_err);
    jp.block_err = p.block_err;
    p.chunk = logit_chunk(n, L.planes);
    cudaError_t e;
    if (simt) {
      jp.blocks = 148;
      e = n <= 4 ? launch_f32_few<LSE, 4>(p, hidden, head, st) : launch_f32_few<LSE, F32_FEW_ROWS>(p, hidden, head, st);
    } else {
      jp.blocks = few_blocks(vocab);
      e = few_map(&maps.a, hidden, n, d, d, 1);
      if (e == cudaSuccess) e = few_head_map(&maps.b, head, vocab, d, d, 1);
      if (e == cudaSuccess) e = n <= 16 ? launch_few<LSE, 16>(maps, p, st) : launch_few<LSE, 64>(maps, p, st);
    }
    if (e == cudaSuccess) e = join(n, 0);
    return cuda_status(e);
  }
  const void* w = nullptr;
  cudaError_t e = head_operand(L, ws, head, vocab, d, f32, &w, st);
  const bool few = n <= FEW_ROWS;   // up to 64 rows: bound by reading the head
  const int wp = f32 ? L.dp : d;
  if (e == cudaSuccess)
    e = few ? few_head_map(&maps.b, w, vocab, d, wp, L.planes) : load_map(&maps.b, w, d, wp, vocab, L.planes);
  for (int r0 = 0; r0 < n && e == cudaSuccess; r0 += L.rows) {
    const int nr = n - r0 < L.rows ? n - r0 : L.rows;
    RowParams rp{};
    rp.n = nr; rp.d = d; rp.vocab = vocab; rp.clear_err = r0 == 0;
    rp.targets = (const char*)targets + (size_t)r0 * target_bytes; rp.target_bytes = target_bytes;
    rp.hidden = (const char*)hidden + (size_t)r0 * d * (f32 ? 4 : 2);
    rp.rows = (bf16*)(ws + L.rows_b); rp.pitch = L.dp; rp.perm = (int*)(ws + L.perm); rp.target = (int*)(ws + L.target);
    rp.n_valid = (int*)(ws + L.n_valid); rp.err = (unsigned*)ws;
    rp.loss_out = loss + r0; rp.lse_out = lse + r0;
    e = launch_order_rows(rp, f32, (int2*)(ws + L.counts), st);
    if (e == cudaSuccess)
      e = few ? few_map(&maps.a, ws + L.rows_b, nr, d, L.dp, L.planes)
              : load_map(&maps.a, ws + L.rows_b, d, L.dp, nr, L.planes);
    if (e != cudaSuccess) break;
    p.n_rows = p.part_pitch = nr;
    p.n_valid = jp.n_valid = rp.n_valid;
    p.target = rp.target;
    jp.perm = rp.perm;
    p.tile_n = logit_tile(L.rows, vocab);   // the same for every pass: the parts are laid out for it
    p.chunk = logit_chunk(n, L.planes);
    if (few) e = nr <= 16 ? launch_few<LSE, 16>(maps, p, st) : launch_few<LSE, 64>(maps, p, st);
    else e = launch_products<LSE>(maps, p, (long long)div_up(nr, TILE) * div_up(vocab, p.tile_n), st);
    if (e == cudaSuccess) e = join(nr, r0);
  }
  return cuda_status(e);
}

extern "C" armt_status armt_token_loss(armt_dtype dtype, int n, int vocab, int d, const void* hidden, const void* head,
                                       const void* targets, int target_bytes, float scale, float* loss, float* lse,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  return token_loss(dtype, n, vocab, d, hidden, head, targets, target_bytes, scale, loss, lse, workspace,
                    workspace_bytes, stream, 0);
}

extern "C" armt_status armt_token_loss_grad(armt_dtype dtype, int n, int vocab, int d, const void* hidden,
                                            const void* head, const void* targets, int target_bytes, float scale,
                                            const float* lse, const float* d_loss, void* d_hidden, void* d_head,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  armt_status s = check_sizes(dtype, n, vocab, d);
  if (s != ARMT_OK) return s;
  if (!hidden || !head || !targets || !lse || !d_loss || (!d_hidden && !d_head) || !workspace ||
      !std::isfinite(scale) || (target_bytes != 4 && target_bytes != 8) || !aligned16(hidden) || !aligned16(head) ||
      !aligned16(workspace) || !aligned16(d_hidden) || !aligned16(d_head) || !aligned_to(targets, target_bytes) ||
      !aligned_to(lse, 4) || !aligned_to(d_loss, 4))
    return ARMT_ERR_INVALID_ARG;
  const bool f32 = dtype == ARMT_FP32;
  const Layout L(n, vocab, d, f32, true);
  if (workspace_bytes < L.total) return ARMT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  char* ws = (char*)workspace;
  const void* w = nullptr;
  cudaError_t e = head_operand(L, ws, head, vocab, d, f32, &w, st);
  RowParams rp{};
  rp.n = n; rp.d = d; rp.vocab = vocab; rp.clear_err = 1;
  rp.targets = targets; rp.target_bytes = target_bytes; rp.hidden = hidden;
  rp.rows = (bf16*)(ws + L.rows_b); rp.pitch = L.dp; rp.perm = (int*)(ws + L.perm); rp.target = (int*)(ws + L.target);
  rp.n_valid = (int*)(ws + L.n_valid); rp.err = (unsigned*)ws;
  rp.twice = L.two_terms;
  rp.d_loss = d_loss; rp.lse_in = lse; rp.g = (float*)(ws + L.g); rp.lse = (float*)(ws + L.lse);
  rp.g_max = (float*)(ws + L.g_max);
  if (e == cudaSuccess) e = launch_order_rows(rp, f32, (int2*)(ws + L.counts), st);
  const int wp = f32 ? L.dp : d;
  LossMaps mp{}, mg{};   // PROB, GRAD
  if (e == cudaSuccess) e = load_map(&mp.a, ws + L.rows_b, d, L.dp, L.g_rows, L.planes);
  if (e == cudaSuccess) e = load_map(&mp.b, w, d, wp, vocab, L.planes);
  mg.b = mp.b;
  mg.c = mp.a;
  if (e == cudaSuccess && d_head)
    e = L.dw_splits > 1 ? make_map(&mg.out0, ws + L.dw, true, d, L.dq, L.vc, L.dw_splits, 32, 32)
                        : make_map(&mg.out0, d_head, f32, d, d, vocab, 1, f32 ? 32 : 64, 32);
  if (e == cudaSuccess && d_hidden) e = make_map(&mg.out1, ws + L.dh, true, d, L.dq, L.g_rows, L.splits, 32, 32);
  LossParams p{};
  p.n_rows = n; p.d = d; p.vocab = vocab; p.planes = L.planes; p.scale = scale;
  p.n_valid = rp.n_valid; p.perm = rp.perm; p.target = rp.target; p.lse = rp.lse; p.g = rp.g; p.g_max = rp.g_max; p.err = rp.err;
  p.want_dw = d_head != nullptr; p.want_dh = d_hidden != nullptr; p.dw_bf16 = !f32; p.k_split = L.k_split;
  p.dw_splits = L.dw_splits; p.dw_k = L.dw_k;
  const bool few = n <= FEW_ROWS;
  if (e == cudaSuccess && few) e = few_map(&mp.a, ws + L.rows_b, n, d, L.dp, L.planes);
  if (e == cudaSuccess && few) e = few_head_map(&mp.b, w, vocab, d, wp, L.planes);
  const int mt = div_up(L.g_rows, TILE), dt = div_up(d, TILE);
  for (int v0 = 0; v0 < vocab && e == cudaSuccess; v0 += L.vc) {
    p.v0 = v0;
    p.vc = vocab - v0 < L.vc ? vocab - v0 : L.vc;
    p.panels = div_up(p.vc, BK);
    p.splits = div_up(p.vc, L.k_split);
    p.dh_add = v0 > 0;
    if (L.two_terms) e = load_map(&mg.a, ws + L.p, L.g_rows, L.g_rows, p.vc, 1);
    else if (few) e = load_map(&mg.a, ws + L.p, n, few_cols(n), p.vc, L.planes);
    else e = load_map(&mg.a, ws + L.p, 64, 64, n, p.panels * L.planes);
    if (e == cudaSuccess && !few) e = make_map(&mp.out0, ws + L.p, false, 64, 64, n, p.panels * L.planes, 64, 32);
    p.chunk = logit_chunk(n, L.planes);
    const int nt = div_up(p.vc, TILE);
    p.tile_n = logit_tile(n, p.vc);
    p.p_out = (bf16*)(ws + L.p);
    p.p_trans = few;
    if (e == cudaSuccess)
      e = !few ? launch_products<PROB>(mp, p, (long long)mt * div_up(p.vc, p.tile_n), st)
          : f32_few(f32, n, d) ? (n <= 4 ? launch_f32_few<PROB, 4>(p, hidden, head, st)
                                         : launch_f32_few<PROB, F32_FEW_ROWS>(p, hidden, head, st))
               : (n <= 16 ? launch_few<PROB, 16>(mp, p, st) : launch_few<PROB, 64>(mp, p, st));
    LossParams pg = p;
    pg.n_rows = L.g_rows;
    pg.two_terms = L.two_terms;
    pg.chunk = f32 ? F32_CHUNK : GRAD_CHUNK;
    const long long jobs = (p.want_dw ? (long long)nt * dt * L.dw_splits : 0) + (p.want_dh ? (long long)mt * dt * p.splits : 0);
    if (e == cudaSuccess) e = launch_products<GRAD>(mg, pg, jobs, st);
    if (e == cudaSuccess && d_head && L.dw_splits > 1) {
      JoinRows jr{};
      jr.part = (const float*)(ws + L.dw); jr.splits = L.dw_splits; jr.rows = L.vc; jr.pitch = L.dq; jr.n = p.vc; jr.d = d;
      jr.g_max = rp.g_max; jr.scale = scale; jr.err = rp.err;
      jr.out = (char*)d_head + (size_t)v0 * d * (f32 ? 4 : 2);
      e = launch_join_rows(jr, f32, st);
    }
  }
  if (e == cudaSuccess) {
    JoinRows jr{};
    jr.part = (const float*)(ws + L.dh); jr.splits = L.splits; jr.rows = L.g_rows; jr.pitch = L.dq; jr.two_terms = L.two_terms;
    jr.n = n; jr.d = d; jr.perm = rp.perm; jr.n_valid = rp.n_valid; jr.g_max = rp.g_max; jr.scale = scale;
    jr.err = rp.err; jr.out = d_hidden; jr.head = d_head; jr.head_n = (long long)vocab * d;
    e = launch_join_rows(jr, f32, st);
  }
  return cuda_status(e);
}

// Read by the host after the stream has finished: whether a bounded wait ran
// out in the last call that used this workspace.
extern "C" armt_status armt_workspace_status(const void* workspace, void* stream) {
  if (!workspace) return ARMT_ERR_INVALID_ARG;
  unsigned err = 0;
  cudaError_t e = cudaMemcpyAsync(&err, workspace, sizeof(err), cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e);
  return err ? ARMT_ERR_DEVICE_TIMEOUT : ARMT_OK;
}

// The bounded-wait error path on demand: a loss of `rows` zero rows (16 k-blocks,
// more than the stages) whose copies are never issued.  Every wait of the
// products then runs out (about one second), the blocks leave and free their
// tensor memory, the join finds the error and writes NaN.
extern "C" armt_status armt_test_loss_wait(int rows, void* stream) {
  const int v = 600, d = 1024;
  size_t need = 0;
  armt_status s = armt_token_loss_workspace(ARMT_BF16, rows, v, d, 0, &need);
  if (s != ARMT_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const size_t data = ((size_t)rows + v) * d * 2 + (size_t)rows * 16 + 1024;
  char* buf = nullptr;
  cudaError_t e = cudaMallocAsync((void**)&buf, data + need, st);
  if (e != cudaSuccess) return cuda_status(e);
  char* hidden = buf + need;
  char* head = hidden + (size_t)rows * d * 2;
  char* targets = head + (size_t)v * d * 2;
  float* loss = (float*)(targets + (size_t)rows * 8);
  float host = 0.f;
  e = cudaMemsetAsync(buf, 0, data + need, st);
  s = cuda_status(e);
  if (s == ARMT_OK)
    s = token_loss(ARMT_BF16, rows, v, d, hidden, head, targets, 8, 1.f, loss, loss + rows, buf, need, stream, 1);
  if (s == ARMT_OK) s = cuda_status(cudaMemcpyAsync(&host, loss, sizeof(float), cudaMemcpyDeviceToHost, st));
  if (s == ARMT_OK) s = armt_workspace_status(buf, stream);   // waits for the stream
  if (s == ARMT_ERR_DEVICE_TIMEOUT && !std::isnan(host)) s = ARMT_OK;
  cudaFreeAsync(buf, st);
  return s;
}
