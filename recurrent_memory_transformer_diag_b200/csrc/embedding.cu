// Token embedding and the gradient of its table.
//
//   out[n] = scale * table[id_n]                 (0 where id_n is outside [0, V))
//   d_table[v] = (d_table[v]) + scale * sum of d_out[n] over n with id_n = v
//
// Both are bound by memory traffic.  The gradient sums each table row's tokens
// in the order of n, so the result does not depend on the schedule: no
// floating-point atomics.  Two ways, by the number of tokens:
//
//   few tokens: a block owns up to 32 table rows and looks through all ids; one
//     launch, nothing to sort.
//   many tokens: a stable radix sort of (id, n) by 9 bits a pass (in one block
//     up to 8192 tokens); then the
//     sorted list is cut into chunks of 8 to 64 tokens, a worker per chunk adds up
//     its runs of equal ids and writes those that lie inside it.  Runs that
//     cross chunks leave one partial sum per chunk, joined in order by a last
//     kernel, so a token that makes up much of the input is still spread over
//     the device.  Rows that no token names are zeroed by further blocks of
//     the same launch.
#include <cmath>

#include "armt_internal.cuh"
#include "vec8.cuh"

namespace armt {

namespace {

// ---------------------------------------------------------------- lookup
constexpr int LOOKUP_UNROLL = 4;

template <typename T>
__global__ void __launch_bounds__(256) embed_kernel(const void* ids, int id_bytes, const T* table, float scale, T* out,
                                                    long long total, int vecs, int vocab, int d) {
  const long long base = (long long)blockIdx.x * (256 * LOOKUP_UNROLL) + threadIdx.x;
  Vec8<T> x[LOOKUP_UNROLL];
#pragma unroll
  for (int u = 0; u < LOOKUP_UNROLL; ++u) {
    const long long k = base + u * 256;
    x[u].zero();
    if (k < total) {
      const long long row = k / vecs;
      const int c = (int)(k - row * vecs) * 8;
      const long long id = load_id(ids, id_bytes, row);
      if (id >= 0 && id < vocab) x[u].load(table + id * d + c);
    }
  }
#pragma unroll
  for (int u = 0; u < LOOKUP_UNROLL; ++u) {
    const long long k = base + u * 256;
    if (k < total) {
      float v[8];
      x[u].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= scale;
      x[u].set(v);
      x[u].store(out + k * 8);
    }
  }
}

// ---------------------------------------------------------------- gradient, few tokens
// Most tokens for the one-launch gradient.  Its time grows with the tokens of
// one row, which one group of threads adds up: 870 tokens with a few frequent
// ids (table 1323 x 1168) took 148 us here and 22 us sorted; 128 tokens 7 us.
constexpr int SCAN_MAX = 128;
// Table rows of a block: enough blocks for the device where the table is small.
int scan_rows(int vocab) { return vocab >= 32 * 592 ? 32 : (vocab >= 592 ? vocab / 592 : 1); }

template <typename T>
__device__ __forceinline__ void write_row(T* dst, const float* acc, float scale, bool accumulate) {
  float v[8];
  Vec8<T> y;
  if (accumulate) {
    y.load(dst);
    y.get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(acc[i], scale, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = acc[i] * scale;
  }
  y.set(v);
  y.store(dst);
}

template <typename T>
__global__ void __launch_bounds__(256) embed_grad_scan_kernel(const void* ids, int id_bytes, const T* d_out,
                                                              float scale, T* d_table, int n, int vocab, int d,
                                                              int accumulate, int block_rows) {
  __shared__ unsigned char s_n[SCAN_MAX];    // tokens of the block's rows, in order
  __shared__ unsigned char s_row[SCAN_MAX];
  __shared__ int s_warp[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int v0 = blockIdx.x * block_rows;
  int found = 0;
  for (int b = 0; b < n; b += 256) {
    const int i = b + threadIdx.x;
    int r = -1;
    if (i < n) {
      const long long id = load_id(ids, id_bytes, i);
      if (id >= v0 && id < v0 + block_rows && id < vocab) r = (int)(id - v0);
    }
    const unsigned mask = __ballot_sync(0xffffffffu, r >= 0);
    if (lane == 0) s_warp[warp] = __popc(mask);
    __syncthreads();
    int at = found;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) at += s_warp[w];
      found += s_warp[w];
    }
    if (r >= 0) {
      at += __popc(mask & ((1u << lane) - 1));
      s_n[at] = (unsigned char)i;
      s_row[at] = (unsigned char)r;
    }
    __syncthreads();
  }
  const int rows = min(block_rows, vocab - v0), vecs = d / 8;
  for (int k = threadIdx.x; k < rows * vecs; k += 256) {
    const int r = k / vecs, c = (k - r * vecs) * 8;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    bool any = false;
    for (int q = 0; q < found;) {
      Vec8<T> x[4];   // the row's next four tokens
      int m = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        while (q < found && s_row[q] != r) ++q;
        if (q < found) {
          x[u].load(d_out + (long long)s_n[q] * d + c);
          ++q;
          m = u + 1;
        }
      }
      any = any || m > 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u < m) {
          float v[8];
          x[u].get(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += v[i];
        }
      }
    }
    if (any || !accumulate) write_row(d_table + (long long)(v0 + r) * d + c, acc, scale, accumulate != 0);
  }
}

// ---------------------------------------------------------------- stable radix sort
constexpr int RADIX_BITS = 9;
constexpr int RADIX = 1 << RADIX_BITS;
constexpr int SORT_WARPS = 8;
constexpr int SORT_STEPS = 8;                               // keys per lane
constexpr int SORT_TILE = SORT_WARPS * 32 * SORT_STEPS;     // keys per block

// Keys: the id, or `vocab` where it is outside [0, vocab), so those sort last.
__device__ __forceinline__ int sort_key(const void* ids, int id_bytes, const int* keys, int i, int vocab) {
  if (keys) return keys[i];
  const long long id = load_id(ids, id_bytes, i);
  return id >= 0 && id < vocab ? (int)id : vocab;
}

// Lanes of the warp with the same digit (RADIX for a lane past the end).
__device__ __forceinline__ unsigned same_digit(int dg) {
  unsigned same = 0xffffffffu;
#pragma unroll
  for (int b = 0; b <= RADIX_BITS; ++b) {
    const bool bit = (dg >> b) & 1;
    const unsigned m = __ballot_sync(0xffffffffu, bit);
    same &= bit ? m : ~m;
  }
  return same;
}

// Counts of the block's digits: hist[block][digit].
__global__ void __launch_bounds__(256) sort_count_kernel(const void* ids, int id_bytes, const int* keys, int n,
                                                         int vocab, int shift, int* hist, int* clear) {
  __shared__ int cnt[RADIX];
  for (int i = threadIdx.x; i < RADIX; i += 256) cnt[i] = 0;
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0;
  __syncthreads();
  const int base = blockIdx.x * SORT_TILE;
#pragma unroll
  for (int k = 0; k < SORT_TILE / 256; ++k) {
    const int i = base + k * 256 + threadIdx.x;
    if (i < n) atomicAdd(&cnt[(sort_key(ids, id_bytes, keys, i, vocab) >> shift) & (RADIX - 1)], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < RADIX; i += 256) hist[(long long)blockIdx.x * RADIX + i] = cnt[i];
}

// Moves the block's keys to their places, in order.  Each block adds up the
// counts before it by itself (blocks x RADIX counts, from L2: 8 MB in all for
// 131072 tokens, but with the square of them: 134 GB, tens of milliseconds a
// pass, for 16 million).
__global__ void __launch_bounds__(256) sort_move_kernel(const void* ids, int id_bytes, const int* keys, const int* pos,
                                                        int n, int vocab, int shift, const int* hist, int* out_keys,
                                                        int* out_pos) {
  __shared__ int warp_cnt[SORT_WARPS][RADIX];
  __shared__ int start[RADIX];
  __shared__ int s_scan[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < SORT_WARPS * RADIX; i += 256) (&warp_cnt[0][0])[i] = 0;
  // digit totals and the counts of earlier blocks: two digits a thread
  int before[2] = {0, 0}, all[2] = {0, 0};
#pragma unroll 8
  for (int b = 0; b < (int)gridDim.x; ++b) {
    const int2 c = *reinterpret_cast<const int2*>(hist + (long long)b * RADIX + 2 * threadIdx.x);
    all[0] += c.x;
    all[1] += c.y;
    if (b < (int)blockIdx.x) {
      before[0] += c.x;
      before[1] += c.y;
    }
  }
  int incl = all[0] + all[1];
  const int mine = incl;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int excl = incl - mine;
  for (int w = 0; w < warp; ++w) excl += s_scan[w];
  start[2 * threadIdx.x] = excl + before[0];
  start[2 * threadIdx.x + 1] = excl + all[0] + before[1];
  __syncthreads();
  // ranks inside the warp's 32 x SORT_STEPS consecutive keys
  const int base = blockIdx.x * SORT_TILE + warp * 32 * SORT_STEPS;
  int key[SORT_STEPS], rank[SORT_STEPS];
#pragma unroll
  for (int s = 0; s < SORT_STEPS; ++s) {
    const int i = base + s * 32 + lane;
    key[s] = i < n ? sort_key(ids, id_bytes, keys, i, vocab) : -1;
  }
#pragma unroll
  for (int s = 0; s < SORT_STEPS; ++s) {
    const bool in = base + s * 32 + lane < n;
    const int dg = in ? (key[s] >> shift) & (RADIX - 1) : RADIX;   // RADIX: past the end
    const unsigned same = same_digit(dg);
    const int below = __popc(same & ((1u << lane) - 1));
    int old = 0;
    if (in && below == 0) {
      old = warp_cnt[warp][dg];
      warp_cnt[warp][dg] = old + __popc(same);
    }
    old = __shfl_sync(0xffffffffu, old, __ffs(same) - 1);
    rank[s] = old + below;
    __syncwarp();
  }
  __syncthreads();
  for (int dg = threadIdx.x; dg < RADIX; dg += 256) {   // per digit: where each warp's keys start
    int at = start[dg];
#pragma unroll
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int c = warp_cnt[w][dg];
      warp_cnt[w][dg] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < SORT_STEPS; ++s) {
    const int i = base + s * 32 + lane;
    if (i < n) {
      const int at = warp_cnt[warp][(key[s] >> shift) & (RADIX - 1)] + rank[s];
      out_keys[at] = key[s];
      out_pos[at] = pos ? pos[i] : i;
    }
  }
}

// All passes in one block, for up to BLOCK_SORT_MAX tokens: keys in registers,
// moved through shared memory (one launch instead of two a pass).
constexpr int BLOCK_SORT_MAX = 8192;
constexpr int BLOCK_SORT_WARPS = 32;
constexpr int BLOCK_SORT_STEPS = BLOCK_SORT_MAX / (32 * BLOCK_SORT_WARPS);
constexpr int BLOCK_SORT_SMEM = 2 * BLOCK_SORT_MAX * 4 + BLOCK_SORT_WARPS * RADIX * 2;

__global__ void __launch_bounds__(1024, 1) sort_block_kernel(const void* ids, int id_bytes, int n, int vocab,
                                                             int* out_keys, int* out_pos, int* clear) {
  extern __shared__ int dyn[];
  __shared__ int s_scan[16];
  int* s_key = dyn;
  int* s_pos = dyn + BLOCK_SORT_MAX;
  unsigned short* cnt = reinterpret_cast<unsigned short*>(dyn + 2 * BLOCK_SORT_MAX);   // [warp][digit]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a warp's keys are consecutive, 256 of them: the fewer warps have any, the
  // less there is to add up (870 tokens: 14.8 us with 32 warps of 32)
  constexpr int per_warp = 32 * BLOCK_SORT_STEPS;
  const int warps = (n + per_warp - 1) / per_warp;
  const int base = warp * per_warp;
  int key[BLOCK_SORT_STEPS], pos[BLOCK_SORT_STEPS];
#pragma unroll
  for (int s = 0; s < BLOCK_SORT_STEPS; ++s) {
    const int i = base + s * 32 + lane;
    pos[s] = i;
    key[s] = i < n ? sort_key(ids, id_bytes, nullptr, i, vocab) : -1;
  }
  if (threadIdx.x == 0) *clear = 0;
  for (int shift = 0; shift < 31 && (shift == 0 || (vocab >> shift) != 0); shift += RADIX_BITS) {
    for (int i = threadIdx.x; i < warps * RADIX / 2; i += 1024) reinterpret_cast<int*>(cnt)[i] = 0;
    __syncthreads();
    int rank[BLOCK_SORT_STEPS];
#pragma unroll
    for (int s = 0; s < BLOCK_SORT_STEPS; ++s) {
      if (base + s * 32 >= n) break;   // the whole warp
      const bool in = key[s] >= 0;
      const int dg = in ? (key[s] >> shift) & (RADIX - 1) : RADIX;
      const unsigned same = same_digit(dg);
      const int below = __popc(same & ((1u << lane) - 1));
      int old = 0;
      if (in && below == 0) {
        old = cnt[warp * RADIX + dg];
        cnt[warp * RADIX + dg] = (unsigned short)(old + __popc(same));
      }
      rank[s] = __shfl_sync(0xffffffffu, old, __ffs(same) - 1) + below;
      __syncwarp();
    }
    __syncthreads();
    int total = 0, incl = 0;   // a thread per digit: exclusive sums over the warps, then over the digits
    if (threadIdx.x < RADIX) {
#pragma unroll 8
      for (int w = 0; w < warps; ++w) {
        const int c = cnt[w * RADIX + threadIdx.x];
        cnt[w * RADIX + threadIdx.x] = (unsigned short)total;
        total += c;
      }
      incl = total;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) s_scan[warp] = incl;
    }
    __syncthreads();
    if (threadIdx.x < RADIX) {
      int start = incl - total;
      for (int w = 0; w < warp; ++w) start += s_scan[w];
#pragma unroll 8
      for (int w = 0; w < warps; ++w) cnt[w * RADIX + threadIdx.x] += (unsigned short)start;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < BLOCK_SORT_STEPS; ++s) {
      if (key[s] >= 0) {
        const int at = cnt[warp * RADIX + ((key[s] >> shift) & (RADIX - 1))] + rank[s];
        s_key[at] = key[s];
        s_pos[at] = pos[s];
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < BLOCK_SORT_STEPS; ++s) {
      const int i = base + s * 32 + lane;
      if (i < n) {
        key[s] = s_key[i];
        pos[s] = s_pos[i];
      }
    }
  }
#pragma unroll
  for (int s = 0; s < BLOCK_SORT_STEPS; ++s) {
    if (key[s] >= 0) {
      out_keys[base + s * 32 + lane] = key[s];
      out_pos[base + s * 32 + lane] = pos[s];
    }
  }
}

// ---------------------------------------------------------------- sums over the sorted tokens
constexpr int CHUNK_MIN = 8, CHUNK_MAX = 64;   // tokens of a worker: fewer where that keeps the device busy
constexpr int AHEAD = 8;           // rows in flight per thread
constexpr int FILL_ROWS = 64;      // table rows of a zeroing block

struct SumParams {
  const int* keys;
  const int* pos;
  int n, vocab, d;
  int tpw;                 // threads of a worker: a thread owns 8 columns
  int workers;             // per block
  int chunk;               // tokens of a worker
  int chunks, col_blocks;  // columns in blocks of 8 tpw
  int sum_blocks;          // blocks before the zeroing ones
  float scale;
  int accumulate;
  float* part;             // [chunks][2][d]: run that comes in from the chunk before, run that goes on
  int2* open;              // runs that go on over a chunk's end: (chunk, id)
  int* n_open;
};

template <typename T>
__global__ void __launch_bounds__(256) embed_grad_sum_kernel(const SumParams p, const T* d_out, T* d_table) {
  if ((int)blockIdx.x >= p.sum_blocks) {   // rows that no token names
    __shared__ unsigned char present[FILL_ROWS];
    const int v0 = ((int)blockIdx.x - p.sum_blocks) * FILL_ROWS;
    if (threadIdx.x < FILL_ROWS) {
      const int v = v0 + threadIdx.x;
      int lo = 0, hi = p.n;   // first token with an id of at least v
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.keys[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      present[threadIdx.x] = lo < p.n && p.keys[lo] == v;
    }
    __syncthreads();
    const int rows = min(FILL_ROWS, p.vocab - v0), vecs = p.d / 8;
    for (int k = threadIdx.x; k < rows * vecs; k += 256) {
      const int r = k / vecs;
      if (present[r]) continue;
      Vec8<T> z;
      z.zero();
      z.store(d_table + (long long)(v0 + r) * p.d + (k - r * vecs) * 8);
    }
    return;
  }
  const int worker = threadIdx.x / p.tpw, t = threadIdx.x - worker * p.tpw;
  const int cb = blockIdx.x % p.col_blocks;
  const int chunk = (int)(blockIdx.x / p.col_blocks) * p.workers + worker;
  const int col = (cb * p.tpw + t) * 8;
  if (worker >= p.workers || chunk >= p.chunks || col >= p.d) return;
  const int i0 = chunk * p.chunk, i1 = min(p.n, i0 + p.chunk);
  const int prev = i0 > 0 ? p.keys[i0 - 1] : -1;
  int cur = p.keys[i0];
  bool comes_in = cur == prev;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  auto finish = [&](bool goes_on) {
    if (cur >= p.vocab) return;
    if (comes_in || goes_on) {
      float* dst = p.part + ((long long)chunk * 2 + (comes_in ? 0 : 1)) * p.d + col;
      reinterpret_cast<float4*>(dst)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (goes_on && !comes_in && col == 0) p.open[atomicAdd(p.n_open, 1)] = make_int2(chunk, cur);
    } else {
      write_row(d_table + (long long)cur * p.d + col, acc, p.scale, p.accumulate != 0);
    }
  };
  for (int i = i0; i < i1; i += AHEAD) {
    Vec8<T> x[AHEAD];
    int key[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      key[u] = p.vocab;
      x[u].zero();
      if (i + u < i1) {
        key[u] = p.keys[i + u];
        if (key[u] < p.vocab) x[u].load(d_out + (long long)p.pos[i + u] * p.d + col);
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (i + u < i1) {
        if (key[u] != cur) {
          finish(false);
          cur = key[u];
          comes_in = false;
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = 0.f;
        }
        float v[8];
        x[u].get(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += v[k];
      }
    }
  }
  finish(i1 < p.n && p.keys[i1] == cur);
}

// Runs over several chunks: their partial sums in order.  A piece of work is
// 256 columns of a run; a warp does those of a run over up to 32 further
// chunks by itself, the block shares a longer one (8 groups of chunks side by
// side).
template <typename T>
__global__ void __launch_bounds__(256) embed_grad_join_kernel(const SumParams p, T* d_table) {
  __shared__ float s[8][256 + 8];
  __shared__ int s_long[8];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;   // 8 columns, warp
  const int col_blocks = (p.d + 255) / 256;
  const long long work = (long long)*p.n_open * col_blocks;
  auto add = [&](float* acc, long long row, int col) {   // one partial sum
    Vec8<float> v;
    v.load(p.part + row * p.d + col);
    float f[8];
    v.get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += f[i];
  };
  // a block's eight pieces lie a grid apart: those of one long run go to different blocks
  for (long long k0 = blockIdx.x; k0 < work; k0 += (long long)gridDim.x * 8) {
    const long long k = k0 + (long long)y * gridDim.x;
    bool longer = false;
    if (k < work) {
      const int2 run = p.open[k / col_blocks];
      const int col = (int)(k % col_blocks) * 256 + x * 8;
      // further chunks that the run reaches: those that begin with its id
      const long long c = run.x + 1ll + x;
      const unsigned in = __ballot_sync(0xffffffffu, c < p.chunks && p.keys[c * p.chunk] == run.y);
      longer = in == 0xffffffffu;
      const int count = __popc(in);
      if (!longer && col < p.d) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        add(acc, run.x * 2ll + 1, col);
#pragma unroll 4
        for (int i = 1; i <= count; ++i) add(acc, (run.x + i) * 2ll, col);
        write_row(d_table + (long long)run.y * p.d + col, acc, p.scale, p.accumulate != 0);
      }
    }
    if (x == 0) s_long[y] = longer;
    __syncthreads();
    for (int w = 0; w < 8; ++w) {
      if (!s_long[w]) continue;   // the same for all threads
      const long long kw = k0 + (long long)w * gridDim.x;
      const int2 run = p.open[kw / col_blocks];
      const int col = (int)(kw % col_blocks) * 256 + x * 8;
      int count = 0;
      for (int more = 256; more == 256; count += more) {
        const long long c = run.x + 1ll + count + threadIdx.x;
        more = __syncthreads_count(c < p.chunks && p.keys[c * p.chunk] == run.y);
      }
      const int per = (count + 7) / 8, a = run.x + 1 + y * per, b = min(run.x + 1 + count, a + per);
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (col < p.d) {
        if (y == 0) add(acc, run.x * 2ll + 1, col);
#pragma unroll 4
        for (int c = a; c < b; ++c) add(acc, c * 2ll, col);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[y][i * 33 + x] = acc[i];
      __syncthreads();
      if (y == 0 && col < p.d) {
        for (int g = 1; g < 8; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += s[g][i * 33 + x];
        write_row(d_table + (long long)run.y * p.d + col, acc, p.scale, p.accumulate != 0);
      }
      __syncthreads();
    }
    __syncthreads();
  }
}

struct GradLayout {
  int tiles, chunk, chunks;
  size_t hist, keys[2], pos[2], part, open, n_open, total;
  GradLayout(int n, int d) {
    tiles = (n + SORT_TILE - 1) / SORT_TILE;
    chunk = CHUNK_MIN;
    while (chunk < CHUNK_MAX && n / chunk > 2048) chunk *= 2;
    chunks = (n + chunk - 1) / chunk;
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o += (bytes + 255) & ~(size_t)255; return at; };
    n_open = take(4);
    hist = take((size_t)tiles * RADIX * 4);
    for (int k = 0; k < 2; ++k) {
      keys[k] = take((size_t)n * 4);
      pos[k] = take((size_t)n * 4);
    }
    part = take((size_t)chunks * 2 * d * 4);
    open = take((size_t)chunks * 8);
    total = o;
  }
};

template <typename T>
cudaError_t embed_grad(int n, int vocab, int d, const void* ids, int id_bytes, const T* d_out, float scale,
                       T* d_table, int accumulate, char* ws, cudaStream_t st) {
  if (n <= SCAN_MAX) {
    const int rows = scan_rows(vocab);
    embed_grad_scan_kernel<T><<<(vocab + rows - 1) / rows, 256, 0, st>>>(ids, id_bytes, d_out, scale, d_table, n, vocab,
                                                                        d, accumulate, rows);
    return cudaGetLastError();
  }
  const GradLayout L(n, d);
  int* hist = (int*)(ws + L.hist);
  int* n_open = (int*)(ws + L.n_open);
  const int *keys = nullptr, *pos = nullptr;
  if (n <= BLOCK_SORT_MAX) {
    cudaError_t e = cudaFuncSetAttribute(sort_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BLOCK_SORT_SMEM);
    if (e != cudaSuccess) return e;
    keys = (int*)(ws + L.keys[0]);
    pos = (int*)(ws + L.pos[0]);
    sort_block_kernel<<<1, 1024, BLOCK_SORT_SMEM, st>>>(ids, id_bytes, n, vocab, (int*)keys, (int*)pos, n_open);
  } else {
    int to = 0;
    for (int shift = 0; shift < 31 && (shift == 0 || (vocab >> shift) != 0); shift += RADIX_BITS) {   // keys are 0 .. vocab
      sort_count_kernel<<<L.tiles, 256, 0, st>>>(ids, id_bytes, keys, n, vocab, shift, hist, shift ? nullptr : n_open);
      int* ok = (int*)(ws + L.keys[to]);
      int* op = (int*)(ws + L.pos[to]);
      sort_move_kernel<<<L.tiles, 256, 0, st>>>(ids, id_bytes, keys, pos, n, vocab, shift, hist, ok, op);
      keys = ok;
      pos = op;
      to ^= 1;
    }
  }
  SumParams p{};
  p.keys = keys; p.pos = pos; p.n = n; p.vocab = vocab; p.d = d;
  const int vecs = d / 8;
  p.tpw = vecs < 256 ? vecs : 256;
  p.workers = 256 / p.tpw;
  p.chunk = L.chunk;
  p.chunks = L.chunks;
  p.col_blocks = (vecs + p.tpw - 1) / p.tpw;
  p.sum_blocks = (p.chunks + p.workers - 1) / p.workers * p.col_blocks;
  p.scale = scale;
  p.accumulate = accumulate;
  p.part = (float*)(ws + L.part);
  p.open = (int2*)(ws + L.open);
  p.n_open = n_open;
  const int fill = accumulate ? 0 : (vocab + FILL_ROWS - 1) / FILL_ROWS;
  embed_grad_sum_kernel<T><<<p.sum_blocks + fill, 256, 0, st>>>(p, d_out, d_table);
  const long long pieces = (long long)p.chunks * ((d + 255) / 256);   // at most
  embed_grad_join_kernel<T><<<(int)(pieces < 148 * 8 ? pieces : 148 * 8), 256, 0, st>>>(p, d_table);
  return cudaGetLastError();
}

}  // namespace

}  // namespace armt

using namespace armt;

extern "C" armt_status armt_embed(armt_dtype dtype, int n, int vocab, int d, const void* ids, int id_bytes,
                                  const void* table, float scale, void* out, void* stream) {
  const armt_status s = check_sizes(dtype, n, vocab, d);
  if (s != ARMT_OK) return s;
  if (!ids || !table || !out || (id_bytes != 4 && id_bytes != 8) || !std::isfinite(scale) || !aligned16(table) ||
      !aligned16(out) || !aligned_to(ids, id_bytes))
    return ARMT_ERR_INVALID_ARG;
  const int vecs = d / 8;
  const long long total = (long long)n * vecs;
  const long long blocks = (total + 256 * LOOKUP_UNROLL - 1) / (256 * LOOKUP_UNROLL);
  if (blocks > 0x7fffffffll) return ARMT_ERR_SHAPE;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == ARMT_BF16)
    embed_kernel<bf16><<<(unsigned)blocks, 256, 0, st>>>(ids, id_bytes, (const bf16*)table, scale, (bf16*)out, total,
                                                        vecs, vocab, d);
  else
    embed_kernel<float><<<(unsigned)blocks, 256, 0, st>>>(ids, id_bytes, (const float*)table, scale, (float*)out,
                                                         total, vecs, vocab, d);
  return cuda_status(cudaGetLastError());
}

extern "C" armt_status armt_embed_grad_workspace(armt_dtype dtype, int n, int vocab, int d, size_t* bytes) {
  if (!bytes) return ARMT_ERR_INVALID_ARG;
  *bytes = 0;
  const armt_status s = check_sizes(dtype, n, vocab, d);
  if (s != ARMT_OK) return s;
  *bytes = n <= SCAN_MAX ? 0 : GradLayout(n, d).total;
  return ARMT_OK;
}

extern "C" armt_status armt_embed_grad(armt_dtype dtype, int n, int vocab, int d, const void* ids, int id_bytes,
                                       const void* d_out, float scale, void* d_table, int accumulate, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const armt_status s = armt_embed_grad_workspace(dtype, n, vocab, d, &need);
  if (s != ARMT_OK) return s;
  if (!ids || !d_out || !d_table || (id_bytes != 4 && id_bytes != 8) || !std::isfinite(scale) ||
      (accumulate != 0 && accumulate != 1) || !aligned16(d_out) || !aligned16(d_table) ||
      !aligned_to(ids, id_bytes) || workspace_bytes < need ||
      (need && (!workspace || !aligned16(workspace))))
    return ARMT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == ARMT_BF16)
    return cuda_status(embed_grad<bf16>(n, vocab, d, ids, id_bytes, (const bf16*)d_out, scale, (bf16*)d_table,
                                        accumulate, (char*)workspace, st));
  return cuda_status(embed_grad<float>(n, vocab, d, ids, id_bytes, (const float*)d_out, scale, (float*)d_table,
                                       accumulate, (char*)workspace, st));
}
