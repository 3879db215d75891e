// Token embedding and the gradient of its table.
//
//   out[n] = scale * table[id_n]                 (0 where id_n is outside [0, V))
//   d_table[v] = (d_table[v]) + scale * sum of d_out[n] over n with id_n = v
//
// Both are bound by memory traffic.  The gradient sums each table row's tokens
// in the order of n, so the result does not depend on the schedule: no
// floating-point atomics.  Two ways, by the number of tokens:
//
//   few tokens: a block owns 32 table rows and looks through all ids; one
//     launch, nothing to sort.
//   many tokens: a stable radix sort of (id, n) by 9 bits a pass; then the
//     sorted list is cut into chunks of 64 tokens, a worker per chunk adds up
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
constexpr int SCAN_MAX = 2048;      // most tokens for the one-launch gradient
constexpr int SCAN_ROWS = 32;       // table rows of a block

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
                                                              int accumulate) {
  __shared__ unsigned short s_n[SCAN_MAX];    // tokens of the block's rows, in order
  __shared__ unsigned char s_row[SCAN_MAX];
  __shared__ int s_warp[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int v0 = blockIdx.x * SCAN_ROWS;
  int found = 0;
  for (int b = 0; b < n; b += 256) {
    const int i = b + threadIdx.x;
    int r = -1;
    if (i < n) {
      const long long id = load_id(ids, id_bytes, i);
      if (id >= v0 && id < v0 + SCAN_ROWS && id < vocab) r = (int)(id - v0);
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
      s_n[at] = (unsigned short)i;
      s_row[at] = (unsigned char)r;
    }
    __syncthreads();
  }
  const int rows = min(SCAN_ROWS, vocab - v0), vecs = d / 8;
  for (int k = threadIdx.x; k < rows * vecs; k += 256) {
    const int r = k / vecs, c = (k - r * vecs) * 8;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    bool any = false;
    for (int q = 0; q < found; ++q) {
      if (s_row[q] != r) continue;
      any = true;
      Vec8<T> x;
      x.load(d_out + (long long)s_n[q] * d + c);
      float v[8];
      x.get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
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
// counts before it by itself (blocks x RADIX counts, from L2).
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
  for (int b = 0; b < (int)gridDim.x; ++b) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = hist[(long long)b * RADIX + 2 * threadIdx.x + k];
      all[k] += c;
      if (b < (int)blockIdx.x) before[k] += c;
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
    const unsigned same = __match_any_sync(0xffffffffu, dg);
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

// ---------------------------------------------------------------- sums over the sorted tokens
constexpr int CHUNK = 64;          // tokens of a worker
constexpr int AHEAD = 8;           // rows in flight per thread
constexpr int FILL_ROWS = 64;      // table rows of a zeroing block

struct SumParams {
  const int* keys;
  const int* pos;
  int n, vocab, d;
  int tpw;                 // threads of a worker: a thread owns 8 columns
  int workers;             // per block
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
  const int i0 = chunk * CHUNK, i1 = min(p.n, i0 + CHUNK);
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

// Runs over several chunks: their partial sums in order, 16 groups of chunks
// side by side, 64 columns a block.
template <typename T>
__global__ void __launch_bounds__(256) embed_grad_join_kernel(const SumParams p, T* d_table) {
  __shared__ float4 s[256];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;   // 4 columns, group
  const int col_blocks = (p.d + 63) / 64;
  const long long work = (long long)*p.n_open * col_blocks;
  for (long long k = blockIdx.x; k < work; k += gridDim.x) {
    const int2 run = p.open[k / col_blocks];
    const int col = (int)(k % col_blocks) * 64 + x * 4;
    // the run's last chunk: the last token with its id
    int lo = (run.x + 1) * CHUNK, hi = p.n;   // first token behind the run
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.keys[mid] <= run.y) lo = mid + 1;
      else hi = mid;
    }
    const int last = (lo - 1) / CHUNK, count = last - run.x;   // chunks after the first
    const int per = (count + 15) / 16, a = run.x + 1 + y * per, b = min(last + 1, a + per);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < p.d) {
      if (y == 0) acc = *reinterpret_cast<const float4*>(p.part + ((long long)run.x * 2 + 1) * p.d + col);
#pragma unroll 8
      for (int c = a; c < b; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(p.part + (long long)c * 2 * p.d + col);
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
      }
    }
    __syncthreads();
    s[threadIdx.x] = acc;
    __syncthreads();
    if (y == 0 && (x & 1) == 0 && col < p.d) {   // 8 columns a thread
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int g = 0; g < 16; ++g) {
        const float4 l = s[g * 16 + x], r = s[g * 16 + x + 1];
        v[0] += l.x; v[1] += l.y; v[2] += l.z; v[3] += l.w;
        v[4] += r.x; v[5] += r.y; v[6] += r.z; v[7] += r.w;
      }
      write_row(d_table + (long long)run.y * p.d + col, v, p.scale, p.accumulate != 0);
    }
  }
}

struct GradLayout {
  int tiles, chunks;
  size_t hist, keys[2], pos[2], part, open, n_open, total;
  GradLayout(int n, int d) {
    tiles = (n + SORT_TILE - 1) / SORT_TILE;
    chunks = (n + CHUNK - 1) / CHUNK;
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
    embed_grad_scan_kernel<T><<<(vocab + SCAN_ROWS - 1) / SCAN_ROWS, 256, 0, st>>>(ids, id_bytes, d_out, scale, d_table,
                                                                                 n, vocab, d, accumulate);
    return cudaGetLastError();
  }
  const GradLayout L(n, d);
  int* hist = (int*)(ws + L.hist);
  int* n_open = (int*)(ws + L.n_open);
  const int *keys = nullptr, *pos = nullptr;
  int to = 0;
  for (int shift = 0; shift == 0 || (vocab >> shift) != 0; shift += RADIX_BITS) {   // keys are 0 .. vocab
    sort_count_kernel<<<L.tiles, 256, 0, st>>>(ids, id_bytes, keys, n, vocab, shift, hist, shift ? nullptr : n_open);
    int* ok = (int*)(ws + L.keys[to]);
    int* op = (int*)(ws + L.pos[to]);
    sort_move_kernel<<<L.tiles, 256, 0, st>>>(ids, id_bytes, keys, pos, n, vocab, shift, hist, ok, op);
    keys = ok;
    pos = op;
    to ^= 1;
  }
  SumParams p{};
  p.keys = keys; p.pos = pos; p.n = n; p.vocab = vocab; p.d = d;
  const int vecs = d / 8;
  p.tpw = vecs < 256 ? vecs : 256;
  p.workers = 256 / p.tpw;
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
  embed_grad_join_kernel<T><<<148 * 4, 256, 0, st>>>(p, d_table);
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
      !aligned16(out))
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
      (accumulate != 0 && accumulate != 1) || !aligned16(d_out) || !aligned16(d_table) || workspace_bytes < need ||
      (need && (!workspace || !aligned16(workspace))))
    return ARMT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == ARMT_BF16)
    return cuda_status(embed_grad<bf16>(n, vocab, d, ids, id_bytes, (const bf16*)d_out, scale, (bf16*)d_table,
                                        accumulate, (char*)workspace, st));
  return cuda_status(embed_grad<float>(n, vocab, d, ids, id_bytes, (const float*)d_out, scale, (float*)d_table,
                                       accumulate, (char*)workspace, st));
}
