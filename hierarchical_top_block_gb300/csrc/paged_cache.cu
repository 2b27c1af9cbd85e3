// The paged cache's write and its eviction.
//
// Write: the new tokens' rows of K and V go to their pages, and the weights kept beside the pages are cleared there.
// It moves 8 d bytes a (token, head); 8 lanes (d = 64) or 16 (d = 128) take a row, 16 bytes a lane.
//
// Eviction: of the len keys of a (sequence, KV head) the `keep` of the largest accumulated weight stay (the first
// `sinks` and the last `recent` always, ties to the lower index) and are put, in their order, into new pages.  Two
// kernels: the choice (a radix selection over the weights, 8 bits a pass, by a cluster of blocks a head; its result is
// the list of the kept keys, ascending) and the move of their rows.  The choice reads 4 bytes a key, the move
// reads and writes 4 d + 4 a kept key.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"
#include "pdl.cuh"

namespace pisa {
namespace {

// ---- write -----------------------------------------------------------------------------
constexpr int WRITE_THREADS = 128;

struct WriteParams {
  const uint16_t* x[2];
  uint16_t* y[2];
  float* w;  // nullable
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* row_start;
  long long stride[2];
  int B, R, H, P, M, s_bits;
  uint32_t* err;
};

// The sequence of query row `row` (-1: none): the last one that begins at or before it and holds it.
__device__ __forceinline__ int sequence_of(const int32_t* row_start, int B, int R, int row) {
  if (!row_start) return row / (R / B);
  int lo = 0, hi = B;  // first sequence with row_start[b + 1] > row
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(row_start + mid + 1) > row)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo < B ? lo : -1;
}

// A thread has one 16-byte piece of K and of V: four rows' pieces were slower (64000 rows x 8 heads, d = 128: 86 us and 80
// with one; 64 x 8 rows 6.3 and 4.2).
template <int D>
__global__ void __launch_bounds__(WRITE_THREADS) paged_write_kernel(WriteParams p) {
  constexpr int LANES = D / 8, RPB = WRITE_THREADS / LANES;  // lanes a row, rows a block
  const int part = threadIdx.x % LANES;
  const int cap = p.M << p.s_bits;
  if (blockIdx.x == 0)  // sequences without rows are looked at too
    for (int b = threadIdx.x; b < p.B; b += WRITE_THREADS) {
      bool bad;
      paged_seq(p.row_start, p.seq_len, p.B, p.R, cap, b, bad);
      if (bad) report_error(p.err, ERR_BAD_INDEX);
    }
  const long long u = (long long)blockIdx.x * RPB + threadIdx.x / LANES;  // row * H + head
  if (u >= (long long)p.R * p.H) return;
  const int row = (int)whole_quotient(u, p.H), head = (int)(u - (long long)row * p.H);
  const uint4 k = ldg16(p.x[0] + row * p.stride[0] + head * D + part * 8);
  const uint4 v = ldg16(p.x[1] + row * p.stride[1] + head * D + part * 8);
  const int b = sequence_of(p.row_start, p.B, p.R, row);
  if (b < 0) return;
  bool bad;
  const PagedSeq s = paged_seq(p.row_start, p.seq_len, p.B, p.R, cap, b, bad);
  const int t = row - s.first;
  if (t < 0 || t >= s.n) return;
  const int c = s.L + t, page = __ldg(p.table + (size_t)b * p.M + (c >> p.s_bits));
  if ((unsigned)page >= (unsigned)p.P) {
    report_error(p.err, ERR_BAD_INDEX);
    return;
  }
  const long long at = (((long long)page * p.H + head) << p.s_bits) + (c & ((1 << p.s_bits) - 1));
  *reinterpret_cast<uint4*>(p.y[0] + at * D + part * 8) = k;
  *reinterpret_cast<uint4*>(p.y[1] + at * D + part * 8) = v;
  if (p.w && part == 0) p.w[at] = 0.f;
}

// ---- eviction: the choice ----------------------------------------------------------------
constexpr int PICK_THREADS = 512, PICK_WARPS = PICK_THREADS / 32;
constexpr uint32_t MAX_CLUSTER = 8;
constexpr int PICK_CACHED = 12288;  // weights a block keeps in shared memory at most (a multiple of 4); further ones are read again

struct EvictParams {
  uint16_t* K;
  uint16_t* V;
  float* w;
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* new_table;
  int32_t* new_len;
  int32_t* kept;  // [B][H][keep]
  int B, H, P, M, M_new, s_bits, keep, sinks, recent, cached;
  uint32_t* err;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// A word of shared memory of block `rank` of the cluster, at the place that p has here.
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, uint32_t rank) {
  uint32_t addr, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Weights as whole numbers in the same order: 0 for a key that is not there, 1 for NaN, all ones for a key that stays
// whatever its weight; -0 counts as 0.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 1;
  const uint32_t u = __float_as_uint(w + 0.f);  // (-0 + 0 = 0)
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(PICK_THREADS) paged_pick_kernel(EvictParams p) {
  pdl_trigger();
  extern __shared__ __align__(16) uint32_t cached[];  // [p.cached]
  __shared__ uint32_t hist[2][256];     // of passes in turn
  __shared__ uint32_t part[8][256];     // the first pass's, a lane's mod 8: weights have few exponents
  __shared__ uint32_t warp_sum[2][PICK_WARPS];
  __shared__ uint32_t totals[2];        // this block's keys above the limit, and at it
  __shared__ uint32_t found[3];         // digit, keys above it, keys that have it
  const uint32_t rank = cluster_rank(), blocks = cluster_size();
  const int bh = blockIdx.x / blocks, b = bh / p.H, h = bh - b * p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = __ldg(p.seq_len + b);
  if (n < 0 || n > p.M << p.s_bits) {  // (all blocks of the cluster)
    if (rank == 0 && threadIdx.x == 0 && h == 0) report_error(p.err, ERR_BAD_INDEX);
    if (rank == 0)
      for (int i = threadIdx.x; i < p.keep; i += PICK_THREADS) p.kept[(size_t)bh * p.keep + i] = -1;
    return;
  }
  // this block's keys, four a lane at a time (they lie in one page); a whole number of 128 for each warp, so that the
  // warps' shares follow one another
  constexpr int STEP = 128 * PICK_WARPS;
  const int share = (int)((((long long)n + blocks - 1) / blocks + STEP - 1) / STEP * STEP);
  const int c0 = min((long long)n, (long long)rank * share), c1 = min((long long)n, (long long)(rank + 1) * share);
  const int32_t* table = p.table + (size_t)b * p.M;
  auto weights_at = [&](int page, int c) {
    return __ldg(reinterpret_cast<const float4*>(p.w + ((((size_t)page * p.H + h)) << p.s_bits) + (c & ((1 << p.s_bits) - 1))));
  };
  auto order_of = [&](int page, int c, float w) -> uint32_t {
    return page == p.P || c >= n ? 0 : c < p.sinks || c >= n - p.recent ? 0xffffffffu : weight_order(w);
  };
  auto orders_of = [&](int page, int c, float4 w) {
    return make_uint4(order_of(page, c, w.x), order_of(page, c + 1, w.y), order_of(page, c + 2, w.z), order_of(page, c + 3, w.w));
  };
  auto order = [&](int i) {  // of keys c0 + i .. + 3
    if (i < p.cached) return *reinterpret_cast<const uint4*>(cached + i);
    const int page = page_of(table, p.P, (c0 + i) >> p.s_bits, p.err);
    return orders_of(page, c0 + i, page == p.P ? make_float4(0.f, 0.f, 0.f, 0.f) : weights_at(page, c0 + i));
  };
  for (int i = threadIdx.x; i < 8 * 256; i += PICK_THREADS) part[0][i] = 0;
  __syncthreads();
  const int mine = c1 - c0;
  constexpr int BATCH = 4;  // groups of four keys a thread has under way
  for (int i0 = 4 * threadIdx.x; i0 < mine; i0 += 4 * BATCH * PICK_THREADS) {
    int page[BATCH];
    float4 w[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + 4 * u * PICK_THREADS;
      page[u] = i < mine ? page_of(table, p.P, (c0 + i) >> p.s_bits, p.err) : p.P;
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      w[u] = page[u] == p.P ? make_float4(0.f, 0.f, 0.f, 0.f) : weights_at(page[u], c0 + i0 + 4 * u * PICK_THREADS);
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + 4 * u * PICK_THREADS;
      const uint4 x = orders_of(page[u], c0 + i, w[u]);
      if (i < mine && i < p.cached) *reinterpret_cast<uint4*>(cached + i) = x;
      if (x.x) atomicAdd(&part[lane & 7][x.x >> 24], 1u);
      if (x.y) atomicAdd(&part[lane & 7][x.y >> 24], 1u);
      if (x.z) atomicAdd(&part[lane & 7][x.z >> 24], 1u);
      if (x.w) atomicAdd(&part[lane & 7][x.w >> 24], 1u);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 256; i += PICK_THREADS) {
    uint32_t t = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) t += part[u][i];
    hist[0][i] = t;
  }
  // the limit: the want-th largest, 8 bits a pass
  uint32_t limit = 0, want = p.keep;
  bool all = false;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* now = hist[pass & 1];
    uint32_t* next = hist[(pass & 1) ^ 1];
    if (pass > 0) {
      auto count = [&](uint32_t x) {
        if (x && x >> (shift + 8) == limit >> (shift + 8)) atomicAdd(&now[(x >> shift) & 255], 1u);
      };
#pragma unroll 4
      for (int i = 4 * threadIdx.x; i < mine; i += 4 * PICK_THREADS) {
        const uint4 x = order(i);
        count(x.x);
        count(x.y);
        count(x.z);
        count(x.w);
      }
    }
    cluster_sync();
    uint32_t count = 0;
    if (threadIdx.x < 256) {
      uint32_t its[MAX_CLUSTER];
#pragma unroll
      for (uint32_t k = 0; k < MAX_CLUSTER; ++k) its[k] = k < blocks ? peer_word(&now[255 - threadIdx.x], k) : 0;
#pragma unroll
      for (uint32_t k = 0; k < MAX_CLUSTER; ++k) count += its[k];
    }
    // `next` was last read before the barrier
    for (int i = threadIdx.x; i < 256; i += PICK_THREADS) next[i] = 0;
    // sums from the largest digit down
    uint32_t sum = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) warp_sum[0][warp] = sum;
    if (threadIdx.x == 0) found[0] = 256;
    __syncthreads();
    if (threadIdx.x < 256) {
      for (int k = 0; k < warp; ++k) sum += warp_sum[0][k];
      if (sum >= want && sum - count < want) {
        found[0] = 255 - threadIdx.x;
        found[1] = sum - count;
        found[2] = count;
      }
    }
    __syncthreads();
    if (found[0] == 256) {  // fewer keys than wanted (in the first pass alone): every key stays
      all = true;
      break;
    }
    limit |= found[0] << shift;
    want -= found[1];
    if (found[2] == want) {  // all keys of these digits stay: the further ones need not be looked at
      limit -= limit > 0;
      want = 0;
      break;
    }
    __syncthreads();
  }
  if (all) limit = 0, want = 0;  // every key is above it
  // keys above the limit, and at it, of which the first `want` stay: this block's, and those of the blocks before
  const int per = share / PICK_WARPS, w0 = min(mine, warp * per), w1 = min(mine, (warp + 1) * per);
  // (keys above it in the low half of a word, at it in the high one)
  auto kinds = [&](const uint4& x) {
    auto kind = [&](uint32_t v) { return v > limit ? 1u : v == limit && v != 0 ? 0x10000u : 0u; };
    return make_uint4(kind(x.x), kind(x.y), kind(x.z), kind(x.w));
  };
  uint32_t gt = 0, eq = 0;
#pragma unroll 4
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    const uint4 k = kinds(order(i));
    const uint32_t both = k.x + k.y + k.z + k.w;
    gt += both & 0xffffu;
    eq += both >> 16;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_sum[0][warp] = gt;
    warp_sum[1][warp] = eq;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    uint32_t t = 0;
    for (int k = 0; k < PICK_WARPS; ++k) t += warp_sum[threadIdx.x][k];
    totals[threadIdx.x] = t;
  }
  cluster_sync();
  uint32_t before[2] = {0, 0}, every[2] = {0, 0};
  uint32_t its[MAX_CLUSTER][2];
#pragma unroll
  for (uint32_t k = 0; k < MAX_CLUSTER; ++k)
#pragma unroll
    for (int e = 0; e < 2; ++e) its[k][e] = k < blocks ? peer_word(&totals[e], k) : 0;
#pragma unroll
  for (uint32_t k = 0; k < MAX_CLUSTER; ++k)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      every[e] += its[k][e];
      if (k < rank) before[e] += its[k][e];
    }
  for (int k = 0; k < warp; ++k) before[0] += warp_sum[0][k], before[1] += warp_sum[1][k];
  int32_t* kept = p.kept + (size_t)bh * p.keep;
#pragma unroll 2
  for (int i0 = w0; i0 < w1; i0 += 128) {
    const int i = i0 + 4 * lane;
    const uint4 k = i < w1 ? kinds(order(i)) : make_uint4(0, 0, 0, 0);
    const uint32_t mine4 = k.x + k.y + k.z + k.w;
    uint32_t sum = mine4;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    uint32_t g = before[0] + ((sum - mine4) & 0xffffu), q = before[1] + ((sum - mine4) >> 16);
    auto put = [&](uint32_t kind, int c) {
      if (kind == 0) return;
      const uint32_t to = g + min(q, want);
      if ((kind == 1 || q < want) && to < (uint32_t)p.keep) kept[to] = c;
      g += kind & 1;
      q += kind >> 16;
    };
    put(k.x, c0 + i);
    put(k.y, c0 + i + 1);
    put(k.z, c0 + i + 2);
    put(k.w, c0 + i + 3);
    sum = __shfl_sync(0xffffffffu, sum, 31);
    before[0] += sum & 0xffffu;
    before[1] += sum >> 16;
  }
  const uint32_t stay = every[0] + min(every[1], want);
  for (uint32_t i = stay + rank * PICK_THREADS + threadIdx.x; i < (uint32_t)p.keep; i += blocks * PICK_THREADS) kept[i] = -1;
  if (h == 0 && rank == 0 && threadIdx.x == 0) p.new_len[b] = (int)min(stay, (uint32_t)p.keep);
  cluster_sync();  // nobody's shared memory goes away before it has been read
}

// ---- eviction: the move --------------------------------------------------------------------
constexpr int MOVE_THREADS = 128;

template <int D, int RPT>
__global__ void __launch_bounds__(MOVE_THREADS) paged_move_kernel(EvictParams p) {
  constexpr int LANES = D / 8, RPB = MOVE_THREADS / LANES;
  const int part = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  const int bh = blockIdx.y, b = bh / p.H, h = bh - b * p.H, in_page = (1 << p.s_bits) - 1;
  const int j0 = blockIdx.x * RPB * RPT + sub;
  long long to[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {  // (the tables are not the choice's)
    const int j = j0 + i * RPB;
    to[i] = -1;
    if (j < p.keep) {
      const int page = __ldg(p.new_table + (size_t)b * p.M_new + (j >> p.s_bits));
      to[i] = (unsigned)page < (unsigned)p.P ? (((long long)page * p.H + h) << p.s_bits) + (j & in_page) : -2;
    }
  }
  pdl_wait();
  int src[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    src[i] = to[i] != -1 ? p.kept[(size_t)bh * p.keep + j0 + i * RPB] : -1;
    if (src[i] >= 0 && to[i] == -2) {
      report_error(p.err, ERR_BAD_INDEX);
      src[i] = -1;
    }
  }
  uint4 x[RPT][2];
  float w[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    if (src[i] < 0) continue;
    const int page = __ldg(p.table + (size_t)b * p.M + (src[i] >> p.s_bits));
    if ((unsigned)page >= (unsigned)p.P) {  // (unless somebody changes the table under the call)
      src[i] = -1;
      continue;
    }
    const long long from = (((long long)page * p.H + h) << p.s_bits) + (src[i] & in_page);
    x[i][0] = *reinterpret_cast<const uint4*>(p.K + from * D + part * 8);
    x[i][1] = *reinterpret_cast<const uint4*>(p.V + from * D + part * 8);
    if (part == 0) w[i] = p.w[from];
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    if (src[i] < 0) continue;
    *reinterpret_cast<uint4*>(p.K + to[i] * D + part * 8) = x[i][0];
    *reinterpret_cast<uint4*>(p.V + to[i] * D + part * 8) = x[i][1];
    if (part == 0) p.w[to[i]] = w[i];
  }
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

cudaError_t launch_paged_write(const uint16_t* k, const uint16_t* v, long long k_stride, long long v_stride, uint16_t* Kp,
                               uint16_t* Vp, float* w, const int32_t* table, const int32_t* seq_len,
                               const int32_t* row_start, const Problem& pr, const Pages& pg, uint32_t* err, cudaStream_t s) {
  WriteParams p{{k, v}, {Kp, Vp}, w, table, seq_len, row_start, {k_stride, v_stride},
                pr.B,   pr.N,     pr.H_kv, pg.P, pg.M, pg.s_bits, err};
  const long long rows = (long long)pr.N * pr.H_kv;
  const int rpb = WRITE_THREADS * 8 / pr.d;
  const unsigned grid = (unsigned)((rows + rpb - 1) / rpb);
  if (pr.d == 128)
    paged_write_kernel<128><<<grid, WRITE_THREADS, 0, s>>>(p);
  else
    paged_write_kernel<64><<<grid, WRITE_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

size_t paged_evict_workspace_bytes(const Problem& pr, int keep) { return up256((size_t)pr.B * pr.H_kv * keep * 4); }

cudaError_t launch_paged_evict(uint16_t* Kp, uint16_t* Vp, float* w, const int32_t* table, const int32_t* seq_len,
                               const int32_t* new_table, int32_t* new_len, int32_t* kept, int keep, int sinks, int recent,
                               int new_max_pages, const Problem& pr, const Pages& pg, int num_sms, uint32_t* err, cudaStream_t s) {
  EvictParams p{Kp, Vp, w,    table, seq_len,       new_table,  new_len, kept,  pr.B,
                pr.H_kv,  pg.P, pg.M,  new_max_pages, pg.s_bits, keep,    sinks, recent, 0,   err};
  cudaError_t e = allow_shared<paged_pick_kernel>(PICK_CACHED * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // blocks a head: as many as find room at once (two a SM), where there are keys for them (with 1, 2, 4, 8: 8 heads of 32768
  // keys 62, 33, 19, 16 us, 64 heads 64, 35, 25, 37, 240 heads of 8000 keys 26, 34, 50, 91)
  unsigned blocks = MAX_CLUSTER;
  while (blocks > 1 && ((long long)pr.B * pr.H_kv * blocks > 2ll * num_sms || ((long long)pg.M << pg.s_bits) <= 1024ll * blocks)) blocks /= 2;
  cfg.gridDim = dim3((unsigned)pr.B * pr.H_kv * blocks);
  cfg.blockDim = dim3(PICK_THREADS);
  // no more shared memory than the longest sequence wants
  const long long share = ((((long long)pg.M << pg.s_bits) + blocks - 1) / blocks + 2047) / 2048 * 2048;
  p.cached = (int)std::min<long long>(PICK_CACHED, share);
  cfg.dynamicSmemBytes = (size_t)p.cached * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, paged_pick_kernel, p)) != cudaSuccess) return e;
  // two rows a thread where they fill the SMs, one where latency counts (64 x 8192 rows 106.7 us and 109.9 with one, 107.2 with
  // four; 8 x 250 rows 13.4 and 12.4, 14.4 with four)
  const int one = MOVE_THREADS * 8 / pr.d, rpt = (long long)pr.B * pr.H_kv * keep >= 32ll * num_sms * one ? 2 : 1;
  const dim3 grid((unsigned)((keep + one * rpt - 1) / (one * rpt)), (unsigned)(pr.B * pr.H_kv));
  auto move = pr.d == 128 ? (rpt == 2 ? paged_move_kernel<128, 2> : paged_move_kernel<128, 1>)
                          : (rpt == 2 ? paged_move_kernel<64, 2> : paged_move_kernel<64, 1>);
  return launch_pdl(move, grid, dim3(MOVE_THREADS), 0, s, p);
}

}  // namespace pisa
