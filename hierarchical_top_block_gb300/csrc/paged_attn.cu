// Attention of new tokens over the paged cache of their sequences: one token (decode), a few (drafts), a chunk of a
// prompt or a whole one, in ragged batches.
//
//   z_tc = scale q_t . k_c for the keys c that token t sees,   o_t = sum_c softmax(z_t)_c v_c,   lse_t = log sum_c e^z_tc
//
// in one pass over the keys with a running reference (cache_attn.cuh, paged_tc.cu).  Few query rows a sequence
// (G_Q heads x tokens): the kernel here, on mma.sync, bound by the bytes of the cache.  Many: paged_tc.cu.
#include <algorithm>

#include "cache_attn.cuh"
#include "kernels.cuh"
#include "paged.cuh"
#include "pdl.cuh"

namespace pisa {

bool encode_page_map(CUtensorMap* map, const void* base, int d, int S, int H_kv, int P, int keys) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)S, (uint64_t)H_kv, (uint64_t)P};
  const uint64_t strides[3] = {(uint64_t)d * 2, (uint64_t)S * d * 2, (uint64_t)H_kv * S * d * 2};
  const uint32_t box[4] = {64, (uint32_t)keys, 1, 1};
  return encode_tensor_map(map, base, 4, dims, strides, box);
}

bool encode_token_map(CUtensorMap* map, const uint16_t* q, int d, int GQ, int H_kv, int R, long long q_stride, int rows) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)GQ, (uint64_t)H_kv, (uint64_t)R};
  const uint64_t strides[3] = {(uint64_t)d * 2, (uint64_t)GQ * d * 2, (uint64_t)q_stride * 2};
  const uint32_t box[4] = {64, (uint32_t)GQ, 1, (uint32_t)(rows / GQ)};
  return encode_tensor_map(map, q, 4, dims, strides, box);
}

namespace {

constexpr int THREADS = 128;
constexpr int few_blocks(int rows) { return rows > 8 ? 2 : 4; }  // a SM

// Tiles of 8 NH rows (few tiles of 8 are as fast as of 16 with many sequences, and 14.4 : 15.7 us with one of 8000 keys).  A
// block's four warps take the granules of a segment in turn, each with a ring of its own that
// it fills by TMA.  A granule lies in one page (KEYS <= S).
template <int D, int KEYS, int NH>
struct FewCfg {
  // Granules a warp has under way: 16 KB a warp with 16 rows, 8 KB with 8, where four blocks a SM have to find room (two of
  // 8 KB leave it to three: 64 sequences of 8192 keys, 32 / 8 heads, d = 64: 178 us).
  static constexpr int SLOTS = NH * 2048 / (KEYS * D);
  static constexpr int PER_SM = few_blocks(8 * NH);
  using Tile = CacheTile<D, 16, KEYS, NH>;
  static constexpr uint32_t RING = 4 * SLOTS * Tile::BYTES, OUT = 4 * 8 * NH * D * 4;
  static constexpr uint32_t SMEM = RING > OUT ? RING : OUT;  // the outputs meet where the granules were
};

template <int D, int KEYS, int NH>
__global__ void __launch_bounds__(THREADS, FewCfg<D, KEYS, NH>::PER_SM)
    paged_few_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV, PagedParams p) {
  pdl_trigger();
  using C = FewCfg<D, KEYS, NH>;
  using Tile = typename C::Tile;
  constexpr int ROWS = 8 * NH;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* po = reinterpret_cast<float*>(smem);  // [4][ROWS][D]
  __shared__ uint64_t full[4][C::SLOTS];
  __shared__ float sn[4][16], sl[4][16];
  __shared__ float2 ml[ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  uint8_t* ring = smem + warp * C::SLOTS * Tile::BYTES;
  if (lane == 0) {
    prefetch_map(&mapK);
    prefetch_map(&mapV);
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&full[warp][i], 1);
    mbar_fence_init();
  }
  __syncwarp();
  PagedWalk w;
  w.init(p, blockIdx.x, blockIdx.x == 0 && warp == 0);
  uint32_t s = 0, got = 0;  // granules used and fetched
  bool failed = false;
  while (w.next(p, blockIdx.x)) {
    const int rows = w.rows(p);
    const int first = w.k0 * PAGED_KT, key_end = min(w.seen(p, rows - 1), w.k1 * PAGED_KT);
    const int granules = (key_end - first + KEYS - 1) / KEYS, mine = max(0, (granules - warp + 3) >> 2);
    const int32_t* table = p.table + (size_t)w.b * p.M;
    int pages = p.P;  // of the 32 granules of this warp from `batch` on, one a lane
    auto look = [&](int batch) {
      const int g = batch + lane;
      pages = g < mine ? page_of(table, p.P, (first + (warp + 4 * g) * KEYS) >> p.s_bits, p.err) : p.P;
    };
    uint32_t none = 0;  // slots whose granule has no page
    auto fetch = [&](int i) {  // granule i of this warp
      if ((i & 31) == 0) look(i);
      const int page = __shfl_sync(0xffffffffu, pages, i & 31), slot = got % C::SLOTS;
      none = page == p.P ? none | 1u << slot : none & ~(1u << slot);
      if (lane == 0) {
        const int row = (first + (warp + 4 * i) * KEYS) & ((1 << p.s_bits) - 1);
        uint8_t* dst = ring + slot * Tile::BYTES;
        mbar_arrive_expect_tx(&full[warp][slot], Tile::BYTES);
#pragma unroll
        for (int c = 0; c < Tile::PIECES; ++c) {
          tma_load_4d(dst + c * (KEYS * 128), &mapK, &full[warp][slot], 64 * c, row, w.head, page);
          tma_load_4d(dst + Tile::SIDE + c * (KEYS * 128), &mapV, &full[warp][slot], 64 * c, row, w.head, page);
        }
      }
      ++got;
    };
    auto wait = [&](uint32_t n, uint64_t limit = WAIT_LIMIT_NS) {
      return mbar_wait_warp(&full[warp][n % C::SLOTS], (n / C::SLOTS) & 1, p.err, limit);
    };
#pragma unroll
    for (int i = 0; i < C::SLOTS; ++i)
      if (i < mine && !failed) fetch(i);
    typename Tile::Query qr;
    Tile::load_q(qr, [&](int i) {
      if (i >= rows) return (const uint16_t*)nullptr;
      const int m = w.tile * ROWS + i, tok = m >> p.gq_bits;
      return p.q + (w.s.first + tok) * p.q_stride + ((size_t)w.head * p.GQ + (m - (tok << p.gq_bits))) * D;
    }, p.sl2, r, q);
    int seen[NH][2];
    const int least = w.seen(p, 0);
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) seen[h][e] = w.seen(p, 8 * h + 2 * q + e);
    typename Tile::State st;
    Tile::clear(st);
    const typename Tile::Scales sc{};
    for (int i = 0; i < mine && !failed; ++i, ++s) {
      if (!wait(s)) {
        failed = true;
        break;
      }
      const int key = first + (warp + 4 * i) * KEYS, slot = s % C::SLOTS, n = min(KEYS, key_end - key);
      if (!(none >> slot & 1)) {
        if (key + KEYS <= least) {
          Tile::template add<false, true>(st, ring + slot * Tile::BYTES, sc, qr, n, r, q);
        } else {
          int lim[NH][2];
#pragma unroll
          for (int h = 0; h < NH; ++h) lim[h][0] = seen[h][0] - key, lim[h][1] = seen[h][1] - key;
          Tile::template add<true, true>(st, ring + slot * Tile::BYTES, sc, qr, n, r, q, lim);
        }
      }
      __syncwarp();  // the slot has been read
      if (i + C::SLOTS < mine) fetch(i + C::SLOTS);
    }
    if (failed)  // copies still in flight land before their memory is used again (bounded)
      for (; s < got; ++s) wait(s, 100000000ull);
    join_warps<Tile, D>(st, po, sn, sl, ml, rows);
    if (w.slot < 0) {
      for (int i = threadIdx.x; i < rows * D / 2; i += THREADS) {
        const int row = 2 * i / D, c = 2 * i - row * D;
        const size_t at = w.row_at(p, row);
        float lse;
        const float f = finish_row(ml[row].x, ml[row].y, lse);
        const float2 x = *reinterpret_cast<const float2*>(po + 2 * i);
        *reinterpret_cast<uint32_t*>(p.o + at * D + c) = f == 0.f ? 0u : pack_bf16x2(x.x * f, x.y * f);
        if (c == 0 && p.lse) p.lse[at] = lse;
      }
    } else {
      float* dst = p.part_o + (size_t)w.slot * ROWS * D;
      for (int i = threadIdx.x; i < rows * D; i += THREADS) dst[i] = po[i];
      if (threadIdx.x < rows) p.part_ml[(size_t)w.slot * ROWS + threadIdx.x] = ml[threadIdx.x];
    }
    fence_proxy_async();  // the next copies go where po was
    __syncthreads();
  }
  if (threadIdx.x == 0) p.split[blockIdx.x] = w.split(p, blockIdx.x);
}

// Joins the parts of the jobs that span blocks: blockIdx.x is the block where the job begins, blockIdx.y takes its share of
// the job's rows.  A row is joined by one warp where there are few parts, by more where there are more: they take the parts
// in turn, BATCH of them in flight, and meet in shared memory.
template <int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) paged_join_kernel(PagedParams p) {
  constexpr int V = D / 32, BATCH = 4, WARP_BITS = WARPS == 16 ? 4 : 2;
  __shared__ float so[WARPS][D];
  __shared__ float2 sml[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  const PagedSplit x = p.split[blockIdx.x];
  PagedWalk w;
  if (!w.take(x)) return;
  const int c0 = blockIdx.x, c1 = x.c1, slot0 = x.slot0;
  const int parts = c1 - c0 + 1, bits = parts <= 4 ? 0 : parts <= 32 ? 2 : WARP_BITS, W = 1 << bits;  // warps a row
  const int turn = warp & (W - 1), rows = w.rows(p);
  for (int row0 = blockIdx.y << (WARP_BITS - bits); row0 < rows; row0 += (int)gridDim.y << (WARP_BITS - bits)) {
    const int row = row0 + (warp >> bits);
    const bool live = row < rows;
    float m = NEG_INF, l = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int c = c0 + turn; live && c <= c1; c += W * BATCH) {
      float2 ml[BATCH];
      float x[BATCH][V];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int cc = c + u * W;
        ml[u] = make_float2(NEG_INF, 0.f);
        if (cc > c1) continue;
        const size_t at = ((size_t)(cc == c0 ? slot0 : 2 * cc) << p.row_bits) + row;
        ml[u] = p.part_ml[at];
        const float* src = p.part_o + at * D + lane * V;
        if constexpr (V == 4)
          *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(src);
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < BATCH; ++u) top = fmaxf(top, ml[u].x);
      const float f0 = m == NEG_INF ? 0.f : fast_exp2(m - top);
      if (m != NEG_INF) l *= f0;
      m = top;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] *= f0;
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        if (ml[u].x == NEG_INF) {
          l += ml[u].y;  // 0, or NaN where every logit was
          continue;
        }
        const float f = fast_exp2(ml[u].x - m);
        l += ml[u].y * f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += x[u][i] * f;
      }
    }
    if (W > 1) {  // (the same for the whole block)
#pragma unroll
      for (int i = 0; i < V; ++i) so[warp][lane * V + i] = acc[i];
      if (lane == 0) sml[warp] = make_float2(m, l);
      __syncthreads();
      if (turn == 0) {
        m = NEG_INF;
        for (int u = 0; u < W; ++u) m = fmaxf(m, sml[warp + u].x);
        l = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        for (int u = 0; u < W; ++u) {
          const float2 ml = sml[warp + u];
          const float f = ml.x == NEG_INF ? 0.f : fast_exp2(ml.x - m);
          l += ml.x == NEG_INF ? ml.y : ml.y * f;
          if (f != 0.f)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += so[warp + u][lane * V + i] * f;
        }
      }
      __syncthreads();
    }
    if (!live || turn != 0) continue;
    float lse;
    const float f = finish_row(m, l, lse);
    const size_t at = w.row_at(p, row);
    uint32_t y[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) y[i] = f == 0.f ? 0u : pack_bf16x2(acc[2 * i] * f, acc[2 * i + 1] * f);
    uint16_t* dst = p.o + at * D + lane * V;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = y[0];
    if (p.lse && lane == 0) p.lse[at] = lse;
  }
}

constexpr int MAX_SMS = 152;  // this GPU's: the scratch does not depend on the device at hand

// Which kernel, by the query rows a sequence has on average (their own numbers are on the device; any kernel takes any).
// 32 sequences of 8192 keys, 8 KV heads, few-row against tensor-core kernel: d = 64, 8 rows 97 : 95 us, 16 rows 92 : 97, 24
// rows 166 : 96; d = 128, 8 rows 170 : 168, 16 rows 170 : 171, 24 rows 319 : 172 (the few-row kernel then reads the keys
// twice).  A mean says little of a mixed batch: with four heads a group, 128 tokens of as many sequences of 4000 keys and one
// chunk of 256 after 30000 take 1104 : 489 us (alone 315 and, on tensor cores, 115); 255 of 1000 keys and a prompt of 700
// 227 : 290 (170 and 27).
struct Plan {
  bool tc;
  int rows, blocks, stop;
};
Plan paged_plan(const Problem& p, const Pages& pg) {
  const long long rows = ((long long)p.N * p.GQ + p.B - 1) / (p.B > 0 ? p.B : 1);  // a sequence has on average
  const int few = rows > 8 || p.GQ > 8 ? 16 : 8;
  Plan plan = rows > 16 ? Plan{true, PAGED_TC_ROWS, MAX_SMS, 3} : Plan{false, few, few_blocks(few) * MAX_SMS, 2};
  // no more blocks (and scratch) than there can be steps: every sequence has at most one tile that is not full
  const long long tiles = (long long)p.N * p.GQ / plan.rows + p.B;
  const long long steps = (((long long)pg.M << pg.s_bits) + PAGED_KT - 1) / PAGED_KT;
  plan.blocks = (int)std::min<long long>(plan.blocks, p.H_kv * tiles * steps);
  return plan;
}

template <int D, int KEYS, int NH>
cudaError_t launch_few(const PagedParams& p, cudaStream_t s) {
  using C = FewCfg<D, KEYS, NH>;
  CUtensorMap mapK, mapV;
  if (!encode_page_map(&mapK, p.K, D, 1 << p.s_bits, p.H_kv, p.P, KEYS) ||
      !encode_page_map(&mapV, p.V, D, 1 << p.s_bits, p.H_kv, p.P, KEYS))
    return cudaErrorInvalidValue;
  auto kern = paged_few_kernel<D, KEYS, NH>;
  const cudaError_t e = allow_shared<paged_few_kernel<D, KEYS, NH>>(C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<p.blocks, THREADS, C::SMEM, s>>>(mapK, mapV, p);
  return cudaGetLastError();
}
template <int D, int KEYS>
cudaError_t launch_few_rows(const PagedParams& p, cudaStream_t s) {
  return p.row_bits > 3 ? launch_few<D, KEYS, 2>(p, s) : launch_few<D, KEYS, 1>(p, s);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int bits_of(int x) {  // of a power of two
  int b = 0;
  while ((1 << b) < x) ++b;
  return b;
}

}  // namespace

size_t paged_workspace_bytes(const Problem& p, const Pages& pg) {
  const Plan plan = paged_plan(p, pg);
  const size_t parts = (size_t)2 * plan.blocks * plan.rows;
  return up256(parts * p.d * 4) + up256(parts * 8) + up256((size_t)plan.blocks * sizeof(PagedSplit));
}

cudaError_t launch_paged_attn(const uint16_t* q, long long q_stride, const uint16_t* Kp, const uint16_t* Vp,
                              const int32_t* table, const int32_t* seq_len, const int32_t* row_start, uint16_t* o,
                              float* lse, void* ws, const Problem& pr, const Pages& pg, int num_sms, uint32_t* err,
                              cudaStream_t s) {
  PagedParams p = {};
  p.q = q;
  p.K = Kp;
  p.V = Vp;
  p.table = table;
  p.seq_len = seq_len;
  p.row_start = row_start;
  p.o = o;
  p.lse = lse;
  p.q_stride = q_stride;
  p.B = pr.B;
  p.R = pr.N;
  p.H_q = pr.H_q;
  p.H_kv = pr.H_kv;
  p.GQ = pr.GQ;
  p.P = pg.P;
  p.M = pg.M;
  p.s_bits = pg.s_bits;
  p.causal = pr.causal;
  p.sl2 = pr.scale * LOG2E;
  p.err = err;
  const Plan plan = paged_plan(pr, pg);
  p.gq_bits = bits_of(pr.GQ);
  p.row_bits = bits_of(plan.rows);
  p.blocks = plan.blocks;
  p.inverse = ~0ull / p.blocks + 1;
  p.stop = plan.stop;
  const size_t parts = (size_t)2 * p.blocks * plan.rows;
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.part_o = reinterpret_cast<float*>(at);
  at += up256(parts * pr.d * 4);
  p.part_ml = reinterpret_cast<float2*>(at);
  at += up256(parts * 8);
  p.split = reinterpret_cast<PagedSplit*>(at);
  cudaError_t e;
  if (plan.tc)
    e = launch_paged_tc(p, pr.d, s);
  else if (pr.d == 128)
    e = launch_few_rows<128, 16>(p, s);
  else
    e = pg.s_bits > 4 ? launch_few_rows<64, 32>(p, s) : launch_few_rows<64, 16>(p, s);
  if (e != cudaSuccess) return e;
  // Blocks for the rows of a job that spans blocks.  Tiles of 256: eight (1024 tokens after 15360 of 32 / 8 heads 190.7 us,
  // with 4 and 16 190.8 and 192.8; 64 rows over 32768 keys 40.7, 43.4, 40.6; drafted tokens 43.4, 43.0, 45.0).  Few rows: one a
  // row where there are few jobs, which then have many parts (16 heads over 32768 keys, one KV head, with 4, 8 and 16:
  // 41, 28, 22 us), else one for four (64 sequences of 4000 keys 165.7, 166.3, 168.9).
  const long long rows = (long long)p.R * p.GQ, jobs = p.H_kv * (rows / plan.rows + std::min<long long>(p.B, rows));
  if (plan.tc)
    return launch_pdl(pr.d == 128 ? paged_join_kernel<128, 16> : paged_join_kernel<64, 16>,
                      dim3((unsigned)p.blocks, 8), dim3(32 * 16), 0, s, p);
  return launch_pdl(pr.d == 128 ? paged_join_kernel<128, 4> : paged_join_kernel<64, 4>,
                    dim3((unsigned)p.blocks, (unsigned)(jobs < num_sms ? plan.rows : plan.rows / 4)), dim3(32 * 4), 0, s, p);
}

}  // namespace pisa
