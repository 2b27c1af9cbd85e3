// Attention of a batch over prefixes that its sequences share: R query rows in P groups, the
// rows of group p over all keys of prefix p (a bf16 or an 8-bit cache), joined with what each
// row attended on its own.
//
// Reading the prefix once for the whole group is the point: G_Q n_p query rows share each key, so
// with few rows the reads bound the work, and with many the products do (4 d operations a row
// and key).  Few rows: the kernel here, on mma.sync.  Many: prefix_tc.cu.
#include <algorithm>

#include "cache_attn.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "prefix_plan.cuh"

namespace pisa {
namespace {

constexpr int THREADS = 128;

// Joins a finished row's prefix part with its own part (log-sum-exp `own`) and writes one element.
__device__ __forceinline__ void write_out(const PrefixParams& p, size_t at, size_t row, bool write_lse, float acc,
                                          float m, float l, float own) {
  float fa, fo, lse;
  join_own(m, l, own, fa, fo, lse);
  float v = fa == 0.f ? 0.f : acc * fa;
  if (p.o_own && fo != 0.f) v += bf16_to_f32(p.o_own[at]) * fo;
  p.o[at] = f32_to_bf16_rne(v);
  if (write_lse && p.lse) p.lse[row] = lse;
}

// Few rows: tiles of 8 NH on mma.sync.  A block's four warps take the granules of a segment in turn,
// each with a ring of its own that it fills by TMA.
constexpr int few_blocks(int rows) { return rows > 8 ? 2 : 4; }  // a SM

template <int D, int BITS, int NH>
struct FewCfg {
  // A granule: 4 KB of K and of V, at most 32 keys (d = 64, bf16: 8 rows x 8 heads, 32768 keys take 12.2 us with 32
  // keys and 13.3 with 16).  Granules a warp has under way: one with 8 KB and the registers of 8 rows, where
  // four blocks a SM hide more than deeper rings with three (d = 128, codes, 26.5 against 27.0 and with four
  // granules 41 when measured; 16 rows, two blocks: 32.0 with two granules, 34.4 with one).
  static constexpr int KEYS = D * BITS <= 1024 ? 32 : 16;
  static constexpr int SLOTS = D * BITS == 512 || (NH == 2 && D == 128) ? 2 : 1;
  static constexpr int PER_SM = few_blocks(8 * NH);
  using Tile = CacheTile<D, BITS, KEYS, NH>;
  static constexpr uint32_t RING = 4 * SLOTS * Tile::BYTES, OUT = 4 * 8 * NH * D * 4;
  static constexpr uint32_t SMEM = RING > OUT ? RING : OUT;  // the outputs meet where the granules were
};

template <int D, int BITS, int NH>
__global__ void __launch_bounds__(THREADS, FewCfg<D, BITS, NH>::PER_SM) prefix_few_kernel(const __grid_constant__ CUtensorMap mapK,
                                                                const __grid_constant__ CUtensorMap mapV,
                                                                PrefixParams p) {
  pdl_trigger();
  using C = FewCfg<D, BITS, NH>;
  using Tile = typename C::Tile;
  constexpr int ROWS = 8 * NH;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* po = reinterpret_cast<float*>(smem);  // [4][ROWS][D]
  __shared__ uint64_t full[4][C::SLOTS];
  __shared__ float sn[4][16], sl[4][16], bo[ROWS];
  __shared__ float2 ml[ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  WarpRing<Tile, C::SLOTS> ring{smem + warp * C::SLOTS * Tile::BYTES, full[warp]};
  if (lane == 0) {
    prefetch_map(&mapK);
    prefetch_map(&mapV);
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&full[warp][i], 1);
    mbar_fence_init();
  }
  __syncwarp();
  PrefixWalk w;
  w.init(p, blockIdx.x, blockIdx.x == 0 && warp == 0);
  uint32_t s = 0, got = 0;  // granules used and fetched
  bool failed = false;
  while (w.next(p, blockIdx.x)) {
    const int m0 = w.tile * ROWS;                           // first query row of the tile
    const int rows = min(ROWS, w.g.n * p.GQ - m0);          // query row m: token m / G, head m % G
    auto q_row = [&](int i) {
      const int m = m0 + i, tok = m >> p.gq_bits;
      return ((size_t)(w.g.first + tok) * p.H_q + (size_t)w.head * p.GQ + (m - tok * p.GQ));
    };
    const int ph = w.p * p.H_kv + w.head;
    const int first = w.k0 * PREFIX_KT, key_end = min(w.g.len, w.k1 * PREFIX_KT);
    const int granules = key_end > first ? (key_end - first + C::KEYS - 1) / C::KEYS : 0;
#pragma unroll
    for (int i = 0; i < C::SLOTS; ++i)
      if (warp + 4 * i < granules && !failed) ring.fetch(got++, &mapK, &mapV, first + (warp + 4 * i) * C::KEYS, ph, lane);
    typename Tile::Query qr;
    Tile::load_q(qr, [&](int i) { return i < rows ? p.q + q_row(i) * D : nullptr; }, p.sl2, r, q);
    const float* ks = BITS == 8 ? p.ks + (size_t)ph * p.N_cap : nullptr;
    const float* vs = BITS == 8 ? p.vs + (size_t)ph * p.N_cap : nullptr;
    typename Tile::State st;
    Tile::clear(st);
    typename Tile::Scales sc, next_sc;
    auto scales = [&](typename Tile::Scales& x, int g) {
      if (g < granules) Tile::load_scales(x, ks, vs, first + g * C::KEYS, min(C::KEYS, key_end - first - g * C::KEYS), r);
    };
    scales(sc, warp);
    for (int g = warp; g < granules && !failed; g += 4, ++s) {
      scales(next_sc, g + 4);
      if (!ring.wait(s, p.err)) {
        failed = true;
        break;
      }
      Tile::add(st, ring.at(s), sc, qr, min(C::KEYS, key_end - first - g * C::KEYS), r, q);
      __syncwarp();  // the slot has been read
      if (g + 4 * C::SLOTS < granules) ring.fetch(got++, &mapK, &mapV, first + (g + 4 * C::SLOTS) * C::KEYS, ph, lane);
      sc = next_sc;
    }
    if (failed)  // copies still in flight land before their memory is used again (bounded)
      for (; s < got; ++s) ring.wait(s, p.err, 100000000ull);
    // read before any row is written: lse may be lse_own
    if (threadIdx.x < rows) bo[threadIdx.x] = p.lse_own ? p.lse_own[q_row(threadIdx.x)] : NEG_INF;
    join_warps<Tile, D>(st, po, sn, sl, ml, rows);
    if (w.slot < 0) {
      for (int i = threadIdx.x; i < rows * D; i += THREADS) {
        const int row = i / D, c = i - row * D;
        const size_t orow = q_row(row);
        write_out(p, orow * D + c, orow, c == 0, po[i], ml[row].x, ml[row].y, bo[row]);
      }
    } else {
      float* dst = p.part_o + (size_t)w.slot * ROWS * D;
      for (int i = threadIdx.x; i < rows * D; i += THREADS) dst[i] = po[i];
      if (threadIdx.x < rows) p.part_ml[(size_t)w.slot * ROWS + threadIdx.x] = ml[threadIdx.x];
    }
    fence_proxy_async();  // the next copies go where po was
    __syncthreads();
  }
}

// Joins the parts of every job that spans blocks.  A (row, query head) is joined by WARPS warps of a block's four: a
// part is D floats, one 16-byte (8-byte) piece a lane; the warps take the parts in turn, BATCH of them in
// flight, each with its own running maximum, and meet in shared memory.  Latency bounds it (launch 1 us, wait
// for the kernel before 1.7, bounds 1, sums 1-2), so few rows have all four warps each, and many have two, so that
// all rows are under way at once (217 tokens of 16 heads in five groups: the call takes 35.1 us, with four
// warps 38.6; 4 tokens of 32 heads, 38 parts a row: 23.0 with four, 25.4 with two).  BATCH 5: 64 tokens of 32 heads,
// 19 parts a row, took 47.0 us when chosen, with 8 (the registers spill) 48.8, with 4 48.7.
template <int D, int WARPS>
__global__ void __launch_bounds__(THREADS, 8) prefix_join_kernel(PrefixParams p) {
  constexpr int V = D / 32, BATCH = 5, PER = THREADS / 32 / WARPS;  // rows a block
  __shared__ float so[PER][WARPS][D];
  __shared__ float2 sml[PER][WARPS];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WARPS, sub = (threadIdx.x >> 5) / WARPS;
  static_assert(PER <= 2, "a barrier each");
  auto meet = [&] {
    if (sub == 0)
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
    else
      asm volatile("barrier.cta.sync 2, %0;" ::"n"(32 * WARPS) : "memory");
  };
  bool waited = false;  // the parts are written by the kernel before, the groups' bounds are not
  for (long long i = (long long)blockIdx.x * PER + sub; i < (long long)p.R * p.H_q; i += (long long)gridDim.x * PER) {
    const int row = (int)quotient(i, p.H_q), hq = (int)(i - (long long)row * p.H_q);
    int gp = 0;
    if (p.P > 1) {
      int lo = 0, hi = p.P;  // first group with row_start[g + 1] > row
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.row_start + mid + 1) > row)
          hi = mid;
        else
          lo = mid + 1;
      }
      gp = lo;
      if (gp >= p.P) continue;
    }
    const PrefixGroup g = prefix_group(p, gp);
    if (row < g.first || row >= g.first + g.n) continue;
    const int head = hq >> p.gq_bits;
    const int mrow = (row - g.first) * p.GQ + (hq - head * p.GQ);
    const int tile = mrow >> p.row_bits, local = mrow - (tile << p.row_bits);
    PrefixCut cut;
    long long s0 = 0;
    if (p.P == 1) {
      cut = prefix_cut_one(p, g);
    } else {
      if (!waited) pdl_wait();
      waited = true;
      cut = prefix_cut(p, p.base[p.P], (int)p.base[p.P + 1]);
      s0 = p.base[gp];
    }
    s0 += ((long long)head * g.tiles + tile) * (g.steps + cut.extra);  // the job's first position; its steps follow `extra`
    // (in range as long as nobody changes lengths or bounds under the call)
    const int c0 = min(cut.block_of(s0 + cut.extra), p.blocks - 1), c1 = min(cut.block_of(s0 + cut.extra + g.steps - 1), p.blocks - 1);
    if (c0 == c1) continue;  // finished by its block
    const int slot0 = 2 * c0 + (cut.start(c0) >= s0 ? 0 : 1);  // 1: the block had a job before
    const size_t at = (size_t)i * D + lane * V;
    float own = NEG_INF, own_o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) own_o[j] = 0.f;
    if (warp == 0 && p.lse_own) {  // (rows that the kernel before finished are others)
      own = p.lse_own[i];
      if constexpr (V == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p.o_own + at);
        own_o[0] = bf16_lo(x.x), own_o[1] = bf16_hi(x.x), own_o[2] = bf16_lo(x.y), own_o[3] = bf16_hi(x.y);
      } else {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p.o_own + at);
        own_o[0] = bf16_lo(x), own_o[1] = bf16_hi(x);
      }
    }
    if (!waited) pdl_wait();
    waited = true;
    float m = NEG_INF, l = 0.f, acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int c = c0 + warp; c <= c1; c += WARPS * BATCH) {
      float2 ml[BATCH];
      float x[BATCH][V];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int cc = c + u * WARPS;
        const bool in = cc <= c1;
        const size_t at = ((size_t)(cc == c0 || !in ? slot0 : 2 * cc) << p.row_bits) + local;
        ml[u] = in ? p.part_ml[at] : make_float2(NEG_INF, 0.f);
        const float* src = p.part_o + at * D + lane * V;
        if constexpr (V == 4)
          *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(src);
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < BATCH; ++u) top = fmaxf(top, ml[u].x);
      // sums in two factors of 2^(m - top): with value scales that differ by far it may be below fp32's range
      // where the sum times it is not
      const float h0 = m == NEG_INF ? 0.f : fast_exp2(0.5f * (m - top)), f0 = h0 * h0;
      if (m != NEG_INF) l = l * h0 * h0;
      m = top;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] *= f0;
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        if (ml[u].x == NEG_INF) {
          l += ml[u].y;  // 0, or NaN where every logit was
          continue;
        }
        const float h = fast_exp2(0.5f * (ml[u].x - m)), f = h * h;
        l += ml[u].y * h * h;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += x[u][j] * f;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) so[sub][warp][lane * V + j] = acc[j];
    if (lane == 0) sml[sub][warp] = make_float2(m, l);
    meet();
    if (warp == 0) {
      m = NEG_INF;
#pragma unroll
      for (int u = 0; u < WARPS; ++u) m = fmaxf(m, sml[sub][u].x);
      l = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.f;
#pragma unroll
      for (int u = 0; u < WARPS; ++u) {
        const float2 ml = sml[sub][u];
        if (ml.x == NEG_INF) {
          l += ml.y;
          continue;
        }
        const float h = fast_exp2(0.5f * (ml.x - m)), f = h * h;
        l += ml.y * h * h;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += so[sub][u][lane * V + j] * f;
      }
      float fa, fo, lse;
      join_own(m, l, own, fa, fo, lse);
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[j] = fa == 0.f ? 0.f : acc[j] * fa;
        if (fo != 0.f) v[j] += own_o[j] * fo;
      }
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(p.o + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      else
        *reinterpret_cast<uint32_t*>(p.o + at) = pack_bf16x2(v[0], v[1]);
      __syncwarp();  // lse may be lse_own: every lane has read it
      if (p.lse && lane == 0) p.lse[i] = lse;
    }
    meet();
  }
  if (!waited) pdl_wait();  // what comes next on the stream waits for this kernel alone
}

constexpr int MAX_SMS = 152;  // this GPU's: the scratch does not depend on the device at hand

// Which kernel, by the query rows a group has on average (the groups' own sizes are on the device; any kernel
// takes any).  The few-row kernel reads the prefix again for every 16 rows, the tensor-core one pays for its
// start (first scores after 6 us) and for 256 rows whether they are there or not.  At 8 KV heads x 32768 keys
// of d = 128, few-row against tensor-core kernel: codes, 32 rows 31 : 37 us, 48 rows 42 : 38; bf16, 16 rows 32 : 35,
// 32 rows 47 : 36; d = 64: codes, 32 rows 24 : 29, 64 rows 39 : 30; bf16, 16 rows 16 : 21, 32 rows 24 : 21.
// Uneven groups, one of 200 tokens among 60 of one, 16 / 4 heads, for which the average says few rows: 1024 codes each
// 52 : 82 us, 8192 codes 280 : 280.
struct Plan {
  bool tc;
  int rows, blocks, stop;
};
Plan prefix_plan(const Problem& p, bool codes) {
  const long long rows = ((long long)p.N * p.GQ + p.B - 1) / (p.B > 0 ? p.B : 1);
  const bool tc = rows > (codes ? 32 : 16);
  const int few = rows > 8 ? 16 : 8;
  Plan plan = tc ? Plan{true, TC_ROWS, MAX_SMS, 3} : Plan{false, few, few_blocks(few) * MAX_SMS, 2};
  // no more blocks (and scratch) than there can be steps: every group has at most one tile that is not full
  const long long tiles = (long long)p.N * p.GQ / plan.rows + p.B, steps = (p.N_cap + PREFIX_KT - 1) / PREFIX_KT;
  plan.blocks = (int)std::min<long long>(plan.blocks, p.H_kv * tiles * steps);
  return plan;
}

template <int D, int BITS, int NH>
cudaError_t launch_few(const PrefixParams& p, cudaStream_t s) {
  using C = FewCfg<D, BITS, NH>;
  CUtensorMap mapK, mapV;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.N_cap, (uint64_t)p.P * p.H_kv};
  const uint64_t strides[2] = {(uint64_t)C::Tile::ROWB, (uint64_t)p.N_cap * C::Tile::ROWB};
  const uint32_t box[3] = {BITS == 8 ? (uint32_t)D : 64u, (uint32_t)C::KEYS, 1};
  auto encode = [&](CUtensorMap* map, const void* base) {
    return BITS == 8 ? encode_byte_tensor_map(map, base, 3, dims, strides, box, C::Tile::SPAN)
                     : encode_tensor_map(map, base, 3, dims, strides, box);
  };
  if (!encode(&mapK, p.K) || !encode(&mapV, p.V)) return cudaErrorInvalidValue;
  auto kern = prefix_few_kernel<D, BITS, NH>;
  const cudaError_t e = allow_shared<prefix_few_kernel<D, BITS, NH>>(C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<p.blocks, THREADS, C::SMEM, s>>>(mapK, mapV, p);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_few_d(const PrefixParams& p, cudaStream_t s) {
  if (p.ks) return p.row_bits > 3 ? launch_few<D, 8, 2>(p, s) : launch_few<D, 8, 1>(p, s);
  return p.row_bits > 3 ? launch_few<D, 16, 2>(p, s) : launch_few<D, 16, 1>(p, s);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t prefix_workspace_bytes(const Problem& p) {
  size_t most = 0;  // of both kinds of cache
  for (bool codes : {false, true}) {
    const Plan plan = prefix_plan(p, codes);
    most = std::max(most, (size_t)2 * plan.blocks * plan.rows);
  }
  return up256(most * p.d * 4) + up256(most * 8) + up256((size_t)(p.B + 2) * 8);
}

cudaError_t launch_prefix_attn(const uint16_t* q, const void* Kp, const void* Vp, const float* k_scale,
                               const float* v_scale, const int32_t* prefix_len, const int32_t* row_start,
                               const uint16_t* o_own, const float* lse_own, uint16_t* o, float* lse, void* ws,
                               const Problem& pr, int num_sms, uint32_t* err, cudaStream_t s) {
  PrefixParams p;
  p.q = q;
  p.K = static_cast<const uint8_t*>(Kp);
  p.V = static_cast<const uint8_t*>(Vp);
  p.ks = k_scale;
  p.vs = v_scale;
  p.prefix_len = prefix_len;
  p.row_start = row_start;
  p.o_own = o_own;
  p.lse_own = lse_own;
  p.o = o;
  p.lse = lse;
  p.P = pr.B;
  p.R = pr.N;
  p.H_q = pr.H_q;
  p.H_kv = pr.H_kv;
  p.GQ = pr.GQ;
  p.N_cap = pr.N_cap;
  p.sl2 = pr.scale * LOG2E;
  p.err = err;
  const Plan plan = prefix_plan(pr, k_scale != nullptr);
  auto bits = [](int x) {  // of a power of two
    int b = 0;
    while ((1 << b) < x) ++b;
    return b;
  };
  p.gq_bits = bits(pr.GQ);
  p.row_bits = bits(plan.rows);
  p.blocks = plan.blocks;
  p.stop = plan.stop;
  const size_t parts = (size_t)2 * p.blocks * plan.rows;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.part_o = reinterpret_cast<float*>(w);
  w += up256(parts * pr.d * 4);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += up256(parts * 8);
  p.base = reinterpret_cast<long long*>(w);
  // Launched without the programmatic attribute: the call's inputs are there when the kernel starts, so the join,
  // launched with it, may read them before it waits for the parts.
  cudaError_t e;
  if (plan.tc)
    e = launch_prefix_tc(p, pr.d, s);
  else
    e = pr.d == 128 ? launch_few_d<128>(p, s) : launch_few_d<64>(p, s);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)p.R * p.H_q;
  const int warps = rows <= 8ll * num_sms ? 4 : 2;  // a row
  const dim3 grid((unsigned)std::min<long long>((rows * warps + 3) / 4, (long long)num_sms * 16));
  auto join = pr.d == 128 ? (warps == 4 ? prefix_join_kernel<128, 4> : prefix_join_kernel<128, 2>)
                          : (warps == 4 ? prefix_join_kernel<64, 4> : prefix_join_kernel<64, 2>);
  return launch_pdl(join, grid, dim3(THREADS), 0, s, p);
}

}  // namespace pisa
