// Attention of new tokens over selected 64-key blocks of the 8-bit cache: T queries a sequence
// (one in a decode step, several where tokens were drafted), query t at position seq_len[b] + t,
// each with its own block list per KV head, shared by the G_Q heads of the group.
//
// Work: K * 64 rows of 2 d + 8 bytes a (b, h_kv, t) against 4 G_Q d operations a row, at most 60 a
// byte: the reads bound it, so what counts is bytes in flight.  A block of four warps per (b, h_kv, t): the
// warps take the list's granules (KEYS keys) in turn, each with a ring of its own that it fills by TMA
// as far ahead as the ring goes.  Where there are few (b, h_kv, t), a cluster of up to eight blocks shares
// one list and the partial results meet through distributed shared memory, so that every size is one
// launch and needs no scratch memory.
//
// Measured (d = 128): 64 x 8 lists of 16 blocks, four query heads each (139 MB) 28.5 us, 4.9 TB/s; 152 x 2 lists of
// 32, sixteen heads each (164 MB) 33.6 us, 4.9 TB/s; 24 x 5 drafted tokens x 2 lists of 32 30-31 us (126 MB, a third
// of it from HBM); one list of 16 blocks under 16 heads 7.3 us, where launch, list, first copy and the
// cluster's two meetings follow one another.
#include <cooperative_groups.h>

#include "cache_attn.cuh"
#include "kernels.cuh"

namespace pisa {
namespace {

namespace cg = cooperative_groups;
constexpr int THREADS = 128;

struct SparseParams {
  const uint16_t* q;
  const float* ks;
  const float* vs;
  const int32_t* idx;
  const int32_t* seq_len;
  const int32_t* new_len;
  uint16_t* o;
  float* lse;
  int T, H_q, H_kv, GQ, Ksel, N_cap;
  float sl2;
  uint32_t* err;
};

// The granules of a list: its blocks in use, each cut into 64 / KEYS; of these every `of`-th, from the
// caller's first on, is the caller's.
template <int KEYS>
struct Granules {
  static constexpr int PER = 64 / KEYS;
  int blk;        // lane i: the list's i-th block in use
  int pos;        // the query's position
  int g, of, end; // next granule, stride, granules in all
  // `entry`: this lane's list entry, `use` whether it is in use; `scratch` [32] is this warp's.
  __device__ __forceinline__ void begin(int entry, bool use, int* scratch, int position, int mine, int n) {
    const int lane = threadIdx.x & 31;
    const uint32_t bits = __ballot_sync(0xffffffffu, use);
    if (use) scratch[__popc(bits & ((1u << lane) - 1u))] = entry;
    __syncwarp();
    blk = scratch[lane];  // (past the last one: never asked for)
    pos = position;
    g = mine;
    of = n;
    end = PER * __popc(bits);
  }
  // The caller's next granule with a visible key: its first key, or -1 at the end.  Warp-uniform.
  __device__ __forceinline__ int next() {
    while (g < end) {
      const int key0 = __shfl_sync(0xffffffffu, blk, g / PER) * 64 + KEYS * (g % PER);
      g += of;
      if (key0 <= pos) return key0;
    }
    return -1;
  }
};

template <int D, int NH>
struct SparseCfg {
  // Up to eight query heads: one granule of 32 keys under way a warp and four blocks a SM hide more than deeper
  // rings (64 x 8 lists of 16 blocks: 27.5 us when chosen; with two granules and three blocks 33.7).  Sixteen: the state
  // takes twice the registers, and two granules with two blocks are better (24 x 5 drafted tokens, lists of
  // 32 blocks: 29.3 us; one granule and three blocks 35.3, three and two 29.6).
  static constexpr int KEYS = 32, SLOTS = NH, PER_SM = NH == 1 ? 4 : 2;
  using Tile = CacheTile<D, 8, KEYS, NH>;
  static constexpr uint32_t RING = 4 * SLOTS * Tile::BYTES, OUT = 4 * 8 * NH * D * 4;
  static constexpr uint32_t SMEM = RING > OUT ? RING : OUT;  // the outputs meet where the granules were
};

template <int D, int NH>
__global__ void __launch_bounds__(THREADS, SparseCfg<D, NH>::PER_SM) sparse_cache_kernel(const __grid_constant__ CUtensorMap mapK,
                                                                    const __grid_constant__ CUtensorMap mapV,
                                                                    SparseParams p, int cluster) {
  using C = SparseCfg<D, NH>;
  using Tile = typename C::Tile;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* po = reinterpret_cast<float*>(smem);  // [4][8 NH][D]
  __shared__ uint64_t full[4][C::SLOTS];
  __shared__ float sn[4][16], sl[4][16];
  __shared__ float2 ml[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  if (lane == 0) {
    prefetch_map(&mapK);
    prefetch_map(&mapV);
  }
  const int rank = blockIdx.x % cluster;
  const long long pair = blockIdx.x / cluster;  // (b, h_kv, t)
  const int t = (int)(pair % p.T);
  const int bh = (int)(pair / p.T);
  const int b = bh / p.H_kv, hk = bh - b * p.H_kv;
  __shared__ int scratch[4][32];
  const int entry = lane < p.Ksel ? __ldg(p.idx + (size_t)pair * p.Ksel + lane) : -1;
  const int n_new = p.new_len ? p.new_len[b] : p.T, before = p.seq_len[b];
  const bool fits = n_new >= 0 && n_new <= p.T && before >= 0 && before <= p.N_cap - n_new;
  if (!fits && threadIdx.x == 0) report_error(p.err, ERR_BAD_INDEX);
  if (!fits || t >= n_new) return;  // the same for every block of the cluster
  const int pos = before + t;
  if (warp == 0 && entry >= ((p.N_cap + 63) >> 6)) report_error(p.err, ERR_BAD_INDEX);
  Granules<C::KEYS> list;
  list.begin(entry, entry >= 0 && entry <= (pos >> 6), scratch[warp], pos, rank * 4 + warp, 4 * cluster);
  WarpRing<Tile, C::SLOTS> ring{smem + warp * C::SLOTS * Tile::BYTES, full[warp]};
  if (lane == 0) {
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&full[warp][i], 1);
    mbar_fence_init();
  }
  __syncwarp();

  const float* ks = p.ks + (size_t)bh * p.N_cap;
  const float* vs = p.vs + (size_t)bh * p.N_cap;
  int keys[C::SLOTS];  // first keys of the granules in flight, the oldest first
  uint32_t got = 0, s = 0;
#pragma unroll
  for (int i = 0; i < C::SLOTS; ++i) {
    keys[i] = list.next();
    if (keys[i] >= 0) ring.fetch(got++, &mapK, &mapV, keys[i], bh, lane);
  }
  const size_t row0 = ((size_t)b * p.T + t) * p.H_q + (size_t)hk * p.GQ;
  typename Tile::Query qr;
  Tile::load_q(qr, [&](int i) { return i < p.GQ ? p.q + (row0 + i) * D : nullptr; }, p.sl2, r, q);
  typename Tile::State st;
  Tile::clear(st);
  typename Tile::Scales sc;
  if (keys[0] >= 0) Tile::load_scales(sc, ks, vs, keys[0], min(C::KEYS, pos + 1 - keys[0]), r);
  bool failed = false;
  while (keys[0] >= 0) {
    const int key0 = keys[0];
#pragma unroll
    for (int i = 0; i + 1 < C::SLOTS; ++i) keys[i] = keys[i + 1];
    keys[C::SLOTS - 1] = list.next();
    typename Tile::Scales next_sc;
    if (keys[0] >= 0) Tile::load_scales(next_sc, ks, vs, keys[0], min(C::KEYS, pos + 1 - keys[0]), r);
    if (!ring.wait(s, p.err)) {
      failed = true;
      break;
    }
    Tile::add(st, ring.at(s), sc, qr, min(C::KEYS, pos + 1 - key0), r, q);
    __syncwarp();  // the slot has been read
    if (keys[C::SLOTS - 1] >= 0) ring.fetch(got++, &mapK, &mapV, keys[C::SLOTS - 1], bh, lane);
    ++s;
    sc = next_sc;
  }
  if (failed)  // copies still in flight land before their memory is used again (bounded)
    for (; s < got; ++s) ring.wait(s, p.err, 100000000ull);
  join_warps<Tile, D>(st, po, sn, sl, ml, p.GQ);
  if (cluster == 1) {
    for (int i = threadIdx.x; i < p.GQ * D / 2; i += THREADS) {
      const float l = ml[2 * i / D].y, inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
      reinterpret_cast<uint32_t*>(p.o + row0 * D)[i] = pack_bf16x2(po[2 * i] * inv, po[2 * i + 1] * inv);
    }
    if (p.lse && threadIdx.x < p.GQ) {
      const float2 x = ml[threadIdx.x];
      p.lse[row0 + threadIdx.x] = x.y == 0.f ? NEG_INF : (x.x + log2f(x.y)) * LN2;
    }
    return;
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  // four columns a thread: one round trip to the other blocks where a column each took up to eight
  for (int i = 4 * (rank * THREADS + threadIdx.x); i < p.GQ * D; i += 4 * THREADS * cluster) {
    const int row = i / D;
    float2 x[8];
    float4 a[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)  // all of them under way at once
      if (c < cluster) {
        x[c] = *cl.map_shared_rank(&ml[row], c);
        a[c] = *cl.map_shared_rank(reinterpret_cast<float4*>(&po[i]), c);
      }
    float m = NEG_INF, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < cluster) m = fmaxf(m, x[c].x);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < cluster) {
        if (x[c].x == NEG_INF) {
          l += x[c].y;  // 0, or NaN where every logit was
          continue;
        }
        l += times_exp2(x[c].y, x[c].x - m);
        const float f = fast_exp2(x[c].x - m);
        acc.x += a[c].x * f;
        acc.y += a[c].y * f;
        acc.z += a[c].z * f;
        acc.w += a[c].w * f;
      }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    *reinterpret_cast<uint2*>(p.o + row0 * D + i) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (p.lse && i % D == 0) p.lse[row0 + row] = l == 0.f ? NEG_INF : (m + log2f(l)) * LN2;
  }
  cl.sync();  // no block leaves while another reads its shared memory
}

template <int D, int NH>
cudaError_t launch_t(const int8_t* Kq, const int8_t* Vq, const SparseParams& p, const Problem& pr, int cluster,
                     cudaStream_t s) {
  using C = SparseCfg<D, NH>;
  CUtensorMap mapK, mapV;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)pr.N_cap, (uint64_t)pr.B * pr.H_kv};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)pr.N_cap * D};
  const uint32_t box[3] = {(uint32_t)D, (uint32_t)C::KEYS, 1};
  if (!encode_byte_tensor_map(&mapK, Kq, 3, dims, strides, box, C::Tile::SPAN) ||
      !encode_byte_tensor_map(&mapV, Vq, 3, dims, strides, box, C::Tile::SPAN))
    return cudaErrorInvalidValue;
  auto kern = sparse_cache_kernel<D, NH>;
  cudaError_t e = allow_shared<sparse_cache_kernel<D, NH>>(C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)pr.B * pr.H_kv * pr.N * cluster));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, mapK, mapV, p, cluster);
}

}  // namespace

cudaError_t launch_sparse_cache(const uint16_t* q, const int8_t* Kq, const int8_t* Vq, const float* k_scale,
                                const float* v_scale, const int32_t* idx, const int32_t* seq_len,
                                const int32_t* new_len, uint16_t* o, float* lse, const Problem& pr, int num_sms,
                                uint32_t* err, cudaStream_t s) {
  SparseParams p;
  p.q = q;
  p.ks = k_scale;
  p.vs = v_scale;
  p.idx = idx;
  p.seq_len = seq_len;
  p.new_len = new_len;
  p.o = o;
  p.lse = lse;
  p.T = pr.N;
  p.H_q = pr.H_q;
  p.H_kv = pr.H_kv;
  p.GQ = pr.GQ;
  p.Ksel = pr.K;
  p.N_cap = pr.N_cap;
  p.sl2 = pr.scale * LOG2E;
  p.err = err;
  const long long pairs = (long long)pr.B * pr.H_kv * pr.N;
  // Blocks in a cluster, while every warp keeps granules of its own: two as long as all of them are resident at
  // once, more only while they are with half of the room left, since a cluster's blocks need free places in one
  // group of SMs.  (d = 128, lists of 32 blocks, 16 heads each: 38 lists 12.0 us with four blocks and 18.2 with
  // eight, 76 lists 15.1 with two and 21.6 with four, 152 lists 19.5 with two and 22.0 with one; lists of 16
  // blocks, four heads each: 32 lists 6.8 us with eight, 72 7.8 with four and 8.5 with eight, 152 10.0 with two
  // and 13.7 with four, 304 15.1 with two and 16.0 with one.)
  const bool wide = pr.GQ > 8;
  const long long room = (wide ? 2LL : 4LL) * num_sms;
  int cluster = 1;
  while (cluster < 8 && pairs * cluster * 2 <= (cluster == 1 ? room : room / 2) && 4 * cluster < 2 * pr.K) cluster *= 2;
  if (pr.d == 128)
    return wide ? launch_t<128, 2>(Kq, Vq, p, pr, cluster, s) : launch_t<128, 1>(Kq, Vq, p, pr, cluster, s);
  return wide ? launch_t<64, 2>(Kq, Vq, p, pr, cluster, s) : launch_t<64, 1>(Kq, Vq, p, pr, cluster, s);
}

}  // namespace pisa
