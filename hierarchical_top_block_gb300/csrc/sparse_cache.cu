// Attention of new tokens over selected 64-key blocks of the 8-bit cache: T queries a sequence
// (one in a decode step, several where tokens were drafted), query t at position seq_len[b] + t,
// each with its own block list per KV head, shared by the G_Q heads of the group.
//
// Work: K * 64 rows of 2 d + 8 bytes a (b, h_kv, t) against 4 G_Q d operations a row, at most 60 a
// byte: the reads bound it, so what counts is bytes in flight.  A block per (b, h_kv, t): one warp copies
// the list's half blocks (32 keys, 8 KB at d = 128) into a ring by TMA, as far ahead as the ring goes
// (64 KB, two blocks a SM), four warps take them in turn.  Where there are few (b, h_kv, t), a cluster of up to
// eight blocks shares one list and the partial results meet through distributed shared memory, so
// that every size is one launch and needs no scratch memory.
#include <cooperative_groups.h>

#include "cache_attn.cuh"
#include "kernels.cuh"

namespace pisa {
namespace {

namespace cg = cooperative_groups;
constexpr int THREADS = 160;  // four computing warps and the copying one

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

// The half blocks of a list that hold a visible key, in order: of each block in use (bits of b0) its
// first half, and its second one (b1).  A block of the cluster takes every `cluster`-th.
struct HalfBlocks {
  uint32_t b0, b1;
  int blk;       // this lane's list entry
  int l, half;   // place of the last one given
  int s, rank, cluster;
  __device__ __forceinline__ void begin(int r, int c) {
    l = -1;
    half = 1;
    s = 0;
    rank = r;
    cluster = c;
  }
  // The next one of this block's: its first key, or -1 at the end.  Warp-uniform.
  __device__ __forceinline__ int next() {
    while (true) {
      if (half == 0) {
        half = 1;
        if (!((b1 >> l) & 1u)) continue;
      } else {
        const uint32_t rest = l < 0 ? b0 : l == 31 ? 0u : b0 & (0xfffffffeu << l);
        if (rest == 0) return -1;
        l = __ffs(rest) - 1;
        half = 0;
      }
      if ((s++ & (cluster - 1)) == rank) return __shfl_sync(0xffffffffu, blk, l) * 64 + 32 * half;
    }
  }
};

template <int D, bool HI>
__global__ void __launch_bounds__(THREADS, 2) sparse_cache_kernel(const __grid_constant__ CUtensorMap mapK,
                                                               const __grid_constant__ CUtensorMap mapV, SparseParams p,
                                                               int cluster) {
  using Tile = CacheTile<D, 8>;
  using Ring = GranuleRing<D, 8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* po = reinterpret_cast<float*>(smem + Ring::SLOTS * Tile::BYTES);  // [4][16][D]
  __shared__ Ring ring;
  __shared__ float sm[4][16], sn[4][16], sl[4][16];
  __shared__ float2 ml[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  const int rank = blockIdx.x % cluster;
  const long long pair = blockIdx.x / cluster;  // (b, h_kv, t)
  const int t = (int)(pair % p.T);
  const int bh = (int)(pair / p.T);
  const int b = bh / p.H_kv, hk = bh - b * p.H_kv;
  HalfBlocks list;
  list.blk = lane < p.Ksel ? __ldg(p.idx + (size_t)pair * p.Ksel + lane) : -1;
  const int n_new = p.new_len ? p.new_len[b] : p.T, before = p.seq_len[b];
  const bool fits = n_new >= 0 && n_new <= p.T && before >= 0 && before <= p.N_cap - n_new;
  if (!fits && threadIdx.x == 0) report_error(p.err, ERR_BAD_INDEX);
  if (!fits || t >= n_new) return;  // the same for every block of the cluster
  const int pos = before + t;
  {
    const int nblk = (p.N_cap + 63) >> 6;
    if (warp == 4 && list.blk >= nblk) report_error(p.err, ERR_BAD_INDEX);
    const bool in = list.blk >= 0 && list.blk <= (pos >> 6);
    list.b0 = __ballot_sync(0xffffffffu, in);
    list.b1 = __ballot_sync(0xffffffffu, in && list.blk * 64 + 32 <= pos);
    list.begin(rank, cluster);
  }
  if (threadIdx.x == 0) ring.init(1);
  __syncthreads();

  const size_t row0 = ((size_t)b * p.T + t) * p.H_q + (size_t)hk * p.GQ;
  if (warp == 4) {
    // ------------------------------ copies ------------------------------
    uint32_t s = 0;
    for (int key0 = list.next(); key0 >= 0; key0 = list.next(), ++s) {
      if (!mbar_wait_warp(&ring.empty[s % Ring::SLOTS], ((s / Ring::SLOTS) & 1) ^ 1, p.err)) break;
      if (lane == 0) Tile::copy(smem + (s % Ring::SLOTS) * Tile::BYTES, &mapK, &mapV, &ring.full[s % Ring::SLOTS], key0, bh);
    }
    // copies still in flight land before shared memory goes away (bounded; the others wait for theirs too)
    for (uint32_t u = s > Ring::SLOTS ? s - Ring::SLOTS : 0; u < s; ++u)
      mbar_wait_warp(&ring.full[u % Ring::SLOTS], (u / Ring::SLOTS) & 1, p.err, 100000000ull);
  } else {
    typename Tile::Query qr;
    Tile::template load_q<HI>(qr, r < p.GQ ? p.q + (row0 + r) * D : nullptr,
                              r + 8 < p.GQ ? p.q + (row0 + r + 8) * D : nullptr, p.sl2, q);
    const float* ks = p.ks + (size_t)bh * p.N_cap;
    const float* vs = p.vs + (size_t)bh * p.N_cap;
    typename Tile::State st;
    Tile::clear(st);
    uint32_t s = 0;
    auto mine = [&]() {  // this warp's next half block
      int key0 = list.next();
      while (key0 >= 0 && (int)(s & 3) != warp) {
        ++s;
        key0 = list.next();
      }
      return key0;
    };
    int key0 = mine();
    typename Tile::Scales sc, next_sc;
    if (key0 >= 0) Tile::load_scales(sc, ks, vs, key0, min(Tile::KEYS, pos + 1 - key0), q);
    while (key0 >= 0) {
      const uint32_t slot = s % Ring::SLOTS, phase = (s / Ring::SLOTS) & 1;
      ++s;
      const int after = mine();
      if (after >= 0) Tile::load_scales(next_sc, ks, vs, after, min(Tile::KEYS, pos + 1 - after), q);
      if (!mbar_wait_warp(&ring.full[slot], phase, p.err)) break;
      Tile::template add<HI>(st, smem_u32(smem + slot * Tile::BYTES), sc, qr, min(Tile::KEYS, pos + 1 - key0), r, q);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[slot]);
      key0 = after;
      sc = next_sc;
    }
    join_warps<D, 8, HI, 1>(st, po, sm, sn, sl, ml, p.GQ, [] { asm volatile("bar.sync 1, 128;" ::: "memory"); });
    if (cluster == 1) {
      for (int i = threadIdx.x; i < p.GQ * D / 2; i += 128) {
        const float l = ml[2 * i / D].y, inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        reinterpret_cast<uint32_t*>(p.o + row0 * D)[i] = pack_bf16x2(po[2 * i] * inv, po[2 * i + 1] * inv);
      }
      if (p.lse && threadIdx.x < p.GQ) {
        const float2 x = ml[threadIdx.x];
        p.lse[row0 + threadIdx.x] = x.y == 0.f ? NEG_INF : (x.x + log2f(x.y)) * LN2;
      }
    }
  }
  if (cluster == 1) return;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  if (warp < 4) {
    for (int i = rank * 128 + threadIdx.x; i < p.GQ * D; i += 128 * cluster) {
      const int row = i / D;
      float m = NEG_INF, l = 0.f, acc = 0.f;
      for (int c = 0; c < cluster; ++c) m = fmaxf(m, cl.map_shared_rank(&ml[row], c)->x);
      for (int c = 0; c < cluster; ++c) {
        const float2 x = *cl.map_shared_rank(&ml[row], c);
        if (x.x == NEG_INF) {
          l += x.y;  // 0, or NaN where every logit was
          continue;
        }
        const float f = fast_exp2(x.x - m);
        l += x.y * f;
        acc += *cl.map_shared_rank(&po[i], c) * f;
      }
      p.o[row0 * D + i] = f32_to_bf16_rne(l > 0.f ? acc / l : l == 0.f ? 0.f : l);
      if (p.lse && i % D == 0) p.lse[row0 + row] = l == 0.f ? NEG_INF : (m + log2f(l)) * LN2;
    }
  }
  cl.sync();  // no block leaves while another reads its shared memory
}

template <int D, bool HI>
cudaError_t launch_t(const CUtensorMap& mapK, const CUtensorMap& mapV, const SparseParams& p, long long pairs,
                     int cluster, cudaStream_t s) {
  constexpr size_t smem = GranuleRing<D, 8>::SLOTS * CacheTile<D, 8>::BYTES + 4 * 16 * D * sizeof(float);
  auto kern = sparse_cache_kernel<D, HI>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * cluster));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
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
  CUtensorMap mapK, mapV;
  const uint64_t dims[3] = {(uint64_t)pr.d, (uint64_t)pr.N_cap, (uint64_t)pr.B * pr.H_kv};
  const uint64_t strides[2] = {(uint64_t)pr.d, (uint64_t)pr.N_cap * pr.d};
  const uint32_t box[3] = {(uint32_t)pr.d, 32, 1};
  if (!encode_byte_tensor_map(&mapK, Kq, 3, dims, strides, box, pr.d) ||
      !encode_byte_tensor_map(&mapV, Vq, 3, dims, strides, box, pr.d))
    return cudaErrorInvalidValue;
  const long long pairs = (long long)pr.B * pr.H_kv * pr.N;
  // enough blocks for two an SM, while every warp keeps a half block of its own
  int cluster = 1;
  while (cluster < 8 && pairs * cluster * 2 <= 2LL * num_sms && 4 * cluster < 2 * pr.K) cluster *= 2;
  const bool hi = pr.GQ > 8;
  if (pr.d == 128)
    return hi ? launch_t<128, true>(mapK, mapV, p, pairs, cluster, s) : launch_t<128, false>(mapK, mapV, p, pairs, cluster, s);
  return hi ? launch_t<64, true>(mapK, mapV, p, pairs, cluster, s) : launch_t<64, false>(mapK, mapV, p, pairs, cluster, s);
}

}  // namespace pisa
