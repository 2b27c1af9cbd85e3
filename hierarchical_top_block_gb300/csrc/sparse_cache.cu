// Attention of new tokens over selected 64-key blocks of the 8-bit cache: T queries a sequence
// (one in a decode step, several where tokens were drafted), query t at position seq_len[b] + t,
// each with its own block list per KV head, shared by the G_Q heads of the group.
//
// Work: K * 64 rows of 2 d + 8 bytes a (b, h_kv, t) against 4 G_Q d operations a row, at most 60 a
// byte: the reads bound it.  One group of warps per (b, h_kv, t) takes the list's half blocks
// (32 keys) in turn; where there are few groups (a single sequence), a group is a cluster of up to
// eight blocks whose partial results meet through distributed shared memory, so that every size
// is one launch and needs no scratch memory.
#include <cooperative_groups.h>

#include "cache_attn.cuh"
#include "kernels.cuh"

namespace pisa {
namespace {

namespace cg = cooperative_groups;
constexpr int THREADS = 128;

struct SparseParams {
  const uint16_t* q;
  const uint8_t* K;
  const uint8_t* V;
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

template <int D, bool HI>
__global__ void __launch_bounds__(THREADS) sparse_cache_kernel(SparseParams p, int cluster) {
  using Tile = CacheTile<D, 8>;
  __shared__ float po[4 * 16 * D];
  __shared__ float pm[4][16], pl[4][16], bm[16], bl[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  const int rank = blockIdx.x % cluster;
  const long long pair = blockIdx.x / cluster;  // (b, h_kv, t)
  const int t = (int)(pair % p.T);
  const long long bh = pair / p.T;
  const int b = (int)(bh / p.H_kv), hk = (int)(bh - (long long)b * p.H_kv);
  const int n_new = p.new_len ? p.new_len[b] : p.T, before = p.seq_len[b];
  const bool fits = n_new >= 0 && n_new <= p.T && before >= 0 && before <= p.N_cap - n_new;
  if (!fits && threadIdx.x == 0) report_error(p.err, ERR_BAD_INDEX);
  if (!fits || t >= n_new) return;  // the same for every block of the cluster
  const int pos = before + t;
  const int nblk = (p.N_cap + 63) >> 6;

  uint32_t qa[Tile::QW], qb[Tile::QW];
  const size_t row0 = ((size_t)b * p.T + t) * p.H_q + (size_t)hk * p.GQ;
  Tile::load_q(p.q + (row0 + r) * D, r < p.GQ, q, qa);
  Tile::load_q(p.q + (row0 + r + 8) * D, HI && r + 8 < p.GQ, q, qb);

  const int32_t* list = p.idx + ((size_t)bh * p.T + t) * p.Ksel;
  const uint8_t* K = p.K + (size_t)bh * p.N_cap * D;
  const uint8_t* V = p.V + (size_t)bh * p.N_cap * D;
  const float* ks = p.ks + (size_t)bh * p.N_cap;
  const float* vs = p.vs + (size_t)bh * p.N_cap;
  typename Tile::State st;
  Tile::clear(st);
  for (int g = rank * 4 + warp; g < 2 * p.Ksel; g += 4 * cluster) {
    const int blk = __ldg(list + (g >> 1));
    if (blk >= nblk && lane == 0) report_error(p.err, ERR_BAD_INDEX);
    if (blk < 0 || blk >= nblk) continue;
    const long long key0 = (long long)blk * 64 + 32 * (g & 1);
    const int n = (int)min((long long)Tile::KEYS, pos + 1 - key0);
    if (n <= 0) continue;
    typename Tile::Regs regs;
    Tile::load(regs, K, V, ks, vs, key0, n, r, q);
    Tile::template add<HI>(st, regs, qa, qb, n, p.sl2, q);
  }
  join_warps<D, 8, HI>(st, po, pm, pl, bm, bl, p.GQ);
  if (cluster == 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < p.GQ * D; i += THREADS) {
      const int row = i / D;
      p.o[row0 * D + i] = f32_to_bf16_rne(bl[row] > 0.f ? po[i] / bl[row] : bl[row] == 0.f ? 0.f : bl[row]);
    }
    if (p.lse && threadIdx.x < p.GQ)
      p.lse[row0 + threadIdx.x] = bl[threadIdx.x] == 0.f ? NEG_INF : (bm[threadIdx.x] + log2f(bl[threadIdx.x])) * LN2;
    return;
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  for (int i = rank * THREADS + threadIdx.x; i < p.GQ * D; i += THREADS * cluster) {
    const int row = i / D;
    float m = NEG_INF, l = 0.f, acc = 0.f;
    for (int c = 0; c < cluster; ++c) m = fmaxf(m, *cl.map_shared_rank(&bm[row], c));
    for (int c = 0; c < cluster; ++c) {
      const float mc = *cl.map_shared_rank(&bm[row], c);
      const float lc = *cl.map_shared_rank(&bl[row], c);
      if (mc == NEG_INF) {
        l += lc;  // 0, or NaN where every logit was
        continue;
      }
      const float f = fast_exp2(mc - m);
      l += lc * f;
      acc += *cl.map_shared_rank(&po[i], c) * f;
    }
    p.o[row0 * D + i] = f32_to_bf16_rne(l > 0.f ? acc / l : l == 0.f ? 0.f : l);
    if (p.lse && i % D == 0) p.lse[row0 + row] = l == 0.f ? NEG_INF : (m + log2f(l)) * LN2;
  }
  cl.sync();  // no block leaves while another reads its shared memory
}

template <int D, bool HI>
cudaError_t launch_t(const SparseParams& p, long long pairs, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * cluster));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sparse_cache_kernel<D, HI>, p, cluster);
}

}  // namespace

cudaError_t launch_sparse_cache(const uint16_t* q, const int8_t* Kq, const int8_t* Vq, const float* k_scale,
                                const float* v_scale, const int32_t* idx, const int32_t* seq_len,
                                const int32_t* new_len, uint16_t* o, float* lse, const Problem& pr, int num_sms,
                                uint32_t* err, cudaStream_t s) {
  SparseParams p;
  p.q = q;
  p.K = reinterpret_cast<const uint8_t*>(Kq);
  p.V = reinterpret_cast<const uint8_t*>(Vq);
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
  // enough blocks for two an SM, while every warp keeps a half block of its own
  int cluster = 1;
  while (cluster < 8 && pairs * cluster * 2 <= 2LL * num_sms && 4 * cluster < 2 * pr.K) cluster *= 2;
  const bool hi = pr.GQ > 8;
  if (pr.d == 128) return hi ? launch_t<128, true>(p, pairs, cluster, s) : launch_t<128, false>(p, pairs, cluster, s);
  return hi ? launch_t<64, true>(p, pairs, cluster, s) : launch_t<64, false>(p, pairs, cluster, s);
}

}  // namespace pisa
