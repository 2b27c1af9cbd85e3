// The attention weight that every key of the paged cache has got from the new tokens:
//
//   w_c (+)= sum over the tokens t that see key c and the query heads of its KV head of  exp(scale q_t . k_c - lse_t)
//
// with the tokens' log-sum-exps from the attention.  On the tensor cores with the keys as the products' rows,
//   S^T = K Q^T (256 keys x NQ query rows, fp32 in tensor memory),
// so that a thread of the epilogue has one key and sums 2^(S scale log2 e - lse log2 e) over its columns in
// registers, without meeting another thread.  2 d operations and one exponential a pair of key and row: with d = 128
// both pipes are about equally busy.  With few rows (a decode step) K is read once and bounds it.
//
// A job is (sequence, KV head, 256 keys); its steps are the tiles of NQ query rows that see one of the keys.  The jobs'
// steps form one line that is cut into equal ranges, as the attention's (paged.cuh); of a job that spans blocks each
// stores its sums, and a second kernel adds them in order.  Results are the same in every run.
//
// Roles: epilogue warps, a producer (TMA: K by pages, Q), a warp that issues the
// MMAs, a warp that puts the rows' log-sum-exps into shared memory.  TMEM: two stages of two halves of 128 columns.
// Every wait is bounded.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"
#include "pdl.cuh"

namespace pisa {
namespace {

constexpr int KEYS = 256;                   // a job
// Epilogue warps: sixteen, a warpgroup a stage and half of the keys, or for few rows eight, a warpgroup a half.
constexpr int epilogue_warps(int nq) { return nq > 16 ? 16 : 8; }
constexpr int K_SLOTS = 2, L_SLOTS = 3;

// Jobs of key tiles: tile i has the keys 256 i .., and begins with the first tile of query rows that sees one of them.
// p.row_bits: rows of a query tile.
struct KeyJobs {
  int tiles, rows, shift, L;  // key tiles a head; tiles of query rows; tokens a tile, 2 to this
  bool causal;
  __device__ __forceinline__ KeyJobs(const PagedParams& p, const PagedSeq& s) {
    shift = p.row_bits - p.gq_bits;
    rows = (s.n + (1 << shift) - 1) >> shift;
    if (!p.accumulate) rows = max(rows, 1);  // (the weights of a sequence without new tokens are cleared)
    tiles = rows > 0 ? (s.L + s.n + KEYS - 1) / KEYS : 0;
    L = s.L;
    causal = p.causal && s.n > 0;
  }
  __device__ __forceinline__ int first(int i) const { return causal ? max(0, KEYS * i - L) >> shift : 0; }
  __device__ __forceinline__ int steps(int i) const { return rows - first(i); }
  // Steps of the tiles before tile k.  From the first tile i0 that begins behind the old keys on, first(i) =
  // (256 / TT) i - ceil(L / TT), since a tile's TT tokens divide 256.
  __device__ __forceinline__ long long before(int k) const {
    long long sum = (long long)k * rows;
    const int i0 = (L + KEYS - 1) / KEYS;
    if (causal && k > i0) {
      const long long n = k - i0;
      sum -= ((((long long)i0 + k - 1) * n / 2) << (8 - shift)) - n * ((L + (1 << shift) - 1) >> shift);
    }
    return sum;
  }
  __device__ __forceinline__ long long span(int extra) const { return before(tiles) + (long long)tiles * extra; }
  __device__ __forceinline__ int tile_at(long long x, int extra) const { return tile_of(*this, x, extra); }
};
using KeyWalk = PagedLine<KeyJobs>;

template <int D, int NQ>
struct Cfg {
  static constexpr uint32_t K_BYTES = KEYS * D * 2, Q_BYTES = NQ * D * 2;
  static constexpr int Q_SLOTS = 3;
  static constexpr int EPILOGUE = epilogue_warps(NQ), PRODUCER = EPILOGUE, ISSUER = EPILOGUE + 1;  // warps
  static constexpr int THREADS = 32 * (EPILOGUE + 3);
  static constexpr size_t TILES = K_SLOTS * K_BYTES + Q_SLOTS * Q_BYTES;
};

struct Shared {
  uint64_t k_full[K_SLOTS], k_empty[K_SLOTS], q_full[3], q_empty[3];
  uint64_t l_full[L_SLOTS], l_empty[L_SLOTS], s_full[2][2], s_empty[2][2], x_full[2], x_empty[2], drain;
  __align__(16) float neg[L_SLOTS][128];  // -lse log2 e of a tile's rows
  float sum[2][128];                      // of the second stage's warps, for the first's
  uint32_t tmem;
};

// Adds the sum of a key to its weight, or puts it there.
__device__ __forceinline__ void put_weight(const PagedParams& p, const KeyWalk& w, int c, float sum) {
  if (c >= w.s.L + w.s.n) return;
  const int page = page_of(p.table + (size_t)w.b * p.M, p.P, c >> p.s_bits, p.err);
  if (page == p.P) return;
  float* at = p.w + (((size_t)page * p.H_kv + w.head) << p.s_bits) + (c & ((1 << p.s_bits) - 1));
  *at = p.accumulate ? *at + sum : sum;
}

__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&x)[32]) { tmem_ld32(at, x); }
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&x)[16]) { tmem_ld16(at, x); }

// Adds COLS columns of x (from column c on of the tile) with the rows' terms at `neg`.  MASK 1: columns lo .. hi - 1 alone; 2:
// of them those whose row saw something, whatever the product made of it.
template <int COLS, int MASK>
__device__ __forceinline__ void add_columns(const uint32_t (&x)[COLS], const float* neg, unsigned long long sl2, int lo, int hi,
                                            unsigned long long (&sum)[2]) {
#pragma unroll
  for (int c = 0; c < COLS; c += 4) {
    const float4 l = *reinterpret_cast<const float4*>(neg + c);
    float a, b, e, f;
    unpack_f32x2(fma_f32x2(pack_u32x2(x[c], x[c + 1]), sl2, pack_f32x2(l.x, l.y)), a, b);
    unpack_f32x2(fma_f32x2(pack_u32x2(x[c + 2], x[c + 3]), sl2, pack_f32x2(l.z, l.w)), e, f);
    if constexpr (MASK > 0) {
      if (c < lo || c >= hi || (MASK == 2 && l.x == NEG_INF)) a = NEG_INF;
      if (c + 1 < lo || c + 1 >= hi || (MASK == 2 && l.y == NEG_INF)) b = NEG_INF;
      if (c + 2 < lo || c + 2 >= hi || (MASK == 2 && l.z == NEG_INF)) e = NEG_INF;
      if (c + 3 < lo || c + 3 >= hi || (MASK == 2 && l.w == NEG_INF)) f = NEG_INF;
    }
    sum[0] = add_f32x2(sum[0], pack_f32x2(fast_exp2(a), fast_exp2(b)));
    sum[1] = add_f32x2(sum[1], pack_f32x2(fast_exp2(e), fast_exp2(f)));
  }
}

template <int D, int NQ>
__global__ void __launch_bounds__(Cfg<D, NQ>::THREADS, 1)
    paged_weights_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapQ, PagedParams p) {
  pdl_trigger();
  using C = Cfg<D, NQ>;
  constexpr int DH = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sK = smem;
  uint8_t* sQ = smem + K_SLOTS * C::K_BYTES;
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::TILES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* err = p.err;
  if (warp == C::PRODUCER) {
    if (lane == 0) {
      prefetch_map(&mapK);
      prefetch_map(&mapQ);
      for (int i = 0; i < K_SLOTS; ++i) {
        mbar_init(&sh.k_full[i], 1);
        mbar_init(&sh.k_empty[i], 1);
      }
      for (int i = 0; i < C::Q_SLOTS; ++i) {
        mbar_init(&sh.q_full[i], 1);
        mbar_init(&sh.q_empty[i], 1);
      }
      for (int i = 0; i < L_SLOTS; ++i) {
        mbar_init(&sh.l_full[i], 1);
        mbar_init(&sh.l_empty[i], 8);  // (two warpgroups use a tile's)
      }
      for (int i = 0; i < 2; ++i)
        for (int g = 0; g < 2; ++g) {
          mbar_init(&sh.s_full[i][g], 1);
          mbar_init(&sh.s_empty[i][g], 4);
        }
      for (int g = 0; g < 2; ++g) {
        mbar_init(&sh.x_full[g], 4);
        mbar_init(&sh.x_empty[g], 4);
      }
      mbar_init(&sh.drain, 1);
      mbar_fence_init();
    }
    __syncwarp();
  } else if (warp == C::ISSUER) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  KeyWalk w;
  w.init(p, blockIdx.x, blockIdx.x == 0 && warp == 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  uint32_t nt = 0, jobs = 0;  // steps and jobs so far
  bool failed = false;

  if (warp < C::EPILOGUE) {
    // ------------------------------ epilogue ------------------------------
    const int half = (warp >> 2) & 1, mine = warp >> 3, key = 128 * half + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const unsigned long long sl2 = pack_f32x2(p.sl2, p.sl2);
    while (!failed && w.next(p, blockIdx.x)) {
      const KeyJobs j(p, w.s);
      const int c = w.tile * KEYS + key, t0 = j.first(w.tile) + w.k0;
      float total = 0.f;
      for (int t = w.k0; t < w.k1; ++t, ++nt) {
        if (C::EPILOGUE == 16 && (int)(nt & 1) != mine) continue;
        const int m0 = (t0 + t - w.k0) * NQ, hi = (w.s.n << p.gq_bits) - m0;  // rows in use: those before hi
        const int lo = p.causal ? ((c - w.s.L) << p.gq_bits) - m0 : 0;        // that see the key: from lo on
        const uint32_t st = nt & 1, ls = nt % L_SLOTS;
        const bool l_here = mbar_try_wait(&sh.l_full[ls], (nt / L_SLOTS) & 1), s_here = mbar_try_wait(&sh.s_full[st][half], (nt >> 1) & 1);
        if (!__all_sync(0xffffffffu, l_here && s_here) && (!mbar_wait_warp(&sh.l_full[ls], (nt / L_SLOTS) & 1, err) ||
                                                           !mbar_wait_warp(&sh.s_full[st][half], (nt >> 1) & 1, err))) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem + lanes + st * 256 + half * 128;
        const bool mask = __any_sync(0xffffffffu, lo > 0) || hi < NQ;
        unsigned long long sum[2] = {0ull, 0ull};
        constexpr int COLS = NQ < 32 ? NQ : 32;
#pragma unroll
        for (int cc = 0; cc < NQ; cc += COLS) {
          uint32_t x[COLS];
          load_columns(at + cc, x);
          tmem_wait_ld();
          if (!mask)
            add_columns<COLS, 0>(x, sh.neg[ls] + cc, sl2, 0, 0, sum);
          else if (cc < hi)
            add_columns<COLS, 1>(x, sh.neg[ls] + cc, sl2, lo - cc, hi - cc, sum);
        }
        auto summed = [&] {
          float a, b, e, f;
          unpack_f32x2(sum[0], a, b);
          unpack_f32x2(sum[1], e, f);
          return (a + b) + (e + f);
        };
        float y = summed();
        if (__any_sync(0xffffffffu, y != y)) {  // perhaps of a row that saw nothing (looked for here alone: 1% of a tile)
          sum[0] = sum[1] = 0ull;
#pragma unroll 1
          for (int cc = 0; cc < min(NQ, hi); cc += 16) {
            uint32_t x[16];
            load_columns(at + cc, x);
            tmem_wait_ld();
            add_columns<16, 2>(x, sh.neg[ls] + cc, sl2, lo - cc, hi - cc, sum);
          }
          y = summed();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.s_empty[st][half]);
          mbar_arrive(&sh.l_empty[ls]);
        }
        total += y;
      }
      if (failed) break;
      if constexpr (C::EPILOGUE == 16) {  // the two stages' sums meet
        if (mine == 1) {
          if (!mbar_wait_warp(&sh.x_empty[half], (jobs & 1) ^ 1, err)) break;
          sh.sum[half][key & 127] = total;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.x_full[half]);
          ++jobs;
          continue;
        }
        if (!mbar_wait_warp(&sh.x_full[half], jobs & 1, err)) break;
        total += sh.sum[half][key & 127];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.x_empty[half]);
        ++jobs;
      }
      if (w.slot < 0)
        put_weight(p, w, c, total);
      else
        p.part_o[(size_t)w.slot * KEYS + key] = total;
    }
  } else if (warp == C::PRODUCER) {
    // ------------------------------ producer ------------------------------
    const int box_bits = min(p.s_bits, 7);
    const int piece = lane & (DH - 1), box = lane / DH;  // this lane's copy of a K tile (256 keys: at most 16 copies)
    const bool copies = box << box_bits < KEYS;
    while (!failed && w.next(p, blockIdx.x)) {
      const KeyJobs j(p, w.s);
      const int key = w.tile * KEYS + (box << box_bits), in = box << box_bits;
      const int page = copies && key < w.s.L + w.s.n ? page_of(p.table + (size_t)w.b * p.M, p.P, key >> p.s_bits, err) : p.P;
      const uint32_t ks = jobs % K_SLOTS;
      if (!mbar_wait_warp(&sh.k_empty[ks], ((jobs / K_SLOTS) & 1) ^ 1, err)) break;
      if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[ks], C::K_BYTES);
      __syncwarp();
      if (copies)
        tma_load_4d(sK + ks * C::K_BYTES + (in >> 7) * (128 * D * 2) + piece * (128 * 128) + (in & 127) * 128, &mapK,
                    &sh.k_full[ks], 64 * piece, key & ((1 << p.s_bits) - 1), w.head, page);
      __syncwarp();
      ++jobs;
      const int t0 = j.first(w.tile);
      for (int t = w.k0; t < w.k1; ++t, ++nt) {
        const uint32_t qs = nt % C::Q_SLOTS;
        if (!mbar_wait_warp(&sh.q_empty[qs], ((nt / C::Q_SLOTS) & 1) ^ 1, err)) {
          failed = true;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full[qs], C::Q_BYTES);
          for (int i = 0; i < DH; ++i)
            tma_load_4d(sQ + qs * C::Q_BYTES + i * (NQ * 128), &mapQ, &sh.q_full[qs], 64 * i, 0, w.head,
                        w.s.first + ((t0 + t) << (p.row_bits - p.gq_bits)) + (p.R == 0 ? 1 : 0));
        }
        __syncwarp();
      }
    }
    // copies still in flight land before shared memory goes away (bounded; at once unless a wait failed)
    if (lane == 0) {
      for (uint32_t u = jobs > K_SLOTS ? jobs - K_SLOTS : 0; u < jobs; ++u)
        mbar_wait(&sh.k_full[u % K_SLOTS], (u / K_SLOTS) & 1, err, 100000000ull);
      for (uint32_t u = nt > C::Q_SLOTS ? nt - C::Q_SLOTS : 0; u < nt; ++u)
        mbar_wait(&sh.q_full[u % C::Q_SLOTS], (u / C::Q_SLOTS) & 1, err, 100000000ull);
    }
    __syncwarp();
  } else if (warp == C::ISSUER) {
    // ------------------------------ MMAs ------------------------------
    // (A step's barriers are asked for together: one after the other they took 150 clocks each though nothing was
    // missing, 425 us for 2048 tokens of 32 / 8 heads over 32768 keys.)
    constexpr uint32_t id = idesc_bf16_f32(128, NQ);
    const uint64_t k_desc = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint32_t hi = (uint32_t)(k_desc >> 32), k_lo = (uint32_t)k_desc, q_lo = (uint32_t)smem_desc_sw128(smem_u32(sQ), 16, 1024);
    auto desc = [&](uint32_t lo) { return pack_u32x2(lo, hi); };
    Ring<K_SLOTS> ks;
    Ring<C::Q_SLOTS> qs;
    Ring<2> st;
    while (!failed && w.next(p, blockIdx.x)) {
      for (int t = w.k0; t < w.k1 && !failed; ++t) {
        const bool k = t > w.k0 || mbar_try_wait(&sh.k_full[ks.slot], ks.phase), q = mbar_try_wait(&sh.q_full[qs.slot], qs.phase);
        const bool s0 = mbar_try_wait(&sh.s_empty[st.slot][0], st.phase ^ 1), s1 = mbar_try_wait(&sh.s_empty[st.slot][1], st.phase ^ 1);
        if (!__all_sync(0xffffffffu, k && q && s0 && s1))
          failed = (t == w.k0 && !mbar_wait_warp(&sh.k_full[ks.slot], ks.phase, err)) ||
                   !mbar_wait_warp(&sh.q_full[qs.slot], qs.phase, err) || !mbar_wait_warp(&sh.s_empty[st.slot][0], st.phase ^ 1, err) ||
                   !mbar_wait_warp(&sh.s_empty[st.slot][1], st.phase ^ 1, err);
        if (failed) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t a = k_lo + ((ks.slot * C::K_BYTES + half * (128 * D * 2)) >> 4), b = q_lo + ((qs.slot * C::Q_BYTES) >> 4);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              umma_bf16(tmem + st.slot * 256 + half * 128, desc(a + (((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4)),
                        desc(b + (((s >> 2) * (NQ * 128) + (s & 3) * 32) >> 4)), id, s > 0 ? 1u : 0u);
            umma_commit(&sh.s_full[st.slot][half]);
          }
          umma_commit(&sh.q_empty[qs.slot]);
          if (t == w.k1 - 1) umma_commit(&sh.k_empty[ks.slot]);
        }
        __syncwarp();
        qs.next();
        st.next();
      }
      ks.next();
    }
    if (elect_one()) {  // every MMA issued has completed before the tensor memory is released (bounded)
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, err);
    }
    __syncwarp();
  } else {
    // ------------------------------ the rows' log-sum-exps ------------------------------
    constexpr int PER = (NQ + 31) / 32;
    while (!failed && w.next(p, blockIdx.x)) {
      const KeyJobs j(p, w.s);
      const int t0 = j.first(w.tile);
      auto read = [&](int t, float (&x)[PER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int m = (t0 + t) * NQ + 32 * i + lane, tok = m >> p.gq_bits;
          x[i] = NEG_INF;
          if (t < w.k1 && tok < w.s.n)
            x[i] = __ldg(p.lse_in + (size_t)(w.s.first + tok) * p.H_q + w.head * p.GQ + (m - (tok << p.gq_bits)));
        }
      };
      float next[PER];
      read(w.k0, next);
      for (int t = w.k0; t < w.k1; ++t, ++nt) {
        const uint32_t ls = nt % L_SLOTS;
        float x[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = next[i];
        read(t + 1, next);
        if (!mbar_wait_warp(&sh.l_empty[ls], ((nt / L_SLOTS) & 1) ^ 1, err)) {
          failed = true;
          break;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)  // a row that saw nothing gives nothing
          if (32 * i + lane < NQ) sh.neg[ls][32 * i + lane] = x[i] == NEG_INF ? NEG_INF : -x[i] * LOG2E;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.l_full[ls]);
      }
    }
    if (lane == 0) p.split[blockIdx.x] = w.split(p, blockIdx.x);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the parts of the jobs that span blocks, a key a thread.
__global__ void __launch_bounds__(KEYS) paged_weights_join_kernel(PagedParams p) {
  pdl_wait();
  const PagedSplit x = p.split[blockIdx.x];
  KeyWalk w;
  if (!w.take(x)) return;
  float sum = p.part_o[(size_t)x.slot0 * KEYS + threadIdx.x];
  for (int c = blockIdx.x + 1; c <= x.c1; ++c) sum += p.part_o[(size_t)2 * c * KEYS + threadIdx.x];
  put_weight(p, w, w.tile * KEYS + threadIdx.x, sum);
}

constexpr int MAX_SMS = 152;  // this GPU's: the scratch does not depend on the device at hand

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int D, int NQ>
cudaError_t launch_t(const PagedParams& p, cudaStream_t s) {
  using C = Cfg<D, NQ>;
  CUtensorMap mapK, mapQ = {};
  if (!encode_page_map(&mapK, p.K, D, 1 << p.s_bits, p.H_kv, p.P, 1 << std::min(p.s_bits, 7))) return cudaErrorInvalidValue;
  // (without rows the map is over one token, behind which the copies begin: nothing is read, any address does)
  if (!encode_token_map(&mapQ, p.R > 0 ? p.q : p.K, D, p.GQ, p.H_kv, std::max(p.R, 1), p.q_stride, NQ)) return cudaErrorInvalidValue;
  constexpr size_t smem = C::TILES + sizeof(Shared);
  static_assert(smem <= 227 * 1024, "a block's shared memory");
  const cudaError_t e = allow_shared<paged_weights_kernel<D, NQ>>(smem);
  if (e != cudaSuccess) return e;
  paged_weights_kernel<D, NQ><<<p.blocks, C::THREADS, smem, s>>>(mapK, mapQ, p);
  return cudaGetLastError();
}

}  // namespace

size_t paged_weights_workspace_bytes(const Problem& p) {
  return up256((size_t)2 * MAX_SMS * KEYS * 4) + up256((size_t)MAX_SMS * sizeof(PagedSplit));
}

cudaError_t launch_paged_weights(const uint16_t* q, long long q_stride, const float* lse, const uint16_t* Kp, float* w,
                                 const int32_t* table, const int32_t* seq_len, const int32_t* row_start, bool accumulate,
                                 void* ws, const Problem& pr, const Pages& pg, uint32_t* err, cudaStream_t s) {
  PagedParams p = {};
  p.q = q;
  p.lse_in = lse;
  p.K = Kp;
  p.w = w;
  p.table = table;
  p.seq_len = seq_len;
  p.row_start = row_start;
  p.q_stride = q_stride;
  p.B = pr.B;
  p.R = pr.N;
  p.H_q = pr.H_q;
  p.H_kv = pr.H_kv;
  p.GQ = pr.GQ;
  p.P = pg.P;
  p.M = pg.M;
  p.s_bits = pg.s_bits;
  while ((1 << p.gq_bits) < pr.GQ) ++p.gq_bits;
  p.causal = pr.causal;
  p.accumulate = accumulate;
  p.sl2 = pr.scale * LOG2E;
  p.err = err;
  // rows a sequence on average: tiles of 16 where one does (32 sequences of 8192 keys, 8 KV heads, d = 128, against tiles of
  // 128: 4 rows 92.8 : 99.8 us, 16 rows 93.1 : 100.8, 24 rows 100.8 : 100.3, 64 rows 146 : 112; a mixed batch, 128 x 1 token
  // of 4000 keys and 256 after 30000, accumulated, 420 : 280, alone 182 and 65; 255 of 1000 and a prompt of 700 117 : 182)
  const bool few = (long long)pr.N * pr.GQ <= 16ll * pr.B;
  p.row_bits = few ? 4 : 7;
  p.stop = 1;
  const long long keys = (((long long)pg.M << pg.s_bits) + KEYS - 1) / KEYS;  // tiles a sequence may have
  const long long steps = keys * (((long long)pr.N * pr.GQ >> p.row_bits) + pr.B) * pr.H_kv;
  p.blocks = (int)std::min<long long>(MAX_SMS, std::max(1ll, steps));
  p.inverse = ~0ull / p.blocks + 1;
  p.part_o = static_cast<float*>(ws);
  p.split = reinterpret_cast<PagedSplit*>(static_cast<uint8_t*>(ws) + up256((size_t)2 * MAX_SMS * KEYS * 4));
  cudaError_t e;
  if (pr.d == 128)
    e = few ? launch_t<128, 16>(p, s) : launch_t<128, 128>(p, s);
  else
    e = few ? launch_t<64, 16>(p, s) : launch_t<64, 128>(p, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_weights_join_kernel, dim3(p.blocks), dim3(KEYS), 0, s, p);
}

}  // namespace pisa
