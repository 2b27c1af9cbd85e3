// Attention over shared prefixes on the tensor cores of the 5th generation: 256 query rows of one
// (group, KV head) a tile, 128 keys a step.
//
//   S = Q K^T (fp32 in tensor memory), P = 2^(S scale log2 e - m) as bf16 back into tensor memory
//   over S, O += P V in tensor memory, l = sum of the unrounded P
//
// m is a row's reference, not its running maximum: it is raised, and O multiplied by 2^(old - new),
// only when the maximum has grown by more than 2^8 past it (P stays below 2^8, far from the end of
// bf16's and of fp32's range, and the final division by l is exact whatever m is).  With the usual logits that
// happens in a job's first steps alone, so O is left where the MMA accumulates it.  P is rounded
// to bf16 (half a step, 2^-8 of each weight, the size of the output's own rounding).
//
// The 8-bit cache: four warps widen the codes to bf16 (exact) into the swizzled tiles that the MMA
// reads; the key's scale multiplies the logit and the value's scale the weight, both in fp32.
//
// Roles: two softmax warpgroups, one for each 128 rows of the tile (a row a thread), so that one
// tile's softmax runs while the tensor pipe works for the other; a producer warp (TMA); a warp that
// issues the MMAs; with the 8-bit cache the widening warpgroup.  TMEM: S of half i at 128 i (its first 64
// columns hold P afterwards), O of half i at 256 + 128 i.  MMAs of one thread run in order, so S(j + 1)
// of a half is issued right behind its O += P V of step j, which reads P from the same columns.
// Every wait is bounded.
#include <algorithm>

#include "cache_attn.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "prefix_plan.cuh"

namespace pisa {
namespace {

constexpr int ROWS = TC_ROWS, HALF = 128, KT = PREFIX_KT;
constexpr float MAX_GROWTH = 8.f;  // log2 units the maximum may pass a row's reference

template <int D, int BITS>
struct Cfg {
  static constexpr int THREADS = BITS == 8 ? 512 : 384;
  static constexpr int PRODUCER = BITS == 8 ? 12 : 8, ISSUER = PRODUCER + 1;  // warps
  static constexpr uint32_t QH_BYTES = HALF * D * 2;    // 128 query rows
  static constexpr uint32_t TILE = KT * D * 2;          // a K or V tile in bf16
  static constexpr uint32_t RAW = KT * D;               // in codes
  static constexpr int SLOTS = BITS == 8 ? 3 : 5;       // bf16 tiles: K, V, K, ...
  static constexpr int RSLOTS = BITS == 8 ? 3 : 0;       // tiles of codes
  static constexpr size_t SMEM = 1024 + 2 * QH_BYTES + SLOTS * TILE + RSLOTS * RAW;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t full[5], empty[5];          // bf16 tiles
  uint64_t raw_full[4], raw_empty[4];  // tiles of codes
  uint64_t sc_full[4];                 // a step's scales
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drain;
};

template <int R>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// One query row's finished part: to the output (the whole job) or to the block's partial slot.
template <int D>
__device__ __forceinline__ void finish_row(const PrefixParams& p, const PrefixWalk& w, int local, uint32_t o_tmem,
                                           float m, float l, bool live) {
  size_t orow = 0;
  float fa = 0.f, fo = 0.f, lse = 0.f;
  if (live && w.slot < 0) {
    const int mrow = w.tile * ROWS + local, tok = mrow / p.GQ;
    orow = (size_t)(w.g.first + tok) * p.H_q + (size_t)w.head * p.GQ + (mrow - tok * p.GQ);
    join_own(m, l, p.lse_own ? p.lse_own[orow] : NEG_INF, fa, fo, lse);
    if (p.lse) p.lse[orow] = lse;
  }
  float* dst = p.part_o + ((size_t)(w.slot < 0 ? 0 : w.slot) * ROWS + local) * D;
  if (live && w.slot >= 0) p.part_ml[(size_t)w.slot * ROWS + local] = make_float2(m, l);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t r[32];
    tmem_ld32(o_tmem + c, r);
    tmem_wait_ld();
    if (!live) continue;
    if (w.slot < 0) {
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        uint4 own = make_uint4(0, 0, 0, 0);
        if (p.o_own && fo != 0.f) own = *reinterpret_cast<const uint4*>(p.o_own + orow * D + c + j);
        const uint32_t ow[4] = {own.x, own.y, own.z, own.w};
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a = fa == 0.f ? 0.f : __uint_as_float(r[j + 2 * e]) * fa;
          float b = fa == 0.f ? 0.f : __uint_as_float(r[j + 2 * e + 1]) * fa;
          if (p.o_own && fo != 0.f) {
            a += bf16_lo(ow[e]) * fo;
            b += bf16_hi(ow[e]) * fo;
          }
          v[e] = pack_bf16x2(a, b);
        }
        *reinterpret_cast<uint4*>(p.o + orow * D + c + j) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<uint4*>(dst + c + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
    }
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(Cfg<D, BITS>::THREADS, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapV, PrefixParams p) {
  pdl_trigger();
  using C = Cfg<D, BITS>;
  constexpr int DH = D / 64;  // 64-column halves of a row
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sT = sQ + 2 * C::QH_BYTES;
  uint8_t* sR = sT + C::SLOTS * C::TILE;
  __shared__ Bars bar;
  __shared__ __align__(16) float sc[BITS == 8 ? 4 : 1][2][KT];  // scales of the step: keys', values'
  __shared__ uint32_t tmem_base_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* err = p.err;

  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&bar.full[i], BITS == 8 ? 4 : 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], 4);
      mbar_init(&bar.sc_full[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_done[i], 1);
    }
    mbar_init(&bar.drain, 1);
    mbar_fence_init();
  }
  if (warp == C::ISSUER) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;

  PrefixWalk w;
  w.init(p, blockIdx.x, blockIdx.x == 0 && warp == 0);

  if (warp < 8) {
    // ------------------------------ softmax ------------------------------
    if constexpr (BITS == 8) set_regs_up<184>();
    const int half = warp >> 2;
    const int local = half * HALF + (warp & 3) * 32 + lane;  // row in the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lanes + 128 * half, o_tmem = tmem + lanes + 256 + 128 * half;
    uint32_t it = 0, step0 = 0;  // this half's steps; the block's steps
    bool failed = false;
    while (!failed && w.next(p, blockIdx.x)) {
      const int rows = min(ROWS, w.g.n * p.GQ - w.tile * ROWS);
      const int nk = w.k1 - w.k0;
      if (half * HALF >= rows) {  // the tile has no second half
        step0 += nk;
        continue;
      }
      const bool live = local < rows, any = half * HALF + (warp & 3) * 32 < rows;
      float m = NEG_INF, top = NEG_INF;  // reference and maximum, log2 units
      unsigned long long l2 = pack_f32x2(0.f, 0.f);
      for (int j = 0; j < nk; ++j, ++it) {
        const int valid = min(KT, w.g.len - (w.k0 + j) * KT);
        const uint32_t gs = step0 + j;
        if (!mbar_wait_warp(&bar.s_full[half], it & 1, err)) {
          failed = true;
          break;
        }
        if constexpr (BITS == 8) {  // done already (S was formed from the same tile): makes the scales visible
          if (!mbar_wait_warp(&bar.sc_full[gs & 3], (gs >> 2) & 1, err)) {
            failed = true;
            break;
          }
        }
        tc_fence_after();
        if (any) {
          uint32_t s[KT];
#pragma unroll
          for (int c = 0; c < KT; c += 32) tmem_ld32(s_tmem + c, *reinterpret_cast<uint32_t(*)[32]>(s + c));
          tmem_wait_ld();
          if constexpr (BITS == 8) {
            const float4* ks = reinterpret_cast<const float4*>(sc[gs & 3][0]);
#pragma unroll
            for (int c = 0; c < KT; c += 4) {
              const float4 f = ks[c / 4];
              float x[4];
              unpack_f32x2(mul_f32x2(pack_u32x2(s[c], s[c + 1]), pack_f32x2(f.x, f.y)), x[0], x[1]);
              unpack_f32x2(mul_f32x2(pack_u32x2(s[c + 2], s[c + 3]), pack_f32x2(f.z, f.w)), x[2], x[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[c + e] = __float_as_uint(x[e]);
            }
          }
          if (valid < KT) {
#pragma unroll
            for (int c = 0; c < KT; ++c)
              if (c >= valid) s[c] = __float_as_uint(NEG_INF);
          }
          float mx[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
          for (int c = 0; c < KT; c += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(s[c + e])), __uint_as_float(s[c + 4 + e]));
          }
          top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.sl2);
          if (__any_sync(0xffffffffu, top > m + MAX_GROWTH)) {
            // the reference follows the maximum; O (of the steps before) with it
            const float f = top == NEG_INF ? 1.f : fast_exp2(m - top);
            m = top;
            float a, b;
            unpack_f32x2(l2, a, b);
            l2 = pack_f32x2(a * f, b * f);
            if (j > 0) {
              if (!mbar_wait_warp(&bar.o_done[half], (it - 1) & 1, err)) {
                failed = true;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t r[16];
                tmem_ld16(o_tmem + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                tmem_st16(o_tmem + c, r);
              }
              tmem_wait_st();
            }
          }
          const float ref = m == NEG_INF ? 0.f : -m;
          const unsigned long long sl2 = pack_f32x2(p.sl2, p.sl2), ref2 = pack_f32x2(ref, ref);
#pragma unroll
          for (int c = 0; c < KT; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x, y;
              unpack_f32x2(fma_f32x2(pack_u32x2(s[c + e], s[c + e + 1]), sl2, ref2), x, y);
              x = fast_exp2(x);
              y = fast_exp2(y);
              unsigned long long xy = pack_f32x2(x, y);
              l2 = add_f32x2(l2, xy);
              if constexpr (BITS == 8) {
                const float2 f = *reinterpret_cast<const float2*>(&sc[gs & 3][1][c + e]);
                unpack_f32x2(mul_f32x2(xy, pack_f32x2(f.x, f.y)), x, y);
              }
              pk[e / 2] = pack_bf16x2(x, y);
            }
            tmem_st16(s_tmem + c / 2, pk);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[half]);
      }
      step0 += nk;
      if (failed) break;
      if (!mbar_wait_warp(&bar.o_done[half], (it - 1) & 1, err)) {
        failed = true;
        break;
      }
      tc_fence_after();
      float a, b;
      unpack_f32x2(l2, a, b);
      if (any) finish_row<D>(p, w, local, o_tmem, m, a + b, live);
      tc_fence_before();
    }
  } else if (warp == C::PRODUCER) {
    // ------------------------------ producer ------------------------------
    if constexpr (BITS == 8) set_regs_down<64>();
    uint32_t nt = 0, seg = 0;  // tiles (K, V, K, ...) and segments so far
    bool failed = false;
    while (!failed && w.next(p, blockIdx.x)) {
      const int rows = min(ROWS, w.g.n * p.GQ - w.tile * ROWS), halves = rows > HALF ? 2 : 1;
      if (!mbar_wait_warp(&bar.q_empty, (seg & 1) ^ 1, err)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar.q_full, halves * C::QH_BYTES);
        for (int h = 0; h < halves; ++h)
          for (int c = 0; c < DH; ++c)
            tma_load_4d(sQ + h * C::QH_BYTES + c * (HALF * 128), &mapQ, &bar.q_full, 64 * c, 0, w.head,
                        w.g.first + (w.tile * ROWS + h * HALF) / p.GQ);
      }
      ++seg;
      const int ph = w.p * p.H_kv + w.head;
      for (int j = 0; j < w.k1 - w.k0 && !failed; ++j) {
        const int key0 = (w.k0 + j) * KT;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++nt) {
          if constexpr (BITS == 8) {
            const int st = nt % C::RSLOTS;
            if (!mbar_wait_warp(&bar.raw_empty[st], ((nt / C::RSLOTS) & 1) ^ 1, err)) {
              failed = true;
              break;
            }
            if (lane == 0) {
              // rows past the cache's end are not copied; what the slot holds there is finite, and masked
              const uint32_t bytes = (uint32_t)min(KT, p.N_cap - key0) * D;
              mbar_arrive_expect_tx(&bar.raw_full[st], bytes);
              bulk_load(sR + st * C::RAW, (kv ? p.V : p.K) + ((size_t)ph * p.N_cap + key0) * D, bytes, &bar.raw_full[st]);
            }
          } else {
            const int st = nt % C::SLOTS;
            if (!mbar_wait_warp(&bar.empty[st], ((nt / C::SLOTS) & 1) ^ 1, err)) {
              failed = true;
              break;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(&bar.full[st], C::TILE);
              for (int c = 0; c < DH; ++c)
                tma_load_3d(sT + st * C::TILE + c * (KT * 128), kv ? &mapV : &mapK, &bar.full[st], 64 * c, key0, ph);
            }
          }
        }
      }
    }
    // copies still in flight land before shared memory goes away (bounded; at once unless a wait failed)
    if (lane == 0) {
      if (seg > 0) mbar_wait(&bar.q_full, (seg - 1) & 1, err, 100000000ull);
      constexpr uint32_t N = BITS == 8 ? C::RSLOTS : C::SLOTS;
      for (uint32_t u = nt > N ? nt - N : 0; u < nt; ++u)
        mbar_wait(BITS == 8 ? &bar.raw_full[u % N] : &bar.full[u % N], (u / N) & 1, err, 100000000ull);
    }
    __syncwarp();
  } else if (warp == C::ISSUER) {
    // ------------------------------ MMAs ------------------------------
    if constexpr (BITS == 8) set_regs_down<64>();
    constexpr uint32_t id_qk = idesc_bf16_f32(HALF, KT);
    constexpr uint32_t id_pv = idesc_bf16_f32(HALF, D) | (1u << 16);  // V: d contiguous, N-major
    uint32_t gs = 0, seg = 0, it[2] = {0, 0};
    bool failed = false;
    auto tile_full = [&](uint32_t n) { return mbar_wait_warp(&bar.full[n % C::SLOTS], (n / C::SLOTS) & 1, err); };
    auto qk = [&](int h, uint32_t n) {
      const uint32_t a = smem_u32(sQ) + h * C::QH_BYTES, b = smem_u32(sT) + (n % C::SLOTS) * C::TILE;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        umma_bf16(tmem + 128 * h, smem_desc_sw128(a + (s >> 2) * (HALF * 128) + (s & 3) * 32, 16, 1024),
                  smem_desc_sw128(b + (s >> 2) * (KT * 128) + (s & 3) * 32, 16, 1024), id_qk, s > 0 ? 1u : 0u);
      umma_commit(&bar.s_full[h]);
    };
    while (!failed && w.next(p, blockIdx.x)) {
      const int rows = min(ROWS, w.g.n * p.GQ - w.tile * ROWS), halves = rows > HALF ? 2 : 1;
      const int nk = w.k1 - w.k0;
      if (!mbar_wait_warp(&bar.q_full, seg & 1, err) || !tile_full(2 * gs)) break;
      ++seg;
      tc_fence_after();
      if (lane == 0) {
        for (int h = 0; h < halves; ++h) qk(h, 2 * gs);
        umma_commit(&bar.empty[(2 * gs) % C::SLOTS]);
        if (nk == 1) umma_commit(&bar.q_empty);
      }
      __syncwarp();
      for (int j = 0; j < nk && !failed; ++j, ++gs) {
        const uint32_t nv = 2 * gs + 1, nn = 2 * gs + 2;
        if (!tile_full(nv)) {
          failed = true;
          break;
        }
        if constexpr (BITS == 16) {
          // values past the prefix's end are multiplied by weights of 0: they have to be finite
          const int valid = max(0, min(KT, w.g.len - (w.k0 + j) * KT));
          if (valid < KT) {
            uint8_t* t = sT + (nv % C::SLOTS) * C::TILE;
            for (int c = 0; c < DH; ++c)
              for (int i = valid * 8 + lane; i < KT * 8; i += 32)
                *reinterpret_cast<uint4*>(t + c * (KT * 128) + i * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
          }
        }
        for (int h = 0; h < halves; ++h) {
          if (!mbar_wait_warp(&bar.p_full[h], it[h] & 1, err)) {
            failed = true;
            break;
          }
          ++it[h];
          tc_fence_after();
          if (lane == 0) {
            const uint32_t b = smem_u32(sT) + (nv % C::SLOTS) * C::TILE;
#pragma unroll
            for (int s = 0; s < KT / 16; ++s)
              umma_bf16_ts(tmem + 256 + 128 * h, tmem + 128 * h + 8 * s, smem_desc_sw128(b + s * 2048, KT * 128, 1024),
                           id_pv, (j > 0 || s > 0) ? 1u : 0u);
            umma_commit(&bar.o_done[h]);
            if (h == halves - 1) umma_commit(&bar.empty[nv % C::SLOTS]);
          }
          __syncwarp();
          if (j + 1 < nk) {
            if (h == 0 && !tile_full(nn)) {
              failed = true;
              break;
            }
            tc_fence_after();
            if (lane == 0) {
              qk(h, nn);
              if (h == halves - 1) {
                umma_commit(&bar.empty[nn % C::SLOTS]);
                if (j + 2 == nk) umma_commit(&bar.q_empty);
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) {  // every MMA issued has completed before the tensor memory is released (bounded)
      umma_commit(&bar.drain);
      mbar_wait(&bar.drain, 0, err);
    }
    __syncwarp();
  } else if (BITS == 8 && warp < 12) {
    // ------------------------------ codes to bf16 ------------------------------
    if constexpr (BITS == 8) {
      set_regs_down<80>();
      const int t = threadIdx.x - 256;
      constexpr int CH = D / 16;  // 16-code chunks a row
      uint32_t nt = 0, gs = 0;
      bool failed = false;
      while (!failed && w.next(p, blockIdx.x)) {
        const size_t row0 = ((size_t)w.p * p.H_kv + w.head) * p.N_cap;
        for (int j = 0; j < w.k1 - w.k0 && !failed; ++j, ++gs) {
          const int key = (w.k0 + j) * KT + t;
          const float ks = key < w.g.len ? __ldg(p.ks + row0 + key) : 0.f;
          const float vs = key < w.g.len ? __ldg(p.vs + row0 + key) : 0.f;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++nt) {
            const int rs = nt % C::RSLOTS, cs = nt % C::SLOTS;
            if (!mbar_wait_warp(&bar.raw_full[rs], (nt / C::RSLOTS) & 1, err) ||
                !mbar_wait_warp(&bar.empty[cs], ((nt / C::SLOTS) & 1) ^ 1, err)) {
              failed = true;
              break;
            }
            if (kv == 0) {
              // the slots of the scales and of the tiles turn together: the tile slot that was just
              // found free was last used after the softmax of the step four before had read these
              sc[gs & 3][0][t] = ks;
              sc[gs & 3][1][t] = vs;
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.sc_full[gs & 3]);
            }
            const uint8_t* src = sR + rs * C::RAW;
            uint8_t* dst = sT + cs * C::TILE;
#pragma unroll 4
            for (int i = t; i < KT * CH; i += 128) {
              const int row = i / CH, c = i % CH;
              const uint4 x = *reinterpret_cast<const uint4*>(src + i * 16);
              const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[2 * e] = widen_codes(__byte_perm(wd[e], 0, 0x4140));
                o[2 * e + 1] = widen_codes(__byte_perm(wd[e], 0, 0x4342));
              }
              uint8_t* r = dst + (c >> 2) * (KT * 128) + row * 128;
              const int ch = 2 * (c & 3);
              *reinterpret_cast<uint4*>(r + ((ch ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(r + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bar.full[cs]);
              mbar_arrive(&bar.raw_empty[rs]);
            }
          }
        }
      }
    }
  } else {
    if constexpr (BITS == 8) set_regs_down<64>();
  }
  __syncthreads();
  if (warp == C::ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int BITS>
cudaError_t launch_t(const PrefixParams& p, cudaStream_t s) {
  using C = Cfg<D, BITS>;
  CUtensorMap mapQ, mapK, mapV;
  {
    // 128 rows of one KV head's group: (64 columns, G_Q heads, 1 KV head, 128 / G_Q tokens)
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.GQ, (uint64_t)p.H_kv, (uint64_t)p.R};
    const uint64_t strides[3] = {(uint64_t)D * 2, (uint64_t)p.GQ * D * 2, (uint64_t)p.H_q * D * 2};
    const uint32_t box[4] = {64, (uint32_t)p.GQ, 1, (uint32_t)(HALF / p.GQ)};
    if (!encode_tensor_map(&mapQ, p.q, 4, dims, strides, box)) return cudaErrorInvalidValue;
  }
  mapK = mapV = mapQ;  // not used by the 8-bit cache, whose tiles are plain bulk copies
  if (BITS == 16) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.N_cap, (uint64_t)p.P * p.H_kv};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)p.N_cap * D * 2};
    const uint32_t box[3] = {64, (uint32_t)KT, 1};
    if (!encode_tensor_map(&mapK, p.K, 3, dims, strides, box)) return cudaErrorInvalidValue;
    if (!encode_tensor_map(&mapV, p.V, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  auto kern = prefix_tc_kernel<D, BITS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<p.blocks, C::THREADS, C::SMEM, s>>>(mapQ, mapK, mapV, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixParams& p, int d, cudaStream_t s) {
  if (d == 128) return p.ks ? launch_t<128, 8>(p, s) : launch_t<128, 16>(p, s);
  return p.ks ? launch_t<64, 8>(p, s) : launch_t<64, 16>(p, s);
}

}  // namespace pisa
