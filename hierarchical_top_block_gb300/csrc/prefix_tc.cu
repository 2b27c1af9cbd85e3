// Attention over shared prefixes on the tensor cores of the 5th generation: up to 256 query rows of
// one (group, KV head) a tile, 128 keys a step, one block a SM.
//
//   S = Q K^T (fp32 in tensor memory), P = 2^(S scale log2 e - m) as bf16 back into tensor memory
//   over S, O += P V in tensor memory, l = sum of the unrounded P
//
// m is a row's reference, not its running maximum: it is raised, and O multiplied by 2^(old - new),
// only when the maximum has grown by more than 2^8 past it (P stays below 2^8, far from the end of
// bf16's and of fp32's range, and the division by l at the end is exact whatever m is).  With the
// usual logits that happens in a job's first steps alone, so O is left where the MMA accumulates it.
// P is rounded to bf16 (half a step, 2^-8 of each weight, the size of the output's own rounding).
//
// Two streams keep the tensor pipe busy while the softmax of the other one runs, a warpgroup for
// each.  With more than 128 rows a stream is a half of the rows, and both use the same tiles; with
// fewer, both streams have all rows, one the even steps and one the odd ones, each with its own
// m, l and O, which are joined when a job's segment ends.
//
// The 8-bit cache: four warps widen the codes to bf16 (exact) into the swizzled tiles that the MMA
// reads; the key's scale multiplies the logit and the value's scale the weight, both in fp32.
//
// Roles: two softmax warpgroups (a row a thread); a producer warp (TMA); a warp that issues the MMAs;
// with the 8-bit cache the widening warpgroup.  TMEM: S of stream i at 128 i (its first 64 columns
// hold P afterwards), O of stream i at 256 + 128 i.  The MMAs of one thread run in order, so a stream's
// next S is issued right behind its O += P V, which reads P from the same columns.  Every wait is
// bounded.
#include <algorithm>

#include "kernels.cuh"
#include "pdl.cuh"
#include "prefix_plan.cuh"

namespace pisa {
namespace {

constexpr int ROWS = TC_ROWS, KT = PREFIX_KT;
constexpr float MAX_GROWTH = 8.f;  // log2 units the maximum may pass a row's reference

template <int D, int BITS>
struct Cfg {
  static constexpr int THREADS = BITS == 8 ? 512 : 384;
  static constexpr int PRODUCER = BITS == 8 ? 12 : 8, ISSUER = PRODUCER + 1, WORKERS = ISSUER + 1;  // warps
  static constexpr uint32_t QT_BYTES = 128 * D * 2;     // 128 query rows
  static constexpr uint32_t TILE = KT * D * 2;          // a K or V tile in bf16
  static constexpr uint32_t RAW = KT * D;               // in codes
  static constexpr int SLOTS = BITS == 8 ? 3 : 5;
  static constexpr int RSLOTS = 3;
  static constexpr size_t TILES = 2 * QT_BYTES + SLOTS * TILE + (BITS == 8 ? RSLOTS * RAW : 0);
};

constexpr int SC_SLOTS = 4;

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t full[5], empty[5];          // bf16 tiles
  uint64_t raw_full[3], raw_empty[3];  // tiles of codes
  uint64_t sc_full[SC_SLOTS];          // a step's scales
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t x_full, x_done;             // the streams' meeting at the end of a segment
  uint64_t drain;
};

// What follows the tiles in shared memory (all of it dynamic: with five bf16 tiles there is room for
// 3 KB beside them, and none for an alignment gap).
template <int BITS>
struct Shared {
  Bars bar;
  float2 ml[2][128];                               // the streams' maxima and sums, when they meet
  PrefixWalk walks[BITS == 8 ? 14 : 10];           // each working warp's walk over the segments: the
                                                   // softmax needs the registers
  uint32_t tmem;
  __align__(16) float sc[BITS == 8 ? SC_SLOTS : 1][2][BITS == 8 ? KT : 4];  // scales of a step: keys', values'
};

// Two int8 codes in bytes 0 and 2 of y (bytes 1 and 3: anything) -> bf16x2.  A code is m - 128 s
// (s its top bit, m the seven below): (128 + m) - 128 (1 + s), both exact bf16 numbers whose
// bits are 0x4300 | m and 0x4300 | (code & 0x80).
__device__ __forceinline__ uint32_t widen_codes(uint32_t y) {
  const uint32_t a = (y & 0x007f007fu) | 0x43004300u, c = (y & 0x00800080u) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(c));
  return r;
}

template <int R>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// A segment's streams: by rows (`lag` 1: both use every tile) or by steps (`lag` 2: stream = step
// mod 2).  The tiles' order is that of their use: K 0 .. lag - 1, then V j and K j + lag.
struct Segment {
  int rows, nk, lag;
  __device__ __forceinline__ Segment(const PrefixParams& p, const PrefixWalk& w) {
    rows = min(ROWS, w.g.n * p.GQ - w.tile * ROWS);
    nk = w.k1 - w.k0;
    lag = rows > ROWS / 2 ? 1 : 2;
  }
  __device__ __forceinline__ int tiles() const { return 2 * nk; }
  // Tile i of the order: returns its step, and whether it is a V.
  __device__ __forceinline__ int tile(int i, bool& is_v) const {
    const int head = min(lag, nk), both = 2 * (nk - head);
    if (i < head) {
      is_v = false;
      return i;
    }
    i -= head;
    if (i < both) {
      is_v = (i & 1) == 0;
      return is_v ? i >> 1 : head + (i >> 1);
    }
    is_v = true;
    return nk - head + (i - both);
  }
};

// Where a finished query row goes: the output (the whole job was this segment) or a part's slot.
struct RowOut {
  bool live;
  int slot;
  size_t orow;
  float own;         // the row's own log-sum-exp
  float fa, fo;
  float* part;
};
template <int D>
__device__ __forceinline__ RowOut row_out(const PrefixParams& p, const PrefixWalk& w, int local, bool live) {
  RowOut r;
  r.live = live;
  r.slot = w.slot;
  const int mrow = w.tile * ROWS + local, tok = mrow / p.GQ;
  r.orow = (size_t)(w.g.first + tok) * p.H_q + (size_t)w.head * p.GQ + (mrow - tok * p.GQ);
  r.own = live && w.slot < 0 && p.lse_own ? p.lse_own[r.orow] : NEG_INF;
  r.part = p.part_o + ((size_t)(w.slot < 0 ? 0 : w.slot) * ROWS + local) * D;
  r.fa = r.fo = 0.f;
  return r;
}
// The row's factors, and (stats) its log-sum-exp or maximum and sum.
__device__ __forceinline__ void put_stats(const PrefixParams& p, RowOut& r, int local, float m, float l, bool stats) {
  if (!r.live) return;
  if (r.slot < 0) {
    float lse;
    join_own(m, l, r.own, r.fa, r.fo, lse);
    if (stats && p.lse) p.lse[r.orow] = lse;
  } else if (stats) {
    p.part_ml[(size_t)r.slot * ROWS + local] = make_float2(m, l);
  }
}
// 32 columns from c on of the row's output sums, relative to its maximum.
template <int D>
__device__ __forceinline__ void put_columns(const PrefixParams& p, const RowOut& r, int c, const uint32_t (&x)[32]) {
  if (!r.live) return;
  if (r.slot < 0) {
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      uint4 own = make_uint4(0, 0, 0, 0);
      const bool with = p.o_own && r.fo != 0.f;
      if (with) own = *reinterpret_cast<const uint4*>(p.o_own + r.orow * D + c + j);
      const uint32_t ow[4] = {own.x, own.y, own.z, own.w};
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a = r.fa == 0.f ? 0.f : __uint_as_float(x[j + 2 * e]) * r.fa;
        float b = r.fa == 0.f ? 0.f : __uint_as_float(x[j + 2 * e + 1]) * r.fa;
        if (with) {
          a += bf16_lo(ow[e]) * r.fo;
          b += bf16_hi(ow[e]) * r.fo;
        }
        v[e] = pack_bf16x2(a, b);
      }
      *reinterpret_cast<uint4*>(p.o + r.orow * D + c + j) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      *reinterpret_cast<uint4*>(r.part + c + j) = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(Cfg<D, BITS>::THREADS, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapV, PrefixParams p) {
  pdl_trigger();
  using C = Cfg<D, BITS>;
  constexpr int DH = D / 64;  // 64-column pieces of a Q or K row
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sT = sQ + 2 * C::QT_BYTES;
  uint8_t* sR = sT + C::SLOTS * C::TILE;
  Shared<BITS>& sh = *reinterpret_cast<Shared<BITS>*>(smem + C::TILES);
  Bars& bar = sh.bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x;
  uint32_t* err = p.err;

  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&bar.full[i], BITS == 8 ? 4 : 1);  // the widening warps; or the copy
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < C::RSLOTS; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], 4);
    }
    for (int i = 0; i < SC_SLOTS; ++i) mbar_init(&bar.sc_full[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_done[i], 1);
    }
    mbar_init(&bar.x_full, 8);
    mbar_init(&bar.x_done, 8);
    mbar_init(&bar.drain, 1);
    mbar_fence_init();
  }
  if (warp == C::ISSUER) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  const PrefixWalk& w = sh.walks[warp < C::WORKERS ? warp : 0];
  if (warp < C::WORKERS) {
    PrefixWalk first;
    first.init(p, block, block == 0 && warp == 0);
    if (lane == 0) sh.walks[warp] = first;
    __syncwarp();
  }
  auto next_segment = [&]() {
    PrefixWalk at = sh.walks[warp];
    __syncwarp();
    const bool more = at.next(p, block);
    if (lane == 0) sh.walks[warp] = at;
    __syncwarp();
    return more;
  };

  if (warp < 8) {
    // ------------------------------ softmax ------------------------------
    set_regs_up<BITS == 8 ? 192 : 216>();
    const int h = warp >> 2;                                 // stream
    const int trow = (warp & 3) * 32 + lane;                 // TMEM lane
    const int q = lane & 3;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lanes + 128 * h, o_tmem = tmem + lanes + 256 + 128 * h;
    uint32_t it[2] = {0, 0}, step0 = 0, meets = 0;           // the streams' steps; all steps
    bool failed = false;
    while (!failed && next_segment()) {
      const Segment sg(p, w);
      const int local = (sg.lag == 1 ? 128 * h : 0) + trow;  // row in the tile
      const bool live = local < sg.rows, any = local - lane < sg.rows;
      // rows r, r + 8, r + 16, r + 24 of the warp's 32: a lane holds a quarter of the columns of each, so a key's
      // scales are wanted by eight lanes only and fit in registers
      float m[4], top[4];              // reference and maximum, log2 units
      unsigned long long l2[4];        // a lane's share of the sum, even and odd columns
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = top[i] = NEG_INF;
        l2[i] = pack_f32x2(0.f, 0.f);
      }
      uint32_t n = it[h];
      for (int j = sg.lag == 1 ? 0 : h; j < sg.nk; j += sg.lag, ++n) {
        const int valid = min(KT, w.g.len - (w.k0 + j) * KT);
        const uint32_t gs = step0 + j;
        float2 kf[BITS == 8 ? 16 : 1];
        if constexpr (BITS == 8) {
          if (!mbar_wait_warp(&bar.sc_full[gs % SC_SLOTS], (gs / SC_SLOTS) & 1, err)) {
            failed = true;
            break;
          }
#pragma unroll
          for (int g = 0; g < 16; ++g) kf[g] = *reinterpret_cast<const float2*>(&sh.sc[gs % SC_SLOTS][0][8 * g + 2 * q]);
        }
        if (!mbar_wait_warp(&bar.s_full[h], n & 1, err)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (any) {
          uint32_t s[2][64];  // [rows below / from 16][four a group of 8 columns]
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) tmem_ld_16x64(s_tmem + ((uint32_t)(16 * i) << 16) + 64 * c, &s[i][32 * c]);
          tmem_wait_ld();
          if constexpr (BITS == 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int g = 0; g < 16; ++g)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  float x, y;
                  unpack_f32x2(mul_f32x2(pack_u32x2(s[i][4 * g + e], s[i][4 * g + e + 1]), pack_f32x2(kf[g].x, kf[g].y)), x, y);
                  s[i][4 * g + e] = __float_as_uint(x);
                  s[i][4 * g + e + 1] = __float_as_uint(y);
                }
          }
          if (valid < KT) {
#pragma unroll
            for (int g = 0; g < 16; ++g)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (8 * g + 2 * q + c >= valid)
#pragma unroll
                  for (int i = 0; i < 2; ++i) s[i][4 * g + c] = s[i][4 * g + 2 + c] = __float_as_uint(NEG_INF);
          }
          bool moved = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* x = &s[i >> 1][2 * (i & 1)];
            float a = NEG_INF, b = NEG_INF;
#pragma unroll
            for (int g = 0; g < 16; g += 2) {
              a = fmaxf(fmaxf(a, __uint_as_float(x[4 * g])), __uint_as_float(x[4 * g + 1]));
              b = fmaxf(fmaxf(b, __uint_as_float(x[4 * g + 4])), __uint_as_float(x[4 * g + 5]));
            }
            a = fmaxf(a, b);
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            top[i] = fmaxf(top[i], a * p.sl2);
            moved = moved || top[i] > m[i] + MAX_GROWTH;
          }
          if (__any_sync(0xffffffffu, moved)) {
            // the references follow the maxima; O (of the steps before) with them
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[i] = top[i] == NEG_INF ? 1.f : fast_exp2(m[i] - top[i]);
              m[i] = top[i];
              l2[i] = mul_f32x2(l2[i], pack_f32x2(f[i], f[i]));
            }
            if (n != it[h]) {
              if (!mbar_wait_warp(&bar.o_done[h], (n - 1) & 1, err)) {
                failed = true;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 2 * D; c += 16) {  // columns c mod D of rows below 16, then from 16
                const bool up = c >= D;
                const uint32_t at = o_tmem + ((up ? 16u : 0u) << 16) + (up ? c - D : c);
                const float fa = up ? f[2] : f[0], fb = up ? f[3] : f[1];
                uint32_t r[8];
                tmem_ld_16x16(at, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * ((e & 2) ? fb : fa));
                tmem_st_16x16(at, r);
              }
            }
          }
          const unsigned long long sl2 = pack_f32x2(p.sl2, p.sl2);
          unsigned long long ref[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = m[i] == NEG_INF ? 0.f : -m[i];
            ref[i] = pack_f32x2(x, x);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)  // 64 keys
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t pk[16];
#pragma unroll
              for (int g = 0; g < 8; ++g) {
                float2 vf = make_float2(1.f, 1.f);
                if constexpr (BITS == 8) vf = *reinterpret_cast<const float2*>(&sh.sc[gs % SC_SLOTS][1][64 * c + 8 * g + 2 * q]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // row r + 16 i + 8 e
                  const uint32_t* x = &s[i][32 * c + 4 * g + 2 * e];
                  float a, b;
                  unpack_f32x2(fma_f32x2(pack_u32x2(x[0], x[1]), sl2, ref[2 * i + e]), a, b);
                  a = fast_exp2(a);
                  b = fast_exp2(b);
                  const unsigned long long ab = pack_f32x2(a, b);
                  l2[2 * i + e] = add_f32x2(l2[2 * i + e], ab);
                  if constexpr (BITS == 8) unpack_f32x2(mul_f32x2(ab, pack_f32x2(vf.x, vf.y)), a, b);
                  pk[2 * g + e] = pack_bf16x2(a, b);
                }
              }
              tmem_st_16x32(s_tmem + ((uint32_t)(16 * i) << 16) + 32 * c, pk);
            }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[h]);
      }
      // the streams' steps of this segment
      const uint32_t n0 = sg.lag == 1 ? sg.nk : (sg.nk + 1) / 2, n1 = sg.lag == 1 ? sg.nk : sg.nk / 2;
      it[0] += n0;
      it[1] += n1;
      step0 += sg.nk;
      if (failed) break;
      // from here on a row a thread: each row's maximum and sum go through shared memory
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack_f32x2(l2[i], a, b);
        a += b;
        a += __shfl_xor_sync(0xffffffffu, a, 1);
        a += __shfl_xor_sync(0xffffffffu, a, 2);
        if (q == 0) sh.ml[h][(warp & 3) * 32 + 8 * i + (lane >> 2)] = make_float2(m[i], a);
      }
      __syncwarp();
      RowOut out = row_out<D>(p, w, local, live);
      if (sg.lag == 1) {
        if (!mbar_wait_warp(&bar.o_done[h], (it[h] - 1) & 1, err)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (any) {
          const float2 ml = sh.ml[h][trow];
          put_stats(p, out, local, ml.x, ml.y, true);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t r[32];
            tmem_ld32(o_tmem + c, r);
            tmem_wait_ld();
            put_columns<D>(p, out, c, r);
          }
        }
        tc_fence_before();
        __syncwarp();  // sh.ml has been read
      } else {
        // both streams have parts of every row: joined here, half of the columns by each warpgroup
        if (!mbar_wait_warp(&bar.o_done[0], (it[0] - 1) & 1, err) ||
            (n1 > 0 && !mbar_wait_warp(&bar.o_done[1], (it[1] - 1) & 1, err))) {
          failed = true;
          break;
        }
        if (lane == 0) mbar_arrive(&bar.x_full);
        if (!mbar_wait_warp(&bar.x_full, meets & 1, err)) {  // (the row's own log-sum-exp has been read by both)
          failed = true;
          break;
        }
        tc_fence_after();
        if (any) {
          const float2 a = sh.ml[0][trow], b = sh.ml[1][trow];
          const float m = fmaxf(a.x, b.x);
          const float f0 = a.x == NEG_INF ? 0.f : fast_exp2(a.x - m), f1 = b.x == NEG_INF ? 0.f : fast_exp2(b.x - m);
          const float l = (a.x == NEG_INF ? a.y : a.y * f0) + (b.x == NEG_INF ? b.y : b.y * f1);
          put_stats(p, out, local, m, l, h == 0);
          const uint32_t o0 = tmem + lanes + 256;
#pragma unroll 1
          for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 32) {
            uint32_t r[32], r1[32];
            tmem_ld32(o0 + c, r);
            if (n1 > 0) tmem_ld32(o0 + 128 + c, r1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float x = __uint_as_float(r[e]) * f0;
              if (n1 > 0) x = fmaf(__uint_as_float(r1[e]), f1, x);
              r[e] = __float_as_uint(x);
            }
            put_columns<D>(p, out, c, r);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.x_done);
        if (!mbar_wait_warp(&bar.x_done, meets & 1, err)) {  // both O have been read: the next segment may write them
          failed = true;
          break;
        }
        ++meets;
      }
    }
  } else if (warp == C::PRODUCER) {
    // ------------------------------ producer ------------------------------
    set_regs_down<BITS == 8 ? 56 : 72>();
    constexpr uint32_t N = BITS == 8 ? C::RSLOTS : C::SLOTS;
    uint32_t nt = 0, seg = 0;  // tiles and segments so far
    bool failed = false;
    while (!failed && next_segment()) {
      const Segment sg(p, w);
      if (!mbar_wait_warp(&bar.q_empty, (seg & 1) ^ 1, err)) break;
      if (lane == 0) {
        const int streams = sg.lag == 1 ? 2 : 1;
        mbar_arrive_expect_tx(&bar.q_full, streams * C::QT_BYTES);
        for (int h = 0; h < streams; ++h)
          for (int c = 0; c < DH; ++c)
            tma_load_4d(sQ + h * C::QT_BYTES + c * (128 * 128), &mapQ, &bar.q_full, 64 * c, 0, w.head,
                        w.g.first + (w.tile * ROWS + h * 128) / p.GQ);
      }
      ++seg;
      const int ph = w.p * p.H_kv + w.head;
      for (int i = 0; i < sg.tiles(); ++i, ++nt) {
        bool is_v;
        const int key0 = (w.k0 + sg.tile(i, is_v)) * KT;
        const int st = nt % N;
        uint64_t* full = BITS == 8 ? &bar.raw_full[st] : &bar.full[st];
        if (!mbar_wait_warp(BITS == 8 ? &bar.raw_empty[st] : &bar.empty[st], ((nt / N) & 1) ^ 1, err)) {
          failed = true;
          break;
        }
        if (lane == 0) {
          if constexpr (BITS == 8) {
            mbar_arrive_expect_tx(full, C::RAW);
            uint8_t* dst = sR + st * C::RAW;
            tma_load_3d(dst, is_v ? &mapV : &mapK, full, 0, key0, ph);
          } else {
            mbar_arrive_expect_tx(full, C::TILE);
            uint8_t* dst = sT + st * C::TILE;
            for (int c = 0; c < DH; ++c) tma_load_3d(dst + c * (KT * 128), is_v ? &mapV : &mapK, full, 64 * c, key0, ph);
          }
        }
      }
    }
    // copies still in flight land before shared memory goes away (bounded; at once unless a wait failed)
    if (lane == 0) {
      if (seg > 0) mbar_wait(&bar.q_full, (seg - 1) & 1, err, 100000000ull);
      for (uint32_t u = nt > N ? nt - N : 0; u < nt; ++u)
        mbar_wait(BITS == 8 ? &bar.raw_full[u % N] : &bar.full[u % N], (u / N) & 1, err, 100000000ull);
    }
    __syncwarp();
  } else if (warp == C::ISSUER) {
    // ------------------------------ MMAs ------------------------------
    set_regs_down<BITS == 8 ? 56 : 72>();
    constexpr uint32_t id_qk = idesc_bf16_f32(128, KT);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, D) | (1u << 16);  // V: d contiguous, N-major
    uint32_t nt = 0, seg = 0, it[2] = {0, 0};
    bool failed = false;
    // tile n is here (v_valid: a V tile's keys in use)
    auto tile_here = [&](uint32_t n, int v_valid) {
      if (!mbar_wait_warp(&bar.full[n % C::SLOTS], (n / C::SLOTS) & 1, err)) return false;
      if (BITS == 16 && v_valid < KT) {
        // values past the prefix's end are multiplied by weights of 0: they have to be finite
        uint8_t* t = sT + (n % C::SLOTS) * C::TILE;
        for (int c = 0; c < DH; ++c)
          for (int i = max(0, v_valid) * 8 + lane; i < KT * 8; i += 32)
            *reinterpret_cast<uint4*>(t + c * (KT * 128) + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
        __syncwarp();
      }
      return true;
    };
    // descriptors of the first tile and Q slot: the others differ in the address field alone (16-byte units)
    const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024), k_desc = smem_desc_sw128(smem_u32(sT), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(sT), KT * 128, 1024);
    auto qk = [&](int h, int qs, uint32_t n) {  // S of stream h = Q (slot qs) K^T
      const uint64_t a = q_desc + qs * (C::QT_BYTES >> 4), b = k_desc + (n % C::SLOTS) * (C::TILE >> 4);
      const uint32_t d = tmem + 128 * h;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        umma_bf16(d, a + (((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4), b + (((s >> 2) * (KT * 128) + (s & 3) * 32) >> 4),
                       id_qk, s > 0 ? 1u : 0u);
      umma_commit(&bar.s_full[h]);
    };
    auto pv = [&](int h, uint32_t n, bool first) {  // O of stream h (+)= P V
      const uint64_t b = v_desc + (n % C::SLOTS) * (C::TILE >> 4);
      const uint32_t d = tmem + 256 + 128 * h, a = tmem + 128 * h;
#pragma unroll
      for (int s = 0; s < KT / 16; ++s)
        umma_bf16_ts(d, a + 8 * s, b + ((s * 16 * 128) >> 4), id_pv, s > 0 ? 1u : first ? 0u : 1u);
      umma_commit(&bar.o_done[h]);
    };
    while (!failed && next_segment()) {
      const Segment sg(p, w);
      if (!mbar_wait_warp(&bar.q_full, seg & 1, err)) break;
      ++seg;
      const int head = min(sg.lag, sg.nk);
      for (int j = 0; j < head && !failed; ++j, ++nt) {
        if (!tile_here(nt, KT)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          if (sg.lag == 1) {
            qk(0, 0, nt);
            qk(1, 1, nt);
          } else {
            qk(j, 0, nt);
          }
          umma_commit(&bar.empty[nt % C::SLOTS]);
          if (j == sg.nk - 1) umma_commit(&bar.q_empty);
        }
        __syncwarp();
      }
      for (int j = 0; j < sg.nk && !failed; ++j) {
        const uint32_t nv = nt++;
        const bool more = j + sg.lag < sg.nk;
        const uint32_t nn = more ? nt++ : 0;
        if (!tile_here(nv, w.g.len - (w.k0 + j) * KT)) {
          failed = true;
          break;
        }
        const int h0 = sg.lag == 1 ? 0 : j & 1, h1 = sg.lag == 1 ? 1 : h0;
        for (int h = h0; h <= h1; ++h) {
          if (!mbar_wait_warp(&bar.p_full[h], it[h] & 1, err)) {
            failed = true;
            break;
          }
          ++it[h];
          tc_fence_after();
          if (elect_one()) {
            pv(h, nv, j < sg.lag);
            if (h == h1) umma_commit(&bar.empty[nv % C::SLOTS]);
          }
          __syncwarp();
          if (more) {
            if (h == h0 && !tile_here(nn, KT)) {
              failed = true;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              qk(h, sg.lag == 1 ? h : 0, nn);
              if (h == h1) {
                umma_commit(&bar.empty[nn % C::SLOTS]);
                if (j + sg.lag == sg.nk - 1) umma_commit(&bar.q_empty);
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (elect_one()) {  // every MMA issued has completed before the tensor memory is released (bounded)
      umma_commit(&bar.drain);
      mbar_wait(&bar.drain, 0, err);
    }
    __syncwarp();
  } else if (BITS == 8 && warp < 12) {
    // ------------------------------ codes to bf16 ------------------------------
    if constexpr (BITS == 8) {
      set_regs_down<72>();
      const int t = threadIdx.x - 256;
      uint32_t nt = 0, step0 = 0;
      bool failed = false;
      while (!failed && next_segment()) {
        const Segment sg(p, w);
        const size_t row0 = ((size_t)w.p * p.H_kv + w.head) * p.N_cap;
        for (int i = 0; i < sg.tiles(); ++i, ++nt) {
          bool is_v;
          const int j = sg.tile(i, is_v);
          const int key = (w.k0 + j) * KT + t;
          float ks = 0.f, vs = 0.f;
          if (!is_v && key < w.g.len) {
            ks = __ldg(p.ks + row0 + key);
            vs = __ldg(p.vs + row0 + key);
          }
          const int rs = nt % C::RSLOTS, cs = nt % C::SLOTS;
          if (!mbar_wait_warp(&bar.raw_full[rs], (nt / C::RSLOTS) & 1, err) ||
              !mbar_wait_warp(&bar.empty[cs], ((nt / C::SLOTS) & 1) ^ 1, err)) {
            failed = true;
            break;
          }
          if (!is_v) {
            // these scales' places were last used four steps before, whose softmax is done: the slot just
            // found free held a tile that was used after it
            const uint32_t gs = step0 + j;
            sh.sc[gs % SC_SLOTS][0][t] = ks;
            sh.sc[gs % SC_SLOTS][1][t] = vs;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sc_full[gs % SC_SLOTS]);
          }
          const uint8_t* src = sR + rs * C::RAW;
          uint8_t* dst = sT + cs * C::TILE;
          // 16 codes a piece; eight lanes take two rows of four pieces, so that their stores meet all banks
#pragma unroll
          for (int u = 0; u < D / 16; ++u) {
            const int row = (t >> 2) + 32 * (u & 3), c = (t & 3) + 4 * (u >> 2);
            const uint4 x = *reinterpret_cast<const uint4*>(src + row * D + c * 16);
            const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[2 * e] = widen_codes(__byte_perm(wd[e], 0, 0x4140));
              o[2 * e + 1] = widen_codes(__byte_perm(wd[e], 0, 0x4342));
            }
            uint8_t* piece = dst + (u >> 2) * (KT * 128) + row * 128;
            const int ch = 2 * (c & 3);
            *reinterpret_cast<uint4*>(piece + ((ch ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(piece + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bar.full[cs]);
            mbar_arrive(&bar.raw_empty[rs]);
          }
        }
        step0 += sg.nk;
      }
    }
  } else {
    set_regs_down<BITS == 8 ? 56 : 72>();
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
    const uint32_t box[4] = {64, (uint32_t)p.GQ, 1, (uint32_t)(128 / p.GQ)};
    if (!encode_tensor_map(&mapQ, p.q, 4, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const uint64_t rowb = (uint64_t)D * BITS / 8;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.N_cap, (uint64_t)p.P * p.H_kv};
  const uint64_t strides[2] = {rowb, (uint64_t)p.N_cap * rowb};
  const uint32_t box[3] = {BITS == 8 ? (uint32_t)D : 64u, (uint32_t)KT, 1};  // 128 keys
  auto encode = [&](CUtensorMap* map, const void* base) {
    return BITS == 8 ? encode_byte_tensor_map(map, base, 3, dims, strides, box, 0)
                     : encode_tensor_map(map, base, 3, dims, strides, box);
  };
  if (!encode(&mapK, p.K) || !encode(&mapV, p.V)) return cudaErrorInvalidValue;
  constexpr size_t smem = C::TILES + sizeof(Shared<BITS>);
  static_assert(smem <= 227 * 1024, "a block's shared memory");
  auto kern = prefix_tc_kernel<D, BITS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<p.blocks, C::THREADS, smem, s>>>(mapQ, mapK, mapV, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixParams& p, int d, cudaStream_t s) {
  if (d == 128) return p.ks ? launch_t<128, 8>(p, s) : launch_t<128, 16>(p, s);
  return p.ks ? launch_t<64, 8>(p, s) : launch_t<64, 16>(p, s);
}

}  // namespace pisa
