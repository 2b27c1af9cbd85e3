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
//
// A bf16 cache: bf16 operands, P rounded to bf16 (half a step, 2^-8 of each weight, the size of the
// output's own rounding).  An 8-bit cache: fp16 operands.  Four warps widen the codes, whole numbers,
// into the swizzled tiles that the MMA reads (two instructions a pair; to bf16 it would be four); Q is
// brought to at most 2 in magnitude by a power of two a row and kept as fp16 in place (exact but for
// elements below 2^-14 of the row's largest, which keep 2^-25 of it); the key's scale multiplies the
// fp32 logit, and the value's scale the weight before it is rounded, 2^-11 of it (2^-32 of the row's
// largest at least, codes.cuh).  The reference then follows the largest product of a weight and its value's
// scale.  A step's largest logit and largest scale together bound that; only where the bound asks for a raise
// are logits and scales added key by key (in a job's first steps, and in later ones whose largest belong to
// different keys).
//
// Two streams keep the tensor pipe busy while the softmax of the other one runs, a warpgroup for
// each.  With more than 128 rows a stream is a half of the rows, and both use the same tiles; with
// fewer, both streams have all rows, one the even steps and one the odd ones, each with its own
// m, l and O, which are joined when a job's segment ends.
//
// Roles: two softmax warpgroups; a producer warp (TMA); a warp that issues the MMAs;
// with the 8-bit cache the widening warpgroup.  TMEM: S of stream i at 128 i (its first 64 columns
// hold P afterwards), O of stream i at 256 + 128 i.  The MMAs of one thread run in order, so a stream's
// next S is issued right behind its O += P V, which reads P from the same columns.  Every wait is
// bounded.
//
// Measured (d = 128): 256 tokens of 32 / 2 heads after 131072 bf16 keys 379-392 us, 1.40-1.45 PFLOP/s; a step of
// 256 rows takes 3300 clocks, of which the products alone would take 2048 and their operands' way through
// shared memory, with the copies, up to 2560; the rest is the softmax's latency that two streams do
// not hide.  (Weights handed over in halves, so that O += P V starts earlier: no gain.  Pairs of SMs
// that share the tiles, halving the operands' reads: slower, each step then waits for the other SM.)  With
// codes a step takes 4100 clocks (472 us): the widened tiles are written and read once more.  Short
// prefixes pay for the start (7 us to the first scores of codes, 5 of bf16), the parts' 128 KB a SM
// (3-5 us) and the join (5 us).
#include <algorithm>

#include "codes.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "prefix_plan.cuh"

namespace pisa {
namespace {

constexpr int ROWS = TC_ROWS, KT = PREFIX_KT;
constexpr float MAX_GROWTH = 8.f;  // log2 units the maximum may pass a row's reference
constexpr float SCALE_CEILING = 100.f;  // what log2 of larger value scales counts as (their rows' outputs may overflow)

template <int D, int BITS>
struct Cfg {
  static constexpr int THREADS = BITS == 8 ? 512 : 384;
  static constexpr int PRODUCER = BITS == 8 ? 12 : 8, ISSUER = PRODUCER + 1;  // warps
  static constexpr uint32_t QT_BYTES = 128 * D * 2;     // 128 query rows
  static constexpr uint32_t TILE = KT * D * 2;          // a K or V tile in bf16
  static constexpr uint32_t RAW = KT * D;               // in codes
  // registers a thread of the softmax, of the widening and of the producing and issuing warpgroup, of 512 x 128
  // and 384 x 168 at launch.  The softmax holds 128 logits: with less it spills (256 tokens of 32 / 2 heads,
  // 131072 keys: 466 us for codes with 208 / 56 / 40, 478 with 208 / 40 / 56; with 200 a fifth more, with 192 a third;
  // bf16 398 us with 208 / 88, 416 with 200 / 104)
  static constexpr int REGS_SOFTMAX = 208, REGS_WIDEN = 56, REGS_ISSUE = BITS == 8 ? 40 : 88;
  static_assert(BITS == 8 ? 2 * REGS_SOFTMAX + REGS_WIDEN + REGS_ISSUE <= 4 * 128
                          : 2 * REGS_SOFTMAX + REGS_ISSUE <= 3 * 168, "registers of the block");
  static constexpr int SLOTS = BITS == 8 ? 3 : 5;
  static constexpr int RSLOTS = 3;
  static constexpr size_t TILES = 2 * QT_BYTES + SLOTS * TILE + (BITS == 8 ? RSLOTS * RAW : 0);
};

constexpr int SC_SLOTS = 4;

struct Bars {
  uint64_t q_full, q_ready, q_empty;   // Q copied; brought to fp16 (8-bit cache); no longer read
  uint64_t full[5], empty[5];          // bf16 tiles
  uint64_t raw_full[3], raw_empty[3];  // tiles of codes
  uint64_t sc_full[SC_SLOTS];          // a step's scales
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t x_full, x_done;             // the streams' meeting at the end of a segment
  uint64_t drain;
};

// A softmax warp's counts so far: steps of each stream, all steps, meetings of the streams, segments.
struct Counts {
  uint32_t it[2], steps, meets, segs;
};

// A warp's walk over the block's segments: in its registers, or in shared memory where those are scarce.
template <bool SHARED>
struct Walk {
  PrefixWalk w;
  __device__ __forceinline__ void start(const PrefixWalk& from, PrefixWalk*) { w = from; }
  __device__ __forceinline__ bool next(const PrefixParams& p, int block) { return w.next(p, block); }
  __device__ __forceinline__ const PrefixWalk& now() const { return w; }
};
template <>
struct Walk<true> {
  PrefixWalk* at;
  __device__ __forceinline__ void start(const PrefixWalk& from, PrefixWalk* place) {
    at = place;
    keep(from);
  }
  __device__ __forceinline__ bool next(const PrefixParams& p, int block) {
    PrefixWalk w = *at;
    __syncwarp();
    const bool more = w.next(p, block);
    keep(w);
    return more;
  }
  __device__ __forceinline__ const PrefixWalk& now() const { return *at; }
  __device__ __forceinline__ void keep(const PrefixWalk& w) {
    if ((threadIdx.x & 31) == 0) *at = w;
    __syncwarp();
  }
};

template <int BITS>
struct ForCodes {};
template <>
struct ForCodes<8> {
  __align__(16) float sc[SC_SLOTS][3][KT];  // scales of a step: keys', values'; what the values' add to a logit (log2)
  uint32_t top[SC_SLOTS][4];                // largest of a widening warp's value scales, as bits
  float q_factor[ROWS];                     // logit factor of a row: scale log2 e times its power of two
};

// What follows the tiles in shared memory (all of it dynamic: with five bf16 tiles there is room for
// 3 KB beside them, and none for an alignment gap).
template <int BITS>
struct Shared {
  Bars bar;
  float2 ml[2][128];                               // the streams' maxima and sums, when they meet
  PrefixWalk walks[BITS == 8 ? 14 : 8];            // each warp's walk, where its registers are wanted
  Counts counts[8];
  uint32_t tmem;
  ForCodes<BITS> code;
};

// One row of Q in its swizzled tile, bf16 -> fp16 times the power of two that brings its largest
// element to [1, 2); returns sl2 over that power.
template <int D>
__device__ __forceinline__ float normalise_row(uint8_t* tile, int row, float sl2) {
  auto at = [&](int c) {
    return reinterpret_cast<uint4*>(tile + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
  };
  uint4 x[D / 8];
#pragma unroll
  for (int c = 0; c < D / 8; ++c) x[c] = *at(c);
  uint32_t most[2] = {0, 0};  // largest magnitudes of two halves of a word each: as integers they are in order
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    most[0] = __vmaxu2(most[0], __vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu));
    most[1] = __vmaxu2(most[1], __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu));
  }
  const uint32_t both = __vmaxu2(most[0], most[1]);
  const uint32_t top = min(max(max(both >> 23, (both >> 7) & 0x1ffu), 1u), 253u);  // exponent (infinities stay so)
  const float down = __uint_as_float((254u - top) << 23);                          // 2^(127 - top)
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    uint32_t* w = &x[c].x;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_f16x2(bf16_lo(w[e]) * down, bf16_hi(w[e]) * down);
    *at(c) = x[c];
  }
  return sl2 * __uint_as_float(top << 23);
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

// Where a finished query row goes: the output (the whole job was this segment) or a part's slot.  The output
// sums are read from tensor memory in the accumulators' layout (a lane has pairs of columns of rows r and
// r + 8), so that a store fills whole 32-byte sectors of eight rows: a row a thread it took twice as long.
struct RowOut {
  bool live;
  size_t orow;
  float fa, fo;  // factors of the sums and of the row's own output
};
// The row's place and factors; `stats`: this lane writes its log-sum-exp, or maximum and sum.  Warp-wide.
__device__ __forceinline__ RowOut row_out(const PrefixParams& p, const PrefixWalk& w, int local, bool live, float m, float l,
                                          bool stats) {
  RowOut r;
  r.live = live;
  r.fa = 1.f;
  r.fo = 0.f;
  if (w.slot >= 0) {
    r.orow = (size_t)w.slot * ROWS + local;
    if (live && stats) p.part_ml[r.orow] = make_float2(m, l);
    return r;
  }
  const int mrow = w.tile * ROWS + local, tok = mrow >> p.gq_bits;
  r.orow = (size_t)(w.g.first + tok) * p.H_q + (size_t)w.head * p.GQ + (mrow - tok * p.GQ);
  float lse;
  join_own(m, l, live && p.lse_own ? p.lse_own[r.orow] : NEG_INF, r.fa, r.fo, lse);
  __syncwarp();  // lse may be lse_own: all four lanes of a row have read it
  if (live && stats && p.lse) p.lse[r.orow] = lse;
  return r;
}
// 32 columns from c on of rows r and r + 8 of a half of 16, x[4 g + 2 e + i]: column c + 8 g + 2 q + i of row r + 8 e.
template <int D>
__device__ __forceinline__ void put_columns(const PrefixParams& p, const PrefixWalk& w, const RowOut (&r)[2], int c, int q,
                                            const uint32_t (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!r[e].live) continue;
    const size_t at = r[e].orow * D + c + 2 * q;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float a = __uint_as_float(x[4 * g + 2 * e]), b = __uint_as_float(x[4 * g + 2 * e + 1]);
      if (w.slot >= 0) {
        *reinterpret_cast<float2*>(p.part_o + at + 8 * g) = make_float2(a, b);
        continue;
      }
      float v0 = r[e].fa == 0.f ? 0.f : a * r[e].fa, v1 = r[e].fa == 0.f ? 0.f : b * r[e].fa;
      if (p.o_own && r[e].fo != 0.f) {
        const uint32_t own = *reinterpret_cast<const uint32_t*>(p.o_own + at + 8 * g);
        v0 += bf16_lo(own) * r[e].fo;
        v1 += bf16_hi(own) * r[e].fo;
      }
      *reinterpret_cast<uint32_t*>(p.o + at + 8 * g) = pack_bf16x2(v0, v1);
    }
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

  // The producer sets up the barriers and starts to fetch at once; the others meet when they and the tensor
  // memory are there.
  if (warp == C::PRODUCER) {
    if (lane == 0) {
      prefetch_map(&mapQ);
      prefetch_map(&mapK);
      prefetch_map(&mapV);
      mbar_init(&bar.q_full, 1);
      mbar_init(&bar.q_ready, 8);
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
    __syncwarp();
    asm volatile("barrier.cta.arrive 1, %0;" ::"n"(C::THREADS) : "memory");
  } else if (warp == C::ISSUER) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  PrefixWalk first;  // (the first segment is found here: with all registers, and in one piece of code)
  first.init(p, block, block == 0 && warp == 0);
  const bool any_work = first.next(p, block);
  uint32_t tmem = 0;
  if (warp != C::PRODUCER) {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(C::THREADS) : "memory");
    tc_fence_after();
    tmem = sh.tmem;
  }

  if (warp < 8) {
    // ------------------------------ softmax ------------------------------
    set_regs_up<C::REGS_SOFTMAX>();
    const int h = warp >> 2;                                 // stream
    const int trow = (warp & 3) * 32 + lane;                 // TMEM lane
    const int q = lane & 3;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lanes + 128 * h, o_tmem = tmem + lanes + 256 + 128 * h;
    Walk<true> walk;
    walk.start(first, &sh.walks[warp]);
    Counts& count = sh.counts[warp];
    if (lane == 0) count = Counts{};
    __syncwarp();
    bool failed = false;
    for (bool more_work = any_work; !failed && more_work; more_work = walk.next(p, block)) {
      const PrefixWalk& w = walk.now();
      const Segment sg(p, w);
      const int local = (sg.lag == 1 ? 128 * h : 0) + trow;  // row in the tile
      const bool any = local - lane < sg.rows;
      // rows r, r + 8, r + 16, r + 24 of the warp's 32: a lane holds a quarter of the columns of each, so it wants
      // a quarter of the keys' scales
      float m[4];                      // reference, log2 units
      float sl2[4];                    // logit factor
      if constexpr (BITS == 8) {
        const uint32_t seg = count.segs;
        if (!mbar_wait_warp(&bar.q_full, seg & 1, err)) break;
        if (sg.lag == 1 || h == 0) sh.code.q_factor[128 * h + trow] = normalise_row<D>(sQ + h * C::QT_BYTES, trow, p.sl2);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_ready);
        if (!mbar_wait_warp(&bar.q_ready, seg & 1, err)) break;
      }
      unsigned long long l2[4];        // a lane's share of the sum, even and odd columns
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = NEG_INF;
        l2[i] = pack_f32x2(0.f, 0.f);
        sl2[i] = p.sl2;
        if constexpr (BITS == 8) sl2[i] = sh.code.q_factor[(sg.lag == 1 ? 128 * h : 0) + (warp & 3) * 32 + 8 * i + (lane >> 2)];
      }
      uint32_t n = count.it[h], gs = count.steps + (sg.lag == 1 ? 0 : h);
      bool begun = false;  // O holds sums of this segment
      for (int j = sg.lag == 1 ? 0 : h; j < sg.nk; j += sg.lag, ++n, gs += sg.lag) {
        const int valid = min(KT, w.g.len - (w.k0 + j) * KT);
        float most = 0.f;  // codes: what the step's largest value scale adds to a logit (a bound)
        if constexpr (BITS == 8) {
          if (!mbar_wait_warp(&bar.sc_full[gs % SC_SLOTS], (gs / SC_SLOTS) & 1, err)) {
            failed = true;
            break;
          }
          const uint4 x = *reinterpret_cast<const uint4*>(sh.code.top[gs % SC_SLOTS]);
          // 2^(exponent + 1) is above the largest; scales beyond 2^100 are taken as that
          const float log2_above = (float)((int)(max(max(x.x, x.y), max(x.z, x.w)) >> 23) - 126);
          most = fminf(fmaxf(log2_above, SCALE_FLOOR), SCALE_CEILING) - WEIGHT_ROOM;
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
            for (int g = 0; g < 16; ++g) {
              const float2 kf = *reinterpret_cast<const float2*>(&sh.code.sc[gs % SC_SLOTS][0][8 * g + 2 * q]);
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  float x, y;
                  unpack_f32x2(mul_f32x2(pack_u32x2(s[i][4 * g + e], s[i][4 * g + e + 1]), pack_f32x2(kf.x, kf.y)), x, y);
                  s[i][4 * g + e] = __float_as_uint(x);
                  s[i][4 * g + e + 1] = __float_as_uint(y);
                }
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
          float top[4];
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
            top[i] = a * sl2[i] + most;
            moved = moved || top[i] > m[i] + MAX_GROWTH;
          }
          bool raise = __any_sync(0xffffffffu, moved);
          if constexpr (BITS == 8) {
            if (raise) {  // the maxima themselves
#pragma unroll
              for (int i = 0; i < 4; ++i) top[i] = NEG_INF;
#pragma unroll
              for (int g = 0; g < 16; ++g) {
                const float2 lv = *reinterpret_cast<const float2*>(&sh.code.sc[gs % SC_SLOTS][2][8 * g + 2 * q]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t* x = &s[i >> 1][4 * g + 2 * (i & 1)];
                  float a, b;
                  unpack_f32x2(fma_f32x2(pack_u32x2(x[0], x[1]), pack_f32x2(sl2[i], sl2[i]), pack_f32x2(lv.x, lv.y)), a, b);
                  top[i] = fmaxf(fmaxf(top[i], a), b);
                }
              }
              moved = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                moved = moved || top[i] > m[i] + MAX_GROWTH;
              }
              raise = __any_sync(0xffffffffu, moved);
            }
          }
          if (raise) {
            // the references follow the maxima; O (of the steps before) with them
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float to = fmaxf(m[i], top[i]), by = to == NEG_INF ? 0.f : m[i] - to;
              f[i] = fast_exp2(by);
              m[i] = to;
              const float h = fast_exp2(0.5f * by);  // (l times 2^by, where l is large and 2^by below fp32's range too)
              l2[i] = mul_f32x2(mul_f32x2(l2[i], pack_f32x2(h, h)), pack_f32x2(h, h));
            }
            if (begun) {
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
                if constexpr (BITS == 8) vf = *reinterpret_cast<const float2*>(&sh.code.sc[gs % SC_SLOTS][1][64 * c + 8 * g + 2 * q]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // row r + 16 i + 8 e
                  const uint32_t* x = &s[i][32 * c + 4 * g + 2 * e];
                  float a, b;
                  unpack_f32x2(fma_f32x2(pack_u32x2(x[0], x[1]), pack_f32x2(sl2[2 * i + e], sl2[2 * i + e]), ref[2 * i + e]), a, b);
                  a = fast_exp2(a);
                  b = fast_exp2(b);
                  const unsigned long long ab = pack_f32x2(a, b);
                  l2[2 * i + e] = add_f32x2(l2[2 * i + e], ab);
                  if constexpr (BITS == 8) unpack_f32x2(mul_f32x2(ab, pack_f32x2(vf.x, vf.y)), a, b);
                  pk[2 * g + e] = BITS == 8 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
                }
              }
              tmem_st_16x32(s_tmem + ((uint32_t)(16 * i) << 16) + 32 * c, pk);
            }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[h]);
        begun = true;
      }
      // the streams' steps of this segment
      const uint32_t n0 = sg.lag == 1 ? sg.nk : (sg.nk + 1) / 2, n1 = sg.lag == 1 ? sg.nk : sg.nk / 2;
      const uint32_t it[2] = {count.it[0] + n0, count.it[1] + n1}, meets = count.meets;
      __syncwarp();
      if (lane == 0) count = Counts{{it[0], it[1]}, count.steps + sg.nk, meets + (sg.lag == 1 ? 0 : 1), count.segs + 1};
      __syncwarp();
      if (failed) break;
      float l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack_f32x2(l2[i], a, b);
        a += b;
        a += __shfl_xor_sync(0xffffffffu, a, 1);
        l[i] = a + __shfl_xor_sync(0xffffffffu, a, 2);
      }
      const int row0 = (sg.lag == 1 ? 128 * h : 0) + (warp & 3) * 32 + (lane >> 2);  // the first of the lane's rows
      if (sg.lag == 1) {
        if (!mbar_wait_warp(&bar.o_done[h], (it[h] - 1) & 1, err)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (any)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            RowOut out[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = row0 + 8 * (i + e);
              out[e] = row_out(p, w, row, row < sg.rows, m[i + e], l[i + e], q == 0);
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t r[16];
              tmem_ld_16x32(o_tmem + ((uint32_t)(8 * i) << 16) + c, r);
              tmem_wait_ld();
              put_columns<D>(p, w, out, c, q, r);
            }
          }
        tc_fence_before();
      } else {
        // both streams have parts of every row: joined here, rows below 16 of 32 by one warpgroup, the others by
        // the other one
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (q == 0) sh.ml[h][row0 + 8 * i] = make_float2(m[i], l[i]);
        __syncwarp();
        if (!mbar_wait_warp(&bar.o_done[0], (it[0] - 1) & 1, err) ||
            (n1 > 0 && !mbar_wait_warp(&bar.o_done[1], (it[1] - 1) & 1, err))) {
          failed = true;
          break;
        }
        if (lane == 0) mbar_arrive(&bar.x_full);
        if (!mbar_wait_warp(&bar.x_full, meets & 1, err)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (any) {
          RowOut out[2];
          float f0[2], f1[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = row0 + 16 * h + 8 * e;
            const float2 a = sh.ml[0][row], b = sh.ml[1][row];
            const float top = fmaxf(a.x, b.x);
            f0[e] = a.x == NEG_INF ? 0.f : fast_exp2(a.x - top);
            f1[e] = b.x == NEG_INF ? 0.f : fast_exp2(b.x - top);
            const float sum = (a.x == NEG_INF ? a.y : times_exp2(a.y, a.x - top)) + (b.x == NEG_INF ? b.y : times_exp2(b.y, b.x - top));
            out[e] = row_out(p, w, row, row < sg.rows, top, sum, q == 0);
          }
          const uint32_t o0 = tmem + lanes + 256 + ((uint32_t)(16 * h) << 16);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t r[16], r1[16];
            tmem_ld_16x32(o0 + c, r);
            if (n1 > 0) tmem_ld_16x32(o0 + 128 + c, r1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int e = (k >> 1) & 1;
              float x = __uint_as_float(r[k]) * f0[e];
              if (n1 > 0) x = fmaf(__uint_as_float(r1[k]), f1[e], x);
              r[k] = __float_as_uint(x);
            }
            put_columns<D>(p, w, out, c, q, r);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.x_done);
        if (!mbar_wait_warp(&bar.x_done, meets & 1, err)) {  // both O have been read: the next segment may write them
          failed = true;
          break;
        }
      }
    }
  } else if (BITS == 8 && warp < 12) {
    // ------------------------------ codes to fp16 ------------------------------
    if constexpr (BITS == 8) {
      set_regs_down<C::REGS_WIDEN>();
      const int t = threadIdx.x - 256;
      Walk<true> walk;
      walk.start(first, &sh.walks[warp]);
      uint32_t nt = 0, step0 = 0;
      bool failed = false;
      for (bool more_work = any_work; !failed && more_work; more_work = walk.next(p, block)) {
        const PrefixWalk& w = walk.now();
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
            sh.code.sc[gs % SC_SLOTS][0][t] = ks;
            sh.code.sc[gs % SC_SLOTS][1][t] = vs;
            sh.code.sc[gs % SC_SLOTS][2][t] = fminf(scale_log2(vs), SCALE_CEILING - WEIGHT_ROOM);
            const uint32_t mag = __float_as_uint(vs) & 0x7fffffffu;
            const uint32_t most = __reduce_max_sync(0xffffffffu, mag <= 0x7f800000u ? mag : 0u);  // (not of a NaN)
            if (lane == 0) sh.code.top[gs % SC_SLOTS][warp - 8] = most;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sc_full[gs % SC_SLOTS]);
          }
          // 16 codes a piece; eight lanes take two rows of four pieces, so that their stores meet all banks
          const uint8_t* src = sR + rs * C::RAW + (t >> 2) * D + (t & 3) * 16;
          uint8_t* dst = sT + cs * C::TILE + (t >> 2) * 128;
          const int swz = (t >> 2) & 7, c0 = ((2 * (t & 3)) ^ swz) << 4, c1 = ((2 * (t & 3) + 1) ^ swz) << 4;
#pragma unroll
          for (int u = 0; u < D / 16; ++u) {  // rows 32 (u mod 4) further, columns 64 (u / 4)
            const uint4 x = *reinterpret_cast<const uint4*>(src + 32 * (u & 3) * D + 64 * (u >> 2));
            const uint32_t w0 = x.x ^ 0x80808080u, w1 = x.y ^ 0x80808080u, w2 = x.z ^ 0x80808080u, w3 = x.w ^ 0x80808080u;
            uint8_t* row = dst + (u >> 2) * (KT * 128) + 32 * (u & 3) * 128;
            *reinterpret_cast<uint4*>(row + c0) =
                make_uint4(widen_f16<0x4140>(w0), widen_f16<0x4342>(w0), widen_f16<0x4140>(w1), widen_f16<0x4342>(w1));
            *reinterpret_cast<uint4*>(row + c1) =
                make_uint4(widen_f16<0x4140>(w2), widen_f16<0x4342>(w2), widen_f16<0x4140>(w3), widen_f16<0x4342>(w3));
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
    // The producing and issuing warps are two of one warpgroup: all of it changes its registers by one instruction.
    set_regs_down<C::REGS_ISSUE>();
    if (warp == C::PRODUCER) {
      // ------------------------------ producer ------------------------------
      constexpr uint32_t N = BITS == 8 ? C::RSLOTS : C::SLOTS;
      Walk<BITS == 8> walk;
      walk.start(first, &sh.walks[BITS == 8 ? warp : 0]);
      uint32_t nt = 0, seg = 0;  // tiles and segments so far
      bool failed = false;
      for (bool more_work = any_work; !failed && more_work; more_work = walk.next(p, block)) {
        const PrefixWalk& w = walk.now();
        const Segment sg(p, w);
        if (!mbar_wait_warp(&bar.q_empty, (seg & 1) ^ 1, err)) break;
        if (lane == 0) {
          const int streams = sg.lag == 1 ? 2 : 1;
          mbar_arrive_expect_tx(&bar.q_full, streams * C::QT_BYTES);
          for (int h = 0; h < streams; ++h)
            for (int c = 0; c < DH; ++c)
              tma_load_4d(sQ + h * C::QT_BYTES + c * (128 * 128), &mapQ, &bar.q_full, 64 * c, 0, w.head,
                          w.g.first + ((w.tile * ROWS + h * 128) >> p.gq_bits));
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
      // fp16 operands have format 0 where bf16 have 1; V: d contiguous, N-major
      constexpr uint32_t formats = BITS == 8 ? (1u << 7) | (1u << 10) : 0u;
      constexpr uint32_t id_qk = idesc_bf16_f32(128, KT) & ~formats;
      constexpr uint32_t id_pv = (idesc_bf16_f32(128, D) & ~formats) | (1u << 16);
      Walk<BITS == 8> walk;
      walk.start(first, &sh.walks[BITS == 8 ? warp : 0]);
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
      // descriptors of the first tile and Q slot: the others differ in the address field alone (16-byte units of
      // the low word)
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sT), 16, 1024);
      const uint32_t k_hi = (uint32_t)(k_desc >> 32), q_lo = (uint32_t)smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint32_t k_lo = (uint32_t)k_desc, v_lo = (uint32_t)smem_desc_sw128(smem_u32(sT), KT * 128, 1024);
      auto desc = [&](uint32_t lo) { return pack_u32x2(lo, k_hi); };  // (8-row groups of 1024 bytes in all of them)
      auto qk = [&](int h, int qs, uint32_t n) {  // S of stream h = Q (slot qs) K^T
        const uint32_t a = q_lo + qs * (C::QT_BYTES >> 4), b = k_lo + (n % C::SLOTS) * (C::TILE >> 4), d = tmem + 128 * h;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          umma_bf16(d, desc(a + (((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4)),
                    desc(b + (((s >> 2) * (KT * 128) + (s & 3) * 32) >> 4)), id_qk, s > 0 ? 1u : 0u);
        umma_commit(&bar.s_full[h]);
      };
      auto pv = [&](int h, uint32_t n, bool first) {  // O of stream h (+)= P V
        const uint32_t b = v_lo + (n % C::SLOTS) * (C::TILE >> 4), d = tmem + 256 + 128 * h, a = tmem + 128 * h;
#pragma unroll
        for (int s = 0; s < KT / 16; ++s)
          umma_bf16_ts(d, a + 8 * s, desc(b + ((s * 16 * 128) >> 4)), id_pv, s > 0 ? 1u : first ? 0u : 1u);
        umma_commit(&bar.o_done[h]);
      };
      for (bool more_work = any_work; !failed && more_work; more_work = walk.next(p, block)) {
        const PrefixWalk& w = walk.now();
        const Segment sg(p, w);
        if (!mbar_wait_warp(BITS == 8 ? &bar.q_ready : &bar.q_full, seg & 1, err)) break;
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
    }
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
  cudaError_t e = allow_shared<prefix_tc_kernel<D, BITS>>(smem);
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
