// Attention of many new tokens over the paged cache on the tensor cores of the 5th generation: tiles of up to 256 query
// rows (tokens x heads of one KV head), 128 keys a step, one block a SM.
//
//   S = Q K^T (fp32 in tensor memory), P = 2^(S scale log2 e - m) as bf16 back into tensor memory over S,
//   O += P V in tensor memory, l = sum of the unrounded P
//
// m is a row's reference, not its running maximum: a segment's first step sets it to 8 above the step's maximum, and
// later ones take it as it is.  Only where a lane's sum of a step's weights (32 keys of a row) passes 1 are the maxima found,
// the reference raised to 8 above them, O multiplied by 2^(old - new) and the step's weights made again.  So no weight is above
// 1 (a value at the end of bf16's range gives a finite product), a row's largest is 2^-8 at least, and the division by l at
// the end is exact whatever m is.  With the usual logits that
// hardly happens, so most steps look for no maximum at all (with one a step: 4096 tokens after 28672 of 32 / 8 heads
// 1550 us).  P is rounded to bf16, half a step (2^-8) of each weight, as the output is.
//
// Two streams keep the tensor pipe busy while the softmax of the other one runs, a warpgroup for each.  With more than
// 128 rows a stream is a half of the rows, and both use the same tiles; with fewer, both streams have all rows, one
// the even steps and one the odd ones, each with its own m, l and O, joined when a job's segment ends.
//
// A step's keys come in copies of min(S, 128) tokens of a page, issued by as many lanes of the producing warps.  Copies for pages that are not there, or that begin behind
// the sequence's last key, are given a page number past the pool and read as zeros.  Logits are masked by row only
// in steps that pass the last key which the warp's first row sees, and in steps with such a page.
//
// Roles: two softmax warpgroups; two producer warps (TMA); a warp that issues the MMAs.  TMEM: NB buffers of 128 columns
// for S (the first 64 of one hold P afterwards), then O of both streams.  With d = 64 there is room for a third buffer,
// so that a stream finds its next S made when it has handed over its P.  The MMAs of one thread run in order, so the next
// S of a buffer is issued right behind the O += P V that reads P from it.  Every wait is bounded.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"
#include "pdl.cuh"

namespace pisa {
namespace {

constexpr int ROWS = PAGED_TC_ROWS, KT = PAGED_KT;
constexpr float MOST = 1.f;  // a lane's sum of a row's weights in a step above which the references are raised
constexpr float ROOM = 8.f;  // how far above the maxima (log2 units)

constexpr int THREADS = 384, PRODUCER = 8, ISSUER = 9, PRODUCER2 = 10;  // warps
// Registers a thread of the softmax and of the other warpgroup, of 384 x 168 at launch: the softmax holds 128 logits.
constexpr int REGS_SOFTMAX = 208, REGS_ISSUE = 88;
static_assert(2 * REGS_SOFTMAX + REGS_ISSUE <= 3 * 168, "registers of the block");

template <int D>
struct Cfg {
  static constexpr int NB = D == 64 ? 3 : 2;         // buffers of S
  static constexpr int K_SLOTS = D == 64 ? 5 : 3, V_SLOTS = D == 64 ? 4 : 2;  // tiles
  static constexpr uint32_t QT_BYTES = 128 * D * 2;  // 128 query rows
  static constexpr uint32_t TILE = KT * D * 2;       // a K or V tile
  static constexpr size_t TILES = 2 * QT_BYTES + (K_SLOTS + V_SLOTS) * TILE;
  static_assert(NB * 128 + 2 * D <= 512, "tensor memory");
};

template <int D>
struct Bars {
  uint64_t q_full, q_empty;             // Q copied; no longer read
  uint64_t k_full[Cfg<D>::K_SLOTS], k_empty[Cfg<D>::K_SLOTS], v_full[Cfg<D>::V_SLOTS], v_empty[Cfg<D>::V_SLOTS];
  uint64_t s_full[Cfg<D>::NB], p_full[Cfg<D>::NB], o_done[Cfg<D>::NB];  // of a buffer of S: made, P in it, O += P V made
  uint64_t x_full, x_done;              // the streams' meeting at the end of a segment
  uint64_t drain;
};

// A softmax warp's counts so far: products, meetings of the streams.
struct Counts {
  uint32_t made, meets;
};

// What follows the tiles in shared memory.
template <int D>
struct Shared {
  Bars<D> bar;
  float2 ml[2][64];       // a stream's maxima and sums of the rows that the other one writes, when they meet
  PagedWalk walks[11];    // each warp's walk: registers are wanted elsewhere
  Counts counts[8];
  uint32_t tmem;
};

// A warp's walk over the block's segments, in shared memory.
struct Walk {
  PagedWalk* at;
  __device__ __forceinline__ void start(const PagedWalk& from, PagedWalk* place) {
    at = place;
    keep(from);
  }
  __device__ __forceinline__ bool next(const PagedParams& p, int block) {
    PagedWalk w = *at;
    __syncwarp();
    const bool more = w.next(p, block);
    keep(w);
    return more;
  }
  __device__ __forceinline__ const PagedWalk& now() const { return *at; }
  __device__ __forceinline__ void keep(const PagedWalk& w) {
    if ((threadIdx.x & 31) == 0) *at = w;
    __syncwarp();
  }
};

template <int R>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// A segment's streams: by rows (`lag` 1: both use every tile) or by steps (`lag` 2: stream = step mod 2).  Its products
// are numbered in the order in which they are made, streams in turn: product u is of stream u mod 2 and step u / 2 (by
// rows) or u (by steps), and S of u lies in buffer (products before the segment + u) mod NB.  S of u + NB is issued right
// behind the O += P V of u, which reads P from the same buffer.
struct Segment {
  int rows, nk, lag;
  __device__ __forceinline__ Segment(const PagedParams& p, const PagedWalk& w) {
    rows = w.rows(p);
    nk = w.k1 - w.k0;
    lag = rows > ROWS / 2 ? 1 : 2;
  }
  __device__ __forceinline__ int products() const { return lag == 1 ? 2 * nk : nk; }
};

// Where a finished query row goes: the output (the whole job was this segment) or a part's slot.  The output sums are
// read from tensor memory in the accumulators' layout (a lane has pairs of columns of rows r and r + 8), so that a
// store fills whole 32-byte sectors of eight rows.
struct RowOut {
  bool live;
  size_t orow;
  float f;  // factor of the sums
};
// The row's place and factor; `stats`: this lane writes its log-sum-exp, or maximum and sum.
__device__ __forceinline__ RowOut row_out(const PagedParams& p, const PagedWalk& w, int local, bool live, float m, float l,
                                          bool stats) {
  RowOut r;
  r.live = live;
  r.f = 1.f;
  if (w.slot >= 0) {
    r.orow = (size_t)w.slot * ROWS + local;
    if (live && stats) p.part_ml[r.orow] = make_float2(m, l);
    return r;
  }
  r.orow = w.row_at(p, local);
  float lse;
  r.f = finish_row(m, l, lse);
  if (live && stats && p.lse) p.lse[r.orow] = lse;
  return r;
}
// 32 columns from c on of rows r and r + 8 of a half of 16, x[4 g + 2 e + i]: column c + 8 g + 2 q + i of row r + 8 e.
template <int D>
__device__ __forceinline__ void put_columns(const PagedParams& p, const PagedWalk& w, const RowOut (&r)[2], int c, int q,
                                            const uint32_t (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!r[e].live) continue;
    const size_t at = r[e].orow * D + c + 2 * q;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float a = __uint_as_float(x[4 * g + 2 * e]), b = __uint_as_float(x[4 * g + 2 * e + 1]);
      if (w.slot >= 0)
        *reinterpret_cast<float2*>(p.part_o + at + 8 * g) = make_float2(a, b);
      else
        *reinterpret_cast<uint32_t*>(p.o + at + 8 * g) = r[e].f == 0.f ? 0u : pack_bf16x2(a * r[e].f, b * r[e].f);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapV, PagedParams p) {
  pdl_trigger();
  using C = Cfg<D>;
  constexpr int DH = D / 64;  // 64-column pieces of a Q or K row
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sT = sQ + 2 * C::QT_BYTES;
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem + C::TILES);
  Bars<D>& bar = sh.bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x;
  uint32_t* err = p.err;
  const int box_bits = min(p.s_bits, 7);  // a copy's keys, 2 to this

  // The first producer sets up the barriers and starts to fetch at once; the others meet when they and the tensor memory
  // are there.
  if (warp == PRODUCER) {
    if (lane == 0) {
      prefetch_map(&mapQ);
      prefetch_map(&mapK);
      prefetch_map(&mapV);
      mbar_init(&bar.q_full, 1);
      mbar_init(&bar.q_empty, 1);
      for (int i = 0; i < C::K_SLOTS; ++i) {
        mbar_init(&bar.k_full[i], 1);
        mbar_init(&bar.k_empty[i], 1);
      }
      for (int i = 0; i < C::V_SLOTS; ++i) {
        mbar_init(&bar.v_full[i], 1);
        mbar_init(&bar.v_empty[i], 1);
      }
      for (int i = 0; i < C::NB; ++i) {
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
    asm volatile("barrier.cta.arrive 1, %0;" ::"n"(THREADS) : "memory");
  } else if (warp == ISSUER) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  PagedWalk first;  // (the first segment is found here: with all registers, and in one piece of code)
  first.init(p, block, block == 0 && warp == 0);
  const bool any_work = first.next(p, block);
  uint32_t tmem = 0;
  if (warp != PRODUCER) {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(THREADS) : "memory");
    tc_fence_after();
    tmem = sh.tmem;
  }

  if (warp < 8) {
    // ------------------------------ softmax ------------------------------
    set_regs_up<REGS_SOFTMAX>();
    const int h = warp >> 2;                                 // stream
    const int q = lane & 3;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tmem = tmem + lanes + 128 * C::NB + D * h;
    Walk walk;
    walk.start(first, &sh.walks[warp]);
    Counts& count = sh.counts[warp];
    if (lane == 0) count = Counts{};
    __syncwarp();
    bool failed = false;
    for (bool more_work = any_work; !failed && more_work; more_work = walk.next(p, block)) {
      const PagedWalk& w = walk.now();
      const Segment sg(p, w);
      const int warp_row = (sg.lag == 1 ? 128 * h : 0) + (warp & 3) * 32;  // the warp's first row in the tile
      const int row0 = warp_row + (lane >> 2);                             // the first of the lane's four, 8 apart
      const bool any = warp_row < sg.rows;
      const int total = w.s.L + w.s.n, least = w.seen(p, warp_row);
      const int32_t* table = p.table + (size_t)w.b * p.M;
      // the page of the copy that this lane stands for, of step j (looked at a step later: the load is not waited for)
      const int first_key = w.k0 * KT, nk = sg.nk, lag = sg.lag;
      const int look_end = (lane << box_bits) < KT ? min(total, w.k1 * KT) : 0;
      auto look = [&](int j) {
        const int key = first_key + j * KT + (lane << box_bits);
        return key < look_end ? __ldg(table + (key >> p.s_bits)) : 0;
      };
      float m[4];                // references, log2 units
      unsigned long long l2[4];  // a lane's share of the sum, even and odd columns
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = NEG_INF;
        l2[i] = pack_f32x2(0.f, 0.f);
      }
      const unsigned long long sl2 = pack_f32x2(p.sl2, p.sl2);
      const uint32_t made = count.made;  // products before the segment
      uint32_t u = made + h;
      // O += P V of product v has been made.  (A wait may not be two phases ahead of its barrier.  The one before it in
      // v's buffer, of product v - NB, is known to be done: S of v was issued behind it.)
      auto o_done = [&](uint32_t v) { return mbar_wait_warp(&bar.o_done[v % C::NB], (v / C::NB) & 1, err); };
      bool begun = false;  // O holds sums of this segment
      bool blank = true;   // a row of the warp has no reference yet
      int page = look(lag == 1 ? 0 : h);
      for (int j = lag == 1 ? 0 : h; j < nk; j += lag, u += 2) {
        const uint32_t buf = u % C::NB, s_tmem = tmem + lanes + 128 * buf;
        const int key0 = first_key + j * KT;
        const unsigned none = __ballot_sync(0xffffffffu, (unsigned)page >= (unsigned)p.P);  // copies that have none
        page = look(j + lag);
        if (!mbar_wait_warp(&bar.s_full[buf], (u / C::NB) & 1, err)) {
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
          if (key0 + KT > least) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int lim = w.seen(p, row0 + 8 * i) - key0 - 2 * q;
#pragma unroll
              for (int g = 0; g < 16; ++g)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (8 * g + c >= lim) s[i >> 1][4 * g + 2 * (i & 1) + c] = __float_as_uint(NEG_INF);
            }
          }
          if (none) {
#pragma unroll
            for (int g = 0; g < 16; ++g)
              if (none >> (8 * g >> box_bits) & 1)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int c = 0; c < 4; ++c) s[i][4 * g + c] = __float_as_uint(NEG_INF);
          }
          // P against the references, and its sums
          unsigned long long sum[4];
          auto weights = [&] {
            unsigned long long ref[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = m[i] == NEG_INF ? 0.f : -m[i];
              ref[i] = pack_f32x2(x, x);
              sum[i] = 0ull;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)  // 64 keys
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t pk[16];
#pragma unroll
                for (int g = 0; g < 8; ++g)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {  // row r + 16 i + 8 e
                    const uint32_t* x = &s[i][32 * c + 4 * g + 2 * e];
                    float a, b;
                    unpack_f32x2(fma_f32x2(pack_u32x2(x[0], x[1]), sl2, ref[2 * i + e]), a, b);
                    a = fast_exp2(a);
                    b = fast_exp2(b);
                    sum[2 * i + e] = add_f32x2(sum[2 * i + e], pack_f32x2(a, b));
                    pk[2 * g + e] = pack_bf16x2(a, b);
                  }
                tmem_st_16x32(s_tmem + ((uint32_t)(16 * i) << 16) + 32 * c, pk);
              }
          };
          bool again = blank;
          if (!again) {
            weights();
            uint32_t far = 0;  // bits of the rows
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float a, b;
              unpack_f32x2(sum[i], a, b);
              far |= a + b > MOST ? 1u << i : 0u;
            }
            again = __any_sync(0xffffffffu, far);
            if (again) {  // (what lies in the rows behind the tile's last asks for nothing)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (row0 + 8 * i >= sg.rows) far &= ~(1u << i);
              again = __any_sync(0xffffffffu, far);
            }
          }
          if (again) {
            // the references follow the maxima, O (of the steps before) with them
            float f[4];
            bool none_seen = false;
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
              const float to = fmaxf(m[i], a * p.sl2 + ROOM);
              f[i] = to == NEG_INF ? 1.f : fast_exp2(m[i] - to);
              m[i] = to;
              none_seen = none_seen || (row0 + 8 * i < sg.rows && to == NEG_INF);
              l2[i] = mul_f32x2(l2[i], pack_f32x2(f[i], f[i]));
            }
            blank = __any_sync(0xffffffffu, none_seen);
            if (begun) {
              if (!o_done(u - 2)) {
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
            tmem_wait_st();  // the weights made before lie in the same columns, and two stores may land in any order
            weights();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) l2[i] = add_f32x2(l2[i], sum[i]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[buf]);
        begun = true;
      }
      const uint32_t all = sg.products(), meets = count.meets;
      const bool both = all > 1;  // the second stream has steps
      __syncwarp();
      if (lane == 0) count = Counts{made + all, meets + (sg.lag == 1 ? 0 : 1)};
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
      if (sg.lag == 1) {
        if (!o_done(made + all - 2 + h)) {
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
        // both streams have parts of every row: joined here, rows below 16 of 32 by one warpgroup, the others by the
        // other one
        float2* other = &sh.ml[h][(warp & 3) * 16 + (lane >> 2)];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (q == 0) other[8 * e] = h == 0 ? make_float2(m[2 + e], l[2 + e]) : make_float2(m[e], l[e]);
        __syncwarp();
        if ((both && !o_done(made + all - 2)) || !o_done(made + all - 1)) {  // in this order: the products' own
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
            const float2 mine = h == 0 ? make_float2(m[e], l[e]) : make_float2(m[2 + e], l[2 + e]);
            const float2 its = sh.ml[1 - h][(warp & 3) * 16 + (lane >> 2) + 8 * e];
            const float2 a = h == 0 ? mine : its, b = h == 0 ? its : mine;
            const float top = fmaxf(a.x, b.x);
            f0[e] = a.x == NEG_INF ? 0.f : fast_exp2(a.x - top);
            f1[e] = b.x == NEG_INF ? 0.f : fast_exp2(b.x - top);
            // (without a reference a sum is 0, or NaN where every logit was)
            const float sum = (a.x == NEG_INF ? a.y : a.y * f0[e]) + (b.x == NEG_INF ? b.y : b.y * f1[e]);
            out[e] = row_out(p, w, row, row < sg.rows, top, sum, q == 0);
          }
          const uint32_t o0 = tmem + lanes + 128 * C::NB + ((uint32_t)(16 * h) << 16);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t r[16], r1[16];
            tmem_ld_16x32(o0 + c, r);
            if (both) tmem_ld_16x32(o0 + D + c, r1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int e = (k >> 1) & 1;
              float x = __uint_as_float(r[k]) * f0[e];
              if (both) x = fmaf(__uint_as_float(r1[k]), f1[e], x);
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
    if (warp == 0 && lane == 0) p.split[block] = walk.now().split(p, block);
  } else {
    // The producing and issuing warps are two of one warpgroup: all of it changes its registers by one instruction.
    set_regs_down<REGS_ISSUE>();
    if (warp == PRODUCER || warp == PRODUCER2) {
      // ------------------------------ producers: Q and K; V ------------------------------
      // A warp each: a copy takes its warp 80 clocks, and a tile of pages of 16 tokens 8 or 16 copies.
      const bool is_v = warp == PRODUCER2;
      Walk walk;
      walk.start(first, &sh.walks[is_v ? 10 : 8]);
      uint32_t seg = 0, nt = 0;  // segments and tiles so far
      const uint32_t slots = is_v ? C::V_SLOTS : C::K_SLOTS;
      uint64_t *const full = is_v ? bar.v_full : bar.k_full, *const empty = is_v ? bar.v_empty : bar.k_empty;
      const CUtensorMap* map = is_v ? &mapV : &mapK;
      uint32_t slot = 0, phase = 0;
      bool failed = false;
      const int piece = lane & (DH - 1), in_tile = lane / DH << box_bits;  // this lane's copy of a tile
      const bool copies = in_tile < KT;
      uint8_t* const dst = sT + (is_v ? C::K_SLOTS * C::TILE : 0) + piece * (KT * 128) + in_tile * 128;
      const int in_page = (1 << p.s_bits) - 1;
      for (bool more_work = any_work; !failed && more_work; more_work = walk.next(p, block)) {
        const PagedWalk& w = walk.now();
        const Segment sg(p, w);
        if (!is_v) {
          if (!mbar_wait_warp(&bar.q_empty, (seg & 1) ^ 1, err)) break;
          if (lane == 0) {
            const int streams = sg.lag == 1 ? 2 : 1;
            mbar_arrive_expect_tx(&bar.q_full, streams * C::QT_BYTES);
            for (int h = 0; h < streams; ++h)
              for (int c = 0; c < DH; ++c)
                tma_load_4d(sQ + h * C::QT_BYTES + c * (128 * 128), &mapQ, &bar.q_full, 64 * c, 0, w.head,
                            w.s.first + ((w.tile * ROWS + h * 128) >> p.gq_bits));
          }
        }
        ++seg;
        const int total = w.s.L + w.s.n, head = w.head, nk = sg.nk;
        int key = w.k0 * KT + in_tile;
        const int end = w.k1 * KT;
        const int32_t* table = p.table + (size_t)w.b * p.M;
        // the page of this lane's copy (read two steps ahead, so that nobody waits for it)
        auto entry_of = [&](int c) { return copies && c < end && c < total ? __ldg(table + (c >> p.s_bits)) : -1; };
        int entry = entry_of(key), next = entry_of(key + KT);
        for (int j = 0; j < nk; ++j, key += KT) {
          const int later = entry_of(key + 2 * KT);
          if (!mbar_wait_warp(empty + slot, phase ^ 1, err)) {
            failed = true;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(full + slot, C::TILE);
          __syncwarp();
          if (copies)
            tma_load_4d(dst + slot * C::TILE, map, full + slot, 64 * piece, key & in_page, head,
                        (unsigned)entry < (unsigned)p.P ? entry : p.P);
          if (entry >= p.P) report_error(err, ERR_BAD_INDEX);
          __syncwarp();
          entry = next;
          next = later;
          if (++slot == slots) slot = 0, phase ^= 1;
          ++nt;
        }
      }
      // copies still in flight land before shared memory goes away (bounded; at once unless a wait failed)
      if (lane == 0) {
        if (seg > 0 && !is_v) mbar_wait(&bar.q_full, (seg - 1) & 1, err, 100000000ull);
        for (uint32_t u = nt > slots ? nt - slots : 0; u < nt; ++u) mbar_wait(full + u % slots, (u / slots) & 1, err, 100000000ull);
      }
      __syncwarp();
    } else if (warp == ISSUER) {
      // ------------------------------ MMAs ------------------------------
      constexpr uint32_t id_qk = idesc_bf16_f32(128, KT);
      constexpr uint32_t id_pv = idesc_bf16_f32(128, D) | (1u << 16);  // V: d contiguous, N-major
      Walk walk;
      walk.start(first, &sh.walks[9]);
      // A product's tiles and its P are asked for together, so that little time passes between two products' MMAs: the
      // tensor pipe's queue is short.  (One wait after the other, 150 clocks each though nothing was missing: 1490 us for
      // 4096 tokens after 28672 of 32 / 8 heads.  One lane that does everything, 1667 us: issuing wants a converged warp.
      // Two warps in turn, 1720 us: their MMAs mix, and a stream gets its next S later.)
      uint32_t seg = 0, made = 0;  // segments, products so far
      Ring<C::K_SLOTS> kr;         // the next tiles
      Ring<C::V_SLOTS> vr;
      bool failed = false;
      // descriptors of the first tile and Q slot: the others differ in the address field alone (16-byte units of the
      // low word)
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sT), 16, 1024);
      const uint32_t k_hi = (uint32_t)(k_desc >> 32), q_lo = (uint32_t)smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint32_t k_lo = (uint32_t)k_desc, v_lo = (uint32_t)smem_desc_sw128(smem_u32(sT + C::K_SLOTS * C::TILE), KT * 128, 1024);
      auto desc = [&](uint32_t lo) { return pack_u32x2(lo, k_hi); };  // (8-row groups of 1024 bytes in all of them)
      auto qk = [&](uint32_t buf, int qs, uint32_t slot) {  // S of a buffer = Q (slot qs) K^T
        const uint32_t a = q_lo + qs * (C::QT_BYTES >> 4), b = k_lo + slot * (C::TILE >> 4), d = tmem + 128 * buf;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          umma_bf16(d, desc(a + (((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4)),
                    desc(b + (((s >> 2) * (KT * 128) + (s & 3) * 32) >> 4)), id_qk, s > 0 ? 1u : 0u);
        umma_commit(&bar.s_full[buf]);
      };
      auto pv = [&](uint32_t buf, int h, uint32_t slot, bool first) {  // O of stream h (+)= P V
        const uint32_t b = v_lo + slot * (C::TILE >> 4), d = tmem + 128 * C::NB + D * h, a = tmem + 128 * buf;
#pragma unroll
        for (int s = 0; s < KT / 16; ++s)
          umma_bf16_ts(d, a + 8 * s, desc(b + ((s * 16 * 128) >> 4)), id_pv, s > 0 ? 1u : first ? 0u : 1u);
        umma_commit(&bar.o_done[buf]);
      };
      for (bool more_work = any_work; !failed && more_work; more_work = walk.next(p, block)) {
        const PagedWalk& w = walk.now();
        const Segment sg(p, w);
        const int end = w.s.L + w.s.n - w.k0 * KT;  // the sequence's end, from the segment's first key
        const int all = sg.products();
        const bool by_rows = sg.lag == 1;
        uint32_t ks = 0, vs = 0;  // slots of the K and V tiles in use
        auto score = [&](int u) {  // S of product u (elected lane)
          qk((made + u) % C::NB, by_rows ? u & 1 : 0, ks);
          if (!by_rows || (u & 1)) umma_commit(&bar.k_empty[ks]);
          if (u == all - 1) umma_commit(&bar.q_empty);
        };
        if (!mbar_wait_warp(&bar.q_full, seg & 1, err)) break;
        ++seg;
        for (int u = 0; u < min(C::NB, all) && !failed; ++u) {
          if (!by_rows || (u & 1) == 0) {
            failed = !mbar_wait_warp(&bar.k_full[kr.slot], kr.phase, err);
            ks = kr.slot;
            kr.next();
          }
          tc_fence_after();
          if (!failed && elect_one()) score(u);
          __syncwarp();
        }
        for (int u = 0; u < all && !failed; ++u) {
          const uint32_t g = made + u;
          const bool new_v = !by_rows || (u & 1) == 0, more = u + C::NB < all;
          const bool new_k = more && (!by_rows || ((u + C::NB) & 1) == 0);
          // what the product needs: its V, the K of the S behind it, its P (where a tile is there already: P's barrier again)
          uint64_t* const p_bar = &bar.p_full[g % C::NB];
          const uint32_t p_phase = (g / C::NB) & 1;
          uint64_t *v_bar = p_bar, *k_bar = p_bar;
          uint32_t v_phase = p_phase, k_phase = p_phase;
          if (new_v) {
            v_bar = &bar.v_full[vr.slot];
            v_phase = vr.phase;
            vs = vr.slot;
            vr.next();
          }
          if (new_k) {
            k_bar = &bar.k_full[kr.slot];
            k_phase = kr.phase;
            ks = kr.slot;
            kr.next();
          }
          const bool v = mbar_try_wait(v_bar, v_phase), k = mbar_try_wait(k_bar, k_phase), pp = mbar_try_wait(p_bar, p_phase);
          if (!__all_sync(0xffffffffu, v && k && pp))
            failed = !mbar_wait_warp(v_bar, v_phase, err) || !mbar_wait_warp(k_bar, k_phase, err) || !mbar_wait_warp(p_bar, p_phase, err);
          if (failed) break;
          if (new_v) {
            const int v_valid = end - (by_rows ? u >> 1 : u) * KT;
            if (v_valid < KT) {
              // values past the sequence's end are multiplied by weights of 0: they have to be finite
              uint8_t* t = sT + (C::K_SLOTS + vs) * C::TILE;
              for (int c = 0; c < DH; ++c)
                for (int i = max(0, v_valid) * 8 + lane; i < KT * 8; i += 32)
                  *reinterpret_cast<uint4*>(t + c * (KT * 128) + i * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async();
              __syncwarp();
            }
          }
          tc_fence_after();
          if (elect_one()) {
            pv(g % C::NB, u & 1, vs, u < 2);
            if (!by_rows || (u & 1)) umma_commit(&bar.v_empty[vs]);
            if (more) score(u + C::NB);
          }
          __syncwarp();
        }
        made += all;
      }
      if (elect_one()) {  // every MMA issued has completed before the tensor memory is released (bounded)
        umma_commit(&bar.drain);
        mbar_wait(&bar.drain, 0, err);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (warp == ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_t(const PagedParams& p, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap mapQ, mapK, mapV;
  const int box = 1 << std::min(p.s_bits, 7);
  if (!encode_token_map(&mapQ, p.q, D, p.GQ, p.H_kv, p.R, p.q_stride, 128) ||
      !encode_page_map(&mapK, p.K, D, 1 << p.s_bits, p.H_kv, p.P, box) ||
      !encode_page_map(&mapV, p.V, D, 1 << p.s_bits, p.H_kv, p.P, box))
    return cudaErrorInvalidValue;
  constexpr size_t smem = C::TILES + sizeof(Shared<D>);
  static_assert(smem <= 227 * 1024, "a block's shared memory");
  const cudaError_t e = allow_shared<paged_tc_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  paged_tc_kernel<D><<<p.blocks, THREADS, smem, s>>>(mapQ, mapK, mapV, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams& p, int d, cudaStream_t s) {
  return d == 128 ? launch_t<128>(p, s) : launch_t<64>(p, s);
}

}  // namespace pisa
