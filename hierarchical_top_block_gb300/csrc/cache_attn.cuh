// Attention of up to 16 query rows of one KV head over keys of a cache, by one warp: the part that the
// attention over selected blocks of the 8-bit cache and the attention over a shared prefix (few
// rows) have in common.
//
// Formulas, for query row i and key c with codes k8, v8 and row scales ks, vs (a bf16 cache: k, v
// themselves and scales 1):
//   z_ic = scale ks_c (q_i . k8_c),   p_ic = 2^(z_ic - n_i),   l_i = sum_c p_ic,   o_i = sum_c (p_ic vs_c) v8_c
// (z in log2 units): one pass over the keys.  n is a reference that the largest z (of codes: z + log2 vs, less
// WEIGHT_ROOM) passes by 2^8 at most: it is raised, and o and l multiplied by 2^(old - new), only when that
// has grown by more.
// The result is o_i / l_i, and n_i + log2 l_i the log-sum-exp, whatever n is.
//
// The products run on mma.sync (m16n8k16, fp32 sums) with the keys as rows and the query rows as the
// eight columns, so that a group of up to eight query heads wastes nothing:
//   S^T = K Q^T   (16 keys x 8 rows a product),   O^T += V^T P^T   (16 columns of V x 8 rows)
// P^T comes out of S^T by one 8 x 8 transposition of fp16 pairs a tile (movmatrix).
//
// With codes both operands are fp16: codes are whole numbers up to 127, exact there and two
// instructions a pair away (bf16 takes four, and its weights carry 8 bits); q is brought to at most
// 2 in magnitude by a power of two a row, so that it is exact but for elements below 2^-14 of the row's
// largest, which keep 2^-25 of it; and the weight with its value's scale, p vs, is rounded to fp16:
// 2^-11 of it, and 2^-32 of the row's largest one at least (codes.cuh).  A bf16 cache keeps bf16 operands, and
// its weights are rounded to bf16 (2^-8).  l sums the unrounded weights.
//
// A granule of 32 or 16 keys lies in shared memory as TMA wrote it, rows of 128 bytes (64 for codes of
// d = 64) in the swizzle of that width, first K, then V.
//   K: lane 4 r + q reads, of the keys r ^ 4 (r & 1) of each group of eight, the 16 bytes at 64 j + 16 q
//      (chunks of 64 bytes j).  The contraction index may be permuted if both operands are: Q is loaded
//      with the same order.
//   V: lane 4 r + q reads, of keys 16 kk + {2 q, (2 q + 1) ^ 4} and the same + 8, 16 (or 8) bytes at 16 r;
//      the two keys that the operand wants in one register are paired while the codes are widened, so
//      the transposition costs one permutation.
// The keys' order within a group of eight (odd ones four apart from their place) makes the eight
// lanes of a quarter-warp read eight different 16-byte columns in both.
#pragma once

#include "codes.cuh"

namespace pisa {

// Products without side effects (the compiler may order them among the loads that feed them).
__device__ __forceinline__ void product_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void product_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements, row r in lanes 4 r .. 4 r + 3, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// D: head dimension; BITS: 8 (codes) or 16 (bf16); KEYS a granule; NH: groups of eight query rows.
template <int D, int BITS, int KEYS, int NH>
struct CacheTile {
  static constexpr int MT = KEYS / 16;               // products of 16 keys
  static constexpr int G8 = KEYS / 8;                // groups of eight keys
  static constexpr int DT = D / 16;                  // products of 16 columns of V
  static constexpr int ROWB = D * BITS / 8;          // bytes a cache row
  static constexpr int SPAN = ROWB < 128 ? 64 : 128; // bytes a row in shared memory (a swizzle's width)
  static constexpr int PIECES = ROWB / SPAN;         // such pieces a row: boxes of a copy
  static constexpr uint32_t SIDE = KEYS * ROWB;      // K or V of a granule
  static constexpr uint32_t BYTES = 2 * SIDE;
  static constexpr int KCH = ROWB / 64;              // 16-byte pieces of a K row a lane holds
  static constexpr int VW = ROWB / 32;               // words of a V row a lane holds
  static constexpr int QW = D / 8;                   // words of a Q row a lane holds
  static constexpr int ROWS = 8 * NH;

  // The d that row r (up = 0) or r + 8 (up = 1) of column product t stands for.
  __device__ static __forceinline__ int column(int t, int up, int r) {
    if constexpr (BITS == 8) return (D / 8) * r + 2 * t + up;
    return 64 * (t >> 2) + 8 * r + 2 * (t & 3) + up;
  }
  // The key of row n of a group of eight.
  __device__ static __forceinline__ int key_of(int n) { return n ^ ((n & 1) << 2); }
  // Shared-memory offset of 16-byte column c of a granule's row.
  __device__ static __forceinline__ uint32_t at(int row, int c) {
    if constexpr (SPAN == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return (c >> 3) * (KEYS * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  }

  // Issues the copies of keys key0 .. of head `bh` to `dst` (one thread; maps with boxes of KEYS rows).
  __device__ static __forceinline__ void copy(uint8_t* dst, const CUtensorMap* mapK, const CUtensorMap* mapV,
                                              uint64_t* bar, int key0, int bh) {
    mbar_arrive_expect_tx(bar, BYTES);
    constexpr int STEP = BITS == 8 ? SPAN : SPAN / 2;  // elements a piece
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      tma_load_3d(dst + c * (KEYS * SPAN), mapK, bar, STEP * c, key0, bh);
      tma_load_3d(dst + SIDE + c * (KEYS * SPAN), mapV, bar, STEP * c, key0, bh);
    }
  }

  struct Query {
    uint32_t w[NH][QW];   // query row 8 h + r, in K's order
    float s[NH][2];       // logit factors (log2 units, the rows' powers of two with them) of rows 8 h + 2 q + {0, 1}
  };
  // row(i): where query row i starts, null where there is none.
  template <typename Row>
  __device__ static __forceinline__ void load_q(Query& x, Row row_at, float sl2, int r, int q) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const uint16_t* row = row_at(8 * h + r);
      uint32_t top = 1;  // largest exponent field of the row
#pragma unroll
      for (int j = 0; j < QW / 4; ++j) {
        // codes: 16 values at 64 (j / 2) + 16 q (two pieces); bf16: 8 values at 32 j + 8 q
        const int c = BITS == 8 ? 64 * (j >> 1) + 16 * q + 8 * (j & 1) : 32 * j + 8 * q;
        const uint4 v = row ? ldg16(row + c) : make_uint4(0, 0, 0, 0);
        x.w[h][4 * j] = v.x;
        x.w[h][4 * j + 1] = v.y;
        x.w[h][4 * j + 2] = v.z;
        x.w[h][4 * j + 3] = v.w;
      }
      x.s[h][0] = x.s[h][1] = sl2;
      if constexpr (BITS == 8) {
#pragma unroll
        for (int j = 0; j < QW; ++j) top = max(top, max((x.w[h][j] >> 7) & 0xffu, (x.w[h][j] >> 23) & 0xffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = min(top, 253u);                                        // (infinities stay so)
        const float down = __uint_as_float((254u - top) << 23);      // 2^(127 - top)
#pragma unroll
        for (int j = 0; j < QW; ++j) x.w[h][j] = pack_f16x2(bf16_lo(x.w[h][j]) * down, bf16_hi(x.w[h][j]) * down);
        const float f = sl2 * __uint_as_float(top << 23);            // sl2 2^(top - 127), of row r
        x.s[h][0] = __shfl_sync(0xffffffffu, f, 4 * (2 * q));
        x.s[h][1] = __shfl_sync(0xffffffffu, f, 4 * (2 * q + 1));
      }
    }
  }

  // A lane's scales of a granule: of its key in each group of eight.
  struct Scales {
    float k[BITS == 8 ? G8 : 1], v[BITS == 8 ? G8 : 1];
  };
  __device__ static __forceinline__ void load_scales(Scales& s, const float* ks, const float* vs, long long key0, int n,
                                                     int r) {
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < G8; ++i) {
        const int c = 8 * i + key_of(r);
        s.k[i] = c < n ? __ldg(ks + key0 + c) : 0.f;
        s.v[i] = c < n ? __ldg(vs + key0 + c) : 0.f;
      }
    }
  }

  // The running state of rows 8 h + 2 q + {0, 1}; l (the two rows') is a lane's share of the sum until
  // the end.  o[t][h]: columns (t, 0) of the two rows, then columns (t, 1).
  struct State {
    float n[NH][2];
    unsigned long long l[NH];
    float o[DT][NH][4];
  };
  __device__ static __forceinline__ void clear(State& s) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      s.n[h][0] = s.n[h][1] = NEG_INF;
      s.l[h] = pack_f32x2(0.f, 0.f);
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int h = 0; h < NH; ++h) s.o[t][h][0] = s.o[t][h][1] = s.o[t][h][2] = s.o[t][h][3] = 0.f;
  }
  // The largest over a column's lanes (those of equal q).
  __device__ static __forceinline__ float column_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
  }

  // Adds the first `n` keys of the granule at `g` in shared memory.
  __device__ static __forceinline__ void add(State& st, const uint8_t* g, const Scales& sc, const Query& qr, int n, int r,
                                             int q) {
    float s[MT][NH][4];  // keys of groups 2 i (elements 0, 1: rows 2 q, 2 q + 1) and 2 i + 1 (2, 3)
    const int krow = key_of(r);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < NH; ++h) s[i][h][0] = s[i][h][1] = s[i][h][2] = s[i][h][3] = 0.f;
#pragma unroll
    for (int j = 0; j < KCH; ++j) {
      uint4 x[G8];
#pragma unroll
      for (int i = 0; i < G8; ++i) x[i] = *reinterpret_cast<const uint4*>(g + at(8 * i + krow, 4 * j + q));
      // the sums of the key tiles in turn: each waits for its product before
#pragma unroll
      for (int e = 0; e < (BITS == 8 ? 4 : 2); ++e)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if constexpr (BITS == 8) {
            auto word = [&](const uint4& v) { return (e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w) ^ 0x80808080u; };
            const uint32_t u0 = word(x[2 * i]), u1 = word(x[2 * i + 1]);
            const uint32_t a0 = widen_f16<0x4140>(u0), a1 = widen_f16<0x4140>(u1), a2 = widen_f16<0x4342>(u0),
                           a3 = widen_f16<0x4342>(u1);
#pragma unroll
            for (int h = 0; h < NH; ++h) product_f16(s[i][h], a0, a1, a2, a3, qr.w[h][8 * j + 2 * e], qr.w[h][8 * j + 2 * e + 1]);
          } else {
            const uint4 u0 = x[2 * i], u1 = x[2 * i + 1];
#pragma unroll
            for (int h = 0; h < NH; ++h)
              product_bf16(s[i][h], e ? u0.z : u0.x, e ? u1.z : u1.x, e ? u0.w : u0.y, e ? u1.w : u1.y,
                           qr.w[h][4 * j + 2 * e], qr.w[h][4 * j + 2 * e + 1]);
          }
        }
    }
    // logits, and the maximum of them with the values' scales
    float lv[BITS == 8 ? G8 : 1];
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < G8; ++i) lv[i] = scale_log2(sc.v[i]);
    }
    bool moved = false;
    float top[NH][2];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const unsigned long long f = pack_f32x2(qr.s[h][0], qr.s[h][1]);
      float x0 = NEG_INF, x1 = NEG_INF;
#pragma unroll
      for (int i = 0; i < G8; ++i) {
        float* z = &s[i >> 1][h][2 * (i & 1)];
        unsigned long long y = mul_f32x2(pack_f32x2(z[0], z[1]), BITS == 8 ? mul_f32x2(f, pack_f32x2(sc.k[i], sc.k[i])) : f);
        unpack_f32x2(y, z[0], z[1]);
        if (8 * i + krow >= n) z[0] = z[1] = NEG_INF;
        float a = z[0], b = z[1];
        if constexpr (BITS == 8) {
          a += lv[i];
          b += lv[i];
        }
        x0 = fmaxf(x0, a);
        x1 = fmaxf(x1, b);
      }
      top[h][0] = column_max(x0);
      top[h][1] = column_max(x1);
      moved = moved || top[h][0] > st.n[h][0] + 8.f || top[h][1] > st.n[h][1] + 8.f;
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float f[2], l[2];
        unpack_f32x2(st.l[h], l[0], l[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float to = fmaxf(st.n[h][e], top[h][e]), by = to == NEG_INF ? 0.f : st.n[h][e] - to;
          f[e] = fast_exp2(by);  // 0 before the first keys
          // (n covers the values' scales too: where those rise by far, l is large and may keep what f does not)
          l[e] = times_exp2(l[e], by);
          st.n[h][e] = to;
        }
        st.l[h] = pack_f32x2(l[0], l[1]);
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          st.o[t][h][0] *= f[0];
          st.o[t][h][1] *= f[1];
          st.o[t][h][2] *= f[0];
          st.o[t][h][3] *= f[1];
        }
      }
    }
    uint32_t pt[MT][NH][2];  // P^T: rows 8 h + r, keys 2 q, 2 q + 1 of groups 2 i and 2 i + 1
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      // a row that has seen no key (or only logits of -inf) has n = -inf: its weights are 0
      const unsigned long long ref = pack_f32x2(st.n[h][0] == NEG_INF ? 0.f : -st.n[h][0], st.n[h][1] == NEG_INF ? 0.f : -st.n[h][1]);
#pragma unroll
      for (int i = 0; i < G8; ++i) {
        const float* z = &s[i >> 1][h][2 * (i & 1)];
        float a, b;
        unpack_f32x2(add_f32x2(pack_f32x2(z[0], z[1]), ref), a, b);
        a = fast_exp2(a);
        b = fast_exp2(b);
        unsigned long long ab = pack_f32x2(a, b);
        st.l[h] = add_f32x2(st.l[h], ab);
        if constexpr (BITS == 8) {  // a masked key's scale reads as 0
          unpack_f32x2(mul_f32x2(ab, pack_f32x2(sc.v[i], sc.v[i])), a, b);
          pt[i >> 1][h][i & 1] = transpose8(pack_f16x2(a, b));
        } else {
          pt[i >> 1][h][i & 1] = transpose8(pack_bf16x2(a, b));
        }
      }
    }
    const uint8_t* gv = g + SIDE;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      uint32_t v[4][VW];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = 16 * i + 8 * (u >> 1) + key_of(2 * q + (u & 1));
        if constexpr (VW == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(gv + at(row, r >> 1) + 8 * (r & 1));
          v[u][0] = x.x;
          v[u][1] = x.y;
        } else {
#pragma unroll
          for (int j = 0; j < VW / 4; ++j) {
            const uint4 x = *reinterpret_cast<const uint4*>(gv + at(row, 8 * j + r));
            v[u][4 * j] = x.x;
            v[u][4 * j + 1] = x.y;
            v[u][4 * j + 2] = x.z;
            v[u][4 * j + 3] = x.w;
          }
        }
        if constexpr (BITS == 16) {
          if (row >= n) {  // a weight of 0 times whatever lies there
#pragma unroll
            for (int j = 0; j < VW; ++j) v[u][j] = 0;
          }
        }
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        if constexpr (BITS == 8) {  // four columns: bytes of two keys interleaved, then widened
          const uint32_t x0 = v[0][w] ^ 0x80808080u, x1 = v[1][w] ^ 0x80808080u;
          const uint32_t x2 = v[2][w] ^ 0x80808080u, x3 = v[3][w] ^ 0x80808080u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t a = __byte_perm(x0, x1, e ? 0x7362 : 0x5140), b = __byte_perm(x2, x3, e ? 0x7362 : 0x5140);
            const uint32_t a0 = widen_f16<0x4140>(a), a1 = widen_f16<0x4342>(a), a2 = widen_f16<0x4140>(b),
                           a3 = widen_f16<0x4342>(b);
#pragma unroll
            for (int h = 0; h < NH; ++h) product_f16(st.o[2 * w + e][h], a0, a1, a2, a3, pt[i][h][0], pt[i][h][1]);
          }
        } else {
          const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410), a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
          const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410), a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
          for (int h = 0; h < NH; ++h) product_bf16(st.o[w][h], a0, a1, a2, a3, pt[i][h][0], pt[i][h][1]);
        }
      }
    }
  }
};

// One warp's granules: a ring of SLOTS in shared memory that the warp fills (lane 0, TMA) and empties
// itself.  Granule s is in slot s mod SLOTS; phases are waited for in order.
template <typename Tile, int SLOTS>
struct WarpRing {
  uint8_t* mem;
  uint64_t* full;  // [SLOTS], initialised with one arrival
  __device__ __forceinline__ void fetch(uint32_t s, const CUtensorMap* mapK, const CUtensorMap* mapV, int key0, int bh,
                                        int lane) {
    if (lane == 0) Tile::copy(mem + (s % SLOTS) * Tile::BYTES, mapK, mapV, &full[s % SLOTS], key0, bh);
  }
  __device__ __forceinline__ bool wait(uint32_t s, uint32_t* err, uint64_t limit = WAIT_LIMIT_NS) {
    return mbar_wait_warp(&full[s % SLOTS], (s / SLOTS) & 1, err, limit);
  }
  __device__ __forceinline__ const uint8_t* at(uint32_t s) const { return mem + (s % SLOTS) * Tile::BYTES; }
};

// Joins the states of a block's four warps into shared memory.  po [4][ROWS][D] and sn, sl [4][16] are
// scratch; afterwards ml holds each row's reference and sum and po its output sums (`rows` rows are in
// use).  All 128 threads.
template <typename Tile, int D>
__device__ __forceinline__ void join_warps(typename Tile::State& st, float* po, float (*sn)[16], float (*sl)[16],
                                           float2* ml, int rows) {
  constexpr int ROWS = Tile::ROWS, NH = ROWS / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    float l[2];
    unpack_f32x2(st.l[h], l[0], l[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
      if (r == 0) {
        sn[warp][8 * h + 2 * q + e] = st.n[h][e];
        sl[warp][8 * h + 2 * q + e] = l[e];
      }
    }
  }
  __syncthreads();  // (and every warp is done with its granules: po may lie over them)
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * h + 2 * q + e;
      float n = NEG_INF, l = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) n = fmaxf(n, sn[k][row]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // without a reference a sum is 0, or NaN where every logit was
        const float a = sn[k][row], b = sl[k][row];
        l += a == NEG_INF ? b : times_exp2(b, a - n);
      }
      if (warp == 0 && r == 0 && row < rows) ml[row] = make_float2(n, l);
      const float f = st.n[h][e] == NEG_INF ? 0.f : fast_exp2(st.n[h][e] - n);
      if (row < rows) {
        float* dst = po + ((size_t)warp * ROWS + row) * D;
#pragma unroll
        for (int t = 0; t < Tile::DT; ++t) {
          const float a = f == 0.f ? 0.f : st.o[t][h][e] * f, b = f == 0.f ? 0.f : st.o[t][h][2 + e] * f;
          *reinterpret_cast<float2*>(dst + Tile::column(t, 0, r)) = make_float2(a, b);
        }
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D; i += 128)
    po[i] = (po[i] + po[i + ROWS * D]) + (po[i + 2 * ROWS * D] + po[i + 3 * ROWS * D]);
  __syncthreads();
}

}  // namespace pisa
