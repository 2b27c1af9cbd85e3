// Attention of 16 query rows of one KV head over keys of a cache, by one warp: the part that the
// attention over selected blocks of the 8-bit cache and the attention over a shared prefix (few
// rows) have in common.
//
// Formulas, for query row i and key c with codes k8, v8 and row scales ks, vs (a bf16 cache: k, v
// themselves and scales 1):
//   z_ic = scale ks_c (q_i . k8_c),   l_i = sum_c 2^(z_ic - m_i),   o_i = sum_c 2^(z_ic + log2 vs_c - n_i) v8_c
// (z in log2 units), m and n the running maxima of the two exponents: one pass over the keys.  The
// result is o_i 2^(n_i - m_i) / l_i.
//
// The products run on mma.sync (m16n8k16, fp32 sums).  With codes both operands are fp16: codes are
// whole numbers up to 127, exact there and two instructions a pair away (bf16 takes four, and its
// weights carry 8 bits); q is brought to at most 2 in magnitude by a power of two a row, so that it
// is exact but for elements below 2^-14 of the row's largest, which keep 2^-25 of it; and the weight
// with its value's scale, at most 1, is rounded to fp16: 2^-11 of the weight, and 2^-25 of the row's
// largest one at least.  A bf16 cache keeps bf16 operands, and its weights are rounded to bf16 (2^-8).
// l sums the unrounded weights.
//
// A granule of 32 keys of codes (16 of bf16) lies in shared memory as TMA wrote it, rows of 128
// bytes (64 for codes of d = 64) in the swizzle of that width, first K, then V.
//   K: lane 4 r + q reads, of key 8 nt + r ^ 4 (r & 1), the 16 bytes at 64 j + 16 q (chunks of 64 bytes
//      j).  The contraction index may be permuted if both operands are: Q is loaded with the same order.
//   V: lane 4 r + q reads, of keys 16 kk + {2 q, (2 q + 1) ^ 4} and the same + 8, 16 (or 8) bytes at 16 r;
//      the two keys that the B operand wants in one register are paired while the codes are widened,
//      so the transposition costs one permutation.  n-tile i of the output holds column i of every
//      lane's bytes.
// The keys' order within a group of eight (odd ones four apart from their place) makes the eight
// lanes of a quarter-warp read eight different 16-byte columns in both.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace pisa {

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Codes with their top bit flipped (code + 128) in two bytes of x -> fp16x2: 0x6400 | u is 1024 + u.
template <int SEL>
__device__ __forceinline__ uint32_t widen_f16(uint32_t x) {
  const uint32_t y = __byte_perm(x, 0x64646464u, SEL);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x64806480u));  // 1152
  return r;
}

template <int D, int BITS>
struct CacheTile {
  static constexpr int KEYS = BITS == 8 ? 32 : 16;   // keys a granule
  static constexpr int NT = KEYS / 8, KK = KEYS / 16, NDT = D / 8;
  static constexpr int ROWB = D * BITS / 8;          // bytes a cache row
  static constexpr int SPAN = ROWB < 128 ? 64 : 128; // bytes a row in shared memory (a swizzle's width)
  static constexpr int PIECES = ROWB / SPAN;         // such pieces a row: boxes of a copy
  static constexpr uint32_t SIDE = KEYS * ROWB;      // K or V of a granule
  static constexpr uint32_t BYTES = 2 * SIDE;
  static constexpr int KCH = ROWB / 64;              // 16-byte pieces of a K row a lane holds
  static constexpr int VW = ROWB / 32;               // words of a V row a lane holds
  static constexpr int QW = D / 8;                   // words of a Q row a lane holds

  // The MMA's n index (column of a lane's output pair) of n-tile i stands for this d.
  __device__ static __forceinline__ int column(int i, int n) {
    if constexpr (BITS == 8) return (D / 8) * n + i;
    return 64 * (i >> 3) + 8 * n + (i & 7);
  }
  // The key of column n of a group of eight.
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
    uint32_t a[QW], b[QW];  // rows r and r + 8, in K's order
    float s[2];             // logit factors, log2 units (the rows' powers of two with them)
  };
  // One lane's part of query rows r (`ra`) and r + 8 (`rb`); absent rows: null.
  template <bool HI>
  __device__ static __forceinline__ void load_q(Query& x, const uint16_t* ra, const uint16_t* rb, float sl2, int q) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t(&w)[QW] = h ? x.b : x.a;
      const uint16_t* row = h ? rb : ra;
      x.s[h] = sl2;
      if (h == 1 && !HI) {
#pragma unroll
        for (int j = 0; j < QW; ++j) w[j] = 0;
        continue;
      }
      uint32_t top = 0;  // largest exponent field of the row
#pragma unroll
      for (int j = 0; j < QW / 4; ++j) {
        // codes: 16 values at 64 (j / 2) + 16 q (two pieces); bf16: 8 values at 32 j + 8 q
        const int c = BITS == 8 ? 64 * (j >> 1) + 16 * q + 8 * (j & 1) : 32 * j + 8 * q;
        const uint4 v = row ? ldg16(row + c) : make_uint4(0, 0, 0, 0);
        w[4 * j] = v.x;
        w[4 * j + 1] = v.y;
        w[4 * j + 2] = v.z;
        w[4 * j + 3] = v.w;
        if constexpr (BITS == 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max((w[4 * j + e] >> 7) & 0xffu, (w[4 * j + e] >> 23) & 0xffu));
        }
      }
      if constexpr (BITS == 8) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = min(max(top, 1u), 253u);                               // (infinities stay so)
        const float down = __uint_as_float((254u - top) << 23);      // 2^(127 - top)
        x.s[h] = sl2 * __uint_as_float(top << 23);                   // sl2 2^(top - 127)
#pragma unroll
        for (int j = 0; j < QW; ++j) w[j] = pack_f16x2(bf16_lo(w[j]) * down, bf16_hi(w[j]) * down);
      }
    }
  }

  // A lane's scales of a granule: of the keys of its accumulator columns.
  struct Scales {
    float k[BITS == 8 ? 2 * NT : 1], v[BITS == 8 ? 2 * NT : 1];
  };
  __device__ static __forceinline__ void load_scales(Scales& s, const float* ks, const float* vs, long long key0, int n,
                                                     int q) {
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        const int c = 8 * (i >> 1) + key_of(2 * q + (i & 1));
        s.k[i] = c < n ? __ldg(ks + key0 + c) : 0.f;
        s.v[i] = c < n ? __ldg(vs + key0 + c) : 0.f;
      }
    }
  }

  // The running state of 16 rows (row r in element 0 and o[.][0..1], row r + 8 in the others); l is a
  // lane's share of the sum until the end.
  struct State {
    float m[2], n[2], l[2];
    float o[NDT][4];
  };
  __device__ static __forceinline__ void clear(State& s) {
    s.m[0] = s.m[1] = s.n[0] = s.n[1] = NEG_INF;
    s.l[0] = s.l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < NDT; ++i) s.o[i][0] = s.o[i][1] = s.o[i][2] = s.o[i][3] = 0.f;
  }

  // Adds the first `n` keys of the granule at shared-memory address `g`.  HI: rows 8 .. 15 are in use.
  template <bool HI>
  __device__ static __forceinline__ void add(State& st, uint32_t g, const Scales& sc, const Query& qr, int n, int r,
                                             int q) {
    float s[NT][4];
    const int krow = key_of(r);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KCH; ++j) {
        const uint4 x = lds16(g + at(8 * nt + krow, 4 * j + q));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if constexpr (BITS == 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int a = 8 * j + 2 * e;
            const uint32_t u = w[e] ^ 0x80808080u;
            mma_f16_16816(s[nt], qr.a[a], HI ? qr.b[a] : 0u, qr.a[a + 1], HI ? qr.b[a + 1] : 0u, widen_f16<0x4140>(u),
                          widen_f16<0x4342>(u));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int a = 4 * j + 2 * e;
            mma_bf16_16816(s[nt], qr.a[a], HI ? qr.b[a] : 0u, qr.a[a + 1], HI ? qr.b[a + 1] : 0u, w[2 * e], w[2 * e + 1]);
          }
        }
      }
    }
    // logits, and the maxima of z and of z + log2 vs
    float lv[BITS == 8 ? 2 * NT : 1];
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) lv[i] = fast_log2(sc.v[i]);  // a masked key's scale reads as 0: -inf
    }
    float mx[2] = {NEG_INF, NEG_INF}, nx[2] = {NEG_INF, NEG_INF};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool in = 8 * nt + key_of(2 * q + c) < n;
#pragma unroll
        for (int h = 0; h < (HI ? 2 : 1); ++h) {
          float& z = s[nt][2 * h + c];
          z = in ? z * (BITS == 8 ? sc.k[2 * nt + c] * qr.s[h] : qr.s[h]) : NEG_INF;
          mx[h] = fmaxf(mx[h], z);
          if constexpr (BITS == 8) nx[h] = fmaxf(nx[h], z + lv[2 * nt + c]);
        }
      }
    bool moved = false;
    float cf[2] = {1.f, 1.f};
#pragma unroll
    for (int h = 0; h < (HI ? 2 : 1); ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      if constexpr (BITS == 8) {
        nx[h] = fmaxf(nx[h], __shfl_xor_sync(0xffffffffu, nx[h], 1));
        nx[h] = fmaxf(nx[h], __shfl_xor_sync(0xffffffffu, nx[h], 2));
      } else {
        nx[h] = mx[h];
      }
      if (mx[h] > st.m[h]) {
        st.l[h] *= fast_exp2(st.m[h] - mx[h]);  // 0 before the first keys
        st.m[h] = mx[h];
      }
      if (nx[h] > st.n[h]) {
        cf[h] = fast_exp2(st.n[h] - nx[h]);
        st.n[h] = nx[h];
        moved = true;
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < NDT; ++i) {
        st.o[i][0] *= cf[0];
        st.o[i][1] *= cf[0];
        if (HI) {
          st.o[i][2] *= cf[1];
          st.o[i][3] *= cf[1];
        }
      }
    }
    uint32_t pa[KK][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !HI) {
          pa[nt >> 1][2 * (nt & 1) + 1] = 0u;
          continue;
        }
        // a row that has seen no key (or only logits of -inf) has m = -inf: its weights are 0
        const float rm = st.m[h] == NEG_INF ? 0.f : st.m[h];
        const float p0 = fast_exp2(s[nt][2 * h] - rm), p1 = fast_exp2(s[nt][2 * h + 1] - rm);
        st.l[h] += p0 + p1;
        if constexpr (BITS == 8) {
          const float rn = st.n[h] == NEG_INF ? 0.f : st.n[h];
          pa[nt >> 1][2 * (nt & 1) + h] =
              pack_f16x2(fast_exp2(s[nt][2 * h] + lv[2 * nt] - rn), fast_exp2(s[nt][2 * h + 1] + lv[2 * nt + 1] - rn));
        } else {
          pa[nt >> 1][2 * (nt & 1) + h] = pack_bf16x2(p0, p1);
        }
      }
    }
    const uint32_t gv = g + SIDE;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t v[4][VW];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = 16 * kk + 8 * (u >> 1) + key_of(2 * q + (u & 1));
        if constexpr (VW == 2) {
          const uint2 x = lds8(gv + at(row, r >> 1) + 8 * (r & 1));
          v[u][0] = x.x;
          v[u][1] = x.y;
        } else {
#pragma unroll
          for (int j = 0; j < VW / 4; ++j) {
            const uint4 x = lds16(gv + at(row, 8 * j + r));
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
      if constexpr (BITS == 8) {
#pragma unroll
        for (int w = 0; w < VW; ++w) {  // four columns: bytes of two keys interleaved, then widened
          const uint32_t x0 = v[0][w] ^ 0x80808080u, x1 = v[1][w] ^ 0x80808080u;
          const uint32_t x2 = v[2][w] ^ 0x80808080u, x3 = v[3][w] ^ 0x80808080u;
          const uint32_t a01 = __byte_perm(x0, x1, 0x5140), a23 = __byte_perm(x0, x1, 0x7362);
          const uint32_t b01 = __byte_perm(x2, x3, 0x5140), b23 = __byte_perm(x2, x3, 0x7362);
          mma_f16_16816(st.o[4 * w], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], widen_f16<0x4140>(a01), widen_f16<0x4140>(b01));
          mma_f16_16816(st.o[4 * w + 1], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], widen_f16<0x4342>(a01), widen_f16<0x4342>(b01));
          mma_f16_16816(st.o[4 * w + 2], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], widen_f16<0x4140>(a23), widen_f16<0x4140>(b23));
          mma_f16_16816(st.o[4 * w + 3], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], widen_f16<0x4342>(a23), widen_f16<0x4342>(b23));
        }
      } else {
#pragma unroll
        for (int i = 0; i < NDT; ++i) {
          const int w = (i >> 3) * 4 + ((i & 7) >> 1);
          const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
          mma_bf16_16816(st.o[i], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], __byte_perm(v[0][w], v[1][w], sel),
                         __byte_perm(v[2][w], v[3][w], sel));
        }
      }
    }
  }
};

// A ring of granules between the warp that copies (TMA) and the four that compute.  Granule s of the
// block's whole sequence is taken by the warps of key part s mod PARTS, 4 / PARTS of them (one a row
// tile).  The slots are a multiple of the parts, so a slot's granules all go to the same warps, and
// each of them waits for every phase of the slot in turn (a parity says nothing to a waiter that is two
// phases off: copies may land out of order).
template <int D, int BITS>
struct GranuleRing {
  static constexpr int SLOTS = D == 128 ? 8 : 16;
  static_assert(SLOTS % 4 == 0, "");
  uint64_t full[SLOTS], empty[SLOTS];
  __device__ __forceinline__ void init(int takers) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], takers);
    }
    mbar_fence_init();
  }
};

// Joins the states of the warps that share rows into shared memory.  Warp w holds row tile w mod RT
// for key part w / RT.  po [4][16][D] and st [4][16] (m, l) are scratch; afterwards ml holds each row's
// maximum and sum and po its output sums relative to that maximum, rows of the tiles in order (the
// tiles' first `rows` rows are in use).  All 128 threads of the computing warps; `sync` is their barrier.
template <int D, int BITS, bool HI, int RT, typename Sync>
__device__ __forceinline__ void join_warps(typename CacheTile<D, BITS>::State& st, float* po, float (*sm)[16],
                                           float (*sn)[16], float (*sl)[16], float2* ml, int rows, Sync sync) {
  using T = CacheTile<D, BITS>;
  constexpr int PARTS = 4 / RT;
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3, rt = warp % RT;
#pragma unroll
  for (int h = 0; h < (HI ? 2 : 1); ++h) {
    st.l[h] += __shfl_xor_sync(0xffffffffu, st.l[h], 1);
    st.l[h] += __shfl_xor_sync(0xffffffffu, st.l[h], 2);
    if (q == 0) {
      sm[warp][r + 8 * h] = st.m[h];
      sn[warp][r + 8 * h] = st.n[h];
      sl[warp][r + 8 * h] = st.l[h];
    }
  }
  sync();
#pragma unroll
  for (int h = 0; h < (HI ? 2 : 1); ++h) {
    const int row = r + 8 * h;
    float m = NEG_INF, l = 0.f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) m = fmaxf(m, sm[rt + RT * k][row]);
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {  // without a maximum a sum is 0, or NaN where every logit was
      const float a = sm[rt + RT * k][row], b = sl[rt + RT * k][row];
      l += a == NEG_INF ? b : b * fast_exp2(a - m);
    }
    if (warp < RT && q == 0 && 16 * rt + row < rows) ml[16 * rt + row] = make_float2(m, l);
    const float f = st.n[h] == NEG_INF ? 0.f : fast_exp2(st.n[h] - m);
    if (16 * rt + row < rows) {
#pragma unroll
      for (int i = 0; i < T::NDT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          po[((size_t)warp * 16 + row) * D + T::column(i, 2 * q + c)] = f == 0.f ? 0.f : st.o[i][2 * h + c] * f;
    }
  }
  sync();
  if (PARTS > 1) {
    for (int i = threadIdx.x & 127; i < rows * D; i += 128) {
      float a = po[i];
#pragma unroll
      for (int k = 1; k < PARTS; ++k) a += po[i + k * RT * 16 * D];
      po[i] = a;
    }
    sync();
  }
}

}  // namespace pisa
