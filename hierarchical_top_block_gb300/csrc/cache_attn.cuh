// Attention of up to 16 query rows of one KV head over keys of a cache, by one warp: the part
// that the attention over selected blocks of the 8-bit cache and the attention over a shared
// prefix (few rows) have in common.
//
// Formulas, for query row i and key c with codes k8, v8 and row scales ks, vs (a bf16 cache: k, v
// themselves and scales 1):
//   z_ic = scale ks_c (q_i . k8_c),  o_i = sum_c e^(z_ic - m_i) vs_c v8_c,  l_i = sum_c e^(z_ic - m_i)
// with the running maximum m_i, so one pass over the keys does.  Codes are whole numbers up to
// 127, exact in bf16, so the products run on mma.sync (m16n8k16, fp32 sums) with the raw codes;
// ks multiplies the fp32 logit and vs the fp32 weight.  The weight is rounded to bf16 for the
// second product (half a step, 2^-8 of each weight, as large as the rounding of the bf16 output);
// l sums the unrounded weights.
//
// Every byte of the cache is used once, so nothing is staged in shared memory: a warp loads a
// granule (8 KB at d = 128: 32 keys of codes, 16 of bf16) straight into the registers that the
// MMA wants.
//   K: lane 4 r + q holds, of key 8 nt + r, the 16 bytes at 64 j + 16 q (chunks of 64 bytes j).  The
//      contraction index may be permuted if both operands are: Q is loaded with the same order.
//   V: lane 4 r + q holds, of keys 16 kk + 2 q + {0, 1, 8, 9}, 16 (or 8) bytes at 16 r; the two keys
//      that the B operand wants in one register are paired while the codes are widened, so the
//      transposition costs nothing.  n-tile i of the output holds column i of every lane's bytes.
#pragma once

#include "common.cuh"

namespace pisa {

// Two int8 codes in bytes 0 and 2 of y (bytes 1 and 3: anything) -> bf16x2.  A code is m - 128 s
// (s its top bit, m the seven below): (128 + m) - 128 (1 + s), both exact bf16 numbers whose
// bits are 0x4300 | m and 0x4300 | (code & 0x80).
__device__ __forceinline__ uint32_t widen_codes(uint32_t y) {
  const uint32_t a = (y & 0x007f007fu) | 0x43004300u, c = (y & 0x00800080u) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(c));
  return r;
}

template <int D, int BITS>
struct CacheTile {
  static constexpr int KEYS = BITS == 8 ? 32 : 16;  // keys a granule
  static constexpr int NT = KEYS / 8, KK = KEYS / 16, NDT = D / 8;
  static constexpr int ROWB = D * BITS / 8;     // bytes a cache row
  static constexpr int KCH = ROWB / 64;         // 16-byte pieces of a K row a lane holds
  static constexpr int VW = ROWB / 32;          // words of a V row a lane holds
  static constexpr int QW = D / 8;              // words of a Q row a lane holds

  // The MMA's n index (column of a lane's output pair) of n-tile i stands for this d.
  __device__ static __forceinline__ int column(int i, int n) {
    if constexpr (BITS == 8) return (D / 8) * n + i;
    return 64 * (i >> 3) + 8 * n + (i & 7);
  }

  // One lane's part of a query row, in K's order; zeros for an absent row.
  __device__ static __forceinline__ void load_q(const uint16_t* row, bool in, int q, uint32_t (&w)[QW]) {
#pragma unroll
    for (int j = 0; j < QW / 4; ++j) {
      // codes: 16 values at 64 (j / 2) + 16 q (two pieces); bf16: 8 values at 32 j + 8 q
      const int at = BITS == 8 ? 64 * (j >> 1) + 16 * q + 8 * (j & 1) : 32 * j + 8 * q;
      const uint4 x = in ? ldg16(row + at) : make_uint4(0, 0, 0, 0);
      w[4 * j] = x.x;
      w[4 * j + 1] = x.y;
      w[4 * j + 2] = x.z;
      w[4 * j + 3] = x.w;
    }
  }

  struct Regs {
    uint4 k[NT * KCH];
    uint32_t v[KK * 4 * VW];
    float ks[2 * NT], vs[2 * NT];
  };

  // Loads keys key0 .. key0 + n - 1 (n <= KEYS) of one head's rows; later keys read as the first
  // one (K) and as zero (V): they are masked, and their bytes are not touched.
  __device__ static __forceinline__ void load(Regs& g, const uint8_t* K, const uint8_t* V, const float* ks,
                                              const float* vs, long long key0, int n, int r, int q) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const long long key = key0 + (8 * nt + r < n ? 8 * nt + r : 0);
#pragma unroll
      for (int j = 0; j < KCH; ++j) g.k[nt * KCH + j] = ldg16(K + key * ROWB + 64 * j + 16 * q);
    }
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = 16 * kk + 2 * q + (u & 1) + 8 * (u >> 1);
        const uint8_t* row = V + (key0 + i) * ROWB;
        uint32_t* dst = g.v + (kk * 4 + u) * VW;
        if constexpr (VW == 2) {
          const uint2 x = i < n ? __ldg(reinterpret_cast<const uint2*>(row + 8 * r)) : make_uint2(0, 0);
          dst[0] = x.x;
          dst[1] = x.y;
        } else {
#pragma unroll
          for (int j = 0; j < VW / 4; ++j) {
            const uint4 x = i < n ? ldg16(row + 128 * j + 16 * r) : make_uint4(0, 0, 0, 0);
            dst[4 * j] = x.x;
            dst[4 * j + 1] = x.y;
            dst[4 * j + 2] = x.z;
            dst[4 * j + 3] = x.w;
          }
        }
      }
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        const int c = 8 * (i >> 1) + 2 * q + (i & 1);
        g.ks[i] = c < n ? __ldg(ks + key0 + c) : 0.f;
        g.vs[i] = c < n ? __ldg(vs + key0 + c) : 0.f;
      }
    }
  }

  // The running state of 16 rows (row r in m[0], l[0], o[.][0..1], row r + 8 in the others); l is
  // a lane's share of the sum until finish().  Logits in log2 units.
  struct State {
    float m[2], l[2];
    float o[NDT][4];
  };
  __device__ static __forceinline__ void clear(State& s) {
    s.m[0] = s.m[1] = NEG_INF;
    s.l[0] = s.l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < NDT; ++i) s.o[i][0] = s.o[i][1] = s.o[i][2] = s.o[i][3] = 0.f;
  }

  // Adds the granule's n keys to the state.  HI: rows 8 .. 15 are in use.
  template <bool HI>
  __device__ static __forceinline__ void add(State& st, const Regs& g, const uint32_t (&qa)[QW],
                                             const uint32_t (&qb)[QW], int n, float sl2, int q) {
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KCH; ++j) {
        const uint4 x = g.k[nt * KCH + j];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if constexpr (BITS == 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int a = 8 * j + 2 * e;
            mma_bf16_16816(s[nt], qa[a], HI ? qb[a] : 0u, qa[a + 1], HI ? qb[a + 1] : 0u,
                           widen_codes(__byte_perm(w[e], 0, 0x4140)), widen_codes(__byte_perm(w[e], 0, 0x4342)));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int a = 4 * j + 2 * e;
            mma_bf16_16816(s[nt], qa[a], HI ? qb[a] : 0u, qa[a + 1], HI ? qb[a + 1] : 0u, w[2 * e], w[2 * e + 1]);
          }
        }
      }
    }
    float mx[2] = {NEG_INF, NEG_INF};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool in = 8 * nt + 2 * q + c < n;
        const float f = BITS == 8 ? g.ks[2 * nt + c] * sl2 : sl2;
        s[nt][c] = in ? s[nt][c] * f : NEG_INF;
        mx[0] = fmaxf(mx[0], s[nt][c]);
        if (HI) {
          s[nt][2 + c] = in ? s[nt][2 + c] * f : NEG_INF;
          mx[1] = fmaxf(mx[1], s[nt][2 + c]);
        }
      }
    bool moved = false;
    float cf[2] = {1.f, 1.f};
#pragma unroll
    for (int h = 0; h < (HI ? 2 : 1); ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      if (mx[h] > st.m[h]) {
        cf[h] = fast_exp2(st.m[h] - mx[h]);  // 0 for the first keys
        st.m[h] = mx[h];
        st.l[h] *= cf[h];
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
        const float ref = st.m[h] == NEG_INF ? 0.f : st.m[h];
        const float p0 = fast_exp2(s[nt][2 * h] - ref), p1 = fast_exp2(s[nt][2 * h + 1] - ref);
        st.l[h] += p0 + p1;
        // a masked key's scale is 0 here, whatever its place in the cache holds
        pa[nt >> 1][2 * (nt & 1) + h] = BITS == 8 ? pack_bf16x2(p0 * g.vs[2 * nt], p1 * g.vs[2 * nt + 1]) : pack_bf16x2(p0, p1);
      }
    }
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const uint32_t* v = g.v + kk * 4 * VW;
#pragma unroll
      for (int i = 0; i < NDT; ++i) {
        uint32_t b0, b1;
        if constexpr (BITS == 8) {
          const int w = i >> 2;
          const uint32_t sel = (uint32_t)(i & 3) * 0x1111u + 0x4400u;
          b0 = widen_codes(__byte_perm(v[w], v[VW + w], sel));
          b1 = widen_codes(__byte_perm(v[2 * VW + w], v[3 * VW + w], sel));
        } else {
          const int w = (i >> 3) * 4 + ((i & 7) >> 1);
          const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
          b0 = __byte_perm(v[w], v[VW + w], sel);
          b1 = __byte_perm(v[2 * VW + w], v[3 * VW + w], sel);
        }
        mma_bf16_16816(st.o[i], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], b0, b1);
      }
    }
  }

  // Row sums over the four lanes of a row.
  template <bool HI>
  __device__ static __forceinline__ void finish(State& s) {
#pragma unroll
    for (int h = 0; h < (HI ? 2 : 1); ++h) {
      s.l[h] += __shfl_xor_sync(0xffffffffu, s.l[h], 1);
      s.l[h] += __shfl_xor_sync(0xffffffffu, s.l[h], 2);
    }
  }
};

// Joins the four warps' states of one block into shared memory: po [4][16][D] (written here) with
// pm, pl [4][16]; afterwards the block's row maxima are in bm, its sums in bl and its output sums,
// relative to bm, in po[0].  `rows` rows are in use.  All threads of a 128-thread block.
template <int D, int BITS, bool HI>
__device__ __forceinline__ void join_warps(typename CacheTile<D, BITS>::State& st, float* po, float (*pm)[16],
                                           float (*pl)[16], float* bm, float* bl, int rows) {
  using T = CacheTile<D, BITS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  T::template finish<HI>(st);
  if (q == 0) {
    pm[warp][r] = st.m[0];
    pl[warp][r] = st.l[0];
    pm[warp][r + 8] = HI ? st.m[1] : NEG_INF;
    pl[warp][r + 8] = HI ? st.l[1] : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < (HI ? 2 : 1); ++h) {
    const int row = r + 8 * h;
    float m = pm[0][row];
#pragma unroll
    for (int w = 1; w < 4; ++w) m = fmaxf(m, pm[w][row]);
    const float f = st.m[h] == NEG_INF ? 0.f : fast_exp2(st.m[h] - m);
    if (row < rows) {
#pragma unroll
      for (int i = 0; i < T::NDT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          po[((size_t)warp * 16 + row) * D + T::column(i, 2 * q + c)] = f == 0.f ? 0.f : st.o[i][2 * h + c] * f;
    }
  }
  if (threadIdx.x < 16) {
    const int row = threadIdx.x;
    float m = pm[0][row], l = 0.f;
#pragma unroll
    for (int w = 1; w < 4; ++w) m = fmaxf(m, pm[w][row]);
#pragma unroll
    for (int w = 0; w < 4; ++w)  // without a maximum a sum is 0, or NaN where every logit was
      l += pm[w][row] == NEG_INF ? pl[w][row] : pl[w][row] * fast_exp2(pm[w][row] - m);
    bm[row] = m;
    bl[row] = l;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D; i += 128) {
    const float a = po[i] + po[16 * D + i], b = po[32 * D + i] + po[48 * D + i];
    po[i] = a + b;
  }
}

}  // namespace pisa
