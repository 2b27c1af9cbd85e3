// The attention weight that every key of the paged cache has got from the new tokens:
//
//   w_c (+)= sum over the tokens t that see key c and the query heads of its KV head of  exp(scale q_t . k_c - lse_t)
//
// with the tokens' log-sum-exps from the attention.  A key belongs to one block, which goes over the query rows
// in order: results are the same in every run.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace pisa {
namespace {

constexpr int THREADS = 128, QT = 16;  // keys a block; query rows at a time

struct WeightParams {
  const uint16_t* q;
  const float* lse;
  const uint16_t* K;
  float* w;
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* row_start;
  long long q_stride;
  int B, R, H_q, H, GQ, gq_bits, P, M, s_bits, causal, accumulate;
  float sl2;
  uint32_t* err;
};

// One key a thread, its row in registers; the query rows go through shared memory.
template <int D>
__global__ void __launch_bounds__(THREADS) paged_weights_kernel(WeightParams p) {
  __shared__ __align__(16) float sq[QT][D];
  __shared__ float sl[QT];
  const int b = blockIdx.z, h = blockIdx.y;
  bool bad;
  const PagedSeq s = paged_seq(p.row_start, p.seq_len, p.B, p.R, p.M << p.s_bits, b, bad);
  if (bad && blockIdx.x == 0 && h == 0 && threadIdx.x == 0) report_error(p.err, ERR_BAD_INDEX);
  const int total = s.L + s.n;
  for (int c0 = blockIdx.x * THREADS; c0 < total; c0 += gridDim.x * THREADS) {
    const int c = c0 + threadIdx.x;
    int page = p.P;
    if (c < total) page = page_of(p.table + (size_t)b * p.M, p.P, c >> p.s_bits, p.err);
    const size_t at = (((size_t)page * p.H + h) << p.s_bits) + (c & ((1 << p.s_bits) - 1));
    uint32_t k[D / 2];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint4 x = page < p.P ? ldg16(p.K + at * D + 8 * i) : make_uint4(0, 0, 0, 0);
      k[4 * i] = x.x, k[4 * i + 1] = x.y, k[4 * i + 2] = x.z, k[4 * i + 3] = x.w;
    }
    float sum = 0.f;
    const int rows = s.n << p.gq_bits, first = p.causal ? max(0, c0 - s.L) << p.gq_bits : 0;
    for (int m0 = first; m0 < rows; m0 += QT) {
      __syncthreads();
      for (int i = threadIdx.x; i < QT * D; i += THREADS) {
        const int m = m0 + i / D, t = m >> p.gq_bits;
        sq[i / D][i % D] = m < rows ? bf16_to_f32(p.q[(s.first + t) * p.q_stride + (size_t)((h << p.gq_bits) + m - (t << p.gq_bits)) * D + i % D]) : 0.f;
      }
      if (threadIdx.x < QT) {
        const int m = m0 + threadIdx.x, t = m >> p.gq_bits;
        sl[threadIdx.x] = m < rows ? p.lse[(size_t)(s.first + t) * p.H_q + (h << p.gq_bits) + m - (t << p.gq_bits)] * LOG2E : POS_INF;
      }
      __syncthreads();
      for (int i = 0; i < QT; ++i) {
        float a = 0.f, e = 0.f;
#pragma unroll
        for (int j = 0; j < D / 2; j += 2) {
          const float4 x = *reinterpret_cast<const float4*>(&sq[i][2 * j]);
          a = fmaf(x.x, bf16_lo(k[j]), a);
          e = fmaf(x.y, bf16_hi(k[j]), e);
          a = fmaf(x.z, bf16_lo(k[j + 1]), a);
          e = fmaf(x.w, bf16_hi(k[j + 1]), e);
        }
        const int t = (m0 + i) >> p.gq_bits;
        // a row that saw nothing (lse = -inf) gives nothing
        if (m0 + i < rows && sl[i] != NEG_INF && (!p.causal || c <= s.L + t)) sum += fast_exp2(fmaf(a + e, p.sl2, -sl[i]));
      }
    }
    if (c < total && page < p.P) p.w[at] = p.accumulate ? p.w[at] + sum : sum;
  }
}

}  // namespace

cudaError_t launch_paged_weights(const uint16_t* q, long long q_stride, const float* lse, const uint16_t* Kp, float* w,
                                 const int32_t* table, const int32_t* seq_len, const int32_t* row_start, bool accumulate,
                                 const Problem& pr, const Pages& pg, uint32_t* err, cudaStream_t s) {
  WeightParams p{q,     lse,     Kp,    w,    table, seq_len,   row_start, q_stride,   pr.B,
                 pr.N,  pr.H_q,  pr.H_kv, pr.GQ, 0,    pg.P,      pg.M,      pg.s_bits, pr.causal,
                 accumulate, pr.scale * LOG2E, err};
  while ((1 << p.gq_bits) < pr.GQ) ++p.gq_bits;
  const long long most = (((long long)pg.M << pg.s_bits) + THREADS - 1) / THREADS;
  const dim3 grid((unsigned)std::min<long long>(most, 65535), (unsigned)pr.H_kv, (unsigned)pr.B);
  if (pr.d == 128)
    paged_weights_kernel<128><<<grid, THREADS, 0, s>>>(p);
  else
    paged_weights_kernel<64><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pisa
