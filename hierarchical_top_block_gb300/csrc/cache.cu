// The 8-bit key/value cache: rows are quantised as they are written, and read back as bf16.
//
// A row x (d values of one key or value head) is stored as int8 codes and one fp32 scale:
//   a = max_i |x_i|,  scale = a / 127,  code_i = sign(x_i) floor(127 |x_i| / a + 1/2)
// (a = 0: codes and scale 0; a row with an infinity or a NaN: codes 0, scale NaN, so that the row
// reads back as NaN).  The scale is per (token, head): a row never changes after it was written,
// so tokens can be appended one at a time and the attention can keep the codes as whole numbers
// (they are exact in bf16) and apply the scale to the fp32 logit or weight.
//
// Rounding half away from zero makes the codes exact with one fp32 reciprocal a row: with
// X, M < 2^8 the integer significands of x and a and e the difference of their exponents,
// 127 |x| / a = 127 X / (M 2^e), so a value that is not half-way between two codes is at least
// 1 / (2 M 2^e) > 2^-(e+9) from half-way, while its size is below 2^(8-e).  Multiplying by
// (127 / a)(1 + 2^-20) moves it by less than 2^(8.3-e-20) = 2^-(e+11.7) (the two roundings included), too
// little to cross, and moves an exact half-way value up, never down.
//
// Both kernels move bytes: 16 lanes (d = 128) or 8 lanes (d = 64) take a row, 8 values a lane, so
// every access of a warp is whole 128-byte lines; a thread has RPT rows in flight, four when there are
// rows for every SM, one when latency counts (8 heads x 131072 rows of K and V at d = 128 written 250 us with
// four, 281 with one, read back 117 and 167; 64 x 8 rows written 3.1 and 2.1 us, 7 x 4 x 333 rows of d = 64
// read 2.7 and 2.3).  A block takes its rows and ends: resident blocks that walk over the rows read
// 127 us.
#include "kernels.cuh"

namespace pisa {
namespace {

constexpr int THREADS = 128;

// n / d of n < 2^31 as one product: with 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d) < 2^32 + 1, n m / 2^(31+s)
// exceeds n / d by n (m d - 2^(31+s)) / (d 2^(31+s)) < 2^31 2^s / (d 2^(31+s)) = 1 / d: the whole part is that of n / d.
struct Divisor {
  uint64_t m;
  uint32_t d, shift;
};
Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {((1ull << (31 + s)) + d - 1) / d, d, 31 + s};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor& d) { return (uint32_t)((n * d.m) >> d.shift); }

struct CacheParams {
  const uint16_t* x[2];  // write: K and V rows in
  uint16_t* y[2];        // values out (read: the rows; write: nullable)
  int8_t* q[2];
  float* s[2];
  const int32_t* start;  // first cache row of each sequence (nullable: 0)
  const int32_t* count;  // rows of each sequence in use (nullable: T)
  uint32_t rows;         // B * H * T, below 2^31
  Divisor H, T;
  int N_cap;
  uint32_t* err;
};

// The place of row `row` of [B][H][T]: its cache row, or -1 where there is none (behind the
// sequence's count, or a sequence whose rows do not fit: nothing of it is read or written).
__device__ __forceinline__ long long cache_row(const CacheParams& p, uint32_t row) {
  const uint32_t bh = quotient(row, p.T), t = row - bh * p.T.d, b = quotient(bh, p.H);
  const int first = p.start ? __ldg(p.start + b) : 0, n = p.count ? __ldg(p.count + b) : (int)p.T.d;
  if (first < 0 || n < 0 || n > (int)p.T.d || first > p.N_cap - n) {
    report_error(p.err, ERR_BAD_INDEX);
    return -1;
  }
  return t < (uint32_t)n ? (long long)bh * p.N_cap + first + t : -1;
}

template <int D, int RPT, bool VALUES>
__global__ void __launch_bounds__(THREADS) cache_write_kernel(CacheParams p) {
  constexpr int LANES = D / 8, RPB = THREADS / LANES;  // lanes a row, rows a block and step
  const int part = threadIdx.x % LANES, kv = blockIdx.y;
  int8_t* q = kv ? p.q[1] : p.q[0];
  float* s = kv ? p.s[1] : p.s[0];
  uint16_t* y = kv ? p.y[1] : p.y[0];
  const uint16_t* x = kv ? p.x[1] : p.x[0];  // may be the values out as well: each lane reads its part before it writes it
  const uint64_t first = (uint64_t)blockIdx.x * RPB * RPT + threadIdx.x / LANES;
  uint4 w[RPT];
  long long at[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const uint64_t row = first + (uint64_t)i * RPB;
    at[i] = row < p.rows ? cache_row(p, (uint32_t)row) : -1;
    w[i] = at[i] >= 0 ? *reinterpret_cast<const uint4*>(x + row * D + 8 * part) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    // the largest |x| by its bits (bf16 magnitudes order as integers; NaN above infinity), two at a time
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) a = __vmaxu2(a, u[j] & 0x7fff7fffu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, o));
    a = max(a >> 16, a & 0xffffu);
    const float amax = __uint_as_float(a << 16);
    const bool finite = a < 0x7f80u;
    const float scale = finite ? __fdiv_rn(amax, 127.f) : __uint_as_float(0x7fc00000u);
    // 127 / a overflows below 2^-121: both sides times 2^64 there (exact)
    const float up = amax < 5.421010862427522e-20f ? 1.8446744073709552e19f : 1.f;
    const float inv = a == 0 || !finite ? 0.f : __fdiv_rn(127.f, amax * up) * (1.f + 9.5367431640625e-07f);
    float t[8];         // the codes
    uint32_t bits[8];   // the codes in their low bytes
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j % 2 == 0 && !finite) u[j / 2] = 0;
      float v = j % 2 ? bf16_hi(u[j / 2]) : bf16_lo(u[j / 2]);
      if (up != 1.f) v *= up;
      // |v inv| + 1/2 is cut to a whole number by its sum with 2^23 towards zero, and the code, subtracted
      // from that again, is left in two's complement by a sum with 1.5 2^23
      const uint32_t sign = __float_as_uint(v) & 0x80000000u;
      const float big = __uint_as_float(0x4b000000u | sign);
      t[j] = __fadd_rn(__fadd_rz(__fmaf_rn(v, inv, __uint_as_float(0x3f000000u | sign)), big), -big);
      bits[j] = __float_as_uint(__fadd_rn(t[j], 12582912.f));
    }
    if (at[i] < 0) continue;
    uint32_t code[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      code[h] = __byte_perm(__byte_perm(bits[4 * h], bits[4 * h + 1], 0x0040),
                            __byte_perm(bits[4 * h + 2], bits[4 * h + 3], 0x0040), 0x5410);
    *reinterpret_cast<uint2*>(q + at[i] * D + 8 * part) = make_uint2(code[0], code[1]);
    if (part == 0) s[at[i]] = scale;
    if (VALUES) {
      uint4 v;
      v.x = pack_bf16x2(t[0] * scale, t[1] * scale);
      v.y = pack_bf16x2(t[2] * scale, t[3] * scale);
      v.z = pack_bf16x2(t[4] * scale, t[5] * scale);
      v.w = pack_bf16x2(t[6] * scale, t[7] * scale);
      if (y) *reinterpret_cast<uint4*>(y + (first + (uint64_t)i * RPB) * D + 8 * part) = v;
    }
  }
}

template <int D, int RPT>
__global__ void __launch_bounds__(THREADS) cache_read_kernel(CacheParams p) {
  constexpr int LANES = D / 8, RPB = THREADS / LANES;
  const int part = threadIdx.x % LANES;
  const int kv = p.y[0] == nullptr ? 1 : blockIdx.y;  // K, V or both
  const int8_t* __restrict__ q = kv ? p.q[1] : p.q[0];
  const float* __restrict__ s = kv ? p.s[1] : p.s[0];
  uint16_t* y = kv ? p.y[1] : p.y[0];
  const uint64_t first = (uint64_t)blockIdx.x * RPB * RPT + threadIdx.x / LANES;
  uint2 w[RPT];
  float sc[RPT];
  long long at[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const uint64_t row = first + (uint64_t)i * RPB;
    at[i] = row < p.rows ? cache_row(p, (uint32_t)row) : -1;
    w[i] = at[i] >= 0 ? __ldg(reinterpret_cast<const uint2*>(q + at[i] * D + 8 * part)) : make_uint2(0, 0);
    sc[i] = at[i] >= 0 ? __ldg(s + at[i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    if (at[i] < 0) continue;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = (float)(int8_t)(w[i].x >> (8 * j)) * sc[i];
      f[4 + j] = (float)(int8_t)(w[i].y >> (8 * j)) * sc[i];
    }
    uint4 v;
    v.x = pack_bf16x2(f[0], f[1]);
    v.y = pack_bf16x2(f[2], f[3]);
    v.z = pack_bf16x2(f[4], f[5]);
    v.w = pack_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4*>(y + (first + (uint64_t)i * RPB) * D + 8 * part) = v;
  }
}

// Blocks of `rpt` rows a thread.
unsigned blocks_for(uint32_t rows, int d, int rpt) {
  const uint32_t step = (uint32_t)(THREADS / (d / 8) * rpt);
  return (rows + step - 1) / step;
}
// Rows a thread: four once one would fill every SM's threads.
int rows_per_thread(uint32_t rows, int d, int num_sms) { return blocks_for(rows, d, 1) > 2048u / THREADS * num_sms ? 4 : 1; }

template <int D, int RPT>
void write_with(const CacheParams& c, cudaStream_t s) {
  const dim3 grid(blocks_for(c.rows, D, RPT), 2);
  if (c.y[0] || c.y[1])
    cache_write_kernel<D, RPT, true><<<grid, THREADS, 0, s>>>(c);
  else
    cache_write_kernel<D, RPT, false><<<grid, THREADS, 0, s>>>(c);
}
template <int D, int RPT>
void read_with(const CacheParams& c, cudaStream_t s) {
  cache_read_kernel<D, RPT><<<dim3(blocks_for(c.rows, D, RPT), c.y[0] && c.y[1] ? 2 : 1), THREADS, 0, s>>>(c);
}

CacheParams params_of(const Problem& p, uint32_t* err) {
  CacheParams c{};
  c.rows = (uint32_t)p.B * (uint32_t)p.H_kv * (uint32_t)p.N;
  c.H = divisor((uint32_t)p.H_kv);
  c.T = divisor((uint32_t)p.N);
  c.N_cap = p.N_cap;
  c.err = err;
  return c;
}

}  // namespace

cudaError_t launch_cache_write(const uint16_t* k, const uint16_t* v, int8_t* Kq, int8_t* Vq, float* k_scale,
                               float* v_scale, const int32_t* seq_len, const int32_t* new_len, uint16_t* k_out,
                               uint16_t* v_out, const Problem& p, int num_sms, uint32_t* err, cudaStream_t s) {
  CacheParams c = params_of(p, err);
  c.x[0] = k;
  c.x[1] = v;
  c.y[0] = k_out;
  c.y[1] = v_out;
  c.q[0] = Kq;
  c.q[1] = Vq;
  c.s[0] = k_scale;
  c.s[1] = v_scale;
  c.start = seq_len;
  c.count = new_len;
  const bool one = rows_per_thread(c.rows, p.d, num_sms) == 1;
  if (p.d == 128)
    one ? write_with<128, 1>(c, s) : write_with<128, 4>(c, s);
  else
    one ? write_with<64, 1>(c, s) : write_with<64, 4>(c, s);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const int8_t* Kq, const int8_t* Vq, const float* k_scale, const float* v_scale,
                              const int32_t* start, const int32_t* len, uint16_t* k_out, uint16_t* v_out,
                              const Problem& p, int num_sms, uint32_t* err, cudaStream_t s) {
  CacheParams c = params_of(p, err);
  c.y[0] = k_out;
  c.y[1] = v_out;
  c.q[0] = const_cast<int8_t*>(Kq);
  c.q[1] = const_cast<int8_t*>(Vq);
  c.s[0] = const_cast<float*>(k_scale);
  c.s[1] = const_cast<float*>(v_scale);
  c.start = start;
  c.count = len;
  const bool one = rows_per_thread(c.rows, p.d, num_sms) == 1;
  if (p.d == 128)
    one ? read_with<128, 1>(c, s) : read_with<128, 4>(c, s);
  else
    one ? read_with<64, 1>(c, s) : read_with<64, 4>(c, s);
  return cudaGetLastError();
}

}  // namespace pisa
