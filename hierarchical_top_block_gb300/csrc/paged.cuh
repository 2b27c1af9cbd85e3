// The paged cache, and how the attention over it is divided over thread blocks.
//
// Keys and values of all sequences lie in pages [P][H_kv][S][d], S = 2^s_bits tokens; key c of sequence b is row
// c mod S of page table[b][c / S].  Sequence b has L = seq_len[b] keys before its n new tokens, whose
// query rows are first .. first + n - 1; token t sees the keys 0 .. L + t (or all L + n).
//
// A job is (sequence, KV head, tile of ROWS query rows: ROWS / G_Q tokens of G_Q heads); it takes the keys that its
// last token sees in steps of PAGED_KT.  The jobs' steps, one job after the other, form one line that is cut into
// equal ranges, one a block: whatever the lengths, every block gets the same work.  A job that lies in one block
// is finished there; of one that spans blocks each stores its part (row maxima, sums and output sums), and a
// second kernel joins them.  A block has at most two such parts: the first job of its range and the last.  On
// the line every job begins with `extra` empty steps, as long as a block stops for it (rows written, others
// fetched): 880 jobs of 2 to 47 steps over 152 blocks, d = 64, took 191 us with them and 234 without.  The cut depends on
// the sizes alone, so results are the same in every run.
//
// With the causal mask the jobs of a head have different numbers of steps; their sums have a closed form:
// a tile of TT tokens (a power of two) ends at token (i + 1) TT, so it takes floor((L + 127 + (i + 1) TT) / 128)
// steps, which is floor((a + i + 1) / c) with c = 128 / TT and a = floor((L + 127) / TT).
#pragma once

#include "common.cuh"

namespace pisa {

constexpr int PAGED_KT = 128;  // keys a step

// A job that spans blocks, written by the one where it begins: its parts are slot0, then the first slots of the blocks behind
// it up to c1 (c1 < 0: there is no such job).
struct __align__(16) PagedSplit {
  int b, first, n, L;  // sequence; its first row, rows and keys before them
  int head, tile, c1, slot0;
};

struct PagedParams {
  const uint16_t* q;
  const uint16_t* K;
  const uint16_t* V;
  float* w;                  // (the weights' kernels)
  const float* lse_in;       // (the same)
  const int32_t* table;      // [B][M]
  const int32_t* seq_len;    // [B]
  const int32_t* row_start;  // [B + 1], nullable: R / B rows each
  uint16_t* o;
  float* lse;                // nullable
  float* part_o;             // [2 blocks][ROWS][d] output sums relative to the row maximum
  float2* part_ml;           // [2 blocks][ROWS] row maximum (log2 units) and sum
  PagedSplit* split;         // [blocks] the job that a block leaves unfinished, where it has its beginning
  long long q_stride;        // elements between rows of q
  int B, R, H_q, H_kv, GQ, P, M;
  int s_bits, gq_bits, row_bits;  // S, G_Q and ROWS are 2 to these
  int causal, accumulate;
  int blocks, stop;          // thread blocks the line is cut for; steps that a second job in a block costs
  unsigned long long inverse;  // ceil(2^64 / blocks)
  float sl2;
  uint32_t* err;
};

struct PagedSeq {
  int first, n, L;  // first row, rows (0 where the lengths do not fit: the sequence is left out), keys before them
};
// `bad`: the inputs are out of range.
__device__ __forceinline__ PagedSeq paged_seq(const int32_t* row_start, const int32_t* seq_len, int B, int R, int cap,
                                              int b, bool& bad) {
  PagedSeq s;
  int lo = row_start ? __ldg(row_start + b) : b * (R / B), hi = row_start ? __ldg(row_start + b + 1) : lo + R / B;
  bad = lo < 0 || hi < lo || hi > R;
  lo = min(max(lo, 0), R);
  hi = min(max(hi, lo), R);
  s.first = lo;
  s.n = hi - lo;
  s.L = __ldg(seq_len + b);
  if (s.L < 0 || s.L > cap - s.n) {
    bad = true;
    s.n = s.L = 0;
  }
  return s;
}
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b, bool& bad) {
  return paged_seq(p.row_start, p.seq_len, p.B, p.R, p.M << p.s_bits, b, bad);
}

// a / b of numbers >= 0, in 32 bits where they fit.
__device__ __forceinline__ long long whole_quotient(long long a, long long b) {
  return (a >> 32) || (b >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// The tile of a head that holds its position x < span(extra).
template <class Jobs>
__device__ __forceinline__ int tile_of(const Jobs& j, long long x, int extra) {
  int lo = 0, hi = j.tiles - 1;  // the last tile that begins at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (j.before(mid) + (long long)mid * extra <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The steps of a sequence's jobs, the same for each of its KV heads.
struct PagedJobs {
  int tiles, tt_bits;  // tiles a head; tokens a tile, 2 to this
  int L, n, causal;
  __device__ __forceinline__ PagedJobs(const PagedParams& p, const PagedSeq& s) {
    tt_bits = p.row_bits - p.gq_bits;
    tiles = (s.n + (1 << tt_bits) - 1) >> tt_bits;
    L = s.L;
    n = s.n;
    causal = p.causal;
  }
  // Keys that the last token of tile i sees.
  __device__ __forceinline__ int keys(int i) const { return L + (causal ? min(n, (i + 1) << tt_bits) : n); }
  __device__ __forceinline__ int steps(int i) const { return (keys(i) + PAGED_KT - 1) / PAGED_KT; }
  // Steps of the tiles before tile k <= tiles.
  __device__ __forceinline__ long long before(int k) const {
    if (k == 0) return 0;
    if (!causal) return (long long)k * steps(0);
    const int last = k == tiles ? steps(k - 1) : -1;  // (it may be ragged)
    if (last >= 0 && --k == 0) return last;
    long long sum;
    const int a0 = L + PAGED_KT - 1;
    if (tt_bits >= 8) {
      sum = (long long)k * (a0 / PAGED_KT) + ((long long)k * (k + 1) << (tt_bits - 8));
    } else {
      const int a = a0 >> tt_bits;
      sum = floors(a + k) - floors(a);
    }
    return sum + max(last, 0);
  }
  // sum of floor(j / c) for j = 0 .. m, c = 128 / TT
  __device__ __forceinline__ long long floors(int m) const {
    const int c_bits = 7 - tt_bits, q = m >> c_bits, r = m - (q << c_bits);
    return ((long long)q * (q - 1) >> 1 << c_bits) + (long long)q * (r + 1);
  }
  __device__ __forceinline__ long long span(int extra) const { return before(tiles) + (long long)tiles * extra; }
  __device__ __forceinline__ int tile_at(long long x, int extra) const { return tile_of(*this, x, extra); }
};

// The cut of S positions over the blocks: every block in use has one at least, so a job's parts are in consecutive
// blocks.  x / blocks of x < 2^64 / blocks as one product: with m = ceil(2^64 / blocks) = (2^64 + e) / blocks, e < blocks,
// x m / 2^64 exceeds x / blocks by x e / (blocks 2^64) < 1 / blocks.
struct PagedCut {
  long long S;
  int extra;
  __device__ __forceinline__ int used(const PagedParams& p) const { return (int)max(min(S, (long long)p.blocks), 1ll); }
  __device__ __forceinline__ long long start(const PagedParams& p, int block) const {
    if (S <= p.blocks) return block;
    return p.blocks == 1 ? S * block : (long long)__umul64hi((unsigned long long)S * block, p.inverse);
  }
  // The block that holds position s: the last one that starts at or before it.
  __device__ __forceinline__ int block_of(const PagedParams& p, long long s) const {
    return S <= p.blocks ? (int)s : (int)whole_quotient((s + 1) * p.blocks - 1, S);
  }
};
__device__ __forceinline__ PagedCut paged_cut_of(const PagedParams& p, long long S, long long jobs) {
  if (S <= p.blocks || p.blocks == 1) return PagedCut{S, 0};  // a step a block
  const long long len = (long long)__umul64hi((unsigned long long)S, p.inverse), with = S + jobs * p.stop;
  // with many jobs a block; or where the longest range is no longer with the empty steps than with one stop
  return jobs > p.blocks || (jobs > 1 && with <= (len + p.stop) * p.blocks) ? PagedCut{with, p.stop} : PagedCut{S, 0};
}

// Walks a block's range job by job.  Every thread of a warp holds the same state.
template <class Jobs>
struct PagedLine {
  long long at, end;  // next position and end of the range
  long long gbase;    // first position of the current sequence
  long long job_end;  // the position behind the current job
  long long length;   // the line's
  int b;              // current sequence
  short extra;        // empty steps before a job's own
  bool begun;         // a segment of the range is behind
  PagedSeq s;
  // current segment
  int head, tile, k0, k1;  // KV head, tile, steps [k0, k1) of the job
  int slot;                // -1: the whole job; else the part's slot (2 block + 0 or 1)

  // Warp-wide.  `report`: this warp reports bad inputs.
  __device__ __forceinline__ void init(const PagedParams& p, int block, bool report) {
    const int lane = threadIdx.x & 31;
    begun = false;
    b = 0;
    gbase = 0;
    job_end = -1;
    // sums over the sequences before and with a lane's own: steps and jobs
    long long S = 0, jobs = 0;
    auto sums = [&](int i0, long long& x, long long& n) {
      x = n = 0;
      bool bad = false;
      if (i0 + lane < p.B) {
        const Jobs j(p, paged_seq(p, i0 + lane, bad));
        x = p.H_kv * j.before(j.tiles);
        n = (long long)p.H_kv * j.tiles;
      }
      if (report && bad) report_error(p.err, ERR_BAD_INDEX);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        const long long k = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) x += y, n += k;
      }
    };
    long long x, n;
    for (int i0 = 0; i0 < p.B; i0 += 32) {
      sums(i0, x, n);
      S += __shfl_sync(0xffffffffu, x, 31);
      jobs += __shfl_sync(0xffffffffu, n, 31);
    }
    const PagedCut cut = paged_cut_of(p, S, jobs);
    extra = (short)cut.extra;
    length = cut.S;
    at = end = 0;
    if (block >= cut.used(p)) return;
    at = cut.start(p, block);
    end = cut.start(p, block + 1);
    if (at >= end) return;
    // the sequence that holds position `at`
    long long before = 0;
    for (int i0 = 0; i0 < p.B; i0 += 32) {
      if (p.B > 32) sums(i0, x, n);  // (else they are there)
      const long long upto = before + x + n * extra;
      const unsigned past = __ballot_sync(0xffffffffu, upto > at);
      if (past) {
        const int l = __ffs(past) - 1;
        b = i0 + l;
        const long long begin = __shfl_sync(0xffffffffu, upto, max(l - 1, 0));
        gbase = l > 0 ? begin : before;
        break;
      }
      before = __shfl_sync(0xffffffffu, upto, 31);
    }
    bool bad;
    s = paged_seq(p, b, bad);
  }

  // Moves to the next segment; false at the end of the range.
  __device__ __forceinline__ bool next(const PagedParams& p, int block) {
    for (;;) {
      if (at >= end) return false;
      const Jobs j(p, s);
      long long off;  // in the job
      if (at == job_end && tile + 1 < j.tiles) {  // the head's next
        ++tile;
        off = 0;
        job_end += extra + j.steps(tile);
      } else if (at >= job_end) {
        const long long span = j.span(extra);
        off = at - gbase;
        if (off >= p.H_kv * span) {  // at < end <= the line's length: a later sequence holds it
          gbase += p.H_kv * span;
          if (++b >= p.B) return false;  // (unless somebody changes the lengths under the call)
          bool bad;
          s = paged_seq(p, b, bad);
          job_end = -1;  // (of another sequence)
          continue;
        }
        head = (int)whole_quotient(off, span);
        off -= head * span;
        tile = j.tile_at(off, extra);
        off -= j.before(tile) + (long long)tile * extra;
        job_end = at - off + extra + j.steps(tile);
      } else {
        off = extra;  // behind the job's empty steps
      }
      if (off < extra) {  // the empty steps
        at = min(end, at + extra - off);
        continue;
      }
      const int steps = j.steps(tile);
      k0 = (int)(off - extra);
      k1 = (int)min((long long)steps, k0 + (end - at));
      slot = (k0 == 0 && k1 == steps) ? -1 : 2 * block + (begun ? 1 : 0);
      begun = true;
      at += k1 - k0;
      return true;
    }
  }

  // Behind the last segment: the job that goes on in the next blocks, if it begins in this one.
  __device__ __forceinline__ PagedSplit split(const PagedParams& p, int block) const {
    PagedSplit x = {b, s.first, s.n, s.L, head, tile, -1, slot};
    if (begun && slot >= 0 && k0 == 0)
      x.c1 = PagedCut{length, extra}.block_of(p, job_end - 1);
    if (x.c1 <= block) x.c1 = -1;
    return x;
  }
  // For the kernel that joins.
  __device__ __forceinline__ bool take(const PagedSplit& x) {
    b = x.b;
    s.first = x.first;
    s.n = x.n;
    s.L = x.L;
    head = x.head;
    tile = x.tile;
    return x.c1 >= 0;
  }
};

// The attention's: jobs of query tiles.
struct PagedWalk : PagedLine<PagedJobs> {
  // Keys that query row `row` of the tile sees.
  __device__ __forceinline__ int seen(const PagedParams& p, int row) const {
    const int tok = min(((tile << p.row_bits) + row) >> p.gq_bits, s.n - 1);
    return s.L + (p.causal ? tok + 1 : s.n);
  }
  // Query rows of the tile, and the place of one among all rows and heads.
  __device__ __forceinline__ int rows(const PagedParams& p) const {
    return min(1 << p.row_bits, (s.n << p.gq_bits) - (tile << p.row_bits));
  }
  __device__ __forceinline__ size_t row_at(const PagedParams& p, int row) const {
    const int m = (tile << p.row_bits) + row, tok = m >> p.gq_bits;
    return (size_t)(s.first + tok) * p.H_q + (size_t)head * p.GQ + (m - (tok << p.gq_bits));
  }
};

// The page of keys from c0 on (c0 < cap): its number, or P (whose rows a copy reads as zeros) where the entry names
// none; no row sees those keys.  Entries from P on are reported.
__device__ __forceinline__ int page_of(const int32_t* table, int P, int entry, uint32_t* err) {
  const int page = __ldg(table + entry);
  if (page >= P) report_error(err, ERR_BAD_INDEX);
  return page < 0 || page >= P ? P : page;
}

// The tensor-core kernel (paged_tc.cu): tiles of PAGED_TC_ROWS rows, one block a SM.
constexpr int PAGED_TC_ROWS = 256;
cudaError_t launch_paged_tc(const PagedParams& p, int d, cudaStream_t s);

// The slots of a ring in turn, with the parity of their phase.
template <uint32_t N>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

// A finished row: the factor of its output sums, and its log-sum-exp.
__device__ __forceinline__ float finish_row(float m, float l, float& lse) {
  lse = l == 0.f ? NEG_INF : (m + log2f(l)) * LN2;
  return l == 0.f ? 0.f : 1.f / l;
}

// A map over the query rows of one KV head's group: boxes of `rows`, (64 columns, G_Q heads, 1 KV head, rows / G_Q tokens).
bool encode_token_map(CUtensorMap* map, const uint16_t* q, int d, int GQ, int H_kv, int R, long long q_stride, int rows);
// A map over pages [P][H_kv][S][d]: boxes of `keys` rows of 64 columns.
bool encode_page_map(CUtensorMap* map, const void* base, int d, int S, int H_kv, int P, int keys);

}  // namespace pisa
