// How the attention over shared prefixes is divided over thread blocks.
//
// A job is (group p, KV head, tile of ROWS query rows); it takes the group's prefix in steps of
// PREFIX_KT keys.  The jobs' steps, one job after the other, form one line, cut into equal ranges,
// one a block: whatever the number of groups, rows and keys, every block gets the same work.  A job
// that lies in one block is finished there; of a job that spans blocks, each block stores its part
// (row maxima, sums and output sums), and a second kernel joins them.  A block has at most two such
// parts: the first job of its range and the last.  The cut depends on the sizes alone, so results
// are the same in every run.
//
// The ranges begin at S b / blocks, rounded down, not at multiples of a rounded length: the jobs of one
// head (tiles of its query rows) read the same keys, and with the exact quotient their blocks begin at
// few different keys, walk over the prefix side by side, and all but the first find it in the L2 (256
// tokens of 32 / 2 heads after 131072 bf16 keys, 32 jobs over 152 blocks: 388 us, with multiples 403).
//
// A block that meets a second job stops for it: the rows of the first are written, those of the
// next fetched.  On the line every job therefore begins with `extra` empty steps, as long as that stop;
// where the jobs end on the blocks' bounds anyway, or the empty steps would make the ranges longer than
// a stop does, there are none.  (Five groups of 217 tokens of 16 / 4 heads in all, d = 128, 20 jobs of up to 79
// steps over 152 blocks: codes 43.0 us with a stop of 3 steps, 44.9 with 2, 43.1 with 4 and 5, 48.0 with none;
// bf16 33.7, 34.2, 34.0 and 34.6, 36.5.  One prefix of 32768 keys differs by less than 1%.  Few rows, three groups of
// two tokens over 20000 codes: 28.1 us with 2, 28.3 with 1, 28.7 with 3, 29.9 with none.)
#pragma once

#include <cfloat>

#include "common.cuh"

namespace pisa {

struct PrefixParams {
  const uint16_t* q;
  const uint8_t* K;
  const uint8_t* V;
  const float* ks;           // null: a bf16 cache
  const float* vs;
  const int32_t* prefix_len; // [P]
  const int32_t* row_start;  // [P + 1], nullable: one group of all R rows
  const uint16_t* o_own;     // nullable (both)
  const float* lse_own;
  uint16_t* o;
  float* lse;                // nullable
  float* part_o;             // [2 blocks][ROWS][d] output sums relative to the row maximum
  float2* part_ml;           // [2 blocks][ROWS] row maximum (log2 units) and sum
  long long* base;           // [P + 2] first step of each group, the line's length, `extra` (with one group: not written)
  int P, R, H_q, H_kv, GQ, N_cap;
  int gq_bits, row_bits;     // G_Q and ROWS are 2 to these
  int blocks;                // thread blocks the steps are divided over
  int stop;                  // steps that a second job in a block costs
  float sl2;
  uint32_t* err;
};

constexpr int PREFIX_KT = 128;  // keys a step

struct PrefixGroup {
  int first, n, len;      // first row, rows, prefix keys
  int tiles, steps;       // tiles a head; steps a job (an empty prefix has one, with no key)
};

__device__ __forceinline__ PrefixGroup prefix_group(const PrefixParams& p, int i) {
  PrefixGroup g;
  int lo = p.row_start ? __ldg(p.row_start + i) : 0, hi = p.row_start ? __ldg(p.row_start + i + 1) : p.R;
  lo = min(max(lo, 0), p.R);
  hi = min(max(hi, lo), p.R);
  g.first = lo;
  g.n = hi - lo;
  g.len = min(max(__ldg(p.prefix_len + i), 0), p.N_cap);
  g.tiles = (int)((((long long)g.n << p.gq_bits) + (1 << p.row_bits) - 1) >> p.row_bits);
  g.steps = max(1, (g.len + PREFIX_KT - 1) / PREFIX_KT);
  return g;
}
__device__ __forceinline__ long long group_jobs(const PrefixParams& p, const PrefixGroup& g) {
  return (long long)p.H_kv * g.tiles;
}

// a / b of numbers >= 0, in 32 bits where they fit (a fifth of the time).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a >> 32) || (b >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// The line's cut: S positions over `blocks` blocks.  Job j of a group whose first position is `base` has its
// steps from base + j (steps + extra) + extra on.
struct PrefixCut {
  long long S;
  int blocks, extra;
  __device__ __forceinline__ long long start(int block) const { return quotient(S * block, blocks); }
  // The block that holds position s: the last one that starts at or before it.
  __device__ __forceinline__ int block_of(long long s) const { return (int)quotient((s + 1) * blocks - 1, S); }
};
// Every block in use has a position, so a job's parts are in consecutive blocks.
__device__ __forceinline__ PrefixCut prefix_cut(const PrefixParams& p, long long S, int extra) {
  return PrefixCut{S, (int)max(min(S, (long long)p.blocks), 1ll), extra};
}
// S steps in so many jobs; `even(len)`: ranges of len steps never meet a second job.
template <class Even>
__device__ __forceinline__ PrefixCut prefix_cut(const PrefixParams& p, long long S, long long jobs, Even even) {
  const PrefixCut c = prefix_cut(p, S, 0);
  const long long len = quotient(S, c.blocks), with = S + jobs * p.stop;
  if (jobs <= 1 || (len * c.blocks == S && even(len))) return c;
  // the longest range, with its stop or with the empty steps
  return with <= (len + p.stop) * c.blocks ? prefix_cut(p, with, p.stop) : c;
}
__device__ __forceinline__ PrefixCut prefix_cut_one(const PrefixParams& p, const PrefixGroup& g) {
  return prefix_cut(p, group_jobs(p, g) * g.steps, group_jobs(p, g),
                    [&](long long len) { return quotient(g.steps, len) * len == g.steps; });
}

// Walks a block's range job by job.  Every thread of a warp holds the same state.
struct PrefixWalk {
  long long at, end;      // next step and end of the range
  long long gbase;        // first step of the current group
  int p;                  // current group
  short extra;            // empty steps before a job's own
  bool begun;             // a segment of the range is behind
  PrefixGroup g;
  // current segment
  int head, tile, k0, k1; // KV head, tile, steps [k0, k1) of the job
  int slot;               // -1: the whole job; else the part's slot (2 block + 0 or 1)

  // Warp-wide.  `record`: this warp writes the groups' first steps and reports bad inputs.
  __device__ __forceinline__ void init(const PrefixParams& prm, int block, bool record) {
    const int lane = threadIdx.x & 31;
    if (record) {
      for (int i = lane; i < prm.P; i += 32) {
        const int n = __ldg(prm.prefix_len + i);
        bool bad = n < 0 || n > prm.N_cap;
        if (prm.row_start) {
          const int a = __ldg(prm.row_start + i), b = __ldg(prm.row_start + i + 1);
          bad = bad || a < 0 || b < a || b > prm.R;
        }
        if (bad) report_error(prm.err, ERR_BAD_INDEX);
      }
    }
    begun = false;
    p = 0;
    gbase = 0;
    if (prm.P == 1) {  // (nobody reads `base` then)
      g = prefix_group(prm, 0);
      const PrefixCut cut = prefix_cut_one(prm, g);
      extra = (short)cut.extra;
      range(cut, block);
      return;
    }
    const PrefixGroup mine = prefix_group(prm, min(lane, prm.P - 1));
    auto group = [&](int i) { return i < 32 ? mine : prefix_group(prm, i); };  // a lane's own
    long long S = 0, jobs = 0;
    for (int i = lane; i < prm.P; i += 32) {
      const PrefixGroup x = group(i);
      jobs += group_jobs(prm, x);
      S += group_jobs(prm, x) * x.steps;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      jobs += __shfl_xor_sync(0xffffffffu, jobs, o);
    }
    const PrefixCut cut = prefix_cut(prm, S, jobs, [&](long long len) {
      bool even = true;
      for (int i = lane; i < prm.P; i += 32) {
        const PrefixGroup x = group(i);
        even = even && (x.tiles == 0 || quotient(x.steps, len) * len == x.steps);
      }
      return (bool)__all_sync(0xffffffffu, even);
    });
    extra = (short)cut.extra;
    range(cut, block);
    if (record && lane == 0) {
      prm.base[prm.P] = cut.S;
      prm.base[prm.P + 1] = extra;
    }
    if (at >= end && !record) return;
    // the group that holds position `at`
    long long before = 0;
    bool found = false;
    for (int i0 = 0; i0 < prm.P && !(found && !record); i0 += 32) {
      const int i = i0 + lane;
      long long s = 0;
      if (i < prm.P) {
        const PrefixGroup x = group(i);
        s = group_jobs(prm, x) * (x.steps + extra);
      }
      long long x = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (record && i < prm.P) prm.base[i] = before + x - s;
      const unsigned past = __ballot_sync(0xffffffffu, before + x > at);
      if (past && !found) {
        const int l = __ffs(past) - 1;
        p = i0 + l;
        gbase = before + __shfl_sync(0xffffffffu, x - s, l);
        found = true;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    g = prefix_group(prm, p);
  }

  __device__ __forceinline__ void range(const PrefixCut& cut, int block) {
    at = end = 0;
    if (block >= cut.blocks) return;
    at = cut.start(block);
    end = cut.start(block + 1);
  }

  // Moves to the next segment; false at the end of the range.
  __device__ __forceinline__ bool next(const PrefixParams& prm, int block) {
    if (at >= end) return false;
    long long job, off;  // of the group; position in the job
    for (;;) {
      const long long span = g.steps + extra;
      const long long all = group_jobs(prm, g) * span;
      if (at >= gbase + all) {
        gbase += all;
        g = prefix_group(prm, ++p);  // at < end <= the line's length: a later group holds it
        continue;
      }
      job = quotient(at - gbase, span);
      off = at - gbase - job * span;
      if (off >= extra) break;
      at = min(end, at + extra - off);  // the empty steps
      if (at == end) return false;
    }
    head = (int)quotient(job, g.tiles);
    tile = (int)(job - (long long)head * g.tiles);
    k0 = (int)(off - extra);
    k1 = (int)min((long long)g.steps, k0 + (end - at));
    slot = (k0 == 0 && k1 == g.steps) ? -1 : 2 * block + (begun ? 1 : 0);
    begun = true;
    at += k1 - k0;
    return true;
  }
};

// One (row, head): joins its prefix part (maximum m and sum l, log2 units; acc relative to m) with
// what the row attended on its own.  Returns the factors of acc and of the own output, and the
// joined log-sum-exp (natural).  Rows that nothing was attended for: both 0, -inf.  Without an
// own part (own = -inf) its factor is 0 whatever the prefix part holds, NaN included; where nothing
// was attended for in the prefix, the own part is returned as it is.
__device__ __forceinline__ void join_own(float m, float l, float own, float& f_acc, float& f_own, float& lse) {
  // prefix part: weight l at scale 2^m; own part: weight 1 at scale 2^(own log2 e), which is finite where own is
  // (a mask of the type's lowest value may stand behind it)
  float mo = own * LOG2E;
  if (fabsf(own) <= FLT_MAX) mo = fminf(fmaxf(mo, -FLT_MAX), FLT_MAX);
  float M = fmaxf(m, mo);
  if (M == NEG_INF) M = 0.f;
  const float a = fast_exp2(m - M), b = own == NEG_INF ? 0.f : fast_exp2(mo - M);
  const float prefix = times_exp2(l, m - M), t = prefix + b;
  f_acc = t == 0.f ? 0.f : a / t;
  f_own = b == 0.f ? 0.f : b / t;
  lse = prefix == 0.f ? own : (M + log2f(t)) * LN2;
}

// The tensor-core kernel (prefix_tc.cu): tiles of TC_ROWS rows, one block a SM.
constexpr int TC_ROWS = 256;
cudaError_t launch_prefix_tc(const PrefixParams& p, int d, cudaStream_t s);

}  // namespace pisa
