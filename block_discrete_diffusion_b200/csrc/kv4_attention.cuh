// kv4_attention.cuh -- what the two forms of attention over the 4-bit cache share: how the work is divided among the
// CTAs, what a row sees, and the rows left for joining.
//
// A unit of work is (sequence, KV head, tile of query rows) with a cost of its key steps.  Lengths are known on the
// device only and differ, so the units are laid end to end and every CTA takes an equal stretch of the line: it may
// finish one unit, take several whole, and begin another.  A unit that lies within one stretch is written out
// directly; a stretch's first and last pieces may be parts, which go to the CTA's two slots of the workspace, and
// the merge kernel joins them.  Equal stretches keep all SMs busy to the end whatever the lengths are; a fixed
// number of splits for each sequence left them waiting for the longest one.
#pragma once

#include "kv4.cuh"
#include "kv4_kernels.h"

namespace dg {

struct SeqView {
  int len, n;   // positions, query rows
};

// A sequence's length and row count; nothing to do for one whose counts do not fit (each kernel reports them once).
__device__ __forceinline__ SeqView seq_view(const Kv4View& c, const Kv4Attn& a, int seq, bool report = false) {
  SeqView v;
  v.len = c.lens[seq];
  v.n = a.n_rows ? a.n_rows[seq] : a.rows;
  if (v.len < 0 || (long long)v.len > (long long)c.max_pages * kPage || v.n < 0 || v.n > a.rows) {
    if (report) report_error(c.head, DEV_ERR_BAD_COUNT);
    v.len = v.n = 0;
  }
  return v;
}

// positions that row j of n sees
__device__ __forceinline__ int row_limit(const SeqView& v, int j, int causal) {
  return causal ? max(0, min(v.len, v.len - v.n + j + 1)) : v.len;
}

// Units of one sequence: tiles of TILE rows of the group (row r of the group: query row r / G, head r % G of the
// group) for every KV head, each of `cost` steps of STEP positions (one step where there is nothing to see: the
// row still has to be written).
template <int TILE, int STEP>
struct SeqWork {
  int tiles, cost;
  __device__ __forceinline__ SeqWork(const SeqView& v, int G) {
    tiles = (int)(((long long)v.n * G + TILE - 1) / TILE);
    cost = max(1, (v.len + STEP - 1) / STEP);
  }
  __device__ __forceinline__ long long total(int n_kv) const { return (long long)tiles * n_kv * cost; }
};

// A CTA's stretch of the line: `left` steps from step `step` of unit `unit` of sequence `seq` on.
struct Stretch {
  long long left;
  int seq, unit, step;
  bool at_begin;   // the next piece is the stretch's first
};

// One piece: steps [s0, s1) of a unit of `cost` steps.
struct Piece {
  SeqView v;
  int seq, head, tile, s0, s1, cost;
  bool first;
  __device__ __forceinline__ bool whole() const { return s0 == 0 && s1 == cost; }
};

template <int TILE, int STEP>
__device__ __forceinline__ bool next_piece(const Kv4View& c, const Kv4Attn& a, Stretch& st, Piece& p) {
  const int G = a.n_q / c.n_kv;
  while (st.left > 0 && st.seq < c.n_seq) {
    p.v = seq_view(c, a, st.seq);
    const SeqWork<TILE, STEP> w(p.v, G);
    if (st.unit >= w.tiles * c.n_kv) {
      ++st.seq;
      st.unit = st.step = 0;
      continue;
    }
    p.seq = st.seq;
    p.head = st.unit / w.tiles;
    p.tile = st.unit % w.tiles;
    p.cost = w.cost;
    p.s0 = st.step;
    p.s1 = (int)min((long long)w.cost, st.step + st.left);
    p.first = st.at_begin;
    st.at_begin = false;
    st.left -= p.s1 - p.s0;
    st.step = 0;
    ++st.unit;
    return true;
  }
  return false;
}

// Line header in the workspace, for the merge kernel: base[s] is the line position of sequence s's first unit.
struct LineHeader {
  long long share;
};
__host__ __device__ __forceinline__ long long* line_base(void* line) {
  return reinterpret_cast<long long*>(line) + 2;
}

// Whole CTA of NT threads (a multiple of 32): this CTA's stretch.  CTA 0 also leaves the line's header.
template <int TILE, int STEP, int NT>
__device__ Stretch find_stretch(const Kv4View& c, const Kv4Attn& a) {
  __shared__ long long warp_sums[NT / 32];
  __shared__ Stretch found;
  const int G = a.n_q / c.n_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool lead = blockIdx.x == 0;
  auto cost = [&](int s) {
    if (s >= c.n_seq) return 0ll;
    return SeqWork<TILE, STEP>(seq_view(c, a, s, lead), G).total(c.n_kv);
  };
  // exclusive prefix over the CTA's threads, and their total
  auto scan = [&](long long v, long long& total) {
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    return before + s - v;
  };
  long long total = 0, part, mine = 0, at = 0;
  for (int s0 = 0; s0 < c.n_seq; s0 += NT) {
    mine = cost(s0 + threadIdx.x);
    at = total + scan(mine, part);
    total += part;
    if (lead && s0 + (int)threadIdx.x < c.n_seq) line_base(a.line)[s0 + threadIdx.x] = at;
  }
  const long long share = max((long long)a.min_share, (total + gridDim.x - 1) / gridDim.x);
  const long long begin = share * blockIdx.x;
  if (lead && threadIdx.x == 0) reinterpret_cast<LineHeader*>(a.line)->share = share;
  if (threadIdx.x == 0) found = Stretch{0, c.n_seq, 0, 0, true};
  __syncthreads();
  if (begin < total) {
    long long base = 0;
    for (int s0 = 0; s0 < c.n_seq; s0 += NT) {
      if (c.n_seq > NT) {   // (else `mine` and `at` still hold the only round)
        mine = cost(s0 + threadIdx.x);
        at = base + scan(mine, part);
        base += part;
      }
      if (mine > 0 && at <= begin && begin < at + mine) {
        const int s = s0 + threadIdx.x;
        const SeqWork<TILE, STEP> w(seq_view(c, a, s), G);
        found = Stretch{min(share, total - begin), s, (int)((begin - at) / w.cost), (int)((begin - at) % w.cost), true};
      }
    }
  }
  __syncthreads();
  return found;
}

// the workspace slot of a piece that is part of a unit
__device__ __forceinline__ size_t slot_of(const Piece& p) { return 2 * (size_t)blockIdx.x + (p.first ? 0 : 1); }

// Power of two that brings a row's largest magnitude between 2^14 and 2^15 (the exponent is kept where both
// powers are normal numbers): then fp16 holds the row exactly, down to 2^-39 of that magnitude.
__device__ __forceinline__ void row_powers(float amax, float& down, float& up) {
  const int e = min(253, max(15, (int)((__float_as_uint(amax) >> 23) & 255))) - 127;
  down = __uint_as_float((uint32_t)(141 - e) << 23);
  up = __uint_as_float((uint32_t)(113 + e) << 23);
}

}  // namespace dg
