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

#include <type_traits>

#include "kv4.cuh"
#include "kv4_kernels.h"

namespace dg {

struct SeqView {
  int len, n;   // positions, query rows
};

// a / b and a % b of line positions (64-bit division only where 32 bits do not do: it is a long routine)
__device__ __forceinline__ long long line_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// mbar_wait by a whole warp, which leaves it together: the lanes see a phase end at different polls, and what
// follows (tcgen05.ld and .st, products) must be reached by all of them at once.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, DEV_ERR_TIMEOUT_ATTN));
}

// bytes [src, src + bytes) of global memory to shared memory, counted on bar
__device__ __forceinline__ void bulk_load(uint64_t* bar, void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

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

// query row of row r of the group (r / group by a multiplication: r < 2^31; a division by a variable costs 150 cycles)
__device__ __forceinline__ int group_row(const Kv4Attn& a, int r) {
  return (int)((__umulhi((uint32_t)r, a.group_mul) + (uint32_t)r) >> a.group_shift);
}

// The unit of a cluster, from the grid (tile, KV head, CTAs of the cluster for each sequence); this CTA's rank of n.
struct Unit {
  int tile, head, seq, rank, n;
};
__device__ __forceinline__ Unit cluster_unit() {
  Unit u;
  u.tile = blockIdx.x;
  u.head = blockIdx.y;
  asm("mov.u32 %0, %%clusterid.z;" : "=r"(u.seq));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(u.rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(u.n));
  return u;
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

// One piece: steps [s0, s1) of a unit of `cost` steps.
struct Piece {
  SeqView v;
  int seq, head, tile, s0, s1, cost;
  bool first;   // the first of its CTA's stretch
  __device__ __forceinline__ bool whole() const { return s0 == 0 && s1 == cost; }
};

// Line header in the workspace, for the merge kernel: base[s] is the line position of sequence s's first unit.
struct LineHeader {
  long long share;
};
__host__ __device__ __forceinline__ long long* line_base(void* line) {
  return reinterpret_cast<long long*>(line) + 2;
}

// A CTA's stretch of the line, walked piece by piece.  Each warp walks it for itself, without shared memory or
// barriers: lane l holds the counts of sequence 32 w + l of the current window, so a window costs one round of loads.
template <int TILE, int STEP>
struct Stretch {
  const Kv4View& c;
  const Kv4Attn& a;
  int G, lane;
  SeqView mine;            // counts of sequence window + lane
  int window;
  long long left;          // steps that the stretch still has
  int seq, unit, step;     // where it goes on
  bool at_begin;

  __device__ __forceinline__ void load(int w, bool report = false) {
    window = w;
    mine = SeqView{0, 0};
    if (w + lane < c.n_seq) mine = seq_view(c, a, w + lane, report);
  }
  __device__ __forceinline__ long long cost_of_mine() const {
    return SeqWork<TILE, STEP>(mine, G).total(c.n_kv);
  }
  // exclusive prefix of v over the lanes; the sum in `total`
  __device__ __forceinline__ long long scan(long long v, long long& total) const {
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    return s - v;
  }

  // Whole warp.  `lead`: the one warp of the grid that leaves the header and reports counts that do not fit.
  __device__ __forceinline__ Stretch(const Kv4View& c_, const Kv4Attn& a_, bool lead)
      : c(c_), a(a_), G(a_.group), lane(threadIdx.x & 31), left(0), seq(c_.n_seq), unit(0), step(0),
        at_begin(true) {
    long long total = 0, part, at = 0;
#pragma unroll 1
    for (int w = 0; w < c.n_seq; w += 32) {
      load(w, lead);
      at = total + scan(cost_of_mine(), part);
      total += part;
      if (lead && w + lane < c.n_seq) line_base(a.line)[w + lane] = at;
    }
    const long long share = max((long long)a.min_share, line_div(total + gridDim.x - 1, gridDim.x));
    const long long begin = share * blockIdx.x;
    if (lead && lane == 0) reinterpret_cast<LineHeader*>(a.line)->share = share;
    if (begin >= total) return;
    left = min(share, total - begin);
    long long base = 0;
#pragma unroll 1
    for (int w = 0; w < c.n_seq; w += 32) {
      if (c.n_seq > 32) {   // (else `mine` and `at` still hold the only window)
        load(w);
        at = base + scan(cost_of_mine(), part);
        base += part;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, at <= begin && begin < at + cost_of_mine());
      if (hit) {
        const int l = __ffs(hit) - 1;
        const long long off = begin - __shfl_sync(0xffffffffu, at, l);
        const int cost = max(1, (__shfl_sync(0xffffffffu, mine.len, l) + STEP - 1) / STEP);
        seq = w + l;
        unit = (int)line_div(off, cost);
        step = (int)(off - (long long)unit * cost);
        return;
      }
    }
  }

  __device__ __forceinline__ bool next(Piece& p) {
    while (left > 0 && seq < c.n_seq) {
      if (seq >= window + 32) load(seq & ~31);
      p.v.len = __shfl_sync(0xffffffffu, mine.len, seq & 31);
      p.v.n = __shfl_sync(0xffffffffu, mine.n, seq & 31);
      const SeqWork<TILE, STEP> w(p.v, G);
      if (unit >= w.tiles * c.n_kv) {
        ++seq;
        unit = step = 0;
        continue;
      }
      p.seq = seq;
      p.head = unit / w.tiles;
      p.tile = unit % w.tiles;
      p.cost = w.cost;
      p.s0 = step;
      p.s1 = (int)min((long long)w.cost, step + left);
      p.first = at_begin;
      at_begin = false;
      left -= p.s1 - p.s0;
      step = 0;
      ++unit;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ float2 dsmem_ld_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float dsmem_ld_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void dsmem_st_f2(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void dsmem_st4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The reference of a row's weights: p = 2^(s - reference), in fp16 for the product with v.  A reference 2^-Shift below
// the row's largest score uses the upper part of fp16's range, so that small weights, of which a long context may have
// many, keep their bits down to 2^-(14 + Shift) of the largest and a value down to 2^-(25 + Shift).  Shift is left out of
// sums and statistics by itself, since these count from the reference.  Beyond 2^20 fp32 scores lie too far apart for it.
template <int Shift>
__device__ __forceinline__ float reference_of(float top) {
  return fabsf(top) < 1048576.f ? top - (float)Shift : top;
}

// Channels in a 16-byte chunk of a part of the many-rows form: fp16 for a bf16 output, fp32 for an fp16 one.
template <typename T>
constexpr int kPartPer = std::is_same<T, __half>::value ? 4 : 8;

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
