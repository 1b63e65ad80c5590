// kv4_attention.cu -- attention over the paged 4-bit cache.
//
// o = softmax(scale q k^T) v over the positions [0, len) of a sequence (causal: row j of n sees positions up to
// len - n + j), with k and v dequantised on the way to the tensor cores.  Statistics and sums are in fp32; the
// operands are fp16: k and v are exact in it (6 significant bits), q is made exact by a power of two per row,
// and p is rounded once, by 2^-11 of itself, or by 2^-32 (many rows) or 2^-40 (few) of the row's largest where that is
// more (reference_of); the row's sum takes it unrounded.
#include <math.h>

#include "kv4_attention.cuh"

namespace dg {

namespace {

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  // (volatile: no product, and so no load that it waits for, falls behind the copy that refills a slot)
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// ---------------------------------------------------------------------------------------------
// few rows: single tokens and other tiles of at most 8 rows of a KV head
// ---------------------------------------------------------------------------------------------
// A call of few units whose lengths cannot differ much runs a cluster for each unit, which joins its CTAs' rows through
// distributed shared memory in the same launch; others divide the line of all units evenly (kv4_attention.cuh) and
// join in a second launch.
//
// 4 warps; a warp takes every fourth page of the CTA's piece of a unit.  It keeps a ring of whole blocks in shared
// memory (one bulk copy each: a block is contiguous), dequantises them into m16n8k16 fragments and multiplies S = K
// Q^T and O^T += V^T P^T: positions and channels are the 16-wide side, the rows the 8-wide one, so a tile of 8 rows
// wastes no tensor work, and a row's statistics lie with the same lanes in S and in O^T.  Bound by the cache's bytes:
// mma.sync is enough, since 8 rows x 2 operations a value stay far below its rate.
constexpr int kFewWarps = 4;               // warps of a CTA; three CTAs an SM keep 24 blocks in flight
constexpr int kFewStages = 2;
constexpr int kMaxCluster = kKv4MaxCluster;
constexpr int kFewShift = 15;              // p in [0, 2^15]: its reference is the largest score met so far, less this

template <int DH>
struct FewSmem {
  alignas(16) uint8_t ring[kFewWarps][kFewStages][Kv4<DH>::kBytes];
  uint64_t full[kFewWarps][kFewStages];
  float m[kFewWarps][kKv4FewTile], l[kFewWarps][kKv4FewTile];
};

// Cluster: grid (tile, KV head, CTA of the cluster for each sequence); else the CTAs divide the line.
template <int DH, typename T, bool Cluster>
__global__ void __launch_bounds__(32 * kFewWarps, kv4_few_ctas(DH))
    kv4_attend_few_kernel(Kv4View c, int layer, Kv4Attn a) {
  using F = Kv4<DH>;
  constexpr int NJ = DH / 16;            // 16-channel steps of a row
  extern __shared__ __align__(16) uint8_t smem_raw[];
  FewSmem<DH>& sm = *reinterpret_cast<FewSmem<DH>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_trigger();
  if (lane == 0) {
    for (int s = 0; s < kFewStages; ++s) mbar_init(&sm.full[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait();

  const int G = a.group;
  const Unit unit = Cluster ? cluster_unit() : Unit{0, 0, 0, 0, 1};
  int phase = 0;                // copies that each stage of the ring has seen, one bit each: its barrier's parity
  bool ok = true;
  // one piece of work
  auto work = [&](const Piece& pc) {
    const int seq = pc.seq, head = pc.head;
    const SeqView sv = pc.v;
    const int r0 = pc.tile * kKv4FewTile;         // row r of the group: query row r / G, head r % G of the group
    const int nr = min(kKv4FewTile, sv.n * G - r0);
    const int limit = row_limit(sv, group_row(a, r0 + nr - 1), a.causal);   // the tile's last row sees the most
    const int all = row_limit(sv, group_row(a, r0), a.causal);                // every row sees positions below this
    const int p0 = pc.s0, p1 = min((limit + kPage - 1) / kPage, pc.s1);
    const int n_mine = p1 - p0 > warp ? (p1 - p0 - warp + kFewWarps - 1) / kFewWarps : 0;

    // page i of this warp: p0 + warp + 4 i; ids are read 32 at a time, one a lane
    const int32_t* table = c.table + (size_t)seq * c.max_pages + p0 + warp;
    int ids = 0;
    auto page_id = [&](int i) {   // whole warp, i ascending
      if ((i & 31) == 0) {
        ids = -1;
        if (i + lane < n_mine) {
          ids = table[(i + lane) * kFewWarps];
          if (ids < 0 || ids >= c.n_pages) {
            report_error(c.head, DEV_ERR_BAD_INDEX);
            ids = -1;
          }
        }
      }
      return __shfl_sync(0xffffffffu, ids, i & 31);
    };
    const uint8_t* plane = c.pool + ((size_t)layer * c.n_pages * c.n_kv + head) * F::kBytes;
    auto fetch = [&](int i) {     // whole warp: start the copy of its page i; a page that is not there is not copied
      const int id = page_id(i);
      if (lane == 0) {
        uint64_t* bar = &sm.full[warp][i % kFewStages];
        if (id >= 0) {
          mbar_arrive_expect_tx(bar, F::kBytes);
          bulk_load(bar, sm.ring[warp][i % kFewStages], plane + (size_t)id * c.n_kv * F::kBytes, F::kBytes);
        } else {
          mbar_arrive(bar);
        }
      }
      return id >= 0;
    };
    uint32_t present = 0;         // by stage
    for (int i = 0; i < kFewStages && i < n_mine; ++i) present |= (uint32_t)fetch(i) << i;

    // Q fragments: row g, channels DH/4 t + 4 j + {0..3}, times a power of two that makes them exact in fp16
    uint32_t qf[NJ][2];
    float fac[2];                 // rows 2t, 2t + 1: scale log2(e) and the power of two taken out
    {
      const int r = r0 + g, qj = group_row(a, r);
      float x[DH / 4];
#pragma unroll
      for (int i = 0; i < DH / 4; ++i) x[i] = 0.f;
      if (g < nr) {
        const T* q = static_cast<const T*>(a.q) + seq * a.q_seq + qj * a.q_row + (head * G + r - qj * G) * a.q_head +
                     DH / 4 * t;
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(q)[i];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[8 * i + 2 * e] = Half<T>::lo(w[e]);
            x[8 * i + 2 * e + 1] = Half<T>::hi(w[e]);
          }
        }
      }
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < DH / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float down, up;
      row_powers(amax, down, up);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        qf[j][0] = pack_f16x2(x[4 * j] * down, x[4 * j + 1] * down);
        qf[j][1] = pack_f16x2(x[4 * j + 2] * down, x[4 * j + 3] * down);
      }
      const float f = a.scale * 1.4426950408889634f * up;
      fac[0] = __shfl_sync(0xffffffffu, f, 8 * t);
      fac[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
    int lim[2];                   // positions that rows 2t, 2t + 1 see
#pragma unroll
    for (int e = 0; e < 2; ++e) lim[e] = 2 * t + e < nr ? row_limit(sv, group_row(a, r0 + 2 * t + e), a.causal) : 0;

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[NJ][4];               // O^T: channels DH/8 g + 2 j + {0, 1}, rows 2t, 2t + 1
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    int i = 0;
    for (; i < n_mine; ++i) {
      const int st = i % kFewStages;
      ok = warp_wait(&sm.full[warp][st], (phase >> st) & 1, c.head + KV4_WORD_WAIT);
      if (!ok) break;
      phase ^= 1 << st;
      const bool here = (present >> st) & 1;
      const int base = (p0 + warp + i * kFewWarps) * kPage;
      if (here) {
        const uint8_t* block = sm.ring[warp][st];
        float s[4][4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.f;
        uint32_t sw[4];   // scales of positions g and g + 8 of each tile, kH blocks each
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          const uint8_t* sc = block + F::kSk + lane * 8 * F::kH + 2 * kt * F::kH;
          sw[kt] = F::kH == 2 ? *reinterpret_cast<const uint32_t*>(sc) : *reinterpret_cast<const uint16_t*>(sc);
        }
        // the four tiles side by side: four independent chains of products
#pragma unroll
        for (int jh = 0; jh < F::kH; ++jh) {
          uint32_t w[4][4];
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) {
            const uint4 q = *reinterpret_cast<const uint4*>(block + ((kt * F::kH + jh) * 32 + lane) * 16);
            w[kt][0] = q.x;
            w[kt][1] = q.y;
            w[kt][2] = q.z;
            w[kt][3] = q.w;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
              uint32_t s0, s1;
              if constexpr (F::kH == 2) {
                s0 = jh ? scale_pair<1, 1>(sw[kt]) : scale_pair<0, 0>(sw[kt]);
                s1 = jh ? scale_pair<3, 3>(sw[kt]) : scale_pair<2, 2>(sw[kt]);
              } else {
                s0 = scale_pair<0, 0>(sw[kt]);
                s1 = scale_pair<1, 1>(sw[kt]);
              }
              uint32_t f[4];
              e2m1_to_f16(w[kt][j], f);
              const uint32_t af[4] = {mul_f16x2(f[0], s0), mul_f16x2(f[1], s1), mul_f16x2(f[2], s0),
                                      mul_f16x2(f[3], s1)};
              mma_16816(s[kt], af, qf[4 * jh + j][0], qf[4 * jh + j][1]);
            }
        }
        // base-2 scores, masked; the block's row maxima over the positions (lanes with the same t)
        float top[2] = {-INFINITY, -INFINITY};
        const bool whole = base + kPage <= all && nr == kKv4FewTile;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = s[kt][e] * fac[e & 1];
            if (!whole && base + kt * 16 + g + 8 * (e >> 1) >= lim[e & 1]) v = -INFINITY;
            s[kt][e] = v;
            top[e & 1] = max_nan(top[e & 1], v);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = max_nan(top[e], __shfl_xor_sync(0xffffffffu, top[e], 4));
          top[e] = max_nan(top[e], __shfl_xor_sync(0xffffffffu, top[e], 8));
          top[e] = reference_of<kFewShift>(max_nan(top[e], __shfl_xor_sync(0xffffffffu, top[e], 16)));
        }
        // (references follow the largest scores in the same order)
        const float n0 = max_nan(m[0], top[0]), n1 = max_nan(m[1], top[1]);   // (a NaN score makes its row NaN)
        if (__any_sync(0xffffffffu, n0 != m[0] || n1 != m[1])) {
          const float f0 = n0 == m[0] ? 1.f : fast_exp2(m[0] - n0), f1 = n1 == m[1] ? 1.f : fast_exp2(m[1] - n1);
          l[0] *= f0;
          l[1] *= f1;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            o[j][0] *= f0;
            o[j][1] *= f1;
            o[j][2] *= f0;
            o[j][3] *= f1;
          }
          m[0] = n0;
          m[1] = n1;
        }
        // a row that sees nothing yet keeps m = -inf: its scores are -inf, its p 0
        const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
        uint32_t pf[4][2];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          const float q0 = fast_exp2(s[kt][0] - b0), q1 = fast_exp2(s[kt][1] - b1);
          const float q2 = fast_exp2(s[kt][2] - b0), q3 = fast_exp2(s[kt][3] - b1);
          l[0] += q0 + q2;
          l[1] += q1 + q3;
          pf[kt][0] = transpose_8x8(pack_f16x2(q0, q1));   // [position g][row 2t, 2t+1] -> [row g][positions 2t, 2t+1]
          pf[kt][1] = transpose_8x8(pack_f16x2(q2, q3));
        }
        const int left = sv.len - base;   // V of positions at or beyond the length is stale: its scale becomes 0
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          const int blk = F::kH == 2 ? g : g >> 1;
          uint32_t sw = *reinterpret_cast<const uint32_t*>(block + F::kSv + (blk * 4 + t) * 16 + 4 * kt);
          if (left < kPage) {
            const int pos = kt * 16 + 2 * t;
            uint32_t keep = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) keep |= pos + (e & 1) + 8 * (e >> 1) < left ? 0xffu << (8 * e) : 0u;
            sw &= keep;
          }
          const uint32_t s01 = scale_pair<0, 1>(sw), s23 = scale_pair<2, 3>(sw);
#pragma unroll
          for (int jh = 0; jh < F::kH; ++jh) {
            const uint4 q = *reinterpret_cast<const uint4*>(block + F::kV + ((kt * F::kH + jh) * 32 + lane) * 16);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t f[4];
              e2m1_to_f16(w[j], f);
              const uint32_t af[4] = {mul_f16x2(f[0], s01), mul_f16x2(f[1], s01), mul_f16x2(f[2], s23),
                                      mul_f16x2(f[3], s23)};
              mma_16816(o[4 * jh + j], af, pf[kt][0], pf[kt][1]);
            }
          }
        }
      }
      if (!here) m[0] = m[1] = NAN;   // a page that is none: the rows that it belongs to are not to be taken for whole
      __syncwarp();   // every lane has read the stage
      if (i + kFewStages < n_mine) {
        const bool again = fetch(i + kFewStages);
        present = (present & ~(1u << st)) | ((uint32_t)again << st);
      }
    }
    // (a wait that ran out: the error word tells; the copies still in flight land in this CTA's memory, so wait on)
    for (int k = i; k < n_mine && k < i + kFewStages; ++k)
      mbar_wait(&sm.full[warp][k % kFewStages], (phase >> (k % kFewStages)) & 1, nullptr, 0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
    }
    // join the warps: O [warp][row][channel] in the warp's own stages
    float* po = reinterpret_cast<float*>(sm.ring[warp][0]);
    float* part = reinterpret_cast<float*>(sm.ring[0][1]);   // a cluster's CTA: its joined rows
    float* part_lse = part + kKv4FewTile * DH;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) po[(2 * t + (e & 1)) * DH + DH / 8 * g + 2 * j + (e >> 1)] = o[j][e];
    if (g == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sm.m[warp][2 * t + e] = m[e];
        sm.l[warp][2 * t + e] = l[e];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nr * (DH / 2); i += 32 * kFewWarps) {
      const int row = i / (DH / 2), ch = i % (DH / 2) * 2;
      float top = sm.m[0][row];
#pragma unroll
      for (int w = 1; w < kFewWarps; ++w) top = max_nan(top, sm.m[w][row]);
      float den = 0.f, v0 = 0.f, v1 = 0.f;
      if (top != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
          const float f = fast_exp2(sm.m[w][row] - top);
          const float2 x = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(sm.ring[w][0]) + row * DH + ch);
          den += f * sm.l[w][row];
          v0 += f * x.x;
          v1 += f * x.y;
        }
        v0 /= den;
        v1 /= den;
      }
      // (the shift in both terms, so that their rounding is that of the score and of a sum from its largest)
      const float lse2 = top == -INFINITY ? -INFINITY : top + kFewShift + log2f(den * (1.f / (1 << kFewShift)));
      const int r = r0 + row, j = group_row(a, r), h = head * G + r - j * G;
      if (Cluster && unit.n > 1) {
        *reinterpret_cast<float2*>(part + row * DH + ch) = make_float2(v0, v1);
        if (ch == 0) part_lse[row] = lse2;
      } else if (pc.whole()) {
        T* dst = static_cast<T*>(a.out) + seq * a.o_seq + j * a.o_row + h * a.o_head + ch;
        *reinterpret_cast<uint32_t*>(dst) = Half<T>::pack(v0, v1);
        if (a.lse && ch == 0) a.lse[((size_t)seq * a.rows + j) * a.n_q + h] = lse2 * 0.6931471805599453f;
      } else {
        const size_t at = slot_of(pc) * kKv4FewTile + row;
        *reinterpret_cast<float2*>(static_cast<float*>(a.part_o) + at * DH + ch) = make_float2(v0, v1);
        if (ch == 0) a.part_lse[at] = lse2;
      }
    }
    if (Cluster && unit.n > 1) {
      // every CTA of the cluster joins its share of the rows' channel pairs from all of them
      cluster_sync();
      const int n = unit.n;
      const uint32_t o_addr = smem_u32(part), lse_addr = smem_u32(part_lse);
      for (int i = unit.rank * 32 * kFewWarps + threadIdx.x; i < nr * (DH / 2); i += n * 32 * kFewWarps) {
        const int row = i / (DH / 2), ch = i % (DH / 2) * 2;
        float le[kMaxCluster];
        float2 x[kMaxCluster];
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          le[k] = k < n ? dsmem_ld_f1(dsmem_map(lse_addr + 4 * row, k)) : -INFINITY;
          x[k] = k < n ? dsmem_ld_f2(dsmem_map(o_addr + 4 * (row * DH + ch), k)) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) top = max_nan(top, le[k]);
        float den = 0.f, v0 = 0.f, v1 = 0.f;
        if (top != -INFINITY) {
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k) {
            const float f = k < n ? fast_exp2(le[k] - top) : 0.f;
            den += f;
            v0 += f * x[k].x;
            v1 += f * x[k].y;
          }
          v0 /= den;
          v1 /= den;
        }
        const int r = r0 + row, j = group_row(a, r), h = head * G + r - j * G;
        T* dst = static_cast<T*>(a.out) + seq * a.o_seq + j * a.o_row + h * a.o_head + ch;
        *reinterpret_cast<uint32_t*>(dst) = Half<T>::pack(v0, v1);
        if (a.lse && ch == 0)
          a.lse[((size_t)seq * a.rows + j) * a.n_q + h] =
              (top == -INFINITY ? -INFINITY : top + log2f(den)) * 0.6931471805599453f;
      }
      cluster_sync();   // this CTA's rows stay until all have read them
    }
  };
  if constexpr (Cluster) {
    Piece pc;
    pc.tile = unit.tile;
    pc.head = unit.head;
    pc.seq = unit.seq;
    pc.v = seq_view(c, a, pc.seq, threadIdx.x == 0);
    if (pc.tile * kKv4FewTile >= pc.v.n * G) return;   // (the whole cluster)
    const int pages = (pc.v.len + kPage - 1) / kPage;
    const int per = (pages + unit.n - 1) / unit.n;
    pc.cost = max(1, pages);
    pc.s0 = unit.n == 1 ? 0 : min(pages, unit.rank * per);
    pc.s1 = unit.n == 1 ? pc.cost : min(pages, pc.s0 + per);
    pc.first = true;
    work(pc);
  } else {
    Stretch<kKv4FewTile, kKv4FewStep> stretch(c, a, blockIdx.x == 0 && warp == 0);
    Piece pc;
    while (stretch.next(pc)) {
      work(pc);
      fence_proxy_async_smem();            // (rows were joined in the rings: before the next copies into them)
      if (!__syncthreads_and(ok)) break;   // (the rings are free again; a warp that gave up has told)
    }
  }
}

// ---------------------------------------------------------------------------------------------
// joining the splits: one warp for each (sequence, row, head)
// ---------------------------------------------------------------------------------------------
// Each piece left its normalised row and base-2 log-sum-exp; the row is their mean with weights 2^(lse - max).  The
// pieces of a unit are those of the CTAs whose stretches meet it: the first CTA's last piece, then first pieces.
struct Pieces {
  int c0, c1;      // CTAs; one alone has written the row out itself
  size_t first;    // slot of CTA c0's piece
  __device__ __forceinline__ size_t slot(int cta) const { return cta == c0 ? first : 2 * (size_t)cta; }
};
template <int TILE, int STEP>
__device__ __forceinline__ Pieces pieces_of(const Kv4View& c, const Kv4Attn& a, int seq, const SeqView& v, int head,
                                            int tile) {
  const SeqWork<TILE, STEP> w(v, a.group);
  const long long share = reinterpret_cast<const LineHeader*>(a.line)->share;
  const long long start = line_base(a.line)[seq] + ((long long)head * w.tiles + tile) * w.cost;
  Pieces p;
  p.c0 = (int)line_div(start, share);
  p.c1 = (int)line_div(start + w.cost - 1, share);
  p.first = 2 * (size_t)p.c0 + (start != p.c0 * share ? 1 : 0);
  return p;
}

// few rows: a CTA for each (sequence, row, head), whose warps share out the pieces (one token behind 32768 positions
// has 56 a row: one warp walking them spent 4 us waiting for its loads)
constexpr int kMergeWarps = 8;
template <int DH, typename T>
__global__ void __launch_bounds__(32 * kMergeWarps) kv4_merge_few_kernel(Kv4View c, Kv4Attn a) {
  pdl_trigger();
  pdl_wait();
  constexpr int kPer = DH / 32;
  __shared__ float tops[kMergeWarps], dens[kMergeWarps], accs[kMergeWarps][DH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.group;
  const int h = blockIdx.x % a.n_q, j = blockIdx.x / a.n_q % a.rows, seq = blockIdx.x / a.n_q / a.rows;
  const SeqView v = seq_view(c, a, seq);
  if (j >= v.n) return;
  const int r = j * G + h % G;
  const Pieces p = pieces_of<kKv4FewTile, kKv4FewStep>(c, a, seq, v, h / G, r / kKv4FewTile);
  if (p.c0 == p.c1) return;
  const size_t row = r % kKv4FewTile;
  // this warp's pieces c0 + warp, c0 + warp + 8, ...: running maximum, eight at a time
  float top = -INFINITY, den = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int s0 = p.c0 + warp; s0 <= p.c1; s0 += 8 * kMergeWarps) {
    float le[8], x[8][kPer];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = s0 + k * kMergeWarps;
      le[k] = -INFINITY;
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[k][e] = 0.f;
      if (s <= p.c1) {
        const size_t slot = p.slot(s) * kKv4FewTile + row;
        le[k] = a.part_lse[slot];
        const float* src = static_cast<const float*>(a.part_o) + slot * DH + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
          const float2 y = *reinterpret_cast<const float2*>(src + e);
          x[k][e] = y.x;
          x[k][e + 1] = y.y;
        }
      }
    }
    float now = top;
#pragma unroll
    for (int k = 0; k < 8; ++k) now = max_nan(now, le[k]);
    if (now == -INFINITY) continue;
    const float keep = fast_exp2(top - now);
    den *= keep;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= keep;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = fast_exp2(le[k] - now);
      den += f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += f * x[k][e];
    }
    top = now;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) accs[warp][lane * kPer + e] = acc[e];
  if (lane == 0) {
    tops[warp] = top;
    dens[warp] = den;
  }
  __syncthreads();
  for (int ch = threadIdx.x * 2; ch < DH; ch += 64 * kMergeWarps) {
    float m = tops[0], d = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) m = max_nan(m, tops[w]);
    if (m != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float f = fast_exp2(tops[w] - m);
        d += f * dens[w];
        v0 += f * accs[w][ch];
        v1 += f * accs[w][ch + 1];
      }
    }
    const float inv = d == 0.f ? 0.f : 1.f / d;
    T* dst = static_cast<T*>(a.out) + seq * a.o_seq + j * a.o_row + h * a.o_head + ch;
    *reinterpret_cast<uint32_t*>(dst) = Half<T>::pack(v0 * inv, v1 * inv);
    if (a.lse && ch == 0) a.lse[((size_t)seq * a.rows + j) * a.n_q + h] = (m + log2f(d)) * 0.6931471805599453f;
  }
}

// many rows: a CTA for 64 group rows of a (sequence, KV head); thread = (row, pair of 8-channel chunks): loads of the
// same chunk by neighbouring rows are contiguous
constexpr int kMergeRows = 64;
template <int DH, typename T>
__global__ void __launch_bounds__(kMergeRows* DH / 16) kv4_merge_many_kernel(Kv4View c, Kv4Attn a) {
  pdl_trigger();
  pdl_wait();
  constexpr int kPer = kPartPer<T>;
  const int G = a.group;
  const int seq = blockIdx.z, head = blockIdx.y;
  const SeqView v = seq_view(c, a, seq);
  const int r = blockIdx.x * kMergeRows + threadIdx.x % kMergeRows, chunk = threadIdx.x / kMergeRows * 2;
  if (r >= v.n * G) return;
  const Pieces p = pieces_of<kKv4ManyTile, kKv4ManyStep>(c, a, seq, v, head, r / kKv4ManyTile);
  if (p.c0 == p.c1) return;
  const size_t row = r % kKv4ManyTile;
  const float2* stat = reinterpret_cast<const float2*>(a.part_lse);   // (lse, power of two)
  float top = -INFINITY;
#pragma unroll 8
  for (int s = p.c0; s <= p.c1; ++s) top = max_nan(top, stat[p.slot(s) * kKv4ManyTile + row].x);
  float acc[16], den = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  if (top != -INFINITY) {
#pragma unroll 4
    for (int s = p.c0; s <= p.c1; ++s) {
      const size_t slot = p.slot(s);
      const float2 st = stat[slot * kKv4ManyTile + row];
      const float f = fast_exp2(st.x - top), g = f * st.y;
      const uint4* src = static_cast<const uint4*>(a.part_o) +
                         (slot * (DH / kPer) + (size_t)chunk * (8 / kPer)) * kKv4ManyTile + row;
      den += f;
#pragma unroll
      for (int u = 0; u < 16 / kPer; ++u) {
        const uint4 y = src[u * kKv4ManyTile];
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kPer == 4) {
            acc[4 * u + e] += g * __uint_as_float(w[e]);
          } else {
            acc[8 * u + 2 * e] += g * Half<__half>::lo(w[e]);
            acc[8 * u + 2 * e + 1] += g * Half<__half>::hi(w[e]);
          }
        }
      }
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int j = group_row(a, r), h = head * G + r - j * G;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + seq * a.o_seq + j * a.o_row + h * a.o_head + chunk * 8);
#pragma unroll
  for (int u = 0; u < 2; ++u)
    dst[u] = make_uint4(Half<T>::pack(acc[8 * u] * inv, acc[8 * u + 1] * inv),
                        Half<T>::pack(acc[8 * u + 2] * inv, acc[8 * u + 3] * inv),
                        Half<T>::pack(acc[8 * u + 4] * inv, acc[8 * u + 5] * inv),
                        Half<T>::pack(acc[8 * u + 6] * inv, acc[8 * u + 7] * inv));
  if (a.lse && chunk == 0) a.lse[((size_t)seq * a.rows + j) * a.n_q + h] = (top + log2f(den)) * 0.6931471805599453f;
}

template <int DH, typename T>
cudaError_t launch_few(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st) {
  static unsigned long long done = 0;
  const cudaError_t e = once_per_device(&done, [] {
    cudaError_t e = cudaFuncSetAttribute(kv4_attend_few_kernel<DH, T, false>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(FewSmem<DH>));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv4_attend_few_kernel<DH, T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               sizeof(FewSmem<DH>));
    return e != cudaSuccess
               ? e
               : cudaFuncSetAttribute(kv4_attend_few_kernel<DH, T, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  if (a.cluster) {
    const int tiles = (a.rows * a.group + kKv4FewTile - 1) / kKv4FewTile;
    return launch_k(kv4_attend_few_kernel<DH, T, true>, dim3(tiles, c.n_kv, c.n_seq * a.cluster), dim3(32 * kFewWarps),
                    sizeof(FewSmem<DH>), st, a.cluster, c, layer, a);
  }
  return launch_k(kv4_attend_few_kernel<DH, T, false>, dim3(a.n_ctas), dim3(32 * kFewWarps),
                  sizeof(FewSmem<DH>), st, 1,
                  c, layer, a);
}

template <int DH, typename T>
cudaError_t launch_merge(const Kv4View& c, const Kv4Attn& a, bool few, cudaStream_t st) {
  if (few) {
    const size_t rows = (size_t)c.n_seq * a.rows * a.n_q;
    return launch_k(kv4_merge_few_kernel<DH, T>, dim3((unsigned)rows), dim3(32 * kMergeWarps), 0, st, 1, c, a);
  }
  const dim3 grid((a.rows * a.group + kMergeRows - 1) / kMergeRows, c.n_kv, c.n_seq);
  return launch_k(kv4_merge_many_kernel<DH, T>, grid, dim3(kMergeRows * DH / 16), 0, st, 1, c, a);
}

}  // namespace

cudaError_t kv4_attend_few(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st) {
  if (c.dh == 128)
    return a.fp16 ? launch_few<128, __half>(c, layer, a, st) : launch_few<128, __nv_bfloat16>(c, layer, a, st);
  return a.fp16 ? launch_few<64, __half>(c, layer, a, st) : launch_few<64, __nv_bfloat16>(c, layer, a, st);
}

cudaError_t kv4_attend_merge(const Kv4View& c, const Kv4Attn& a, bool few, cudaStream_t st) {
  if (c.dh == 128)
    return a.fp16 ? launch_merge<128, __half>(c, a, few, st) : launch_merge<128, __nv_bfloat16>(c, a, few, st);
  return a.fp16 ? launch_merge<64, __half>(c, a, few, st) : launch_merge<64, __nv_bfloat16>(c, a, few, st);
}

}  // namespace dg
