// kv4_canvas.cu -- attention over the paged 4-bit cache for many rows: canvases and prompt chunks, on tcgen05.
//
// A CTA works on 256 rows of a KV head (two 128-row tiles) and steps of one page, so each dequantised page serves
// 256 rows.  Warp roles (512 threads):
//   warps 0-3    softmax of tile 0, warps 4-7 softmax of tile 1 (thread = row): Q into shared memory, S from TMEM,
//                P = 2^(S - m) in fp16 back into S's columns of TMEM, running sum, the finished row out
//   warps 8-11   dequantise: pages' blocks from a ring of three in shared memory to fp16 K and V tiles in the 128-byte
//                swizzled layout of the tensor core, a ring of eight
//   warp 12      issues the products of tile 0, warp 15 those of tile 1: S = Q K^T of a step, O += P V of the step two
//                before
//   warp 13      walks the CTA's stretch and hands its pieces to the others, up to four ahead
//   warp 14      copies the pages' blocks into their ring, one bulk copy each
//
// Two S of 64 columns a tile fill TMEM beside the two O, so while a tile's exponentials of one step run, its next S is
// there already and the tensor core works on the other products; with one S of 128 columns each tile waited for its
// products and then they for it (5000 cycles for 128 positions, of which 2200 of products and 2050 of exponentials).
// P as the tensor core's operand in TMEM and not in shared memory takes 128 KB off the 384 KB that 128 positions
// cost there; the blocks come by bulk copies because loads into registers were waited for by each tile's proxy fence.
//
// A call whose units fit the SMs in clusters runs one for each unit, whose CTAs each join a share of its rows, and
// the second launch falls away.  A row goes from TMEM into its place in the Q tile and from there in one piece into
// the shared memory of the CTA that joins it.  Such a call is a chain of latencies (one canvas behind 2048 positions:
// 19.4 us, 6 of them its six steps), so Q is copied asynchronously while the lengths are read, a thread scales a row
// of it from registers (1.5 us less than sixteen rounds of loads, shuffles and stores), and query rows are found without
// divisions by the group's size.
//
// The scale multiplies each code in fp16, exactly.  V's codes come in pairs of positions, so V is laid down with its
// positions in the order 16 t + 4 tile + (pair), which makes each lane's share contiguous; P's columns are stored in
// the same order, which only renames registers.  The running maximum is lazy: O and the sum are rescaled when a row's
// maximum has grown by more than 2^8; it is taken 2^7 low, so P stays below 2^15 and has most of fp16's range.
#include <math.h>

#include "kv4_attention.cuh"

namespace dg {

namespace {

constexpr int kManyThreads = 512;
// Registers a thread after the split of the launch's 4 x 128: two softmax groups, the dequantisers, the issuers.
constexpr int kRegsSoftmax = 152, kRegsDequant = 120, kRegsIssue = 88;
constexpr int kRegsLaunch = 128;
static_assert(2 * kRegsSoftmax + kRegsDequant + kRegsIssue <= 4 * kRegsLaunch,
              "register split above what the CTA was launched with");
constexpr int kRing = 8;       // fp16 tiles of 64 positions
constexpr int kRaw = 3;        // pages' blocks
constexpr float kLazy = 8.f;   // log2 units
constexpr int kManyShift = 7;  // log2 of P's largest value where the reference has just followed (reference_of)
constexpr float kFar = 1048576.f;   // a reference from here on is subtracted from rounded scores
constexpr int kMaxManyCluster = kKv4MaxManyCluster;

template <int DH>
struct ManySmem {
  static constexpr uint32_t kQ = 128u * DH * 2u;       // a Q tile
  static constexpr uint32_t kTile = 64u * DH * 2u;     // a K or V tile
  static constexpr size_t kBytes =
      1024 + 2 * kQ + kRing * kTile + kRaw * Kv4<DH>::kBytes + 640 + 8 * (256 + kMaxManyCluster);
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(kRing * kTile + kRaw * Kv4<DH>::kBytes >= (256u + kMaxManyCluster - 1) * DH * 4u,
                "the rings hold the rows in fp32 that a cluster's CTA joins: of each of n, 1/n of 256, rounded up");
};

// A piece of work as the roles need it.
struct Task {
  int seq, head, row0, nr;      // its rows: [row0, row0 + nr) of the sequence's group rows
  int s0, steps;                // its pages that some row sees: [s0, s0 + steps); steps < 0: no more pieces
  int len, n, whole, slot;
};
constexpr int kTasks = 4;
constexpr int kTaskReaders = 15;   // warps that read a task

struct ManyBars {
  uint64_t task_full[kTasks], task_empty[kTasks];
  Task task[kTasks];
  uint64_t q_full[2], s_full[2][2], p_ready[2][2], pv_done[2][2];   // by tile, by S buffer
  uint64_t kv_full[kRing], kv_empty[kRing], raw_full[kRaw], raw_empty[kRaw];
  int raw_there[kRaw];   // 0: the table names no page here: its scores are NaN, and so are the rows that see it
  uint64_t drained[2];    // a tile's products, after a wait that ran out
  uint32_t tmem, copies;  // (of blocks, started)
  int lost;               // a wait of this CTA ran out
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of packed words to this warp's lanes
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* r) {
  tmem_st32(taddr, reinterpret_cast<const float*>(r));
}
// D[tmem] (+)= A[tmem] * B[smem desc]^T, 16-bit inputs, fp32 accumulate; one thread issues.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive without release semantics: for tensor memory, whose accesses tcgen05.wait and tcgen05.fence order.
__device__ __forceinline__ void mbar_arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// kind::f16 with fp16 operands, fp32 accumulators, both K-major
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The reading end of the tasks, one for each warp.
struct Tasks {
  ManyBars* bars;
  int* err;
  uint32_t i = 0;
  __device__ __forceinline__ bool next(Task& t) {   // whole warp
    const int k = i % kTasks;
    if (!warp_wait(&bars->task_full[k], (i / kTasks) & 1, err)) {
      bars->lost = 1;
      return false;
    }
    t = bars->task[k];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->task_empty[k]);
    ++i;
    return t.steps >= 0;
  }
};

// Cluster: grid (tile, KV head, CTA of the cluster for each sequence); else the CTAs divide the line.
template <int DH, typename T, bool Cluster>
__global__ void __launch_bounds__(kManyThreads, 1) kv4_attend_many_kernel(Kv4View c, int layer, Kv4Attn a) {
  using F = Kv4<DH>;
  using C = ManySmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = base;
  uint8_t* kv_s = q_s + 2 * C::kQ;
  uint8_t* raw_s = kv_s + kRing * C::kTile;
  ManyBars* bars = reinterpret_cast<ManyBars*>(raw_s + kRaw * F::kBytes);
  // a cluster's CTA: its rows' lse and powers of two
  float2* stat_s = reinterpret_cast<float2*>(raw_s + kRaw * F::kBytes + 640);
  static_assert(sizeof(ManyBars) <= 640, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = c.head + KV4_WORD_WAIT;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->q_full[x], 4);
      mbar_init(&bars->drained[x], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->s_full[x][b], 1);
        mbar_init(&bars->pv_done[x][b], 1);
        mbar_init(&bars->p_ready[x][b], 4);
      }
    }
    for (int b = 0; b < kRing; ++b) {
      mbar_init(&bars->kv_full[b], 4);
      mbar_init(&bars->kv_empty[b], 2);   // both issuers
    }
    for (int k = 0; k < kRaw; ++k) {
      mbar_init(&bars->raw_full[k], 1);
      mbar_init(&bars->raw_empty[k], 4);
    }
    for (int k = 0; k < kTasks; ++k) {
      mbar_init(&bars->task_full[k], 1);
      mbar_init(&bars->task_empty[k], kTaskReaders);
    }
    fence_mbar_init();
    bars->lost = 0;
  }
  if (warp == 12) tmem_alloc(&bars->tmem, 512);   // tile x: S [128 x, +64) and [128 x + 64, +64), O [256 + 128 x, ..)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  pdl_wait();

  const int G = a.group;
  const Unit unit = Cluster ? cluster_unit() : Unit{0, 0, 0, 0, 1};
  Tasks tasks{bars, err};
  Task pc;
  bool ok = true;

  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDequant));
    // ------------------------------ dequantise ------------------------------
    // K: warp w takes the page's 16-position tile w.  V: tiles 2 hv + {0, 1} with hv = (w & 1) ^ (g & 1), so that the lanes of
    // a store meet different banks, and half w >> 1 of a lane's channels.
    const int w = warp - 8, g = lane >> 2, t = lane & 3;
    const int hv = (w & 1) ^ (g & 1);
    uint32_t item = 0, page = 0;                 // K and V tiles laid down, pages read so far
    while (tasks.next(pc)) {
      for (int i = 0; i < pc.steps; ++i, ++page) {
        const int left = pc.len - (pc.s0 + i) * kPage;   // positions of this page that exist
        const uint32_t slot = page % kRaw;
        ok = ok && warp_wait(&bars->raw_full[slot], (page / kRaw) & 1, err);
        const uint8_t* blk = raw_s + slot * F::kBytes;
        const bool there = ok && bars->raw_there[slot];
        uint4 k[F::kH];
        uint32_t v[2][2 * F::kH], ks, vs[2];
        {
          const uint8_t* s = blk + F::kSk + lane * 8 * F::kH + 2 * w * F::kH;
          ks = F::kH == 2 ? *reinterpret_cast<const uint32_t*>(s) : *reinterpret_cast<const uint16_t*>(s);
#pragma unroll
          for (int jh = 0; jh < F::kH; ++jh) {
            // (lanes t 2 and 3 take the channel halves in the other order, for the banks)
            const int jk = F::kH == 2 ? jh ^ (t >> 1) : 0;
            k[jh] = *reinterpret_cast<const uint4*>(blk + ((w * F::kH + jk) * 32 + lane) * 16);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int vt = 2 * hv + u;
            vs[u] = *reinterpret_cast<const uint32_t*>(blk + F::kSv + ((F::kH == 2 ? g : g >> 1) * 4 + t) * 16 + 4 * vt);
            if constexpr (F::kH == 2) {
              const uint4 q = *reinterpret_cast<const uint4*>(blk + F::kV + ((vt * 2 + (w >> 1)) * 32 + lane) * 16);
              v[u][0] = q.x;
              v[u][1] = q.y;
              v[u][2] = q.z;
              v[u][3] = q.w;
            } else {
              const uint2 q = *reinterpret_cast<const uint2*>(blk + F::kV + (vt * 32 + lane) * 16 + 8 * (w >> 1));
              v[u][0] = q.x;
              v[u][1] = q.y;
            }
          }
        }
        // a page that is not there: K is code 0 at scale NaN, V any code at scale 0
        if (!there) {
          ks = 0xffffffffu;
          vs[0] = vs[1] = 0;
#pragma unroll
          for (int jh = 0; jh < F::kH; ++jh) k[jh] = make_uint4(0, 0, 0, 0);
        }
        // ---- K ----
        {
          const int b = item % kRing;
          ok = ok && warp_wait(&bars->kv_empty[b], ((item / kRing) & 1) ^ 1, err);
          const int row = 16 * w + g;   // and row + 8
#pragma unroll
          for (int jh = 0; jh < F::kH; ++jh) {
            const int jk = F::kH == 2 ? jh ^ (t >> 1) : 0;
            uint32_t s0, s1;
            if constexpr (F::kH == 2) {
              const uint32_t two = jk ? ks >> 8 : ks;
              s0 = scale_pair<0, 0>(two);
              s1 = scale_pair<2, 2>(two);
            } else {
              s0 = scale_pair<0, 0>(ks);
              s1 = scale_pair<1, 1>(ks);
            }
            const uint32_t wd[4] = {k[jh].x, k[jh].y, k[jh].z, k[jh].w};
            const int plane64 = F::kH == 2 ? t >> 1 : 0;
            const int chunk0 = F::kH == 2 ? (t & 1) * 4 + 2 * jk : 2 * t;
            uint8_t* rp = kv_s + (size_t)b * C::kTile + plane64 * 8192 + row * 128;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t f0[4], f1[4];
              e2m1_to_f16(wd[2 * q], f0);
              e2m1_to_f16(wd[2 * q + 1], f1);
              const int off = ((chunk0 + q) ^ g) << 4;   // (row and row + 8 have the same swizzle)
              *reinterpret_cast<uint4*>(rp + off) = make_uint4(mul_f16x2(f0[0], s0), mul_f16x2(f0[2], s0),
                                                              mul_f16x2(f1[0], s0), mul_f16x2(f1[2], s0));
              *reinterpret_cast<uint4*>(rp + 1024 + off) = make_uint4(mul_f16x2(f0[1], s1), mul_f16x2(f0[3], s1),
                                                                     mul_f16x2(f1[1], s1), mul_f16x2(f1[3], s1));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->kv_full[b]);
          ++item;
        }
        // ---- V ----
        {
          const int b = item % kRing;
          ok = ok && warp_wait(&bars->kv_empty[b], ((item / kRing) & 1) ^ 1, err);
          uint8_t* dst = kv_s + (size_t)b * C::kTile;
          uint32_t s01[2], s23[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (left < kPage) {   // positions at or beyond the length are stale: scale 0
              const int pos = 16 * (2 * hv + u) + 2 * t;
              uint32_t keep = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) keep |= pos + (e & 1) + 8 * (e >> 1) < left ? 0xffu << (8 * e) : 0u;
              vs[u] &= keep;
            }
            s01[u] = scale_pair<0, 1>(vs[u]);
            s23[u] = scale_pair<2, 3>(vs[u]);
          }
          const int chunk = 2 * t + hv;
          const int ch0 = DH / 8 * g + DH / 16 * (w >> 1);   // first channel (a multiple of 4 or 8)
#pragma unroll
          for (int j = 0; j < 2 * F::kH; ++j) {
            uint32_t f0[4], f1[4];
            e2m1_to_f16(v[0][j], f0);
            e2m1_to_f16(v[1][j], f1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ch = ch0 + 2 * j + e;
              *reinterpret_cast<uint4*>(dst + ch * 128 + ((chunk ^ (ch & 7)) << 4)) =
                  make_uint4(mul_f16x2(f0[e], s01[0]), mul_f16x2(f0[2 + e], s23[0]), mul_f16x2(f1[e], s01[1]),
                             mul_f16x2(f1[2 + e], s23[1]));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars->kv_full[b]);
            // The block's slot is free only now that all its values have been used: an arrival behind the loads alone
            // let the next copy meet loads of V that were still under way
            mbar_arrive(&bars->raw_empty[slot]);
          }
          ++item;
        }
      }
    }
    if (!ok) bars->lost = 1;
    if constexpr (Cluster) {
      __syncwarp();
      if (unit.n > 1) cluster_sync();
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 13) {
      // ------------------------------ pieces ------------------------------
      auto task_of = [&](const Piece& p) {
        const int row0 = p.tile * kKv4ManyTile, nr = min(kKv4ManyTile, p.v.n * G - row0);
        const int limit = row_limit(p.v, group_row(a, row0 + nr - 1), a.causal);   // the last row sees the most
        const int steps = max(0, min((limit + kKv4ManyStep - 1) / kKv4ManyStep, p.s1) - p.s0);
        return Task{p.seq, p.head, row0, nr, p.s0, steps, p.v.len, p.v.n, p.whole(), (int)slot_of(p)};
      };
      const Task none{0, 0, 0, 0, 0, -1, 0, 0, 0, 0};
      if constexpr (Cluster) {
        // one piece: this CTA's share of the unit's pages; the unit may have no rows
        const int n = unit.n;
        Piece p;
        p.tile = unit.tile;
        p.head = unit.head;
        p.seq = unit.seq;
        p.v = seq_view(c, a, p.seq, lane == 0);
        const int pages = (p.v.len + kPage - 1) / kPage, per = (pages + n - 1) / n;
        p.cost = max(1, pages);
        p.s0 = n == 1 ? 0 : min(pages, unit.rank * per);
        p.s1 = n == 1 ? p.cost : min(pages, p.s0 + per);
        p.first = true;
        if (lane == 0) {
          const bool some = p.tile * kKv4ManyTile < p.v.n * G;
          bars->task[0] = some ? task_of(p) : none;
          bars->task[1] = none;
          mbar_arrive(&bars->task_full[0]);
          mbar_arrive(&bars->task_full[1]);
        }
      } else {
        Stretch<kKv4ManyTile, kKv4ManyStep> stretch(c, a, blockIdx.x == 0);
        Piece p;
        for (uint32_t i = 0;; ++i) {
          const int k = i % kTasks;
          const bool more = stretch.next(p);
          ok = warp_wait(&bars->task_empty[k], ((i / kTasks) & 1) ^ 1, err);
          if (!ok) break;
          if (lane == 0) {
            bars->task[k] = more ? task_of(p) : none;
            mbar_arrive(&bars->task_full[k]);
          }
          __syncwarp();
          if (!more) break;
        }
      }
    } else if (warp == 14) {
      // ------------------------------ blocks ------------------------------
      uint32_t page = 0;
      while (tasks.next(pc) && ok) {
        const int32_t* table = c.table + (size_t)pc.seq * c.max_pages;
        const uint8_t* plane = c.pool + ((size_t)layer * c.n_pages * c.n_kv + pc.head) * F::kBytes;
        int ids = -1;   // 32 pages' ids at a time, one a lane
        for (int i = 0; i < pc.steps; ++i, ++page) {
          if ((i & 31) == 0) {
            const bool wanted = i + lane < pc.steps;   // (the steps end at the last page that a row sees)
            ids = wanted ? table[pc.s0 + i + lane] : -1;
            if (wanted && (ids < 0 || ids >= c.n_pages)) {
              report_error(c.head, DEV_ERR_BAD_INDEX);
              ids = -1;
            }
          }
          const int id = __shfl_sync(0xffffffffu, ids, i & 31);
          const uint32_t slot = page % kRaw;
          ok = warp_wait(&bars->raw_empty[slot], ((page / kRaw) & 1) ^ 1, err);
          if (!ok) break;
          if (lane == 0) {
            bars->raw_there[slot] = id >= 0;
            if (id >= 0) {
              mbar_arrive_expect_tx(&bars->raw_full[slot], F::kBytes);
              bulk_load(&bars->raw_full[slot], raw_s + slot * F::kBytes, plane + (size_t)id * c.n_kv * F::kBytes,
                        F::kBytes);
            } else {
              mbar_arrive(&bars->raw_full[slot]);
            }
          }
          __syncwarp();
        }
      }
      bars->copies = page;
    } else {
      // ------------------------------ products of tile x ------------------------------
      // (the whole warp waits, lane 0 issues)
      const int x = warp == 12 ? 0 : 1;
      constexpr uint32_t idesc_s = idesc_f16_f32(128, 64);
      constexpr uint32_t idesc_o = idesc_f16_f32(128, DH);
      // low words of the operands' descriptors (start address / 16; a shared-memory address fits the field)
      const uint32_t q_lo = (smem_u32(q_s + x * C::kQ) >> 4) | 1u << 16, kv_lo = (smem_u32(kv_s) >> 4) | 1u << 16;
      const uint32_t desc_hi = (uint32_t)(smem_desc_sw128(0) >> 32);
      auto desc_of = [&](uint32_t lo) { return (uint64_t)desc_hi << 32 | lo; };
      const uint32_t t_s = tmem + x * 128, t_o = tmem + 256 + x * 128;
      uint32_t item = 0, n_step = 0, n_piece = 0;   // K and V tiles of all pieces; steps and pieces of this tile
      auto full = [&](uint32_t it) {
        ok = ok && warp_wait(&bars->kv_full[it % kRing], (it / kRing) & 1, err);
      };
      while (tasks.next(pc)) {
        const int steps = pc.steps;
        if (steps == 0) continue;   // (nothing to see: the softmax warps write the rows without any product)
        if (x * 128 >= pc.nr) {     // no rows in this tile: let the buffers go
          for (int i = 0; i < 2 * steps; ++i, ++item) {
            full(item);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->kv_empty[item % kRing]);
          }
          continue;
        }
        ok = ok && warp_wait(&bars->q_full[x], n_piece++ & 1, err);
        // S of step h, from K tile item + 2 h, into buffer (n_step of h) & 1.  Its columns are free: S there was read
        // before P took their place, and P there was multiplied before (products complete in order)
        auto issue_s = [&](int h, uint32_t buf) {
          const uint32_t b = (item + 2 * h) % kRing;
          full(item + 2 * h);
          tc_fence_after();
          if (lane == 0) {
            const uint32_t bd = kv_lo + b * (C::kTile >> 4);
            if (ok) {
#pragma unroll
              for (int kk = 0; kk < DH / 16; ++kk)
                umma_bf16(t_s + 64 * buf, desc_of(q_lo + (kk / 4) * (16384 >> 4) + (kk % 4) * 2),
                          desc_of(bd + (kk / 4) * (8192 >> 4) + (kk % 4) * 2), idesc_s, kk != 0);
            }
            umma_commit(&bars->s_full[x][buf]);
            umma_commit(&bars->kv_empty[b]);
          }
          __syncwarp();
        };
        issue_s(0, n_step & 1);
        if (steps > 1) issue_s(1, (n_step & 1) ^ 1);
        for (int i = 0; i < steps; ++i, ++n_step) {
          const uint32_t it = item + 2 * i + 1, b = it % kRing, buf = n_step & 1;
          full(it);
          ok = ok && warp_wait(&bars->p_ready[x][buf], (n_step >> 1) & 1, err);
          tc_fence_after();
          if (lane == 0) {
            const uint32_t bd = kv_lo + b * (C::kTile >> 4);
            if (ok) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_f16_ts(t_o, t_s + 64 * buf + kk * 8, desc_of(bd + kk * 2), idesc_o, (i | kk) != 0);
            }
            umma_commit(&bars->pv_done[x][buf]);
            umma_commit(&bars->kv_empty[b]);
          }
          __syncwarp();
          if (i + 2 < steps) issue_s(i + 2, buf);
        }
        item += 2 * steps;
      }
    }
    if (!ok) bars->lost = 1;
    __syncwarp();
    if constexpr (Cluster) {
      if (unit.n > 1) cluster_sync();
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------ softmax ------------------------------
    const int x = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lane_off + 256 + x * 128;
    uint8_t* qtile = q_s + x * C::kQ + (warp & 3) * 32 * 128;   // this warp's 32 rows
    auto q_chunk = [&](int row, int i) {         // 16-byte chunk i of the warp's row
      return reinterpret_cast<uint4*>(qtile + (i / 8) * 16384 + row * 128 + (((i & 7) ^ (row & 7)) << 4));
    };
    // The warp's rows of Q as they are into their places, dh / 8 lanes a row; of n query rows.  (Those behind the
    // last one are set to zero when the others are scaled.)
    auto load_q = [&](int seq, int head, int row0, int n) {
      constexpr int kLanes = DH / 8, kRows = 32 / kLanes;
      const int first = x * 128 + (warp & 3) * 32 + lane / kLanes;   // row of round 0, then kRows further each
      int qj = group_row(a, row0 + first), qg = row0 + first - qj * G;
      const int dj = group_row(a, kRows), dg = kRows - dj * G;
      const T* q = static_cast<const T*>(a.q) + seq * a.q_seq + (head * G) * a.q_head + lane % kLanes * 8;
#pragma unroll 4
      for (int i = 0; i < 32 / kRows; ++i) {
        if (qj < n) cp_async16(q_chunk(i * kRows + lane / kLanes, lane % kLanes), q + qj * a.q_row + qg * a.q_head);
        qj += dj;
        qg += dg;
        if (qg >= G) {
          qg -= G;
          ++qj;
        }
      }
    };
    bool met = false;                            // the cluster, before its rows are written
    if constexpr (Cluster) {
      // (while the walker reads the length too)
      load_q(unit.seq, unit.head, unit.tile * kKv4ManyTile, a.n_rows ? min(a.n_rows[unit.seq], a.rows) : a.rows);
    }
    uint32_t n_step = 0;                         // steps of this tile so far
    while (tasks.next(pc)) {
      const int steps = pc.steps;
      if (x * 128 >= pc.nr) continue;            // (the issuer skips this tile too)
      const bool valid = x * 128 + r < pc.nr;
      // a row behind the last one goes along with its limit, so that its warp's shortcuts hold
      const int rr = pc.row0 + (valid ? x * 128 + r : pc.nr - 1);
      const int j = group_row(a, rr), h = pc.head * G + rr - j * G;
      const int limit = row_limit(SeqView{pc.len, pc.n}, j, a.causal);
      float sl2 = 0.f;
      // (The S products of the last piece, which read these rows, are complete: this warp has read the last S)
      if (!Cluster && steps > 0) load_q(pc.seq, pc.head, pc.row0, pc.n);
      // A cluster's copies were started before the piece was known: also a CTA without steps waits for its own before
      // its rows go through the Q tile
      cp_async_wait_all();
      __syncwarp();
      if (steps > 0) {
        // Q to fp16 in its place, times a power of two, a thread a row
        uint4 w[DH / 8];
        uint32_t top[4] = {0, 0, 0, 0};   // largest magnitudes: 16-bit floats in the order of their bits
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) w[i] = *q_chunk(lane, i);   // (all before the first store)
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) {
          if (!valid) w[i] = make_uint4(0, 0, 0, 0);
          top[0] = __vmaxu2(top[0], w[i].x & 0x7fff7fffu);
          top[1] = __vmaxu2(top[1], w[i].y & 0x7fff7fffu);
          top[2] = __vmaxu2(top[2], w[i].z & 0x7fff7fffu);
          top[3] = __vmaxu2(top[3], w[i].w & 0x7fff7fffu);
        }
        top[0] = __vmaxu2(__vmaxu2(top[0], top[1]), __vmaxu2(top[2], top[3]));
        float down, up;
        row_powers(Half<T>::lo(max(top[0] & 0xffffu, top[0] >> 16)), down, up);
#pragma unroll
        for (int i = 0; i < DH / 8; ++i)
          *q_chunk(lane, i) = make_uint4(pack_f16x2(Half<T>::lo(w[i].x) * down, Half<T>::hi(w[i].x) * down),
                                         pack_f16x2(Half<T>::lo(w[i].y) * down, Half<T>::hi(w[i].y) * down),
                                         pack_f16x2(Half<T>::lo(w[i].z) * down, Half<T>::hi(w[i].z) * down),
                                         pack_f16x2(Half<T>::lo(w[i].w) * down, Half<T>::hi(w[i].w) * down));
        sl2 = fmaxf(a.scale * 1.4426950408889634f * up, 1e-44f);   // (above 0, so that -inf stays -inf)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full[x]);
      }
      float m_used = -INFINITY, l = 0.f;
      bool far = false;                          // the reference is kFar or more
      for (int i = 0; i < steps; ++i, ++n_step) {
        const uint32_t buf = n_step & 1;
        const uint32_t t_s = tmem + lane_off + x * 128 + 64 * buf;
        ok = ok && warp_wait(&bars->s_full[x][buf], (n_step >> 1) & 1, err);
        tc_fence_after();
        const int kmax = limit - (pc.s0 + i) * kKv4ManyStep;   // positions of this step that the row sees
        float s[64];
        tmem_ld32(t_s, s);
        tmem_ld32(t_s + 32, s + 32);
        tmem_wait_ld();
        if (!__all_sync(0xffffffffu, kmax >= kKv4ManyStep)) {
#pragma unroll
          for (int e = 0; e < 64; ++e) s[e] = e < kmax ? s[e] : -INFINITY;
        }
        // the row's maximum (raw scores; the scale is positive)
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 2) top[e / 2 & 3] = max3(top[e / 2 & 3], s[e], s[e + 1]);
        // the reference follows when the maximum has grown by more than kLazy (the first finite one: above -inf)
        const float tmax = reference_of<kManyShift>(fmaxf(max3(top[0], top[1], top[2]), top[3]) * sl2);
        const bool grow = tmax > m_used + kLazy;
        float factor = sl2;
        if (__any_sync(0xffffffffu, grow || far)) {
          const float m_new = grow ? tmax : m_used;
          const float alpha = grow && m_used != -INFINITY ? fast_exp2(m_used - m_new) : 1.f;
          l *= alpha;
          m_used = m_new;
          far = fabsf(m_used) >= kFar && m_used != -INFINITY;
          if (__any_sync(0xffffffffu, far)) {
            // The reference is a rounded product; this far out the exact products of the multiply-add below lie up to
            // half a unit of it off, which is more than P has room for.  So the scores are rounded as it was
            factor = 1.f;
#pragma unroll
            for (int e = 0; e < 64; ++e) s[e] *= sl2;
          }
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O holds the steps before this one once the last of their products is complete
            ok = ok && warp_wait(&bars->pv_done[x][buf ^ 1], ((n_step - 1) >> 1) & 1, err);
            tc_fence_after();
#pragma unroll 1
            for (int cb = 0; cb < DH; cb += 32) {
              float o[32];
              tmem_ld32(t_o + cb, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(t_o + cb, o);
            }
          }
        }
        // P over S, in V's order: words 4 ch .. 4 ch + 3 (chunk ch = 2 t + b) are the pairs t of the 8-position groups
        // 4 b .. 4 b + 3.  (Nothing seen yet: every score is -inf, p is 0.)
        const float m_ref = m_used == -INFINITY ? 0.f : m_used;
        const uint64_t sl2x2 = pack_f32x2(factor, factor), negm2 = pack_f32x2(-m_ref, -m_ref);
        uint64_t sum[2] = {0, 0};
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const uint64_t y = ffma_f32x2(pack_f32x2(s[e], s[e + 1]), sl2x2, negm2);
          const float p0 = fast_exp2(lo_f32(y)), p1 = fast_exp2(hi_f32(y));
          sum[e / 2 & 1] = fadd_f32x2(sum[e / 2 & 1], pack_f32x2(p0, p1));
          pk[8 * (e / 2 % 4) + e / 8] = pack_f16x2(p0, p1);   // pair e / 2 = 4 group + t -> word 8 t + group
        }
        tmem_st32u(t_s, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&bars->p_ready[x][buf]);
        const uint64_t both = fadd_f32x2(sum[0], sum[1]);
        l += lo_f32(both) + hi_f32(both);
      }
      // ---- the row out ----
      if (steps > 0) {
        // (one barrier a buffer: the products of the last two steps may both be under way here)
        ok = ok && warp_wait(&bars->pv_done[x][(n_step - 1) & 1], ((n_step - 1) >> 1) & 1, err);
        tc_fence_after();
      }
      const bool some = steps > 0 && l != 0.f;   // (a row may see nothing; a NaN sum goes through)
      const float inv = some ? 1.f / l : 0.f;
      const float lse2 = some ? m_used + kManyShift + log2f(l * (1.f / (1 << kManyShift))) : -INFINITY;
      T* dst = static_cast<T*>(a.out) + pc.seq * a.o_seq + j * a.o_row + h * a.o_head;
      const size_t at = (size_t)pc.slot * kKv4ManyTile + x * 128 + r;
      // A part for a bf16 output in fp16: half the bytes of fp32.  A power of two brings the row's largest magnitude up
      // to 2^14 .. 2^15 (a mean of |v| <= 61440 is never above fp16's range), so a value is off by 2^-11 of itself at
      // most, or by 2^-39 of that largest one.  For an fp16 output, whose own rounding that is, in fp32.  16-byte chunks
      // of the tile's rows lie side by side, so that a warp's stores and the merge's loads are contiguous
      constexpr int kPer = kPartPer<T>;   // channels of a chunk
      const bool joined = (Cluster && unit.n > 1) || !pc.whole;
      float factor = inv, up = 1.f;
      if (kPer == 8 && joined) {
        float most = 0.f;
#pragma unroll 1
        for (int cb = 0; cb < DH; cb += 32) {
          float o[32];
          tmem_ld32(t_o + cb, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) most = max3(most, fabsf(o[e]), fabsf(o[e + 1]));
        }
        float down;
        row_powers(some ? most * inv : 0.f, down, up);
        up = fminf(up, 1.f);
        factor = inv * fmaxf(down, 1.f);
      }
      auto chunk_of = [](const float(&o)[32], int e) {
        if constexpr (kPer == 4)
          return make_uint4(__float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                            __float_as_uint(o[e + 3]));
        else
          return make_uint4(pack_f16x2(o[e], o[e + 1]), pack_f16x2(o[e + 2], o[e + 3]),
                            pack_f16x2(o[e + 4], o[e + 5]), pack_f16x2(o[e + 6], o[e + 7]));
      };
      uint4* part = static_cast<uint4*>(a.part_o) + (size_t)pc.slot * kKv4ManyTile * (DH / kPer) + x * 128 + r;
      if (Cluster && unit.n > 1) {
        // Each CTA of the cluster joins its share of the rows.  A row goes into this warp's part of the Q tile, whose
        // products are complete, and from there in one piece to the CTA that joins it: as the lanes hold the rows, a
        // store would meet a line for each lane
        const int per = (pc.nr + unit.n - 1) / unit.n, owner = min((x * 128 + r) / per, unit.n - 1);
        const int place = unit.rank * per + x * 128 + r - owner * per;
        const uint32_t to = dsmem_map(smem_u32(kv_s) + place * (16 * DH / kPer), owner);
        const uint32_t to_stat = dsmem_map(smem_u32(stat_s + place), owner);
        cluster_sync();   // the others' rings are free once all their products are complete
        met = true;
        if (valid) dsmem_st_f2(to_stat, make_float2(lse2, up));
        constexpr int kLanes = DH / 8, kRows = 32 / kLanes;   // the Q tile holds dh / 8 chunks of a row
#pragma unroll
        for (int half = 0; half < 8 / kPer; ++half) {
#pragma unroll
          for (int cb = 0; cb < DH / 8 * kPer; cb += 32) {
            float o[32];
            tmem_ld32(t_o + half * (DH / 2) + cb, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = some ? o[e] * factor : 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += kPer) *q_chunk(lane, (cb + e) / kPer) = chunk_of(o, e);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32 / kRows; ++i) {
            const int row = i * kRows + lane / kLanes;
            const uint32_t at = __shfl_sync(0xffffffffu, to, row) + (half * kLanes + lane % kLanes) * 16;
            if (x * 128 + (warp & 3) * 32 + row < pc.nr) dsmem_st4(at, *q_chunk(row, lane % kLanes));
          }
          __syncwarp();
        }
      } else {
#pragma unroll
        for (int cb = 0; cb < DH; cb += 32) {
          float o[32];
          tmem_ld32(t_o + cb, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = some ? o[e] * factor : 0.f;
          if (valid && ok) {
            if (pc.whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                *reinterpret_cast<uint4*>(dst + cb + e) =
                    make_uint4(Half<T>::pack(o[e], o[e + 1]), Half<T>::pack(o[e + 2], o[e + 3]),
                               Half<T>::pack(o[e + 4], o[e + 5]), Half<T>::pack(o[e + 6], o[e + 7]));
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += kPer) part[(cb + e) / kPer * kKv4ManyTile] = chunk_of(o, e);
            }
          }
        }
        if (valid && ok) {
          if (!pc.whole)
            reinterpret_cast<float2*>(a.part_lse)[at] = make_float2(lse2, up);
          else if (a.lse)
            a.lse[((size_t)pc.seq * a.rows + j) * a.n_q + h] = lse2 * 0.6931471805599453f;
        }
      }
      tc_fence_before();   // O is read before the next piece's products overwrite it (they wait for p_ready)
    }
    if (!ok) bars->lost = 1;
    // (a cluster's CTA goes on with all its warps: everyone back to the registers of the launch)
    if constexpr (Cluster) {
      cp_async_wait_all();
      __syncwarp();
      if (unit.n > 1 && !met) cluster_sync();
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (bars->lost) {
    // Nobody has waited for what may still be under way: copies into this CTA's memory, products that read it and write
    // its tensor memory
    if (warp == 14)
      for (uint32_t n = bars->copies, k = 1; k <= kRaw && k <= n; ++k)
        mbar_wait(&bars->raw_full[(n - k) % kRaw], ((n - k) / kRaw) & 1, nullptr, 0);
    if ((warp == 12 || warp == 15) && lane == 0) {
      uint64_t* bar = &bars->drained[warp == 12 ? 0 : 1];
      umma_commit(bar);
      mbar_wait(bar, 0, nullptr, 0);
    }
    __syncthreads();
  }
  if (warp == 12) tmem_dealloc(tmem, 512);
  if (Cluster && unit.n > 1) {
    // every CTA of the cluster has its share of the unit's rows from all of them, and joins it, a thread for a
    // 16-byte chunk at a time
    cluster_sync();
    const int n = unit.n, nr = bars->task[0].nr;                 // (0: the unit has no rows)
    const int per = (nr + n - 1) / n, first = unit.rank * per, mine = min(per, nr - first);
    constexpr int kPer = kPartPer<T>, kChunks = DH / kPer;
    for (int i = threadIdx.x; i < mine * kChunks; i += kManyThreads) {
      const int at = i / kChunks, chunk = i % kChunks;
      float2 st[kMaxManyCluster];
      float top = -INFINITY;
      uint4 v[kMaxManyCluster];
#pragma unroll
      for (int k = 0; k < kMaxManyCluster; ++k) {   // (all loads before the first use)
        st[k] = k < n ? stat_s[k * per + at] : make_float2(-INFINITY, 1.f);
        v[k] = k < n ? reinterpret_cast<const uint4*>(kv_s)[(k * per + at) * kChunks + chunk] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < kMaxManyCluster; ++k) top = max_nan(top, st[k].x);
      float acc[kPer], den = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
      if (top != -INFINITY) {
#pragma unroll
        for (int k = 0; k < kMaxManyCluster; ++k) {
          const float f = fast_exp2(st[k].x - top), g = f * st[k].y;
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          den += f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kPer == 4) {
              acc[e] += g * __uint_as_float(w[e]);
            } else {
              acc[2 * e] += g * Half<__half>::lo(w[e]);
              acc[2 * e + 1] += g * Half<__half>::hi(w[e]);
            }
          }
        }
      }
      const float inv = den == 0.f ? 0.f : 1.f / den;
      const int rr = unit.tile * kKv4ManyTile + first + at, j = group_row(a, rr), h = unit.head * G + rr - j * G;
      T* dst = static_cast<T*>(a.out) + unit.seq * a.o_seq + j * a.o_row + h * a.o_head + chunk * kPer;
#pragma unroll
      for (int e = 0; e < kPer; e += 4)
        *reinterpret_cast<uint2*>(dst + e) = make_uint2(Half<T>::pack(acc[e] * inv, acc[e + 1] * inv),
                                                        Half<T>::pack(acc[e + 2] * inv, acc[e + 3] * inv));
      if (a.lse && chunk == 0)
        a.lse[((size_t)unit.seq * a.rows + j) * a.n_q + h] = (top + log2f(den)) * 0.6931471805599453f;
    }
  }
}

template <int DH, typename T>
cudaError_t prepare_many() {
  static unsigned long long done = 0;
  return once_per_device(&done, [] {
    const cudaError_t e = cudaFuncSetAttribute(kv4_attend_many_kernel<DH, T, false>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ManySmem<DH>::kBytes);
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(kv4_attend_many_kernel<DH, T, true>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)ManySmem<DH>::kBytes);
  });
}

template <int DH>
int clusters_at_once(int n) {
  if (prepare_many<DH, __nv_bfloat16>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, n);
  cfg.blockDim = dim3(kManyThreads);
  cfg.dynamicSmemBytes = ManySmem<DH>::kBytes;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = n;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int count = 0;
  if (cudaOccupancyMaxActiveClusters(&count, kv4_attend_many_kernel<DH, __nv_bfloat16, true>, &cfg) == cudaSuccess)
    return count;
  cudaGetLastError();   // (a size the device does not take is an answer, not an error of the call)
  return 0;
}

template <int DH, typename T>
cudaError_t launch_many(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st) {
  constexpr int kBytes = (int)ManySmem<DH>::kBytes;
  const cudaError_t e = prepare_many<DH, T>();
  if (e != cudaSuccess) return e;
  if (a.cluster) {
    const int tiles = (a.rows * a.group + kKv4ManyTile - 1) / kKv4ManyTile;
    return launch_k(kv4_attend_many_kernel<DH, T, true>, dim3(tiles, c.n_kv, c.n_seq * a.cluster), dim3(kManyThreads),
                    kBytes, st, a.cluster, c, layer, a);
  }
  return launch_k(kv4_attend_many_kernel<DH, T, false>, dim3(a.n_ctas), dim3(kManyThreads), kBytes, st, 1, c, layer, a);
}

}  // namespace

int kv4_many_clusters(int dh, int n) {
  static int known[2][64][kMaxManyCluster + 1];   // by head size and device: count + 1, 0 where not asked for yet
  int dev = 0;
  if (n < 1 || n > kMaxManyCluster || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int v = __atomic_load_n(&known[dh == 128][dev][n], __ATOMIC_RELAXED);
  if (v == 0) {
    v = (dh == 128 ? clusters_at_once<128>(n) : clusters_at_once<64>(n)) + 1;
    __atomic_store_n(&known[dh == 128][dev][n], v, __ATOMIC_RELAXED);
  }
  return v - 1;
}

cudaError_t kv4_attend_many(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st) {
  if (c.dh == 128)
    return a.fp16 ? launch_many<128, __half>(c, layer, a, st) : launch_many<128, __nv_bfloat16>(c, layer, a, st);
  return a.fp16 ? launch_many<64, __half>(c, layer, a, st) : launch_many<64, __nv_bfloat16>(c, layer, a, st);
}

}  // namespace dg
