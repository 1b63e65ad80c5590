// kv4_canvas.cu -- attention over the paged 4-bit cache for many rows: canvases and prompt chunks, on tcgen05.
//
// A CTA works on 256 rows of a KV head (two 128-row tiles) and steps of 128 positions (two pages), so each dequantised
// step serves 256 rows.  Warp roles (416 threads):
//   warps 0-3    softmax of tile 0, warps 4-7 softmax of tile 1 (thread = row): the row of Q into shared memory, S from
//                TMEM, P = 2^(S - m) in fp16 to shared memory, running sum, the finished row out
//   warps 8-11   dequantise: codes and scales from global memory into registers, one step ahead; fp16 K and V tiles
//                in the 128-byte swizzled layout of the tensor core, through a ring of three buffers
//   warp 12      issues the products: S_x = Q_x K^T and O_x += P_x V in the order
//                S_0(0) S_1(0) | PV_0(t) S_0(t+1) PV_1(t) S_1(t+1) ..., one tile's products under the other's softmax
// The scale multiplies each code in fp16, exactly.  V's codes come in pairs of positions, so V is laid down with its
// positions in the order 16 t + 4 tile + (pair), which makes each lane's share contiguous; P's columns are stored in the same
// order, which only renames registers.  The running maximum is lazy: O and the sum are rescaled when a row's
// maximum has grown by more than 2^8, so P stays below 2^8.
#include <math.h>

#include "kv4_attention.cuh"

namespace dg {

namespace {

constexpr int kManyThreads = 416;
constexpr int kRing = 3;
constexpr float kLazy = 8.f;   // log2 units

template <int DH>
struct ManySmem {
  static constexpr uint32_t kTile = 128u * DH * 2u;   // a Q, K or V tile
  static constexpr uint32_t kP = 128u * 128u * 2u;
  static constexpr size_t kBytes = 1024 + 2 * kTile + kRing * kTile + 2 * kP + 256;
};

struct ManyBars {
  uint64_t q_full[2], s_full[2], s_free[2], p_ready[2], pv_done[2];
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint32_t tmem;
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

// kind::f16 with fp16 operands, fp32 accumulators, both K-major
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// steps of 128 positions that the rows of a piece have to look at, within [s0, s1)
__device__ __forceinline__ int piece_steps(const Piece& p, int G, int causal, int& nr) {
  nr = (int)min((long long)kKv4ManyTile, (long long)p.v.n * G - (long long)p.tile * kKv4ManyTile);
  const int limit = row_limit(p.v, (p.tile * kKv4ManyTile + nr - 1) / G, causal);
  return max(0, min((limit + kKv4ManyStep - 1) / kKv4ManyStep, p.s1) - p.s0);
}

template <int DH, typename T>
__global__ void __launch_bounds__(kManyThreads, 1) kv4_attend_many_kernel(Kv4View c, int layer, Kv4Attn a) {
  using F = Kv4<DH>;
  using C = ManySmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = base;
  uint8_t* kv_s = q_s + 2 * C::kTile;
  uint8_t* p_s = kv_s + kRing * C::kTile;
  ManyBars* bars = reinterpret_cast<ManyBars*>(p_s + 2 * C::kP);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = c.head + KV4_WORD_WAIT;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->q_full[x], 4);
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->s_free[x], 4);
      mbar_init(&bars->p_ready[x], 4);
      mbar_init(&bars->pv_done[x], 1);
    }
    for (int b = 0; b < kRing; ++b) {
      mbar_init(&bars->kv_full[b], 4);
      mbar_init(&bars->kv_empty[b], 1);
    }
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(&bars->tmem, 512);   // S_0 [0,128) S_1 [128,256) O_0 [256,..) O_1 [384,..)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  pdl_wait();

  const int G = a.n_q / c.n_kv;
  Stretch stretch = find_stretch<kKv4ManyTile, kKv4ManyStep, kManyThreads>(c, a);
  Piece pc;
  bool ok = true;

  if (warp >= 8 && warp < 12) {
    // ------------------------------ dequantise ------------------------------
    const int w = warp - 8, g = lane >> 2, t = lane & 3;
    const int pg = w >> 1;                       // this warp's page of a step
    uint32_t item = 0;                           // K and V tiles laid down so far
    while (next_piece<kKv4ManyTile, kKv4ManyStep>(c, a, stretch, pc)) {
      int nr;
      const int steps = piece_steps(pc, G, a.causal, nr);
      const int n_pages = (pc.v.len + kPage - 1) / kPage;
      const int32_t* table = c.table + (size_t)pc.seq * c.max_pages;
      const uint8_t* plane = c.pool + ((size_t)layer * c.n_pages * c.n_kv + pc.head) * F::kBytes;
      // this warp's page of step i, or null
      int ids = -1;
      auto block_of = [&](int i) -> const uint8_t* {   // whole warp, i ascending
        if ((i & 31) == 0) {
          const int page = 2 * (pc.s0 + i + lane) + pg;
          ids = i + lane < steps && page < n_pages ? table[page] : -1;
          if (i + lane < steps && page < n_pages && (ids < 0 || ids >= c.n_pages)) {
            report_error(c.head, DEV_ERR_BAD_INDEX);
            ids = -1;
          }
        }
        const int id = __shfl_sync(0xffffffffu, ids, i & 31);
        return id < 0 ? nullptr : plane + (size_t)id * c.n_kv * F::kBytes;
      };
      // K: 16-position tiles 2 (w & 1) + {0, 1}; V: tiles 2 h + {0, 1} with h = (w & 1) ^ (g & 1), so that the lanes of
      // a store meet different banks
      const int hv = (w & 1) ^ (g & 1);
      uint4 ck[2][F::kH], cv[2][F::kH];
      uint32_t sk[2], sv[2];
      auto load = [&](const uint8_t* blk) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int kt = 2 * (w & 1) + u, vt = 2 * hv + u;
          sk[u] = sv[u] = 0;
#pragma unroll
          for (int jh = 0; jh < F::kH; ++jh) ck[u][jh] = cv[u][jh] = make_uint4(0, 0, 0, 0);
          if (blk) {
            const uint8_t* s = blk + F::kSk + lane * 8 * F::kH + 2 * kt * F::kH;
            sk[u] = F::kH == 2 ? *reinterpret_cast<const uint32_t*>(s) : *reinterpret_cast<const uint16_t*>(s);
            sv[u] = *reinterpret_cast<const uint32_t*>(blk + F::kSv + ((F::kH == 2 ? g : g >> 1) * 4 + t) * 16 + 4 * vt);
#pragma unroll
            for (int jh = 0; jh < F::kH; ++jh) {
              // (K: lanes t 2 and 3 take the channel halves in the other order, for the banks)
              const int jk = F::kH == 2 ? jh ^ (t >> 1) : 0;
              ck[u][jh] = *reinterpret_cast<const uint4*>(blk + ((kt * F::kH + jk) * 32 + lane) * 16);
              cv[u][jh] = *reinterpret_cast<const uint4*>(blk + F::kV + ((vt * F::kH + jh) * 32 + lane) * 16);
            }
          }
        }
      };
      if (steps > 0) load(block_of(0));
      for (int i = 0; i < steps; ++i) {
        uint4 k[2][F::kH], v[2][F::kH];
        uint32_t ks[2], vs[2];
        const int left = pc.v.len - (pc.s0 + i) * kKv4ManyStep - pg * kPage;   // positions of this page that exist
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          ks[u] = sk[u];
          vs[u] = sv[u];
#pragma unroll
          for (int jh = 0; jh < F::kH; ++jh) {
            k[u][jh] = ck[u][jh];
            v[u][jh] = cv[u][jh];
          }
        }
        if (i + 1 < steps) load(block_of(i + 1));
        // ---- K ----
        {
          const int b = item % kRing;
          ok = ok && mbar_wait(&bars->kv_empty[b], ((item / kRing) & 1) ^ 1, err, DEV_ERR_TIMEOUT_ATTN);
          uint8_t* dst = kv_s + (size_t)b * C::kTile;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int row = pg * kPage + 16 * (2 * (w & 1) + u) + g;   // and row + 8
#pragma unroll
            for (int jh = 0; jh < F::kH; ++jh) {
              const int jk = F::kH == 2 ? jh ^ (t >> 1) : 0;
              uint32_t s0, s1;
              if constexpr (F::kH == 2) {
                const uint32_t two = jk ? ks[u] >> 8 : ks[u];
                s0 = scale_pair<0, 0>(two);
                s1 = scale_pair<2, 2>(two);
              } else {
                s0 = scale_pair<0, 0>(ks[u]);
                s1 = scale_pair<1, 1>(ks[u]);
              }
              const uint32_t wd[4] = {k[u][jh].x, k[u][jh].y, k[u][jh].z, k[u][jh].w};
              const int plane64 = F::kH == 2 ? t >> 1 : 0;
              const int chunk0 = F::kH == 2 ? (t & 1) * 4 + 2 * jk : 2 * t;
              uint8_t* rp = dst + plane64 * 16384 + row * 128;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t f0[4], f1[4];
                e2m1_to_f16(wd[2 * q], f0);
                e2m1_to_f16(wd[2 * q + 1], f1);
                const int off = ((chunk0 + q) ^ (row & 7)) << 4;   // (row + 8 has the same swizzle)
                *reinterpret_cast<uint4*>(rp + off) = make_uint4(mul_f16x2(f0[0], s0), mul_f16x2(f0[2], s0),
                                                                mul_f16x2(f1[0], s0), mul_f16x2(f1[2], s0));
                *reinterpret_cast<uint4*>(rp + 1024 + off) = make_uint4(mul_f16x2(f0[1], s1), mul_f16x2(f0[3], s1),
                                                                       mul_f16x2(f1[1], s1), mul_f16x2(f1[3], s1));
              }
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
          ok = ok && mbar_wait(&bars->kv_empty[b], ((item / kRing) & 1) ^ 1, err, DEV_ERR_TIMEOUT_ATTN);
          uint8_t* dst = kv_s + (size_t)b * C::kTile + pg * (DH * 128);
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
#pragma unroll
          for (int jh = 0; jh < F::kH; ++jh) {
            const uint32_t w0[4] = {v[0][jh].x, v[0][jh].y, v[0][jh].z, v[0][jh].w};
            const uint32_t w1[4] = {v[1][jh].x, v[1][jh].y, v[1][jh].z, v[1][jh].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t f0[4], f1[4];
              e2m1_to_f16(w0[j], f0);
              e2m1_to_f16(w1[j], f1);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int ch = DH / 8 * g + 8 * jh + 2 * j + e;
                *reinterpret_cast<uint4*>(dst + ch * 128 + ((chunk ^ ((2 * j + e) & 7)) << 4)) =
                    make_uint4(mul_f16x2(f0[e], s01[0]), mul_f16x2(f0[2 + e], s23[0]), mul_f16x2(f1[e], s01[1]),
                               mul_f16x2(f1[2 + e], s23[1]));
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->kv_full[b]);
          ++item;
        }
      }
    }
  } else if (warp == 12) {
    // ------------------------------ products ------------------------------
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16_f32(128, 128);
      constexpr uint32_t idesc_o = idesc_f16_f32(128, DH);
      uint32_t item = 0, n_tile[2] = {0, 0}, n_piece[2] = {0, 0};   // items used, steps of each tile, pieces of each tile
      while (next_piece<kKv4ManyTile, kKv4ManyStep>(c, a, stretch, pc)) {
        int nr;
        const int steps = piece_steps(pc, G, a.causal, nr);
        if (steps == 0) continue;   // (nothing to see: the softmax warps write the rows without any product)
        const int nx = nr > 128 ? 2 : 1;
        for (int x = 0; x < nx; ++x) {
          ok = ok && mbar_wait(&bars->q_full[x], n_piece[x] & 1, err, DEV_ERR_TIMEOUT_ATTN);
          ++n_piece[x];
        }
        auto issue_s = [&](int x, int i) {
          const uint32_t it = item + 2 * i, b = it % kRing;
          ok = ok && mbar_wait(&bars->kv_full[b], (it / kRing) & 1, err, DEV_ERR_TIMEOUT_ATTN);
          ok = ok && mbar_wait(&bars->s_free[x], ((n_tile[x] + i) & 1) ^ 1, err, DEV_ERR_TIMEOUT_ATTN);
          tc_fence_after();
          if (ok) {
            const uint8_t* kb = kv_s + (size_t)b * C::kTile;
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
              const uint64_t ad =
                  desc_advance(smem_desc_sw128(smem_u32(q_s + x * C::kTile + (kk / 4) * 16384)), (kk % 4) * 32);
              const uint64_t bd = desc_advance(smem_desc_sw128(smem_u32(kb + (kk / 4) * 16384)), (kk % 4) * 32);
              umma_bf16(tmem + x * 128, ad, bd, idesc_s, kk != 0);
            }
          }
          umma_commit(&bars->s_full[x]);
          if (x == nx - 1) umma_commit(&bars->kv_empty[b]);
        };
        auto issue_pv = [&](int x, int i) {
          const uint32_t it = item + 2 * i + 1, b = it % kRing;
          ok = ok && mbar_wait(&bars->kv_full[b], (it / kRing) & 1, err, DEV_ERR_TIMEOUT_ATTN);
          ok = ok && mbar_wait(&bars->p_ready[x], (n_tile[x] + i) & 1, err, DEV_ERR_TIMEOUT_ATTN);
          tc_fence_after();
          if (ok) {
            const uint8_t* vb = kv_s + (size_t)b * C::kTile;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint64_t ad =
                  desc_advance(smem_desc_sw128(smem_u32(p_s + x * C::kP + (kk / 4) * 16384)), (kk % 4) * 32);
              const uint64_t bd = desc_advance(smem_desc_sw128(smem_u32(vb + (kk / 4) * (DH * 128))), (kk % 4) * 32);
              umma_bf16(tmem + 256 + x * 128, ad, bd, idesc_o, (i | kk) != 0);
            }
          }
          umma_commit(&bars->pv_done[x]);
          if (x == nx - 1) umma_commit(&bars->kv_empty[b]);
        };
        for (int x = 0; x < nx; ++x) issue_s(x, 0);
        for (int i = 0; i < steps; ++i)
          for (int x = 0; x < nx; ++x) {
            issue_pv(x, i);
            if (i + 1 < steps) issue_s(x, i + 1);
          }
        item += 2 * steps;
        for (int x = 0; x < nx; ++x) n_tile[x] += steps;
      }
    }
  } else {
    // ------------------------------ softmax ------------------------------
    const int x = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + x * 128;
    const uint32_t t_o = tmem + lane_off + 256 + x * 128;
    uint8_t* prow = p_s + x * C::kP + r * 128;
    uint8_t* qrow = q_s + x * C::kTile + r * 128;
    uint32_t n_tile = 0;                         // steps of this tile so far
    while (next_piece<kKv4ManyTile, kKv4ManyStep>(c, a, stretch, pc)) {
      int nr;
      const int steps = piece_steps(pc, G, a.causal, nr);
      if (x * 128 >= nr) continue;               // (the issuer skips this tile too)
      const bool valid = x * 128 + r < nr;
      // a row behind the last one goes along with its limit, so that its warp's shortcuts hold
      const int rr = pc.tile * kKv4ManyTile + (valid ? x * 128 + r : nr - 1);
      const int j = rr / G, h = pc.head * G + rr % G;
      const int limit = row_limit(pc.v, j, a.causal);
      float sl2 = 0.f;
      if (steps > 0) {
        // Q: this thread's row to fp16 in the swizzled layout, times a power of two (the S products of the last
        // piece, which read this row, are complete: this warp has read the last S)
        const T* q = static_cast<const T*>(a.q) + pc.seq * a.q_seq + j * a.q_row + h * a.q_head;
        uint4 raw[DH / 8];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) {
          raw[i] = valid ? reinterpret_cast<const uint4*>(q)[i] : make_uint4(0, 0, 0, 0);
          const uint32_t wd[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(Half<T>::lo(wd[e])), fabsf(Half<T>::hi(wd[e]))));
        }
        float down, up;
        row_powers(amax, down, up);
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) {
          uint32_t wd[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) wd[e] = pack_f16x2(Half<T>::lo(wd[e]) * down, Half<T>::hi(wd[e]) * down);
          *reinterpret_cast<uint4*>(qrow + (i / 8) * 16384 + (((i & 7) ^ (r & 7)) << 4)) =
              make_uint4(wd[0], wd[1], wd[2], wd[3]);
        }
        sl2 = a.scale * 1.4426950408889634f * up;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full[x]);
      }
      float m_used = -INFINITY, l = 0.f;
      for (int i = 0; i < steps; ++i, ++n_tile) {
        ok = ok && mbar_wait(&bars->s_full[x], n_tile & 1, err, DEV_ERR_TIMEOUT_ATTN);
        tc_fence_after();
        const int kmax = limit - (pc.s0 + i) * kKv4ManyStep;   // positions of this step that the row sees
        const bool full = kmax >= kKv4ManyStep;
        auto p_pass = [&](float m_ref, float& rmax) {
          uint64_t lt2 = 0;
          const uint64_t sl2x2 = pack_f32x2(sl2, sl2), negm2 = pack_f32x2(-m_ref, -m_ref);
          rmax = -INFINITY;
#pragma unroll
          for (int cb = 0; cb < 128; cb += 64) {
            float s[64];
            tmem_ld32(t_s + cb, s);
            tmem_ld32(t_s + cb + 32, s + 32);
            tmem_wait_ld();
            uint32_t pk[32];
            if (full) {
#pragma unroll
              for (int e = 0; e < 64; e += 2) {
                rmax = fmaxf(rmax, fmaxf(s[e], s[e + 1]));
                const uint64_t y = ffma_f32x2(pack_f32x2(s[e], s[e + 1]), sl2x2, negm2);
                const float p0 = fast_exp2(lo_f32(y)), p1 = fast_exp2(hi_f32(y));
                lt2 = fadd_f32x2(lt2, pack_f32x2(p0, p1));
                pk[e / 2] = pack_f16x2(p0, p1);
              }
            } else {
              float lt = 0.f;
#pragma unroll
              for (int e = 0; e < 64; e += 2) {
                const bool v0 = cb + e < kmax, v1 = cb + e + 1 < kmax;   // masked: p = 0
                if (v0) rmax = fmaxf(rmax, s[e]);
                if (v1) rmax = fmaxf(rmax, s[e + 1]);
                const float p0 = v0 ? fast_exp2(fmaf(s[e], sl2, -m_ref)) : 0.f;
                const float p1 = v1 ? fast_exp2(fmaf(s[e + 1], sl2, -m_ref)) : 0.f;
                lt += p0 + p1;
                pk[e / 2] = pack_f16x2(p0, p1);
              }
              lt2 = fadd_f32x2(lt2, pack_f32x2(lt, 0.f));
            }
            // position order of V: chunk 2 t + h holds pairs t of 8-position groups 4 h .. 4 h + 3
            uint8_t* out = prow + (cb / 64) * 16384;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              const int at = 16 * (ch & 1) + (ch >> 1);
              *reinterpret_cast<uint4*>(out + ((ch ^ (r & 7)) << 4)) =
                  make_uint4(pk[at], pk[at + 4], pk[at + 8], pk[at + 12]);
            }
          }
          return lo_f32(lt2) + hi_f32(lt2);
        };
        // PV of the step before is complete (products complete in order), so O and P are free here
        float rmax = -INFINITY, lt = 0.f;
        bool redo = m_used == -INFINITY;
        if (!__any_sync(0xffffffffu, redo)) {
          lt = p_pass(m_used, rmax);
          redo = rmax * sl2 > m_used + kLazy;
        }
        if (__any_sync(0xffffffffu, redo)) {
          rmax = -INFINITY;
#pragma unroll
          for (int cb = 0; cb < 128; cb += 64) {
            float s[64];
            tmem_ld32(t_s + cb, s);
            tmem_ld32(t_s + cb + 32, s + 32);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (cb + e < kmax) rmax = fmaxf(rmax, s[e]);
          }
          const float tmax = rmax * sl2;
          const bool grow = redo && tmax > m_used + kLazy;
          const float m_new = grow ? tmax : m_used;
          const float alpha = (grow && m_used != -INFINITY) ? fast_exp2(m_used - m_new) : 1.f;
          l *= alpha;
          m_used = m_new;
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int cb = 0; cb < DH; cb += 32) {
              float o[32];
              tmem_ld32(t_o + cb, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(t_o + cb, o);
            }
            tmem_wait_st();
          }
          lt = p_pass(m_used, rmax);
        }
        l += lt;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->s_free[x]);
          mbar_arrive(&bars->p_ready[x]);
        }
      }
      // ---- the row out ----
      if (steps > 0) {
        ok = ok && mbar_wait(&bars->pv_done[x], (n_tile - 1) & 1, err, DEV_ERR_TIMEOUT_ATTN);
        tc_fence_after();
      }
      const bool some = steps > 0 && l != 0.f;   // (a row may see nothing; a NaN sum goes through)
      const float inv = some ? 1.f / l : 0.f;
      const float lse2 = some ? m_used + log2f(l) : -INFINITY;
      const bool whole = pc.whole();
      T* dst = static_cast<T*>(a.out) + pc.seq * a.o_seq + j * a.o_row + h * a.o_head;
      const size_t at = slot_of(pc) * kKv4ManyTile + x * 128 + r;
      __half* part = static_cast<__half*>(a.part_o) + at * DH;
#pragma unroll
      for (int cb = 0; cb < DH; cb += 32) {
        float o[32];
        tmem_ld32(t_o + cb, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = some ? o[e] * inv : 0.f;
        if (valid && ok) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(dst + cb + e) =
                  make_uint4(Half<T>::pack(o[e], o[e + 1]), Half<T>::pack(o[e + 2], o[e + 3]),
                             Half<T>::pack(o[e + 4], o[e + 5]), Half<T>::pack(o[e + 6], o[e + 7]));
          } else {
            // a part in fp16: half the bytes of fp32, and 2^-11 of a mean of |v| <= 61440 at most
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(part + cb + e) =
                  make_uint4(pack_f16x2(o[e], o[e + 1]), pack_f16x2(o[e + 2], o[e + 3]),
                             pack_f16x2(o[e + 4], o[e + 5]), pack_f16x2(o[e + 6], o[e + 7]));
          }
        }
      }
      if (valid && ok) {
        if (!whole)
          a.part_lse[at] = lse2;
        else if (a.lse)
          a.lse[((size_t)pc.seq * a.rows + j) * a.n_q + h] = lse2 * 0.6931471805599453f;
      }
      tc_fence_before();   // O is read before the next piece's products overwrite it (they wait for p_ready)
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int DH, typename T>
cudaError_t launch_many(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st) {
  static unsigned long long done = 0;
  if (first_on_device(&done)) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_attend_many_kernel<DH, T>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ManySmem<DH>::kBytes);
    if (e != cudaSuccess) return e;
  }
  return launch_k(kv4_attend_many_kernel<DH, T>, dim3(a.n_ctas), dim3(kManyThreads), ManySmem<DH>::kBytes, st, 1, c,
                  layer, a);
}

}  // namespace

cudaError_t kv4_attend_many(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st) {
  if (c.dh == 128)
    return a.fp16 ? launch_many<128, __half>(c, layer, a, st) : launch_many<128, __nv_bfloat16>(c, layer, a, st);
  return a.fp16 ? launch_many<64, __half>(c, layer, a, st) : launch_many<64, __nv_bfloat16>(c, layer, a, st);
}

}  // namespace dg
