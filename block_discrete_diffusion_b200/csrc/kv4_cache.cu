// kv4_cache.cu -- the paged 4-bit cache: rows in and out, and its pages.
//
// Rows.  A CTA owns one (sequence, page, KV head) block, so every byte of a page has one writer.  A thread takes
// whole words of the block (positions g and g + 8 of K, a quad of positions of V) with 8 channels, so that a
// row's loads and stores are contiguous over the lanes; two neighbours share a scale.  Only words that some other row
// shares are read first.  Bound by memory: a value costs 2 bytes on one side and 0.5625 on the other; all of a
// thread's loads are under way before the first is used (32 KB of rows a CTA).  32767 positions in and out take 71 us
// (4.9 TB/s); that every CTA looks at all pages of its sequence's rows before it stores costs 4 us of them.
//
// Pages.  The book (lengths, reference counts, tables) is a few hundred KB at most and its updates depend on one
// another through a prefix sum, so one CTA does each of them in one launch; whatever moves page contents is left as a
// list of (from, to) for a second launch over the whole GPU (whose CTAs are placed while the first runs; one launch
// whose other CTAs wait for the list measured 33.5 us instead of 23.5 for 32 copies of 2.2 MB).  Nothing changes when
// a call cannot be carried out whole: the error word tells.
#include <type_traits>

#include "kv4.cuh"
#include "kv4_kernels.h"

namespace dg {

namespace {

// 8 elements (16 bytes) of a row
template <typename T>
__device__ __forceinline__ uint4 load8(const void* base, long long at) {
  return *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
}
template <typename T>
__device__ __forceinline__ void widen8(uint4 q, float (&x)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    x[2 * c] = Half<T>::lo(w[c]);
    x[2 * c + 1] = Half<T>::hi(w[c]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(void* base, long long at, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(static_cast<T*>(base) + at) =
      make_uint4(Half<T>::pack(x[0], x[1]), Half<T>::pack(x[2], x[3]), Half<T>::pack(x[4], x[5]),
                 Half<T>::pack(x[6], x[7]));
}

// Scale byte of the 16 values that this lane and its neighbour (lane ^ 1) hold; the values become quotients on the grid
// that to_e2m1_word rounds.  Both lanes take part.
__device__ __forceinline__ uint32_t to_quotients(float (&x)[8]) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(x[i]));
  amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const uint32_t byte = ue5m3_scale(amax);
  const float s = ue5m3_to_f32(byte);
  const float r = s > 0.f ? fast_rcp(s) : 0.f;
  const uint64_t rr = pack_f32x2(r, r);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t y = on_grid2(pack_f32x2(x[i], x[i + 1]), rr);
    x[i] = lo_f32(y);
    x[i + 1] = hi_f32(y);
  }
  return byte;
}

// v's bits of `mask` into *p
__device__ __forceinline__ void merge_words(uint2* p, uint2 v, uint32_t mask) {
  if (mask != 0xffffffffu) {
    const uint2 o = *p;
    v = make_uint2((o.x & ~mask) | (v.x & mask), (o.y & ~mask) | (v.y & mask));
  }
  *p = v;
}
__device__ __forceinline__ void merge_words(uint4* p, uint4 v, uint32_t mask) {
  if (mask != 0xffffffffu) {
    const uint4 o = *p;
    v = make_uint4((o.x & ~mask) | (v.x & mask), (o.y & ~mask) | (v.y & mask), (o.z & ~mask) | (v.z & mask),
                   (o.w & ~mask) | (v.w & mask));
  }
  *p = v;
}

// 8 channels of two neighbouring positions of a transposed V (positions side by side, channels `stride` elements
// apart): each word holds both positions of a channel
template <typename T>
__device__ __forceinline__ void load_pairs(const void* base, long long at, long long stride, float (&x0)[8],
                                           float (&x1)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const T*>(base) + at + c * stride);
    x0[c] = Half<T>::lo(w);
    x1[c] = Half<T>::hi(w);
  }
}

// Rows [len - n, len) of every sequence into (Write) or out of its pages.  2 DH threads: each takes two half blocks
// of K (8 channels of two positions) and one of V (8 channels of four positions).  Whole: one sequence's prefix, V
// transposed.
template <int DH, typename T, bool Write, bool Whole>
__global__ void __launch_bounds__(2 * DH) kv4_rows_kernel(Kv4View c, int layer, Kv4Rows r) {
  using F = Kv4<DH>;
  constexpr int kThreads = 2 * DH, kBlocks = DH / 16;
  pdl_trigger();
  pdl_wait();
  const int seq = Whole ? r.only - 1 : blockIdx.z, head = blockIdx.y;
  const int len = c.lens[seq];
  const int n = r.n_rows ? r.n_rows[seq] : r.rows;
  if (n == 0 && !Whole) return;
  if (Whole && n != len) {
    if (threadIdx.x == 0) report_error(c.head, DEV_ERR_BAD_COUNT);
    return;
  }
  const long long cap = (long long)c.max_pages * kPage;
  if (n < 0 || n > r.rows || n > len || len > cap) {
    if (threadIdx.x == 0) report_error(c.head, DEV_ERR_BAD_COUNT);
    return;
  }
  const int start = len - n;
  const int lp = start / kPage + blockIdx.x;
  if ((long long)lp * kPage >= len) return;
  const int32_t* table = c.table + (size_t)seq * c.max_pages;
  const int page = min(max(table[lp], 0), c.n_pages - 1);   // (looked at below; in the pool whatever it is)
  // All of the call's pages of this sequence are looked at by each of its CTAs before its first store, so that the rows
  // move whole or not at all.  Whole CTA, once its loads of rows are under way
  auto refused = [&] {
    int bad = 0;
    for (int i = start / kPage + threadIdx.x; (long long)i * kPage < len; i += kThreads) {
      const int p = table[i];
      const bool in = p >= 0 && p < c.n_pages;
      bad |= !in || (Write && c.refs[p] != 1);   // (a page with other owners is nobody's to write)
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) report_error(c.head, DEV_ERR_BAD_INDEX);
    return bad != 0;
  };
  uint8_t* block = c.pool + (((size_t)layer * c.n_pages + page) * c.n_kv + head) * F::kBytes;
  const int lo = max(start - lp * kPage, 0), hi = min(len - lp * kPage, kPage);   // positions of this page
  const long long row0 = (long long)lp * kPage - start;                          // row of the page's position 0
  const long long kb = (Whole ? 0 : seq * r.k_seq) + head * r.k_head;
  const long long vb = (Whole ? 0 : seq * r.v_seq) + head * r.v_head;
  const int u = threadIdx.x & 1, b = threadIdx.x / 2 % kBlocks, rest = threadIdx.x / 2 / kBlocks;   // rest: 0 .. 15

  // K: two pairs of positions p, p + 8
  const int t = b / F::kH, jh = b % F::kH;
  int kp[2];
  bool in0[2], in1[2];
  uint2* k_words[2];
  uint8_t* k_scale[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int pair = rest + 16 * i, kt = pair / 8, g = pair % 8;
    kp[i] = kt * 16 + g;
    in0[i] = kp[i] >= lo && kp[i] < hi;
    in1[i] = kp[i] + 8 >= lo && kp[i] + 8 < hi;
    k_words[i] = reinterpret_cast<uint2*>(block + ((kt * F::kH + jh) * 32 + g * 4 + t) * 16) + u;
    k_scale[i] = block + F::kSk + (g * 4 + t) * 8 * F::kH + 2 * kt * F::kH + jh;   // position p; p + 8 is kH further
  }
  // V: positions 2t, 2t + 1, 2t + 8, 2t + 9 of a tile
  const int vt = rest / 4, vq = rest % 4, vp = vt * 16 + 2 * vq;
  bool in[4];
  uint32_t v_mask = 0, s_mask = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int p = vp + (e & 1) + 8 * (e >> 1);
    in[e] = p >= lo && p < hi;
    v_mask |= in[e] ? 0x0f0fu << (16 * (e >> 1) + 4 * (e & 1)) : 0u;
    s_mask |= in[e] ? 0xffu << (8 * e) : 0u;
  }
  const int v_h = F::kH == 2 ? u : 0, v_g = F::kH == 2 ? b : 2 * b + u;
  uint4* v_words = reinterpret_cast<uint4*>(block + F::kV + ((vt * F::kH + v_h) * 32 + v_g * 4 + vq) * 16);
  uint32_t* v_scale = reinterpret_cast<uint32_t*>(block + F::kSv + ((b * 4 + vq) * 4 + vt) * 4);
  const int ch = b * 16 + 8 * u;
  auto k_at = [&](int p) { return kb + (row0 + p) * r.k_row + ch; };
  // (Whole: channel ch of position p; a pair's two positions share a word, which lies inside the caller's rows of
  // positions even where the second one is behind the end)
  auto vt_at = [&](int pair) { return vb + ch * r.v_row + lp * (long long)kPage + vp + 8 * pair; };
  auto v_at = [&](int e) { return vb + (row0 + vp + (e & 1) + 8 * (e >> 1)) * r.v_row + ch; };

  if constexpr (Write) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 k0[2], k1[2], v[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k0[i] = in0[i] ? load8<T>(r.k, k_at(kp[i])) : zero;
      k1[i] = in1[i] ? load8<T>(r.k, k_at(kp[i] + 8)) : zero;
    }
    float x[4][8];
    if constexpr (Whole) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[e][k] = 0.f;
      if (in[0]) load_pairs<T>(r.v, vt_at(0), r.v_row, x[0], x[1]);
      if (in[2]) load_pairs<T>(r.v, vt_at(1), r.v_row, x[2], x[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = in[e] ? load8<T>(r.v, v_at(e)) : zero;
    }
    if (refused()) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!__any_sync(0xffffffffu, in0[i] || in1[i])) continue;   // (single tokens: most warps have nothing)
      float x0[8], x1[8];
      widen8<T>(k0[i], x0);
      widen8<T>(k1[i], x1);
      const uint32_t s0 = to_quotients(x0), s1 = to_quotients(x1);
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = to_e2m1_word(x0[4 * j], x0[4 * j + 1], x1[4 * j], x1[4 * j + 1], x0[4 * j + 2], x0[4 * j + 3],
                            x1[4 * j + 2], x1[4 * j + 3]);
      if (in0[i] || in1[i])
        merge_words(k_words[i], make_uint2(w[0], w[1]), (in0[i] ? 0x00ff00ffu : 0u) | (in1[i] ? 0xff00ff00u : 0u));
      if (u == 0 && in0[i]) k_scale[i][0] = (uint8_t)s0;
      if (u == 0 && in1[i]) k_scale[i][F::kH] = (uint8_t)s1;
    }
    if (!__any_sync(0xffffffffu, v_mask != 0)) return;
    uint32_t s = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (!Whole) widen8<T>(v[e], x[e]);
      s |= to_quotients(x[e]) << (8 * e);
    }
    if (v_mask) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = to_e2m1_word(x[0][2 * j], x[1][2 * j], x[0][2 * j + 1], x[1][2 * j + 1], x[2][2 * j], x[3][2 * j],
                            x[2][2 * j + 1], x[3][2 * j + 1]);
      merge_words(v_words, make_uint4(w[0], w[1], w[2], w[3]), v_mask);
      if (u == 0) *v_scale = s_mask == 0xffffffffu ? s : (*v_scale & ~s_mask) | (s & s_mask);
    }
  } else {
    const bool some = __any_sync(0xffffffffu, in0[0] || in1[0] || in0[1] || in1[1] || v_mask);
    uint2 kw[2];
    float ks0[2], ks1[2];
    uint4 vw;
    uint32_t vs;
    if (some) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        kw[i] = *k_words[i];
        ks0[i] = ue5m3_to_f32(k_scale[i][0]);
        ks1[i] = ue5m3_to_f32(k_scale[i][F::kH]);
      }
      vw = *v_words;
      vs = *v_scale;
    }
    if (refused() || !some) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[2] = {kw[i].x, kw[i].y};
      float x0[8], x1[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t o[4];
        e2m1_to_f16(w[j], o);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x0[4 * j + 2 * e] = Half<__half>::lo(o[2 * e]) * ks0[i];
          x0[4 * j + 2 * e + 1] = Half<__half>::hi(o[2 * e]) * ks0[i];
          x1[4 * j + 2 * e] = Half<__half>::lo(o[2 * e + 1]) * ks1[i];
          x1[4 * j + 2 * e + 1] = Half<__half>::hi(o[2 * e + 1]) * ks1[i];
        }
      }
      if (in0[i]) store8<T>(r.k, k_at(kp[i]), x0);
      if (in1[i]) store8<T>(r.k, k_at(kp[i] + 8), x1);
    }
    const uint32_t w[4] = {vw.x, vw.y, vw.z, vw.w};
    float x[4][8], sv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sv[e] = ue5m3_to_f32((vs >> (8 * e)) & 0xff);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o[4];
      e2m1_to_f16(w[j], o);
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // o[e]: channel e & 1, positions 2 (e >> 1) + {0, 1} of the quad
        x[2 * (e >> 1)][2 * j + (e & 1)] = Half<__half>::lo(o[e]) * sv[2 * (e >> 1)];
        x[2 * (e >> 1) + 1][2 * j + (e & 1)] = Half<__half>::hi(o[e]) * sv[2 * (e >> 1) + 1];
      }
    }
    if constexpr (Whole) {
#pragma unroll
      for (int pair = 0; pair < 2; ++pair)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          T* dst = static_cast<T*>(r.v) + vt_at(pair) + k * r.v_row;
          const uint32_t w = Half<T>::pack(x[2 * pair][k], x[2 * pair + 1][k]);
          if (in[2 * pair + 1])
            *reinterpret_cast<uint32_t*>(dst) = w;
          else if (in[2 * pair])   // (the position behind the prefix stays as it was)
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w;
        }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (in[e]) store8<T>(r.v, v_at(e), x[e]);
    }
  }
}

template <int DH, typename T>
cudaError_t launch_rows(const Kv4View& c, int layer, const Kv4Rows& r, bool write, cudaStream_t st) {
  const int pages = (int)(((long long)r.rows + kPage - 2) / kPage + 1);   // the rows may begin at a page's last position
  const dim3 grid(pages < c.max_pages ? pages : c.max_pages, c.n_kv, r.only ? 1 : c.n_seq);
  if (r.only) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return launch_k(write ? kv4_rows_kernel<DH, T, true, true> : kv4_rows_kernel<DH, T, false, true>, grid,
                      dim3(2 * DH), 0, st, 1, c, layer, r);
    return cudaErrorInvalidValue;
  }
  return launch_k(write ? kv4_rows_kernel<DH, T, true, false> : kv4_rows_kernel<DH, T, false, false>, grid, dim3(2 * DH),
                  0, st, 1, c, layer, r);
}

__device__ __forceinline__ int pages_of(long long len) { return (int)((len + kPage - 1) / kPage); }

// One CTA.  (P is at most max_pages pages.)
constexpr int kCheckThreads = 256;
__global__ void __launch_bounds__(kCheckThreads) kv4_check_prefix_kernel(Kv4View c, int slot, int P) {
  pdl_trigger();
  pdl_wait();
  const bool fits = c.lens[slot] == P;
  int bad = 0;
  for (int i = threadIdx.x; fits && i < pages_of(P); i += kCheckThreads) {
    const int page = c.table[(size_t)slot * c.max_pages + i];
    bad |= page < 0 || page >= c.n_pages;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x != 0) return;
  const int code = !fits ? DEV_ERR_BAD_COUNT : bad ? DEV_ERR_BAD_INDEX : 0;
  c.head[KV4_WORD_PREFIX] = code;
  if (code) report_error(c.head, code);
}

// ---------------------------------------------------------------------------------------------
// the book
// ---------------------------------------------------------------------------------------------
constexpr int kBookThreads = 1024;
constexpr int kMaxSeq = 4096;     // sequences of a cache (dg_kv4_cache): one word of shared memory each

// exclusive prefix sum over the CTA's threads; *total: the sum (all threads)
__device__ int block_scan(int v, int* total) {
  __shared__ int warp_sums[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const int w = warp_sums[lane];
    int ws = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, ws, o);
      if (lane >= o) ws += u;
    }
    warp_sums[lane] = ws - w;
    if (lane == 31) warp_sums[32] = ws;
  }
  __syncthreads();
  const int before = warp_sums[warp] + s - v;
  *total = warp_sums[32];
  __syncthreads();
  return before;
}

// What a sequence needs to grow by `count`: pages it has, whether it copies its last one, pages to take.
struct Growth {
  int have, copy, need, last;
  int bad;   // 0, or the code of what does not fit
};
__device__ Growth growth(const Kv4View& c, const int32_t* counts, int seq) {
  Growth g{0, 0, 0, -1, 0};
  const int len = c.lens[seq], n = counts[seq];
  const long long now = (long long)len + n;
  if (n < 0 || len < 0 || now > (long long)c.max_pages * kPage) {
    g.bad = DEV_ERR_BAD_COUNT;
    return g;
  }
  g.have = pages_of(len);
  if (n > 0 && len % kPage) {
    g.last = c.table[(size_t)seq * c.max_pages + g.have - 1];
    if (g.last < 0 || g.last >= c.n_pages) {
      g.bad = DEV_ERR_BAD_INDEX;
      return g;
    }
    g.copy = c.refs[g.last] > 1;
  }
  g.need = g.copy + pages_of(now) - g.have;
  return g;
}

__global__ void __launch_bounds__(kBookThreads) kv4_extend_kernel(Kv4View c, const int32_t* counts) {
  pdl_trigger();
  pdl_wait();
  __shared__ int first[kMaxSeq + 1];   // index of a sequence's first page among the pages taken
  __shared__ int bad, n_moves, n_free;
  if (threadIdx.x == 0) bad = n_moves = n_free = 0;
  __syncthreads();
  // thread i: sequences [i per, i per + per), in order
  const int per = (c.n_seq + kBookThreads - 1) / kBookThreads;
  int mine = 0;
  for (int s = threadIdx.x * per; s < min(c.n_seq, (int)(threadIdx.x + 1) * per); ++s) {
    const Growth g = growth(c, counts, s);
    if (g.bad) atomicMax(&bad, g.bad);
    mine += g.need;
  }
  int total;
  int at = block_scan(mine, &total);
  for (int s = threadIdx.x * per; s < min(c.n_seq, (int)(threadIdx.x + 1) * per); ++s) {
    first[s] = at;
    at += growth(c, counts, s).need;
  }
  if (threadIdx.x == 0) first[c.n_seq] = total;
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) {
      report_error(c.head, bad);
      c.head[KV4_WORD_MOVES] = 0;
    }
    return;
  }
  // the `total` lowest free pages (into c.map), 4 counts a thread at a time
  for (int base = 0; base < c.n_pages && n_free < total; base += 4 * kBookThreads) {
    const int p = base + 4 * threadIdx.x;
    int v[4], k = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = p + e < c.n_pages && c.refs[p + e] == 0;
      k += v[e];
    }
    int found;
    const int before = n_free;   // (read before the scan's barriers: thread 0 adds to it after them)
    int rank = before + block_scan(k, &found);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (v[e]) {
        if (rank < total) c.map[rank] = p + e;
        ++rank;
      }
    if (threadIdx.x == 0) n_free += found;
    __syncthreads();
  }
  if (n_free < total) {
    if (threadIdx.x == 0) {
      report_error(c.head, DEV_ERR_NO_PAGES);
      c.head[KV4_WORD_MOVES] = 0;
    }
    return;
  }
  for (int i = threadIdx.x; i < total; i += kBookThreads) {
    int lo = 0, hi = c.n_seq - 1;   // the last sequence whose first page is at or before i
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (first[mid] <= i) lo = mid; else hi = mid - 1;
    }
    const int len = c.lens[lo], k = i - first[lo];
    const int have = pages_of(len);
    const int copy = first[lo + 1] - first[lo] - (pages_of((long long)len + counts[lo]) - have);
    const int page = c.map[i];
    int32_t* entry = c.table + (size_t)lo * c.max_pages + have - copy + k;
    if (k < copy) {
      const int m = atomicAdd(&n_moves, 1);
      c.move_src[m] = *entry;
      c.move_dst[m] = page;
      atomicSub(c.refs + *entry, 1);
    }
    *entry = page;
    c.refs[page] = 1;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < c.n_seq; s += kBookThreads) c.lens[s] += counts[s];
  if (threadIdx.x == 0) c.head[KV4_WORD_MOVES] = n_moves;
}

// Sequences dst[i] become second owners of src[i]'s pages, one warp for each pair.
__global__ void __launch_bounds__(kBookThreads) kv4_fork_kernel(Kv4View c, const int32_t* src, const int32_t* dst, int n) {
  pdl_trigger();
  pdl_wait();
  __shared__ int times[kMaxSeq];   // how often a sequence is a destination
  __shared__ int bad;
  for (int s = threadIdx.x; s < c.n_seq; s += kBookThreads) times[s] = 0;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= c.n_seq || b < 0 || b >= c.n_seq || c.lens[b] != 0 || c.lens[a] < 0 ||
        (long long)c.lens[a] > (long long)c.max_pages * kPage)
      bad = 1;
    else
      atomicAdd(times + b, 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n && !bad; i += kBookThreads)
    if (times[dst[i]] != 1 || times[src[i]] != 0) bad = 1;
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) report_error(c.head, DEV_ERR_BAD_INDEX);
    return;
  }
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += kBookThreads / 32) {
    const int a = src[i], b = dst[i], len = c.lens[a];
    for (int k = lane; k < pages_of(len); k += 32) {
      const int page = c.table[(size_t)a * c.max_pages + k];
      c.table[(size_t)b * c.max_pages + k] = page;
      if (page >= 0 && page < c.n_pages) atomicAdd(c.refs + page, 1);
    }
    if (lane == 0) c.lens[b] = len;
  }
}

__global__ void __launch_bounds__(kBookThreads) kv4_free_kernel(Kv4View c, const int32_t* slots, int n) {
  pdl_trigger();
  pdl_wait();
  __shared__ int times[kMaxSeq];
  __shared__ int bad;
  for (int s = threadIdx.x; s < c.n_seq; s += kBookThreads) times[s] = 0;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    const int s = slots[i];
    if (s < 0 || s >= c.n_seq)
      bad = 1;
    else if (atomicAdd(times + s, 1))
      bad = 1;
  }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) report_error(c.head, DEV_ERR_BAD_INDEX);
    return;
  }
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += kBookThreads / 32) {
    const int s = slots[i];
    const int pages = min(pages_of(max(c.lens[s], 0)), c.max_pages);
    for (int k = lane; k < pages; k += 32) {
      int32_t* entry = c.table + (size_t)s * c.max_pages + k;
      const int page = *entry;
      if (page >= 0 && page < c.n_pages) atomicSub(c.refs + page, 1);
      *entry = -1;
    }
    __syncwarp();
    if (lane == 0) c.lens[s] = 0;
  }
}

// Live pages above the count of live pages move, in order, to the free places below it.
__global__ void __launch_bounds__(kBookThreads) kv4_compact_kernel(Kv4View c) {
  pdl_trigger();
  pdl_wait();
  int live = 0;
  for (int p = threadIdx.x; p < c.n_pages; p += kBookThreads) live += c.refs[p] > 0;
  int n_live;
  block_scan(live, &n_live);
  int n_holes = 0, n_moves = 0;
  for (int base = 0; base < c.n_pages; base += 4 * kBookThreads) {
    const int p = base + 4 * threadIdx.x;
    int hole[4], move[4], nh = 0, nm = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = p + e < c.n_pages;
      const bool used = in && c.refs[p + e] > 0;
      hole[e] = in && p + e < n_live && !used;
      move[e] = p + e >= n_live && used;
      nh += hole[e];
      nm += move[e];
    }
    int th, tm;
    int rh = n_holes + block_scan(nh, &th), rm = n_moves + block_scan(nm, &tm);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (hole[e]) c.move_dst[rh++] = p + e;
      if (move[e]) c.move_src[rm++] = p + e;
    }
    n_holes += th;
    n_moves += tm;
  }
  __syncthreads();   // as many holes as moves: both lists are whole and visible to the CTA
  for (int m = threadIdx.x; m < n_moves; m += kBookThreads) {
    const int s = c.move_src[m], d = c.move_dst[m];
    c.map[s] = d;
    c.refs[d] = c.refs[s];
    c.refs[s] = 0;
  }
  if (threadIdx.x == 0) {
    c.head[KV4_WORD_MOVES] = n_moves;
    c.head[KV4_WORD_LIVE] = n_live;
  }
}

// Page contents: move m takes page move_src[m] to move_dst[m] in every layer.  No page is both a source and a
// destination, so the order does not matter.  With Remap the page tables follow (c.map of a moved page).
constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = kMoveThreads * 16 * 8;   // bytes a CTA copies at a time: 8 loads in flight a thread

template <bool Remap>
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(Kv4View c, size_t page_bytes) {
  pdl_trigger();
  pdl_wait();
  const int moves = c.head[KV4_WORD_MOVES];
  const int per = (int)((page_bytes + kMoveChunk - 1) / kMoveChunk);
  const long long work = (long long)moves * c.n_layers * per;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const int part = (int)(w % per);
    const int layer = (int)(w / per % c.n_layers), m = (int)(w / per / c.n_layers);
    const size_t plane = (size_t)layer * c.n_pages;
    const size_t off = (size_t)part * kMoveChunk;
    const uint4* s = reinterpret_cast<const uint4*>(c.pool + (plane + c.move_src[m]) * page_bytes + off);
    uint4* d = reinterpret_cast<uint4*>(c.pool + (plane + c.move_dst[m]) * page_bytes + off);
    const int n = (int)(min((size_t)kMoveChunk, page_bytes - off) / 16);
    uint4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e * kMoveThreads + (int)threadIdx.x < n) v[e] = s[e * kMoveThreads + threadIdx.x];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e * kMoveThreads + (int)threadIdx.x < n) d[e * kMoveThreads + threadIdx.x] = v[e];
  }
  if (Remap && moves > 0) {
    const int n_live = c.head[KV4_WORD_LIVE];
    const long long entries = (long long)c.n_seq * c.max_pages;
    for (long long i = (long long)blockIdx.x * kMoveThreads + threadIdx.x; i < entries;
         i += (long long)gridDim.x * kMoveThreads) {
      const int page = c.table[i];
      if (page >= n_live && page < c.n_pages) c.table[i] = c.map[page];
    }
  }
}

// For at most `moves` moved pages.  Sixteen CTAs an SM where there can be that much work: with the eight that fit at
// once half of a 30-layer pool took 93 us instead of 85.
template <bool Remap>
cudaError_t launch_moves(const Kv4View& c, long long moves, int n_sms, cudaStream_t st) {
  const size_t page_bytes = (size_t)c.n_kv * 72 * c.dh;
  const long long work = moves * c.n_layers * (long long)((page_bytes + kMoveChunk - 1) / kMoveChunk);
  const int grid = (int)(work < 16 * n_sms ? work + 1 : 16 * n_sms);
  return launch_k(kv4_move_kernel<Remap>, dim3(grid), dim3(kMoveThreads), 0, st, 1, c, page_bytes);
}

}  // namespace

cudaError_t kv4_rows(const Kv4View& c, int layer, const Kv4Rows& r, bool write, cudaStream_t st) {
  if (c.dh == 128)
    return r.fp16 ? launch_rows<128, __half>(c, layer, r, write, st)
                  : launch_rows<128, __nv_bfloat16>(c, layer, r, write, st);
  return r.fp16 ? launch_rows<64, __half>(c, layer, r, write, st)
                : launch_rows<64, __nv_bfloat16>(c, layer, r, write, st);
}

cudaError_t kv4_check_prefix(const Kv4View& c, int slot, int P, cudaStream_t st) {
  return launch_k(kv4_check_prefix_kernel, dim3(1), dim3(kCheckThreads), 0, st, 1, c, slot, P);
}

cudaError_t kv4_extend(const Kv4View& c, const int32_t* counts, int n_sms, cudaStream_t st) {
  const cudaError_t e = launch_k(kv4_extend_kernel, dim3(1), dim3(kBookThreads), 0, st, 1, c, counts);
  return e != cudaSuccess ? e : launch_moves<false>(c, c.n_seq, n_sms, st);   // a copy for each sequence at most
}

cudaError_t kv4_fork(const Kv4View& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t st) {
  return launch_k(kv4_fork_kernel, dim3(1), dim3(kBookThreads), 0, st, 1, c, src, dst, n);
}

cudaError_t kv4_free(const Kv4View& c, const int32_t* slots, int n, cudaStream_t st) {
  return launch_k(kv4_free_kernel, dim3(1), dim3(kBookThreads), 0, st, 1, c, slots, n);
}

cudaError_t kv4_compact(const Kv4View& c, int n_sms, cudaStream_t st) {
  const cudaError_t e = launch_k(kv4_compact_kernel, dim3(1), dim3(kBookThreads), 0, st, 1, c);
  return e != cudaSuccess ? e : launch_moves<true>(c, c.n_pages / 2, n_sms, st);   // as many holes as moves
}

}  // namespace dg
