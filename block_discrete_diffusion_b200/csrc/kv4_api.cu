// kv4_api.cu -- entry points of the paged 4-bit cache (include/dg.h): argument checks and launches.  Host code only.
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>

#include <algorithm>

#include "dg.h"
#include "kv4_kernels.h"

#define DG_API extern "C" __attribute__((visibility("default")))

using namespace dg;

namespace {

dg_status bad(const char* fn, const char* why, dg_status st = DG_ERR_INVALID_ARG) {
  char msg[256];
  snprintf(msg, sizeof msg, "%s: %s", fn, why);
  return record_error(st, msg);
}

dg_status launched(const char* fn, cudaError_t e) {
  return e == cudaSuccess ? DG_OK : bad(fn, cudaGetErrorString(e), DG_ERR_CUDA);
}

constexpr int kMaxPages = 1 << 24;

const char* shape_error(const dg_kv4_cache* c) {
  if (!c) return "null cache";
  if (c->d_head != 64 && c->d_head != 128) return "d_head must be 64 or 128";
  if (c->n_layers <= 0 || c->n_kv <= 0 || c->n_pages <= 0 || c->n_seq <= 0 || c->max_pages <= 0)
    return "sizes must be positive";
  if (c->n_seq > 4096) return "n_seq must be at most 4096";
  if (c->n_pages > kMaxPages || c->max_pages > kMaxPages) return "n_pages and max_pages must be at most 2^24";
  if ((long long)c->n_seq * c->max_pages >= 1ll << 30) return "n_seq * max_pages must be below 2^30";
  if ((long long)c->n_seq * c->n_kv > 65535) return "n_seq * n_kv must be at most 65535";
  // (n_pages * n_kv * 72 * d_head is below 2^54)
  if ((1ll << 54) / c->n_layers < (long long)c->n_pages * c->n_kv * 72 * c->d_head)
    return "the pool must be at most 2^54 bytes";
  return nullptr;
}

size_t pad4(size_t n) { return (n + 3) & ~size_t(3); }

size_t pool_bytes(const dg_kv4_cache* c) {
  return (size_t)c->n_layers * c->n_pages * c->n_kv * 72 * c->d_head;
}
size_t table_words(const dg_kv4_cache* c) { return pad4((size_t)c->n_seq * c->max_pages); }
size_t book_words(const dg_kv4_cache* c) {
  return KV4_HEAD_WORDS + pad4(c->n_seq) + 4 * pad4(c->n_pages) + table_words(c);
}

bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

dg_status check_cache(const char* fn, const dg_kv4_cache* c) {
  if (const char* why = shape_error(c)) return bad(fn, why);
  if (!aligned16(c->d_pool) || !aligned16(c->d_book)) return bad(fn, "pool and book must be 16-byte aligned device buffers");
  if (c->pool_bytes < pool_bytes(c)) return bad(fn, "pool too small", DG_ERR_CAPACITY);
  if (c->book_bytes < 4 * book_words(c)) return bad(fn, "book too small", DG_ERR_CAPACITY);
  return DG_OK;
}

Kv4View view(const dg_kv4_cache* c) {
  Kv4View v{};
  int32_t* w = static_cast<int32_t*>(c->d_book);
  auto take = [&](size_t words) {
    int32_t* p = w;
    w += words;
    return p;
  };
  v.pool = static_cast<uint8_t*>(c->d_pool);
  v.head = take(KV4_HEAD_WORDS);
  v.lens = take(pad4(c->n_seq));
  v.refs = take(pad4(c->n_pages));
  v.table = take(table_words(c));
  v.move_src = take(pad4(c->n_pages));
  v.move_dst = take(pad4(c->n_pages));
  v.map = take(pad4(c->n_pages));
  v.n_layers = c->n_layers;
  v.n_kv = c->n_kv;
  v.dh = c->d_head;
  v.n_pages = c->n_pages;
  v.n_seq = c->n_seq;
  v.max_pages = c->max_pages;
  return v;
}

int current_sms() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// Whether some of the n elements of a dimension, d_head channels each, lie on one another: as outputs they would race.
bool overlap(long long n, int64_t stride, int d_head) { return n > 1 && stride < d_head && -stride < d_head; }

// How a call's work is divided: the form, and the CTAs among which it goes.  The host knows no lengths, so where they
// matter it goes by max_pages, the length that a sequence may have: with a table of 512 pages one token behind 577
// positions takes 11.0 us instead of 7.6, one canvas behind 2048 24.3 instead of 19.7 (a line and a second launch).
struct Plan {
  bool few;
  int cluster, n_ctas, min_share;
  size_t tile, row_bytes, stat_bytes;   // rows of a workspace slot, bytes of a row in it, of its lse and power
  size_t bytes(const dg_kv4_cache* c) const {
    return line_bytes(c) + 2 * (size_t)n_ctas * tile * (row_bytes + stat_bytes);
  }
  static size_t line_bytes(const dg_kv4_cache* c) { return (16 + 8 * (size_t)c->n_seq + 255) & ~size_t(255); }
};

constexpr size_t kWorkspaceSlack = 256;   // the parts begin at a multiple of it

// Rows of a KV head up to which the few-rows form runs whatever the lengths (32 sequences of 8192 positions, 8 KV
// heads: 8 rows 68 us, 32 rows 208 us, 64 rows 402 us; the other form 258 to 262 us for any of them).
constexpr int kFewRows = 32;

Plan plan_of(const dg_kv4_cache* c, int n_q, int rows) {
  Plan p{};
  const int sms = current_sms();
  const long long group_rows = (long long)rows * (n_q / c->n_kv);
  const int few_ctas = sms * kv4_few_ctas(c->d_head);
  // A cluster for each unit where the sequences cannot be long: one launch and no parts in memory (one token behind
  // 577 positions: 11.7 -> 7.0 us).  Longer units want more warps than a cluster of such CTAs has (32768 positions:
  // 21.2 us on the line, 24.8 in clusters of 16 CTAs, 24.3 of 12-warp CTAs that fill an SM), and units of different
  // lengths leave SMs idle: from about 24 pages a CTA on that costs more than the second launch.  Where the many-rows
  // form stands on the other side, its clusters win from 10 to 12 pages a CTA on (128 rows, 4 pages a CTA 8.3 us,
  // 12.2 in the other form; 10 pages 12.5 and 13.5; 24 pages 20.3 and 14.7; 48 rows, 6 pages 11.6 and 11.4, 12 pages
  // 15.8 and 14.5; heads of 64, 128 rows, 12 pages 13.3 and 13.9).
  const long long units = (group_rows + kKv4FewTile - 1) / kKv4FewTile * c->n_kv * c->n_seq;
  int n = kKv4MaxCluster;
  while (n > 1 && units * n > few_ctas) n /= 2;
  if (units <= few_ctas && c->max_pages <= (group_rows <= kFewRows ? 24 : n >= 4 ? 12 : 10) * n) p.cluster = n;
  p.few = p.cluster || group_rows <= kFewRows;
  if (p.few) {
    p.n_ctas = few_ctas;
    p.min_share = 4;                               // a page for each warp
    p.tile = kKv4FewTile;
    p.row_bytes = 4 * (size_t)c->d_head;
    p.stat_bytes = 4;
  } else {
    p.n_ctas = sms;                                // one CTA holds an SM
    // Clusters here too where all units' run at once and none is long (see above).  Eight CTAs of a GPC's SMs at
    // most, and fewer clusters than SMs / size would give: with 16 clusters of 8 the last ones waited (2304
    // positions, one canvas, in an earlier form of the join: 36.9 us; 16 clusters of 4 22.6 us, the line 23.8 us; 600
    // positions 30.5, 15.7, 19.6).  One canvas behind 2000 positions 19.2 us, 23.3 on the line; behind 9000 40.2 and
    // 45.0; two behind 6000, 24 pages a CTA, 40.8 and 49.8.  (Sequences of different lengths leave SMs idle, so not
    // up to where equal ones break even, 50 pages a CTA and more.)
    const long long many = (group_rows + kKv4ManyTile - 1) / kKv4ManyTile * c->n_kv * c->n_seq;
    int m = many <= sms ? kKv4MaxManyCluster : 0;
    while (m > 0 && many > kv4_many_clusters(c->d_head, m)) --m;
    if (m > 0 && c->max_pages <= (c->n_seq == 1 ? 32 : 24) * m) p.cluster = m;
    p.min_share = 1;
    p.tile = kKv4ManyTile;
    p.row_bytes = 4 * (size_t)c->d_head;           // (parts for a bf16 output take half of it)
    p.stat_bytes = 8;
  }
  return p;
}

dg_status check_rows(const char* fn, const dg_kv4_cache* c, int layer, const dg_kv4_rows* r, bool out) {
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  if (!r || !aligned16(r->k) || !aligned16(r->v)) return bad(fn, "k and v must be 16-byte aligned device buffers");
  if (layer < 0 || layer >= c->n_layers) return bad(fn, "layer out of range");
  if (r->dtype != DG_DTYPE_BF16 && r->dtype != DG_DTYPE_FP16) return bad(fn, "dtype must be bf16 or fp16");
  if (r->rows <= 0) return bad(fn, "rows must be positive");
  if ((r->k_seq | r->k_row | r->k_head | r->v_seq | r->v_row | r->v_head) & 7)
    return bad(fn, "strides must be multiples of 8 elements");
  const int dh = c->d_head;
  if (out && (overlap(c->n_seq, r->k_seq, dh) || overlap(r->rows, r->k_row, dh) || overlap(c->n_kv, r->k_head, dh) ||
              overlap(c->n_seq, r->v_seq, dh) || overlap(r->rows, r->v_row, dh) || overlap(c->n_kv, r->v_head, dh)))
    return bad(fn, "rows read out must not overlap");
  return DG_OK;
}

Kv4Rows rows_of(const dg_kv4_rows* r) {
  return Kv4Rows{r->k, r->v, r->k_seq, r->k_row, r->k_head, r->v_seq, r->v_row, r->v_head, r->d_rows, r->rows,
                 r->dtype == DG_DTYPE_FP16, 0};
}

}  // namespace

dg_status dg::kv4_check_cache(const char* fn, const dg_kv4_cache* c) { return check_cache(fn, c); }
Kv4View dg::kv4_view(const dg_kv4_cache* c) { return view(c); }

DG_API size_t dg_kv4_pool_bytes(const dg_kv4_cache* c) { return shape_error(c) ? 0 : pool_bytes(c); }
DG_API size_t dg_kv4_book_bytes(const dg_kv4_cache* c) { return shape_error(c) ? 0 : 4 * book_words(c); }

DG_API dg_status dg_kv4_init(const dg_kv4_cache* c, void* stream) {
  const char* fn = "dg_kv4_init";
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  const Kv4View v = view(c);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(c->d_book, 0, 4 * book_words(c), s);
  if (e == cudaSuccess) e = cudaMemsetAsync(v.table, 0xff, 4 * table_words(c), s);
  return launched(fn, e);
}

DG_API dg_status dg_kv4_extend(const dg_kv4_cache* c, const int32_t* d_counts, void* stream) {
  const char* fn = "dg_kv4_extend";
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  if (!d_counts) return bad(fn, "counts are null");
  return launched(fn, kv4_extend(view(c), d_counts, current_sms(), static_cast<cudaStream_t>(stream)));
}

DG_API dg_status dg_kv4_fork(const dg_kv4_cache* c, const int32_t* d_src, const int32_t* d_dst, int n, void* stream) {
  const char* fn = "dg_kv4_fork";
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  if (!d_src || !d_dst) return bad(fn, "src or dst is null");
  if (n <= 0 || n > c->n_seq) return bad(fn, "n must be in [1, n_seq]");
  return launched(fn, kv4_fork(view(c), d_src, d_dst, n, static_cast<cudaStream_t>(stream)));
}

DG_API dg_status dg_kv4_free(const dg_kv4_cache* c, const int32_t* d_slots, int n, void* stream) {
  const char* fn = "dg_kv4_free";
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  if (!d_slots) return bad(fn, "slots are null");
  if (n <= 0 || n > c->n_seq) return bad(fn, "n must be in [1, n_seq]");
  return launched(fn, kv4_free(view(c), d_slots, n, static_cast<cudaStream_t>(stream)));
}

DG_API dg_status dg_kv4_compact(const dg_kv4_cache* c, void* stream) {
  const char* fn = "dg_kv4_compact";
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  return launched(fn, kv4_compact(view(c), current_sms(), static_cast<cudaStream_t>(stream)));
}

DG_API dg_status dg_kv4_append(const dg_kv4_cache* c, int layer, const dg_kv4_rows* r, void* stream) {
  const char* fn = "dg_kv4_append";
  const dg_status st = check_rows(fn, c, layer, r, false);
  if (st != DG_OK) return st;
  return launched(fn, kv4_rows(view(c), layer, rows_of(r), true, static_cast<cudaStream_t>(stream)));
}

DG_API dg_status dg_kv4_read(const dg_kv4_cache* c, int layer, const dg_kv4_rows* r, void* stream) {
  const char* fn = "dg_kv4_read";
  const dg_status st = check_rows(fn, c, layer, r, true);
  if (st != DG_OK) return st;
  return launched(fn, kv4_rows(view(c), layer, rows_of(r), false, static_cast<cudaStream_t>(stream)));
}

DG_API size_t dg_kv4_attend_workspace_bytes(const dg_kv4_cache* c, int n_q, int rows) {
  if (shape_error(c) || n_q <= 0 || n_q % c->n_kv || n_q > 8192 || rows <= 0 || rows > 65536) return 0;
  return plan_of(c, n_q, rows).bytes(c) + kWorkspaceSlack;
}

DG_API dg_status dg_kv4_attend(const dg_kv4_cache* c, int layer, const dg_kv4_attn* a, void* ws, size_t ws_bytes,
                               void* stream) {
  const char* fn = "dg_kv4_attend";
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  if (!a || !aligned16(a->q) || !aligned16(a->out)) return bad(fn, "q and out must be 16-byte aligned device buffers");
  if (layer < 0 || layer >= c->n_layers) return bad(fn, "layer out of range");
  if (a->dtype != DG_DTYPE_BF16 && a->dtype != DG_DTYPE_FP16) return bad(fn, "dtype must be bf16 or fp16");
  if (a->n_q <= 0 || a->n_q % c->n_kv || a->n_q > 8192) return bad(fn, "n_q must be a multiple of n_kv in [1, 8192]");
  if (a->rows <= 0 || a->rows > 65536) return bad(fn, "rows must be in [1, 65536]");
  if (a->causal != 0 && a->causal != 1) return bad(fn, "causal must be 0 or 1");
  if (!(a->scale > 0.f) || !isfinite(a->scale)) return bad(fn, "scale must be positive and finite");
  if ((a->q_seq | a->q_row | a->q_head | a->o_seq | a->o_row | a->o_head) & 7)
    return bad(fn, "strides must be multiples of 8 elements");
  if (overlap(c->n_seq, a->o_seq, c->d_head) || overlap(a->rows, a->o_row, c->d_head) ||
      overlap(a->n_q, a->o_head, c->d_head))
    return bad(fn, "rows of out must not overlap");
  const Plan p = plan_of(c, a->n_q, a->rows);
  if (!ws || ws_bytes < p.bytes(c) + kWorkspaceSlack) return bad(fn, "workspace too small", DG_ERR_CAPACITY);
  Kv4Attn k{};
  k.q = a->q;
  k.out = a->out;
  k.lse = a->lse;
  k.n_rows = a->d_rows;
  k.q_seq = a->q_seq;
  k.q_row = a->q_row;
  k.q_head = a->q_head;
  k.o_seq = a->o_seq;
  k.o_row = a->o_row;
  k.o_head = a->o_head;
  k.n_q = a->n_q;
  k.group = a->n_q / c->n_kv;
  while (1 << k.group_shift < k.group) ++k.group_shift;
  k.group_mul = (uint32_t)(((1ull << 32) * ((1ull << k.group_shift) - k.group)) / k.group + 1);
  k.rows = a->rows;
  k.causal = a->causal;
  k.fp16 = a->dtype == DG_DTYPE_FP16;
  k.scale = a->scale;
  k.cluster = p.cluster;
  k.n_ctas = p.n_ctas;
  k.min_share = p.min_share;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
  k.line = base;
  k.part_o = base + Plan::line_bytes(c);
  k.part_lse = reinterpret_cast<float*>(base + Plan::line_bytes(c) + 2 * (size_t)p.n_ctas * p.tile * p.row_bytes);
  const Kv4View v = view(c);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = p.few ? kv4_attend_few(v, layer, k, s) : kv4_attend_many(v, layer, k, s);
  if (e == cudaSuccess && !p.cluster) e = kv4_attend_merge(v, k, p.few, s);
  return launched(fn, e);
}

DG_API dg_status dg_kv4_error(const dg_kv4_cache* c, void* stream, int* h_code) {
  const char* fn = "dg_kv4_error";
  const dg_status st = check_cache(fn, c);
  if (st != DG_OK) return st;
  if (!h_code) return bad(fn, "h_code is null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t w[4] = {0, 0, 0, 0};
  const Kv4View v = view(c);
  cudaError_t e = cudaMemcpyAsync(w, v.head, sizeof w, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  // a wait that ran out spoils whole outputs, so it comes first; the other word stays for the next call
  const int word = w[KV4_WORD_WAIT] ? KV4_WORD_WAIT : KV4_WORD_ERR;
  if (e == cudaSuccess && w[word]) e = cudaMemsetAsync(v.head + word, 0, 4, s);
  if (e != cudaSuccess) return launched(fn, e);
  *h_code = w[word];
  if (!*h_code) return DG_OK;
  char why[64];
  snprintf(why, sizeof why, "device-side error code %d", *h_code);
  return bad(fn, why, DG_ERR_DEVICE);
}
