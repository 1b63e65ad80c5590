// kv4_kernels.h -- internal launch interface between the 4-bit cache's entry points (kv4_api.cu) and its kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dg_kernels.h"

namespace dg {

// Device view of a cache: the caller's pool and the sections of its book (see dg_kv4_cache in dg.h).
struct Kv4View {
  uint8_t* pool;         // [n_layers][n_pages][n_kv][72 d_head] bytes
  int32_t* head;         // [0] error code, [1] moves of the last page call, [2] live pages of the last compaction,
                         // [3] error code of a wait (apart, since a wait gives up once it is set),
                         // [4] what the last check of a prefix found
  int32_t *lens, *refs, *table;
  int32_t *move_src, *move_dst, *map;   // scratch of the page calls, n_pages words each
  int n_layers, n_kv, dh, n_pages, n_seq, max_pages;
};

enum : int { KV4_WORD_ERR = 0, KV4_WORD_MOVES = 1, KV4_WORD_LIVE = 2, KV4_WORD_WAIT = 3, KV4_WORD_PREFIX = 4, KV4_HEAD_WORDS = 16 };

// K / V rows of an append or a read: element (seq, row, head, c) at seq * s_seq + row * s_row + head * s_head + c.
struct Kv4Rows {
  void *k, *v;
  long long k_seq, k_row, k_head, v_seq, v_row, v_head;
  const int32_t* n_rows;   // rows of each sequence (null: `rows` each)
  int rows;
  int fp16;                // element type: bf16 (0) or fp16 (1)
  // One sequence's whole prefix instead of all sequences' last rows: sequence only - 1 (0: all), whose length has to
  // be `rows`; v then has its positions side by side and its channels v_row apart (bf16).
  int only;
};

cudaError_t kv4_rows(const Kv4View& c, int layer, const Kv4Rows& r, bool write, cudaStream_t st);
// Whether sequence `slot` has P positions, on pages of the pool: 0 or the code that is recorded, in KV4_WORD_PREFIX.
cudaError_t kv4_check_prefix(const Kv4View& c, int slot, int P, cudaStream_t st);

// page bookkeeping; each is one launch on the book, extend and compact with a second one that moves pages
cudaError_t kv4_extend(const Kv4View& c, const int32_t* counts, int n_sms, cudaStream_t st);
cudaError_t kv4_fork(const Kv4View& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t st);
cudaError_t kv4_free(const Kv4View& c, const int32_t* slots, int n, cudaStream_t st);
cudaError_t kv4_compact(const Kv4View& c, int n_sms, cudaStream_t st);

struct Kv4Attn {
  const void* q;
  void* out;
  float* lse;              // [n_seq][rows][n_q] or null
  const int32_t* n_rows;
  long long q_seq, q_row, q_head, o_seq, o_row, o_head;
  int n_q, rows, causal, fp16;
  int group;               // query heads of a KV head
  uint32_t group_mul;      // r / group = (high word of r * group_mul, plus r) >> group_shift
  int group_shift;
  float scale;
  int cluster;             // CTAs of a unit's cluster (the rows are joined there), 0: divide the line
  int n_ctas;              // CTAs among which the work is divided
  int min_share;           // key steps that a CTA takes at least
  void* line;              // header of the division: 16 bytes and n_seq words of 8 bytes
  void* part_o;            // normalised; few rows: fp32 [2 n_ctas][tile][dh]; many: 16-byte chunks of fp16, or of
                           // fp32 for an fp16 output, [2 n_ctas][chunk][tile]
  float* part_lse;         // [2 n_ctas][rows of a tile], base 2; many: pairs of it and the power of two by which the
                           // row's values in part_o are to be multiplied
};

// Few rows of a KV head (single tokens): tiles of 8 rows, steps of one page, mma.sync on fragments dequantised in
// registers.  Many rows (canvases, prompt chunks): tiles of 256 rows, steps of one page, tcgen05.
constexpr int kKv4FewTile = 8, kKv4FewStep = 64, kKv4MaxCluster = 16;
// CTAs of the few-rows form that an SM holds at once: by shared memory, by registers.
constexpr __host__ __device__ int kv4_few_ctas(int dh) { return dh == 128 ? 3 : 4; }
constexpr int kKv4ManyTile = 256, kKv4ManyStep = 64, kKv4MaxManyCluster = 8;
cudaError_t kv4_attend_few(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st);
cudaError_t kv4_attend_many(const Kv4View& c, int layer, const Kv4Attn& a, cudaStream_t st);
// How many clusters of n CTAs of the many-rows form the current device runs at once (0 without a device).
int kv4_many_clusters(int dh, int n);
cudaError_t kv4_attend_merge(const Kv4View& c, const Kv4Attn& a, bool few, cudaStream_t st);

// the checks of a cache's shape and buffers that every entry point makes, and its device view
dg_status kv4_check_cache(const char* fn, const dg_kv4_cache* c);
Kv4View kv4_view(const dg_kv4_cache* c);

// Kernel attributes are per device: `set` (which may run twice where two threads come first at once) runs until it has
// succeeded on the current device; `done` is the kernel's own word of devices.
template <typename F>
cudaError_t once_per_device(unsigned long long* done, F set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (__atomic_load_n(done, __ATOMIC_ACQUIRE) & bit) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) __atomic_fetch_or(done, bit, __ATOMIC_RELEASE);
  return e;
}

}  // namespace dg
