// The paged key/value cache's layout and the sequence table, shared by the cache kernels
// (fl_kv.cu) and the attention kernels (fl_attn.cu, fl_attn_tc.cu).
#pragma once

#include "fl_common.cuh"

namespace fl {
namespace kv {

constexpr int kBlock = FL_KV_BLOCK;  // tokens of a page
constexpr int kScaleBytes = 512;     // key and value scales at the front of a record

__host__ __device__ constexpr int plane_bytes(int D) { return 32 * D; }
__host__ __device__ constexpr int record_bytes(int D) { return kScaleBytes + 128 * D; }
__host__ __device__ constexpr int depth_bytes(int D, bool d8) { return kScaleBytes + (d8 ? 128 : 64) * D; }

// Levels as the cache reads them: 0 ZERO, 1-2 D4, 3 and above D8.
__device__ __forceinline__ int level_of(const uint8_t* levels, size_t i) {
  if (!levels) return 4;
  const int l = __ldg(levels + i);
  return l == 0 ? 0 : l <= 2 ? 2 : 4;
}

struct Batch {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* start;  // NULL: one new token per sequence
  int n_seqs, max_blocks, rows, max_new;
};

enum : int { kErrSeq = 1, kErrPage = 2, kErrWait = 4 };  // bits of an error word

struct Seq {
  int row0, n, len;  // first row, new tokens, cached tokens; n = 0: nothing to do
};

// Sequence i, or n = 0 (and *bad set) where its entries contradict one another or the bounds.
__device__ __forceinline__ Seq seq_of(const Batch& b, int i, bool* bad) {
  Seq s;
  s.len = __ldg(b.lens + i);
  bool ok = s.len >= 0 && s.len / kBlock + (s.len % kBlock != 0) <= b.max_blocks;
  if (b.start) {
    s.row0 = __ldg(b.start + i);
    const int r1 = __ldg(b.start + i + 1);
    ok = ok && s.row0 >= 0 && r1 >= s.row0 && r1 <= b.rows;
    s.n = ok ? r1 - s.row0 : 0;
    ok = ok && s.n <= b.max_new && s.n <= s.len;
  } else {
    s.row0 = i;
    s.n = s.len > 0 ? 1 : 0;
  }
  if (!ok) {
    s.n = 0;
    *bad = true;
  }
  return s;
}

// Byte offsets inside a record (the layout of fl.h).
// Keys: the eight bytes of 16 dims (dim / 16) of slot j in a plane.
__device__ __forceinline__ int key_off(int D, int j, int d16) {
  const int s = (j >> 2) & 3, g = 2 * (j >> 4) + (j & 1);
  return 16 * (32 * ((D / 64) * s + (d16 >> 2)) + 4 * g + (d16 & 3)) + 8 * ((j >> 1) & 1);
}
// Values: the 16 bytes of dims 16 T + g and 16 T + 8 + g over slots 16 t .. 16 t + 15.
__device__ __forceinline__ int val_off(int T, int g, int t) { return 16 * (32 * T + 4 * g + t); }

// Host checks shared by the calls; FL_OK or the failure.
fl_status check_batch(const char* what, const fl_kv_cache* c, const fl_kv_batch* b);
fl_status check_rows(const char* what, const char* name, const void* p, int64_t stride, int width);
inline Batch batch_of(const fl_kv_batch* b) {
  return Batch{b->block_table, b->lens, b->new_start, b->n_seqs, b->max_blocks, b->rows, b->max_new};
}

}  // namespace kv
}  // namespace fl
