// What the two attention kernels (fl_attn.cu, fl_attn_tc.cu) share: the arguments, which pages a
// sequence's new tokens see, and which keys a query sees.
#pragma once

#include "fl_kv.cuh"

namespace fl {
namespace attn {

struct Args {
  const uint8_t* pages;
  int num_pages, kv_heads, heads, group;  // group = heads / kv_heads
  kv::Batch b;
  const uint8_t* levels;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  float scale_log2;  // scale * log2(e): the softmax runs on powers of two
  int window, sinks;
  int min_rows, max_rows;  // the kernel takes sequences whose n * group is in [min_rows, max_rows]
  uint32_t* tickets;  // [grid], zero between calls
  float* partial;     // two pieces per CTA
};

// The pages that a sequence's new tokens see, as one list: pages [0, sink_pages) and
// [win_page, blocks).
struct Geo {
  kv::Seq s;
  int pos0;               // position of the first new token
  int sink_pages, win_page, np;
};

__device__ __forceinline__ Geo geo_of(const Args& a, int i, bool* bad) {
  Geo g;
  g.s = kv::seq_of(a.b, i, bad);
  g.pos0 = g.s.len - g.s.n;
  const int blocks = g.s.len / kv::kBlock + (g.s.len % kv::kBlock != 0);
  g.sink_pages = g.win_page = 0;
  if (a.window > 0) {
    g.win_page = max(g.pos0 - a.window + 1, 0) / kv::kBlock;
    g.sink_pages = min((min(a.sinks, g.s.len) + kv::kBlock - 1) / kv::kBlock, g.win_page);
  }
  g.np = blocks - g.win_page + g.sink_pages;
  const long long rows = (long long)g.s.n * a.group;
  if (rows < a.min_rows || rows > a.max_rows) g.s.n = 0;  // the other kernel's, or nothing to do
  if (g.s.n == 0) g.np = 0;
  return g;
}

__device__ __forceinline__ int page_at(const Geo& g, int p) { return p < g.sink_pages ? p : g.win_page + p - g.sink_pages; }

__device__ __forceinline__ bool sees(const Args& a, int pos, int key) {
  return key <= pos && (a.window == 0 || pos - key < a.window || key < a.sinks);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Codes of eight elements from the high (and low) nibbles of one word, as bf16 pairs, exactly:
// 0x4300 | n is the bf16 value 128 + n, so the pair of nibbles at bits 4 k and 16 + 4 k becomes
//   D8: (128 + h - 144) * 16 + (128 + l) = 16 h + l - 128   (each step exact in bf16)
//   D4: 128 + h - 136 = h - 8                              (times 16, plus 7.5, is the value)
__device__ __forceinline__ uint32_t nib(uint32_t w, int k) { return ((w >> (4 * k)) & 0x000F000Fu) | 0x43004300u; }
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
constexpr uint32_t kMinus136 = 0xC308C308u, kMinus144 = 0xC310C310u, kSixteen = 0x41804180u;
template <bool kD8>
__device__ __forceinline__ uint32_t code_pair(uint32_t hi, uint32_t lo, int k) {
  if (kD8) return fma_bf16x2(add_bf16x2(nib(hi, k), kMinus144), kSixteen, nib(lo, k));
  return add_bf16x2(nib(hi, k), kMinus136);
}

}  // namespace attn
}  // namespace fl
