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
  int takes;          // which sequences this kernel takes (Takes)
  long long budget;   // of chunk_takes
  uint32_t* tickets;  // [grid], zero between calls
  float* partial;     // two pieces per CTA
};

enum Takes : int { kEvery, kShort, kChunk };

// Whether a sequence of `rows` query rows (new tokens times the group) per key/value head that see
// np pages goes to the chunk kernel; the reasons stand at chunk_budget (fl_attn.cu).
constexpr int kShortRows = 64, kChunkRows = 256, kFreeRows = 56;
__host__ __device__ __forceinline__ bool chunk_takes(long long rows, long long np, long long budget) {
  return rows > kShortRows && (rows > kChunkRows || (rows - kFreeRows) * np > budget);
}

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
  if (a.takes != kEvery && chunk_takes((long long)g.s.n * a.group, g.np, a.budget) != (a.takes == kChunk))
    g.s.n = 0;  // the other kernel's
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

// Values of eight elements from the high (and low) nibbles of one word, as four bf16 pairs, exactly.
// A small integer n < 256 is the bf16 bit pattern of n 2^-133 (subnormals and the first binade run
// on without a gap), so one fused multiply-add per pair turns masked bits into a centred value:
//   D8: u 2^-133 * 2^126 - 1          = (u - 128) / 128          (8 significant bits)
//   D4: h 2^-133 * 2^127 - 241 / 2^11 = (16 h - 120.5) / 1024    (|32 h - 241| < 2^8: exact too)
// kFactor<> gives the value back; it goes into the token's scale. Pair k holds the nibbles at bits
// 4 k and 16 + 4 k. 12 (D8) or 9 (D4) instructions per word, against 22 and 11 when each nibble is
// biased and recentred by itself.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
template <bool kD8>
__host__ __device__ constexpr float value_factor() { return kD8 ? 128.f : 1024.f; }
template <bool kD8>
__device__ __forceinline__ void unpack_word(uint32_t hi, uint32_t lo, uint32_t (&r)[4]) {
  if (kD8) {
    const uint32_t x = ((hi << 4) & 0xF0F0F0F0u) | (lo & 0x0F0F0F0Fu);
    const uint32_t y = (hi & 0xF0F0F0F0u) | ((lo >> 4) & 0x0F0F0F0Fu);
    r[0] = fma_bf16x2(x & 0x00FF00FFu, 0x7E807E80u, 0xBF80BF80u);
    r[1] = fma_bf16x2(y & 0x00FF00FFu, 0x7E807E80u, 0xBF80BF80u);
    r[2] = fma_bf16x2(__byte_perm(x, 0u, 0x4341), 0x7E807E80u, 0xBF80BF80u);
    r[3] = fma_bf16x2(__byte_perm(y, 0u, 0x4341), 0x7E807E80u, 0xBF80BF80u);
  } else {
    const uint32_t w = hi >> 8;
    r[0] = fma_bf16x2(hi & 0x000F000Fu, 0x7F007F00u, 0xBDF1BDF1u);
    r[1] = fma_bf16x2(hi & 0x00F000F0u, 0x7D007D00u, 0xBDF1BDF1u);
    r[2] = fma_bf16x2(w & 0x000F000Fu, 0x7F007F00u, 0xBDF1BDF1u);
    r[3] = fma_bf16x2(w & 0x00F000F0u, 0x7D007D00u, 0xBDF1BDF1u);
  }
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ float lds32(const uint8_t* p) { return *reinterpret_cast<const float*>(p); }

__device__ __forceinline__ uint32_t atom_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Sequence whose units hold u: the last i with pre[i] <= u (empty sequences are passed over).
__device__ __forceinline__ int find_seq(const long long* pre, int n, long long u) {
  int lo = 0, hi = n;  // pre[lo] <= u < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace attn

namespace attn_tc {  // fl_attn_tc.cu
size_t partial_bytes(int D, int nsm);
fl_status launch(const attn::Args& a, int D, int nsm, cudaStream_t st);
}  // namespace attn_tc
}  // namespace fl
