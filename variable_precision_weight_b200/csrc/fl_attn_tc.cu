// Attention of prompt chunks (many new tokens per sequence) over the paged cache, on the
// fifth-generation tensor cores.
//
// Mathematics: that of fl_attn.cu. Here the scores S = Q K^T and outputs O += P V are 128 x 128
// tensor-core tiles. The codes enter both products exactly, as bf16 values c / f (f = 128 at D8,
// 1024 at D4: fl_attn.cuh); f times the key's scale multiplies its score column, f times the
// value's scale its probability, so nothing is rounded but P (to bf16, as there and why) and the
// output.
// The running maximum is moved only when a row's grows by more than 8 (2^8 is no danger to fp32
// sums), which leaves O in tensor memory untouched in nearly every step; l and o carry the same
// power of two, so the result is the softmax all the same.
//
// Bound: per step of 128 keys and 256 query rows at D = 128 an SM needs 2048 cycles of MMA and
// 2048 of the exponential unit. Measured: about 6.9 k cycles (2048 tokens over 32k, 16 heads of
// 128: 770 us, 692 TFLOP/s). No unit is full: the exponentials, the unpacking and the products
// each left out take 5% off, the softmax passes left out 20%; what bounds it is the latency of a
// step's hand-offs (scores, softmax, products) with two tiles in flight, all tensor memory holds.
// The 96 registers of the launch spill (256 bytes stored, 500 loaded a thread over the whole kernel).
// A call of whole tiles takes 21.8 us and 3.60 a step (17.0 and 3.11 at D = 64); the join of a tile
// of 256 rows cut into 3, 6, 12 parts 15, 22, 37 us (14, 19, 31), of 100 rows 3, 4, 8.
//
// How: one persistent CTA per SM, 20 warps. Unit = (sequence, key/value head, tile of 256 query
// rows, step of 128 keys = two pages); rows are (token, head of the group) pairs. Each tile's
// units are the steps that some row of it sees. All units of the call, in order, are cut into
// equal contiguous ranges, one per CTA.
//  * Warp 17 streams the pages' planes into a ring (bulk copies): a step's keys with all scales, its
//    values.
//  * Warps 8-15 turn nibbles into bf16 and write them, 128-byte swizzled, as the K-major B
//    operands of both products (K as [key][dim], V as [dim][key]: the cache's fragment order gives
//    eight consecutive elements of either per 16-byte store).
//  * Warp 16 (one lane) issues the MMAs. The two halves of the 256 rows alternate, so that one
//    half's softmax runs under the other's products.
//  * Warps 0-3 and 4-7: softmax of rows 0-127 and 128-255. Pass one over S (tensor memory) finds
//    the rows' maxima, pass two writes P over S; then the epilogue.
//  * A tile cut by a range boundary leaves partials in the workspace, joined in CTA order by the
//    CTA that arrives last. Where it costs little balance, every tile is cut into the same number
//    of parts instead, one per CTA (one part: a whole tile).
#include <algorithm>

#include "fl_attn.cuh"

namespace fl {
namespace attn_tc {

using namespace attn;

__device__ int g_error;

constexpr int kThreads = 640;
constexpr int kTile = 128, kRows = 2 * kTile;  // rows of an MMA, of a unit
constexpr int kStep = 2 * kv::kBlock;          // keys of a unit
constexpr int kSoftWarps = 8, kConvWarp = 8, kConvWarps = 8, kMmaWarp = 16, kLoadWarp = 17;
constexpr int kScaleRing = 4;  // steps whose scales are held; the operand ring keeps fewer in flight
constexpr int kCutSteps = 8;   // what a range's second piece of a tile costs, in steps
constexpr float kSlack = 8.f;  // a row's maximum moves when it grows by more than this (log2)

template <int D>
struct Cfg {
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSlotBytes = kStep * D * 2;  // a K or V operand
  static constexpr int kSlots = D == 128 ? 3 : 4;
  static constexpr int kUnit = kv::kScaleBytes + 64 * D;  // a page's keys or values: both planes
  static constexpr int kRaw = D == 128 ? 6 : 8;
  static constexpr int kSmem = 1024 + kQ + kSlots * kSlotBytes + kRaw * kUnit;
  static constexpr int kPiece = kRows * (D + 2);  // floats of a partial: o by row, then (m, l) per row
};

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Tensor memory as mma fragments: 16 lanes by 8 columns per four registers, lane (g, t) holding
// columns 2 t and 2 t + 1 of rows g (registers 0, 1) and g + 8 (2, 3); 16 registers are 32 columns.
__device__ __forceinline__ void tmem_ld_frag32(uint32_t taddr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_frag32(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
               : "memory");
}
// Packed pairs of such columns: four 32-bit columns per two registers (rows g and g + 8).
__device__ __forceinline__ void tmem_st_pairs16(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Shared-memory matrix descriptor, K-major, 128-byte swizzle: rows of 128 bytes (64 bf16 of K) whose
// 16-byte chunk c lies at c ^ (row % 8), groups of eight rows 1024 bytes apart; descriptor version
// 1. A step of 16 in K moves the start address by 32 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t chunk) { return row * 128u + ((chunk ^ (row & 7u)) << 4); }

// Instruction descriptor of kind::f16: D fp32, A and B bf16, both K-major, M = 128.
__host__ __device__ constexpr uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// ---------------------------------------------------------------- pairs of fp32
// One instruction each; a value that enters every pair (twice) is made once, by a volatile move.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// ---------------------------------------------------------------- units

// Tile tau of a sequence: its rows, their positions, and the steps that they see as one list,
// steps [0, sink) and [first, ..).
struct Tile {
  int r0, nrows, pos_lo, pos_hi, sink, first, n;
};
__device__ __forceinline__ int tiles_of(const Args& a, const Geo& g) { return (g.s.n * a.group + kRows - 1) / kRows; }
__device__ __forceinline__ Tile tile_of(const Args& a, const Geo& g, int tau) {
  Tile t;
  t.r0 = tau * kRows;
  t.nrows = min(kRows, g.s.n * a.group - t.r0);
  t.pos_lo = g.pos0 + t.r0 / a.group;
  t.pos_hi = g.pos0 + (t.r0 + t.nrows - 1) / a.group;
  t.first = t.sink = 0;
  if (a.window > 0) {
    t.first = max(t.pos_lo - a.window + 1, 0) / kStep;
    t.sink = min((min(a.sinks, t.pos_hi + 1) + kStep - 1) / kStep, t.first);
  }
  t.n = t.pos_hi / kStep - t.first + 1 + t.sink;
  return t;
}
__device__ __forceinline__ int step_at(const Tile& t, int p) { return p < t.sink ? p : t.first + p - t.sink; }
// Whether some row of the tile sees a key of the block. A step's other block may have no page (behind
// the window, between the first tokens and it): its table entry is not looked at.
__device__ __forceinline__ bool needs(const Args& a, const Tile& t, int block) {
  const int key0 = block * kv::kBlock;
  return key0 <= t.pos_hi && (a.window == 0 || t.pos_lo - (key0 + kv::kBlock - 1) < a.window || key0 < a.sinks);
}

// A warp's place in the list of units; every lane holds the same.
struct Walk {
  int i, head, tau, tiles;
  int cuts;      // parts of the tile, where every tile is cut alike
  long long ia;  // first unit of the tile
  Geo g;
  Tile t;

  __device__ __forceinline__ void at_seq(const Args& a, int seq) {
    bool bad = false;
    i = seq;
    g = geo_of(a, i, &bad);
    tiles = tiles_of(a, g);
  }
  __device__ void seek(const Args& a, const long long* pre, long long u, bool by_tile) {
    const int lane = threadIdx.x & 31;
    at_seq(a, find_seq(pre, a.b.n_seqs, u));
    const long long per = (pre[i + 1] - pre[i]) / a.kv_heads;
    head = (int)((u - pre[i]) / per);
    ia = pre[i] + head * per;
    for (tau = 0;; tau += 32) {
      const int mine = tau + lane >= tiles ? 0 : by_tile ? 1 : tile_of(a, g, tau + lane).n;
      long long inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, u < ia + inc);
      if (past) {
        const int w = __ffs(past) - 1;
        ia += __shfl_sync(0xffffffffu, inc - mine, w);
        tau += w;
        break;
      }
      ia += __shfl_sync(0xffffffffu, inc, 31);
    }
    t = tile_of(a, g, tau);
  }
  __device__ __forceinline__ void next(const Args& a, const long long* pre) {
    ia += t.n;
    if (++tau == tiles) {
      tau = 0;
      if (++head == a.kv_heads) {
        head = 0;
        do ++i;
        while (pre[i + 1] == pre[i]);  // units remain, so one does
        at_seq(a, i);
      }
    }
    t = tile_of(a, g, tau);
  }
};

// ---------------------------------------------------------------- softmax of a step

// What a lane's four rows see of a half step's columns: keys up to their position, and of those
// the ones in the window or among the first; nothing where the page is not there.
struct Sight {
  int hi[4], lo[4], sink;  // relative to the half step's first key
  __device__ __forceinline__ bool operator()(int r, int x) const { return x <= hi[r] && (x >= lo[r] || x < sink); }
};
__device__ __forceinline__ Sight sight_of(const Args& a, bool there, const int (&pos)[4], int key0) {
  Sight s;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    s.hi[r] = there ? pos[r] - key0 : -1;
    s.lo[r] = a.window > 0 ? max(pos[r] - a.window + 1, 0) - key0 : -key0;
  }
  s.sink = a.sinks - key0;
  return s;
}

// Both passes over a step read S from tensor memory, 32 columns at a time, the next ones on their
// way while these are worked on. Lane (g, t) holds rows 8 r + g of the warp's 32, columns 8 j + 2 t
// and + 1: it needs a quarter of the columns' scales, and four rows share each. (S held in registers
// over both passes took 1.1 times as long: its unrolled code outgrew the instruction cache.)
struct Chunk {
  uint32_t v[2][16];
  __device__ __forceinline__ void load(uint32_t ts) {
    tmem_ld_frag32(ts, v[0]);
    tmem_ld_frag32(ts + (16u << 16), v[1]);
  }
  __device__ __forceinline__ uint64_t pair(int r, int j) const {
    const uint32_t* const p = &v[r >> 1][4 * j + 2 * (r & 1)];
    return pack2(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
};
__device__ __forceinline__ void load_scales(uint64_t (&k)[4], const float* ks) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const uint64_t*>(ks + 8 * j + 2 * t);
}

// Each row's maximum over the scaled scores of 32 columns.
template <bool kMasked>
__device__ __forceinline__ void chunk_max(const Chunk& c, const uint64_t (&k)[4], const Sight& see, int x0, float (&mx)[4]) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float2 z = unpack2(mul2(c.pair(r, j), k[j]));
      if (kMasked) {
        z.x = see(r, x0 + 8 * j + 2 * t) ? z.x : -INFINITY;
        z.y = see(r, x0 + 8 * j + 2 * t + 1) ? z.y : -INFINITY;
      }
      mx[r] = fmaxf(mx[r], fmaxf(z.x, z.y));
    }
}

// P of 32 columns: 2^(z - m) times the value's scale, bf16, stored at tp; adds the powers to l. A
// key that is not seen has weight 0 whatever its value's scale is.
template <bool kMasked>
__device__ __forceinline__ void chunk_probs(const Chunk& c, uint32_t tp, const uint64_t (&k)[4], const uint64_t (&v)[4],
                                            const Sight& see, int x0, const uint64_t (&mneg)[4], float (&l)[4]) {
  const int t = threadIdx.x & 3;
  uint32_t pr[2][8];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float2 z = unpack2(fma2(c.pair(r, j), k[j], mneg[r]));
      if (kMasked) {
        z.x = see(r, x0 + 8 * j + 2 * t) ? z.x : -INFINITY;
        z.y = see(r, x0 + 8 * j + 2 * t + 1) ? z.y : -INFINITY;
      }
      const float ex = exp2_approx(z.x), ey = exp2_approx(z.y);
      l[r] += ex + ey;
      float2 w = unpack2(mul2(pack2(ex, ey), v[j]));
      if (kMasked) {
        w.x = see(r, x0 + 8 * j + 2 * t) ? w.x : 0.f;
        w.y = see(r, x0 + 8 * j + 2 * t + 1) ? w.y : 0.f;
      }
      pr[r >> 1][2 * j + (r & 1)] = bf16x2(w.x, w.y);
    }
  tmem_st_pairs16(tp, pr[0]);
  tmem_st_pairs16(tp + (16u << 16), pr[1]);
}

template <bool kMasked>
__device__ __forceinline__ void step_max(const Args& a, uint32_t ts, const float* ks, const int* alive, const int (&pos)[4],
                                         int key0, float (&mx)[4]) {
  Chunk c[2];
  c[0].load(ts);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const Sight see = kMasked ? sight_of(a, alive[h], pos, key0 + kv::kBlock * h) : Sight();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint64_t k[4];
      load_scales(k, ks + 64 * h + 32 * e);
      wait_ld();
      if (e == 0 || h == 0) c[1 - e].load(ts + 64 * h + 32 * e + 32);
      chunk_max<kMasked>(c[e], k, see, 32 * e, mx);
    }
  }
}

// P over S: keys 64 h .. of P take the columns 32 h .., read before. Arrives at bar[h] when they are stored.
template <bool kMasked>
__device__ __forceinline__ void step_probs(const Args& a, uint32_t ts, const float* ks, const float* vs, const int* alive,
                                           const int (&pos)[4], int key0, const uint64_t (&mneg)[4], float (&l)[4],
                                           uint64_t* bar) {
  Chunk c[2];
  c[0].load(ts);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const Sight see = kMasked ? sight_of(a, alive[h], pos, key0 + kv::kBlock * h) : Sight();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint64_t k[4], v[4];
      load_scales(k, ks + 64 * h + 32 * e);
      load_scales(v, vs + 64 * h + 32 * e);
      wait_ld();
      if (e == 0 || h == 0) c[1 - e].load(ts + 64 * h + 32 * e + 32);
      chunk_probs<kMasked>(c[e], ts + 32 * h + 16 * e, k, v, see, 32 * e, mneg, l);
    }
    wait_st();
    fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar + h);
  }
}

// Word x of quad lane t and word t of quad lane x change places (all 32 lanes).
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t) {
  const bool odd = t & 1, upper = t & 2;
  const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
  const uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
  w[0] = odd ? x : w[0], w[1] = odd ? w[1] : x;
  w[2] = odd ? y : w[2], w[3] = odd ? w[3] : y;
  const uint32_t z0 = __shfl_xor_sync(0xffffffffu, upper ? w[0] : w[2], 2);
  const uint32_t z1 = __shfl_xor_sync(0xffffffffu, upper ? w[1] : w[3], 2);
  w[0] = upper ? z0 : w[0], w[2] = upper ? w[2] : z0;
  w[1] = upper ? z1 : w[1], w[3] = upper ? w[3] : z1;
}

// Joins the pieces of a tile that CTAs c0 .. c1 left, in that order (inside: the tile begins inside
// c0's range, so its piece is that CTA's second): a warp per row, eight rows at a
// time so that enough loads are in flight.
template <int D>
__device__ __forceinline__ void merge_rows(const Args& a, const Walk& w, int c0, int c1, bool inside) {
  using C = Cfg<D>;
  constexpr int kE = D / 32, kB = 8;  // elements of a lane, rows at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r0 = warp; r0 < w.t.nrows; r0 += kB * kSoftWarps) {
    float m[kB], l[kB], o[kB][kE];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      m[b] = -INFINITY;
      l[b] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[b][e] = 0.f;
    }
#pragma unroll 2
    for (int c = c0; c <= c1; ++c) {
      const float* pp = a.partial + (size_t)(2 * c + (c == c0 && inside)) * C::kPiece;
      float v[kB][kE];
      float2 ml[kB];
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int r = min(r0 + b * kSoftWarps, w.t.nrows - 1);
        ml[b] = __ldcg(reinterpret_cast<const float2*>(pp + kRows * D + 2 * r));
        if (kE == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(pp + r * D + 4 * lane));
          v[b][0] = x.x, v[b][1] = x.y, v[b][kE - 2] = x.z, v[b][kE - 1] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(pp + r * D + 2 * lane));
          v[b][0] = x.x, v[b][1] = x.y;
        }
      }
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const float mn = fmaxf(m[b], ml[b].x), mu = mn == -INFINITY ? 0.f : mn;
        const float f0 = exp2_approx(m[b] - mu), f1 = exp2_approx(ml[b].x - mu);
        m[b] = mn;
        l[b] = fmaf(f1, ml[b].y, f0 * l[b]);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[b][e] = fmaf(f1, v[b][e], f0 * o[b][e]);
      }
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int r = r0 + b * kSoftWarps, rr = w.t.r0 + r;
      if (r >= w.t.nrows) break;
      const float inv = l[b] == 0.f ? 0.f : 1.f / l[b];
      uint16_t* const op = a.out + (int64_t)(w.g.s.row0 + rr / a.group) * a.out_stride +
                           (w.head * a.group + rr % a.group) * D + kE * lane;
      const uint32_t lo = bf16x2(o[b][0] * inv, o[b][1] * inv);
      if (kE == 4)
        *reinterpret_cast<uint2*>(op) = make_uint2(lo, bf16x2(o[b][kE - 2] * inv, o[b][kE - 1] * inv));
      else
        *reinterpret_cast<uint32_t*>(op) = lo;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D>;
  constexpr int NR = C::kRaw, NS = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t raw_full[NR], raw_empty[NR], op_full[NS], op_empty[NS];
  __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], sc_full[kScaleRing];
  __shared__ int meta[NR];                              // level of a raw unit's page
  __shared__ __align__(16) float ksc[kScaleRing][kStep], vsc[kScaleRing][kStep];
  __shared__ int alive[kScaleRing][2];
  __shared__ long long pre[FL_KV_MAX_SEQS + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last, s_tiles, s_longest, s_parts;
  __shared__ Walk walks[kLoadWarp + 1];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* const q_smem = smem;
  uint8_t* const op_smem = smem + C::kQ;
  uint8_t* const raw_smem = op_smem + NS * C::kSlotBytes;

  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s_tiles = s_longest = 0;
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kConvWarps);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&op_full[s], kConvWarps);
      mbar_init(&op_empty[s], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&sc_full[s], kConvWarps);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 4);
      mbar_init(&s_full[t], 1);
      mbar_init(&o_full[t], 1);
      mbar_init(&p_full[t][0], 4);
      mbar_init(&p_full[t][1], 4);
    }
    fence_mbar_init();
  }
  pdl_wait();
  __syncthreads();

  // ---- units before each sequence: a warp per sequence, a lane per tile. Equal ranges of all units
  // balance best but cut most tiles twice, and a range's two pieces each fill and drain the pipeline
  // and pass through the workspace. So where tiles cut into equally many parts give no part much
  // longer than a range (kCutSteps), CTAs take parts: a 1021-token prompt's 128 tiles of 1 to 8
  // steps whole (60 -> 41 us), 64 tiles of 17 to 31 steps in two (145 -> 129 us).
  const int n_seqs = a.b.n_seqs;
  auto scan = [&](bool tiles_only) {
    bool bad = false;
    int longest = 0;
    for (int i = warp; i < n_seqs; i += kThreads / 32) {
      const Geo g = geo_of(a, i, &bad);
      const int tiles = tiles_of(a, g);
      long long sum = tiles;
      if (!tiles_only) {
        sum = 0;
        for (int tau = lane; tau < tiles; tau += 32) {
          const int n = tile_of(a, g, tau).n;
          sum += n;
          longest = max(longest, n);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) atomicAdd(&s_tiles, min(tiles, 1024) * a.kv_heads);
      }
      if (lane == 0) pre[i] = sum * a.kv_heads;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) atomicMax(&s_longest, longest);
    if (bad && blockIdx.x == 0) atomicOr(&g_error, (int)kv::kErrSeq);
    __syncthreads();
    if (warp == 0) {
      const int per = (n_seqs + 31) / 32, i0 = min(lane * per, n_seqs), i1 = min(i0 + per, n_seqs);
      long long sum = 0;
      for (int i = i0; i < i1; ++i) sum += pre[i];
      long long inc = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      long long before = inc - sum;
      for (int i = i0; i < i1; ++i) {
        const long long x = pre[i];
        pre[i] = before;
        before += x;
      }
      if (lane == 31) pre[n_seqs] = inc;
    }
    __syncthreads();
  };
  scan(false);
  const long long U = pre[n_seqs];
  const int share = (int)min(U / gridDim.x, (long long)1 << 30);
  // Parts of a tile: as many as there are CTAs for, but a part saves n / parts steps and adds a piece
  // to the join, done by one CTA, so no more than about sqrt(n) (100 tokens over 4k, 8 tiles of 33
  // steps: six parts 69 us, eighteen 86).
  const int parts = s_tiles > 0 ? min((int)(gridDim.x / (unsigned)s_tiles), 1 + (int)sqrtf((float)s_longest)) : 0;
  const bool by_tile = parts > 0 && (s_longest + parts - 1) / parts <= share + kCutSteps;
  const int G = by_tile ? s_tiles * parts : (int)min((long long)gridDim.x, U);
  if ((int)blockIdx.x >= G) return;
  if (by_tile) {
    __syncthreads();
    scan(true);
  }
  if (threadIdx.x == 0) s_parts = by_tile ? parts : 0;  // (read at a join, after the next barrier)
  long long u0 = by_tile ? blockIdx.x / parts : U * blockIdx.x / G, u1 = U * (blockIdx.x + 1) / G;

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;  // columns: S of either half at 0 and 128, O at 256 and 256 + D

  // each warp's place lies in shared memory: it is read at a tile's ends only
  Walk& w = walks[min(warp, kLoadWarp)];
  if (warp <= kLoadWarp) {
    Walk x;
    x.seek(a, pre, u0, by_tile);
    if (by_tile) {  // units are the tile's steps
      const int cuts = min(parts, x.t.n), part = blockIdx.x % parts;  // a short tile has fewer
      x.cuts = cuts;
      x.ia = 0;
      u0 = part < cuts ? (long long)x.t.n * part / cuts : 0;
      u1 = part < cuts ? (long long)x.t.n * (part + 1) / cuts : 0;
    }
    if (lane == 0) w = x;
    __syncwarp();
  }
  auto advance = [&] {
    Walk x = w;
    x.next(a, pre);
    __syncwarp();
    if (lane == 0) w = x;
    __syncwarp();
  };

  // The launch's registers (640 x 96) by role: 8 warps x 128, 8 x 72, 4 x 80.
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- pages -> raw ring
    int unit = 0;
    bool failed = false;
    auto emit = [&](const uint8_t* src, int lv, bool values) {
      const int s = unit % NR;
      if (failed) return;
      if (unit >= NR && !__all_sync(0xffffffffu, mbar_wait(&raw_empty[s], (uint32_t)((unit / NR - 1) & 1)))) {
        failed = true;
        return;
      }
      if (lane == 0) {
        constexpr uint32_t plane = (uint32_t)kv::plane_bytes(D);
        uint8_t* dst = raw_smem + s * C::kUnit;
        const uint32_t head_bytes = values ? 0u : (uint32_t)kv::kScaleBytes;
        meta[s] = lv;
        mbar_expect_tx(&raw_full[s], lv == 0 ? 0u : head_bytes + (lv == 4 ? 2u : 1u) * plane);
        if (lv > 0) {
          const uint8_t* hi = src + kv::kScaleBytes + (values ? plane : 0u);
          bulk_g2s(dst + kv::kScaleBytes - head_bytes, hi - head_bytes, head_bytes + plane, &raw_full[s]);
          if (lv == 4) bulk_g2s(dst + kv::kScaleBytes + plane, hi + 2 * plane, plane, &raw_full[s]);
        }
      }
      __syncwarp();
      ++unit;
    };
    for (long long u = u0; u < u1 && !failed;) {
      const long long ue = min(u1, w.ia + w.t.n);
      const int p0 = (int)(u - w.ia), p1 = (int)(ue - w.ia);
      const uint8_t* src = nullptr;
      int lv = 0;
      for (int p = p0; p < p1 && !failed; ++p) {
        const int k = (p - p0) & 15;
        if (k == 0) {  // sixteen steps' table entries at once, two lanes per step
          lv = 0;
          const int pp = p + (lane >> 1);
          if (pp < p1) {
            const int block = 2 * step_at(w.t, pp) + (lane & 1);
            if (needs(a, w.t, block)) {
              const size_t at = (size_t)w.i * a.b.max_blocks + block;
              const int page = __ldg(a.b.table + at);
              lv = kv::level_of(a.levels, at);
              if (page < 0 || page >= a.num_pages) {  // a ZERO block's entry may be anything
                if (lv > 0) atomicOr(&g_error, (int)kv::kErrPage);
                lv = 0;
              } else {
                src = a.pages + ((size_t)page * a.kv_heads + w.head) * kv::record_bytes(D);
              }
            }
          }
        }
        const uint8_t* cur_src[2];
        int cur_lv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          cur_src[e] = reinterpret_cast<const uint8_t*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), 2 * k + e));
          cur_lv[e] = __shfl_sync(0xffffffffu, lv, 2 * k + e);
        }
#pragma unroll 1
        for (int e = 0; e < 4; ++e)  // the step's keys, then its values
          emit(e & 1 ? cur_src[1] : cur_src[0], e & 1 ? cur_lv[1] : cur_lv[0], e >= 2);
      }
      u = ue;
      if (u < u1) advance();
    }
    if (failed && lane == 0) atomicOr(&g_error, (int)kv::kErrWait);
    // no copy may still be landing when the CTA exits
    for (int k = max(0, unit - NR); k < unit; ++k)
      if (!mbar_wait(&raw_full[k % NR], (uint32_t)((k / NR) & 1)) && lane == 0) atomicOr(&g_error, (int)kv::kErrWait);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issue: one thread
    if (elect_one()) {
      const uint64_t q_desc = sw128_desc(smem_u32(q_smem)), op_desc = sw128_desc(smem_u32(op_smem));
      bool ok = true;
      int base = 0;               // operands before the piece
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
      auto op_wait = [&](int o) { ok = ok && mbar_wait(&op_full[o % NS], (uint32_t)((o / NS) & 1)); };
      auto scores = [&](int t, int o) {
        const uint64_t qd = q_desc + (uint64_t)(t * (kTile * D * 2 / 16)), kd = op_desc + (uint64_t)((o % NS) * (C::kSlotBytes / 16));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t off = (uint64_t)((ks / 4) * (kTile * 128 / 16) + 2 * (ks % 4));
          mma_ss(tmem + 128u * t, qd + off, kd + off, idesc_bf16(kStep), ks > 0);
        }
        mma_commit(&s_full[t]);
      };
      for (long long u = u0; u < u1 && ok;) {
        const long long ue = min(u1, w.ia + w.t.n);
        const int n = (int)(ue - u), nt = w.t.nrows > kTile ? 2 : 1;
        op_wait(base);
        for (int t = 0; t < nt && ok; ++t) {
          ok = mbar_wait(&q_full[t], nq[t]++ & 1u);
          fence_after();
          if (ok) scores(t, base);
        }
        if (ok) mma_commit(&op_empty[base % NS]);
        for (int j = 0; j < n && ok; ++j) {
          const int vo = base + 2 * j + 1, ko = vo + 1;
          op_wait(vo);
          for (int t = 0; t < nt && ok; ++t) {
            const uint64_t vd = op_desc + (uint64_t)((vo % NS) * (C::kSlotBytes / 16));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = ok && mbar_wait(&p_full[t][h], np[t] & 1u);
              if (!ok) break;
              fence_after();
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_ts(tmem + 256u + (uint32_t)(D * t), tmem + 128u * t + 32u * h + 8u * ks,
                       vd + (uint64_t)(h * (D * 128 / 16) + 2 * ks), idesc_bf16(D), j > 0 || h > 0 || ks > 0);
            }
            ++np[t];
            if (!ok) break;
            if (t == nt - 1) mma_commit(&op_empty[vo % NS]);
            if (j == n - 1) mma_commit(&o_full[t]);
            if (j + 1 < n) {
              if (t == 0) {
                op_wait(ko);
                if (!ok) break;
                fence_after();
              }
              scores(t, ko);
              if (t == nt - 1) mma_commit(&op_empty[ko % NS]);
            }
          }
        }
        base += 2 * n;
        u = ue;
        if (u < u1) w.next(a, pre);
      }
      // every MMA is complete before TMEM is freed: the last commit tracks all of them
      if (ok && base > 0) ok = mbar_wait(&op_empty[(base - 1) % NS], (uint32_t)(((base - 1) / NS) & 1));
      if (!ok) atomicOr(&g_error, (int)kv::kErrWait);
    }
    __syncwarp();
  }
  } else if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------------------------------------------------------- raw ring -> operands
    // in the order K0, V0, K1, V1, .. : with three slots a step's keys then wait for the slot of the
    // values two before, free before the scores of the step between are (keys first, K0, K1, V0, ..,
    // took 761 us instead of 751 for 2048 tokens over 32k)
    {
      const int cw = warp - kConvWarp, g = lane >> 2, t = lane & 3;
      int unit = 0, op = 0, step = 0;
      bool failed = false;
      for (long long u = u0; u < u1 && !failed;) {
        const long long ue = min(u1, w.ia + w.t.n);
        const int n = (int)(ue - u);
#pragma unroll 1
        for (int o = 0; o < 2 * n && !failed; ++o, ++op) {
          const bool values = o & 1;
          const int os = op % NS, sr = step % kScaleRing;
          failed = op >= NS && !__all_sync(0xffffffffu, mbar_wait(&op_empty[os], (uint32_t)((op / NS - 1) & 1)));
          uint8_t* const dst = op_smem + os * C::kSlotBytes;
#pragma unroll 1
          for (int pg = 0; pg < 2 && !failed; ++pg, ++unit) {
            const int s = unit % NR;
            if (!__all_sync(0xffffffffu, mbar_wait(&raw_full[s], (uint32_t)((unit / NR) & 1)))) {
              failed = true;
              break;
            }
            const int lv = meta[s];
            const uint8_t* const raw = raw_smem + s * C::kUnit;
            if (!values && lane < 16) {  // 16 of the page's 64 keys' and 64 values' scales per warp
              const int x = 16 * (cw & 3) + lane;
              const float f = lv == 4 ? value_factor<true>() : value_factor<false>();
              const float sc = lv > 0 ? lds32(raw + 64 * cw + 4 * lane) * (cw < 4 ? f * a.scale_log2 : f) : 0.f;
              (cw < 4 ? ksc : vsc)[sr][kv::kBlock * pg + x] = sc;
              if (cw == 0 && lane == 0) alive[sr][pg] = lv > 0;
            }
            // 512 bytes of a plane per warp: at D = 64, with four such blocks, four warps per page
            if (D == 128 || (cw >> 2) == pg) {
              const int b = D == 128 ? cw : cw & 3;
              uint32_t r[4][4];
              uint4 h = make_uint4(0, 0, 0, 0);  // a block that nobody sees: P is 0 there, but the operand must be finite
              if (lv > 0) h = lds128(raw + kv::kScaleBytes + 512 * b + 16 * lane);
              if (lv == 4) {
                const uint4 l = lds128(raw + kv::kScaleBytes + kv::plane_bytes(D) + 512 * b + 16 * lane);
                unpack_word<true>(h.x, l.x, r[0]);
                unpack_word<true>(h.y, l.y, r[1]);
                unpack_word<true>(h.z, l.z, r[2]);
                unpack_word<true>(h.w, l.w, r[3]);
              } else {
                unpack_word<false>(h.x, 0u, r[0]);
                unpack_word<false>(h.y, 0u, r[1]);
                unpack_word<false>(h.z, 0u, r[2]);
                unpack_word<false>(h.w, 0u, r[3]);
              }
              if (!values) {  // words x, y: dims 16 t .. + 15 of a slot, z, w: of the slot two on
                const int s4 = b / (D / 64), S = b % (D / 64);
                const uint32_t row = (uint32_t)(kv::kBlock * pg + 16 * (g >> 1) + 4 * s4 + (g & 1));
                uint8_t* const d = dst + S * (kStep * 128);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  *reinterpret_cast<uint4*>(d + sw128(row + 2 * (x >> 1), 2 * t + (x & 1))) =
                      make_uint4(r[x][0], r[x][1], r[x][2], r[x][3]);
              } else {  // dims 16 b + g (pairs 0, 2) and + 8 (pairs 1, 3), slots 16 t + 4 x ..
                uint8_t* const d = dst + pg * (D * 128);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                  for (int x = 0; x < 2; ++x)
                    *reinterpret_cast<uint4*>(d + sw128((uint32_t)(16 * b + g + 8 * e), 2 * t + x)) =
                        make_uint4(r[2 * x][e], r[2 * x][e + 2], r[2 * x + 1][e], r[2 * x + 1][e + 2]);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[s]);
          }
          if (failed) break;
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&op_full[os]);
            if (!values) mbar_arrive(&sc_full[sr]);
          }
          if (!values) ++step;
        }
        u = ue;
        if (u < u1) advance();
      }
      if (failed && lane == 0) atomicOr(&g_error, (int)kv::kErrWait);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // ---------------------------------------------------------------- softmax, epilogue
    const int t = warp >> 2, row = 32 * (warp & 3) + lane, fg = lane >> 2, ft = lane & 3;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, half = 16u << 16;
    const uint32_t ts = tmem + lanes + 128u * t, to = tmem + lanes + 256u + (uint32_t)(D * t);
    uint8_t* const qs = q_smem + t * (kTile * D * 2);
    int step = 0, cnt = 0, pieces = 0;  // steps of the CTA, of this half, pieces of this half
    bool ok = true;
    for (long long u = u0; u < u1;) {
      const long long ue = min(u1, w.ia + w.t.n);
      const int p0 = (int)(u - w.ia), n = (int)(ue - u);
      const bool live = w.t.nrows > kTile * t;  // this half has rows
      const bool whole = p0 == 0 && n == w.t.n;
      if (live && ok) {
        {
          const int rr = w.t.r0 + min(kTile * t + row, w.t.nrows - 1);
          const uint4* qp = reinterpret_cast<const uint4*>(a.q + (int64_t)(w.g.s.row0 + rr / a.group) * a.q_stride +
                                                           (w.head * a.group + rr % a.group) * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4*>(qs + (c >> 3) * (kTile * 128) + sw128(row, c & 7)) = __ldg(qp + c);
        }
        fence_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
        const int wr = kTile * t + 32 * (warp & 3) + fg;  // rows of this lane in the tile: wr + 8 r
        int pos[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) pos[r] = w.g.pos0 + (w.t.r0 + min(wr + 8 * r, w.t.nrows - 1)) / a.group;
        const int plo = w.g.pos0 + (w.t.r0 + kTile * t) / a.group;
        const int phi = w.g.pos0 + (w.t.r0 + min(kTile * t + kTile, w.t.nrows) - 1) / a.group;
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float l[4] = {0.f, 0.f, 0.f, 0.f};
        // A half that skipped tiles without rows may be laps ahead of sc_full, whose parity alone would
        // then fall through on an older lap. The first step's scores mean that every unpacking warp
        // has passed its keys, so from there on the barriers are in the laps that are waited for; and
        // they stay: the keys kScaleRing steps on need an operand slot that frees after this half's P.
        // The wait may span all the skipped steps, so its limit grows with them (20 us each, against 4).
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], (uint32_t)(cnt & 1), kWaitLimitNs + 20000ull * (uint32_t)(step - cnt)));
        for (int j = 0; j < n && ok; ++j, ++cnt) {
          const int sr = (step + j) % kScaleRing, key0 = kStep * step_at(w.t, p0 + j);
          ok = __all_sync(0xffffffffu, mbar_wait(&sc_full[sr], (uint32_t)(((step + j) / kScaleRing) & 1)) &&
                                           mbar_wait(&s_full[t], (uint32_t)(cnt & 1)));
          if (!ok) break;
          fence_after();
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          bool masked = key0 + kStep - 1 > plo ||
                        (a.window > 0 && key0 <= phi - a.window && key0 + kStep - 1 >= a.sinks) || !alive[sr][0] || !alive[sr][1];
          if (masked)
            step_max<true>(a, ts, ksc[sr], alive[sr], pos, key0, mx);
          else
            step_max<false>(a, ts, ksc[sr], alive[sr], pos, key0, mx);
          bool grow = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            grow = grow || mx[r] > m[r] + kSlack;
          }
          if (__any_sync(0xffffffffu, grow)) {
            float f[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const bool up = mx[r] > m[r] + kSlack;
              f[r] = up ? exp2_approx(m[r] - mx[r]) : 1.f;
              m[r] = up ? mx[r] : m[r];
              l[r] *= f[r];
            }
            if (j > 0) {  // S of this step follows P V of the step before: O is at rest
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  uint32_t v[16];
                  tmem_ld_frag32(to + e * half + 32 * c, v);
                  wait_ld();
#pragma unroll
                  for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * f[2 * e + ((x >> 1) & 1)]);
                  tmem_st_frag32(to + e * half + 32 * c, v);
                }
              }
              wait_st();
            }
          }
          uint64_t mneg[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) mneg[r] = twice(m[r] == -INFINITY ? 0.f : -m[r]);
          if (masked)
            step_probs<true>(a, ts, ksc[sr], vsc[sr], alive[sr], pos, key0, mneg, l, p_full[t]);
          else
            step_probs<false>(a, ts, ksc[sr], vsc[sr], alive[sr], pos, key0, mneg, l, p_full[t]);
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&o_full[t], (uint32_t)(pieces & 1)));
        ++pieces;
        // ---- epilogue: the outputs, or a partial
        if (ok) {
          fence_after();
          float inv[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float x = l[r];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            inv[r] = whole ? (x == 0.f ? 0.f : 1.f / x) : x;  // a partial keeps the sum
          }
          float* const part = a.partial + (size_t)(2 * blockIdx.x + (u != u0)) * C::kPiece;
          uint16_t* op[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int rr = w.t.r0 + wr + 8 * r;
            op[r] = a.out + (int64_t)(w.g.s.row0 + rr / a.group) * a.out_stride + (w.head * a.group + rr % a.group) * D +
                    8 * ft;
          }
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[2][16];
            tmem_ld_frag32(to + 32 * c, v[0]);
            tmem_ld_frag32(to + half + 32 * c, v[1]);
            wait_ld();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // the four lanes of a row trade columns, so that each stores eight in a row
              uint32_t e0[4], e1[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                e0[x] = v[r >> 1][4 * x + 2 * (r & 1)];
                e1[x] = v[r >> 1][4 * x + 2 * (r & 1) + 1];
                if (whole) e0[x] = bf16x2(__uint_as_float(e0[x]) * inv[r], __uint_as_float(e1[x]) * inv[r]);
              }
              quad_transpose(e0, ft);
              if (!whole) quad_transpose(e1, ft);
              if (wr + 8 * r >= w.t.nrows) continue;
              if (whole) {
                *reinterpret_cast<uint4*>(op[r] + 32 * c) = make_uint4(e0[0], e0[1], e0[2], e0[3]);
              } else {
                uint4* const pp = reinterpret_cast<uint4*>(part + (wr + 8 * r) * D + 32 * c + 8 * ft);
                pp[0] = make_uint4(e0[0], e1[0], e0[1], e1[1]);
                pp[1] = make_uint4(e0[2], e1[2], e0[3], e1[3]);
              }
            }
          }
          if (!whole && ft == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (wr + 8 * r < w.t.nrows)
                *reinterpret_cast<float2*>(part + kRows * D + 2 * (wr + 8 * r)) = make_float2(m[r], inv[r]);
          }
          fence_before();
        }
      }
      if (!whole) {
        asm volatile("bar.sync 1, 256;" ::: "memory");
        int c0, c1;
        bool inside = false;
        if (s_parts > 0) {
          c0 = blockIdx.x - blockIdx.x % s_parts;
          c1 = c0 + w.cuts - 1;
        } else {  // CTA of unit v: the largest c with U c / G <= v
          const long long U = pre[n_seqs], G = min((long long)gridDim.x, U);
          c0 = (int)(((w.ia + 1) * G - 1) / U);
          c1 = (int)(((w.ia + w.t.n) * G - 1) / U);
          inside = U * c0 / G < w.ia;
        }
        if (threadIdx.x == 0) s_last = atom_add_acq_rel(a.tickets + c0, 1u) == (uint32_t)(c1 - c0);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (s_last) merge_rows<D>(a, w, c0, c1, inside);
        if (s_last) {
          if (threadIdx.x == 0) a.tickets[c0] = 0u;
        }
      }
      step += n;
      u = ue;
      if (u < u1) advance();
    }
    if (!ok && lane == 0) atomicOr(&g_error, (int)kv::kErrWait);
  }

  fence_before();
  __syncthreads();  // every role is done: no copy in flight, every MMA complete, TMEM reads done
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ---------------------------------------------------------------- host side

template <int D>
static fl_status launch_d(const Args& a, int nsm, cudaStream_t st) {
  auto kern = attn_tc_kernel<D>;
  FL_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem),
                "cudaFuncSetAttribute(attn_tc)");
  FL_CHECK_CUDA(launch_pdl(kern, dim3((unsigned)nsm), dim3(kThreads), (size_t)Cfg<D>::kSmem, st, 1, a), "launch attn_tc");
  return FL_OK;
}

size_t partial_bytes(int D, int nsm) { return (size_t)nsm * 2 * (D == 64 ? Cfg<64>::kPiece : Cfg<128>::kPiece) * 4; }

fl_status launch(const Args& a, int D, int nsm, cudaStream_t st) {
  return D == 64 ? launch_d<64>(a, nsm, st) : launch_d<128>(a, nsm, st);
}

// Reads and clears the error word (-1 if that fails).
int take_device_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_error, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0 && cudaMemcpyToSymbol(g_error, &z, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

}  // namespace attn_tc
}  // namespace fl
