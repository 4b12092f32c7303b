// Attention of prompt chunks (many new tokens per sequence) over the paged cache, on the
// fifth-generation tensor cores.
//
// Mathematics: that of fl_attn.cu. Here the scores S = Q K^T and outputs O += P V are 128 x 128
// tensor-core tiles. The codes enter both products exactly, as bf16 values c / f (f = 128 at D8,
// 1024 at D4: fl_attn.cuh); f times the key's scale multiplies its score column, f times the
// value's scale its probability, so nothing is rounded but P (to bf16) and the output.
// The running maximum is moved only when a row's grows by more than 8 (2^8 is no danger to fp32
// sums), which leaves O in tensor memory untouched in nearly every step; l and o carry the same
// power of two, so the result is the softmax all the same.
//
// Bound: per step of 128 keys and 256 query rows at D = 128 an SM needs 2048 cycles of MMA and
// 2048 of the exponential unit; turning the codes into bf16 costs about a quarter of the issue
// slots of that time, which is why it is done once for 256 rows.
//
// How: one persistent CTA per SM, 16 warps. Unit = (sequence, key/value head, tile of 256 query
// rows, step of 128 keys = two pages); rows are (token, head of the group) pairs. Each tile's
// units are the steps that some row of it sees. All units of the call, in order, are cut into
// equal contiguous ranges, one per CTA.
//  * Warp 13 streams the pages' planes into a ring (bulk copies), keys of a step with its scales,
//    then the values of the step before.
//  * Warps 8-11 turn nibbles into bf16 and write them, 128-byte swizzled, as the K-major B
//    operands of both products (K as [key][dim], V as [dim][key]: the cache's fragment order gives
//    eight consecutive elements of either per 16-byte store).
//  * Warp 12 (one lane) issues the MMAs. The two halves of the 256 rows alternate, so that one
//    half's softmax runs under the other's products.
//  * Warps 0-3 and 4-7: softmax of rows 0-127 and 128-255, one row per thread. Pass one over S
//    (tensor memory) finds the row's maximum, pass two writes P over S; then the epilogue.
//  * A tile cut by a range boundary leaves partials in the workspace, joined in CTA order by the
//    CTA that arrives last.
#include <algorithm>

#include "fl_attn.cuh"

namespace fl {
namespace attn_tc {

using namespace attn;

__device__ int g_error;

constexpr int kThreads = 512;
constexpr int kTile = 128, kRows = 2 * kTile;  // rows of an MMA, of a unit
constexpr int kStep = 2 * kv::kBlock;          // keys of a unit
constexpr int kSoftWarps = 8, kConvWarp = 8, kConvWarps = 4, kMmaWarp = 12, kLoadWarp = 13;
constexpr int kScaleRing = 4;  // steps whose scales are held; the operand ring keeps fewer in flight
constexpr float kSlack = 8.f;  // a row's maximum moves when it grows by more than this (log2)

template <int D>
struct Cfg {
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSlotBytes = kStep * D * 2;  // a K or V operand
  static constexpr int kSlots = D == 128 ? 3 : 4;
  static constexpr int kUnit = kv::kScaleBytes + 64 * D;  // a page's keys or values: both planes
  static constexpr int kRaw = D == 128 ? 6 : 8;
  static constexpr int kSmem = 1024 + kQ + kSlots * kSlotBytes + kRaw * kUnit;
  static constexpr int kPiece = kRows * (D + 2);  // floats of a partial: o as [D/4][row][4], then (m, l) per row
};

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
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
struct f2 {
  uint64_t v;
};
__device__ __forceinline__ f2 pack2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(f2 p, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p.v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
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

// A warp's place in the list of units; every lane holds the same.
struct Walk {
  int i, head, tau, tiles;
  long long ia;  // first unit of the tile
  Geo g;
  Tile t;

  __device__ __forceinline__ void at_seq(const Args& a, int seq) {
    bool bad = false;
    i = seq;
    g = geo_of(a, i, &bad);
    tiles = tiles_of(a, g);
  }
  __device__ void seek(const Args& a, const long long* pre, long long u) {
    const int lane = threadIdx.x & 31;
    at_seq(a, find_seq(pre, a.b.n_seqs, u));
    const long long per = (pre[i + 1] - pre[i]) / a.kv_heads;
    head = (int)((u - pre[i]) / per);
    ia = pre[i] + head * per;
    for (tau = 0;; tau += 32) {
      const int mine = tau + lane < tiles ? tile_of(a, g, tau + lane).n : 0;
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
  __shared__ int s_last;
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* const q_smem = smem;
  uint8_t* const op_smem = smem + C::kQ;
  uint8_t* const raw_smem = op_smem + NS * C::kSlotBytes;

  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
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

  // ---- units before each sequence: a warp per sequence, a lane per tile
  const int n_seqs = a.b.n_seqs;
  {
    bool bad = false;
    for (int i = warp; i < n_seqs; i += kThreads / 32) {
      const Geo g = geo_of(a, i, &bad);
      const int tiles = tiles_of(a, g);
      long long sum = 0;
      for (int tau = lane; tau < tiles; tau += 32) sum += tile_of(a, g, tau).n;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) pre[i] = sum * a.kv_heads;
    }
    if (bad && blockIdx.x == 0) atomicMax(&g_error, (int)kv::kErrSeq);
  }
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
  const long long U = pre[n_seqs];
  const int G = (int)min((long long)gridDim.x, U);
  if ((int)blockIdx.x >= G) return;
  const long long u0 = U * blockIdx.x / G, u1 = U * (blockIdx.x + 1) / G;

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;  // columns: S of either half at 0 and 128, O at 256 and 256 + D

  Walk w;
  if (warp <= kLoadWarp) w.seek(a, pre, u0);

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
      const int blocks = w.g.s.len / kv::kBlock + (w.g.s.len % kv::kBlock != 0);
      const uint8_t *src = nullptr, *prev_src[2] = {nullptr, nullptr};
      int lv = 0, prev_lv[2] = {0, 0};
      for (int p = p0; p < p1 && !failed; ++p) {
        const int k = (p - p0) & 15;
        if (k == 0) {  // sixteen steps' table entries at once, two lanes per step
          lv = 0;
          const int pp = p + (lane >> 1);
          if (pp < p1) {
            const int block = 2 * step_at(w.t, pp) + (lane & 1);
            if (block < blocks) {
              const size_t at = (size_t)w.i * a.b.max_blocks + block;
              const int page = __ldg(a.b.table + at);
              lv = kv::level_of(a.levels, at);
              if (page < 0 || page >= a.num_pages) {
                atomicMax(&g_error, (int)kv::kErrPage);
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
        emit(cur_src[0], cur_lv[0], false);
        emit(cur_src[1], cur_lv[1], false);
        if (p > p0) {
          emit(prev_src[0], prev_lv[0], true);
          emit(prev_src[1], prev_lv[1], true);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          prev_src[e] = cur_src[e];
          prev_lv[e] = cur_lv[e];
        }
      }
      emit(prev_src[0], prev_lv[0], true);
      emit(prev_src[1], prev_lv[1], true);
      u = ue;
      if (u < u1) w.next(a, pre);
    }
    if (failed && lane == 0) atomicMax(&g_error, (int)kv::kErrWait);
    // no copy may still be landing when the CTA exits
    for (int k = max(0, unit - NR); k < unit; ++k)
      if (!mbar_wait(&raw_full[k % NR], (uint32_t)((k / NR) & 1)) && lane == 0) atomicMax(&g_error, (int)kv::kErrWait);
  } else if (warp >= kConvWarp && warp < kConvWarp + kConvWarps) {
    // ---------------------------------------------------------------- raw ring -> operands
    const int cw = warp - kConvWarp, g = lane >> 2, t = lane & 3;
    int unit = 0, op = 0, step = 0;
    bool failed = false;
    auto convert = [&](bool values) {
      const int os = op % NS;
      if (failed) return;
      if (op >= NS && !__all_sync(0xffffffffu, mbar_wait(&op_empty[os], (uint32_t)((op / NS - 1) & 1)))) {
        failed = true;
        return;
      }
      uint8_t* const dst = op_smem + os * C::kSlotBytes;
#pragma unroll 1
      for (int pg = 0; pg < 2; ++pg, ++unit) {
        const int s = unit % NR;
        if (!__all_sync(0xffffffffu, mbar_wait(&raw_full[s], (uint32_t)((unit / NR) & 1)))) {
          failed = true;
          return;
        }
        const int lv = meta[s];
        const uint8_t* const raw = raw_smem + s * C::kUnit;
        if (!values) {  // 16 keys' scales per warp: lanes 0-15 keys, 16-31 values
          const int x = 16 * cw + (lane & 15);
          const float f = lv == 4 ? value_factor<true>() : value_factor<false>();
          const float sc = lv > 0 ? lds32(raw + 256 * (lane >> 4) + 4 * x) * (lane < 16 ? f * a.scale_log2 : f) : 0.f;
          (lane < 16 ? ksc : vsc)[step % kScaleRing][kv::kBlock * pg + x] = sc;
          if (cw == 0 && lane == 0) alive[step % kScaleRing][pg] = lv > 0;
        }
#pragma unroll
        for (int bb = 0; bb < D / 64; ++bb) {
          const int b = D / 64 * cw + bb;  // 512 bytes of a plane
          uint32_t r[4][4];
          if (lv == 0) {  // a block that nobody sees: P is 0 there, the operand must be finite
#pragma unroll
            for (int x = 0; x < 16; ++x) r[x >> 2][x & 3] = 0u;
          } else {
            const uint4 h = lds128(raw + kv::kScaleBytes + 512 * b + 16 * lane);
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
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&op_full[os]);
        if (!values) mbar_arrive(&sc_full[step % kScaleRing]);
      }
      if (!values) ++step;
      ++op;
    };
    for (long long u = u0; u < u1 && !failed;) {
      const long long ue = min(u1, w.ia + w.t.n);
      const int n = (int)(ue - u);
      for (int j = 0; j < n; ++j) {
        convert(false);
        if (j > 0) convert(true);
      }
      convert(true);
      u = ue;
      if (u < u1) w.next(a, pre);
    }
    if (failed && lane == 0) atomicMax(&g_error, (int)kv::kErrWait);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issue
    {
      const uint32_t q_addr = smem_u32(q_smem), op_addr = smem_u32(op_smem);
      bool ok = true;
      int base = 0;                     // operands before the piece
      int nq[2] = {0, 0}, np[2] = {0, 0};
      auto wait = [&](uint64_t* bar, int phase) { ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(phase & 1))); };
      auto op_wait = [&](int o) { wait(&op_full[o % NS], o / NS); };
      auto scores = [&](int t, int o) {
        if (lane == 0) {
          const uint32_t k_addr = op_addr + (uint32_t)(o % NS) * C::kSlotBytes;
          fence_after();
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (uint32_t)(ks / 4) * (kTile * 128) + 32u * (ks % 4);
            mma_ss(tmem + 128u * t, sw128_desc(q_addr + t * (kTile * D * 2) + off), sw128_desc(k_addr + off),
                   idesc_bf16(kStep), ks > 0);
          }
          mma_commit(&s_full[t]);
        }
      };
      for (long long u = u0; u < u1 && ok;) {
        const long long ue = min(u1, w.ia + w.t.n);
        const int n = (int)(ue - u), nt = w.t.nrows > kTile ? 2 : 1;
        op_wait(base);
        for (int t = 0; t < nt && ok; ++t) {
          wait(&q_full[t], nq[t]++);
          if (ok) scores(t, base);
        }
        if (ok && lane == 0) mma_commit(&op_empty[base % NS]);
        for (int j = 0; j < n && ok; ++j) {
          const int vo = base + (j == n - 1 ? 2 * n - 1 : 2 * j + 2), ko = base + 2 * j + 1;
          op_wait(vo);
          if (j + 1 < n) op_wait(ko);
          for (int t = 0; t < nt && ok; ++t) {
            const uint32_t v_addr = op_addr + (uint32_t)(vo % NS) * C::kSlotBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              wait(&p_full[t][h], np[t]);
              if (ok && lane == 0) {
                fence_after();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  mma_ts(tmem + 256u + (uint32_t)(D * t), tmem + 128u * t + 32u * h + 8u * ks,
                         sw128_desc(v_addr + (uint32_t)(h * D * 128) + 32u * ks), idesc_bf16(D), j > 0 || h > 0 || ks > 0);
              }
            }
            ++np[t];
            if (!ok) break;
            if (lane == 0) {
              if (t == nt - 1) mma_commit(&op_empty[vo % NS]);
              if (j == n - 1) mma_commit(&o_full[t]);
            }
            if (j + 1 < n) {
              scores(t, ko);
              if (t == nt - 1 && lane == 0) mma_commit(&op_empty[ko % NS]);
            }
            __syncwarp();
          }
        }
        base += 2 * n;
        u = ue;
        if (u < u1) w.next(a, pre);
      }
      if (!ok && lane == 0) atomicMax(&g_error, (int)kv::kErrWait);
      // every MMA is complete before TMEM is freed: the last commit tracks all of them
      if (ok && base > 0) {
        const int o = base - 1;
        wait(&op_empty[o % NS], o / NS);
        if (!ok && lane == 0) atomicMax(&g_error, (int)kv::kErrWait);
      }
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- softmax, epilogue
    const int t = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + 128u * t, to = tmem + lanes + 256u + (uint32_t)(D * t);
    uint8_t* const qs = q_smem + t * (kTile * D * 2);
    int step = 0, cnt = 0, pieces = 0;  // steps of the CTA, of this half, pieces of this half
    bool ok = true;
    for (long long u = u0; u < u1;) {
      const long long ue = min(u1, w.ia + w.t.n);
      const int p0 = (int)(u - w.ia), n = (int)(ue - u);
      const bool live = w.t.nrows > kTile * t;  // this half has rows
      const bool whole = p0 == 0 && n == w.t.n;
      float m = -INFINITY, l = 0.f;
      if (live && ok) {
        const int rr = w.t.r0 + min(kTile * t + row, w.t.nrows - 1), pos = w.g.pos0 + rr / a.group;
        const int plo = w.g.pos0 + (w.t.r0 + kTile * t) / a.group;
        const int phi = w.g.pos0 + (w.t.r0 + min(kTile * t + kTile, w.t.nrows) - 1) / a.group;
        const uint4* qp = reinterpret_cast<const uint4*>(a.q + (int64_t)(w.g.s.row0 + rr / a.group) * a.q_stride +
                                                         (w.head * a.group + rr % a.group) * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(qs + (c >> 3) * (kTile * 128) + sw128(row, c & 7)) = __ldg(qp + c);
        fence_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
        for (int j = 0; j < n && ok; ++j, ++cnt) {
          const int sr = (step + j) % kScaleRing, key0 = kStep * step_at(w.t, p0 + j);
          ok = __all_sync(0xffffffffu, mbar_wait(&sc_full[sr], (uint32_t)(((step + j) / kScaleRing) & 1)) &&
                                           mbar_wait(&s_full[t], (uint32_t)(cnt & 1)));
          if (!ok) break;
          fence_after();
          bool masked[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k0 = key0 + kv::kBlock * h, k1 = k0 + kv::kBlock - 1;
            masked[h] = !alive[sr][h] || k1 > plo || (a.window > 0 && k0 <= phi - a.window && k1 >= a.sinks);
          }
          // pass one: the row's maximum
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(ts + 32 * c, v);
            wait_ld();
            float z[32];
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(&ksc[sr][32 * c + x]);
              unpack2(mul2(pack2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), pack2(k4.x, k4.y)), z[x], z[x + 1]);
              unpack2(mul2(pack2(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), pack2(k4.z, k4.w)), z[x + 2],
                      z[x + 3]);
            }
            if (masked[c >> 1]) {
              const int kb = key0 + 32 * c;
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (!alive[sr][c >> 1] || !sees(a, pos, kb + x)) z[x] = -INFINITY;
            }
#pragma unroll
            for (int x = 0; x < 32; x += 2) mx = fmaxf(mx, fmaxf(z[x], z[x + 1]));
          }
          const bool grow = mx > m + kSlack || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? mx : m, f = grow ? exp2_approx(m - mn) : 1.f;
            m = mn;
            l *= f;
            if (j > 0) {  // S of this step follows P V of the step before: O is at rest
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(to + 32 * c, v);
                wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * f);
                tmem_st32(to + 32 * c, v);
              }
              wait_st();
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;
          const f2 mneg = pack2(-mu, -mu);
          // pass two: P over S, 64 keys at a time
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pr[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              tmem_ld32(ts + 64 * h + 32 * c, v);
              wait_ld();
              const int kb = 64 * h + 32 * c;
              f2 sum = pack2(0.f, 0.f);
#pragma unroll
              for (int x = 0; x < 32; x += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(&ksc[sr][kb + x]);
                const float4 v4 = *reinterpret_cast<const float4*>(&vsc[sr][kb + x]);
                float e[4];
                unpack2(fma2(pack2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), pack2(k4.x, k4.y), mneg), e[0], e[1]);
                unpack2(fma2(pack2(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), pack2(k4.z, k4.w), mneg), e[2],
                        e[3]);
                bool see[4];
                if (masked[h]) {
#pragma unroll
                  for (int y = 0; y < 4; ++y) {
                    see[y] = alive[sr][h] && sees(a, pos, key0 + kb + x + y);
                    if (!see[y]) e[y] = -INFINITY;
                  }
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) e[y] = exp2_approx(e[y]);
                const f2 e01 = pack2(e[0], e[1]), e23 = pack2(e[2], e[3]);
                sum = add2(sum, add2(e01, e23));
                float q[4];
                unpack2(mul2(e01, pack2(v4.x, v4.y)), q[0], q[1]);
                unpack2(mul2(e23, pack2(v4.z, v4.w)), q[2], q[3]);
                if (masked[h]) {  // a key that is not seen has weight 0 whatever its value's scale is
#pragma unroll
                  for (int y = 0; y < 4; ++y)
                    if (!see[y]) q[y] = 0.f;
                }
                pr[16 * c + x / 2] = bf16x2(q[0], q[1]);
                pr[16 * c + x / 2 + 1] = bf16x2(q[2], q[3]);
              }
              float s0, s1;
              unpack2(sum, s0, s1);
              l += s0 + s1;
            }
            tmem_st32(ts + 32 * h, pr);
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[t][h]);
          }
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&o_full[t], (uint32_t)(pieces & 1)));
        ++pieces;
        // ---- epilogue: the outputs, or a partial
        if (ok) {
          fence_after();
          const bool mine = kTile * t + row < w.t.nrows;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint16_t* const op = a.out + (int64_t)(w.g.s.row0 + rr / a.group) * a.out_stride +
                               (w.head * a.group + rr % a.group) * D;
          float* const part = a.partial + (size_t)(2 * blockIdx.x + (u != u0)) * C::kPiece;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(to + 32 * c, v);
            wait_ld();
            if (mine && whole) {
#pragma unroll
              for (int x = 0; x < 32; x += 8) {
                uint32_t o[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  o[y] = bf16x2(__uint_as_float(v[x + 2 * y]) * inv, __uint_as_float(v[x + 2 * y + 1]) * inv);
                *reinterpret_cast<uint4*>(op + 32 * c + x) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            } else if (mine) {
#pragma unroll
              for (int x = 0; x < 32; x += 4)
                *reinterpret_cast<uint4*>(part + ((size_t)(8 * c + x / 4) * kRows + kTile * t + row) * 4) =
                    make_uint4(v[x], v[x + 1], v[x + 2], v[x + 3]);
            }
          }
          if (mine && !whole)
            *reinterpret_cast<float2*>(part + kRows * D + 2 * (kTile * t + row)) = make_float2(m, l);
          fence_before();
        }
      }
      if (!whole) {
        asm volatile("bar.sync 1, 256;" ::: "memory");
        // CTA of unit v: the largest c with U c / G <= v
        const int c0 = (int)(((w.ia + 1) * G - 1) / U), c1 = (int)(((w.ia + w.t.n) * G - 1) / U);
        if (threadIdx.x == 0) s_last = atom_add_acq_rel(a.tickets + c0, 1u) == (uint32_t)(c1 - c0);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (s_last) {
          const int pad = (w.t.nrows + 31) / 32 * 32;
          for (int x = threadIdx.x; x < pad * (D / 4); x += 32 * kSoftWarps) {
            const int r = x % pad, d4 = x / pad;
            if (r >= w.t.nrows) continue;
            float mm = -INFINITY, ll = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
              // the tile's piece is its CTA's first unless the tile begins inside that CTA's range
              const float* pp = a.partial + (size_t)(2 * c + (U * c / G < w.ia)) * C::kPiece;
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(pp + kRows * D + 2 * r));
              const float4 v = __ldcg(reinterpret_cast<const float4*>(pp + ((size_t)d4 * kRows + r) * 4));
              const float mn = fmaxf(mm, ml.x), mu = mn == -INFINITY ? 0.f : mn;
              const float f0 = exp2_approx(mm - mu), f1 = exp2_approx(ml.x - mu);
              mm = mn;
              ll = fmaf(f1, ml.y, f0 * ll);
              o.x = fmaf(f1, v.x, f0 * o.x);
              o.y = fmaf(f1, v.y, f0 * o.y);
              o.z = fmaf(f1, v.z, f0 * o.z);
              o.w = fmaf(f1, v.w, f0 * o.w);
            }
            const int rr = w.t.r0 + r;
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            uint16_t* const op = a.out + (int64_t)(w.g.s.row0 + rr / a.group) * a.out_stride +
                                 (w.head * a.group + rr % a.group) * D + 4 * d4;
            *reinterpret_cast<uint2*>(op) = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
          }
          if (threadIdx.x == 0) a.tickets[c0] = 0u;
        }
      }
      step += n;
      u = ue;
      if (u < u1) w.next(a, pre);
    }
    if (!ok && lane == 0) atomicMax(&g_error, (int)kv::kErrWait);
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
