// Attention of a few new tokens per sequence (one, a speculation window) over the paged cache.
//
// Mathematics: one pass over the keys with the running maximum m and sum l of the softmax in
// powers of two; a row's state (m, l, o) of any set of keys joins another's by
//   M = max(m1, m2), l = l1 2^(m1-M) + l2 2^(m2-M), o likewise,
// so the keys are split freely. Codes enter the tensor-core products exactly (as bf16
// values, fl_attn.cuh); the key's scale multiplies its score column, the value's its probability.
//
// Rounding: a probability times its value's scale enters the second product as bf16, the one type of
// that product whose exponents hold every scale (fp16 would need the scales brought to one size for
// each page). The error against 64 bits is 0.0022-0.0026 of the output's size, where rounding the
// output alone gives 0.0017; rounding P alone gives 0.0016.
//
// Bound: HBM bytes of the visible records (512 + 128 D at D8, 512 + 64 D at D4 per page and head).
// Measured: 8 streams of 45-49k tokens at D4, 112 us (63 us at the copy rate). The copies alone take
// 88 us and the arithmetic alone 99: unpacking and the softmax, not the MMAs (16% of their pipe).
// Five, six or eleven consumer warps instead of seven took 127, 118 and 120 us.
//
// How: scores and outputs are computed transposed, S^T = K Q^T and O^T = V^T P^T, so that the 64
// keys and the D dims fill the 16-row side of mma.m16n8k16 and the few query rows of one
// key/value head (n_i * group) its 8-column side: eight or sixteen rows cost what they are, not a
// 128-row tile's worth. The record's bytes lie in fragment order, so one 16-byte shared load per
// lane feeds four MMAs, and S^T's accumulators become P^T's operand by one movmatrix per 8 keys.
//  * Unit = (sequence, head, row tile, page). The units of the call, in that order, are cut into
//    equal contiguous ranges, one per CTA (each CTA scans the device lengths itself, so a captured
//    launch follows them). A producer warp streams whole records (one bulk copy each) through a
//    ring of stages; seven consumer warps take the units in turn, each with its own (m, l, o).
//  * At the end of an item (sequence, head, row tile) the warps' states join in shared memory. An
//    item cut by a range boundary leaves partials in the workspace, joined by the CTA that arrives
//    last, in CTA order, so results do not depend on the order of arrival.
#include <math.h>

#include <algorithm>

#include "fl_attn.cuh"

namespace fl {
namespace attn {

__device__ int g_error;

constexpr int kWarps = 7;                       // consumer warps
constexpr int kConsumers = 32 * kWarps;
constexpr int kThreads = kConsumers + 32;       // and the producer warp
constexpr int kMaxGrid = 512;
constexpr int kSmemLimit = 232448 - 12288;      // opt-in shared memory per block, less static use

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;          // floats per row of the joining buffer
  static constexpr int kRec = kv::record_bytes(D);
  static constexpr int kJoin = kWarps * kRows * kPitch * 4;
  static constexpr int kFit = (kSmemLimit - kJoin) / kRec;
  static constexpr int kStages = kFit < 20 ? kFit : 20;
  static constexpr int kSmem = kStages * kRec + kJoin;
  static_assert(kStages >= kWarps, "the consumers' waits count on it");
  static constexpr int kPiece = kRows * (D + 2);  // floats of a partial: o, then (m, l) per row
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ void consumer_bar() { asm volatile("bar.sync 1, %0;" ::"r"(kConsumers) : "memory"); }

// A warp's state for one item: query columns 8 nt + 2 t and + 1 of lane (g, t).
template <int D, int NT>
struct State {
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2];  // l is this lane's share of the keys
};

// One page: scores of its 64 keys, the online softmax step, and the product with its values.
// mask(key, pos) is applied only where the page is not wholly visible.
template <int D, int NT, bool kD8>
__device__ __forceinline__ void page_step(const Args& a, const uint8_t* rec, int key0, bool masked, const int (&pos)[NT][2],
                                          const uint32_t (&qf)[D / 16][NT][2], State<D, NT>& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const uint8_t* const khi = rec + kv::kScaleBytes + 16 * lane;
  const uint8_t* const klo = khi + 2 * kv::plane_bytes(D);
  const uint8_t* const vhi = khi + kv::plane_bytes(D);
  const uint8_t* const vlo = khi + 3 * kv::plane_bytes(D);
  const int slot0 = 16 * (g >> 1) + (g & 1);  // + 4 s, and + 2 for the second half
  float z[4][NT][4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) z[s][nt][c] = 0.f;
#pragma unroll
    for (int S = 0; S < D / 64; ++S) {
      const int off = 512 * ((D / 64) * s + S);
      const uint4 h = lds128(khi + off);
      uint4 l = make_uint4(0, 0, 0, 0);
      if (kD8) l = lds128(klo + off);
#pragma unroll
      for (int w = 0; w < 2; ++w) {  // 8 dims of a lane's 16
        uint32_t x[4], y[4];         // slots 4 s + .. and 4 s + 2 + ..
        unpack_word<kD8>(w ? h.y : h.x, w ? l.y : l.x, x);
        unpack_word<kD8>(w ? h.w : h.z, w ? l.w : l.z, y);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_bf16(z[s][nt], x[2 * e], y[2 * e], x[2 * e + 1], y[2 * e + 1], qf[4 * S + 2 * w + e][nt][0],
                     qf[4 * S + 2 * w + e][nt][1]);
      }
    }
    const float k0 = lds32(rec + 4 * (slot0 + 4 * s)) * (value_factor<kD8>() * a.scale_log2);
    const float k1 = lds32(rec + 4 * (slot0 + 4 * s + 2)) * (value_factor<kD8>() * a.scale_log2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        z[s][nt][c] *= c < 2 ? k0 : k1;
  }
  if (masked) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!sees(a, pos[nt][c & 1], key0 + slot0 + 4 * s + (c & 2))) z[s][nt][c] = -INFINITY;
  }
  float mu[NT][2];
  bool moved = false;
  float alpha[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = st.m[nt][e];
#pragma unroll
      for (int s = 0; s < 4; ++s) mx = fmaxf(mx, fmaxf(z[s][nt][e], z[s][nt][e + 2]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      mu[nt][e] = mx == -INFINITY ? 0.f : mx;  // nothing visible yet: every power below is 0
      alpha[nt][e] = exp2_approx(st.m[nt][e] - mu[nt][e]);
      moved = moved || mx != st.m[nt][e];
      st.m[nt][e] = mx;
    }
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) st.l[nt][e] *= alpha[nt][e];
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.o[dt][nt][c] *= alpha[nt][c & 1];
    }
  }
  uint32_t pf[4][NT][2];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const float v0 = lds32(rec + 256 + 4 * (slot0 + 4 * s)) * value_factor<kD8>();
    const float v1 = lds32(rec + 256 + 4 * (slot0 + 4 * s + 2)) * value_factor<kD8>();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float e = exp2_approx(z[s][nt][c] - mu[nt][c & 1]);
        st.l[nt][c & 1] += e;
        // a key that is not seen has weight 0 whatever its value's scale is
        p[c] = masked && z[s][nt][c] == -INFINITY ? 0.f : e * (c < 2 ? v0 : v1);
      }
      pf[s][nt][0] = transpose8x8(bf16x2(p[0], p[1]));
      pf[s][nt][1] = transpose8x8(bf16x2(p[2], p[3]));
    }
  }
#pragma unroll
  for (int dt = 0; dt < D / 16; ++dt) {
    const uint4 h = lds128(vhi + 512 * dt);
    uint4 l = make_uint4(0, 0, 0, 0);
    if (kD8) l = lds128(vlo + 512 * dt);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint32_t x[4];
      unpack_word<kD8>(s == 0 ? h.x : s == 1 ? h.y : s == 2 ? h.z : h.w, s == 0 ? l.x : s == 1 ? l.y : s == 2 ? l.z : l.w, x);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16(st.o[dt][nt], x[0], x[1], x[2], x[3], pf[s][nt][0], pf[s][nt][1]);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, NT>;
  constexpr int R = C::kRows, NS = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[NS], empty_bar[NS];
  __shared__ int2 meta[NS];  // (block of the sequence, level)
  __shared__ long long pre[FL_KV_MAX_SEQS + 1];
  __shared__ long long wsum[kWarps];
  __shared__ float sm_m[kWarps][R], sm_l[kWarps][R];
  __shared__ int s_last, s_items;
  float* const join = reinterpret_cast<float*>(smem + NS * C::kRec);

  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s_items = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    fence_mbar_init();
  }
  pdl_wait();

  // ---- units before each sequence
  const int n_seqs = a.b.n_seqs, per = (n_seqs + kConsumers - 1) / kConsumers;
  long long mine = 0, inc = 0;
  __syncthreads();
  if (warp < kWarps) {
    bool bad = false;
    int items = 0;
    for (int k = 0; k < per; ++k) {
      const int i = threadIdx.x * per + k;
      if (i >= n_seqs) break;
      const Geo g = geo_of(a, i, &bad);
      mine += (long long)a.kv_heads * ((g.s.n * a.group + R - 1) / R) * g.np;
      if (g.np > 0) items = min(items + a.kv_heads * ((g.s.n * a.group + R - 1) / R), 1 << 20);
    }
    items = __reduce_add_sync(0xffffffffu, min(items, 1 << 20));
    if (lane == 0 && items > 0) atomicAdd(&s_items, items);
    if (bad && blockIdx.x == 0) atomicOr(&g_error, (int)kv::kErrSeq);
    inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 31) wsum[warp] = inc;
  }
  __syncthreads();
  if (warp < kWarps) {
    long long before = inc - mine;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    bool bad = false;
    for (int k = 0; k < per; ++k) {
      const int i = threadIdx.x * per + k;
      if (i >= n_seqs) break;
      pre[i] = before;
      if (per > 1) {
        const Geo g = geo_of(a, i, &bad);
        before += (long long)a.kv_heads * ((g.s.n * a.group + R - 1) / R) * g.np;
      } else {
        before += mine;
      }
      if (i == n_seqs - 1) pre[n_seqs] = before;
    }
  }
  __syncthreads();
  const long long U = pre[n_seqs];
  // A CTA takes at least one unit per warp; where two per warp and item would do, one CTA per item,
  // so that items of equal lengths are not cut (a join through the workspace costs more than the
  // second unit: one stream of 517 tokens took 13.2 us cut, 9.5 us so).
  const long long items = s_items;
  const int G = items <= gridDim.x && U <= 2 * kWarps * items ? (int)items
                                                              : (int)min((long long)gridDim.x, (U + kWarps - 1) / kWarps);
  if ((int)blockIdx.x >= G) return;
  const long long u0 = U * blockIdx.x / G, u1 = U * (blockIdx.x + 1) / G;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    bool failed = false;
    int issued = 0;
    for (long long base = u0; base < u1 && !failed; base += 32) {
      const long long u = base + lane;
      int block = 0, lv = 0;
      const uint8_t* src = nullptr;
      if (u < u1) {
        const int i = find_seq(pre, n_seqs, u);
        bool bad = false;
        const Geo g = geo_of(a, i, &bad);
        const unsigned rem = (unsigned)(u - pre[i]), np = (unsigned)g.np;
        const unsigned item = rem / np, tiles = (unsigned)((g.s.n * a.group + R - 1) / R);
        block = page_at(g, (int)(rem - item * np));
        const size_t at = (size_t)i * a.b.max_blocks + block;
        lv = kv::level_of(a.levels, at);
        const int page = __ldg(a.b.table + at);
        if (page < 0 || page >= a.num_pages) {  // a ZERO block's entry may be anything
          if (lv > 0) atomicOr(&g_error, (int)kv::kErrPage);
          lv = 0;
        } else {
          src = a.pages + ((size_t)page * a.kv_heads + item / tiles) * C::kRec;
        }
      }
      const int cnt = (int)min((long long)32, u1 - base);
      for (int k = 0; k < cnt; ++k, ++issued) {
        const int s = issued % NS;
        if (issued >= NS && !__all_sync(0xffffffffu, mbar_wait(&empty_bar[s], (uint32_t)((issued / NS - 1) & 1)))) {
          failed = true;
          break;
        }
        if (lane == k) {
          const uint32_t bytes = lv == 0 ? 0u : (uint32_t)kv::depth_bytes(D, lv == 4);
          meta[s] = make_int2(block, lv);
          mbar_expect_tx(&full_bar[s], bytes);
          if (bytes) bulk_g2s(smem + s * C::kRec, src, bytes, &full_bar[s]);
        }
        __syncwarp();
      }
    }
    if (failed && lane == 0) atomicOr(&g_error, (int)kv::kErrWait);
    // no copy may still be landing when the CTA exits
    for (int k = max(0, issued - NS); k < issued; ++k)
      if (!mbar_wait(&full_bar[k % NS], (uint32_t)((k / NS) & 1)) && lane == 0) atomicOr(&g_error, (int)kv::kErrWait);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = lane >> 2, t = lane & 3;
  bool failed = false;
  for (long long u = u0; u < u1;) {
    const int i = find_seq(pre, n_seqs, u);
    bool bad = false;
    const Geo geo = geo_of(a, i, &bad);
    const unsigned rem = (unsigned)(u - pre[i]), np = (unsigned)geo.np, item = rem / np;
    const unsigned tiles = (unsigned)((geo.s.n * a.group + R - 1) / R);
    const long long ia = pre[i] + (long long)item * np, ie = ia + np;  // the item's units
    const long long ue = min(u1, ie);
    const int head = (int)(item / tiles), r0 = (int)(item % tiles) * R, nrows = min(R, geo.s.n * a.group - r0);
    const int pos_lo = geo.pos0 + r0 / a.group, pos_hi = geo.pos0 + (r0 + nrows - 1) / a.group;

    // query fragments: column n = 8 nt + g, dims 64 S + 16 t + 4 ks .. + 3
    uint32_t qf[D / 16][NT][2];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = min(8 * nt + g, nrows - 1) + r0;
      const uint16_t* qp = a.q + (int64_t)(geo.s.row0 + r / a.group) * a.q_stride + (head * a.group + r % a.group) * D;
#pragma unroll
      for (int S = 0; S < D / 64; ++S) {
        const uint4 q0 = __ldg(reinterpret_cast<const uint4*>(qp + 64 * S + 16 * t));
        const uint4 q1 = __ldg(reinterpret_cast<const uint4*>(qp + 64 * S + 16 * t + 8));
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          qf[4 * S + ks][nt][0] = w[2 * ks];
          qf[4 * S + ks][nt][1] = w[2 * ks + 1];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        pos[nt][e] = geo.pos0 + (min(8 * nt + 2 * t + e, nrows - 1) + r0) / a.group;
      }
    }
    State<D, NT> st;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        st.m[nt][e] = -INFINITY;
        st.l[nt][e] = 0.f;
      }
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.o[dt][nt][c] = 0.f;
    }
    // this warp's units of the piece: unit k of the CTA goes to warp k % kWarps
    for (int k = (int)(u - u0) + (warp + kWarps - (int)(u - u0) % kWarps) % kWarps; k < (int)(ue - u0) && !failed;
         k += kWarps) {
      const int s = k % NS, lap = k / NS;
      // The stage's previous unit was another warp's, and copies land in any order: a wait for
      // this lap's parity alone would fall through while the previous lap's copy is in flight.
      // Once that unit is consumed (the unit a lap before it is, since this warp's last unit was
      // issued after it and NS >= kWarps), the parity is this lap's own.
      if (!__all_sync(0xffffffffu, (lap == 0 || mbar_wait(&empty_bar[s], (uint32_t)((lap - 1) & 1))) &&
                                       mbar_wait(&full_bar[s], (uint32_t)(lap & 1)))) {
        if (lane == 0) atomicOr(&g_error, (int)kv::kErrWait);
        failed = true;
        break;
      }
      const int2 mt = meta[s];
      const int key0 = mt.x * kv::kBlock, key1 = key0 + kv::kBlock - 1;
      const uint8_t* const rec = smem + s * C::kRec;
      const bool none = mt.y == 0 || key0 > pos_hi ||
                        (a.window > 0 && key0 >= a.sinks && pos_lo - key1 >= a.window);
      const bool masked = key1 > pos_lo || (a.window > 0 && pos_hi - key0 >= a.window && key1 >= a.sinks);
      if (!none) {
        if (mt.y == 4)
          page_step<D, NT, true>(a, rec, key0, masked, pos, qf, st);
        else
          page_step<D, NT, false>(a, rec, key0, masked, pos, qf, st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[s]);
    }
    // ---- join the warps' states
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[nt][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const int r = 8 * nt + 2 * t + e;
        if (g == 0) {
          sm_m[warp][r] = st.m[nt][e];
          sm_l[warp][r] = l;
        }
        float* jp = join + (warp * R + r) * C::kPitch + g;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          jp[16 * dt] = st.o[dt][nt][e];
          jp[16 * dt + 8] = st.o[dt][nt][e + 2];
        }
      }
    consumer_bar();
    const bool whole = u == ia && ue == ie;
    float* part = a.partial + (size_t)(2 * blockIdx.x + (u != u0)) * C::kPiece;
    for (int x = threadIdx.x; x < R * D / 4; x += kConsumers) {
      const int r = x / (D / 4), d = 4 * (x % (D / 4));
      if (r >= nrows) break;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_m[w][r]);
      const float mu = m == -INFINITY ? 0.f : m;
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_approx(sm_m[w][r] - mu);
        const float4 v = *reinterpret_cast<const float4*>(join + (w * R + r) * C::kPitch + d);
        l = fmaf(f, sm_l[w][r], l);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
      }
      if (whole) {
        const int rr = r0 + r;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* op = a.out + (int64_t)(geo.s.row0 + rr / a.group) * a.out_stride +
                       (head * a.group + rr % a.group) * D + d;
        *reinterpret_cast<uint2*>(op) = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = o;
        if (d == 0) {
          part[R * D + 2 * r] = m;
          part[R * D + 2 * r + 1] = l;
        }
      }
    }
    consumer_bar();  // the joining buffer is free again; a partial is written
    if (!whole) {
      // CTA of unit v: the largest c with U c / G <= v
      const int c0 = (int)(((ia + 1) * G - 1) / U), c1 = (int)((ie * G - 1) / U);
      if (threadIdx.x == 0)
        s_last = atom_add_acq_rel(a.tickets + c0, 1u) == (uint32_t)(c1 - c0);
      consumer_bar();
      if (s_last) {
        for (int x = threadIdx.x; x < R * D / 4; x += kConsumers) {
          const int r = x / (D / 4), d = 4 * (x % (D / 4));
          if (r >= nrows) break;
          float m = -INFINITY, l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            // the item's piece is its CTA's first unless the item begins inside that CTA's range
            const float* pp = a.partial + (size_t)(2 * c + (U * c / G < ia)) * C::kPiece;
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(pp + R * D + 2 * r));
            const float4 v = __ldcg(reinterpret_cast<const float4*>(pp + r * D + d));
            const float mn = fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.f : mn;
            const float f0 = exp2_approx(m - mu), f1 = exp2_approx(ml.x - mu);
            m = mn;
            l = fmaf(f1, ml.y, f0 * l);
            o.x = fmaf(f1, v.x, f0 * o.x);
            o.y = fmaf(f1, v.y, f0 * o.y);
            o.z = fmaf(f1, v.z, f0 * o.z);
            o.w = fmaf(f1, v.w, f0 * o.w);
          }
          const int rr = r0 + r;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint16_t* op = a.out + (int64_t)(geo.s.row0 + rr / a.group) * a.out_stride +
                         (head * a.group + rr % a.group) * D + d;
          *reinterpret_cast<uint2*>(op) = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
        }
        if (threadIdx.x == 0) a.tickets[c0] = 0u;
      }
    }
    u = ue;
  }
}

// ---------------------------------------------------------------- host side

struct Ws {
  size_t tickets, tc_tickets, partial, tc_partial, total;
};

// Which kernel takes a sequence: this one reads and unpacks a page again for every 16 rows; the chunk
// kernel does it once for 256, but starts, ends and joins its tiles at 30-50 us more a call. With
// r rows that see p pages, in a call of nk (sequence, head) pairs, this kernel's extra time grows as
// (r - 56) p nk (at 64 rows both read at the same rate), and what it saves shrinks as nk grows, since
// many tiles need few joins. Measured, this kernel against the other, us, eight heads:
//   D = 128   1 x 4k: 128 rows 30, 56; 256 rows 40, 74    1 x 32k: 96 rows 86, 93; 256 rows 192, 132
//             2 x 100k: 64 rows 304, 299; 256 rows 1191, 400    4 x 4k: 128 rows 68, 67
//             8 x 1k: 96 rows 44, 48; 256 rows 88, 64    8 x 4k: 64 rows 68, 87; 128 rows 121, 92
//   D = 64    1 x 4k: 256 rows 30, 64    1 x 32k: 128 rows 79, 82; 256 rows 144, 110
//             2 x 100k: 64 rows 224, 266; 256 rows 861, 335    8 x 4k: 96 rows 65, 74; 128 rows 81, 75
// Over 306 such shapes (1k to 100k tokens, both depths, groups of 2, 4 and 8) the chosen kernel is
// within 12% of the better one, 0.2% on average. Each sequence's own pages count, not the table's
// width, so both kernels are launched where the call's bounds leave the choice open: 5 to 7 us, for
// instance 28 instead of 22 us for 128 rows over 1,000 tokens under a table of 131,072.
static long long chunk_budget(int D, long long nk) {
  return D == 64 ? std::min(400000ll, 12000000 / nk) / nk : std::min(280000ll, 5000000 / nk) / nk;
}

// Rows per tile by the largest number of rows a (sequence, head) has: eight columns cost half the
// MMAs of sixteen.
static int row_tiles(long long max_rows) { return max_rows <= 8 ? 1 : 2; }

static Ws ws_layout(int nsm, int D, long long max_rows, bool chunks) {
  Ws w;
  w.tickets = 0;
  w.tc_tickets = (size_t)kMaxGrid * 4;
  w.partial = 2 * (size_t)kMaxGrid * 4;
  w.tc_partial = w.partial + (size_t)nsm * 2 * (8 * row_tiles(max_rows)) * (D + 2) * 4;
  w.total = w.tc_partial + (chunks ? attn_tc::partial_bytes(D, nsm) : 0);
  return w;
}

template <int D, int NT>
static fl_status launch(const Args& a, int nsm, cudaStream_t st) {
  auto kern = attn_kernel<D, NT>;
  FL_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::kSmem),
                "cudaFuncSetAttribute(attn)");
  FL_CHECK_CUDA(launch_pdl(kern, dim3((unsigned)nsm), dim3(kThreads), (size_t)Cfg<D, NT>::kSmem, st, 1, a),
                "launch attn");
  return FL_OK;
}

// Reads and clears the error word (-1 if that fails).
int take_device_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_error, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0 && cudaMemcpyToSymbol(g_error, &z, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

static bool shape_ok(int n_seqs, int heads, int kv_heads, int head_dim, int max_new) {
  return (head_dim == 64 || head_dim == 128) && kv_heads >= 1 && kv_heads <= 256 && heads >= kv_heads &&
         heads % kv_heads == 0 && heads / kv_heads <= FL_ATTN_MAX_GROUP && n_seqs >= 1 && n_seqs <= FL_KV_MAX_SEQS &&
         max_new >= 1 && max_new <= (1 << 22);
}

}  // namespace attn
}  // namespace fl

extern "C" size_t fl_attn_workspace_bytes(int n_seqs, int heads, int kv_heads, int head_dim, int max_new) {
  using namespace fl;
  const int nsm = std::min(device_sm_count(), attn::kMaxGrid);
  if (nsm <= 0 || !attn::shape_ok(n_seqs, heads, kv_heads, head_dim, max_new)) return 0;
  const long long max_rows = (long long)max_new * (heads / kv_heads);
  return attn::ws_layout(nsm, head_dim, max_rows, max_rows > attn::kShortRows).total;
}

extern "C" fl_status fl_attn_paged(const fl_kv_cache* cache, const fl_kv_batch* batch, const uint8_t* levels,
                                   const uint16_t* q, int64_t q_stride, int heads, float scale, int window, int sinks,
                                   uint16_t* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  using namespace fl;
  const char* what = "fl_attn_paged";
  if (fl_status s = kv::check_batch(what, cache, batch)) return s;
  const int D = cache->head_dim, Hkv = cache->kv_heads;
  if (heads < 1 || heads % Hkv != 0 || heads / Hkv > FL_ATTN_MAX_GROUP)
    return fail(FL_ERR_SHAPE, "%s: heads=%d (a multiple of kv_heads=%d, at most %d times it)", what, heads, Hkv,
                FL_ATTN_MAX_GROUP);
  if (fl_status s = kv::check_rows(what, "q", q, q_stride, heads * D)) return s;
  if (fl_status s = kv::check_rows(what, "out", out, out_stride, heads * D)) return s;
  // 2^117: scale log2(e) times the codes' factor (2^10 at D4) is still finite in fp32
  if (!(fabsf(scale) <= 0x1p117f)) return fail(FL_ERR_ARG, "%s: scale=%g (at most 2^117 in magnitude)", what, scale);
  if (window < 0 || sinks < 0) return fail(FL_ERR_ARG, "%s: window=%d, sinks=%d (>= 0)", what, window, sinks);
  const int nsm = std::min(device_sm_count(), attn::kMaxGrid);
  if (nsm <= 0) return fail(FL_ERR_CUDA, "%s: no CUDA device", what);
  const int group = heads / Hkv, max_rows = batch->max_new * group, nt = attn::row_tiles(max_rows);
  // a sequence's units, and a CTA's, are counted in 32 bits
  const double units = (double)Hkv * ((max_rows + 8 * nt - 1) / (8 * nt)) * batch->max_blocks;
  if (units > 2147483647.0 || units * batch->n_seqs / nsm > 2147483647.0)
    return fail(FL_ERR_SHAPE, "%s: max_new=%d over max_blocks=%d is too large for one call", what, batch->max_new,
                batch->max_blocks);
  // what a sequence of this call can ask for at most
  long long pages = batch->max_blocks;
  if (window > 0)
    pages = std::min(pages, ((long long)window + batch->max_new + 62) / kv::kBlock + 1 + ((long long)sinks + 63) / kv::kBlock);
  const long long budget = attn::chunk_budget(D, (long long)batch->n_seqs * Hkv);
  const bool chunks = attn::chunk_takes(max_rows, pages, budget);
  const attn::Ws wl = attn::ws_layout(nsm, D, max_rows, chunks);
  if (!workspace || workspace_bytes < wl.total)
    return fail(FL_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, workspace ? workspace_bytes : (size_t)0,
                wl.total);
  if (!aligned16(workspace)) return fail(FL_ERR_ALIGN, "%s: workspace not 16-byte aligned", what);
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  attn::Args a;
  a.pages = cache->pages;
  a.num_pages = cache->num_pages;
  a.kv_heads = Hkv;
  a.heads = heads;
  a.group = group;
  a.b = kv::batch_of(batch);
  a.levels = levels;
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.window = window;
  a.sinks = sinks;
  // One sequence that may be a long chunk: the chunk kernel takes it whatever its length turns out to
  // be, and a prompt saves the other launch (about 5 us).
  const bool both = chunks && (batch->n_seqs > 1 || max_rows <= attn::kChunkRows);
  a.takes = both ? attn::kShort : attn::kEvery;
  a.budget = budget;
  a.tickets = reinterpret_cast<uint32_t*>(wsb + wl.tickets);
  a.partial = reinterpret_cast<float*>(wsb + wl.partial);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (both || !chunks) {
    const fl_status s = D == 64 ? (nt == 1 ? attn::launch<64, 1>(a, nsm, st) : attn::launch<64, 2>(a, nsm, st))
                                : (nt == 1 ? attn::launch<128, 1>(a, nsm, st) : attn::launch<128, 2>(a, nsm, st));
    if (s || !both) return s;
  }
  a.takes = both ? attn::kChunk : attn::kEvery;
  a.tickets = reinterpret_cast<uint32_t*>(wsb + wl.tc_tickets);
  a.partial = reinterpret_cast<float*>(wsb + wl.tc_partial);
  return attn_tc::launch(a, D, nsm, st);
}
