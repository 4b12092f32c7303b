// Quantising the paged key/value cache as it is written, and reading it back ("FoQLens"
// landing page, progress table: one stored copy, read to any depth; here the cached tokens).
//
// Mathematics: per token and key/value head, a = max |x_d|, scale = a / 127,
// code_d = rint(127 x_d / a). 127 x_d is exact in fp32 (15 significant bits) and the division
// is IEEE, and no quotient of two bf16 values can round across a half-integer it does not hit
// (it lies at least 2^-17 away, fp32 rounds by at most 2^-18 below 128), so the code equals the
// formula's in exact arithmetic, ties to even. Where 127 a could pass the largest fp32, both sides
// of the division are taken 2^-8 times: the quotient is the same, and an element too small to
// keep its bits has code 0 either way.
//
// Bound: HBM bytes (4 D read and 2 D + 8 written per token-head when appending, the reverse when
// reading). One CTA per (sequence, touched page, key/value head): its 64 x D codes are the unit
// in which the value plane's order (16 tokens of one dim in a 16-byte piece) turns around. Keys
// go from registers straight to their fragment order (eight lanes fill whole 128-byte lines);
// value codes pass through shared memory as bytes and are turned with 4 x 4 byte transposes.
#include "fl_kv.cuh"

namespace fl {
namespace kv {

__device__ int g_error;

constexpr int kThreads = 128;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

// Bytes of four words as a 4 x 4 matrix, transposed: c[i] byte j = r[j] byte i.
__device__ __forceinline__ void transpose4(uint32_t (&r)[4]) {
  const uint32_t t0 = prmt(r[0], r[1], 0x5140), t1 = prmt(r[2], r[3], 0x5140);
  const uint32_t t2 = prmt(r[0], r[1], 0x7362), t3 = prmt(r[2], r[3], 0x7362);
  r[0] = prmt(t0, t1, 0x5410);
  r[1] = prmt(t0, t1, 0x7632);
  r[2] = prmt(t2, t3, 0x5410);
  r[3] = prmt(t2, t3, 0x7632);
}

// u8 codes of 16 consecutive dims (four words, dim order) <-> the key planes' two words, nibble
// n = (d % 8) / 2 + 4 (d % 2): dims 0, 2, 4, 6 in the low half, 1, 3, 5, 7 in the high half.
__device__ __forceinline__ uint32_t pack8(uint32_t lo4, uint32_t hi4) {  // eight nibbles, one per byte
  // even bytes of (lo4, hi4) -> low half, odd -> high half, two nibbles per byte
  const uint32_t ev = prmt(lo4, hi4, 0x6420), od = prmt(lo4, hi4, 0x7531);
  const uint32_t e = (ev & 0x000F000Fu) | ((ev >> 4) & 0x00F000F0u);  // bytes 0 and 2 hold two dims each
  const uint32_t o = (od & 0x000F000Fu) | ((od >> 4) & 0x00F000F0u);
  return prmt(e, o, 0x6420);
}
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t& lo4, uint32_t& hi4) {
  const uint32_t e = prmt(w, 0, 0x4140), o = prmt(w, 0, 0x4342);  // (b0, 0, b1, 0), (b2, 0, b3, 0)
  const uint32_t ev = (e & 0x000F000Fu) | ((e & 0x00F000F0u) << 4);  // dims 0, 2, 4, 6
  const uint32_t od = (o & 0x000F000Fu) | ((o & 0x00F000F0u) << 4);  // dims 1, 3, 5, 7
  lo4 = prmt(ev, od, 0x5140);
  hi4 = prmt(ev, od, 0x7362);
}

// Sixteen bf16 values of a row spread over LPR lanes -> u8 codes (code + 128) and the scale.
template <int LPR>
__device__ __forceinline__ float quantise16(const uint4 (&raw)[2], uint32_t (&code)[4]) {
  const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
  const bool finite = top < 0x7F800000u;  // NaN patterns order above infinity
  const bool live = finite && top != 0u;
  const bool large = top >= 0x7B800000u;  // a >= 2^120: 127 a could be infinite
  const float a = __uint_as_float(top), f = large ? 127.f / 256.f : 127.f, div = large ? a * (1.f / 256.f) : a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t c4 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t ww = w[2 * i + (k >> 1)];
      const float x = __uint_as_float((k & 1) ? (ww & 0xFFFF0000u) : (ww << 16));
      const int c = live ? __float2int_rn(__fdiv_rn(__fmul_rn(x, f), div)) : 0;
      c4 |= (uint32_t)(c + 128) << (8 * k);
    }
    code[i] = c4;
  }
  return finite ? __fdiv_rn(a, 127.f) : __uint_as_float(0x7FC00000u);
}

struct PageJob {
  Seq s;
  int block, head, j0, j1;  // slots [j0, j1) of the block are this call's
  int page, level;     // level 0: the block is ZERO or its page out of range, page is not valid
};

// The CTA's page: grid x = page touched by a sequence's new tokens, y = sequence, z = head.
__device__ __forceinline__ bool page_job(const Batch& b, int num_pages, const uint8_t* levels, PageJob& jb) {
  bool bad = false;
  jb.s = seq_of(b, blockIdx.y, &bad);
  jb.head = blockIdx.z;
  if (bad && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) atomicOr(&g_error, kErrSeq);
  if (jb.s.n == 0) return false;
  const int first = jb.s.len - jb.s.n;
  jb.block = first / kBlock + (int)blockIdx.x;
  if (jb.block * kBlock >= jb.s.len) return false;
  jb.j0 = max(first - jb.block * kBlock, 0);
  jb.j1 = min(jb.s.len - jb.block * kBlock, kBlock);
  const size_t at = (size_t)blockIdx.y * b.max_blocks + jb.block;
  jb.page = __ldg(b.table + at);
  jb.level = level_of(levels, at);
  if (jb.level > 0 && (jb.page < 0 || jb.page >= num_pages)) {
    if (jb.head == 0 && threadIdx.x == 0) atomicOr(&g_error, kErrPage);
    jb.level = 0;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(uint8_t* pages, int num_pages, int kv_heads, const Batch b,
                                                          const uint16_t* k, int64_t ks, const uint16_t* v,
                                                          int64_t vs) {
  constexpr int LPR = D / 16, RPP = kThreads / LPR, P = D + 16;  // lanes per row, rows per pass, code pitch
  __shared__ __align__(16) uint8_t codes[kBlock * P];
  pdl_release();
  pdl_wait();
  PageJob jb;
  if (!page_job(b, num_pages, nullptr, jb) || jb.level == 0) return;
  uint8_t* rec = pages + ((size_t)jb.page * kv_heads + jb.head) * record_bytes(D);
  uint8_t* const khi = rec + kScaleBytes;
  uint8_t* const klo = khi + 2 * plane_bytes(D);
  uint8_t* const vhi = khi + plane_bytes(D);
  uint8_t* const vlo = khi + 3 * plane_bytes(D);
  const int d16 = threadIdx.x % LPR, jr = threadIdx.x / LPR;
  const int64_t row_of_slot0 = (int64_t)jb.s.row0 + (int64_t)jb.block * kBlock - (jb.s.len - jb.s.n);
  const int hoff = jb.head * D + 16 * d16;
  // slots are walked from the four-slot group of the first one, so that four consecutive slots
  // (one 16-byte piece per lane pair of rows) are written together
  for (int base = jb.j0 & ~3; base < jb.j1; base += RPP) {
    const int j = base + jr;
    const bool on = j >= jb.j0 && j < jb.j1;
    uint4 kr[2] = {}, vr[2] = {};
    if (on) {
      const uint4* kp = reinterpret_cast<const uint4*>(k + (row_of_slot0 + j) * ks + hoff);
      const uint4* vp = reinterpret_cast<const uint4*>(v + (row_of_slot0 + j) * vs + hoff);
      kr[0] = __ldg(kp);
      kr[1] = __ldg(kp + 1);
      vr[0] = __ldg(vp);
      vr[1] = __ldg(vp + 1);
    }
    uint32_t kc[4], vc[4];
    const float kscale = quantise16<LPR>(kr, kc), vscale = quantise16<LPR>(vr, vc);
    if (on) {
      uint2 hi, lo;
      hi.x = pack8((kc[0] >> 4) & 0x0F0F0F0Fu, (kc[1] >> 4) & 0x0F0F0F0Fu);
      hi.y = pack8((kc[2] >> 4) & 0x0F0F0F0Fu, (kc[3] >> 4) & 0x0F0F0F0Fu);
      lo.x = pack8(kc[0] & 0x0F0F0F0Fu, kc[1] & 0x0F0F0F0Fu);
      lo.y = pack8(kc[2] & 0x0F0F0F0Fu, kc[3] & 0x0F0F0F0Fu);
      const int o = key_off(D, j, d16);
      *reinterpret_cast<uint2*>(khi + o) = hi;
      *reinterpret_cast<uint2*>(klo + o) = lo;
      *reinterpret_cast<uint4*>(codes + j * P + 16 * d16) = make_uint4(vc[0], vc[1], vc[2], vc[3]);
      if (d16 == 0) {
        reinterpret_cast<float*>(rec)[j] = kscale;
        reinterpret_cast<float*>(rec)[kBlock + j] = vscale;
      }
    }
  }
  __syncthreads();
  // value planes: task = (16 dims T, dims 4 c .. 4 c + 3 and 8 above, 16 slots t)
  for (int task = threadIdx.x; task < D / 16 * 8; task += kThreads) {
    const int t = task & 3, c = (task >> 2) & 1, T = task >> 3;
    const int a0 = max(jb.j0 - 16 * t, 0), a1 = min(jb.j1 - 16 * t, 16);
    if (a0 >= a1) continue;
    uint32_t H[4][4], L[4][4];  // [s][byte], before the transpose
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int bb = 0; bb < 4; ++bb) {
        const int e = (bb >> 1) | ((bb & 1) << 1);  // byte order of slots 0..3: 0, 2, 1, 3
        const uint8_t* cp = codes + (16 * t + 4 * s + e) * P + 16 * T + 4 * c;
        const int jj = 4 * s + e;
        uint32_t w0 = 0, w1 = 0;
        if (jj >= a0 && jj < a1) {
          w0 = *reinterpret_cast<const uint32_t*>(cp);
          w1 = *reinterpret_cast<const uint32_t*>(cp + 8);
        }
        H[s][bb] = ((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u);
        L[s][bb] = (w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u);
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      transpose4(H[s]);
      transpose4(L[s]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = val_off(T, 4 * c + i, t);
      if (a0 == 0 && a1 == 16) {
        *reinterpret_cast<uint4*>(vhi + o) = make_uint4(H[0][i], H[1][i], H[2][i], H[3][i]);
        *reinterpret_cast<uint4*>(vlo + o) = make_uint4(L[0][i], L[1][i], L[2][i], L[3][i]);
      } else {  // the other slots' bytes belong to other tokens
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int jj = 4 * s + e, bb = (e >> 1) | ((e & 1) << 1);
            if (jj >= a0 && jj < a1) {
              vhi[o + 4 * s + bb] = (uint8_t)(H[s][i] >> (8 * bb));
              vlo[o + 4 * s + bb] = (uint8_t)(L[s][i] >> (8 * bb));
            }
          }
      }
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sixteen u8 codes -> bf16(scale (u - 128 + c)), c = 0 (D8) or 7.5 (D4).
__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&code)[4], float scale, float off) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = code[i >> 1] >> (16 * (i & 1));
    r[i] = bf16x2(scale * ((float)(w & 255u) + off), scale * ((float)((w >> 8) & 255u) + off));
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const uint8_t* pages, int num_pages, int kv_heads,
                                                        const Batch b, const uint8_t* levels, uint16_t* k, int64_t ks,
                                                        uint16_t* v, int64_t vs) {
  constexpr int LPR = D / 16, RPP = kThreads / LPR, P = D + 16;
  __shared__ __align__(16) uint8_t codes[kBlock * P];
  pdl_release();
  pdl_wait();
  PageJob jb;
  if (!page_job(b, num_pages, levels, jb)) return;
  const int lv = jb.level;
  const uint8_t* rec = pages + ((size_t)(lv > 0 ? jb.page : 0) * kv_heads + jb.head) * record_bytes(D);
  const uint8_t* const khi = rec + kScaleBytes;
  const uint8_t* const klo = khi + 2 * plane_bytes(D);
  const uint8_t* const vhi = khi + plane_bytes(D);
  const uint8_t* const vlo = khi + 3 * plane_bytes(D);
  const float off = lv == 2 ? -120.5f : -128.f;
  if (lv > 0) {
    for (int task = threadIdx.x; task < D / 16 * 8; task += kThreads) {
      const int t = task & 3, c = (task >> 2) & 1, T = task >> 3;
      if (16 * t >= jb.j1 || 16 * t + 16 <= jb.j0) continue;
      uint4 h[4], l[4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __ldg(reinterpret_cast<const uint4*>(vhi + val_off(T, 4 * c + i, t)));
      if (lv == 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] = __ldg(reinterpret_cast<const uint4*>(vlo + val_off(T, 4 * c + i, t)));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t H[4], L[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          H[i] = s == 0 ? h[i].x : s == 1 ? h[i].y : s == 2 ? h[i].z : h[i].w;
          L[i] = s == 0 ? l[i].x : s == 1 ? l[i].y : s == 2 ? l[i].z : l[i].w;
        }
        transpose4(H);
        transpose4(L);
#pragma unroll
        for (int bb = 0; bb < 4; ++bb) {
          const int e = (bb >> 1) | ((bb & 1) << 1);
          uint8_t* cp = codes + (16 * t + 4 * s + e) * P + 16 * T + 4 * c;
          *reinterpret_cast<uint32_t*>(cp) = ((H[bb] << 4) & 0xF0F0F0F0u) | (L[bb] & 0x0F0F0F0Fu);
          *reinterpret_cast<uint32_t*>(cp + 8) = (H[bb] & 0xF0F0F0F0u) | ((L[bb] >> 4) & 0x0F0F0F0Fu);
        }
      }
    }
  }
  __syncthreads();
  const int d16 = threadIdx.x % LPR, jr = threadIdx.x / LPR;
  const int64_t row_of_slot0 = (int64_t)jb.s.row0 + (int64_t)jb.block * kBlock - (jb.s.len - jb.s.n);
  const int hoff = jb.head * D + 16 * d16;
  for (int base = jb.j0 & ~3; base < jb.j1; base += RPP) {
    const int j = base + jr;
    if (j < jb.j0 || j >= jb.j1) continue;
    uint32_t kc[4] = {}, vc[4] = {};
    float kscale = 0.f, vscale = 0.f;
    if (lv > 0) {
      const int o = key_off(D, j, d16);
      const uint2 hi = __ldg(reinterpret_cast<const uint2*>(khi + o));
      uint2 lo = make_uint2(0, 0);
      if (lv == 4) lo = __ldg(reinterpret_cast<const uint2*>(klo + o));
      uint32_t h0, h1, l0, l1;
      unpack8(hi.x, h0, h1);
      unpack8(lo.x, l0, l1);
      kc[0] = (h0 << 4) | l0;
      kc[1] = (h1 << 4) | l1;
      unpack8(hi.y, h0, h1);
      unpack8(lo.y, l0, l1);
      kc[2] = (h0 << 4) | l0;
      kc[3] = (h1 << 4) | l1;
      const uint4 q = *reinterpret_cast<const uint4*>(codes + j * P + 16 * d16);
      vc[0] = q.x;
      vc[1] = q.y;
      vc[2] = q.z;
      vc[3] = q.w;
      kscale = __ldg(reinterpret_cast<const float*>(rec) + j);
      vscale = __ldg(reinterpret_cast<const float*>(rec) + kBlock + j);
    }
    // a ZERO block's scale is 0 here, so its values are (minus) zero times a code: made +0
    store16(k + (row_of_slot0 + j) * ks + hoff, kc, kscale, lv > 0 ? off : 0.f);
    store16(v + (row_of_slot0 + j) * vs + hoff, vc, vscale, lv > 0 ? off : 0.f);
  }
}

fl_status check_batch(const char* what, const fl_kv_cache* c, const fl_kv_batch* b) {
  if (!c || !b) return fail(FL_ERR_ARG, "%s: NULL cache or batch", what);
  if (!c->pages || !b->block_table || !b->lens) return fail(FL_ERR_ARG, "%s: NULL pointer in cache or batch", what);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(FL_ERR_SHAPE, "%s: head_dim=%d (64 or 128)", what, c->head_dim);
  if (c->kv_heads < 1 || c->kv_heads > 256) return fail(FL_ERR_SHAPE, "%s: kv_heads=%d (1..256)", what, c->kv_heads);
  if (c->num_pages < 1) return fail(FL_ERR_SHAPE, "%s: num_pages=%d", what, c->num_pages);
  if (b->n_seqs < 1 || b->n_seqs > FL_KV_MAX_SEQS)
    return fail(FL_ERR_SHAPE, "%s: n_seqs=%d (1..%d)", what, b->n_seqs, FL_KV_MAX_SEQS);
  if (b->max_blocks < 1 || b->max_blocks > (1 << 23))
    return fail(FL_ERR_SHAPE, "%s: max_blocks=%d (1..2^23)", what, b->max_blocks);
  if (b->max_new < 1 || b->max_new > b->rows || b->max_new > (1 << 22))
    return fail(FL_ERR_SHAPE, "%s: max_new=%d, rows=%d (1 <= max_new <= rows, at most 2^22)", what, b->max_new,
                b->rows);
  if (!b->new_start && b->rows < b->n_seqs)
    return fail(FL_ERR_SHAPE, "%s: rows=%d below n_seqs=%d without new_start", what, b->rows, b->n_seqs);
  const uintptr_t bad = reinterpret_cast<uintptr_t>(b->block_table) | reinterpret_cast<uintptr_t>(b->lens) |
                        reinterpret_cast<uintptr_t>(b->new_start);
  if (bad & 3u) return fail(FL_ERR_ALIGN, "%s: block_table, lens and new_start must be 4-byte aligned", what);
  if (!aligned16(c->pages)) return fail(FL_ERR_ALIGN, "%s: pages must be 16-byte aligned", what);
  return FL_OK;
}

fl_status check_rows(const char* what, const char* name, const void* p, int64_t stride, int width) {
  if (!p) return fail(FL_ERR_ARG, "%s: NULL %s", what, name);
  if (stride < width || stride % 8 != 0 || stride > (1ll << 40))
    return fail(FL_ERR_SHAPE, "%s: %s row stride %lld (a multiple of 8, at least %d)", what, name, (long long)stride,
                width);
  if (!aligned16(p)) return fail(FL_ERR_ALIGN, "%s: %s must be 16-byte aligned", what, name);
  return FL_OK;
}

// Pages that n new tokens can touch at most.
static unsigned touched(int max_new, int max_blocks) {
  const long long t = ((long long)max_new + 2 * (kBlock - 1)) / kBlock;
  return (unsigned)(t < max_blocks ? t : max_blocks);
}

// Reads and clears the error word (-1 if that fails).
int take_device_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_error, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0 && cudaMemcpyToSymbol(g_error, &z, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

}  // namespace kv
}  // namespace fl

extern "C" size_t fl_kv_page_bytes(int kv_heads, int head_dim) {
  if ((head_dim != 64 && head_dim != 128) || kv_heads < 1 || kv_heads > 256) return 0;
  return (size_t)kv_heads * fl::kv::record_bytes(head_dim);
}

extern "C" fl_status fl_kv_append(const fl_kv_cache* cache, const fl_kv_batch* batch, const uint16_t* k,
                                  int64_t k_stride, const uint16_t* v, int64_t v_stride, void* stream) {
  using namespace fl;
  const char* what = "fl_kv_append";
  if (fl_status s = kv::check_batch(what, cache, batch)) return s;
  const int width = cache->kv_heads * cache->head_dim;
  if (fl_status s = kv::check_rows(what, "k", k, k_stride, width)) return s;
  if (fl_status s = kv::check_rows(what, "v", v, v_stride, width)) return s;
  const dim3 grid(kv::touched(batch->max_new, batch->max_blocks), (unsigned)batch->n_seqs, (unsigned)cache->kv_heads);
  auto kern = cache->head_dim == 64 ? kv::append_kernel<64> : kv::append_kernel<128>;
  FL_CHECK_CUDA(launch_pdl(kern, grid, dim3(kv::kThreads), 0, static_cast<cudaStream_t>(stream), 1, cache->pages,
                           cache->num_pages, cache->kv_heads, kv::batch_of(batch), k, k_stride, v, v_stride),
                "launch kv_append");
  return FL_OK;
}

extern "C" fl_status fl_kv_read(const fl_kv_cache* cache, const fl_kv_batch* batch, const uint8_t* levels, uint16_t* k,
                                int64_t k_stride, uint16_t* v, int64_t v_stride, void* stream) {
  using namespace fl;
  const char* what = "fl_kv_read";
  if (fl_status s = kv::check_batch(what, cache, batch)) return s;
  const int width = cache->kv_heads * cache->head_dim;
  if (fl_status s = kv::check_rows(what, "k", k, k_stride, width)) return s;
  if (fl_status s = kv::check_rows(what, "v", v, v_stride, width)) return s;
  const dim3 grid(kv::touched(batch->max_new, batch->max_blocks), (unsigned)batch->n_seqs, (unsigned)cache->kv_heads);
  auto kern = cache->head_dim == 64 ? kv::read_kernel<64> : kv::read_kernel<128>;
  FL_CHECK_CUDA(launch_pdl(kern, grid, dim3(kv::kThreads), 0, static_cast<cudaStream_t>(stream), 1, cache->pages,
                           cache->num_pages, cache->kv_heads, kv::batch_of(batch), levels, k, k_stride, v, v_stride),
                "launch kv_read");
  return FL_OK;
}
