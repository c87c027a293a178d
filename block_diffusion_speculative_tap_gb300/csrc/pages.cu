// Rows in and out of the paged target cache.
//
// page_append_kernel: one CTA a row of the batch. The row's K heads (and the
// caller's Q heads) are rotated by the row's position, rotate-half:
//   y_i = x_i cos_i - x_{i+d/2} sin_i,   y_{i+d/2} = x_{i+d/2} cos_i + x_i sin_i
// each product and the sum rounded to fp32, then to bf16, and K and V go to
// the row's slot of its stream's pages: as bf16, or as 4-bit codes with one
// scale a group of 16 dims,
//   s = e4m3(max|y| / 6),  code_i = e2m1(y_i / s)   (both to nearest, ties to
// even; the quantised value is the bf16 one). A thread takes 16 dims of the
// lower half and the 16 they pair with, two whole groups, so neither the
// rotation nor a group's maximum leaves it. Bound by the rows' bytes: each is
// read and written once. The row's stream is found by one load a lane over
// row_start, and the values are loaded before anything depends on it.
//
// page_read_kernel: the rows' values back, as bf16 (a 4-bit value times its
// e4m3 scale has at most six significant bits: exact in bf16).
#include <cuda_fp16.h>

#include "internal.h"
#include "pages.h"
#include "ptx.cuh"

namespace dfl {

namespace {

constexpr int kAppendThreads = 128;

// The stream that holds row `t` (row_start[s] <= t < row_start[s + 1]): the
// number of streams that end at or before t. One warp; S when there is none.
__device__ __forceinline__ int find_stream(const RowsArgs& r, int t) {
  const int lane = threadIdx.x & 31;
  for (int s0 = 0; s0 < r.S; s0 += 32) {
    const bool past = s0 + lane >= r.S || r.row_start[s0 + lane + 1] > t;
    const unsigned hit = __ballot_sync(0xffffffffu, past);
    if (hit) return min(r.S, s0 + __ffs(hit) - 1);
  }
  return r.S;
}

struct Place {
  int pos;      // -1: no such row, leave everything as it is
  int64_t row;  // (page * nkv) * page_size + slot of kv head 0, -1: no slot
};

__device__ __forceinline__ Place find_place(const PagesArgs& c, const RowsArgs& r, int t) {
  Place p{-1, -1};
  const int s = find_stream(r, t);
  if (s >= r.S) return p;
  bool bad;
  const StreamRows q = stream_rows(r, s, &bad);
  const int j = t - q.row0;
  if (bad) flag_status(r.status, DFLASH_STATUS_BAD_ROWS);
  if (j < 0 || j >= q.n) return p;
  p.pos = q.C + j;
  if (r.depth) {
    const int d = r.depth[t];
    if (d < 0 || d > 0x3fffffff) {
      flag_status(r.status, DFLASH_STATUS_BAD_ROWS);
      p.pos = -1;
      return p;
    }
    p.pos = q.C + d;
  }
  const int slot = q.C + j, col = slot >> c.page_log2;
  const int pg = col < c.cols ? c.table[static_cast<int64_t>(s) * c.cols + col] : -1;
  if (pg >= 0 && pg < c.n_pages)
    p.row = static_cast<int64_t>(pg) * c.nkv * c.page + (slot & (c.page - 1));
  else
    flag_status(r.status, DFLASH_STATUS_BAD_PAGE);
  return p;
}

struct Bf16x16 {
  uint4 a, b;
};
__device__ __forceinline__ Bf16x16 load16(const __nv_bfloat16* p) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  return Bf16x16{q[0], q[1]};
}
__device__ __forceinline__ void unpack16(const Bf16x16& x, float (&v)[16]) {
  const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ Bf16x16 pack16(const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return Bf16x16{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const Bf16x16& x) {
  uint4* q = reinterpret_cast<uint4*>(p);
  q[0] = x.a;
  q[1] = x.b;
}

// A group of 16 bf16 values to its e4m3 scale and 16 codes (low nibble first).
__device__ __forceinline__ uint2 quantise16(const Bf16x16& x, uint8_t* scale) {
  float v[16];
  unpack16(x, v);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(v[i]));
  const float want = fminf(__fdiv_rn(top, 6.f), 448.f);
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(want));
  uint32_t sh;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sh) : "h"(s2));
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sh & 0xffffu)));
  *scale = static_cast<uint8_t>(s2 & 0xffu);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = v[8 * i + 2 * e], hi = v[8 * i + 2 * e + 1];
      // an exact division: a value midway between two codes stays midway.
      // A group whose scale is zero keeps its signs and no values.
      const float qa = s > 0.f ? __fdiv_rn(lo, s) : copysignf(0.f, lo);
      const float qb = s > 0.f ? __fdiv_rn(hi, s) : copysignf(0.f, hi);
      asm("{\n\t.reg .b8 b;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
          "mov.b32 %0, {b, 0, 0, 0};\n\t}"
          : "=r"(c[e])
          : "f"(qb), "f"(qa));
    }
    w[i] = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
  }
  return make_uint2(w[0], w[1]);
}

// 16 codes and their scale to bf16.
__device__ __forceinline__ Bf16x16 values16(uint2 codes, uint8_t scale) {
  uint32_t sh;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sh) : "h"(static_cast<uint16_t>(scale)));
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sh & 0xffffu)));
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t c = ((i < 8 ? codes.x : codes.y) >> (4 * (i & 7))) & 15u;
    // e2m1 as fp32: 0, 0.5, 1, 1.5, 2, 3, 4, 6
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float mag = e == 0u ? 0.5f * m : __uint_as_float(((e + 126u) << 23) | (m << 22));
    v[i] = (c & 8u) ? -mag * s : mag * s;
  }
  return pack16(v);
}

struct AppendArgs {
  PagesArgs c;
  RowsArgs r;
  const __nv_bfloat16 *k, *v, *q;
  __nv_bfloat16* q_out;
  int64_t k_ld, v_ld, q_ld, q_out_ld;
  const float2* rope;  // [rope_rows][d / 2], null: no rotation
  int rope_rows, nq;
};

template <bool FP4>
__device__ __forceinline__ void store_group(const AppendArgs& a, uint8_t* base, uint8_t* scales, int64_t row, int dim,
                                            const Bf16x16& x) {
  const int d = a.c.d;
  if (FP4) {
    uint8_t s;
    const uint2 w = quantise16(x, &s);
    *reinterpret_cast<uint2*>(base + row * (d / 2) + dim / 2) = w;
    scales[row * (d / 16) + dim / 16] = s;
  } else {
    store16(reinterpret_cast<__nv_bfloat16*>(base) + row * d + dim, x);
  }
}

template <bool FP4>
__global__ void __launch_bounds__(kAppendThreads) page_append_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  const int d = a.c.d, half = d / 2, parts = d / 32;
  const int units = (a.nq + 2 * a.c.nkv) * parts;
  Place place{};
  bool placed = false;
  for (int u0 = 0; u0 < units; u0 += kAppendThreads) {
    const int u = u0 + static_cast<int>(threadIdx.x);
    const int part = u % parts;
    int hd = u / parts;
    // queries, then K heads, then V heads
    const int kind = hd < a.nq ? 0 : hd < a.nq + a.c.nkv ? 1 : 2;
    hd -= kind == 0 ? 0 : kind == 1 ? a.nq : a.nq + a.c.nkv;
    const int d0 = kind == 2 ? part * 32 : part * 16, d1 = kind == 2 ? d0 + 16 : half + d0;
    const bool on = u < units;
    Bf16x16 x0{}, x1{};
    if (on) {
      const __nv_bfloat16* src = (kind == 0   ? a.q + static_cast<int64_t>(t) * a.q_ld
                                  : kind == 1 ? a.k + static_cast<int64_t>(t) * a.k_ld
                                              : a.v + static_cast<int64_t>(t) * a.v_ld) +
                                 static_cast<int64_t>(hd) * d;
      x0 = load16(src + d0);
      x1 = load16(src + d1);
    }
    if (!placed) {
      place = find_place(a.c, a.r, t);
      placed = true;
      if (place.pos >= 0 && a.rope && place.pos >= a.rope_rows) {
        flag_status(a.r.status, DFLASH_STATUS_BAD_ROWS);
        place.pos = -1;
      }
      if (place.pos < 0) return;  // the whole CTA: one row
    }
    if (!on) continue;
    if (kind != 2 && a.rope) {
      const float4* cs = reinterpret_cast<const float4*>(a.rope + static_cast<int64_t>(place.pos) * half + d0);
      float lo[16], hi[16];
      unpack16(x0, lo);
      unpack16(x1, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 w = cs[i];  // (cos, sin) of two dims
        const float a0 = lo[2 * i], b0 = hi[2 * i], a1 = lo[2 * i + 1], b1 = hi[2 * i + 1];
        lo[2 * i] = __fsub_rn(__fmul_rn(a0, w.x), __fmul_rn(b0, w.y));
        hi[2 * i] = __fadd_rn(__fmul_rn(b0, w.x), __fmul_rn(a0, w.y));
        lo[2 * i + 1] = __fsub_rn(__fmul_rn(a1, w.z), __fmul_rn(b1, w.w));
        hi[2 * i + 1] = __fadd_rn(__fmul_rn(b1, w.z), __fmul_rn(a1, w.w));
      }
      x0 = pack16(lo);
      x1 = pack16(hi);
    }
    if (kind == 0) {
      __nv_bfloat16* dst = a.q_out + static_cast<int64_t>(t) * a.q_out_ld + static_cast<int64_t>(hd) * d;
      store16(dst + d0, x0);
      store16(dst + d1, x1);
    } else if (place.row >= 0) {
      const int64_t row = place.row + static_cast<int64_t>(hd) * a.c.page;
      uint8_t* base = kind == 1 ? a.c.k : a.c.v;
      uint8_t* scales = kind == 1 ? a.c.ks : a.c.vs;
      store_group<FP4>(a, base, scales, row, d0, x0);
      store_group<FP4>(a, base, scales, row, d1, x1);
    }
  }
}

struct ReadArgs {
  PagesArgs c;
  RowsArgs r;
  __nv_bfloat16 *k, *v;
  int64_t k_ld, v_ld;
};

template <bool FP4>
__global__ void __launch_bounds__(kAppendThreads) page_read_kernel(const ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  const Place place = find_place(a.c, a.r, t);
  if (place.pos < 0 || place.row < 0) return;
  const int d = a.c.d, groups = d / 16;
  const int units = 2 * a.c.nkv * groups;
  for (int u = threadIdx.x; u < units; u += kAppendThreads) {
    const int grp = u % groups, kv = (u / groups) / a.c.nkv, hd = (u / groups) % a.c.nkv;
    const int64_t row = place.row + static_cast<int64_t>(hd) * a.c.page;
    const uint8_t* base = kv ? a.c.v : a.c.k;
    Bf16x16 x;
    if (FP4) {
      const uint8_t* sc = kv ? a.c.vs : a.c.ks;
      x = values16(*reinterpret_cast<const uint2*>(base + row * (d / 2) + grp * 8), sc[row * groups + grp]);
    } else {
      x = load16(reinterpret_cast<const __nv_bfloat16*>(base) + row * d + grp * 16);
    }
    __nv_bfloat16* dst = (kv ? a.v + static_cast<int64_t>(t) * a.v_ld : a.k + static_cast<int64_t>(t) * a.k_ld) +
                         static_cast<int64_t>(hd) * d + grp * 16;
    store16(dst, x);
  }
}

}  // namespace

int launch_page_append(const PagesArgs& c, const RowsArgs& r, const __nv_bfloat16* k, int64_t k_ld,
                       const __nv_bfloat16* v, int64_t v_ld, const float2* rope, int rope_rows, const __nv_bfloat16* q,
                       int64_t q_ld, __nv_bfloat16* q_out, int64_t q_out_ld, int nq, bool fp4, cudaStream_t st) {
  AppendArgs a{c, r, k, v, q, q_out, k_ld, v_ld, q_ld, q_out_ld, rope, rope_rows, nq};
  const double row = 2.0 * (nq + 2.0 * c.nkv) * c.d + 2.0 * nq * c.d +
                     2.0 * c.nkv * (fp4 ? c.d / 2 + c.d / 16 : 2 * c.d) + (rope ? 4.0 * c.d : 0.0);
  TraceScope ts(st, "page_append", row * r.T, 0.0);
  const cudaError_t e = launch_pdl(fp4 ? page_append_kernel<true> : page_append_kernel<false>, dim3(r.T),
                                   dim3(kAppendThreads), 0, st, a);
  count_launch();
  return cuda_status(e);
}

int launch_page_read(const PagesArgs& c, const RowsArgs& r, __nv_bfloat16* k, int64_t k_ld, __nv_bfloat16* v,
                     int64_t v_ld, bool fp4, cudaStream_t st) {
  ReadArgs a{c, r, k, v, k_ld, v_ld};
  TraceScope ts(st, "page_read", 2.0 * c.nkv * r.T * (2.0 * c.d + (fp4 ? c.d / 2 + c.d / 16 : 2 * c.d)), 0.0);
  const cudaError_t e = launch_pdl(fp4 ? page_read_kernel<true> : page_read_kernel<false>, dim3(r.T),
                                   dim3(kAppendThreads), 0, st, a);
  count_launch();
  return cuda_status(e);
}

}  // namespace dfl
