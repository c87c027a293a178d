// Attention of a ragged batch's rows over the paged target cache, for tiles
// of up to 16 (query row, head of the group) pairs a kv head: single tokens
// and short blocks, where the cache's bytes are the cost.
//
//   out_r = sum_c softmax_c(scale * q_r . k_c) v_c  over the slots c row r sees
//
// in one pass over the keys: a running maximum m (log2 domain), sum l and
// output O in fp32, rescaled when the maximum moves. One tile of 16 rows is
// the M side of m16n8k16 MMAs; its G heads share every K/V byte.
//
// A CTA's warps take the units (kKeys slots) of the CTA's slice in turn, each
// through its own ring of cp.async stages, so no barrier stands inside the
// loop. The order of the dims inside a dot product and of the output columns
// over the MMA's n-tiles is free; it is chosen so that each lane's fragments
// are whole 16-byte pieces of the rows as they lie in the cache (K: dims of
// piece 4c + t of key g; V: the keys 2t, 2t+1, 2t+8, 2t+9 at piece g, pairs
// of keys joined by byte permutes) and 4-bit codes become fp16 pairs in
// registers, with no pass through shared memory in between. 4-bit values
// (e2m1 times e4m3) are exact in fp16; queries go to fp16 over a power of two
// a row, so they neither overflow nor lose more than fp32's own rounding of
// the largest element (2^-25 of it).
//
// Few rows and long caches: the slots of a stream are cut into slices of
// about equal length over all streams (find_item), a slice's (m, l, O) goes
// to the workspace and page_combine_kernel joins a row's slices.
#include <cuda_fp16.h>

#include "internal.h"
#include "pages.h"
#include "ptx.cuh"

namespace dfl {

namespace {

constexpr int kTileRows = 16;
constexpr int kWarps = 8;

template <int D, bool FP4>
struct Geo {
  static constexpr int kRow = FP4 ? D / 2 : 2 * D;  // bytes of a key's codes or values
  static constexpr int kSc = FP4 ? D / 16 : 0;      // scale bytes a key
  static constexpr int kKeys = FP4 ? 32 : 16;       // keys a unit
  static constexpr int kSub = kKeys / 16;
  static constexpr int kStages = 3;
  static constexpr int kOffV = kKeys * kRow;
  static constexpr int kOffKs = 2 * kKeys * kRow;
  static constexpr int kOffVs = kOffKs + kKeys * kSc;
  static constexpr int kStage = 2 * kKeys * (kRow + kSc);
  static constexpr int kPartLd = D + 4;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = kWarps * kTileRows * (kPartLd + 2) * 4;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  static constexpr float kShift = FP4 ? 8.f : 0.f;  // log2 of the factor P carries into fp16
};

// 16-byte piece of a row at which piece p of key `key` is kept, so that the
// fragment reads of K (pieces of one row over t) and V (one piece over the
// keys 2t) both meet every bank once.
template <int ROW>
__device__ __forceinline__ int swz(int key, int p) {
  if (ROW >= 128) return p ^ ((key & 6) ^ ((key & 1) << 2));
  if (ROW == 64) return p ^ ((key >> 1) & 3);
  return p;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool FP4>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (FP4)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight 4-bit codes (low nibble first) to four fp16 pairs.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two e4m3 scales (low byte first) to an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool half) {
  if (half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, bool FP4>
__global__ void __launch_bounds__(kWarps * 32, FP4 ? 2 : 1) page_attn_kernel(const __grid_constant__ PageAttnArgs a) {
  using G_ = Geo<D, FP4>;
  constexpr int kKeys = G_::kKeys, kRow = G_::kRow, kSub = G_::kSub, kNT = D / 8, kST = G_::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Item item_s;
  __shared__ int have_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    Item it;
    const bool have = find_item(a, static_cast<int>(blockIdx.x), false, &it);
    if (lane == 0) {
      item_s = it;
      have_s = have;
    }
  }
  __syncthreads();
  if (!have_s) return;
  const Item it = item_s;
  bool bad;
  const StreamRows q = stream_rows(a.r, it.s, &bad);

  // this thread's two rows, and what the tile's rows see
  RowView rv[2];
  int lo = 0x7fffffff, lo_max = -1, j_max = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t f = static_cast<int64_t>(it.tile) * kTileRows + g + 8 * i;
    const int j = static_cast<int>(f / a.G);
    rv[i].j = j < q.n ? j : -1;
    rv[i].pos = rv[i].j >= 0 ? row_pos(a.r, q, j) : 0;
    rv[i].back = a.window > 0 ? max(0, rv[i].pos - a.window + 1) : 0;
    if (rv[i].j >= 0) {
      lo = min(lo, rv[i].back);
      lo_max = max(lo_max, rv[i].back);
      j_max = max(j_max, j);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  lo_max = __reduce_max_sync(0xffffffffu, lo_max);
  j_max = __reduce_max_sync(0xffffffffu, j_max);
  const int hi = q.C + (a.mode == DFLASH_MASK_CAUSAL ? j_max + 1 : q.n);
  lo = min(lo, q.C);
  const int sinks = min(a.sinks, hi);
  const UnitRange ur = unit_range(lo, hi, a.sinks, kKeys);
  const int i0 = static_cast<int>(static_cast<long long>(ur.n) * it.split / it.ns);
  const int i1 = static_cast<int>(static_cast<long long>(ur.n) * (it.split + 1) / it.ns);

  // queries as A fragments, in the order of dims that K's pieces give
  uint32_t qa[D / 16][4];
  float sc[2] = {a.scale, a.scale};
  {
    const __nv_bfloat16* qp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t f = static_cast<int64_t>(it.tile) * kTileRows + g + 8 * i;
      const int hd = static_cast<int>(f % a.G);
      qp[i] = rv[i].j >= 0 ? a.q + static_cast<int64_t>(q.row0 + rv[i].j) * a.q_ld + (h * a.G + hd) * D : nullptr;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      constexpr int kPieces = D / 32;  // 16-byte pieces of a row a lane holds
      uint4 w[kPieces];
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const int piece = FP4 ? t * kPieces + c : 4 * c + t;
        w[c] = qp[i] ? *reinterpret_cast<const uint4*>(qp[i] + piece * 8) : make_uint4(0u, 0u, 0u, 0u);
      }
      if (FP4) {
        // over a power of two a row, into fp16
        float v[D / 4];
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[c * 8 + 2 * e] = __uint_as_float(u[e] << 16);
            v[c * 8 + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
          }
        }
#pragma unroll
        for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(v[e]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (top > 0.f && top < INFINITY) ? max(-100, min(126, ilogbf(top))) : 0;
        const float down = ldexpf(1.f, -ex);
        sc[i] *= ldexpf(1.f, ex);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          qa[s][i] = pack2(v[4 * s] * down, v[4 * s + 1] * down, true);
          qa[s][2 + i] = pack2(v[4 * s + 2] * down, v[4 * s + 3] * down, true);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          qa[2 * c][i] = w[c].x;
          qa[2 * c][2 + i] = w[c].y;
          qa[2 * c + 1][i] = w[c].z;
          qa[2 * c + 1][2 + i] = w[c].w;
        }
      }
    }
  }

  float o[kNT][4];
#pragma unroll
  for (int e = 0; e < kNT; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  uint8_t* ring = smem + warp * kST * G_::kStage;
  const uint32_t ring_u = smem_u32(ring);
  const int* table = a.c.table + static_cast<int64_t>(it.s) * a.c.cols;
  auto unit_at = [&](int i) { return i < ur.nsink ? i : ur.first + (i - ur.nsink); };
  int pg[kSub];
  auto fetch_pages = [&](int i) {
#pragma unroll
    for (int b = 0; b < kSub; ++b) {
      pg[b] = -1;
      if (i >= i1) continue;
      const int slot = unit_at(i) * kKeys + 16 * b;
      const bool need = (slot < hi && slot + 16 > lo) || slot < sinks;
      if (!need) continue;
      const int col = slot >> a.c.page_log2;
      const int p = col < a.c.cols ? table[col] : -1;
      if (p >= 0 && p < a.c.n_pages) pg[b] = p;
      else flag_status(a.r.status, DFLASH_STATUS_BAD_PAGE);
    }
  };
  uint32_t pres = 0;  // of the units in flight, newest in the low bits: which 16-slot pieces are there
  auto issue = [&](int i, int stage) {
    pres <<= kSub;
    if (i < i1) {
      const int kb = unit_at(i) * kKeys;
#pragma unroll
      for (int b = 0; b < kSub; ++b) {
        if (pg[b] < 0) continue;
        pres |= 1u << b;
        const int64_t row = (static_cast<int64_t>(pg[b]) * a.c.nkv + h) * a.c.page + ((kb + 16 * b) & (a.c.page - 1));
        const uint8_t* ks = a.c.k + row * kRow;
        const uint8_t* vs = a.c.v + row * kRow;
        const uint32_t d0 = ring_u + stage * G_::kStage + b * 16 * kRow;
#pragma unroll
        for (int p0 = 0; p0 < kRow; p0 += 32) {
          const int p = p0 + lane;
          if (kRow >= 32 || p < kRow) {
            constexpr int kPer = kRow / 16;
            const int key = p / kPer, piece = p % kPer;
            const uint32_t off = key * kRow + swz<kRow>(key, piece) * 16;
            cp16(d0 + off, ks + p * 16);
            cp16(d0 + G_::kOffV + off, vs + p * 16);
          }
        }
        if (FP4) {
          const uint32_t s0 = ring_u + stage * G_::kStage + b * 16 * G_::kSc;
          if (lane < G_::kSc) cp16(s0 + G_::kOffKs + lane * 16, a.c.ks + row * G_::kSc + lane * 16);
          else if (lane >= 16 && lane < 16 + G_::kSc)
            cp16(s0 + G_::kOffVs + (lane - 16) * 16, a.c.vs + row * G_::kSc + (lane - 16) * 16);
        }
      }
    }
    cp_commit();
  };

  // the stages ahead of the first unit; pages of the next one are looked up
  // while a unit's copies are issued
  fetch_pages(i0 + warp);
#pragma unroll
  for (int s = 0; s < kST - 1; ++s) {
    issue(i0 + warp + s * kWarps, s);
    fetch_pages(i0 + warp + (s + 1) * kWarps);
  }
  int stage = 0;
  for (int i = i0 + warp; i < i1; i += kWarps) {
    {
      const int ns = stage + kST - 1 >= kST ? stage - 1 : stage + kST - 1;
      issue(i + (kST - 1) * kWarps, ns);
      fetch_pages(i + kST * kWarps);
    }
    cp_wait<kST - 1>();
    __syncwarp();
    const uint8_t* sp = ring + stage * G_::kStage;
    const int kb = unit_at(i) * kKeys;
    const uint32_t here = (pres >> ((kST - 1) * kSub)) & ((1u << kSub) - 1u);
    const bool whole = here == (1u << kSub) - 1u && kb + kKeys <= q.C && (kb >= lo_max || kb + kKeys <= sinks);

    // ------------------------------------------------ scores
    float s[kKeys / 8][4];
#pragma unroll
    for (int nt = 0; nt < kKeys / 8; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      const int key = nt * 8 + g;
      if (!FP4) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(sp + key * kRow + swz<kRow>(key, 4 * c + t) * 16);
          mma16816<FP4>(s[nt], qa[2 * c], w.x, w.y);
          mma16816<FP4>(s[nt], qa[2 * c + 1], w.z, w.w);
        }
      } else {
        constexpr int kW = D / 32;  // words a lane holds of a key
        uint32_t w[kW];
        const uint8_t* src = sp + key * kRow + (D == 128 ? swz<kRow>(key, t) * 16 : t * (D / 8));
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(src);
          w[0] = x.x;
          w[1 % kW] = x.y;
          w[2 % kW] = x.z;
          w[3 % kW] = x.w;
        } else if (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          w[0] = x.x;
          w[1 % kW] = x.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(src);
        }
        const uint8_t* scp = sp + G_::kOffKs + key * G_::kSc;
        uint32_t two;  // the lane's one or two group scales
        if (D == 128) two = *reinterpret_cast<const uint16_t*>(scp + 2 * t);
        else two = scp[D == 64 ? t : t >> 1] * 0x101u;
        const uint32_t sp2 = e4m3x2(two);
        const uint32_t g0 = __byte_perm(sp2, 0, 0x1010), g1 = __byte_perm(sp2, 0, 0x3232);
#pragma unroll
        for (int x = 0; x < kW; ++x) {
          uint32_t f[4];
          e2m1x8(w[x], f);
          const uint32_t gs = (D == 128 && x >= 2) ? g1 : g0;
          mma16816<FP4>(s[nt], qa[2 * x], hmul2(f[0], gs), hmul2(f[1], gs));
          mma16816<FP4>(s[nt], qa[2 * x + 1], hmul2(f[2], gs), hmul2(f[3], gs));
        }
      }
    }
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < kKeys / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool there = (here >> (nt >> 1)) & 1u;
          if (!there || !sees(a, q, rv[e >> 1], kb + nt * 8 + 2 * t + (e & 1))) s[nt][e] = -INFINITY;
        }
    }

    // ------------------------------------------------ running maximum and sum
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < kKeys / 8; ++nt) {
      mx[0] = fmaxf(mx[0], fmaxf(s[nt][0], s[nt][1]));
      mx[1] = fmaxf(mx[1], fmaxf(s[nt][2], s[nt][3]));
    }
    bool moved = false;
    float al[2], sub[2];
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
      mx[i2] = fmaxf(mx[i2], __shfl_xor_sync(0xffffffffu, mx[i2], 1));
      mx[i2] = fmaxf(mx[i2], __shfl_xor_sync(0xffffffffu, mx[i2], 2));
      const float mn = fmaxf(m[i2], mx[i2] * sc[i2]);
      al[i2] = m[i2] == mn ? 1.f : ex2f(m[i2] - mn);
      moved |= m[i2] != mn;
      m[i2] = mn;
      sub[i2] = mn == -INFINITY ? 0.f : mn - G_::kShift;
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int e = 0; e < kNT; ++e) {
        o[e][0] *= al[0];
        o[e][1] *= al[0];
        o[e][2] *= al[1];
        o[e][3] *= al[1];
      }
      l[0] *= al[0];
      l[1] *= al[1];
    }
    uint32_t pa[kSub][4];
#pragma unroll
    for (int nt = 0; nt < kKeys / 8; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = ex2f(fmaf(s[nt][e], sc[e >> 1], -sub[e >> 1]));
      l[0] += s[nt][0] + s[nt][1];
      l[1] += s[nt][2] + s[nt][3];
      // P to 16 bits for the matrix product (the sum keeps fp32 P): bf16, or
      // fp16 beside 4-bit values
      pa[nt >> 1][(nt & 1) * 2] = pack2(s[nt][0], s[nt][1], FP4);
      pa[nt >> 1][(nt & 1) * 2 + 1] = pack2(s[nt][2], s[nt][3], FP4);
    }

    // ------------------------------------------------ output
#pragma unroll
    for (int b = 0; b < kSub; ++b) {
      // slots that no row of the tile sees may hold anything: their V counts as zero
      uint32_t live[2] = {0xffffffffu, 0xffffffffu};  // of the key pairs (2t, 2t+1) and (2t+8, 2t+9), 16 bits a key
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int slot = kb + 16 * b + 2 * t + (x & 1) + (x >> 1) * 8;
          const bool ok = ((here >> b) & 1u) && ((slot >= lo && slot < hi) || slot < sinks);
          if (!ok) live[x >> 1] &= (x & 1) ? 0x0000ffffu : 0xffff0000u;
        }
      }
      const uint8_t* vp = sp + G_::kOffV + b * 16 * kRow;
      if (!FP4) {
        constexpr int kC = D >= 64 ? D / 64 : 1;
        constexpr int kWords = D >= 64 ? 4 : 2;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          uint32_t w[4][kWords];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = 2 * t + (x & 1) + (x >> 1) * 8;
            if (D >= 64) {
              const uint4 u = *reinterpret_cast<const uint4*>(vp + key * kRow + swz<kRow>(key, 8 * c + g) * 16);
              w[x][0] = u.x;
              w[x][1] = u.y;
              w[x][2 % kWords] = u.z;
              w[x][3 % kWords] = u.w;
            } else {
              const uint2 u =
                  *reinterpret_cast<const uint2*>(vp + key * kRow + swz<kRow>(key, g >> 1) * 16 + (g & 1) * 8);
              w[x][0] = u.x;
              w[x][1] = u.y;
            }
          }
#pragma unroll
          for (int e = 0; e < 2 * kWords; ++e) {
            const unsigned sel = (e & 1) ? 0x7632u : 0x5410u;
            const uint32_t b0 = __byte_perm(w[0][e >> 1], w[1][e >> 1], sel) & live[0];
            const uint32_t b1 = __byte_perm(w[2][e >> 1], w[3][e >> 1], sel) & live[1];
            mma16816<FP4>(o[c * 8 + e], pa[b], b0, b1);
          }
        }
      } else {
        constexpr int kB = D / 16;  // bytes a lane holds of a key: dims (D/8) g ..
        uint32_t w[4][(kB + 3) / 4];
        uint32_t vsc[2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 2 * t + (x & 1) + (x >> 1) * 8;
          if (D == 128) {
            const uint2 u =
                *reinterpret_cast<const uint2*>(vp + key * kRow + swz<kRow>(key, g >> 1) * 16 + (g & 1) * 8);
            w[x][0] = u.x;
            w[x][1 % ((kB + 3) / 4)] = u.y;
          } else if (D == 64) {
            w[x][0] = *reinterpret_cast<const uint32_t*>(vp + key * kRow + g * 4);
          } else {
            w[x][0] = *reinterpret_cast<const uint16_t*>(vp + key * kRow + g * 2);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t* vscp = sp + G_::kOffVs + (b * 16 + 2 * t + 8 * x) * G_::kSc + (g * (D / 8)) / 16;
          vsc[x] = e4m3x2(vscp[0] | (static_cast<uint32_t>(vscp[G_::kSc]) << 8)) & live[x];
        }
#pragma unroll
        for (int x = 0; x < (kB + 3) / 4; ++x) {
          uint32_t f[4][4];
#pragma unroll
          for (int k2 = 0; k2 < 4; ++k2) e2m1x8(w[k2][x], f[k2]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (x * 8 + e >= kNT) continue;
            const unsigned sel = (e & 1) ? 0x7632u : 0x5410u;
            const uint32_t b0 = hmul2(__byte_perm(f[0][e >> 1], f[1][e >> 1], sel), vsc[0]);
            const uint32_t b1 = hmul2(__byte_perm(f[2][e >> 1], f[3][e >> 1], sel), vsc[1]);
            mma16816<FP4>(o[x * 8 + e], pa[b], b0, b1);
          }
        }
      }
    }
    __syncwarp();  // the stage may be written again
    stage = stage + 1 == kST ? 0 : stage + 1;
  }
  cp_wait<0>();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }
  __syncthreads();

  // ---------------------------------------------------- join the warps' parts
  float* po = reinterpret_cast<float*>(smem);
  float* pml = po + kWarps * kTileRows * G_::kPartLd;
  // n-tile e of output half c, column 2t + x of the tile: the dim it holds
  constexpr int kPer = (!FP4 && D == 128) ? 8 : kNT;  // n-tiles of consecutive dims
#pragma unroll
  for (int e = 0; e < kNT; ++e) {
    const int c = e / kPer, r = e % kPer;
    const int d0 = c * 64 + kPer * 2 * t + r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* row = po + (warp * kTileRows + g + 8 * i) * G_::kPartLd;
      row[d0] = o[e][2 * i];
      row[d0 + kPer] = o[e][2 * i + 1];
    }
  }
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      pml[(warp * kTileRows + g + 8 * i) * 2] = m[i];
      pml[(warp * kTileRows + g + 8 * i) * 2 + 1] = l[i];
    }
  }
  __syncthreads();
  const bool keep = it.ns > 1 && it.slot < a.slots;
  for (int x = threadIdx.x; x < kTileRows * (D / 4); x += kWarps * 32) {
    const int r = x / (D / 4), d4 = (x % (D / 4)) * 4;
    const int64_t f = static_cast<int64_t>(it.tile) * kTileRows + r;
    const int j = static_cast<int>(f / a.G);
    if (j >= q.n) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, pml[(w * kTileRows + r) * 2]);
    float den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float wt = ex2f(pml[(w * kTileRows + r) * 2] - M);
        const float4 v = *reinterpret_cast<const float4*>(po + (w * kTileRows + r) * G_::kPartLd + d4);
        den = fmaf(wt, pml[(w * kTileRows + r) * 2 + 1], den);
        acc.x = fmaf(wt, v.x, acc.x);
        acc.y = fmaf(wt, v.y, acc.y);
        acc.z = fmaf(wt, v.z, acc.z);
        acc.w = fmaf(wt, v.w, acc.w);
      }
    }
    if (it.ns > 1) {
      if (!keep) continue;
      const int64_t row = (static_cast<int64_t>(it.slot) * a.c.nkv + h) * kTileRows + r;
      *reinterpret_cast<float4*>(a.part_o + row * D + d4) = acc;
      if (d4 == 0) *reinterpret_cast<float2*>(a.part_ml + row * 2) = make_float2(M, den);
    } else {
      const int hd = static_cast<int>(f - static_cast<int64_t>(j) * a.G);
      const float inv = M == -INFINITY ? 0.f : 1.f / den;
      uint2 w;
      w.x = pack2(acc.x * inv, acc.y * inv, false);
      w.y = pack2(acc.z * inv, acc.w * inv, false);
      *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(q.row0 + j) * a.out_ld + (h * a.G + hd) * D + d4) = w;
    }
  }
}

// Joins the slices of a row: one warp a row of a split tile.
constexpr int kCombineRows = 4;
template <int D>
__global__ void __launch_bounds__(kCombineRows * 32) page_combine_kernel(const __grid_constant__ PageAttnArgs a) {
  constexpr int kE = D / 32;
  __shared__ Item item_s;
  __shared__ int have_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // row_start and lens were complete before the attention kernel let this one start
  if (warp == 0) {
    Item it;
    const bool have = find_item(a, static_cast<int>(blockIdx.x), true, &it);
    if (lane == 0) {
      item_s = it;
      have_s = have;
    }
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (!have_s) return;
  const Item it = item_s;
  const int h = blockIdx.y, r = blockIdx.z * kCombineRows + warp;
  bool bad;
  const StreamRows q = stream_rows(a.r, it.s, &bad);
  const int64_t f = static_cast<int64_t>(it.tile) * a.tile + r;
  const int j = static_cast<int>(f / a.G);
  if (r >= a.tile || j >= q.n || it.slot + it.ns > a.slots) return;
  const int64_t row0 = (static_cast<int64_t>(it.slot) * a.c.nkv + h) * a.tile + r;
  const int64_t step = static_cast<int64_t>(a.c.nkv) * a.tile;
  float M = -INFINITY;
  for (int k = lane; k < it.ns; k += 32) M = fmaxf(M, a.part_ml[(row0 + k * step) * 2]);
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float acc[kE] = {};
  float den = 0.f;
  if (M != -INFINITY) {
#pragma unroll 8
    for (int k = 0; k < it.ns; ++k) {
      const int64_t row = row0 + k * step;
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + row * 2);
      const float w = ex2f(ml.x - M);
      den = fmaf(w, ml.y, den);
      const float* src = a.part_o + row * D + lane * kE;
      float v[kE];
      if (kE == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
      else if (kE == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
      else v[0] = *src;
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] = fmaf(w, v[e], acc[e]);
    }
  }
  const float inv = M == -INFINITY ? 0.f : 1.f / den;
  const int hd = static_cast<int>(f - static_cast<int64_t>(j) * a.G);
  __nv_bfloat16* dst = a.out + static_cast<int64_t>(q.row0 + j) * a.out_ld + (h * a.G + hd) * D + lane * kE;
  if (kE == 4) {
    uint2 w;
    w.x = pack2(acc[0] * inv, acc[1 % kE] * inv, false);
    w.y = pack2(acc[2 % kE] * inv, acc[3 % kE] * inv, false);
    *reinterpret_cast<uint2*>(dst) = w;
  } else if (kE == 2) {
    *reinterpret_cast<uint32_t*>(dst) = pack2(acc[0] * inv, acc[1 % kE] * inv, false);
  } else {
    *dst = __float2bfloat16_rn(acc[0] * inv);
  }
}

template <int D, bool FP4>
int launch_small(const PageAttnArgs& a, const PagePlan& p, cudaStream_t st) {
  using G_ = Geo<D, FP4>;
  auto kern = page_attn_kernel<D, FP4>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G_::kSmem) != cudaSuccess) {
    cudaGetLastError();
    return DFLASH_E_CUDA;
  }
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(p.items), static_cast<unsigned>(a.c.nkv)),
                                   dim3(kWarps * 32), G_::kSmem, st, a);
  count_launch();
  return cuda_status(e);
}

template <int D>
int launch_combine(const PageAttnArgs& a, const PagePlan& p, cudaStream_t st) {
  const cudaError_t e = launch_pdl(page_combine_kernel<D>,
                                   dim3(static_cast<unsigned>(p.split_tiles), static_cast<unsigned>(a.c.nkv),
                                        static_cast<unsigned>((a.tile + kCombineRows - 1) / kCombineRows)),
                                   dim3(kCombineRows * 32), 0, st, a);
  count_launch();
  return cuda_status(e);
}

}  // namespace

PagePlan page_attention_plan(const dflash_pages& c, const dflash_rows& r, int nq) {
  const int G = nq / c.n_kv_heads;
  const bool fp4 = c.format == DFLASH_PAGES_FP4;
  PagePlan p{};
  const int64_t R = static_cast<int64_t>(r.max_rows) * G;
  p.tc = c.head_dim >= 64 && R > kTileRows;
  if (p.tc) {
    p.tile = R > 512 ? 256 : 128;
    p.unit = 128;
    p.target = 152;
    p.min_units = 4;
  } else {
    p.tile = kTileRows;
    p.unit = fp4 ? 32 : 16;
    p.target = 152 * (fp4 ? 2 : 1);
    p.min_units = 2 * kWarps;
  }
  const int64_t per_stream = (static_cast<int64_t>(r.max_rows) * G + p.tile - 1) / p.tile;
  const int64_t by_rows = (static_cast<int64_t>(r.rows) * G + p.tile - 1) / p.tile + c.streams;
  const int64_t tiles = std::min(c.streams * per_stream, by_rows);
  // a stream is split only when its units pass total / target, so all its
  // slices are under twice the target; slices of at most the whole table
  const int64_t cap_units = (static_cast<int64_t>(c.table_cols) * c.page_size + p.unit - 1) / p.unit + 1;
  const bool may_split = cap_units > p.min_units;
  const int64_t per_head = (p.target + c.n_kv_heads - 1) / c.n_kv_heads;
  p.items = tiles + (may_split ? per_head : 0);
  p.slots = may_split ? static_cast<int>(2 * per_head + 1) : 0;
  p.split_tiles = may_split ? std::min(tiles, per_head) : 0;
  return p;
}

int launch_page_attention(const PageAttnArgs& a, const PagePlan& p, bool fp4, cudaStream_t st) {
  const int D = a.c.d;
  int rc;
  {
    TraceScope ts(st, "page_attention", 0.0, 0.0);
    if (p.tc) rc = launch_page_attention_tc(a, p, fp4, st);
    else if (D == 128) rc = fp4 ? launch_small<128, true>(a, p, st) : launch_small<128, false>(a, p, st);
    else if (D == 64) rc = fp4 ? launch_small<64, true>(a, p, st) : launch_small<64, false>(a, p, st);
    else rc = fp4 ? launch_small<32, true>(a, p, st) : launch_small<32, false>(a, p, st);
  }
  if (rc || p.split_tiles == 0) return rc;
  TraceScope ts(st, "page_combine", 0.0, 0.0);
  return D == 128 ? launch_combine<128>(a, p, st) : D == 64 ? launch_combine<64>(a, p, st) : launch_combine<32>(a, p, st);
}

}  // namespace dfl
