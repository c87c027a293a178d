// The paged target cache and the ragged batch of rows that is appended to it
// and attends over it: what the kernels see of dflash_pages and dflash_rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash.h"

namespace dfl {

struct PagesArgs {
  uint8_t* k;        // [n_pages][nkv][page][row bytes]
  uint8_t* v;
  uint8_t* ks;       // 4-bit pages: [n_pages][nkv][page][d / 16] e4m3 scales
  uint8_t* vs;
  const int* table;  // [S][cols]
  int n_pages, page, page_log2, nkv, d, S, cols;
};

struct RowsArgs {
  const int* row_start;  // [S + 1]
  const int* lens;       // [S]
  const int* depth;      // [T] or null
  int T, max_rows, S;
  int cap;               // slots a stream's table reaches
  int* status;           // device status word, may be null
};

struct PageAttnArgs {
  PagesArgs c;
  RowsArgs r;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_ld, out_ld;
  const uint32_t* mask;  // tree mode: [T][mask_ld]
  int mask_ld, mode, window, sinks;
  int nq, G;
  float scale;           // softmax scale times log2(e)
  // work split: an item is one (stream, tile of rows, slice of the keys)
  int unit;              // slots a unit of the split
  int tile;              // rows (query row x head of the group) a tile
  int target;            // items over all kv heads the split aims at
  int min_units;         // fewest units an item is given
  int slots;             // partial slots a kv head in part_o
  float* part_o;         // [slots][nkv][tile][d]
  float* part_ml;        // [slots][nkv][tile][2]
};

__device__ __forceinline__ void flag_status(int* status, int bits) {
  if (status) atomicOr(status, bits);
}

// Rows of stream s, from data only the device sees: never past the buffers
// and never more than max_rows, whatever row_start and lens hold.
struct StreamRows {
  int row0, n, C;
};
__device__ __forceinline__ StreamRows stream_rows(const RowsArgs& r, int s, bool* bad) {
  StreamRows q;
  const int a = r.row_start[s], b = r.row_start[s + 1], c = r.lens[s];
  q.row0 = min(max(a, 0), r.T);
  q.n = min(min(max(b, q.row0), r.T) - q.row0, r.max_rows);
  q.C = min(max(c, 0), r.cap);
  *bad = a != q.row0 || b != q.row0 + q.n || c != q.C;
  return q;
}

// Slots that rows of a stream can see, in units of `unit` slots: the units
// [0, nsink) that hold sinks and the units [first, first + n - nsink).
struct UnitRange {
  int nsink, first, n;
};
__device__ __forceinline__ UnitRange unit_range(int lo, int hi, int sinks, int unit) {
  UnitRange u;
  const int end = (hi + unit - 1) / unit;
  u.first = min(lo / unit, end);
  u.nsink = lo > 0 ? min((min(sinks, hi) + unit - 1) / unit, u.first) : 0;
  u.n = u.nsink + end - u.first;
  return u;
}

// The split of a call's work, the same in every CTA of a call. A stream of n
// rows is mt tiles of `tile` (row, head) pairs; each tile's units are cut into
// ns slices, about total / target units each, so that streams of unequal
// length give slices of equal length.
struct Item {
  int s, tile, split, ns, slot;  // slot: partial slot (ns > 1)
};

// Find item `want` of a call (split_only: tile `want` among the tiles of the
// streams with ns > 1). One warp; every lane gets the answer. Returns false
// past the last one.
__device__ __forceinline__ bool find_item(const PageAttnArgs& a, int want, bool split_only, Item* out) {
  const int lane = threadIdx.x & 31;
  auto units_of = [&](int s, int* mt) -> int {
    bool bad;
    const StreamRows q = stream_rows(a.r, s, &bad);
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) flag_status(a.r.status, DFLASH_STATUS_BAD_ROWS);
    *mt = static_cast<int>((static_cast<int64_t>(q.n) * a.G + a.tile - 1) / a.tile);
    if (q.n == 0) return 0;
    const int lo = a.window > 0 ? max(0, q.C - a.window + 1) : 0;
    return unit_range(lo, q.C + q.n, a.sinks, a.unit).n;
  };
  // total units over the tiles of all streams
  long long total = 0;
  int mt0 = 0, u0 = 0;
  for (int s0 = 0; s0 < a.r.S; s0 += 32) {
    int mt = 0, u = 0;
    if (s0 + lane < a.r.S) u = units_of(s0 + lane, &mt);
    if (s0 == 0) {
      mt0 = mt;
      u0 = u;
    }
    total += static_cast<long long>(mt) * u;
  }
  for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const long long per = (total * a.c.nkv + a.target - 1) / a.target;
  const int upi = static_cast<int>(per > a.min_units ? (per < 0x7fffffffll ? per : 0x7fffffffll) : a.min_units);
  int base = 0, slots = 0;
  for (int s0 = 0; s0 < a.r.S; s0 += 32) {
    int mt = mt0, u = u0;
    if (s0 > 0) {
      mt = u = 0;
      if (s0 + lane < a.r.S) u = units_of(s0 + lane, &mt);
    }
    // a stream whose rows see no slot still has its output written
    const int ns = u > 0 ? static_cast<int>((static_cast<long long>(u) + upi - 1) / upi) : 1;
    const int cnt = split_only ? (ns > 1 ? mt : 0) : mt * ns;
    const int part = ns > 1 ? mt * ns : 0;
    int ic = cnt, ip = part;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, ic, o), y = __shfl_up_sync(0xffffffffu, ip, o);
      if (lane >= o) {
        ic += x;
        ip += y;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, want < base + ic);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int before = base + __shfl_sync(0xffffffffu, ic - cnt, l);
      const int nsl = __shfl_sync(0xffffffffu, ns, l);
      const int slot0 = slots + __shfl_sync(0xffffffffu, ip - part, l);
      const int rel = want - before, tiles = __shfl_sync(0xffffffffu, mt, l);
      const int tile = split_only ? rel : rel / nsl;
      out->s = s0 + l;
      out->ns = nsl;
      out->tile = tiles - 1 - tile;  // the last rows see most: their items start first
      out->split = split_only ? 0 : rel - tile * nsl;
      out->slot = slot0 + tile * nsl + out->split;
      return true;
    }
    base += __shfl_sync(0xffffffffu, ic, 31);
    slots += __shfl_sync(0xffffffffu, ip, 31);
  }
  return false;
}

// What one (query row, head) pair of a tile sees.
struct RowView {
  int j;       // row of its stream, -1: no row
  int pos;     // its position
  int back;    // first slot its window reaches (context part)
};

__device__ __forceinline__ int row_pos(const RowsArgs& r, const StreamRows& q, int j) {
  return q.C + (r.depth ? max(0, min(r.depth[q.row0 + j], 0x3fffffff)) : j);
}

// Whether row v sees slot `slot` of its stream.
__device__ __forceinline__ bool sees(const PageAttnArgs& a, const StreamRows& q, const RowView& v, int slot) {
  if (v.j < 0 || slot < 0) return false;
  if (slot < q.C) return slot >= v.back || slot < a.sinks;
  const int m = slot - q.C;
  if (m >= q.n) return false;
  if (a.mode == DFLASH_MASK_CAUSAL && m > v.j) return false;
  if (a.mode == DFLASH_MASK_TREE &&
      !((a.mask[static_cast<int64_t>(q.row0 + v.j) * a.mask_ld + (m >> 5)] >> (m & 31)) & 1u))
    return false;
  if (a.window == 0 || slot < a.sinks) return true;
  return v.pos - row_pos(a.r, q, m) < a.window;
}

int launch_page_append(const PagesArgs& c, const RowsArgs& r, const __nv_bfloat16* k, int64_t k_ld,
                       const __nv_bfloat16* v, int64_t v_ld, const float2* rope, int rope_rows, const __nv_bfloat16* q,
                       int64_t q_ld, __nv_bfloat16* q_out, int64_t q_out_ld, int nq, bool fp4, cudaStream_t st);
int launch_page_read(const PagesArgs& c, const RowsArgs& r, __nv_bfloat16* k, int64_t k_ld, __nv_bfloat16* v,
                     int64_t v_ld, bool fp4, cudaStream_t st);
// Work split of a call (host side): which kernel, its tile and its workspace.
struct PagePlan {
  bool tc;
  int tile, unit, target, min_units, slots;
  int64_t items, split_tiles;
};
PagePlan page_attention_plan(const dflash_pages& c, const dflash_rows& r, int nq);
int launch_page_attention(const PageAttnArgs& a, const PagePlan& p, bool fp4, cudaStream_t st);
int launch_page_attention_tc(const PageAttnArgs& a, const PagePlan& p, bool fp4, cudaStream_t st);

}  // namespace dfl
