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
  // work split (see Share)
  int unit_log2;         // slots a unit of the split
  int tile, tile_log2;   // rows (query row x head of the group) a tile
  int target;            // CTAs of one wave
  int min_units;         // fewest units a CTA's share has
  int no_split;          // tiles of up to this many units are not split
  float* part_o;         // [2 * target][tile][d]; null: nothing is split
  float* part_ml;        // [2 * target][tile][2]
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
__device__ __forceinline__ UnitRange unit_range(int lo, int hi, int sinks, int unit_log2) {
  UnitRange u;
  const int more = (1 << unit_log2) - 1;
  const int end = (hi + more) >> unit_log2;
  u.first = min(lo >> unit_log2, end);
  u.nsink = lo > 0 ? min((min(sinks, hi) + more) >> unit_log2, u.first) : 0;
  u.n = u.nsink + end - u.first;
  return u;
}

// The split of a call's work, the same in every CTA of a call. Each stream of
// n rows is mt tiles of `tile` (row, head) pairs; a tile's keys are the
// stream's units. All tiles' units, kv head by kv head, stream by stream, make
// one line, and CTA b of B takes the part [total * b / B, total * (b + 1) / B)
// of it: streams of unequal length make equal shares. A share is a run of
// segments, each (part of) one tile; a part goes to the workspace, slot 2b for
// a CTA's first segment and 2b + 1 for its last, and page_combine_kernel joins
// the parts. With many tiles, or short ones, every CTA takes whole tiles
// instead.
__device__ __forceinline__ long long div_up_to_64(long long a, long long b) {  // a >= 0, b > 0; mostly 32 bits
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}
struct Share {
  long long line;   // units of a kv head
  long long tiles;  // tiles of a kv head
  long long ctas;   // B
  bool whole;       // a tile a CTA
  __device__ __forceinline__ long long start(const PageAttnArgs& a, long long b) const {
    return whole ? b : div_up_to_64(line * a.c.nkv * b, ctas);
  }
};
struct Segment {
  int h, s, tile;  // kv head, stream, tile of it
  int u, x0, x1;   // units of the tile, and the part of them
};

__device__ __forceinline__ int stream_units(const PageAttnArgs& a, int s, int* mt, bool flag) {
  bool bad;
  const StreamRows q = stream_rows(a.r, s, &bad);
  if (bad && flag) flag_status(a.r.status, DFLASH_STATUS_BAD_ROWS);
  *mt = (q.n * a.G + (1 << a.tile_log2) - 1) >> a.tile_log2;  // max_rows * G is under 2^31
  if (q.n == 0) return 0;
  const int lo = a.window > 0 ? max(0, q.C - a.window + 1) : 0;
  return unit_range(lo, q.C + q.n, a.sinks, a.unit_log2).n;
}

// One warp; every lane gets the answer.
__device__ __forceinline__ Share share_of(const PageAttnArgs& a) {
  const int lane = threadIdx.x & 31;
  long long line = 0, tiles = 0;
  int most = 0;
  for (int s0 = 0; s0 < a.r.S; s0 += 32) {
    int mt = 0, u = 0;
    if (s0 + lane < a.r.S) u = stream_units(a, s0 + lane, &mt, blockIdx.x == 0 && blockIdx.y == 0);
    line += static_cast<long long>(mt) * u;
    tiles += mt;
    most = max(most, u);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    line += __shfl_xor_sync(0xffffffffu, line, o);
    tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  Share sh;
  sh.line = line;
  sh.tiles = tiles;
  sh.whole = a.part_o == nullptr || most <= a.no_split || tiles * a.c.nkv >= 3ll * a.target;
  if (sh.whole) {
    sh.ctas = tiles * a.c.nkv;
  } else {
    const long long b = div_up_to_64(line * a.c.nkv + a.min_units - 1, a.min_units);
    sh.ctas = b < a.target ? b : a.target;
  }
  return sh;
}

// The segment at place `at` of the line (whole: tile `at`), open to the tile's
// end. One warp.
__device__ __forceinline__ Segment segment_at(const PageAttnArgs& a, const Share& sh, long long at) {
  const int lane = threadIdx.x & 31;
  const long long per = sh.whole ? sh.tiles : sh.line;
  Segment g;
  g.h = static_cast<int>(div_up_to_64(at, per));
  const long long r = at - g.h * per;
  long long base = 0;
  g.s = g.tile = g.u = g.x0 = g.x1 = 0;
  for (int s0 = 0; s0 < a.r.S; s0 += 32) {
    int mt = 0, u = 0;
    if (s0 + lane < a.r.S) u = stream_units(a, s0 + lane, &mt, false);
    const long long cnt = sh.whole ? mt : static_cast<long long>(mt) * u;
    long long inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, r < base + inc);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const long long rel = r - base - __shfl_sync(0xffffffffu, inc - cnt, l);
      g.s = s0 + l;
      g.u = __shfl_sync(0xffffffffu, u, l);
      const int tiles = __shfl_sync(0xffffffffu, mt, l);
      const int tile = static_cast<int>(sh.whole ? rel : div_up_to_64(rel, g.u));
      g.x0 = sh.whole ? 0 : static_cast<int>(rel - static_cast<long long>(tile) * g.u);
      g.x1 = g.u;
      g.tile = tiles - 1 - tile;  // the last rows see most: whole tiles start with them
      return g;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return g;
}

// A CTA's run of segments, kept in shared memory between them.
struct Run {
  Share sh;
  long long at, end;
  Segment seg;
  int left;  // whether seg is one
};
__device__ __forceinline__ void run_begin(const PageAttnArgs& a, Run* run) {
  const Share sh = share_of(a);
  if ((threadIdx.x & 31) == 0) {
    const bool on = blockIdx.x < sh.ctas;
    run->sh = sh;
    run->at = on ? sh.start(a, blockIdx.x) : 0;
    run->end = on ? sh.start(a, blockIdx.x + 1ll) : 0;
  }
  __syncwarp();
}
__device__ __forceinline__ void run_next(const PageAttnArgs& a, Run* run) {
  const long long at = run->at, left = run->end - at;
  Segment sg{};
  if (left > 0) {
    const Share sh = run->sh;
    sg = segment_at(a, sh, at);
    if (!sh.whole && sg.x1 - sg.x0 > left) sg.x1 = sg.x0 + static_cast<int>(left);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) run->at = at + (sh.whole ? 1 : sg.x1 - sg.x0);
  }
  if ((threadIdx.x & 31) == 0) {
    run->seg = sg;
    run->left = left > 0;
  }
  __syncwarp();
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
  bool tc;      // the tensor-memory kernel
  bool split;   // tiles may be split: a workspace and a combine launch
  int tile, unit, target, min_units, no_split;
  int64_t ctas;
};
PagePlan page_attention_plan(const dflash_pages& c, const dflash_rows& r, int nq);
int launch_page_attention(const PageAttnArgs& a, const PagePlan& p, bool fp4, cudaStream_t st);
int launch_page_attention_tc(const PageAttnArgs& a, const PagePlan& p, bool fp4, cudaStream_t st);

}  // namespace dfl
