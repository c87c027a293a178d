// Editing a target's scores before they are verified: penalties for repeated
// tokens, biases, a grammar's mask.
//
// For row n of a stream (the scores after node n of its draft) and token v,
// with c the stream's count of v among its output tokens, p whether v is in
// its prompt, and e the number of nodes on the path from the root (not
// counted: the root is the last committed token) to n that hold v:
//   count = c + e,  seen = p or count > 0
//   x = seen ? (x > 0 ? x / repetition : x * repetition) : x
//   x = x - frequency * count - presence * [count > 0]
//   x = x + (sum of v's biases);   x = -inf where the grammar's bit of v is 0
// in fp32, every operation rounded, the result rounded once to bf16.
//
// logit_rules_kernel: one CTA takes a slice of 2048 tokens of a stream for a
// group of its rows. The tokens of the slice that any rule touches (a count, a
// bias, a drafted node: a few in a thousand) are listed in shared memory; the
// rows are copied under the mask, 16 bytes of scores and a byte of the mask a
// thread, and then the listed scores are edited in place, a thread each: with
// the edits inside the copy nearly every warp had some thread to wait for
// (32 trees of 93 nodes x 151936: 668 us, 327 us this way). Bound by the scores'
// bytes: 5.7 TB/s there; 16 rows of one stream take 4.5 us, a launch's latency.
//
// token_counts_kernel: adds tokens to a stream's counts, one thread a token;
// equal tokens of a warp go in one update, which saturates at 32767.
#include "internal.h"
#include "ptx.cuh"
#include "rules.h"

namespace dfl {

namespace {

constexpr int kThreads = 256;
constexpr int kSlice = kThreads * 8;

__device__ __forceinline__ float penalise(float x, int count, bool prompt, float rep, float freq, float pres) {
  if (prompt || count > 0) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
  if (count > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, static_cast<float>(count))), pres);
  return x;
}

// Rows a thread has in flight: 16 bytes of scores and a byte of the mask each.
constexpr int kBatch = 4;

__global__ void __launch_bounds__(kThreads, 4) logit_rules_kernel(const RulesArgs a) {
  __shared__ __align__(16) float bias[kSlice];
  __shared__ uint32_t path[DFLASH_MAX_TREE_NODES];  // node << 16 | token of the slice
  __shared__ uint32_t marked[kSlice / 32];          // tokens of the slice with a count, a bias or a drafted node
  __shared__ uint16_t list[kSlice];
  __shared__ int n_path, n_list;
  __shared__ uint16_t bid[kThreads];
  __shared__ float bval[kThreads];
  __shared__ int wcount[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = blockIdx.x * kSlice, v = v0 + tid * 8;
  const int n0 = blockIdx.y * a.group, n1 = min(a.N, n0 + a.group);
  const bool on = v < a.V;
  for (int s = blockIdx.z; s < a.S; s += gridDim.z) {
    const int64_t row0 = static_cast<int64_t>(s) * a.N;
    const __nv_bfloat16* in = a.in + row0 * a.V + v;
    __nv_bfloat16* out = a.out + row0 * a.V + v;
    const uint8_t* gram = a.grammar ? reinterpret_cast<const uint8_t*>(a.grammar + row0 * a.words) + (v >> 3) : nullptr;
    uint4 x[kBatch];
    unsigned may[kBatch];
    auto fetch = [&](int n) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        may[i] = 0xffu;
        if (on && n + i < n1) {
          x[i] = *reinterpret_cast<const uint4*>(in + static_cast<int64_t>(n + i) * a.V);
          if (gram) may[i] = gram[static_cast<int64_t>(n + i) * a.words * 4];
        }
      }
    };
    fetch(n0);
    // ------------------------------------------------ what the rules touch in the slice
    uint4 cw = make_uint4(0u, 0u, 0u, 0u);
    if (a.counts && on) cw = *reinterpret_cast<const uint4*>(a.counts + static_cast<int64_t>(s) * a.V + v);
    int e0 = 0, e1 = 0;
    if (a.bias_start) {
      e0 = max(0, min(a.bias_start[s], a.n_bias));
      e1 = max(e0, min(a.bias_start[s + 1], a.n_bias));
    }
    if (tid == 0) n_path = n_list = 0;
    {
      const uint32_t c4[4] = {cw.x, cw.y, cw.z, cw.w};
      unsigned mine = 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) mine |= ((c4[k >> 1] >> (16 * (k & 1))) & 0xffffu) != 0u ? 1u << k : 0u;
      reinterpret_cast<uint8_t*>(marked)[tid] = static_cast<uint8_t>(mine);
    }
    if (e1 > e0) {
      *reinterpret_cast<float4*>(bias + tid * 8) = make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(bias + tid * 8 + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    // drafted tokens; the root's (node 0) are in the counts
    if (a.tokens)
      for (int m = 1 + tid; m < a.N; m += kThreads) {
        const int id = a.tokens[row0 + m];
        if (id >= v0 && id < v0 + kSlice && id < a.V) {
          path[atomicAdd(&n_path, 1)] = static_cast<uint32_t>(m) << 16 | static_cast<uint32_t>(id - v0);
          atomicOr(&marked[(id - v0) >> 5], 1u << ((id - v0) & 31));
        }
      }
    // biases, in list order: equal ids add up in that order
    for (int e = e0; e < e1; e += kThreads) {
      const int id = e + tid < e1 ? a.bias_ids[e + tid] : -1;
      const bool in_slice = id >= v0 && id < v0 + kSlice && id < a.V;
      const unsigned w = __ballot_sync(0xffffffffu, in_slice);
      if (lane == 0) wcount[warp] = __popc(w);
      if (__syncthreads_or(in_slice)) {
        int at = __popc(w & ((1u << lane) - 1u)), total = 0;
        for (int k = 0; k < kThreads / 32; ++k) {
          if (k < warp) at += wcount[k];
          total += wcount[k];
        }
        if (in_slice) {
          bid[at] = static_cast<uint16_t>(id - v0);
          bval[at] = a.bias_vals[e + tid];
          atomicOr(&marked[(id - v0) >> 5], 1u << ((id - v0) & 31));
        }
        __syncthreads();
        if (tid < total) {
          bool first = true;
          for (int k = 0; k < tid; ++k) first &= bid[k] != bid[tid];
          if (first) {
            float sum = bias[bid[tid]];
            for (int k = tid; k < total; ++k)
              if (bid[k] == bid[tid]) sum = __fadd_rn(sum, bval[k]);
            bias[bid[tid]] = sum;
          }
        }
      }
      __syncthreads();  // the lists are written again
    }
    __syncthreads();
    {
      unsigned mine = reinterpret_cast<const uint8_t*>(marked)[tid];
      if (mine) {
        int at = atomicAdd(&n_list, __popc(mine));
        for (; mine; mine &= mine - 1u) list[at++] = static_cast<uint16_t>(tid * 8 + __ffs(mine) - 1);
      }
    }
    // ------------------------------------------------ every score: copied, or -inf by the mask
    for (int n = n0; n < n1; n += kBatch) {
      uint4 y[kBatch];
      unsigned allow[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        y[i] = x[i];
        allow[i] = may[i];
      }
      fetch(n + kBatch);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // two bits of the mask to two halves
          const uint32_t two = (allow[i] >> (2 * k)) & 3u;
          const uint32_t keep = ((two & 1u) | ((two & 2u) << 15)) * 0xffffu;
          w[k] = (w[k] & keep) | (0xff80ff80u & ~keep);
        }
        if (on && n + i < n1)
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(n + i) * a.V) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncthreads();
    // ------------------------------------------------ the few that a rule touches, again
    const int nl = n_list, np = n_path, rows = n1 - n0;
    if (nl > 0) {
      const float rep = a.repetition ? a.repetition[s] : 1.f;
      const float freq = a.frequency ? a.frequency[s] : 0.f;
      const float pres = a.presence ? a.presence[s] : 0.f;
      for (int i = tid; i < nl * rows; i += kThreads) {
        const int n = n0 + i / nl, id = list[i % nl];
        if (a.grammar) {
          const uint32_t word = a.grammar[(row0 + n) * a.words + ((v0 + id) >> 5)];
          if (!((word >> ((v0 + id) & 31)) & 1u)) continue;
        }
        const unsigned c = a.counts ? a.counts[static_cast<int64_t>(s) * a.V + v0 + id] : 0u;
        int count = static_cast<int>(c & 0x7fffu);
        for (int p = 0; p < np; ++p) {
          const int m = path[p] >> 16;
          if (static_cast<int>(path[p] & 0xffffu) != id) continue;
          count += a.node_mask ? (a.node_mask[(row0 + n) * a.mask_ld + (m >> 5)] >> (m & 31)) & 1u : m <= n;
        }
        __nv_bfloat16* at = a.out + (row0 + n) * a.V + v0 + id;
        float f = penalise(__bfloat162float(*at), count, c >> 15, rep, freq, pres);
        if (e1 > e0) f = __fadd_rn(f, bias[id]);
        *at = __float2bfloat16_rn(f);
      }
    }
    __syncthreads();  // the next stream writes the shared lists
  }
}

__global__ void __launch_bounds__(256) token_counts_kernel(uint16_t* counts, const int* tokens, const int* row_start,
                                                           int S, int V, int per, int64_t total, int prompt) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  int s = -1;
  if (i < total) {
    if (!row_start) {
      s = static_cast<int>(i / per);
    } else {
      // the last stream that starts at or before i, if it reaches that far
      int lo = 0, hi = S;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row_start[mid] <= i) lo = mid;
        else hi = mid;
      }
      if (row_start[lo] <= i && i < row_start[lo + 1]) s = lo;
    }
  }
  const int id = s >= 0 ? tokens[i] : -1;
  const bool on = id >= 0 && id < V;
  const long long key = on ? static_cast<long long>(s) * V + id : -1;
  const unsigned same = __match_any_sync(0xffffffffu, static_cast<unsigned long long>(key));
  if (!on || static_cast<int>(threadIdx.x & 31) != __ffs(same) - 1) return;
  unsigned* word = reinterpret_cast<unsigned*>(counts + (key & ~1ll));
  const int sh = (key & 1) ? 16 : 0;
  if (prompt) {
    atomicOr(word, 0x8000u << sh);
    return;
  }
  const unsigned add = __popc(same);
  unsigned old = *reinterpret_cast<volatile unsigned*>(word);
  while (true) {
    const unsigned c = (old >> sh) & 0x7fffu;
    const unsigned n = min(0x7fffu, c + add);
    if (n == c) return;
    const unsigned seen = atomicCAS(word, old, old + ((n - c) << sh));
    if (seen == old) return;
    old = seen;
  }
}

}  // namespace

int launch_logit_rules(const RulesArgs& args, int num_sms, cudaStream_t st) {
  RulesArgs a = args;
  const int slices = (a.V + kSlice - 1) / kSlice;
  // rows a CTA: its counts, biases and drafted tokens are looked up once for
  // all of them, so as many as leave two waves of four CTAs an SM, and whole
  // batches of rows in flight
  const int64_t rows_all = static_cast<int64_t>(a.S) * a.N * slices;
  int64_t group = rows_all / (8ll * num_sms);
  group = (group + kBatch - 1) / kBatch * kBatch;
  a.group = static_cast<int>(group < kBatch ? kBatch : group > a.N ? a.N : group);
  const int groups = (a.N + a.group - 1) / a.group;
  TraceScope ts(st, "logit_rules", static_cast<double>(a.S) * a.V * (4.0 * a.N + (a.counts ? 2.0 : 0.0) +
                                   (a.grammar ? a.N / 8.0 : 0.0)), 0.0);
  const cudaError_t e = launch_pdl(logit_rules_kernel,
                                   dim3(static_cast<unsigned>(slices), static_cast<unsigned>(groups),
                                        static_cast<unsigned>(a.S < 65535 ? a.S : 65535)),
                                   dim3(kThreads), 0, st, a);
  count_launch();
  return cuda_status(e);
}

int launch_token_counts(uint16_t* counts, const int* tokens, const int* row_start, int S, int V, int per,
                        int64_t total, int prompt, cudaStream_t st) {
  TraceScope ts(st, "token_counts", 4.0 * total, 0.0);
  const cudaError_t e = launch_pdl(token_counts_kernel, dim3(static_cast<unsigned>((total + 255) / 256)), dim3(256), 0,
                                   st, counts, tokens, row_start, S, V, per, total, prompt);
  count_launch();
  return cuda_status(e);
}

}  // namespace dfl
