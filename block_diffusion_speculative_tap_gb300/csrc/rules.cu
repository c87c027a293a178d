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
// group of its rows; a thread keeps its 8 tokens' counts and biases in
// registers and streams the rows: 16 bytes of scores in, one byte of the
// mask, 16 bytes out. The drafted tokens and biases that fall into the slice
// (few) wait in shared memory. Bound by the scores' bytes.
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

__global__ void __launch_bounds__(kThreads) logit_rules_kernel(const RulesArgs a) {
  __shared__ float bias[kSlice];
  __shared__ uint32_t path[DFLASH_MAX_TREE_NODES];  // node << 16 | token of the slice
  __shared__ int n_path;
  __shared__ uint16_t bid[kThreads];
  __shared__ float bval[kThreads];
  __shared__ int wcount[kThreads / 32 + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = blockIdx.x * kSlice, v = v0 + tid * 8;
  const int n0 = blockIdx.y * a.group, n1 = min(a.N, n0 + a.group);
  const bool on = v < a.V;
  for (int s = blockIdx.z; s < a.S; s += gridDim.z) {
    if (tid == 0) n_path = 0;
    bool any_bias = false;
    float b[8] = {};
    uint4 cw = make_uint4(0u, 0u, 0u, 0u);
    if (a.counts && on) cw = *reinterpret_cast<const uint4*>(a.counts + static_cast<int64_t>(s) * a.V + v);
    __syncthreads();
    // the drafted tokens of the slice; the root's (node 0) are in the counts
    if (a.tokens)
      for (int m = 1 + tid; m < a.N; m += kThreads) {
        const int id = a.tokens[static_cast<int64_t>(s) * a.N + m];
        if (id >= v0 && id < v0 + kSlice && id < a.V)
          path[atomicAdd(&n_path, 1)] = static_cast<uint32_t>(m) << 16 | static_cast<uint32_t>(id - v0);
      }
    // the biases of the slice, in list order: equal ids add up in that order
    if (a.bias_start) {
      const int e0 = max(0, min(a.bias_start[s], a.n_bias)), e1 = max(e0, min(a.bias_start[s + 1], a.n_bias));
      if (e1 > e0) {
        for (int i = tid; i < kSlice; i += kThreads) bias[i] = 0.f;
        for (int e = e0; e < e1; e += kThreads) {
          __syncthreads();
          const int id = e + tid < e1 ? a.bias_ids[e + tid] : -1;
          const bool in = id >= v0 && id < v0 + kSlice && id < a.V;
          const unsigned w = __ballot_sync(0xffffffffu, in);
          if (lane == 0) wcount[warp] = __popc(w);
          __syncthreads();
          int at = __popc(w & ((1u << lane) - 1u)), total = 0;
          for (int k = 0; k < kThreads / 32; ++k) {
            if (k < warp) at += wcount[k];
            total += wcount[k];
          }
          if (total == 0) continue;
          any_bias = true;
          if (in) {
            bid[at] = static_cast<uint16_t>(id - v0);
            bval[at] = a.bias_vals[e + tid];
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
      }
    }
    __syncthreads();
    if (any_bias)
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = bias[tid * 8 + k];
    const float rep = a.repetition ? a.repetition[s] : 1.f;
    const float freq = a.frequency ? a.frequency[s] : 0.f;
    const float pres = a.presence ? a.presence[s] : 0.f;
    const int np = n_path;
    const bool counted = (cw.x | cw.y | cw.z | cw.w) != 0u;
    const uint32_t c4[4] = {cw.x, cw.y, cw.z, cw.w};
    if (on) {
#pragma unroll 4
      for (int n = n0; n < n1; ++n) {
        const int64_t row = static_cast<int64_t>(s) * a.N + n;
        const uint4 xw = *reinterpret_cast<const uint4*>(a.in + row * a.V + v);
        unsigned may = 0xffu;
        if (a.grammar) may = reinterpret_cast<const uint8_t*>(a.grammar + row * a.words)[v >> 3];
        uint32_t w[4] = {xw.x, xw.y, xw.z, xw.w};
        unsigned extra[8];
        bool drafted = false;
        if (np > 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) extra[k] = 0u;
          for (int p = 0; p < np; ++p) {
            const int m = path[p] >> 16, k0 = static_cast<int>(path[p] & 0xffffu) - tid * 8;
            if (k0 < 0 || k0 >= 8) continue;
            const bool hit = a.node_mask ? (a.node_mask[row * a.mask_ld + (m >> 5)] >> (m & 31)) & 1u : m <= n;
            if (!hit) continue;
            drafted = true;
#pragma unroll
            for (int k = 0; k < 8; ++k) extra[k] += k == k0;
          }
        }
        if (counted || drafted || any_bias) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float x = __uint_as_float((k & 1) ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
            const unsigned c = (c4[k >> 1] >> (16 * (k & 1))) & 0xffffu;
            x = penalise(x, static_cast<int>((c & 0x7fffu) + (drafted ? extra[k] : 0u)), c >> 15, rep, freq, pres);
            x = __fadd_rn(x, b[k]);
            const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(x));
            w[k >> 1] = (k & 1) ? (w[k >> 1] & 0xffffu) | (h << 16) : (w[k >> 1] & 0xffff0000u) | h;
          }
        }
        if (may != 0xffu) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (!((may >> k) & 1u)) w[k >> 1] = (k & 1) ? (w[k >> 1] & 0xffffu) | 0xff800000u : (w[k >> 1] & 0xffff0000u) | 0xff80u;
        }
        *reinterpret_cast<uint4*>(a.out + row * a.V + v) = make_uint4(w[0], w[1], w[2], w[3]);
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
  // rows a CTA: its counts, biases and drafted tokens are read once for all
  // of them, so as many as leave about four CTAs an SM
  const int64_t rows_all = static_cast<int64_t>(a.S) * a.N * slices;
  int64_t group = rows_all / (4ll * num_sms);
  a.group = static_cast<int>(group < 1 ? 1 : group > a.N ? a.N : group);
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
