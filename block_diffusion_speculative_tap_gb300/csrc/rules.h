// Arguments of the logit rules' kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash.h"

namespace dfl {

struct RulesArgs {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int S, N, V, words, mask_ld, n_bias, group;
  const uint16_t* counts;
  const int* tokens;
  const uint32_t* node_mask;
  const float *repetition, *frequency, *presence;
  const int *bias_start, *bias_ids;
  const float* bias_vals;
  const uint32_t* grammar;
};

int launch_logit_rules(const RulesArgs& a, int num_sms, cudaStream_t st);
int launch_token_counts(uint16_t* counts, const int* tokens, const int* row_start, int S, int V, int per,
                        int64_t total, int prompt, cudaStream_t st);

}  // namespace dfl
