// Attention of few packed rows a sequence over a block-scaled cache (fa3_few.cu), as fa3_attn_gqa_block_paged calls it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa3_packed.cuh"

namespace fa3 {

struct FewCall {
  const uint16_t* q;
  const int8_t* k;
  const int8_t* v;
  const float* ks;
  const float* vs;
  const int32_t* q_start;
  const int32_t* kv_lens;
  uint16_t* out;
  float* lse;                      // written (read by the weights)
  int64_t q_stride;
  int n, B, Hq, G, sms;
  float sm_log2;
  int32_t* err;
};

// Whether a call has few enough rows.
bool few_rows(int n, int B, int Hkv, int G, int T_max);
size_t few_rows_workspace(int n, int B, int G, int sms);
cudaError_t few_rows_attn(const FewCall& c, const int32_t* table, int num_pages, int page_size, int max_pages, int block,
                          int Hkv, void* workspace, cudaStream_t s);

// The same of fa3_attn_weights_gqa_block_paged (v, vs and out unused; lse is read).
bool few_rows_weights(int n, int B, int Hkv, int G, int T_max);
cudaError_t few_rows_weights_attn(const FewCall& c, float* weights, const int32_t* table, int num_pages, int page_size,
                                  int max_pages, int block, int Hkv, cudaStream_t s);

}  // namespace fa3
