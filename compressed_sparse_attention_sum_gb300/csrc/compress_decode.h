// Launcher of csa_compress_decode (internal to the library).
#pragma once

#include "rows.h"

namespace csa {

struct CompressDecodeArgs {
  const void *kv, *score;
  long long kv_bs, kv_rs, sc_bs, sc_rs;   // elements
  int sw;                                 // score width: 1 or d
  void *kv_ring, *score_ring;
  int R;                                  // rows of a ring
  const int32_t* seq_lens;
  int kind;
  const float *weight, *bias;
  float eps;
  RopeArgs rope;
  void* out;
  long long out_bs;
  int32_t *first, *counts;
  int b, s_q, d, ratio, coff;
  int* status;
  bool store_here;                        // set by the launcher
};

cudaError_t launch_compress_decode(const CompressDecodeArgs& a, bool bf16, cudaStream_t st);

}  // namespace csa
