// Launchers of the row calls (internal to the library); include/csa_rows.h has
// their definitions.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace csa {

constexpr int kMaxNormWidth = 32768;   // channels of csa_norm's rows
constexpr int kMaxHeadWidth = 512;     // channels of a head's row

enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

struct RopeArgs {
  const int64_t* turns;   // null: no rotation
  int dim, first;
  float scale;
  bool half, back;        // back: by the negative angle
};

// The angle that `turn` (2^-64 turns a position) makes at position pos, in 2^-32 turns: the
// top half of the product modulo 2^64, which is exact, as whole turns drop out.  The factors
// are unsigned: signed ones would overflow at most positions.
__host__ __device__ constexpr uint32_t angle_of(int64_t turn, int pos) {
  return (uint32_t)(((uint64_t)turn * (uint64_t)(int64_t)pos) >> 32);
}

struct RowStrides {
  long long b, t, h;      // elements
};

// Rows [b, s, H, d] of the forward calls.
struct RowsFwd {
  const void* x;
  void* out;
  RowStrides xs, os;
  bool x_bf16, out_bf16;
  int kind;               // kNormNone: rotation only (x and out may differ in type)
  const float *weight, *bias;
  float eps;
  const int32_t* pos;     // null: the token's index
  long long pos_stride;
  RopeArgs rope;
  int b, s, H, d;
  bool in_place;          // out is x: channels that nothing changes stay untouched
};

struct RowsBwd {
  const void *x, *dout;
  void* dx;
  RowStrides xs, gs, ds;
  bool x_bf16, g_bf16, dx_bf16;
  int kind;
  const float* weight;
  float eps;
  const int32_t* pos;
  long long pos_stride;
  RopeArgs rope;
  float *dweight, *dbias; // null: not wanted
  float* parts;           // [CTAs][wanted][d]
  int b, s, H, d;
};

// CTAs whose sums of dweight and dbias go to the workspace.
int rows_bwd_ctas(long long rows, int n);

cudaError_t launch_rows_fwd(const RowsFwd& a, cudaStream_t st);        // d <= kMaxHeadWidth
cudaError_t launch_rows_bwd(const RowsBwd& a, int ctas, cudaStream_t st);
// [rows, n] rows (b = s = 1) of any width up to kMaxNormWidth, no rotation
cudaError_t launch_norm_wide(const RowsFwd& a, cudaStream_t st);
cudaError_t launch_norm_wide_bwd(const RowsBwd& a, int ctas, cudaStream_t st);
// dweight and dbias from the CTAs' parts
cudaError_t launch_sum_parts(const float* parts, int ctas, float* dweight, float* dbias, int n,
                             cudaStream_t st);

}  // namespace csa
