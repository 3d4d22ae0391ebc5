// Internal declarations of the 8-bit path (include/paro_w8a8.h).
#pragma once

#include "paro_block.h"
#include "paro_internal.h"
#include "paro_w8a8.h"

namespace paro {

constexpr float kQ8Max = 127.0f;
// Smallest row maximum a scale is made from (2^-100): 127 / it and the scale stay normal float32.
constexpr float kQ8MinTop = 0x1p-100f;

// Rows of 16-bit elements, read as the library's own vector types.
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using i32x4 = int __attribute__((ext_vector_type(4)));

struct NormArgs {
  int M, D, dtype;
  const void* x;
  const void* residual;  // nullptr: none
  const void* gamma;
  float eps;
  void* residual_out;
  void* y;       // 16-bit output, or
  int8_t* q;     // codes and
  float* scales; // scales
  // the norm and gate after a block (launch_block_norm): x is the block's output
  const void* post_gamma;  // nullptr: no norm
  const void* gate;        // nullptr: none
  uint32_t gate_rows;      // row m takes the gate's row m / gate_rows
  float residual_scale;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st);
hipError_t launch_block_norm(const NormArgs& a, hipStream_t st);
hipError_t launch_quantize_q8(int M, int D, int dtype, const void* x, int8_t* q, float* scales, hipStream_t st);
hipError_t launch_dequantize_q8(int M, int D, const int8_t* q, const float* scales, void* x, int dtype, hipStream_t st);
// The row quantiser behind the transform R.
hipError_t launch_rotate_q8(const DevRot& R, int M, int dtype, const void* x, int8_t* q, float* scales, hipStream_t st);
// R.K == 0 and R.s == nullptr: no transform.
hipError_t launch_pack_q8(const DevRot& R, int N, int dtype, const void* W, int8_t* q, float* scales, hipStream_t st);

// One 8-bit product: y [M][N], or with `gated` y [M][N] = silu(gate) * up from weights [2N][D], or with
// `epilogue` y = act(product + bias) + residual.
struct W8A8Call {
  int M, D, N;
  bool gated;
  const int8_t* x;
  const float* xs;
  const int8_t* w;
  const float* ws;
  void* y;
  int ydtype;
  bool epilogue;
  int act;               // paro_activation
  const void* bias;      // ydtype [N], or nullptr
  const void* residual;  // ydtype [M][N], or nullptr
};
// What a product kernel makes of its sums.
enum Output { kPlain, kGated, kEpilogue };
// A row or two: the weights streamed into registers, no workspace.
bool w8a8_stream_takes(int M, int N);
hipError_t launch_w8a8_stream(const W8A8Call& c, hipStream_t st);
// Up to 64 rows: 16 columns a workgroup, no workspace. Its estimated time (1e30: not taken).
double w8a8_column_us(int M, int D, int N, bool gated);
hipError_t launch_w8a8_column(const W8A8Call& c, hipStream_t st);
// Any number of rows: the tiled product.
struct GemmPlanQ8 {
  int tile;           // which tiling
  int splits;         // of the reduction over D
  size_t part_bytes;  // workspace of the splits' partial sums (0: no split)
  double us;          // estimated time
};
GemmPlanQ8 plan_gemm_w8a8(int M, int D, int N, bool gated);
constexpr int kTilingsQ8 = 7;
struct TilingQ8 {
  int bm, bn;      // rows of x and of w in a tile
  int workgroups;  // that the GPU holds at once
};
TilingQ8 tiling_w8a8(int tile);
// Workspace of a reduction in this many parts (1: none).
size_t part_bytes_w8a8(int M, int N, bool gated, int splits);
hipError_t launch_w8a8_gemm(const W8A8Call& c, const GemmPlanQ8& p, int* part, hipStream_t st);

}  // namespace paro

// For tests, and in no header of the library: which kernel a product takes (0 streamed, 1 by columns, 2 tiled)
// with its tiling and split, what a tiling is, and a product in a given tiling and split (at most one part for
// each 128 channels; the rest as in paro_w8a8_linear and paro_w8a8_gated_linear).
extern "C" {
void paro_internal_w8a8_plan(int M, int D, int N, int gated, int* kernel, int* tile, int* splits);
int paro_internal_w8a8_tiling(int tile, int* bm, int* bn, int* workgroups);  // 0 past the last one
size_t paro_internal_w8a8_tiled_workspace_bytes(int M, int N, int gated, int splits);
paro_status paro_internal_w8a8_tiled(int tile, int splits, int gated, int M, int D, int N, const int8_t* x, const float* xscales,
                                     const int8_t* qweight, const float* wscales, void* y, int ydtype, void* ws, size_t ws_bytes,
                                     void* stream);
paro_status paro_internal_w8a8_tiled_epilogue(int tile, int splits, int M, int D, int N, const int8_t* x, const float* xscales,
                                              const int8_t* qweight, const float* wscales, const void* bias, int activation,
                                              const void* residual, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream);
}
