// Host-side launchers of the 8-bit operators (arguments checked in
// fp8_api.cu; see moe_kernels.h for the conventions).
#pragma once

#include "moe_kernels.h"

namespace moe_host {

moe_status launch_add_rmsnorm(int dtype, const void* x, const void* residual, const void* norm_w, void* res_out,
                              void* xn, uint8_t* q, float* q_scale, int n, int d, float eps, cudaStream_t s);

// mats matrices [rows][cols] in blocks of block_rows (1 or 128) x 128.
moe_status launch_quantize(int dtype, int block_rows, int mats, int rows, int cols, const void* x, uint8_t* q,
                           float* scale, cudaStream_t s);

// One e4m3 operand with its block scales.
struct Fp8Operand {
  const uint8_t* q = nullptr;
  const float* scale = nullptr;
  int64_t ld = 0;  // bytes between rows (the row operands a, sa)
};

// Arguments of a grouped block-scaled e4m3 product.
struct Fp8Gemm {
  int epi = EPI_STORE;       // EPI_STORE (bf16), EPI_F32, EPI_SWIGLU (e4m3 + scales)
  Fp8Operand a, b, b2;       // rows; weights [groups][nout][k] (gate and up for EPI_SWIGLU)
  Fp8Operand sb, sb2, sa;    // the folded shared expert (the last group): weights, and rows (sa.q null: from a)
  int sa_rows = 0;
  const int32_t* offsets = nullptr;
  int groups = 1, max_rows = 0, nout = 0, k = 0;
  void* c = nullptr;         // [max_rows][nout]
  float* c_scale = nullptr;  // EPI_SWIGLU: [max_rows][ceil(nout / 128)]
  bool follows = false;      // the launch before it on the stream is the product that makes a: its end may overlap
  int32_t* hdr = nullptr;    // workspace header
  void* split_ws = nullptr;  // partial sums of cut tiles
  size_t split_bytes = 0;
};

// Most rows, columns (of any operand) and weight rows of all groups: rounded up to
// whole tiles, and a tile further, they still fit an int.
constexpr int64_t kFp8MostExtent = 0x7fffff00;
// Bytes between rows stay below a tensor map's largest stride.
constexpr int64_t kFp8MostStride = (int64_t)1 << 40;

// Start of every workspace of the 8-bit products, the header in it.
constexpr size_t kFp8HeaderBytes = 1024;

// Bytes of partial sums for these sizes (0: no tile is cut).  A launch with fewer
// bytes does not cut its tiles.
size_t gemm_fp8_split_bytes(bool swiglu, int64_t rows, int groups, bool offsets, int nout, int k);

// The tiling of a launch whose partial sums have room: most rows of a tile, 256 of
// them on the MMA's M side (wide) or fewer on its N side, and parts along K.
void gemm_fp8_tiling(bool swiglu, int64_t rows, int groups, bool offsets, int nout, int k, int32_t tiling[3]);

moe_status launch_gemm_fp8(const Fp8Gemm& g, cudaStream_t s);

}  // namespace moe_host
