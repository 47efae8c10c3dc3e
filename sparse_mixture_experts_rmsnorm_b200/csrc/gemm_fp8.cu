// Grouped product of e4m3 operands with block scales:
//   C[r][n] = sum_kb sa[r][kb] * sb[g][n / 128][kb] * sum_{k in kb} A[r][k] * B[g][n][k]
// for the rows r of group g, kb running over blocks of 128 columns.  The inner
// sums and the sum over blocks are fp32.
#include "gemm_fp8_kernels.h"
#include "quant_common.cuh"

namespace moe {

struct Fp8Args {
  moe_host::Fp8Gemm g;
};

__device__ __forceinline__ float silu_f(float z) { return __fdividef(z, 1.f + __expf(-z)); }

__device__ __forceinline__ float e4m3_value(uint8_t v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

// 32 rows x 128 columns per block of 256 threads: warp w takes rows 4w .. 4w + 3,
// lane l columns l, l + 32, l + 64, l + 96.
template <int EPI>
__global__ void __launch_bounds__(256) gemm_fp8_simple_kernel(const Fp8Args args) {
  const moe_host::Fp8Gemm& a = args.g;
  constexpr int NB = EPI == moe_host::EPI_SWIGLU ? 2 : 1;
  __shared__ float xs[32][33];
  __shared__ float ws[NB][128][33];
  __shared__ int tile_sh[3];
  if (threadIdx.x == 0) {
    int t = blockIdx.y, g = 0;
    const int groups = a.offsets ? a.groups : 1;
    tile_sh[0] = -1;
    for (; g < groups; ++g) {
      const int b = a.offsets ? a.offsets[g] : 0, e = a.offsets ? a.offsets[g + 1] : a.max_rows;
      const int tiles = (e - b + 31) / 32;
      if (t < tiles) {
        tile_sh[0] = g;
        tile_sh[1] = b + t * 32;
        tile_sh[2] = e;
        break;
      }
      t -= tiles;
    }
  }
  __syncthreads();
  const int g = tile_sh[0], row0 = tile_sh[1], row_end = tile_sh[2];
  if (g < 0) return;
  const int n0 = blockIdx.x * 128;
  const int nkb = (a.k + 127) / 128, nnb = (a.nout + 127) / 128;
  const bool sh = a.sb.q != nullptr && g == a.groups - 1;
  const uint8_t* A = a.a.q;
  const float* As = a.a.scale;
  int64_t ld = a.a.ld;
  int shift = 0;
  if (sh && a.sa.q != nullptr) {
    A = a.sa.q;
    As = a.sa.scale;
    ld = a.sa.ld;
    shift = a.offsets[g];
  }
  const int warp = warp_id(), lane = lane_id();
  float acc[NB][4][4] = {};
  for (int kb = 0; kb < nkb; ++kb) {
    float in[NB][4][4] = {};
    for (int k0 = kb * 128; k0 < kb * 128 + 128; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < 32 * 32; i += 256) {
        const int r = i / 32, k = k0 + i % 32;
        xs[r][i % 32] = (row0 + r < row_end && k < a.k) ? e4m3_value(A[(size_t)(row0 + r - shift) * ld + k]) : 0.f;
      }
      for (int b = 0; b < NB; ++b) {
        const uint8_t* W = sh ? (b ? a.sb2.q : a.sb.q) : (b ? a.b2.q : a.b.q) + (size_t)g * a.nout * a.k;
        for (int i = threadIdx.x; i < 128 * 32; i += 256) {
          const int n = i / 32, k = k0 + i % 32;
          ws[b][n][i % 32] = (n0 + n < a.nout && k < a.k) ? e4m3_value(W[(size_t)(n0 + n) * a.k + k]) : 0.f;
        }
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int b = 0; b < NB; ++b)
          for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j)
              in[b][i][j] = fmaf(xs[warp * 4 + i][k], ws[b][lane + 32 * j][k], in[b][i][j]);
    }
    for (int b = 0; b < NB; ++b) {
      const float* S = sh ? (b ? a.sb2.scale : a.sb.scale) : (b ? a.b2.scale : a.b.scale) + (size_t)g * nnb * nkb;
      const float sb = S[(size_t)blockIdx.x * nkb + kb];
      for (int i = 0; i < 4; ++i) {
        const int r = row0 + warp * 4 + i;
        if (r >= row_end) continue;
        const float s = As[(size_t)(r - shift) * nkb + kb] * sb;
        for (int j = 0; j < 4; ++j) acc[b][i][j] = fmaf(in[b][i][j], s, acc[b][i][j]);
      }
    }
  }
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + warp * 4 + i;
    if (EPI == moe_host::EPI_SWIGLU) {
      float v[4], m = 0.f;
      for (int j = 0; j < 4; ++j) {
        v[j] = n0 + lane + 32 * j < a.nout ? silu_f(acc[0][i][j]) * acc[NB - 1][i][j] : 0.f;
        m = fmaxf(m, fabsf(v[j]));
      }
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float sc = quant_scale(m), inv = __frcp_rn(sc);
      if (r >= row_end) continue;
      for (int j = 0; j < 4; ++j)
        if (n0 + lane + 32 * j < a.nout) ((uint8_t*)a.c)[(size_t)r * a.nout + n0 + lane + 32 * j] = e4m3x1(v[j] * inv);
      if (lane == 0) a.c_scale[(size_t)r * nnb + blockIdx.x] = sc;
    } else {
      if (r >= row_end) continue;
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + lane + 32 * j;
        if (n >= a.nout) continue;
        if (EPI == moe_host::EPI_F32) ((float*)a.c)[(size_t)r * a.nout + n] = acc[0][i][j];
        else ((bf16*)a.c)[(size_t)r * a.nout + n] = __float2bfloat16_rn(acc[0][i][j]);
      }
    }
  }
}

}  // namespace moe

namespace moe_host {

moe_status launch_gemm_fp8(const Fp8Gemm& g, cudaStream_t s) {
  if (g.max_rows == 0) return MOE_OK;
  const dim3 grid((unsigned)q_blocks(g.nout), (unsigned)((g.max_rows + 31) / 32 + (g.offsets ? g.groups : 0)));
  moe::Fp8Args a;
  a.g = g;
  if (g.epi == EPI_SWIGLU) moe::gemm_fp8_simple_kernel<EPI_SWIGLU><<<grid, 256, 0, s>>>(a);
  else if (g.epi == EPI_F32) moe::gemm_fp8_simple_kernel<EPI_F32><<<grid, 256, 0, s>>>(a);
  else moe::gemm_fp8_simple_kernel<EPI_STORE><<<grid, 256, 0, s>>>(a);
  return launch_status();
}

}  // namespace moe_host
