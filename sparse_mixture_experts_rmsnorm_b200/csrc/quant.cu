// The residual add fused with RMSNorm and an e4m3 output, and the
// quantisation of matrices to e4m3 (see quant_common.cuh for the scales).
//
// The norm is step a1 of the layer ("Mixture of Experts (MoE)" lesson, "The
// concept / Swapping the FFN": the MoE block reads norm(h) of the residual
// stream, and the block before it has just added to that stream):
//   s  = act(x + residual),  r = fl32(1 / sqrt(mean(s^2) + eps)), mean in fp64,
//   v  = fl32(fl32(s * r) * w),  xn = act(v),  (q, q_scale) from v per 128 columns.
// xn has the bits that moe_route gives for h = s.
#include "gemm_fp8_kernels.h"
#include "quant_common.cuh"

namespace moe {

// V consecutive elements of T as one access (V = 1: any alignment).
template <typename T, int V>
struct Pack {
  T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  Pack<T, V> x;
  if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4*>(&x) = *reinterpret_cast<const uint4*>(p);
  else x.v[0] = p[0];
  return x;
}

template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& x) {
  if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&x);
  else p[0] = x.v[0];
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[V], float inv) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                              e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(p) = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  } else {
    p[0] = e4m3x1(v[0] * inv);
  }
}

// Lanes that hold one block of 128 columns, and the passes they take over it:
// V columns per lane and pass.
template <int V>
struct BlockLanes {
  static constexpr int kLanes = V == 8 ? 16 : 32;
  static constexpr int kPasses = Q_BLOCK / (kLanes * V);  // 1, or 4 for V = 1
};

template <int LANES>
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// One block per row (grid-stride); the row s is staged in shared memory in its
// own type.  Every warp takes whole blocks of 128 columns in the second pass,
// so a scale needs no shared memory.
template <typename T, int V>
__global__ void __launch_bounds__(256) add_rmsnorm_kernel(const T* x, const T* residual, const T* __restrict__ w,
                                                          T* res_out, T* xn, uint8_t* __restrict__ q,
                                                          float* __restrict__ q_scale, int n, int d, float eps) {
  extern __shared__ __align__(16) uint8_t row_raw[];
  T* row = reinterpret_cast<T*>(row_raw);
  __shared__ double part[8];
  __shared__ float r_sh;
  constexpr int LANES = BlockLanes<V>::kLanes, PASSES = BlockLanes<V>::kPasses;
  const int warps = blockDim.x >> 5;
  const int nb = (d + Q_BLOCK - 1) / Q_BLOCK;
  for (int t = blockIdx.x; t < n; t += gridDim.x) {
    const size_t base = (size_t)t * d;
    double acc = 0.0;
    for (int i = threadIdx.x * V; i < d; i += blockDim.x * V) {
      Pack<T, V> s = load_pack<T, V>(x + base + i);
      if (residual != nullptr) {
        const Pack<T, V> b = load_pack<T, V>(residual + base + i);
#pragma unroll
        for (int j = 0; j < V; ++j) s.v[j] = from_f32<T>(__fadd_rn(to_f32(s.v[j]), to_f32(b.v[j])));
      }
      if (res_out != nullptr) store_pack<T, V>(res_out + base + i, s);
      store_pack<T, V>(row + i, s);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const double f = (double)to_f32(s.v[j]);
        acc += f * f;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane_id() == 0) part[warp_id()] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
      double sum = 0.0;
      for (int i = 0; i < warps; ++i) sum += part[i];
      r_sh = (float)(1.0 / sqrt(sum / (double)d + (double)eps));
    }
    __syncthreads();
    const float r = r_sh;
    const int unit0 = threadIdx.x / LANES, units = blockDim.x / LANES;
    const int lane = threadIdx.x % LANES;
    // whole warps take part in the shuffles: a unit past the last block has no columns
    for (int b0 = 0; b0 < nb; b0 += units) {
      const int b = b0 + unit0;
      float v[PASSES][V];
      float m = 0.f;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int c = b * Q_BLOCK + (p * LANES + lane) * V;
        if (c < d) {
          const Pack<T, V> s = load_pack<T, V>(row + c), wv = load_pack<T, V>(w + c);
          Pack<T, V> o;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            v[p][j] = __fmul_rn(__fmul_rn(to_f32(s.v[j]), r), to_f32(wv.v[j]));
            m = fmaxf(m, fabsf(v[p][j]));
            o.v[j] = from_f32<T>(v[p][j]);
          }
          if (xn != nullptr) store_pack<T, V>(xn + base + c, o);
        }
      }
      if (q == nullptr) continue;
      const float scale = quant_scale(lanes_max<LANES>(m));
      const float inv = __frcp_rn(scale);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int c = b * Q_BLOCK + (p * LANES + lane) * V;
        if (c < d) store_codes<V>(q + base + c, v[p], inv);
      }
      if (lane == 0 && b < nb) q_scale[(size_t)t * nb + b] = scale;
    }
    __syncthreads();
  }
}

// 1 x 128 blocks: LANES lanes take one block of one row, one pass over the data.
template <typename T, int V>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                            float* __restrict__ scale, int64_t rows, int cols) {
  constexpr int LANES = BlockLanes<V>::kLanes, PASSES = BlockLanes<V>::kPasses;
  const int nb = (cols + Q_BLOCK - 1) / Q_BLOCK;
  const int64_t units = rows * nb;
  const int per_block = blockDim.x / LANES;
  const int lane = threadIdx.x % LANES;
  for (int64_t u0 = (int64_t)blockIdx.x * per_block; u0 < units; u0 += (int64_t)gridDim.x * per_block) {
    const int64_t u = u0 + threadIdx.x / LANES;
    const int64_t r = u / nb;
    const int b = (int)(u - r * nb);
    float v[PASSES][V];
    float m = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int c = b * Q_BLOCK + (p * LANES + lane) * V;
      if (u < units && c < cols) {
        const Pack<T, V> s = load_pack<T, V>(x + r * cols + c);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[p][j] = to_f32(s.v[j]);
          m = fmaxf(m, fabsf(v[p][j]));
        }
      }
    }
    const float sc = quant_scale(lanes_max<LANES>(m));
    const float inv = __frcp_rn(sc);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int c = b * Q_BLOCK + (p * LANES + lane) * V;
      if (u < units && c < cols) store_codes<V>(q + r * cols + c, v[p], inv);
    }
    if (lane == 0 && u < units) scale[u] = sc;
  }
}

// 128 x 128 blocks: a 256-thread block keeps one tile in registers.  Thread i
// holds column group i % (128 / V) of rows i / (128 / V) + step * j.
template <typename T, int V>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                             float* __restrict__ scale, int64_t tiles, int rows,
                                                             int cols) {
  constexpr int ACROSS = Q_BLOCK / V;       // threads across a tile row
  constexpr int STEP = 256 / ACROSS;        // rows per pass
  constexpr int PASSES = Q_BLOCK / STEP;    // 8 (V = 8), 16 (V = 4) or 64 (V = 1)
  __shared__ float part[8];
  const int rb = (rows + Q_BLOCK - 1) / Q_BLOCK, cb = (cols + Q_BLOCK - 1) / Q_BLOCK;
  const int tr = threadIdx.x / ACROSS, tc = (threadIdx.x % ACROSS) * V;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t mat = tile / ((int64_t)rb * cb);
    const int in_mat = (int)(tile - mat * rb * cb);
    const int r0 = (in_mat / cb) * Q_BLOCK, c = (in_mat % cb) * Q_BLOCK + tc;
    const size_t base = (size_t)mat * rows * cols;
    Pack<T, V> s[PASSES];
    float m = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = r0 + tr + p * STEP;
      if (r < rows && c < cols) {
        s[p] = load_pack<T, V>(x + base + (size_t)r * cols + c);
#pragma unroll
        for (int j = 0; j < V; ++j) m = fmaxf(m, fabsf(to_f32(s[p].v[j])));
      }
    }
    m = lanes_max<32>(m);
    __syncthreads();  // the previous tile's maxima have been read
    if (lane_id() == 0) part[warp_id()] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
    const float sc = quant_scale(m);
    const float inv = __frcp_rn(sc);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = r0 + tr + p * STEP;
      if (r < rows && c < cols) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = to_f32(s[p].v[j]);
        store_codes<V>(q + base + (size_t)r * cols + c, v, inv);
      }
    }
    if (threadIdx.x == 0) scale[tile] = sc;
  }
}

}  // namespace moe

namespace moe_host {

template <typename T, int V>
static moe_status add_rmsnorm_t(const void* x, const void* residual, const void* w, void* res_out, void* xn,
                                uint8_t* q, float* q_scale, int n, int d, float eps, cudaStream_t s) {
  static SmemLimit lim;
  const int smem = (int)((size_t)d * sizeof(T));
  const moe_status st = ensure_smem_limit(moe::add_rmsnorm_kernel<T, V>, smem, lim);
  if (st != MOE_OK) return st;
  const int grid = n < sm_count() * 16 ? n : sm_count() * 16;
  moe::add_rmsnorm_kernel<T, V><<<grid, 256, smem, s>>>((const T*)x, (const T*)residual, (const T*)w, (T*)res_out,
                                                        (T*)xn, q, q_scale, n, d, eps);
  return launch_status();
}

moe_status launch_add_rmsnorm(int dtype, const void* x, const void* residual, const void* norm_w, void* res_out,
                              void* xn, uint8_t* q, float* q_scale, int n, int d, float eps, cudaStream_t s) {
  if (n == 0) return MOE_OK;
  const int v = dtype == MOE_BF16 ? 8 : 4;
  const uintptr_t at = (uintptr_t)x | (uintptr_t)residual | (uintptr_t)norm_w | (uintptr_t)res_out | (uintptr_t)xn;
  const bool vec = d % v == 0 && at % 16 == 0 && (uintptr_t)q % 8 == 0;
  if (dtype == MOE_BF16)
    return vec ? add_rmsnorm_t<moe::bf16, 8>(x, residual, norm_w, res_out, xn, q, q_scale, n, d, eps, s)
               : add_rmsnorm_t<moe::bf16, 1>(x, residual, norm_w, res_out, xn, q, q_scale, n, d, eps, s);
  return vec ? add_rmsnorm_t<float, 4>(x, residual, norm_w, res_out, xn, q, q_scale, n, d, eps, s)
             : add_rmsnorm_t<float, 1>(x, residual, norm_w, res_out, xn, q, q_scale, n, d, eps, s);
}

template <typename T, int V>
static moe_status quantize_t(int block_rows, int mats, int rows, int cols, const void* x, uint8_t* q, float* scale,
                             cudaStream_t s) {
  const int nb = q_blocks(cols);
  const int64_t most = (int64_t)sm_count() * 8;
  if (block_rows == 1) {
    const int64_t all = (int64_t)mats * rows;
    const int64_t per_block = 256 / moe::BlockLanes<V>::kLanes;
    const int64_t blocks = (all * nb + per_block - 1) / per_block;
    moe::quantize_rows_kernel<T, V><<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>((const T*)x, q, scale,
                                                                                              all, cols);
    return launch_status();
  }
  const int64_t tiles = (int64_t)mats * q_blocks(rows) * nb;
  moe::quantize_tiles_kernel<T, V><<<(unsigned)(tiles < most ? tiles : most), 256, 0, s>>>((const T*)x, q, scale,
                                                                                           tiles, rows, cols);
  return launch_status();
}

moe_status launch_quantize(int dtype, int block_rows, int mats, int rows, int cols, const void* x, uint8_t* q,
                           float* scale, cudaStream_t s) {
  if (mats == 0 || rows == 0) return MOE_OK;
  const int v = dtype == MOE_BF16 ? 8 : 4;
  const bool vec = cols % v == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)q % 8 == 0;
  if (dtype == MOE_BF16)
    return vec ? quantize_t<moe::bf16, 8>(block_rows, mats, rows, cols, x, q, scale, s)
               : quantize_t<moe::bf16, 1>(block_rows, mats, rows, cols, x, q, scale, s);
  return vec ? quantize_t<float, 4>(block_rows, mats, rows, cols, x, q, scale, s)
             : quantize_t<float, 1>(block_rows, mats, rows, cols, x, q, scale, s);
}

}  // namespace moe_host
