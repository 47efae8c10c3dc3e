// The residual add fused with RMSNorm and an e4m3 output, and the
// quantisation of matrices to e4m3 (see quant_common.cuh for the scales).
//
// The norm is step a1 of the layer ("Mixture of Experts (MoE)" lesson, "The
// concept / Swapping the FFN": the MoE block reads norm(h) of the residual
// stream, and the block before it has just added to that stream):
//   s  = act(x + residual),  r = fl32(1 / sqrt(mean(s^2) + eps)), mean in fp64,
//   v  = fl32(fl32(s * r) * w),  xn = act(v),  (q, q_scale) from v per 128 columns.
// xn has the bits that moe_route gives for h = s.
#include <algorithm>
#include <type_traits>

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

// Many rows: one block per row (grid-stride), the row s staged
// in shared memory in its own type; every warp takes whole blocks of 128 columns
// in the second pass, so a scale needs no shared memory.  Bound by HBM; few
// registers keep many rows in flight: 8192 rows of 7168 bf16 columns with residual
// and every output move at 5.4 to 5.8 TB/s, the register form below at 4.9 at most.
// SHIFTED (V = 1): rows of odd widths start anywhere, so the first pass takes the
// aligned 16-byte pieces between a row's ends, at the same place of a piece in shared
// memory; x, residual and res_out start alike.  With residual and every output, 2048
// rows of 5003 fp32 columns take 41 us (63 by single elements), 8192 of 1027 bf16 33
// (54).
template <typename T, int V, bool SHIFTED, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) add_rmsnorm_staged_kernel(const T* x, const T* residual, const T* __restrict__ w,
                                                          T* res_out, T* xn, uint8_t* __restrict__ q,
                                                          float* __restrict__ q_scale, int n, int d, float eps) {
  extern __shared__ __align__(16) uint8_t row_raw[];
  T* row = reinterpret_cast<T*>(row_raw);
  __shared__ double part[32];
  __shared__ float r_sh;
  constexpr int LANES = BlockLanes<V>::kLanes, PASSES = BlockLanes<V>::kPasses;
  const int warps = blockDim.x >> 5;
  const int nb = (d + Q_BLOCK - 1) / Q_BLOCK;
  for (int t = blockIdx.x; t < n; t += gridDim.x) {
    const size_t base = (size_t)t * d;
    double acc = 0.0;
    // N elements from element at of the row, kept in shared memory from `to`
    auto first_pass = [&](auto count, int at, T* to) {
      constexpr int N = decltype(count)::value;
      Pack<T, N> s = load_pack<T, N>(x + base + at);
      if (residual != nullptr) {
        const Pack<T, N> b = load_pack<T, N>(residual + base + at);
#pragma unroll
        for (int j = 0; j < N; ++j) s.v[j] = from_f32<T>(__fadd_rn(to_f32(s.v[j]), to_f32(b.v[j])));
      }
      if (res_out != nullptr) store_pack<T, N>(res_out + base + at, s);
      store_pack<T, N>(to, s);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const double f = (double)to_f32(s.v[j]);
        acc += f * f;
      }
    };
    const T* kept = row;
    if constexpr (SHIFTED) {
      constexpr int P = 16 / (int)sizeof(T);
      const int shift = (int)((uintptr_t)(x + base) % 16 / sizeof(T)), end = shift + d;
      kept = row + shift;
      for (int i = threadIdx.x * P; i < end; i += blockDim.x * P) {
        if (i >= shift && i + P <= end) {
          first_pass(std::integral_constant<int, P>(), i - shift, row + i);
        } else {
          for (int j = max(i, shift); j < min(i + P, end); ++j)
            first_pass(std::integral_constant<int, 1>(), j - shift, row + j);
        }
      }
    } else {
      for (int i = threadIdx.x * V; i < d; i += blockDim.x * V)
        first_pass(std::integral_constant<int, V>(), i, row + i);
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
          const Pack<T, V> s = load_pack<T, V>(kept + c), wv = load_pack<T, V>(w + c);
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

// One block per row (grid-stride), the row in registers: LANES lanes hold NBW
// blocks of 128 columns, UNITS apart, so that every sum and every block's largest
// magnitude is a few shuffles away.  For few rows (NBW = 1 spreads a row of up to
// 1024 LANES lanes over one block: latency) and for rows that start unaligned in
// different ways (V = 1).
template <typename T, int V, int NBW>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const T* x, const T* residual, const T* __restrict__ w,
                                                           T* res_out, T* xn, uint8_t* __restrict__ q,
                                                           float* __restrict__ q_scale, int n, int d, float eps) {
  __shared__ double part[32];
  __shared__ float r_sh;
  constexpr int LANES = BlockLanes<V>::kLanes, PASSES = BlockLanes<V>::kPasses;
  const int warps = blockDim.x >> 5;
  const int nb = (d + Q_BLOCK - 1) / Q_BLOCK;
  const int unit0 = threadIdx.x / LANES, units = blockDim.x / LANES;
  const int c0 = (threadIdx.x % LANES) * V;
  for (int t = blockIdx.x; t < n; t += gridDim.x) {
    const size_t base = (size_t)t * d;
    constexpr bool EARLY = NBW == 1;  // few rows: the norm weights are loaded before the sums are joined
    Pack<T, V> s[NBW][PASSES], wv[EARLY ? PASSES : 1];
#pragma unroll
    for (int i = 0; i < NBW; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int c = (unit0 + i * units) * Q_BLOCK + p * (LANES * V) + c0;
        if (c < d) {
          s[i][p] = load_pack<T, V>(x + base + c);
          if (residual != nullptr) {
            const Pack<T, V> b = load_pack<T, V>(residual + base + c);
#pragma unroll
            for (int j = 0; j < V; ++j) s[i][p].v[j] = from_f32<T>(__fadd_rn(to_f32(s[i][p].v[j]), to_f32(b.v[j])));
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) s[i][p].v[j] = from_f32<T>(0.f);
        }
      }
    double acc = 0.0;
#pragma unroll
    for (int i = 0; i < NBW; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int c = (unit0 + i * units) * Q_BLOCK + p * (LANES * V) + c0;
        if (c < d) {
          if (EARLY) wv[p] = load_pack<T, V>(w + c);
          if (res_out != nullptr) store_pack<T, V>(res_out + base + c, s[i][p]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const double f = (double)to_f32(s[i][p].v[j]);
          acc += f * f;
        }
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane_id() == 0) part[warp_id()] = acc;
    __syncthreads();
    if (warp_id() == 0) {
      double sum = lane_id() < warps ? part[lane_id()] : 0.0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane_id() == 0) r_sh = (float)(1.0 / sqrt(sum / (double)d + (double)eps));
    }
    __syncthreads();
    const float r = r_sh;
#pragma unroll
    for (int i = 0; i < NBW; ++i) {
      const int b = unit0 + i * units;
      float v[PASSES][V];
      float m = 0.f;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int c = b * Q_BLOCK + p * (LANES * V) + c0;
        if (c < d) {
          const Pack<T, V> wc = EARLY ? wv[p] : load_pack<T, V>(w + c);
          Pack<T, V> o;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            v[p][j] = __fmul_rn(__fmul_rn(to_f32(s[i][p].v[j]), r), to_f32(wc.v[j]));
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
        const int c = b * Q_BLOCK + p * (LANES * V) + c0;
        if (c < d) store_codes<V>(q + base + c, v[p], inv);
      }
      if (c0 == 0 && b < nb) q_scale[(size_t)t * nb + b] = scale;
    }
  }
}

// The largest magnitude of a pack, NaN aside; bf16 pairs are compared as they are.
template <typename T, int V>
__device__ __forceinline__ float pack_amax(const Pack<T, V>& x) {
  if constexpr (sizeof(T) == 2 && V == 8) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
    __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, fabsf(to_f32(x.v[j])));
    return m;
  }
}

// Blocks of 128 columns that LANES lanes of the row quantisation take at once.
constexpr int Q_UNROLL = 2;

// 1 x 128 blocks: LANES lanes take UNROLL blocks of a row; a thread block takes
// consecutive ones.  A block's two divisions cost as much as its codes when every lane
// does them, so the lanes share the blocks' maxima out (4096 x 14336 bf16: 31 us,
// 5.7 TB/s; all lanes for each block 35.5 us; thread blocks a grid's width apart 43).
// WHOLE: the columns are whole blocks, so block u is the 128 elements from 128 u
// on and no division finds its row.
template <typename T, int V, bool WHOLE>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                            float* __restrict__ scale, int64_t units, int cols) {
  constexpr int LANES = BlockLanes<V>::kLanes, PASSES = BlockLanes<V>::kPasses, UNROLL = Q_UNROLL;
  const int nb = (cols + Q_BLOCK - 1) / Q_BLOCK;
  const int lane = threadIdx.x % LANES;
  const int across = blockDim.x / LANES;  // blocks of 128 columns that the thread block takes at once
  const int64_t u0 = (int64_t)blockIdx.x * across * UNROLL + threadIdx.x / LANES;
  Pack<T, V> s[UNROLL][PASSES];
  int64_t at[UNROLL];  // this lane's first element
  int left[UNROLL];    // columns from there to the row's end
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    const int64_t u = u0 + k * across;
    if (WHOLE) {
      at[k] = u * Q_BLOCK + lane * V;
      left[k] = u < units ? Q_BLOCK : 0;
    } else {
      const int64_t r = u / nb;
      const int c = (int)(u - r * nb) * Q_BLOCK + lane * V;
      at[k] = r * cols + c;
      left[k] = u < units ? cols - c : 0;
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
      if (p * LANES * V < left[k]) s[k][p] = load_pack<T, V>(x + at[k] + p * (LANES * V));
  }
  float m[UNROLL];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    m[k] = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
      if (p * LANES * V < left[k]) m[k] = fmaxf(m[k], pack_amax<T, V>(s[k][p]));
  }
  // the UNROLL maxima together: LANES / UNROLL lanes end up with one of them, whose
  // divisions they do
  int mine = 0;
#pragma unroll
  for (int n = UNROLL / 2, o = LANES / 2; o > 0; n >>= 1, o >>= 1) {
    if (n > 0) {
      const bool upper = lane & o;
      mine += upper ? n : 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = upper ? m[i] : m[i + n], keep = upper ? m[i + n] : m[i];
        m[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
      }
    } else {
      m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    }
  }
  const float my_scale = quant_scale(m[0]);
  const float my_inv = __frcp_rn(my_scale);
  if (lane % (LANES / UNROLL) == 0 && u0 + mine * across < units) scale[u0 + mine * across] = my_scale;
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    const float inv = __shfl_sync(0xffffffffu, my_inv, k * (LANES / UNROLL), LANES);
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
      if (p * LANES * V < left[k]) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = to_f32(s[k][p].v[j]);
        store_codes<V>(q + at[k] + p * (LANES * V), v, inv);
      }
  }
}

// 128 x 128 blocks: a thread block keeps one tile in registers, in its own type,
// between reading it and writing its codes; other blocks of the SM read meanwhile.
// 16-byte bf16 accesses (V = 8): four blocks of 256 threads, 8 x 14336 x 4096 in
// 204 us (6.9 TB/s; 5 blocks 208, 6 283, 3 217, two of 512 threads 272; 217 us on the
// slowest GPU it ran on).  Otherwise two
// blocks of 512, whose tiles need as many registers (8 x 7168 x 2048 fp32 103 us,
// 5.7 TB/s; four of 256 125).
template <int V>
constexpr int kTileThreads = V == 8 ? 256 : 512;
template <int V>
constexpr int kTileBlocks = V == 8 ? 4 : 2;
template <typename T, int V>
__global__ void __launch_bounds__(kTileThreads<V>, kTileBlocks<V>)
    quantize_tiles_kernel(const T* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ scale, int mats, int rows,
                          int cols) {
  constexpr int ACROSS = Q_BLOCK / V;       // threads across a tile row
  constexpr int WARPS = kTileThreads<V> / 32;
  constexpr int STEP = kTileThreads<V> / ACROSS;  // rows per pass
  constexpr int PASSES = Q_BLOCK / STEP;          // 8 (V = 8, 4) or 32 (V = 1)
  __shared__ float part[2][16];
  const int rb = rows / Q_BLOCK + (rows % Q_BLOCK != 0), cb = gridDim.x;
  const int tr = threadIdx.x / ACROSS;
  const int c = blockIdx.x * Q_BLOCK + (threadIdx.x % ACROSS) * V;
  int parity = 0;
  for (int mat = blockIdx.z; mat < mats; mat += gridDim.z)
    for (int br = blockIdx.y; br < rb; br += gridDim.y, parity ^= 1) {
      const size_t at = ((size_t)mat * rows + br * Q_BLOCK + tr) * cols + c;
      const int left = c < cols ? rows - br * Q_BLOCK - tr : 0;  // rows from this thread's first on
      Pack<T, V> s[PASSES];
      float m = 0.f;
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (p * STEP < left) s[p] = load_pack<T, V>(x + at + (size_t)p * STEP * cols);
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (p * STEP < left) m = fmaxf(m, pack_amax<T, V>(s[p]));
      m = lanes_max<32>(m);
      if (lane_id() == 0) part[parity][warp_id()] = m;
      __syncthreads();
      m = lanes_max<WARPS>(part[parity][lane_id() & (WARPS - 1)]);
      const float sc = quant_scale(m);
      const float inv = __frcp_rn(sc);
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (p * STEP < left) {
          float v[V];
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] = to_f32(s[p].v[j]);
          store_codes<V>(q + at + (size_t)p * STEP * cols, v, inv);
        }
      if (threadIdx.x == 0) scale[((size_t)mat * rb + br) * cb + blockIdx.x] = sc;
    }
}

}  // namespace moe

namespace moe_host {

template <typename T, int V>
static moe_status add_rmsnorm_t(const void* x, const void* residual, const void* w, void* res_out, void* xn,
                                uint8_t* q, float* q_scale, int n, int d, float eps, cudaStream_t s) {
  constexpr int LANES = moe::BlockLanes<V>::kLanes;
  const int nb = q_blocks(d);
  const int grid = n < sm_count() * 16 ? n : sm_count() * 16;
  // threads of the register form with nbw blocks of 128 columns per LANES lanes
  auto threads = [&](int nbw) { return ((nb + nbw - 1) / nbw * LANES + 31) / 32 * 32; };
  const bool few = n <= 2 * sm_count() && threads(1) <= 1024;
#define MOE_ADD_RMSNORM(NBW)                                                                                   \
  moe::add_rmsnorm_kernel<T, V, NBW><<<grid, threads(NBW), 0, s>>>((const T*)x, (const T*)residual, (const T*)w, \
                                                                   (T*)res_out, (T*)xn, q, q_scale, n, d, eps)
  // unaligned rows that start alike in x, residual and res_out
  auto alike = [&](const void* p) { return p == nullptr || ((uintptr_t)p - (uintptr_t)x) % 16 == 0; };
  const bool shifted = V == 1 && alike(residual) && alike(res_out) && (uintptr_t)x % sizeof(T) == 0;
  if (few) {
    MOE_ADD_RMSNORM(1);
  } else if (V == 1 && !shifted) {
    if constexpr (V == 1) {
      if (threads(4) <= 1024) MOE_ADD_RMSNORM(4);
      else MOE_ADD_RMSNORM(12);  // d up to 49152
    }
  } else {
    constexpr int P = 16 / (int)sizeof(T);
    const int smem = (int)((size_t)(d + (V == 1 ? P : 0)) * sizeof(T));
    const int blocks = std::max(1, 220 * 1024 / smem);  // that an SM holds
    auto launch = [&](auto kernel, SmemLimit& lim, int threads) -> moe_status {
      const moe_status st = ensure_smem_limit(kernel, smem, lim);
      if (st != MOE_OK) return st;
      kernel<<<grid, threads, smem, s>>>((const T*)x, (const T*)residual, (const T*)w, (T*)res_out, (T*)xn, q, q_scale,
                                         n, d, eps);
      return MOE_OK;
    };
    static SmemLimit lim_short, lim_long;
    // Short rows: about four passes over the row by 64 to 192 threads, up to 256 where an
    // SM holds seven rows or fewer (4096 rows of 14336 bf16 columns with residual 94 us,
    // 110 with 192; 8192 of 7168, where it holds 15, 91 and 105 with 256).  Long ones, of
    // which it holds four at most: 1024 threads an SM (512 rows of 40001 fp32 columns
    // 94 us, 289 with 192 threads; 1024 of 16384 80 and 97).
    const int passes = std::min(192, std::max(64, (d / P + 127) / 128 * 32));
    const moe_status st =
        blocks > 4 ? launch(moe::add_rmsnorm_staged_kernel<T, V, V == 1, 256>, lim_short,
                            std::max(passes, std::min(256, 1792 / blocks / 32 * 32)))
                   : launch(moe::add_rmsnorm_staged_kernel<T, V, V == 1, 1024>, lim_long, 1024 / blocks / 32 * 32);
    if (st != MOE_OK) return st;
  }
#undef MOE_ADD_RMSNORM
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
  if (block_rows == 1) {
    const int64_t units = (int64_t)mats * rows * nb;
    const bool whole = V > 1 && cols % moe::Q_BLOCK == 0;
    const int64_t per_block = 256 / moe::BlockLanes<V>::kLanes * moe::Q_UNROLL;
    const int64_t blocks = (units + per_block - 1) / per_block;
    if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
    if (whole)
      moe::quantize_rows_kernel<T, V, true><<<(unsigned)blocks, 256, 0, s>>>((const T*)x, q, scale, units, cols);
    else
      moe::quantize_rows_kernel<T, V, false><<<(unsigned)blocks, 256, 0, s>>>((const T*)x, q, scale, units, cols);
    return launch_status();
  }
  const dim3 grid((unsigned)nb, (unsigned)std::min(q_blocks(rows), 65535), (unsigned)std::min(mats, 65535));
  moe::quantize_tiles_kernel<T, V><<<grid, moe::kTileThreads<V>, 0, s>>>((const T*)x, q, scale, mats, rows, cols);
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
