// Grouped product of e4m3 operands with block scales on SM pairs
// (tcgen05.mma.cta_group::2.kind::f8f6f4):
//   C[r][n] = sum_kb sa[r][kb] * sb[g][n / 128][kb] * sum_{k in kb} A[r][k] * B[g][n][k]
// for the rows r of group (expert) g, kb running over blocks of 128 columns.
// Epilogues: bf16 or fp32 results, or for the experts' gate and up projections
//   t = silu(gate) * up  in fp32, quantised per row and 128 hidden units.
//
// Scales.  They change every 128 columns, so every k-block of 128 gets its own
// accumulator in one of two 256-column TMEM slots, and eight epilogue warps per
// CTA add it, times its scales, to fp32 sums in registers: 128 of them per
// thread, acc += v * (sa * sb) as packed pairs.  Two warps beside the producer
// and the MMA issuer form the products sa * sb, their inputs loaded two k-blocks
// ahead, and complete the same barrier as the accumulator.  An epilogue warp
// loads its next 16 columns, across k-blocks too, before it adds the last ones.
//
// Two tilings (template parameter WIDE):
//   wide    256 rows of a group on the MMA's M side, 256 weight rows on its N side.
//           A TMEM lane is a row, so a thread's scale is one number and the
//           accumulator is read in the fast 32x32b shape.
//   swapped 256 weight rows on M, a chunk of up to 256 rows, padded to 16, on N (a
//           group of m rows is cut into ceil(m / 256) equal chunks): no work for
//           rows that are not there.  A lane is a weight row and the scales differ
//           by column; in the 16x256b shape (lane l holds rows l / 4 and l / 4 + 8,
//           columns 2 (l % 4) and + 1 of every eight) one product read from shared
//           memory serves four values.
// Measured on B200, the reads and additions of a 256 x 256 k-block of a pair take the
// epilogue about 460 cycles in the 32x32b shape and 980 in the 16x256b shape (which
// moves half as much per access), and its MMAs 512.  A whole wide k-block takes 0.42 us
// (735 cycles) with one tile per pair and about 900 cycles in large calls, not the 512
// that two slots would allow; which hand-over costs the rest has not been measured.
//
// Gate and up.  One view over both matrices (their distance is a stride)
// interleaves them in shared memory, eight gate rows, eight up rows, so a thread
// holds both values of a hidden unit and the activation needs no exchange.  A
// pair's tile is 128 hidden units, one block of the result's scales: only each
// row's largest magnitude crosses between warps (wide) or CTAs (swapped).
//
// Roles (384 threads per CTA, clusters of two; the register file is split
// between the roles with setmaxnreg):
//   warp 0      TMA producer in both CTAs; 3-stage ring of 64 KiB, two k-blocks
//               per stage and (K % 128 == 0) one load per operand and stage;
//   warp 1      TMEM allocation; in the even CTA it issues the MMAs;
//   warps 2, 3  scale products, one warp per TMEM slot;
//   warps 4-11  epilogue: warp w holds TMEM lanes 32 (w % 4) .. + 31 and one half
//               of the tile's columns.
// Few tiles (a handful of rows): chunks get smaller, or each tile is cut along K
// into `splits` parts, so that the weights stream through all SMs; the parts' fp32
// sums meet in the workspace and the pair that comes last adds them in order and
// writes the result.
// Tiles run group by group, a group's chunks in runs of eight per weight tile,
// and are claimed from a counter in the workspace header that the last pair to
// finish sets back to zero.  Data that crosses to the other CTA travels by
// st.async; no TMA load uses cluster multicast.  Every wait is bounded: on
// time-out the block records MOE_ERR_DEVICE_TIMEOUT, stops issuing work, drains
// and returns.
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "gemm_fp8_kernels.h"
#include "quant_common.cuh"
#include "tcgen05_pair.cuh"

namespace moe {

constexpr int F_BK = 128;                             // k-block: 128 e4m3 codes, one 128-byte swizzle row
constexpr int F_KB = 2;                               // k-blocks per stage
constexpr int F_STAGES = 3;
constexpr int F_KBLK_BYTES = 128 * F_BK;              // one k-block of 128 rows: 16 KiB
constexpr int F_W_BYTES = F_KB * F_KBLK_BYTES;        // this CTA's 128 weight rows
constexpr int F_STAGE_BYTES = 2 * F_W_BYTES;          // and up to 128 rows of the chunk
constexpr int F_THREADS = 384;
constexpr int F_EPI_WARP0 = 4, F_EPI_WARPS = 8;
constexpr int F_CHUNK = 256;                          // most rows of a group in one tile (swapped: Fp8Args::chunk)
constexpr int F_RUN = 8;                              // chunks that walk a group's weight tiles together
constexpr int F_XMAPS = 16;                           // row boxes of 8, 16, ..., 128 rows
constexpr int F_TRING = 8;
constexpr int F_SLOTS = 2;                            // rows of scale products, one per TMEM slot
// readers of a published tile index: even CTA: MMA, 2 scale and 8 epilogue
// warps; odd CTA: producer, 2 and 8
constexpr int F_TRING_READERS = 22;
// Rows a group, on average over max_rows (the host knows no more), from which on the
// wide tiling is taken.  It reads its accumulators faster but works on 256 rows whatever
// a group has: of groups of 256 rows on average, half have a second tile of a few rows.
// With nearly even groups, expert FFN of 7168 x 2048 (or
// 4096 x 14336) in a steady loop, wide against swapped: 128 rows a group 507 and
// 461 us, 141 rows 1002 and 948, 256 rows 5464 and 5482 (both at the power limit),
// 1024 rows 1939 and 2290.
constexpr int F_WIDE_ROWS = 256;
constexpr int F_OUT_PITCH = 80;                       // bytes per row of a warp's output block of 64-byte rows
constexpr int F_OUT_BYTES = 16 * F_OUT_PITCH;         // swapped: 16 rows of 32 bf16
constexpr int F_OUT_WIDE_BYTES = 2048;                // wide: 16 rows of 128 bytes, or 32 of 64
// Words of the workspace header (0-3: the error record, 32: the bf16 products' tile
// counter): tiles claimed, pairs finished, and the finished parts of up to 50 cut
// tiles, all of which every launch leaves at zero.  They are in the header, which no
// other call of the library uses as scratch.
constexpr int F_CLAIM_WORD = 40, F_DONE_WORD = 41;
constexpr int F_SPLIT_TILES = 50;
__host__ __device__ constexpr int f8_split_word(int tile) { return tile < 28 ? 4 + tile : 14 + tile; }
static_assert(f8_split_word(27) < 32 && f8_split_word(28) > F_DONE_WORD &&
                  f8_split_word(F_SPLIT_TILES - 1) < (int)kHeaderBytes / 4,
              "counters inside the header, apart from its other words");

// Rows of scale products per slot of 256 (swapped), and floats of a slot.
template <int EPI, bool WIDE>
constexpr int f8_mats() {
  return EPI == moe_host::EPI_SWIGLU && !WIDE ? 2 : 1;
}
template <int EPI, bool WIDE>
constexpr int f8_smem_bytes() {
  return F_STAGES * F_STAGE_BYTES + F_SLOTS * f8_mats<EPI, WIDE>() * F_CHUNK * 4 +
         (WIDE ? F_EPI_WARPS * F_OUT_WIDE_BYTES : EPI == moe_host::EPI_STORE ? F_EPI_WARPS * F_OUT_BYTES : 0) +
         1024;  // + alignment slack
}

struct Fp8Maps {
  CUtensorMap w, ws;       // routed and shared weights
  CUtensorMap x[F_XMAPS];  // the rows: x[i] has boxes of 8 (i + 1) rows
  CUtensorMap xs[F_XMAPS]; // the shared group's rows when they come from their own tensor
};

struct Fp8Args {
  const int32_t* offsets;  // [G+1] device, or nullptr: one group of max_rows rows
  int groups, max_rows;
  int nout;                // output columns per group
  int nk;                  // k-blocks
  int splits;              // parts that a tile's k-blocks are cut into
  unsigned split_magic;    // floor(2^32 / splits) + 1: its high product with an index is the index / splits
  int split_nk, split_rem; // k-blocks per part, one more in the first split_rem parts
  float4* partial;         // [tiles][splits][2][partial_vecs][256]
  int partial_vecs;        // float4 per thread and part
  int n_o;                 // weight tiles per group
  int chunk;               // most rows of a group in one tile: F_CHUNK, less (swapped) where there are few tiles
  int view;                // 1: the maps bring two k-blocks per load (K % 128 == 0)
  int nnb;                 // scale blocks along n
  const float *as, *sas;               // row scales, and those of the shared group's own rows
  const float *bs[2], *sbs[2];         // weight scales, in the order of the matrices in a tile
  int up_first, s_up_first;            // SwiGLU: the up matrix comes first in a tile (it lies lower in memory)
  void* c;
  float* c_scale;
  int vec;                 // 1: rows of C are whole, aligned 16-byte pieces
  int shared_group, shared_a;
  int32_t* hdr;
  uint64_t wait_ns;
};

enum { F_SITE_RING = 8, F_SITE_SCALE = 9, F_SITE_AMAX = 10, F_SITE_SPLIT = 11 };

// ---- tiles --------------------------------------------------------------------
struct Fp8Tile {
  int group, row0, rows, half, o;  // rows [row0, row0 + rows) of C; half: rows that each CTA loads; weight tile o
  int kb0, nk;                     // k-blocks kb0 .. kb0 + nk - 1
  int index, part;                 // of the tile, its parts together; which of them
};

// (chunk is a power of two)
__device__ __forceinline__ int f8_chunks(int m, int chunk) { return (m + chunk - 1) >> (31 - __clz(chunk)); }

// One warp: prefix[g] = first tile of group g (n_o tiles per chunk).
__device__ __forceinline__ void f8_prefix(const int* offs, int* prefix, int groups, int n_o, int chunk) {
  const int lane = lane_id();
  int carry = 0;
  for (int base = 0; base < groups; base += 32) {
    const int g = base + lane;
    const int v = g < groups ? f8_chunks(offs[g + 1] - offs[g], chunk) * n_o : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (g < groups) prefix[g] = carry + x - v;
    carry += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) prefix[groups] = carry;
}

// Swapped tiles divide integers only where a group has several chunks: a decode is on
// the way of a call's first load.
template <bool WIDE, bool SPLIT>
__device__ __forceinline__ Fp8Tile f8_decode(int t, const int* prefix, const int* offs, const Fp8Args& args) {
  Fp8Tile tl;
  tl.part = 0;
  tl.kb0 = 0;
  tl.nk = args.nk;
  if constexpr (SPLIT) {  // at least two parts
    const int index = (int)__umulhi((unsigned)t, args.split_magic);
    tl.part = t - index * args.splits;
    tl.kb0 = tl.part * args.split_nk + min(tl.part, args.split_rem);
    tl.nk = args.split_nk + (tl.part < args.split_rem ? 1 : 0);
    t = index;
  }
  tl.index = t;
  int lo = 0, hi = args.groups - 1;  // last g with prefix[g] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int m = offs[lo + 1] - offs[lo];
  const int ch = f8_chunks(m, args.chunk);
  const int local = t - prefix[lo];
  int c = 0, nc = WIDE ? F_CHUNK : (m + 15) & ~15;
  tl.o = local;
  if (WIDE || ch > 1) {
    if (!WIDE) nc = ((m + ch - 1) / ch + 15) & ~15;
    const int run = local / (args.n_o * F_RUN);
    const int rem = local - run * args.n_o * F_RUN;
    const int in_run = min(F_RUN, ch - run * F_RUN);
    tl.o = rem / in_run;
    c = run * F_RUN + rem - tl.o * in_run;
  }
  tl.group = lo;
  tl.row0 = offs[lo] + c * nc;
  tl.rows = max(0, min(nc, m - c * nc));
  tl.half = WIDE ? min(128, max(8, (tl.rows + 7) & ~7)) : max(8, ((tl.rows + 15) & ~15) >> 1);
  return tl;
}

// ---- waits --------------------------------------------------------------------
__device__ __forceinline__ bool f8_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One thread's bounded wait; CLUSTER: a barrier that the other CTA arrives on.
template <bool CLUSTER>
__device__ __forceinline__ bool f8_wait(uint64_t* bar, uint32_t parity, const Fp8Args& a, volatile int* abort,
                                        int site) {
  auto poll = [&] { return CLUSTER ? f8_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (poll()) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t polls = 1;; ++polls) {
    if (poll()) return true;
    if ((polls & 63u) == 0u) {
      if (*abort) return false;
      if (global_timer_ns() - t0 >= a.wait_ns) {
        record_error(a.hdr, MOE_ERR_DEVICE_TIMEOUT, KID_GEMM_FP8, blockIdx.x, site);
        *abort = 1;
        return false;
      }
    }
  }
}

// Every lane waits; true when all of them saw the phase complete.
template <bool CLUSTER>
__device__ __forceinline__ bool f8_warp_wait(uint64_t* bar, uint32_t parity, const Fp8Args& a, volatile int* abort,
                                             int site) {
  bool ok = CLUSTER ? f8_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  if (__builtin_expect(__all_sync(0xffffffffu, ok), 1)) return true;
  ok = f8_wait<CLUSTER>(bar, parity, a, abort, site);
  return __all_sync(0xffffffffu, ok);
}

// mbar_arrive_expect_tx_cluster with a release: what this thread has done and observed
// so far (an acquired count, with all that it stands for) is passed on to the waiters.
__device__ __forceinline__ void f8_arrive_expect_tx_release(uint32_t bar_cluster, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar_cluster),
               "r"(bytes)
               : "memory");
}

// ---- TMA, MMA and TMEM ----------------------------------------------------------
__device__ __forceinline__ void f8_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  tma_load_2d_pair(dst, map, bar, c0, c1);
}
__device__ __forceinline__ void f8_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void f8_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(0), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void f8_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%3, %3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(c3), "r"(c4)
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 operands, fp32 accumulation, K = 32.
template <int ACCUMULATE>
__device__ __forceinline__ void f8_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "n"(ACCUMULATE)
      : "memory");
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// Instruction descriptor, kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A and B
// e4m3 (bits 7-9 and 10-12 = 0), both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
constexpr uint32_t f8_idesc(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// 16 TMEM lanes x 16 columns: register 4 j + i of lane l holds row l / 4 + 8 (i / 2),
// column 8 j + 2 (l % 4) + i % 2.
#define MOE_TMEM_LD16x16(taddr, r)                                                                                 \
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"                    \
               : "=r"((r)[0]), "=r"((r)[1]), "=r"((r)[2]), "=r"((r)[3]), "=r"((r)[4]), "=r"((r)[5]), "=r"((r)[6]), \
                 "=r"((r)[7])                                                                                      \
               : "r"(taddr))

// 32 TMEM lanes (lane l = TMEM lane l) x 16 columns.
#define MOE_TMEM_LD32x16(taddr, r)                                                                                 \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "   \
               "%13, %14, %15}, [%16];"                                                                            \
               : "=r"((r)[0][0]), "=r"((r)[0][1]), "=r"((r)[0][2]), "=r"((r)[0][3]), "=r"((r)[0][4]),              \
                 "=r"((r)[0][5]), "=r"((r)[0][6]), "=r"((r)[0][7]), "=r"((r)[1][0]), "=r"((r)[1][1]),              \
                 "=r"((r)[1][2]), "=r"((r)[1][3]), "=r"((r)[1][4]), "=r"((r)[1][5]), "=r"((r)[1][6]),              \
                 "=r"((r)[1][7])                                                                                   \
               : "r"(taddr))

// Waits for this thread's TMEM loads; the registers pass through it, so no use of them can move above it.
__device__ __forceinline__ void f8_tmem_wait(uint32_t (&v)[2][8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i >> 3][i & 7]));
}

__device__ __forceinline__ uint64_t pack64(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack64(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
// two fp32 FMAs, each rounded once
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

// Place of column c (0 .. 127) of a half in a row of scale products: the four
// values that a lane takes for two groups of eight columns lie together.
__device__ __forceinline__ int f8_scale_at(int c) {
  return (c & ~15) + ((c & 6) << 1) + ((c & 8) >> 2) + (c & 1);
}

// silu(g) * u in fp32, silu(g) = g / (1 + e^-g): the full exponential and a division
// that are each off by at most 2 ulp.  (The rounded division made the FFN 3 to 14 %
// slower; a bare ex2.approx saves 1 % but is off by 28 ulp near g = -80, where its
// argument is rounded.)  Below g = -87.3 the division gives 0, as silu does to 1e-36.
__device__ __forceinline__ float f8_silu_mul(float g, float u) {
  return __fmul_rn(__fdividef(g, 1.f + expf(-g)), u);
}

// Byte transpose over the four lanes l, l ^ 4, l ^ 8, l ^ 12: lane i = (l / 4) % 4
// of them gets byte i of every lane's word, in lane order.
__device__ __forceinline__ uint32_t f8_transpose_bytes(uint32_t w) {
  const bool b0 = lane_id() & 4, b1 = lane_id() & 8;
  // trade 16-bit halves with the lane two apart, then bytes with the neighbour
  uint32_t p = __shfl_xor_sync(0xffffffffu, w, 8);
  w = b1 ? __byte_perm(w, p, 0x3276) : __byte_perm(w, p, 0x5410);
  p = __shfl_xor_sync(0xffffffffu, w, 4);
  return b0 ? __byte_perm(w, p, 0x3715) : __byte_perm(w, p, 0x6240);
}

// What the main loop of an epilogue warp needs, set up once; barriers and scales as shared-memory addresses.
struct Fp8Drain {
  uint32_t tmem;            // this warp's lanes of slot 0
  uint32_t tempty_remote;   // the even CTA's tempty_bar[0]
  uint32_t tfull, sempty;   // this CTA's barriers of slot 0
  uint32_t scales;          // this lane's first scale product of slot 0
  uint32_t slot, phase;     // slot of the next k-block, and its tfull's phase
};

__device__ __forceinline__ uint32_t ld_shared(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void ld_shared_2x64(uint32_t at, uint64_t (&v)[2]) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(at) : "memory");
}

// Whether the phase has completed, for every lane; without waiting.
__device__ __forceinline__ bool f8_ready(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

__device__ __forceinline__ bool f8_wait_at(uint32_t bar, uint32_t phase, const Fp8Args& args, volatile int* abort,
                                           int site) {
  if (__builtin_expect(f8_ready(bar, phase), 1)) return true;
  return f8_warp_wait<false>(reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(bar)), phase, args, abort, site);
}

// Waits for the accumulator and the scale products of the next k-block.
__device__ __forceinline__ bool f8_next_full(const Fp8Drain& d, const Fp8Args& args, volatile int* abort) {
  if (!f8_wait_at(d.tfull + d.slot * 8u, d.phase, args, abort, SITE_TMEM_FULL)) return false;
  tc_fence_after();
  return true;
}

// Hands the slot back: its accumulator and scale products have been read.
__device__ __forceinline__ void f8_release(const Fp8Drain& d, uint32_t slot) {
  tc_fence_before();
  __syncwarp();
  if (lane_id() == 0) {
    mbar_arrive_cluster_relaxed(d.tempty_remote + slot * 8u);
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(d.sempty + slot * 8u) : "memory");
  }
}

// Adds the k-blocks of one tile to acc[16 columns][16 lanes][8 columns][rows
// l / 4, + 8] (pairs of columns).  NB batches of 16 columns from column col0 of
// the slot.  Every lane calls it; false after a failed wait.
template <int NB, int MATS>
__device__ __forceinline__ bool f8_accumulate(uint64_t (&acc)[8][2][2][2], Fp8Drain& d, int col0, int nk,
                                              const Fp8Args& args, volatile int* abort) {
  uint32_t v[2][2][8];
  auto load = [&](uint32_t slot, int b, uint32_t (&r)[2][8]) {
    const uint32_t at = d.tmem + slot * 256u + (uint32_t)(col0 + b * 16);
    MOE_TMEM_LD16x16(at, r[0]);
    MOE_TMEM_LD16x16(at + (16u << 16), r[1]);
  };
  if (!f8_next_full(d, args, abort)) return false;
  load(d.slot, 0, v[0]);
  // one k-block whose first batch is on its way into v[P]
  auto step = [&](auto first, bool more) -> bool {
    constexpr int P = decltype(first)::value;
    const uint32_t slot = d.slot;
    const uint32_t sc = d.scales + slot * (MATS * F_CHUNK * 4);
    uint64_t s[2][2][2];  // scale products of two batches
    auto scales = [&](int b) {
      ld_shared_2x64(sc + b * 64, s[b & 1][0]);
      if (MATS == 2) ld_shared_2x64(sc + F_CHUNK * 4 + b * 64, s[b & 1][1]);
    };
    scales(0);
    d.slot ^= 1u;
    d.phase ^= d.slot ^ 1u;
    bool ready = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t(&r)[2][8] = v[(P + b) & 1];
      if (b + 1 < NB) scales(b + 1);
      // the next k-block is usually there by now: asked before the last batch is awaited
      if (b + 1 == NB) ready = more && f8_ready(d.tfull + d.slot * 8u, d.phase);
      f8_tmem_wait(r);
      if (b + 1 < NB) {
        load(slot, b + 1, v[(P + b + 1) & 1]);
      } else {
        f8_release(d, slot);
        if (more) {
          if (!ready && !f8_next_full(d, args, abort)) return false;
          tc_fence_after();
          load(d.slot, 0, v[(P + b + 1) & 1]);
        }
      }
#pragma unroll
      for (int l16 = 0; l16 < 2; ++l16)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t* q = s[b & 1][MATS == 2 ? h : 0];
          fma2(acc[b][l16][0][h], pack64(r[l16][2 * h], r[l16][2 * h + 1]), q[0]);
          fma2(acc[b][l16][1][h], pack64(r[l16][4 + 2 * h], r[l16][5 + 2 * h]), q[1]);
        }
    }
    return true;
  };
  for (int kb = 0; kb < nk; kb += 2) {
    if (!step(std::integral_constant<int, 0>(), kb + 1 < nk)) return false;
    if (kb + 1 < nk && !step(std::integral_constant<int, NB & 1>(), kb + 2 < nk)) return false;
  }
  return true;
}

// The wide tiling: acc[16 columns][pairs], lane = row, columns col0 .. + 127.
// (Single FMAs: packed ones measured 3 % slower here.)
// SWIGLU: of every 16 columns the first eight belong to the tile's first matrix.
template <bool SWIGLU>
__device__ __forceinline__ bool f8_accumulate_wide(uint64_t (&acc)[8][8], Fp8Drain& d, int col0, int nk,
                                                   const Fp8Args& args, volatile int* abort) {
  uint32_t v[2][2][8];
  auto load = [&](uint32_t slot, int b, uint32_t (&r)[2][8]) {
    MOE_TMEM_LD32x16(d.tmem + slot * 256u + (uint32_t)(col0 + b * 16), r);
  };
  if (!f8_next_full(d, args, abort)) return false;
  load(d.slot, 0, v[0]);
  auto step = [&](auto last) -> bool {
    constexpr bool MORE = decltype(last)::value;
    const uint32_t slot = d.slot;
    const float s0 = __uint_as_float(ld_shared(d.scales + slot * (F_CHUNK * 4)));
    const float s1 = SWIGLU ? __uint_as_float(ld_shared(d.scales + slot * (F_CHUNK * 4) + 512)) : s0;
    d.slot ^= 1u;
    d.phase ^= d.slot ^ 1u;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      uint32_t(&r)[2][8] = v[b & 1];
      f8_tmem_wait(r);
      if (b < 7) {
        load(slot, b + 1, v[(b + 1) & 1]);
      } else {
        f8_release(d, slot);
        if (MORE) {
          if (!f8_next_full(d, args, abort)) return false;
          load(d.slot, 0, v[0]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 x = unpack64(acc[b][i]), y = unpack64(acc[b][4 + i]);
        x.x = __fmaf_rn(__uint_as_float(r[0][2 * i]), s0, x.x);
        x.y = __fmaf_rn(__uint_as_float(r[0][2 * i + 1]), s0, x.y);
        y.x = __fmaf_rn(__uint_as_float(r[1][2 * i]), s1, y.x);
        y.y = __fmaf_rn(__uint_as_float(r[1][2 * i + 1]), s1, y.y);
        acc[b][i] = pack64(__float_as_uint(x.x), __float_as_uint(x.y));
        acc[b][4 + i] = pack64(__float_as_uint(y.x), __float_as_uint(y.y));
      }
    }
    return true;
  };
  for (int kb = 1; kb < nk; ++kb)
    if (!step(std::true_type())) return false;
  return step(std::false_type());
}

// A warp whose rows are not in the tile: it only hands the slots back.
__device__ __forceinline__ bool f8_pass_over(Fp8Drain& d, int nk, const Fp8Args& args, volatile int* abort) {
  for (int kb = 0; kb < nk; ++kb) {
    if (!f8_next_full(d, args, abort)) return false;
    f8_release(d, d.slot);
    d.slot ^= 1u;
    d.phase ^= d.slot ^ 1u;
  }
  return true;
}

// Writes BYTES (w) of each of the warp's 32 rows, lane = row, to C: row r at
// c + r * ld, `valid` rows, of which the first `bytes` bytes exist.  Through the
// warp's block of shared memory (16 rows of 128 bytes at a time, or 32 of 64), so
// that the stores write whole 128-byte lines: they go out by the line, and 64-byte
// pieces of eight rows per instruction took about twice as long.
// vec: c, ld and bytes are multiples of 16; else elements of ES bytes.
template <int ES, int BYTES>
__device__ __forceinline__ void f8_store_rows(uint8_t* block, const uint4 (&w)[BYTES / 16], uint8_t* c, size_t ld,
                                              int valid, int bytes, bool vec) {
  constexpr int ROWS = F_OUT_WIDE_BYTES / BYTES, PIECES = BYTES / 16;
  const int lane = lane_id();
  // 16-byte piece i of a row lies where no two of eight rows meet in a bank
  auto at = [&](int r, int i) {
    return block + r * BYTES + ((BYTES == 128 ? i ^ (r & 7) : i ^ ((r >> 1) & 3)) << 4);
  };
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += ROWS) {
    __syncwarp();
    if (lane >= r0 && lane < r0 + ROWS) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) *reinterpret_cast<uint4*>(at(lane - r0, i)) = w[i];
    }
    __syncwarp();
    if (vec) {
#pragma unroll
      for (int i = 0; i < ROWS * PIECES / 32; ++i) {
        const int r = i * (32 / PIECES) + lane / PIECES, p = lane % PIECES;
        const uint4 q = *reinterpret_cast<const uint4*>(at(r, p));
        if (r0 + r < valid && p * 16 < bytes) *reinterpret_cast<uint4*>(c + (size_t)(r0 + r) * ld + p * 16) = q;
      }
    } else if constexpr (ES > 1) {
      using T = typename std::conditional<ES == 4, float, bf16>::type;
      constexpr int COLS = BYTES / ES;
      for (int i = lane; i < ROWS * COLS; i += 32) {
        const int r = i / COLS, b = (i % COLS) * ES;
        if (r0 + r < valid && b < bytes)
          *reinterpret_cast<T*>(c + (size_t)(r0 + r) * ld + b) = *reinterpret_cast<const T*>(at(r, b / 16) + b % 16);
      }
    }
  }
}

// SPLIT: tiles (swapped) are cut along K into args.splits parts.
template <int EPI, bool WIDE, bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(F_THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ Fp8Maps maps, const Fp8Args args) {
  constexpr bool SWIGLU = EPI == moe_host::EPI_SWIGLU;
  constexpr int MATS = f8_mats<EPI, WIDE>();
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[F_STAGES];   // used in the even CTA
  __shared__ __align__(8) uint64_t empty_bar[F_STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];        // used in the even CTA
  __shared__ __align__(8) uint64_t sempty_bar[F_SLOTS];  // the slot's scale products have been read
  __shared__ __align__(8) uint64_t amax_bar;             // SwiGLU: every warp's magnitudes are in amax_sh
  __shared__ __align__(8) uint64_t peer_bar[2];          //         the other CTA's have arrived
  __shared__ __align__(8) uint64_t inv_bar;              //         1 / scale of every row is in inv_sh
  __shared__ __align__(8) uint64_t split_bar;            // every warp's part of a cut tile is in the workspace
  __shared__ __align__(8) uint64_t pair_bar;             // ... the odd CTA's too (even CTA)
  __shared__ __align__(8) uint64_t done_bar;             // last_sh is there
  __shared__ volatile int last_sh;
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ __align__(8) uint64_t tr_full[F_TRING];     // a tile index is in tile_ring[j] (both CTAs)
  __shared__ __align__(8) uint64_t tr_empty[F_TRING];    // every reader has taken it (even CTA)
  __shared__ volatile int tile_ring[F_TRING];
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ int offs_sh[TC_MAX_GROUPS + 1];
  __shared__ int prefix_sh[TC_MAX_GROUPS + 1];
  __shared__ unsigned amax_sh[SWIGLU && !WIDE ? F_CHUNK : 1];
  __shared__ volatile float peer_sh[SWIGLU && !WIDE ? 2 : 1][SWIGLU && !WIDE ? F_CHUNK : 1];
  __shared__ __align__(16) float inv_sh[SWIGLU && !WIDE ? F_CHUNK : 4];
  __shared__ __align__(8) uint64_t half_bar[4];          // SwiGLU, wide: both halves of a quarter's rows are in half_sh
  __shared__ float half_sh[SWIGLU && WIDE ? 2 : 1][2][128];

  const int warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int first = (int)cluster_index(), step = (int)cluster_count();
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t smem_base = smem_u32(smem);
  float* scale_ring = reinterpret_cast<float*>(smem + F_STAGES * F_STAGE_BYTES);  // [F_SLOTS][MATS][2][128]

  const int G = args.groups;
  for (int i = threadIdx.x; i <= G; i += blockDim.x)
    offs_sh[i] = args.offsets ? args.offsets[i] : (i == 0 ? 0 : args.max_rows);
  if constexpr (SWIGLU && !WIDE)
    for (int i = threadIdx.x; i < F_CHUNK; i += blockDim.x) amax_sh[i] = 0u;
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  if (warp == 0) f8_prefix(offs_sh, prefix_sh, G, args.n_o, args.chunk);
  if (threadIdx.x == 32) {
    for (int s = 0; s < F_STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 2);  // the MMA's commit and the slot's scale warp
      mbar_init(&tempty_bar[b], 2 * F_EPI_WARPS);
      mbar_init(&sempty_bar[b], F_EPI_WARPS);
      mbar_init(&peer_bar[b], 1);
    }
    mbar_init(&amax_bar, F_EPI_WARPS);
    mbar_init(&inv_bar, F_EPI_WARPS);
    mbar_init(&split_bar, F_EPI_WARPS);
    mbar_init(&pair_bar, 1);
    mbar_init(&done_bar, 1);
    for (int q = 0; q < 4; ++q) mbar_init(&half_bar[q], 2);
    for (int j = 0; j < F_TRING; ++j) {
      mbar_init(&tr_full[j], 1);
      mbar_init(&tr_empty[j], F_TRING_READERS);
    }
    mbar_init(&drain_bar, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(TC_TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before either signals the other
  tc_fence_after();
  // A launch that follows its rows' producer directly (Fp8Gemm::follows) may get this
  // far while that kernel still runs.  From here on memory is read that it writes.
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const uint32_t tmem_base = tmem_base_sh;
  const int total_tiles = prefix_sh[G] * (SPLIT ? args.splits : 1);

  // the next published tile index, for a role of one warp (every lane calls) or one thread
  auto take_warp = [&](int& rs, uint32_t& rph, int& t) -> bool {
    if (!f8_warp_wait<true>(&tr_full[rs], rph, args, &abort_flag, F_SITE_RING)) return false;
    t = tile_ring[rs];
    const uint32_t z = depend_zero((uint32_t)t);  // every lane's read has returned ...
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(&tr_empty[rs], 0) + z);  // ... before the slot is freed
    if (++rs == F_TRING) {
      rs = 0;
      rph ^= 1u;
    }
    return true;
  };

  if (warp < F_EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // ======================= TMA producer (both CTAs) =======================
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        long issued = 0;
        tma_prefetch_map(&maps.w);
        bool ok = true;
        // The even CTA's producer claims tiles and publishes their indices (and
        // finally one past the last) to every role of both CTAs; a tile's
        // successor is published right after the tile's first stage is issued.
        int rs = 0;
        uint32_t rph = 0;
        auto publish = [&](int v) -> bool {
          if (!f8_wait<true>(&tr_empty[rs], rph ^ 1u, args, &abort_flag, F_SITE_RING)) return false;
          tile_ring[rs] = v;
          mbar_arrive(&tr_full[rs]);
          const uint32_t peer_full = map_to_rank(&tr_full[rs], 1);
          mbar_arrive_expect_tx_cluster(peer_full, 4);
          st_async_b32(map_to_rank((const void*)&tile_ring[rs], 1), (uint32_t)v, peer_full);
          if (++rs == F_TRING) {
            rs = 0;
            rph ^= 1u;
          }
          return true;
        };
        auto take = [&](int& v) -> bool {
          if (!f8_wait<true>(&tr_full[rs], rph, args, &abort_flag, F_SITE_RING)) return false;
          v = tile_ring[rs];
          mbar_arrive_cluster_relaxed(map_to_rank(&tr_empty[rs], 0) + depend_zero((uint32_t)v));
          if (++rs == F_TRING) {
            rs = 0;
            rph ^= 1u;
          }
          return true;
        };
        // (no tiles to claim where every pair has at most one)
        const bool claims = total_tiles > step;
        auto claim = [&]() -> int { return claims ? step + atomicAdd(args.hdr + F_CLAIM_WORD, 1) : total_tiles; };
        int t = first;
        int pending = 0;  // even CTA: the claimed successor of the next tile
        if (leader) {
          ok = publish(t);
          if (ok && t < total_tiles) pending = claim();
        } else {
          ok = take(t);
        }
        while (ok && t < total_tiles) {
          const Fp8Tile tl = f8_decode<WIDE, SPLIT>(t, prefix_sh, offs_sh, args);
          const bool sh = tl.group == args.shared_group;
          const CUtensorMap* wm = sh ? &maps.ws : &maps.w;
          const bool own_rows = sh && args.shared_a;
          const CUtensorMap* xm = own_rows ? &maps.xs[tl.half / 8 - 1] : &maps.x[tl.half / 8 - 1];
          const int x_row = (own_rows ? tl.row0 - offs_sh[tl.group] : tl.row0) + (int)rank * (WIDE ? 128 : tl.half);
          const int w_base = sh ? 0 : tl.group * args.nout;
          const int w_row = SWIGLU ? (w_base + tl.o * 128 + (int)rank * 64) / 8 : w_base + tl.o * 256 + (int)rank * 128;
          const uint32_t x_kblk = (uint32_t)(tl.half * F_BK);
          int next = 0;
          bool sent = !leader;
          const int kb_end = tl.kb0 + tl.nk;
          for (int kb = tl.kb0; kb < kb_end; kb += F_KB) {
            if (!f8_wait<false>(&empty_bar[stage], phase ^ 1u, args, &abort_flag, SITE_EMPTY)) {
              ok = false;
              break;
            }
            const uint32_t sa = smem_base + stage * F_STAGE_BYTES;
            const uint32_t full_leader = map_to_rank(&full_bar[stage], 0);
            // a view load brings F_KB k-blocks (zeros past K), else one load per k-block
            const int kb_n = args.view ? F_KB : min(F_KB, kb_end - kb);
            if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2u * (uint32_t)kb_n * (F_KBLK_BYTES + x_kblk));
            if (args.view) {
              if (SWIGLU) f8_load_5d(sa, wm, full_leader, w_row, kb);
              else f8_load_3d(sa, wm, full_leader, 0, w_row, kb);
              f8_load_3d(sa + F_W_BYTES, xm, full_leader, 0, x_row, kb);
            } else {
              for (int j = 0; j < kb_n; ++j) {
                const int c0 = (kb + j) * F_BK;
                if (SWIGLU) f8_load_4d(sa + j * F_KBLK_BYTES, wm, full_leader, c0, w_row);
                else f8_load_2d(sa + j * F_KBLK_BYTES, wm, full_leader, c0, w_row);
                f8_load_2d(sa + F_W_BYTES + j * x_kblk, xm, full_leader, c0, x_row);
              }
            }
            ++issued;
            if (++stage == F_STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            if (!sent) {
              sent = true;
              next = pending;
              if (!publish(next)) {
                ok = false;
                break;
              }
              if (next < total_tiles) pending = claim();
            }
          }
          if (!ok) break;
          if (leader) {
            t = next;
          } else if (!take(t)) {
            break;
          }
        }
        // Drain (even CTA, which owns the full barriers): the last loads of
        // both CTAs have landed before exit.
        if (leader) {
          const long n_drain = issued < F_STAGES ? issued : F_STAGES;
          int s = stage;
          uint32_t ph = phase;
          for (long i = 0; i < n_drain; ++i) {
            if (--s < 0) {
              s = F_STAGES - 1;
              ph ^= 1u;
            }
            mbar_wait_bounded(&full_bar[s], ph, args.wait_ns, nullptr, args.hdr, KID_GEMM_FP8, SITE_DRAIN);
          }
          // every pair has made its last claim before the last one to get here
          // clears the counter for the next launch
          __threadfence();
          if (claims && atomicAdd(args.hdr + F_DONE_WORD, 1) == step - 1) {
            atomicExch(args.hdr + F_CLAIM_WORD, 0);
            atomicExch(args.hdr + F_DONE_WORD, 0);
          }
        }
      }
    } else if (warp == 1) {
      // ======================= MMA issuer (even CTA) =======================
      // The whole warp runs the loop, so that descriptors and addresses stay in
      // uniform registers; one elected lane issues.
      if (leader) {
        int stage = 0, buf = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        int rs = 0, t;
        uint32_t rph = 0;
        const uint64_t desc0 = sw128_desc(smem_base);
        while (ok && take_warp(rs, rph, t) && t < total_tiles) {
          const Fp8Tile tl = f8_decode<WIDE, SPLIT>(t, prefix_sh, offs_sh, args);
          const uint32_t idesc = f8_idesc(256, WIDE ? 256 : 2 * tl.half);
          const uint32_t x_kblk = (uint32_t)(tl.half * F_BK) >> 4;  // in descriptor units of 16 bytes
          const int nk = tl.nk;
          for (int kb = 0; kb < nk; ++kb) {
            const int j = kb & (F_KB - 1);
            if (j == 0 && !f8_warp_wait<false>(&full_bar[stage], phase, args, &abort_flag, SITE_FULL)) {
              ok = false;
              break;
            }
            if (!f8_warp_wait<false>(&tempty_bar[buf], bphase ^ 1u, args, &abort_flag, SITE_TMEM_EMPTY)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const bool last = j == F_KB - 1 || kb + 1 == nk;  // of its stage
            if (elect_one()) {
              const uint64_t wdesc = desc0 + (uint64_t)(stage * (F_STAGE_BYTES >> 4) + j * (F_KBLK_BYTES >> 4));
              const uint64_t xdesc = desc0 + (uint64_t)(stage * (F_STAGE_BYTES >> 4) + (F_W_BYTES >> 4)) + j * x_kblk;
              const uint64_t adesc = WIDE ? xdesc : wdesc, bdesc = WIDE ? wdesc : xdesc;
              const uint32_t d_tmem = tmem_base + (uint32_t)(buf * 256);
              f8_mma<0>(d_tmem, adesc, bdesc, idesc);
#pragma unroll
              for (int kk = 1; kk < F_BK / 32; ++kk)  // K = 32 per MMA: 32 bytes further along the row
                f8_mma<1>(d_tmem, adesc + (uint64_t)(kk * 2), bdesc + (uint64_t)(kk * 2), idesc);
              tc2_commit_both(&tfull_bar[buf]);
              if (last) tc2_commit_both(&empty_bar[stage]);
            }
            __syncwarp();
            buf ^= 1;
            if (buf == 0) bphase ^= 1u;
            if (last && ++stage == F_STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // Drain: every MMA issued here completes before TMEM is freed and
        // before the odd CTA (whose shared memory they read) may exit.
        if (elect_one()) {
          tc2_commit_own(&drain_bar);
          mbar_wait_bounded(&drain_bar, 0, args.wait_ns, nullptr, args.hdr, KID_GEMM_FP8, SITE_DRAIN);
        }
        __syncwarp();
      }
    } else {
      // ======================= scale products (warps 2, 3) =======================
      int rs = 0, t;
      uint32_t rph = 0;
      const int slot = warp & 1;
      uint32_t kc = 0, sphase = 0;  // k-blocks of all tiles so far: k-block kc is in TMEM slot kc % 2
      const int nkb = args.nk;
      bool ok = true;
      while (ok && take_warp(rs, rph, t) && t < total_tiles) {
        const Fp8Tile tl = f8_decode<WIDE, SPLIT>(t, prefix_sh, offs_sh, args);
        const bool sh = tl.group == args.shared_group;
        const bool own_rows = sh && args.shared_a;
        const int nk = tl.nk;
        const float* as = own_rows ? args.sas + (size_t)(tl.row0 - offs_sh[tl.group]) * nkb
                                   : args.as + (size_t)tl.row0 * nkb;
        as += tl.kb0;
        // the two weight scales of a k-block: of the tile's two matrices (SwiGLU), or of
        // the two halves of its columns (wide); else this CTA's only one
        const float* bs0 = (sh ? args.sbs[0] : args.bs[0]) + (size_t)(sh ? 0 : tl.group) * args.nnb * nkb;
        const float* bs1 = (sh ? args.sbs[1] : args.bs[1]) + (size_t)(sh ? 0 : tl.group) * args.nnb * nkb;
        const float* b0 = bs0 + (size_t)(SWIGLU ? tl.o : min(2 * tl.o + (WIDE ? 0 : (int)rank), args.nnb - 1)) * nkb + tl.kb0;
        const float* b1 =
            (SWIGLU ? bs1 + (size_t)tl.o * nkb : bs0 + (size_t)min(2 * tl.o + 1, args.nnb - 1) * nkb) + tl.kb0;
        const int r_base = WIDE ? (int)rank * 128 : 0;  // first row whose products this CTA needs
        constexpr int RP = WIDE ? 4 : 8;                // rows per lane
        float cur[RP], cur_b[2];
        auto load = [&](int kb, float (&v)[RP], float (&b)[2]) {
#pragma unroll
          for (int i = 0; i < RP; ++i) {
            const int r = r_base + lane + 32 * i;
            v[i] = r < tl.rows ? __ldg(as + (size_t)r * nkb + kb) : 0.f;
          }
          b[0] = __ldg(b0 + kb);
          b[1] = SWIGLU || WIDE ? __ldg(b1 + kb) : 0.f;
        };
        const int kb0 = (int)((kc ^ (uint32_t)warp) & 1u);  // this warp's first k-block of the tile
        if (kb0 < nk) load(kb0, cur, cur_b);
        for (int kb = kb0; kb < nk; kb += 2) {
          float nxt[RP], nxt_b[2];
          if (kb + 2 < nk) load(kb + 2, nxt, nxt_b);
          if (!f8_warp_wait<false>(&sempty_bar[slot], sphase ^ 1u, args, &abort_flag, F_SITE_SCALE)) {
            ok = false;
            break;
          }
          sphase ^= 1u;
          float* dst = scale_ring + slot * (MATS * F_CHUNK);
#pragma unroll
          for (int i = 0; i < RP; ++i) {
            const int r = lane + 32 * i;
            if constexpr (WIDE) {
              dst[r] = __fmul_rn(cur[i], cur_b[0]);
              dst[128 + r] = __fmul_rn(cur[i], cur_b[1]);
            } else if (r < 2 * tl.half) {
              const int at = r < tl.half ? f8_scale_at(r) : 128 + f8_scale_at(r - tl.half);
#pragma unroll
              for (int m = 0; m < MATS; ++m) dst[m * F_CHUNK + at] = __fmul_rn(cur[i], cur_b[m]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&tfull_bar[slot]);
#pragma unroll
          for (int i = 0; i < RP; ++i) cur[i] = nxt[i];
          cur_b[0] = nxt_b[0];
          cur_b[1] = nxt_b[1];
        }
        kc += (uint32_t)nk;
      }
    }
  } else {
    // ======================= epilogue (warps 4..11, both CTAs) =======================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int quarter = warp & 3;               // TMEM lanes 32 * quarter .. + 31
    const int hf = (warp - F_EPI_WARP0) >> 2;   // half of the chunk's columns
    const int owner = threadIdx.x - F_EPI_WARP0 * 32;  // SwiGLU: the row whose scale this thread makes
    const uint32_t peer = rank ^ 1u;
    Fp8Drain drain;
    drain.tmem = tmem_base + ((uint32_t)(quarter * 32) << 16);
    drain.tempty_remote = map_to_rank(&tempty_bar[0], 0);
    drain.tfull = smem_u32(tfull_bar);
    drain.sempty = smem_u32(sempty_bar);
    drain.scales = smem_u32(scale_ring) +
                   4u * (uint32_t)(WIDE ? (SWIGLU ? 0 : hf * 128) + quarter * 32 + lane : hf * 128 + (lane & 3) * 4);
    drain.slot = drain.phase = 0;
    uint32_t tiles_done = 0, half_phase = 0;
    int rs = 0, t;
    uint32_t rph = 0;
    bool ok = true;
    // Tiles cut along K: this warp's sums go to the workspace (`vecs` float4 per
    // thread).  Once both CTAs of the pair have written theirs, the even CTA counts
    // the pair's part as done.  Returns 2, with the sums of all parts in `a`, in the
    // pair whose part was the last one, 1 in the others, 0 after a failed wait.
    uint32_t split_phase = 0;
    auto split_join = [&](uint64_t(&a)[64], const Fp8Tile& tl, int vecs) -> int {
      const size_t stride = (size_t)args.partial_vecs * 256;  // of one CTA's part
      float4* const first = args.partial + ((size_t)tl.index * args.splits * 2 + rank) * stride + owner;
      float4* const mine = first + (size_t)tl.part * 2 * stride;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (i >= vecs) break;
        const float2 x = unpack64(a[2 * i]), y = unpack64(a[2 * i + 1]);
        __stcg(mine + i * 256, make_float4(x.x, x.y, y.x, y.y));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&split_bar);
      const uint32_t ph = split_phase;
      split_phase ^= 1u;
      if (warp == F_EPI_WARP0) {
        if (!f8_warp_wait<false>(&split_bar, ph, args, &abort_flag, F_SITE_SPLIT)) return 0;
        if (leader) {
          if (!f8_warp_wait<true>(&pair_bar, ph, args, &abort_flag, F_SITE_SPLIT)) return 0;
          if (lane == 0) {
            // after the barriers: releases the sums of every thread of the pair's epilogues,
            // and acquires those of the other parts, which the releasing arrivals on both
            // CTAs' done_bar pass on to them; the count goes back to zero for the next launch
            unsigned count;
            asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                         : "=r"(count)
                         : "l"(args.hdr + f8_split_word(tl.index)), "r"((unsigned)args.splits - 1u)
                         : "memory");
            const bool last = count == (unsigned)args.splits - 1u;
            last_sh = last;
            mbar_arrive(&done_bar);
            const uint32_t peer_done = map_to_rank(&done_bar, 1);
            f8_arrive_expect_tx_release(peer_done, 4);
            st_async_b32(map_to_rank((const void*)&last_sh, 1), last, peer_done);
          }
        } else if (lane == 0) {
          mbar_arrive_cluster(map_to_rank(&pair_bar, 0));  // releases this CTA's stores to the even CTA
        }
        __syncwarp();
      }
      if (!f8_warp_wait<true>(&done_bar, ph, args, &abort_flag, F_SITE_SPLIT)) return 0;
      if (!last_sh) return 1;
#pragma unroll
      for (int i = 0; i < 64; ++i) a[i] = 0ull;
#pragma unroll
      for (int i0 = 0; i0 < 32; i0 += 4) {
        if (i0 >= vecs) break;
        const float4* src = first + i0 * 256;
#pragma unroll 4  // 16 loads in flight
        for (int p = 0; p < args.splits; ++p, src += 2 * stride) {
#pragma unroll
          for (int i = i0; i < i0 + 4; ++i) {
            const float4 f = __ldcg(src + (i - i0) * 256);
            const float2 x = unpack64(a[2 * i]), y = unpack64(a[2 * i + 1]);
            a[2 * i] = pack64(__float_as_uint(__fadd_rn(x.x, f.x)), __float_as_uint(__fadd_rn(x.y, f.y)));
            a[2 * i + 1] = pack64(__float_as_uint(__fadd_rn(y.x, f.z)), __float_as_uint(__fadd_rn(y.y, f.w)));
          }
        }
      }
      return 2;
    };
    while (ok && take_warp(rs, rph, t) && t < total_tiles) {
      const Fp8Tile tl = f8_decode<WIDE, SPLIT>(t, prefix_sh, offs_sh, args);
      if constexpr (WIDE) {
        const int r_cta = quarter * 32;                          // this warp's rows of the CTA's 128
        const int valid = tl.rows - ((int)rank * 128 + r_cta);   // ... of which this many exist
        if (valid <= 0) {
          // (so does the quarter's other warp: half_bar and half_sh's buffer stay as they are)
          ok = f8_pass_over(drain, tl.nk, args, &abort_flag);
          if (!ok) break;
          continue;
        }
        uint64_t acc[8][8];
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i >> 3][i & 7] = 0ull;
        ok = f8_accumulate_wide<SWIGLU>(acc, drain, hf * 128, tl.nk, args, &abort_flag);
        if (!ok) break;
        uint8_t* stage = smem + F_STAGES * F_STAGE_BYTES + F_SLOTS * MATS * F_CHUNK * 4 +
                         (warp - F_EPI_WARP0) * F_OUT_WIDE_BYTES;
        const size_t row = (size_t)tl.row0 + (int)rank * 128 + r_cta;
        if constexpr (!SWIGLU) {
          constexpr int ES = EPI == moe_host::EPI_F32 ? 4 : 2, COLS = 128 / ES;
          const int n0 = tl.o * 256 + hf * 128;
          const size_t ld = (size_t)args.nout * ES;
          uint8_t* c = reinterpret_cast<uint8_t*>(args.c) + row * ld + (size_t)n0 * ES;
#pragma unroll
          for (int p = 0; p < 128 / COLS; ++p) {  // 32 (fp32) or 64 columns at a time
            const int left = args.nout - (n0 + p * COLS);
            if (left <= 0) break;
            uint4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if constexpr (ES == 4) {
                const uint64_t* a = &acc[2 * p + (i >> 2)][(i & 3) * 2];
                const float2 x = unpack64(a[0]), y = unpack64(a[1]);
                w[i] = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x),
                                  __float_as_uint(y.y));
              } else {
                const uint64_t* a = &acc[4 * p + (i >> 1)][(i & 1) * 4];
                const float2 x = unpack64(a[0]), y = unpack64(a[1]), z = unpack64(a[2]), q = unpack64(a[3]);
                w[i] = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y), pack_bf16x2(z.x, z.y),
                                  pack_bf16x2(q.x, q.y));
              }
            }
            f8_store_rows<ES, 128>(stage, w, c + p * 128, ld, valid, left * ES, args.vec);
          }
        } else {
          const bool up_first = tl.group == args.shared_group ? args.s_up_first : args.up_first;
          const int unit0 = tl.o * 128 + hf * 64;  // this warp's hidden units, 8 per 16 columns
          // the activation in place; the order of the two matrices is the tile's, so
          // the choice stays outside the 64 units
          auto activate = [&](auto up_is_first) {
            constexpr bool UP = decltype(up_is_first)::value;
#pragma unroll
            for (int b = 0; b < 8; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 g = unpack64(acc[b][UP ? 4 + i : i]), u = unpack64(acc[b][UP ? i : 4 + i]);
                acc[b][i] = pack64(__float_as_uint(f8_silu_mul(g.x, u.x)), __float_as_uint(f8_silu_mul(g.y, u.y)));
              }
          };
          if (up_first) activate(std::true_type());
          else activate(std::false_type());
          if (unit0 + 64 > args.nout) {  // units past the last one (nout is even)
#pragma unroll
            for (int b = 0; b < 8; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (unit0 + b * 8 + 2 * i >= args.nout) acc[b][i] = 0ull;
          }
          float m = 0.f;
#pragma unroll
          for (int b = 0; b < 8; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = unpack64(acc[b][i]);
              m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
          // the other half of the row's 128 units is with the warp of the same rows.
          // Two buffers, one per phase of half_bar: that warp reads this tile's value before
          // it arrives for the next one of the quarter's tiles that has rows.
          float* at = &half_sh[half_phase][0][r_cta + lane];
          at[hf * 128] = m;
          __syncwarp();
          if (lane == 0) mbar_arrive(&half_bar[quarter]);
          if (!f8_warp_wait<false>(&half_bar[quarter], half_phase, args, &abort_flag, F_SITE_AMAX)) break;
          half_phase ^= 1u;
          const float scale = quant_scale(fmaxf(m, at[(hf ^ 1) * 128]));
          const float inv = __frcp_rn(scale);
          if (hf == 0 && lane < valid) args.c_scale[(row + lane) * args.n_o + tl.o] = scale;
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t* a = &acc[2 * i + (k >> 1)][(k & 1) * 2];
              const float2 x = unpack64(a[0]), y = unpack64(a[1]);
              q[k] = e4m3x4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
            }
            w[i] = make_uint4(q[0], q[1], q[2], q[3]);
          }
          if (unit0 < args.nout)
            f8_store_rows<1, 64>(stage, w, reinterpret_cast<uint8_t*>(args.c) + row * args.nout + unit0, args.nout, valid,
                             args.nout - unit0, true);
        }
      } else {
      const int cw = tl.half;  // columns of this warp: hf * cw .. + cw - 1
      uint64_t acc[8][2][2][2];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i >> 3][(i >> 2) & 1][(i >> 1) & 1][i & 1] = 0ull;
      // columns past cw in the last batches add up unused values
      if (cw > 96) ok = f8_accumulate<8, MATS>(acc, drain, hf * cw, tl.nk, args, &abort_flag);
      else if (cw > 64) ok = f8_accumulate<6, MATS>(acc, drain, hf * cw, tl.nk, args, &abort_flag);
      else if (cw > 32) ok = f8_accumulate<4, MATS>(acc, drain, hf * cw, tl.nk, args, &abort_flag);
      else if (cw > 16) ok = f8_accumulate<2, MATS>(acc, drain, hf * cw, tl.nk, args, &abort_flag);
      else ok = f8_accumulate<1, MATS>(acc, drain, hf * cw, tl.nk, args, &abort_flag);
      if (!ok) break;
      if constexpr (SPLIT) {
        const int done = split_join(reinterpret_cast<uint64_t(&)[64]>(acc), tl, (cw + 15) / 16 * 4);
        if (done == 0) break;
        if (done == 1) continue;
      }

      const int c_lane = 2 * (lane & 3);  // this lane's first column of every eight
      const int valid = tl.rows - hf * cw;  // rows of this half that exist
      const size_t row0 = (size_t)tl.row0 + hf * cw;
      if constexpr (EPI == moe_host::EPI_F32) {
        const int n_base = tl.o * 256 + (int)rank * 128 + quarter * 32 + (lane >> 2);
        float* C = reinterpret_cast<float*>(args.c);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (b * 16 >= cw) break;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = b * 16 + j * 8 + c_lane, n = n_base + 8 * i;
              const float2 f = unpack64(acc[b][i >> 1][j][i & 1]);
              if (n < args.nout) {
                if (r < valid && r < cw) C[(row0 + r) * args.nout + n] = f.x;
                if (r + 1 < valid && r + 1 < cw) C[(row0 + r + 1) * args.nout + n] = f.y;
              }
            }
        }
      } else if constexpr (EPI == moe_host::EPI_STORE) {
        // 16 rows x 32 columns at a time through this warp's block of shared memory
        uint8_t* stage = smem + F_STAGES * F_STAGE_BYTES + F_SLOTS * MATS * F_CHUNK * 4 +
                         (warp - F_EPI_WARP0) * F_OUT_BYTES;
        const uint32_t st_at = smem_u32(stage) + (uint32_t)((lane & 7) * F_OUT_PITCH + (lane >> 3) * 16);
        const int n0 = tl.o * 256 + (int)rank * 128 + quarter * 32;
        bf16* C = reinterpret_cast<bf16*>(args.c);
        const int left = min(valid, cw);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int r0 = b * 16;
          if (r0 >= left) break;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = unpack64(acc[b][i >> 1][j][i & 1]);
              p[i] = pack_bf16x2(f.x, f.y);
            }
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                             st_at + (uint32_t)(j * 8 * F_OUT_PITCH)),
                         "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3])
                         : "memory");
          }
          __syncwarp();
          if (args.vec) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = i * 8 + (lane >> 2), n = n0 + (lane & 3) * 8;
              const uint4 w = *reinterpret_cast<const uint4*>(stage + r * F_OUT_PITCH + (lane & 3) * 16);
              if (r0 + r < left && n < args.nout) *reinterpret_cast<uint4*>(C + (row0 + r0 + r) * args.nout + n) = w;
            }
          } else {
            for (int r = 0; r < 16 && r0 + r < left; ++r)
              if (n0 + lane < args.nout)
                C[(row0 + r0 + r) * args.nout + n0 + lane] =
                    *reinterpret_cast<const bf16*>(stage + r * F_OUT_PITCH + lane * 2);
          }
        }
      } else {
        const int unit0 = tl.o * 128 + (int)rank * 64 + quarter * 16;  // hidden units of this warp
        const bool up_first = tl.group == args.shared_group ? args.s_up_first : args.up_first;
        // the activation in place: acc[..][0] holds its pair of rows
        float m[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) m[i] = 0.f;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (b * 16 >= cw) break;  // (one jump: unrolled batches are long, and few rows find them cold)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = 0.f, my = 0.f;
#pragma unroll
            for (int l16 = 0; l16 < 2; ++l16) {
              const float2 p = unpack64(acc[b][l16][j][0]), q = unpack64(acc[b][l16][j][1]);
              const bool in = unit0 + l16 * 8 + (lane >> 2) < args.nout;
              const float vx = in ? f8_silu_mul(up_first ? q.x : p.x, up_first ? p.x : q.x) : 0.f;
              const float vy = in ? f8_silu_mul(up_first ? q.y : p.y, up_first ? p.y : q.y) : 0.f;
              mx = fmaxf(mx, fabsf(vx));
              my = fmaxf(my, fabsf(vy));
              acc[b][l16][j][0] = pack64(__float_as_uint(vx), __float_as_uint(vy));
            }
            m[b * 4 + j * 2] = mx;
            m[b * 4 + j * 2 + 1] = my;
          }
        }
        // each row's largest magnitude over the 8 lanes that share its column: a
        // reduce-scatter, after which a lane holds 4 of the 32 rows
#pragma unroll
        for (int o = 16, n = 16; o >= 4; o >>= 1, n >>= 1) {
          const bool upper = lane & o;
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const float give = upper ? m[i] : m[i + n], keep = upper ? m[i + n] : m[i];
            m[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
          }
        }
        const int i0 = ((lane & 16) ? 16 : 0) + ((lane & 8) ? 8 : 0) + ((lane & 4) ? 4 : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = i0 + i;  // b * 4 + j * 2 + e
          const int c = (at >> 1) * 8 + c_lane + (at & 1);
          if (c < cw) atomicMax(&amax_sh[hf * cw + c], __float_as_uint(m[i]));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&amax_bar);
        const uint32_t once = tiles_done & 1u;          // phase of the barriers used once per tile
        const uint32_t pb = tiles_done & 1u, pph = (tiles_done >> 1) & 1u;
        if (!f8_warp_wait<false>(&amax_bar, once, args, &abort_flag, F_SITE_AMAX)) break;
        // one thread per row: trade the magnitude with the other CTA, make the scale
        if (owner == 0) mbar_arrive_expect_tx(&peer_bar[pb], (uint32_t)(2 * tl.half) * 4u);
        unsigned mine = 0u;
        if (owner < 2 * tl.half) {
          mine = amax_sh[owner];
          amax_sh[owner] = 0u;
          st_async_b32(map_to_rank((const void*)&peer_sh[pb][owner], peer), mine, map_to_rank(&peer_bar[pb], peer));
        }
        if (!f8_warp_wait<true>(&peer_bar[pb], pph, args, &abort_flag, F_SITE_AMAX)) break;
        if (owner < 2 * tl.half) {
          const float scale = quant_scale(fmaxf(__uint_as_float(mine), peer_sh[pb][owner]));
          inv_sh[owner < cw ? f8_scale_at(owner) : 128 + f8_scale_at(owner - cw)] = __frcp_rn(scale);
          if (leader && owner < tl.rows) args.c_scale[(size_t)(tl.row0 + owner) * args.n_o + tl.o] = scale;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&inv_bar);
        if (!f8_warp_wait<false>(&inv_bar, once, args, &abort_flag, F_SITE_AMAX)) break;
        ++tiles_done;
        // codes: four consecutive units of one row per lane, 16 bytes of eight rows per store
        uint8_t* C = reinterpret_cast<uint8_t*>(args.c);
        const int item = (lane >> 2) & 3;  // (16-lane half, row of the pair) this lane stores
        const int unit = unit0 + (item >> 1) * 8 + (lane >> 4) * 4;
        const int left = min(valid, cw);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (b * 16 >= cw) break;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 inv = *reinterpret_cast<const float2*>(inv_sh + hf * 128 + b * 16 + (lane & 3) * 4 + j * 2);
            const float2 lo = unpack64(acc[b][0][j][0]), hi = unpack64(acc[b][1][j][0]);
            const uint32_t w = f8_transpose_bytes(e4m3x4(lo.x * inv.x, lo.y * inv.y, hi.x * inv.x, hi.y * inv.y));
            const int r = b * 16 + j * 8 + c_lane + (item & 1);
            if (r < left && unit < args.nout) *reinterpret_cast<uint32_t*>(C + (row0 + r) * args.nout + unit) = w;
          }
        }
      }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TC_TMEM_COLS)
                 : "memory");
}

}  // namespace moe

namespace moe_host {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // gemm_tc.cu

// Tensor map of bytes: dims and strides (of dims 1 ..) as given, 128-byte
// swizzle, zero fill outside.
static bool byte_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row-major [rows][k] matrix, rows ld bytes apart, in boxes of box_rows rows x
// 128 columns; as a view {128, rows, k / 128} the box also spans two k-blocks.
static bool rows_map(CUtensorMap* m, const void* base, int64_t rows, int k, int64_t ld, int box_rows, bool view) {
  if (view) {
    const cuuint64_t dims[3] = {128, (cuuint64_t)rows, (cuuint64_t)(k / 128)}, strides[2] = {(cuuint64_t)ld, 128};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, moe::F_KB};
    return byte_map(m, base, 3, dims, strides, box);
  }
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  return byte_map(m, base, 2, dims, strides, box);
}

// Two [rows][k] matrices `apart` bytes from each other, interleaved by eight
// rows: boxes of eight such groups of each (128 rows).  rows % 8 == 0.
static bool interleaved_map(CUtensorMap* m, const void* low, int64_t apart, int64_t rows, int k, bool view) {
  const cuuint64_t K = (cuuint64_t)k;
  if (view) {
    const cuuint64_t dims[5] = {128, 8, 2, (cuuint64_t)(rows / 8), K / 128};
    const cuuint64_t strides[4] = {K, (cuuint64_t)apart, 8 * K, 128};
    const cuuint32_t box[5] = {128, 8, 2, 8, moe::F_KB};
    return byte_map(m, low, 5, dims, strides, box);
  }
  const cuuint64_t dims[4] = {K, 8, 2, (cuuint64_t)(rows / 8)}, strides[3] = {K, (cuuint64_t)apart, 8 * K};
  const cuuint32_t box[4] = {128, 8, 2, 8};
  return byte_map(m, low, 4, dims, strides, box);
}

// Clusters of two that can be resident at once (one CTA per SM), per device.
template <int EPI, bool WIDE, bool SPLIT>
static int f8_resident_pairs() {
  static std::atomic<int> cache[64] = {};
  const int dev = current_device();
  if (dev >= 0 && dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count() & ~1));
  cfg.blockDim = dim3(moe::F_THREADS);
  cfg.dynamicSmemBytes = moe::f8_smem_bytes<EPI, WIDE>();
  if (cudaOccupancyMaxActiveClusters(&n, moe::gemm_fp8_kernel<EPI, WIDE, SPLIT>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = sm_count() / 2;
  }
  if (n > sm_count() / 2) n = sm_count() / 2;
  if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int EPI, bool WIDE, bool SPLIT>
static moe_status launch_f8_t(const moe::Fp8Maps& maps, const moe::Fp8Args& args, int64_t tile_bound, bool follows,
                              cudaStream_t s) {
  static SmemLimit lim;
  const moe_status st = ensure_smem_limit(moe::gemm_fp8_kernel<EPI, WIDE, SPLIT>, moe::f8_smem_bytes<EPI, WIDE>(), lim);
  if (st != MOE_OK) return st;
  const int64_t pairs = std::min<int64_t>(tile_bound, f8_resident_pairs<EPI, WIDE, SPLIT>());
  cudaLaunchAttribute overlap = {};
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(moe::F_THREADS);
  cfg.dynamicSmemBytes = moe::f8_smem_bytes<EPI, WIDE>();
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = follows ? 1 : 0;
  cudaLaunchKernelEx(&cfg, moe::gemm_fp8_kernel<EPI, WIDE, SPLIT>, maps, args);
  return launch_status();
}

template <int EPI>
static moe_status launch_f8(bool wide, const moe::Fp8Maps& maps, const moe::Fp8Args& args, int64_t tile_bound,
                            bool follows, cudaStream_t s) {
  if (wide) return launch_f8_t<EPI, true, false>(maps, args, tile_bound, follows, s);
  return args.splits > 1 ? launch_f8_t<EPI, false, true>(maps, args, tile_bound, follows, s)
                         : launch_f8_t<EPI, false, false>(maps, args, tile_bound, follows, s);
}

// Weight map of one set of matrices; *up_first: the second lies lower in memory.
static moe_status weight_map(CUtensorMap* m, int epi, const Fp8Operand& b, const Fp8Operand& b2, int64_t rows, int k,
                             bool view, int* up_first) {
  *up_first = 0;
  if (epi != EPI_SWIGLU) return rows_map(m, b.q, rows, k, k, 128, view) ? MOE_OK : MOE_ERR_CUDA;
  *up_first = b2.q < b.q;
  const uint8_t* low = *up_first ? b2.q : b.q;
  const int64_t apart = *up_first ? b.q - b2.q : b2.q - b.q;  // not 0, and below 2^40
  return interleaved_map(m, low, apart, rows, k, view) ? MOE_OK : MOE_ERR_CUDA;
}

// Wide tiles or swapped ones, most rows of a chunk, weight tiles per group, the most
// tiles there can be, and parts that each is cut into along K.
struct Fp8Shape {
  bool wide;
  int chunk, n_o;
  int64_t tiles;
  int splits;
};

// More tiles than SM pairs: the tiling by rows per group (F_WIDE_ROWS), chunks of 256
// rows.  With fewer, a call lasts as long as one tile, so the tile is made shorter,
// by smaller chunks (the weights are then read more often, from L2) or by cutting it
// along K, whichever costs least in hundredths of a microsecond, as measured on B200
// with calls of 1 to 1000 rows, K = 1040 to 7168:
//   a k-block       42 wide, 26 + r^2 / 2400 swapped with r rows (27, 28, 33 and 53
//                   with 32, 64, 128 and 256): the rounds of barriers between MMA and
//                   epilogue below 100 rows, the accumulator reads above;
//   joining p parts 300 + 6 r + 25 p (wide tiles are not cut: smaller chunks always win).
// 200 x 2048 x 7168 takes 23.1 us in chunks of 32 rows, 32.5 as 8 parts of whole
// tiles; 1 x 4096 x 7168 15.9 us in 4 parts, 22.0 uncut.
static Fp8Shape f8_shape(bool swiglu, int64_t rows, int groups, bool offsets, int nout, int k) {
  Fp8Shape f;
  f.wide = rows >= (int64_t)moe::F_WIDE_ROWS * groups;
  f.chunk = moe::F_CHUNK;
  f.n_o = (int)(swiglu ? ((int64_t)nout + 127) / 128 : ((int64_t)nout + 255) / 256);
  f.splits = 1;
  auto tiles = [&](int chunk) { return ((rows + chunk - 1) / chunk + (offsets ? groups : 0)) * f.n_o; };
  f.tiles = tiles(f.chunk);
  const int64_t pairs = sm_count() / 2, nk = q_blocks(k);
  if (f.tiles < 1 || f.tiles > pairs) return f;
  const int64_t per_group = (rows + groups - 1) / groups;
  int64_t best = f.wide ? 42 * nk : INT64_MAX;
  for (int chunk = moe::F_CHUNK; chunk >= 32 && tiles(chunk) <= pairs; chunk /= 2) {
    const int64_t r = std::min<int64_t>(chunk, per_group), t = tiles(chunk);
    const int64_t most = t <= moe::F_SPLIT_TILES ? std::max<int64_t>(1, std::min(pairs / t, nk / 2)) : 1;
    for (int64_t parts = 1; parts <= most; ++parts) {
      const int64_t cost = (26 + r * r / 2400) * ((nk + parts - 1) / parts) + (parts > 1 ? 300 + 6 * r + 25 * parts : 0);
      if (cost >= best) continue;
      best = cost;
      f.wide = false;
      f.chunk = chunk;
      f.tiles = t;
      f.splits = (int)parts;
    }
  }
  return f;
}

// float4 of sums per thread: half of the chunk in 16s
static int f8_partial_vecs(const Fp8Shape& f, int64_t rows) {
  return (int)((std::min<int64_t>(f.chunk, rows) + 31) / 32 * 4);
}

size_t gemm_fp8_split_bytes(bool swiglu, int64_t rows, int groups, bool offsets, int nout, int k) {
  if (rows <= 0) return 0;
  const Fp8Shape f = f8_shape(swiglu, rows, groups, offsets, nout, k);
  return f.splits == 1 ? 0 : (size_t)f.tiles * f.splits * 2 * f8_partial_vecs(f, rows) * 256 * sizeof(float4);
}

void gemm_fp8_tiling(bool swiglu, int64_t rows, int groups, bool offsets, int nout, int k, int32_t tiling[3]) {
  const Fp8Shape f = f8_shape(swiglu, rows, groups, offsets, nout, k);
  tiling[0] = f.wide;
  tiling[1] = f.chunk;
  tiling[2] = f.splits;
}

moe_status launch_gemm_fp8(const Fp8Gemm& g, cudaStream_t s) {
  if (g.max_rows == 0) return MOE_OK;
  const bool swiglu = g.epi == EPI_SWIGLU;
  const int groups = g.offsets ? g.groups : 1;
  const Fp8Shape shape = f8_shape(swiglu, g.max_rows, groups, g.offsets != nullptr, g.nout, g.k);
  const bool wide = shape.wide;
  const bool view = g.k % 128 == 0;
  const bool shared = g.sb.q != nullptr && g.offsets != nullptr;
  const bool shared_a = shared && g.sa.q != nullptr && g.sa_rows > 0;
  moe::Fp8Maps maps;
  moe::Fp8Args args;
  const int64_t w_rows = std::max<int64_t>((int64_t)(shared ? g.groups - 1 : g.groups) * g.nout, 1);
  moe_status st = weight_map(&maps.w, g.epi, g.b, g.b2, w_rows, g.k, view, &args.up_first);
  if (st != MOE_OK) return st;
  args.s_up_first = 0;
  if (shared) {
    st = weight_map(&maps.ws, g.epi, g.sb, g.sb2, g.nout, g.k, view, &args.s_up_first);
    if (st != MOE_OK) return st;
  }
  // row boxes: only those that a chunk can take (one group: its two chunk sizes)
  auto row_maps = [&](CUtensorMap* ms, const Fp8Operand& a, int64_t rows, bool one_group) -> bool {
    const int64_t ch = (rows + shape.chunk - 1) / shape.chunk;
    const int64_t nc = wide ? moe::F_CHUNK : ((rows + ch - 1) / ch + 15) / 16 * 16;
    auto half = [&](int64_t r) { return wide ? std::min<int64_t>(128, (r + 7) / 8 * 8) : (r + 15) / 16 * 8; };
    const int64_t first = half(std::min(nc, rows)), last = half(rows - (ch - 1) * nc);
    for (int i = 0; i < moe::F_XMAPS; ++i) {
      const int64_t box = 8 * (i + 1);
      if (one_group ? (box == first || box == last) : box <= half(std::min<int64_t>(shape.chunk, rows)))
        if (!rows_map(&ms[i], a.q, rows, g.k, a.ld, (int)box, view)) return false;
    }
    return true;
  };
  const int64_t a_rows = shared_a ? std::max<int64_t>((int64_t)g.max_rows - g.sa_rows, 1) : g.max_rows;
  if (!row_maps(maps.x, g.a, a_rows, g.offsets == nullptr)) return MOE_ERR_CUDA;
  if (shared_a && !row_maps(maps.xs, g.sa, g.sa_rows, true)) return MOE_ERR_CUDA;
  args.offsets = g.offsets;
  args.groups = groups;
  args.max_rows = g.max_rows;
  args.nout = g.nout;
  args.nk = q_blocks(g.k);
  args.n_o = shape.n_o;
  args.chunk = shape.chunk;
  args.splits = 1;
  args.partial = nullptr;
  args.partial_vecs = f8_partial_vecs(shape, g.max_rows);
  const size_t split_bytes = gemm_fp8_split_bytes(swiglu, g.max_rows, groups, g.offsets != nullptr, g.nout, g.k);
  if (split_bytes > 0 && split_bytes <= g.split_bytes) {
    args.splits = shape.splits;
    args.split_magic = (unsigned)((1ull << 32) / (unsigned)args.splits + 1);  // exact: there are few tiles
    args.split_nk = args.nk / args.splits;
    args.split_rem = args.nk % args.splits;
    args.partial = static_cast<float4*>(g.split_ws);
  }
  args.view = view ? 1 : 0;
  args.nnb = q_blocks(g.nout);
  args.as = g.a.scale;
  args.sas = g.sa.scale;
  for (int m = 0; m < 2; ++m) {
    args.bs[m] = (swiglu && (m ^ args.up_first)) ? g.b2.scale : g.b.scale;
    args.sbs[m] = (swiglu && (m ^ args.s_up_first)) ? g.sb2.scale : g.sb.scale;
  }
  args.c = g.c;
  args.c_scale = g.c_scale;
  args.vec = (g.nout % (g.epi == EPI_F32 ? 4 : 8) == 0 && (uintptr_t)g.c % 16 == 0) ? 1 : 0;
  args.shared_group = shared ? g.groups - 1 : -1;
  args.shared_a = shared_a ? 1 : 0;
  args.hdr = g.hdr;
  args.wait_ns = wait_limit_ns();
  const int64_t bound = shape.tiles * args.splits;  // the exact count lives on the device
  if (swiglu) return launch_f8<EPI_SWIGLU>(wide, maps, args, bound, g.follows, s);
  if (g.epi == EPI_F32) return launch_f8<EPI_F32>(wide, maps, args, bound, g.follows, s);
  return launch_f8<EPI_STORE>(wide, maps, args, bound, g.follows, s);
}

}  // namespace moe_host
