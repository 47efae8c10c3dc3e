// C-ABI entry points of the 8-bit (e4m3, block-scaled) operators and of the
// layer forward built on them: argument checks, the workspace layout and the
// order of the kernels on the caller's stream.
#include <algorithm>
#include <initializer_list>

#include "gemm_fp8_kernels.h"
#include "quant_common.cuh"
#include "tcgen05.cuh"

namespace moe_host {

// Workspace of the 8-bit layer (every region 256-byte aligned): the header,
// xn and its e4m3 form, the routing buffers, the expert-sorted e4m3 rows with
// their scales, the e4m3 activations with theirs, and the expert outputs.
struct Fp8Layout {
  size_t hdr, xn, xq, xs, logits, idx, gate, counts, offsets, offsets_ext, slot_row, row_token, hist, xq_perm,
      xs_perm, act, act_s, y_perm, y_shared, split, total;
  bool fold;           // the shared expert runs as one more group of the routed products
  int64_t rows;        // R: rows of the expert-sorted buffers
  int64_t act_elems;   // codes and scales that the activation regions hold
  int64_t act_scales;
  size_t split_bytes;  // partial sums of products with few tiles
};

static Fp8Layout fp8_layout(const moe_config* c) {
  Fp8Layout L;
  const size_t es = c->dtype == MOE_BF16 ? 2 : 4;
  const int64_t N = c->n_tokens, d = c->d_model, E = c->n_experts, k = c->top_k;
  const int64_t cap = capacity_of(c);
  int64_t R = N * k;
  if (cap >= 0 && E * cap < R) R = E * cap;
  L.rows = R;
  L.fold = c->d_ff_shared > 0 && c->d_ff_shared == c->d_ff && c->n_experts < moe::TC_MAX_GROUPS;
  const int64_t Rx = R + (L.fold ? N : 0);
  L.act_elems = Rx * c->d_ff;
  L.act_scales = Rx * q_blocks(c->d_ff);
  if (N * (int64_t)c->d_ff_shared > L.act_elems) L.act_elems = N * c->d_ff_shared;
  if (N * (int64_t)q_blocks(c->d_ff_shared) > L.act_scales) L.act_scales = N * q_blocks(c->d_ff_shared);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.hdr = take(kFp8HeaderBytes);
  L.xn = take(N * d * es);
  L.xq = take(N * d);
  L.xs = take(N * q_blocks(c->d_model) * 4);
  L.logits = take(N * E * 4);
  L.idx = take(N * k * 4);
  L.gate = take(N * k * 4);
  L.counts = take(E * 4);
  L.offsets = take((E + 1) * 4);
  L.offsets_ext = take((E + 2) * 4);
  L.slot_row = take(N * k * 4);
  L.row_token = take(N * k * 4);
  L.hist = take(permute_hist_ints(N * k, (int)E) * 4);
  L.xq_perm = take(R * d);
  L.xs_perm = take(R * q_blocks(c->d_model) * 4);
  L.act = take(L.act_elems);
  L.act_s = take(L.act_scales * 4);
  L.y_perm = take(Rx * d * es);
  L.y_shared = take(c->d_ff_shared > 0 && !L.fold ? N * d * es : 0);
  // both products of the routed experts, of one group of as many rows and of the shared expert
  L.split_bytes = 0;
  auto need = [&](int64_t rows, int groups, bool offs, int64_t h) {
    const size_t gate_up = gemm_fp8_split_bytes(true, rows, groups, offs, (int)h, c->d_model);
    const size_t down = gemm_fp8_split_bytes(false, rows, groups, offs, c->d_model, (int)h);
    L.split_bytes = std::max(L.split_bytes, std::max(gate_up, down));
  };
  need(Rx, (int)E + (L.fold ? 1 : 0), true, c->d_ff);
  need(Rx, 1, false, c->d_ff);
  if (c->d_ff_shared > 0) need(N, 1, false, c->d_ff_shared);
  L.split = take(L.split_bytes);
  L.total = o;
  return L;
}

// e4m3 rows must be whole 16-byte units for TMA.
static bool fp8_supported(const moe_config* c) {
  return config_supported(c) && c->d_model % 16 == 0 && c->d_ff % 16 == 0 && c->d_ff_shared % 16 == 0;
}

static moe_status check_fp8(const moe_config* c, const void* ws, size_t ws_bytes) {
  if (!config_ok(c)) return MOE_ERR_INVALID_ARG;
  if (!fp8_supported(c)) return MOE_ERR_UNSUPPORTED;
  if (ws == nullptr || ((uintptr_t)ws % 256) != 0) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < fp8_layout(c).split) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// The layout in a workspace that may have been sized for another number of tokens:
// the partial sums, at its end, have the room that is left.
static Fp8Layout fp8_layout_in(const moe_config* c, size_t ws_bytes) {
  Fp8Layout L = fp8_layout(c);
  L.split_bytes = std::min(L.split_bytes, ws_bytes - L.split);
  return L;
}

#define MOE_TRY(x)                 \
  do {                             \
    moe_status _st = (x);          \
    if (_st != MOE_OK) return _st; \
  } while (0)

static inline char* wsp(void* ws, size_t off) { return static_cast<char*>(ws) + off; }

static inline bool misaligned(std::initializer_list<const void*> ps) {
  uintptr_t at = 0;
  for (const void* p : ps) at |= (uintptr_t)p;
  return at % 16 != 0;
}

// Gate and up lie at the two ends of one tensor-map stride, which has 40 bits.
static inline bool one_view(const void* gate, const void* up) {
  const uintptr_t a = (uintptr_t)gate, b = (uintptr_t)up;
  return a != b && (a < b ? b - a : a - b) < (uintptr_t)1 << 40;
}

// The SwiGLU experts over prepared products: gate/up (activation quantised in
// the epilogue), then down.  p carries the groups and the rows; w2 and its
// shared form the down projection's weights.
static moe_status ffn_fp8_impl(const moe_config* c, Fp8Gemm p, Fp8Operand w_down, Fp8Operand ws_down, int d_ff, void* y,
                               void* ws, const Fp8Layout& L, cudaStream_t s, void* between) {
  Fp8Operand act;
  act.q = (uint8_t*)wsp(ws, L.act);
  act.scale = (float*)wsp(ws, L.act_s);
  act.ld = d_ff;
  p.hdr = (int32_t*)wsp(ws, L.hdr);
  p.split_ws = wsp(ws, L.split);
  p.split_bytes = L.split_bytes;
  p.epi = EPI_SWIGLU;
  p.nout = d_ff;
  p.k = c->d_model;
  p.c = const_cast<uint8_t*>(act.q);
  p.c_scale = const_cast<float*>(act.scale);
  MOE_TRY(launch_gemm_fp8(p, s));
  if (between && cudaEventRecord((cudaEvent_t)between, s) != cudaSuccess) return MOE_ERR_CUDA;
  p.epi = c->dtype == MOE_BF16 ? EPI_STORE : EPI_F32;
  p.a = act;
  p.b = w_down;
  p.b2 = Fp8Operand();
  p.sb = ws_down;
  p.sb2 = p.sa = Fp8Operand();
  p.sa_rows = 0;
  p.nout = c->d_model;
  p.k = d_ff;
  p.c = y;
  p.c_scale = nullptr;
  p.follows = between == nullptr;
  return launch_gemm_fp8(p, s);
}

static Fp8Operand operand(const void* q, const float* scale, int64_t ld = 0) {
  Fp8Operand o;
  o.ld = ld;
  o.q = (const uint8_t*)q;
  o.scale = scale;
  return o;
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

moe_status moe_add_rmsnorm(const moe_config* cfg, const void* x, const void* residual, const void* norm_w,
                           void* res_out, void* xn, void* q, float* q_scale, void* stream) {
  NvtxScope range("moe_add_rmsnorm");
  if (!config_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (cfg->d_model > 49152) return MOE_ERR_UNSUPPORTED;
  if (cfg->n_tokens == 0) return MOE_OK;  // empty tensors may have NULL pointers
  if (!x || !norm_w || (!res_out && !xn && !q) || (q == nullptr) != (q_scale == nullptr)) return MOE_ERR_INVALID_ARG;
  if (xn && xn == res_out) return MOE_ERR_INVALID_ARG;
  return launch_add_rmsnorm(cfg->dtype, x, residual, norm_w, res_out, xn, (uint8_t*)q, q_scale, cfg->n_tokens,
                            cfg->d_model, cfg->rms_eps, (cudaStream_t)stream);
}

moe_status moe_quantize_fp8(int32_t dtype, int32_t block_rows, int32_t n_mats, int32_t rows, int32_t cols,
                            const void* x, void* q, float* scale, void* stream) {
  NvtxScope range("moe_quantize_fp8");
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if ((block_rows != 1 && block_rows != 128) || n_mats < 0 || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (n_mats > 0 && rows > 0 && (!x || !q || !scale)) return MOE_ERR_INVALID_ARG;
  if (cols > kFp8MostExtent) return MOE_ERR_UNSUPPORTED;
  return launch_quantize(dtype, block_rows, n_mats, rows, cols, x, (uint8_t*)q, scale, (cudaStream_t)stream);
}

size_t moe_workspace_size_gemm_fp8(int32_t n_groups, int32_t max_rows, int32_t n_out, int32_t k) {
  if (n_groups < 1 || n_groups > moe::TC_MAX_GROUPS || max_rows < 0 || n_out < 1 || k < 1) return 0;
  return kFp8HeaderBytes + std::max(gemm_fp8_split_bytes(false, max_rows, n_groups, true, n_out, k),
                                    gemm_fp8_split_bytes(false, max_rows, n_groups, false, n_out, k));
}

moe_status moe_gemm_fp8_tiling(int32_t swiglu, int32_t n_groups, int32_t has_offsets, int32_t max_rows, int32_t n_out,
                               int32_t k, int32_t* tiling) {
  if (n_groups < 1 || n_groups > moe::TC_MAX_GROUPS || max_rows < 1 || n_out < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if ((!has_offsets && n_groups != 1) || !tiling) return MOE_ERR_INVALID_ARG;
  gemm_fp8_tiling(swiglu != 0, max_rows, n_groups, has_offsets != 0, n_out, k, tiling);
  return MOE_OK;
}

moe_status moe_gemm_fp8(int32_t n_groups, const int32_t* offsets, int32_t max_rows, int32_t n_out, int32_t k,
                        const void* a, int64_t lda, const float* a_scale, const void* b, const float* b_scale,
                        int32_t c_dtype, void* c, void* ws, size_t ws_bytes, void* stream) {
  NvtxScope range("moe_gemm_fp8");
  if (n_groups < 1 || n_groups > moe::TC_MAX_GROUPS || max_rows < 0 || n_out < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if (offsets == nullptr && n_groups != 1) return MOE_ERR_INVALID_ARG;
  if (c_dtype != MOE_F32 && c_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (ws == nullptr || ((uintptr_t)ws % 256) != 0) return MOE_ERR_INVALID_ARG;
  if (max_rows > 0 && (!a || !a_scale || !b || !b_scale || !c)) return MOE_ERR_INVALID_ARG;
  if (lda < k) return MOE_ERR_INVALID_ARG;
  if (k % 16 || lda % 16 || lda >= kFp8MostStride || misaligned({a, b})) return MOE_ERR_UNSUPPORTED;
  if (max_rows > kFp8MostExtent || k > kFp8MostExtent || (int64_t)n_groups * n_out > kFp8MostExtent)
    return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < kFp8HeaderBytes) return MOE_ERR_WORKSPACE;  // (with no room for parts, no tile is cut)
  Fp8Gemm g;
  g.epi = c_dtype == MOE_BF16 ? EPI_STORE : EPI_F32;
  g.a = operand(a, a_scale, lda);
  g.b = operand(b, b_scale);
  g.offsets = offsets;
  g.groups = n_groups;
  g.max_rows = max_rows;
  g.nout = n_out;
  g.k = k;
  g.c = c;
  g.hdr = (int32_t*)ws;
  g.split_ws = wsp(ws, kFp8HeaderBytes);
  g.split_bytes = ws_bytes - kFp8HeaderBytes;
  return launch_gemm_fp8(g, (cudaStream_t)stream);
}

size_t moe_workspace_size_fp8(const moe_config* cfg) {
  if (!config_ok(cfg)) return 0;
  return fp8_layout(cfg).total;
}

moe_status moe_expert_ffn_fp8(const moe_config* cfg, int32_t n_groups, const int32_t* offsets, int32_t max_rows,
                              const void* x, int64_t ldx, const float* x_scale, const void* w_gate,
                              const float* w_gate_scale, const void* w_up, const float* w_up_scale,
                              const void* w_down, const float* w_down_scale, int32_t d_ff, void* y, void* ws,
                              size_t ws_bytes, void* stream) {
  NvtxScope range("moe_expert_ffn_fp8");
  MOE_TRY(check_fp8(cfg, ws, ws_bytes));
  if (n_groups < 1 || n_groups > moe::TC_MAX_GROUPS || max_rows < 0 || d_ff < 1) return MOE_ERR_INVALID_ARG;
  if (offsets == nullptr && n_groups != 1) return MOE_ERR_INVALID_ARG;
  if (d_ff % 16 || max_rows > kFp8MostExtent || (int64_t)n_groups * std::max(d_ff, cfg->d_model) > kFp8MostExtent)
    return MOE_ERR_UNSUPPORTED;
  const Fp8Layout L = fp8_layout_in(cfg, ws_bytes);
  if ((int64_t)max_rows * d_ff > L.act_elems || (int64_t)max_rows * q_blocks(d_ff) > L.act_scales)
    return MOE_ERR_WORKSPACE;
  if (max_rows == 0) return MOE_OK;
  if (!x || !x_scale || !w_gate || !w_gate_scale || !w_up || !w_up_scale || !w_down || !w_down_scale || !y)
    return MOE_ERR_INVALID_ARG;
  if (ldx < cfg->d_model) return MOE_ERR_INVALID_ARG;
  if (ldx % 16 || ldx >= kFp8MostStride || misaligned({x, w_gate, w_up, w_down}) || !one_view(w_gate, w_up))
    return MOE_ERR_UNSUPPORTED;
  Fp8Gemm p;
  p.a = operand(x, x_scale, ldx);
  p.b = operand(w_gate, w_gate_scale);
  p.b2 = operand(w_up, w_up_scale);
  p.offsets = offsets;
  p.groups = n_groups;
  p.max_rows = max_rows;
  return ffn_fp8_impl(cfg, p, operand(w_down, w_down_scale), Fp8Operand(), d_ff, y, ws, L, (cudaStream_t)stream,
                      nullptr);
}

moe_status moe_layer_forward_fp8(const moe_config* cfg, const moe_weights_fp8* w, const void* h, const void* residual,
                                 const float* bias, void* out, const moe_routing* routing, const moe_trace* trace,
                                 void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_fp8(cfg, ws, ws_bytes));
  if (w == nullptr) return MOE_ERR_INVALID_ARG;
  const bool shared = cfg->d_ff_shared > 0;
  const int N = cfg->n_tokens, d = cfg->d_model, E = cfg->n_experts, k = cfg->top_k, H = cfg->d_ff;
  if (N > 0) {
    if (!h || !out || !w->norm_w || !w->w_router || !w->w_gate || !w->w_gate_scale || !w->w_up || !w->w_up_scale ||
        !w->w_down || !w->w_down_scale)
      return MOE_ERR_INVALID_ARG;
    if (shared && (!w->ws_gate || !w->ws_gate_scale || !w->ws_up || !w->ws_up_scale || !w->ws_down ||
                   !w->ws_down_scale))
      return MOE_ERR_INVALID_ARG;
    if (misaligned({w->w_gate, w->w_up, w->w_down}) || (shared && misaligned({w->ws_gate, w->ws_up, w->ws_down})))
      return MOE_ERR_UNSUPPORTED;
    if (!one_view(w->w_gate, w->w_up) || (shared && !one_view(w->ws_gate, w->ws_up))) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)E * std::max(H, d) > kFp8MostExtent || cfg->d_ff_shared > kFp8MostExtent) return MOE_ERR_UNSUPPORTED;
  }
  cudaStream_t s = (cudaStream_t)stream;
  const Fp8Layout L = fp8_layout_in(cfg, ws_bytes);
  if (L.rows + N > kFp8MostExtent) return MOE_ERR_UNSUPPORTED;
  auto pick = [&](void* user, size_t off) { return user ? user : (void*)wsp(ws, off); };
  void* xn = wsp(ws, L.xn);
  uint8_t* xq = (uint8_t*)wsp(ws, L.xq);
  float* xs = (float*)wsp(ws, L.xs);
  float* logits = (float*)wsp(ws, L.logits);
  float* scores = routing ? routing->scores : nullptr;
  int32_t* idx = (int32_t*)pick(routing ? routing->topk_idx : nullptr, L.idx);
  float* gate = (float*)pick(routing ? routing->topk_gate : nullptr, L.gate);
  int32_t* counts = (int32_t*)pick(routing ? routing->counts : nullptr, L.counts);
  int32_t* offsets = (int32_t*)pick(routing ? routing->offsets : nullptr, L.offsets);
  int32_t* slot_row = (int32_t*)pick(routing ? routing->slot_row : nullptr, L.slot_row);
  int32_t* row_token = (int32_t*)pick(routing ? routing->row_token : nullptr, L.row_token);
  int32_t* offs_ext = (int32_t*)wsp(ws, L.offsets_ext);
  int32_t* hdr = (int32_t*)wsp(ws, L.hdr);
  uint8_t* xq_perm = (uint8_t*)wsp(ws, L.xq_perm);
  float* xs_perm = (float*)wsp(ws, L.xs_perm);
  void* y_perm = wsp(ws, L.y_perm);
  void* y_shared = shared && !L.fold ? wsp(ws, L.y_shared) : nullptr;
  NvtxScope call_range("moe_layer_forward_fp8");
  NvtxStages stages;
  auto mark = [&](void* ev, const char* next) -> moe_status {
    stages.next(next);
    if (ev && cudaEventRecord((cudaEvent_t)ev, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  };
  MOE_TRY(mark(trace ? trace->start : nullptr, "route"));
  // the residual stream: `out` holds h + residual until the combine adds the experts to it
  const void* stream_h = residual ? out : h;
  if (N > 0) {
    // the router reads xn in the act dtype, the experts its e4m3 form; few
    // experts or tokens, or router weights that TMA cannot read: the router's dot
    // products ride along with a second norm
    const bool tc = cfg->dtype == MOE_BF16 && E >= 64 && N >= 512 && !misaligned({w->w_router});
    MOE_TRY(launch_add_rmsnorm(cfg->dtype, h, residual, w->norm_w, residual ? out : nullptr, tc ? xn : nullptr, xq,
                               xs, N, d, cfg->rms_eps, s));
    if (tc)
      MOE_TRY(launch_gemm_tc(EPI_F32, xn, w->w_router, nullptr, nullptr, 1, N, E, d, logits, E, hdr, s));
    else
      MOE_TRY(launch_rmsnorm_router(cfg->dtype, stream_h, w->norm_w, w->w_router, nullptr, logits, N, d, E,
                                    cfg->rms_eps, s));
  }
  MOE_TRY(launch_topk(logits, bias, scores, idx, gate, nullptr, N, E, k, s));
  MOE_TRY(mark(trace ? trace->routed : nullptr, "permute"));
  MOE_TRY(launch_permute(idx, N, k, E, (int)capacity_of(cfg), (int32_t*)wsp(ws, L.hist), offsets, slot_row, row_token,
                         s, L.fold ? offs_ext : nullptr, L.fold ? N : 0, counts));
  // rows of d e4m3 codes move as d / 2 two-byte elements, their scales as fp32 rows
  MOE_TRY(launch_gather(MOE_BF16, xq, slot_row, N, k, xq_perm, d / 2, s, hdr));
  MOE_TRY(launch_gather(MOE_F32, xs, slot_row, N, k, xs_perm, q_blocks(d), s, hdr));
  MOE_TRY(mark(trace ? trace->permuted : nullptr, "gate_up"));
  const int R = (int)L.rows;
  Fp8Gemm p;
  p.a = operand(xq_perm, xs_perm, d);
  p.b = operand(w->w_gate, w->w_gate_scale);
  p.b2 = operand(w->w_up, w->w_up_scale);
  p.offsets = L.fold ? offs_ext : offsets;
  p.groups = L.fold ? E + 1 : E;
  p.max_rows = L.fold ? R + N : R;
  Fp8Operand down_shared;
  if (L.fold) {
    p.sb = operand(w->ws_gate, w->ws_gate_scale);
    p.sb2 = operand(w->ws_up, w->ws_up_scale);
    p.sa = operand(xq, xs, d);
    p.sa_rows = N;
    down_shared = operand(w->ws_down, w->ws_down_scale);
  }
  if (p.max_rows > 0)
    MOE_TRY(ffn_fp8_impl(cfg, p, operand(w->w_down, w->w_down_scale), down_shared, H, y_perm, ws, L, s,
                         trace ? trace->gate_up : nullptr));
  else
    MOE_TRY(mark(trace ? trace->gate_up : nullptr, "gate_up"));
  MOE_TRY(mark(trace ? trace->down : nullptr, "shared"));
  if (y_shared && N > 0) {
    Fp8Gemm ps;
    ps.a = operand(xq, xs, d);
    ps.b = operand(w->ws_gate, w->ws_gate_scale);
    ps.b2 = operand(w->ws_up, w->ws_up_scale);
    ps.max_rows = N;
    MOE_TRY(ffn_fp8_impl(cfg, ps, operand(w->ws_down, w->ws_down_scale), Fp8Operand(), cfg->d_ff_shared, y_shared, ws,
                         L, s, nullptr));
  }
  MOE_TRY(mark(trace ? trace->shared : nullptr, "combine"));
  MOE_TRY(launch_combine(cfg->dtype, stream_h, y_perm, slot_row, gate, y_shared, out, N, d, k, s,
                         L.fold ? offs_ext : nullptr, L.fold ? E : 0));
  return mark(trace ? trace->combined : nullptr, nullptr);
}

}  // extern "C"
