// C-ABI front end of the block calls (include/moe.h): routing by scores, experts in 8 bits and the norms around
// a block.  Argument checks, workspace carving and the launch sequence of each entry point.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "../../include/moe.h"
#include "launch.h"

using namespace moe;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxE = 1024;
constexpr int kMaxRows = 1 << 30;               // index arithmetic in 32 bits
constexpr int kMaxCols = 1 << 20;
constexpr int kMaxNorm = 16384;                 // columns of a row that a block's registers hold

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
cudaStream_t as_stream(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

#define MOE_TRY(expr)                          \
  do {                                         \
    cudaError_t e__ = (expr);                  \
    if (e__ != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

// No exception crosses the C boundary (the tables and locks of launch plans may throw).
template <typename F>
moe_status guarded(F f) noexcept {
  try {
    return f();
  } catch (...) {
    return MOE_ERR_CUDA;
  }
}

bool dtype_ok(moe_dtype t) { return t == MOE_F16 || t == MOE_F32; }
size_t elem_bytes(moe_dtype t) { return t == MOE_F16 ? 2 : 4; }
int lane_elems(moe_dtype t) { return t == MOE_F16 ? 8 : 4; }     // elements of 16 bytes

moe_status check_route(int T, int E, int k, moe_score score) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (k > kRouteMaxK || E > kMaxE || (long long)T * E > 0x7fffffffLL || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_fp8(int T, int d, int f, int E, int S_max, moe_dtype dtype) {
  if (T < 0 || S_max < 0 || d < 1 || f < 1 || E < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F16 || d % 128 || f % 128 || E > kMaxE) return MOE_ERR_UNSUPPORTED;
  if (T > kMaxRows || S_max > kMaxRows || d > kMaxCols || f > kMaxCols) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_norm(int T, int d, int k, moe_dtype dtype) {
  if (T < 0 || d < 1 || k < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (d % lane_elems(dtype) || d > kMaxNorm || T > kMaxRows || k > kRouteMaxK) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The experts' rows, slots and weights come together, with k > 0, or not at all.
bool experts_ok(const void* expert_out, const int32_t* slot_of, const float* topk_w, int k, int S_max) {
  if (k == 0) return !expert_out && !slot_of && !topk_w;
  return slot_of && topk_w && (expert_out || S_max == 0);
}

// Memory of an argument, and whether an output shares some with an input or with another output: blocks write while others
// still read, and a sum may be written before its factor is read.
struct Span {
  const void* p;
  size_t bytes;
};
bool shared_memory(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
bool overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span& i : inputs)
      if (shared_memory(*o, i)) return true;
    for (auto q = o + 1; q != outputs.end(); ++q)
      if (shared_memory(*o, *q)) return true;
  }
  return false;
}

// An empty call launches nothing that would write the status word: it is cleared here, in a workspace that is
// device memory (an empty call needs none).
moe_status clear_status(void* workspace, size_t ws_bytes, cudaStream_t s) {
  if (!workspace || ws_bytes < sizeof(int)) return MOE_OK;
  cudaPointerAttributes at = {};
  if (cudaPointerGetAttributes(&at, workspace) != cudaSuccess) {
    cudaGetLastError();                           // no device, or not a pointer of this process
    return MOE_OK;
  }
  if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return MOE_OK;
  MOE_TRY(cudaMemsetAsync(workspace, 0, sizeof(int), s));
  return MOE_OK;
}

size_t norm_bytes(int T, int d, bool f16) {
  return align_up((size_t)std::max(norm_teams(std::max(T, 1), d, f16), 1) * 2 * d * sizeof(float));
}

}  // namespace

extern "C" {

moe_status moe_route(const void* tokens, moe_dtype dtype, const float* Wg, const float* logits_in,
                     const float* bias, const uint8_t* token_mask, int T, int d, int E, int k, moe_score score,
                     int n_groups, int top_groups, int group_top, int renormalize, float scale, float* logits_out,
                     float* scores_out, int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    if (d < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (n_groups < 1 || top_groups < 1 || top_groups > n_groups || (group_top != 1 && group_top != 2))
      return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    moe_status st = check_route(T, E, k, score);
    if (st != MOE_OK) return st;
    if (E % n_groups || k > E / n_groups * top_groups) return MOE_ERR_INVALID_ARG;
    if (n_groups > kRouteMaxGroups) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!topk_idx || !topk_w || (!logits_in && (!tokens || !Wg || !logits_out))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(tokens) || !aligned16(Wg) || !aligned16(logits_in) || !aligned16(logits_out) || !aligned16(bias) ||
        !aligned16(scores_out) || !aligned16(topk_idx) || !aligned16(topk_w))
      return MOE_ERR_UNSUPPORTED;
    const size_t te = (size_t)T * E * 4, tk = (size_t)T * k * 4;
    if (overlap({{logits_out == logits_in ? nullptr : logits_out, te}, {scores_out, te}, {topk_idx, tk}, {topk_w, tk}},
                {{logits_in ? nullptr : tokens, (size_t)T * d * elem_bytes(dtype)},
                 {logits_in ? nullptr : Wg, (size_t)d * E * 4}, {logits_in, te}, {bias, (size_t)E * 4}, {token_mask, (size_t)T}}))
      return MOE_ERR_INVALID_ARG;
    cudaStream_t s = as_stream(stream);
    if (!logits_in) MOE_TRY(launch_gate_logits(tokens, dtype == MOE_F16, Wg, T, d, E, logits_out, s));
    const ScoreArgs a{logits_in ? logits_in : logits_out, bias, token_mask, T, E, k, score == MOE_SCORE_SIGMOID,
                      n_groups, top_groups, group_top, renormalize != 0, scale,
                      logits_in && logits_out != logits_in ? logits_out : nullptr, scores_out, topk_idx, topk_w};
    MOE_TRY(launch_route(a, s, /*pdl=*/!logits_in));
    return MOE_OK;
  });
}

moe_status moe_route_backward(const float* logits, const int32_t* topk_idx, const float* dtopk_w,
                              const float* dscores, const uint8_t* token_mask, const void* tokens, const float* Wg,
                              moe_dtype dtype, int T, int d, int E, int k, moe_score score, int renormalize,
                              float scale, float* dlogits, float* dWg, const void* dtokens_in, void* dtokens,
                              void* workspace, size_t ws_bytes, moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    moe_status st = check_route(T, E, k, score);
    if (st != MOE_OK) return st;
    if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    const bool deep = dWg || dtokens;
    if (deep && (d < 1 || !dtype_ok(dtype))) return MOE_ERR_INVALID_ARG;
    if (deep && (d % lane_elems(dtype) || d > kMaxCols)) return MOE_ERR_UNSUPPORTED;
    cudaStream_t s = as_stream(stream);
    if (T == 0) {
      if (dWg) MOE_TRY(cudaMemsetAsync(dWg, 0, (size_t)d * E * sizeof(float), s));
      return clear_status(workspace, ws_bytes, s);
    }
    if (!logits || !topk_idx || !dlogits || (!dtopk_w && !dscores)) return MOE_ERR_INVALID_ARG;
    if ((dWg && !tokens) || (dtokens && !Wg) || (dtokens_in && !dtokens)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(dtopk_w) || !aligned16(dscores) ||
        !aligned16(tokens) || !aligned16(Wg) || !aligned16(dlogits) || !aligned16(dWg) || !aligned16(dtokens_in) ||
        !aligned16(dtokens) || !aligned16(workspace))
      return MOE_ERR_UNSUPPORTED;
    size_t need = 0;
    if (deep) {
      st = moe_gate_backward_workspace_size(T, d, E, dtype, &need);
      if (st != MOE_OK) return st;
      if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
    }
    const size_t te = (size_t)T * E * 4, tk = (size_t)T * k * 4, de = (size_t)d * E * 4;
    const size_t td = deep ? (size_t)T * d * elem_bytes(dtype) : 0;
    if (overlap({{dlogits, te}, {dWg, de}, {dtokens, td}, {deep ? workspace : nullptr, need}},
                {{logits, te}, {topk_idx, tk}, {dtopk_w, tk}, {dscores, te}, {token_mask, (size_t)T},
                 {dWg ? tokens : nullptr, td}, {dtokens ? Wg : nullptr, de},
                 {dtokens_in == dtokens ? nullptr : dtokens_in, td}}))
      return MOE_ERR_INVALID_ARG;
    const int f16 = dtype == MOE_F16;
    uint8_t* ws = static_cast<uint8_t*>(workspace) + kAlign;
    int* status = deep ? static_cast<int*>(workspace) : nullptr;
    const RouteScore how{dscores, score == MOE_SCORE_SIGMOID, renormalize != 0, scale};
    const bool tc = deep && f16 && gate_tc_ok(T, d, E, dWg, dtokens);
    if (tc)
      MOE_TRY(launch_gate_tc(logits, topk_idx, dtopk_w, nullptr, nullptr, nullptr, token_mask, k, dlogits,
                             static_cast<const __half*>(tokens), Wg, dWg, static_cast<const __half*>(dtokens_in),
                             static_cast<__half*>(dtokens), ws, status, T, d, E, s, &how));
    else
      MOE_TRY(launch_dlogits(logits, topk_idx, dtopk_w, nullptr, nullptr, nullptr, token_mask, T, E, k, dlogits,
                             status, s, &how));
    if (dWg && !tc)
      MOE_TRY(launch_row_sums(tokens, dlogits, dWg, d, E, 0, nullptr, nullptr, nullptr, 0, 0, 0, nullptr,
                              nullptr, nullptr, token_mask, ws, f16, T, T, 1, /*pdl=*/true, s));
    if (dtokens && !tc) MOE_TRY(launch_gate_dx(dlogits, Wg, dtokens_in, f16, T, d, E, dtokens, s));
    return MOE_OK;
  });
}

moe_status moe_fp8_quantize(const void* W, moe_dtype dtype, int E, int K, int N, uint8_t* Wq, float* scales,
                            moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    if (E < 1 || K < 1 || N < 1 || !dtype_ok(dtype) || !W || !Wq || !scales) return MOE_ERR_INVALID_ARG;
    if (K % 128 || N % 128 || K > kMaxCols || N > kMaxCols) return MOE_ERR_UNSUPPORTED;
    if ((long long)E * (K / 128) * (N / 128) > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(W) || !aligned16(Wq) || !aligned4(scales)) return MOE_ERR_UNSUPPORTED;
    const size_t n = (size_t)E * K * N;
    if (overlap({{Wq, n}, {scales, n / 16384 * 4}}, {{W, n * elem_bytes(dtype)}})) return MOE_ERR_INVALID_ARG;
    MOE_TRY(launch_fp8_weights(W, dtype == MOE_F16, E, K, N, Wq, scales, as_stream(stream)));
    return MOE_OK;
  });
}

moe_status moe_expert_fp8_workspace_size(int T, int d, int f, int E, int S_max, moe_dtype dtype, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe_status st = check_fp8(T, d, f, E, S_max, dtype);
  if (st != MOE_OK) return st;
  *bytes = fp8_ffn_bytes(d, f, E, S_max);
  return MOE_OK;
}

moe_status moe_expert_ffn_fp8(const void* tokens, const int32_t* perm, const int32_t* offsets, const uint8_t* W1q,
                              const float* W1s, const uint8_t* W2q, const float* W2s, moe_dtype dtype, int T, int d,
                              int f, int E, int S_max, void* expert_out, void* workspace, size_t ws_bytes,
                              moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    moe_status st = check_fp8(T, d, f, E, S_max, dtype);
    if (st != MOE_OK) return st;
    if (T == 0 || S_max == 0) return clear_status(workspace, ws_bytes, as_stream(stream));
    if (!tokens || !perm || !offsets || !W1q || !W1s || !W2q || !W2s || !expert_out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(tokens) || !aligned4(perm) || !aligned4(offsets) || !aligned16(W1q) || !aligned4(W1s) ||
        !aligned16(W2q) || !aligned4(W2s) || !aligned16(expert_out) || !aligned16(workspace))
      return MOE_ERR_UNSUPPORTED;
    const size_t need = fp8_ffn_bytes(d, f, E, S_max), w = (size_t)E * d * f;
    if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
    // (expert_out may be tokens: these are in the workspace, in 8 bits, before the first row of it is written)
    if (overlap({{workspace, need}, {expert_out, (size_t)S_max * d * 2}},
                {{perm, (size_t)S_max * 4}, {offsets, (size_t)(E + 1) * 4}, {W1q, w}, {W1s, w / 16384 * 4}, {W2q, w},
                 {W2s, w / 16384 * 4}}) ||
        overlap({{workspace, need}}, {{tokens, (size_t)T * d * 2}}))
      return MOE_ERR_INVALID_ARG;
    MOE_TRY(launch_fp8_ffn(tokens, perm, offsets, W1q, W1s, W2q, W2s, T, d, f, E, S_max, expert_out,
                           static_cast<uint8_t*>(workspace), as_stream(stream)));
    return MOE_OK;
  });
}

moe_status moe_block_norm(const void* residual, const void* expert_out, const int32_t* slot_of, const float* topk_w,
                          const void* shared, const float* post_w, const float* gate, float alpha,
                          const float* next_w, float eps, moe_dtype dtype, int T, int d, int k, int S_max,
                          void* hidden_out, void* normed_out, float* rstd_post, float* rstd_next,
                          moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    if (S_max < 0 || !(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(alpha)) return MOE_ERR_INVALID_ARG;
    moe_status st = check_norm(T, d, k, dtype);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!residual || !experts_ok(expert_out, slot_of, topk_w, k, S_max)) return MOE_ERR_INVALID_ARG;
    if (!hidden_out && !normed_out) return MOE_ERR_INVALID_ARG;
    if (!normed_out != !next_w || (rstd_next && !normed_out) || (rstd_post && !post_w)) return MOE_ERR_INVALID_ARG;
    const bool with_block = k > 0 || shared;
    if (!with_block && (post_w || gate)) return MOE_ERR_INVALID_ARG;           // of a block that is not there
    if (with_block && !hidden_out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(residual) || !aligned16(expert_out) || !aligned4(slot_of) || !aligned4(topk_w) ||
        !aligned16(shared) || !aligned16(post_w) || !aligned16(gate) || !aligned16(next_w) ||
        !aligned16(hidden_out) || !aligned16(normed_out) || !aligned4(rstd_post) || !aligned4(rstd_next))
      return MOE_ERR_UNSUPPORTED;
    const size_t el = elem_bytes(dtype), row = (size_t)d * 4, td = (size_t)T * d * el, t4 = (size_t)T * 4;
    if (overlap({{hidden_out, td}, {normed_out, td}, {rstd_post, t4}, {rstd_next, t4}},
                {{residual == hidden_out ? nullptr : residual, td}, {expert_out, (size_t)S_max * d * el},
                 {slot_of, t4 * k}, {topk_w, t4 * k}, {shared, td}, {post_w, row}, {gate, row}, {next_w, row}}))
      return MOE_ERR_INVALID_ARG;
    const NormArgs a{residual, expert_out, slot_of, topk_w, shared, post_w, gate, next_w, alpha, eps, T, d, k, S_max,
                     with_block, hidden_out, normed_out, rstd_post, rstd_next};
    MOE_TRY(launch_block_norm(a, dtype == MOE_F16, as_stream(stream)));
    return MOE_OK;
  });
}

moe_status moe_block_norm_workspace_size(int T, int d, int k, moe_dtype dtype, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe_status st = check_norm(T, d, k, dtype);
  if (st != MOE_OK) return st;
  *bytes = norm_bytes(T, d, dtype == MOE_F16);
  return MOE_OK;
}

moe_status moe_block_norm_backward(const void* dhidden, const void* dnormed, const void* hidden,
                                   const float* rstd_next, const float* next_w, const void* expert_out,
                                   const int32_t* slot_of, const float* topk_w, const void* shared,
                                   const float* post_w, const float* rstd_post, const float* gate, float alpha,
                                   moe_dtype dtype, int T, int d, int k, int S_max, void* dresidual,
                                   void* dexpert_out, float* dtopk_w, void* dshared, float* dpost_w, float* dgate,
                                   float* dnext_w, void* workspace, size_t ws_bytes, moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    if (S_max < 0 || !std::isfinite(alpha)) return MOE_ERR_INVALID_ARG;
    moe_status st = check_norm(T, d, k, dtype);
    if (st != MOE_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (T == 0) {
      for (float* sum : {dpost_w, dgate, dnext_w})
        if (sum) MOE_TRY(cudaMemsetAsync(sum, 0, (size_t)d * sizeof(float), s));
      return MOE_OK;
    }
    if (!dhidden && !dnormed) return MOE_ERR_INVALID_ARG;
    if (dnormed && (!hidden || !rstd_next || !next_w)) return MOE_ERR_INVALID_ARG;
    if (!experts_ok(expert_out, slot_of, topk_w, k, S_max)) return MOE_ERR_INVALID_ARG;
    if (post_w && !rstd_post) return MOE_ERR_INVALID_ARG;
    if ((dgate && !gate) || (dpost_w && !post_w) || (dnext_w && !dnormed)) return MOE_ERR_INVALID_ARG;
    const bool with_block = k > 0 || shared;
    if (!with_block && (post_w || gate || dshared)) return MOE_ERR_INVALID_ARG;
    if (k == 0 && (dexpert_out || dtopk_w)) return MOE_ERR_INVALID_ARG;
    const bool sums = dpost_w || dgate || dnext_w;
    if (!dresidual && !dexpert_out && !dtopk_w && !dshared && !sums) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dhidden) || !aligned16(dnormed) || !aligned16(hidden) || !aligned4(rstd_next) ||
        !aligned16(next_w) || !aligned16(expert_out) || !aligned4(slot_of) || !aligned4(topk_w) ||
        !aligned16(shared) || !aligned16(post_w) || !aligned4(rstd_post) || !aligned16(gate) ||
        !aligned16(dresidual) || !aligned16(dexpert_out) || !aligned4(dtopk_w) || !aligned16(dshared) ||
        !aligned16(dpost_w) || !aligned16(dgate) || !aligned16(dnext_w) || !aligned16(workspace))
      return MOE_ERR_UNSUPPORTED;
    const bool f16 = dtype == MOE_F16;
    if (sums && (!workspace || ws_bytes < norm_bytes(T, d, f16))) return MOE_ERR_WORKSPACE;
    // (dresidual may be dhidden: a row is read before it is written, by the same threads)
    const size_t el = elem_bytes(dtype), row = (size_t)d * 4, td = (size_t)T * d * el, t4 = (size_t)T * 4;
    const size_t sd = (size_t)S_max * d * el;
    if (overlap({{dresidual, td}, {dexpert_out, sd}, {dtopk_w, t4 * k}, {dshared, td}, {dpost_w, row}, {dgate, row},
                 {dnext_w, row}, {sums ? workspace : nullptr, norm_bytes(T, d, f16)}},
                {{dhidden == dresidual ? nullptr : dhidden, td}, {dnormed, td}, {dnormed ? hidden : nullptr, td},
                 {dnormed ? rstd_next : nullptr, t4}, {dnormed ? next_w : nullptr, row}, {expert_out, sd},
                 {slot_of, t4 * k}, {topk_w, t4 * k}, {shared, td}, {post_w, row}, {post_w ? rstd_post : nullptr, t4},
                 {gate, row}}))
      return MOE_ERR_INVALID_ARG;
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.expert_out = expert_out;
    a.slot_of = slot_of;
    a.topk_w = topk_w;
    a.shared = shared;
    a.post_w = post_w;
    a.gate = gate;
    a.next_w = next_w;
    a.alpha = alpha;
    a.T = T;
    a.d = d;
    a.k = k;
    a.S_max = S_max;
    a.with_block = with_block;
    const int through = dexpert_out || dtopk_w || dshared || dpost_w || dgate;
    const NormGrads b{dhidden, dnormed, hidden, rstd_next, rstd_post, dresidual, dexpert_out, dtopk_w, dshared,
                      dpost_w, dgate, dnext_w, sums ? static_cast<float*>(workspace) : nullptr, through,
                      through && (post_w || dgate)};
    MOE_TRY(launch_block_norm_backward(a, b, f16, s));
    return MOE_OK;
  });
}

}  // extern "C"
