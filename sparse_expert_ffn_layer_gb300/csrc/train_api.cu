// C-ABI front end of the training and adapter calls (include/moe.h): argument checks, workspace
// carving and the launch sequence of each entry point.
#include <algorithm>

#include "../../include/moe.h"
#include "launch.h"

using namespace moe;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxE = 1024;
constexpr int kMaxRank = 128;
constexpr int kMaxRows = 1 << 30;               // index arithmetic in 32 bits
constexpr int kMaxCols = 1 << 20;               // blocks along a grid's second dimension

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
cudaStream_t as_stream(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

#define MOE_TRY(expr)                          \
  do {                                         \
    cudaError_t e__ = (expr);                  \
    if (e__ != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

// No exception crosses the C boundary (the launch plans' tables and locks may throw).
template <typename F>
moe_status guarded(F f) noexcept {
  try {
    return f();
  } catch (...) {
    return MOE_ERR_CUDA;
  }
}

bool dtype_ok(moe_dtype t) { return t == MOE_F16 || t == MOE_F32; }
int lane_elems(moe_dtype t) { return t == MOE_F16 ? 8 : 4; }     // elements of 16 bytes

moe_status check_router(int T, int E, int k) {
  if (T < 0 || E < 1 || (k != 1 && k != 2) || k > E) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || (long long)T * E > 0x7fffffffLL || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_adapter(int T, int d_in, int d_out, int r, int N, int S_max, moe_dtype dtype) {
  if (T < 0 || S_max < 0 || d_in < 1 || d_out < 1 || r < 1 || N < 1) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  const int v = lane_elems(dtype);
  if (N > kMaxE || r > kMaxRank || r % 8 || d_in % v || d_out % v) return MOE_ERR_UNSUPPORTED;
  if (T > kMaxRows || S_max > kMaxRows || d_in > kMaxCols || d_out > kMaxCols) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// An empty call launches nothing that would write the status word: it is cleared here, in a workspace
// that is device memory (an empty call needs none).
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

// [status][dh][partial h][workspace of the sums dA and dB]
size_t hidden_bytes(int r, size_t rows) { return align_up(rows * r * sizeof(float)); }
size_t adapter_sums_at(int d_in, int d_out, int r, int N, int S_max, moe_dtype dtype) {
  size_t b = kAlign + hidden_bytes(r, S_max);
  if (adapter_tall(S_max, N, r, dtype == MOE_F16)) b += hidden_bytes(r, adapter_partial_rows(S_max));
  return b;
}
size_t adapter_bytes(int d_in, int d_out, int r, int N, int S_max, moe_dtype dtype) {
  return adapter_sums_at(d_in, d_out, r, N, S_max, dtype) +
         align_up(row_sums_bytes(d_in, r, d_out, r, dtype == MOE_F16, S_max));
}

}  // namespace

extern "C" {

moe_status moe_balance_workspace_size(int T, int E, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe_status st = check_router(T, E, 1);
  if (st != MOE_OK) return st;
  *bytes = align_up(balance_records_bytes(E));
  return MOE_OK;
}

moe_status moe_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* token_mask,
                            int T, int E, int k, int32_t* counts, float* prob_mean, float* losses,
                            int32_t* n_valid, void* workspace, size_t ws_bytes, moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    moe_status st = check_router(T, E, k);
    if (st != MOE_OK) return st;
    if (!counts || !prob_mean || !losses || !n_valid) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !topk_idx)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(counts) || !aligned16(prob_mean) ||
        !aligned16(losses) || !aligned16(n_valid) || !aligned16(workspace))
      return MOE_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < align_up(balance_records_bytes(E))) return MOE_ERR_WORKSPACE;
    MOE_TRY(launch_balance_loss(logits, topk_idx, token_mask, T, E, k, counts, prob_mean, losses,
                                n_valid, static_cast<float*>(workspace), as_stream(stream)));
    return MOE_OK;
  });
}

moe_status moe_gate_backward_workspace_size(int T, int d, int E, moe_dtype dtype, size_t* bytes) {
  if (!bytes || d < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  moe_status st = check_router(T, E, 1);
  if (st != MOE_OK) return st;
  if (d % lane_elems(dtype) || d > kMaxCols) return MOE_ERR_UNSUPPORTED;
  // either form
  size_t most = row_sums_bytes(d, E, 0, 0, dtype == MOE_F16, T);
  if (dtype == MOE_F16 && E <= 256) most = std::max(most, gate_tc_bytes(T, d, E));
  *bytes = kAlign + align_up(most);
  return MOE_OK;
}

moe_status moe_gate_topk_backward(const float* logits, const int32_t* topk_idx, const float* dtopk_w,
                                  const float* dlosses, const int32_t* counts, const int32_t* n_valid,
                                  const uint8_t* token_mask, const void* tokens, const float* Wg,
                                  moe_dtype dtype, int T, int d, int E, int k, float* dlogits,
                                  float* dWg, const void* dtokens_in, void* dtokens, void* workspace,
                                  size_t ws_bytes, moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    moe_status st = check_router(T, E, k);
    if (st != MOE_OK) return st;
    const bool deep = dWg || dtokens;
    if (deep && (d < 1 || !dtype_ok(dtype))) return MOE_ERR_INVALID_ARG;
    if (deep && (d % lane_elems(dtype) || d > kMaxCols)) return MOE_ERR_UNSUPPORTED;
    cudaStream_t s = as_stream(stream);
    if (T == 0) {
      if (dWg) MOE_TRY(cudaMemsetAsync(dWg, 0, (size_t)d * E * sizeof(float), s));
      return clear_status(workspace, ws_bytes, s);   // (dtokens without rows may be a null pointer)
    }
    if (!logits || !topk_idx || !dlogits || (!dtopk_w && !dlosses)) return MOE_ERR_INVALID_ARG;
    if (dlosses && (!counts || !n_valid)) return MOE_ERR_INVALID_ARG;
    if ((dWg && !tokens) || (dtokens && !Wg) || (dtokens_in && !dtokens)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(dtopk_w) || !aligned4(dlosses) ||
        !aligned4(counts) || !aligned4(n_valid) || !aligned16(tokens) || !aligned16(Wg) ||
        !aligned16(dlogits) || !aligned16(dWg) || !aligned16(dtokens_in) || !aligned16(dtokens) ||
        !aligned16(workspace))
      return MOE_ERR_UNSUPPORTED;
    size_t need = 0;
    if (deep) {
      st = moe_gate_backward_workspace_size(T, d, E, dtype, &need);
      if (st != MOE_OK) return st;
      if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
    }
    if (dtokens && dWg && dtokens == tokens) return MOE_ERR_INVALID_ARG;   // written while read
    const int f16 = dtype == MOE_F16;
    uint8_t* ws = static_cast<uint8_t*>(workspace) + kAlign;
    int* status = deep ? static_cast<int*>(workspace) : nullptr;
    // Masked tokens may hold anything: their rows are left out of dWg's sums (dtokens need no mask:
    // dlogits are zero).
    const bool tc = f16 && gate_tc_ok(T, d, E, dWg, dtokens);
    if (tc)
      MOE_TRY(launch_gate_tc(logits, topk_idx, dtopk_w, dlosses, counts, n_valid, token_mask, k, dlogits,
                             static_cast<const __half*>(tokens), Wg, dWg,
                             static_cast<const __half*>(dtokens_in), static_cast<__half*>(dtokens), ws,
                             status, T, d, E, s));
    else
      MOE_TRY(launch_dlogits(logits, topk_idx, dtopk_w, dlosses, counts, n_valid, token_mask, T, E, k,
                             dlogits, status, s));
    if (dWg && !tc)
      MOE_TRY(launch_row_sums(tokens, dlogits, dWg, d, E, 0, nullptr, nullptr, nullptr, 0, 0, 0, nullptr,
                              nullptr, nullptr, token_mask, ws, f16, T, T, 1, /*pdl=*/true, s));
    if (dtokens && !tc) MOE_TRY(launch_gate_dx(dlogits, Wg, dtokens_in, f16, T, d, E, dtokens, s));
    return MOE_OK;
  });
}

moe_status moe_combine_backward(const void* dout, const void* expert_out, const int32_t* slot_of,
                                const float* topk_w, moe_dtype dtype, int T, int d, int k, int S_max,
                                void* dexpert_out, float* dtopk_w, moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    if (T < 0 || d < 1 || S_max < 0 || (k != 1 && k != 2)) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (T > kMaxRows || d > kMaxCols) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!dexpert_out && !dtopk_w) return MOE_ERR_INVALID_ARG;
    if (!dout || !slot_of || (dexpert_out && !topk_w) || (dtopk_w && !expert_out && S_max > 0))
      return MOE_ERR_INVALID_ARG;
    if (!aligned16(dout) || !aligned16(expert_out) || !aligned16(slot_of) || !aligned16(topk_w) ||
        !aligned16(dexpert_out) || !aligned16(dtopk_w))
      return MOE_ERR_UNSUPPORTED;
    if (dexpert_out && dexpert_out == dout) return MOE_ERR_INVALID_ARG;   // written while read
    MOE_TRY(launch_combine_backward(dout, expert_out, slot_of, topk_w, dtype == MOE_F16, T, d, k, S_max,
                                    dexpert_out, dtopk_w, as_stream(stream)));
    return MOE_OK;
  });
}

moe_status moe_adapter_workspace_size(int T, int d_in, int d_out, int r, int N, int S_max,
                                      moe_dtype dtype, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe_status st = check_adapter(T, d_in, d_out, r, N, S_max, dtype);
  if (st != MOE_OK) return st;
  *bytes = adapter_bytes(d_in, d_out, r, N, S_max, dtype);
  return MOE_OK;
}

moe_status moe_adapter_forward(const void* tokens, const int32_t* perm, const int32_t* offsets,
                               const void* A, const void* B, const float* scale, const void* base,
                               moe_dtype dtype, int T, int d_in, int d_out, int r, int N, int S_max,
                               void* out, float* hidden, void* workspace, size_t ws_bytes,
                               moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    moe_status st = check_adapter(T, d_in, d_out, r, N, S_max, dtype);
    if (st != MOE_OK) return st;
    if (T == 0 || S_max == 0) return clear_status(workspace, ws_bytes, as_stream(stream));
    if (!tokens || !perm || !offsets || !A || !B || !scale || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(tokens) || !aligned4(perm) || !aligned4(offsets) || !aligned16(A) || !aligned16(B) ||
        !aligned4(scale) || !aligned16(base) || !aligned16(out) || !aligned16(hidden) ||
        !aligned16(workspace))
      return MOE_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < adapter_bytes(d_in, d_out, r, N, S_max, dtype)) return MOE_ERR_WORKSPACE;
    if (out == tokens) return MOE_ERR_INVALID_ARG;   // written while read
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* partial = reinterpret_cast<float*>(ws + kAlign + hidden_bytes(r, S_max));
    MOE_TRY(launch_adapter(tokens, A, B, base, out, hidden, partial, scale, perm, offsets,
                           static_cast<int*>(workspace), dtype == MOE_F16, /*transposed=*/false, T, d_in,
                           d_out, r, N, S_max, as_stream(stream)));
    return MOE_OK;
  });
}

moe_status moe_adapter_backward(const void* dout, const void* tokens, const float* hidden,
                                const int32_t* perm, const int32_t* offsets, const void* A,
                                const void* B, const float* scale, const void* dtokens_in,
                                moe_dtype dtype, int T, int d_in, int d_out, int r, int N, int S_max,
                                void* dtokens, float* dA, float* dB, void* workspace, size_t ws_bytes,
                                moe_stream_t stream) {
  return guarded([&]() -> moe_status {
    moe_status st = check_adapter(T, d_in, d_out, r, N, S_max, dtype);
    if (st != MOE_OK) return st;
    // (the tokens' gradient of an empty batch may be a null pointer: it has no rows)
    if (T > 0 && !dtokens && !dA && !dB) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = as_stream(stream);
    if (T == 0 || S_max == 0) {
      if (dA) MOE_TRY(cudaMemsetAsync(dA, 0, (size_t)N * d_in * r * sizeof(float), s));
      if (dB) MOE_TRY(cudaMemsetAsync(dB, 0, (size_t)N * r * d_out * sizeof(float), s));
      return clear_status(workspace, ws_bytes, s);
    }
    if (!dout || !perm || !offsets || !A || !B || !scale) return MOE_ERR_INVALID_ARG;
    if ((dA && !tokens) || (dB && !hidden) || (dtokens_in && !dtokens)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dout) || !aligned16(tokens) || !aligned16(hidden) || !aligned4(perm) ||
        !aligned4(offsets) || !aligned16(A) || !aligned16(B) || !aligned4(scale) ||
        !aligned16(dtokens_in) || !aligned16(dtokens) || !aligned16(dA) || !aligned16(dB) ||
        !aligned16(workspace))
      return MOE_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < adapter_bytes(d_in, d_out, r, N, S_max, dtype)) return MOE_ERR_WORKSPACE;
    if (dtokens && (dtokens == dout || (dA && dtokens == tokens))) return MOE_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* dh = reinterpret_cast<float*>(ws + kAlign);
    float* partial = reinterpret_cast<float*>(ws + kAlign + hidden_bytes(r, S_max));
    const int f16 = dtype == MOE_F16;
    // dh, and with it the tokens' gradient.  Without dtokens only the first product runs (dn = 0),
    // and with neither dtokens nor dA the launch only checks the indices (dk = 0 too).
    MOE_TRY(launch_adapter(dout, B, A, dtokens_in, dtokens, dA ? dh : nullptr, partial, scale, perm,
                           offsets, reinterpret_cast<int*>(ws), f16, /*transposed=*/true, T,
                           dA || dtokens ? d_out : 0, dtokens ? d_in : 0, r, N, S_max, s));
    if (dA || dB)
      MOE_TRY(launch_row_sums(
          tokens, dh, dA, d_in, r, 0, dout, hidden, dB, d_out, r, 1, scale, perm, offsets, nullptr,
          ws + adapter_sums_at(d_in, d_out, r, N, S_max, dtype), f16, T, S_max, N, /*pdl=*/true, s));
    return MOE_OK;
  });
}

}  // extern "C"
