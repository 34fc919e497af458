// api.cu -- the C ABI of libdflash2: handle management, host-side argument
// validation and dispatch to the kernels.  The handle owns one device buffer,
// the 4-byte error word; every other byte a call needs is the caller's.
#include <cuda_runtime.h>

#include <cstdint>
#include <new>

#include "host_checks.h"

namespace {

constexpr int kK = 16;
constexpr int64_t kMaxL = 64;

// What the two attention entry points check alike; fills all of `a` but err (nothing with B or T = 0).
int check_attention(const uint16_t* q, RowStrides qs, const dflash2_kv_cache* cache, const int32_t* cache_len,
                    const uint16_t* k_new, const uint16_t* v_new, RowStrides ns, const uint64_t* tree_mask, int64_t B,
                    int64_t T, int64_t heads, float scale, uint16_t* out, float* lse, const void* workspace,
                    dflash2::AttnArgs* a) {
  if (const int st = check_queries(B, T, heads, cache, scale)) return st;
  if (const int st = view_cache(cache, B, &a->cache)) return st;
  if (B == 0 || T == 0) return DFLASH2_OK;
  // one 32-bit number counts the tiles of 128 keys over all sequences, kv heads and pairs of row tiles
  if (dflash2::tree_attn_units(B, T, heads / cache->heads, cache->heads, a->cache.capacity) >= (int64_t(1) << 31))
    return DFLASH2_ERR_UNSUPPORTED;
  if (!q || !cache_len || !out || (k_new == nullptr) != (v_new == nullptr) || (tree_mask && !k_new))
    return DFLASH2_ERR_INVALID_ARG;
  if (const int st = check_rows(&qs, B, T, heads, cache->head_dim)) return st;
  if (k_new)
    if (const int st = check_rows(&ns, B, T, cache->heads, cache->head_dim)) return st;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(cache_len, 4) ||
      !aligned(tree_mask, 8) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
    return DFLASH2_ERR_MISALIGNED;
  a->q = q;
  a->q_b = qs.b, a->q_t = qs.t, a->q_h = qs.h;
  a->cache_len = cache_len;
  a->k_new = k_new;
  a->v_new = v_new;
  a->new_b = ns.b, a->new_t = ns.t, a->new_h = ns.h;
  a->mask = tree_mask;
  a->B = B;
  a->T = static_cast<int32_t>(T);
  a->heads = static_cast<int32_t>(heads);
  a->group = static_cast<int32_t>(heads / cache->heads);
  a->scale = scale;
  a->out = out;
  a->lse = lse;
  return DFLASH2_OK;
}

}  // namespace

extern "C" {

int dflash2_version(void) { return 100; }

const char* dflash2_status_string(int status) {
  switch (status) {
    case DFLASH2_OK: return "ok";
    case DFLASH2_ERR_INVALID_ARG: return "invalid argument";
    case DFLASH2_ERR_UNSUPPORTED: return "unsupported shape or parameter";
    case DFLASH2_ERR_MISALIGNED: return "misaligned pointer or leading dimension";
    case DFLASH2_ERR_CUDA: return "CUDA runtime error";
    case DFLASH2_ERR_TIMEOUT: return "bounded device wait timed out";
    case DFLASH2_ERR_DEVICE: return "device reported an error";
    case DFLASH2_ERR_WORKSPACE: return "workspace too small";
    default: return "unknown status";
  }
}

int dflash2_create(int device, dflash2_handle** out) {
  if (out == nullptr) return DFLASH2_ERR_INVALID_ARG;
  *out = nullptr;
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || device < 0 || device >= count)
    return DFLASH2_ERR_INVALID_ARG;
  if (cudaSetDevice(device) != cudaSuccess) return DFLASH2_ERR_CUDA;
  dflash2_handle* h = new (std::nothrow) dflash2_handle;
  if (h == nullptr) return DFLASH2_ERR_CUDA;
  h->device = device;
  if (cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
      cudaMalloc(&h->err, sizeof(uint32_t)) != cudaSuccess ||
      cudaMemset(h->err, 0, sizeof(uint32_t)) != cudaSuccess) {
    if (h->err) cudaFree(h->err);
    delete h;
    return DFLASH2_ERR_CUDA;
  }
  *out = h;
  return DFLASH2_OK;
}

int dflash2_destroy(dflash2_handle* h) {
  if (h == nullptr) return DFLASH2_ERR_INVALID_ARG;
  int st = DFLASH2_OK;
  if (h->err) {
    if (cudaSetDevice(h->device) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
      st = DFLASH2_ERR_CUDA;
    cudaFree(h->err);
  }
  delete h;
  return st;
}

int dflash2_num_sms(const dflash2_handle* h) { return h ? h->num_sms : 0; }

int dflash2_get_device_error(dflash2_handle* h, void* stream, uint32_t* bits, int clear) {
  if (bad_handle(h) || bits == nullptr) return DFLASH2_ERR_INVALID_ARG;
  if (const int st = wrong_device(h)) return st;
  cudaStream_t s = as_stream(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return DFLASH2_ERR_CUDA;
  if (cudaMemcpy(bits, h->err, sizeof(uint32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return DFLASH2_ERR_CUDA;
  if (clear && cudaMemset(h->err, 0, sizeof(uint32_t)) != cudaSuccess) return DFLASH2_ERR_CUDA;
  return DFLASH2_OK;
}

int dflash2_topk(dflash2_handle* h, const uint16_t* logits, int64_t rows, int64_t V, int64_t ld,
                 int k, float* vals, int32_t* idx, void* stream) {
  const NvtxRange range("dflash2_topk");
  if (bad_handle(h) || rows < 0 || V < 0 || ld < V) return DFLASH2_ERR_INVALID_ARG;
  if (k != kK || V < kK || V >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (rows == 0) return DFLASH2_OK;
  if (!logits || !vals || !idx) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || (ld % 8) != 0 || !aligned(vals, 4) || !aligned(idx, 4))
    return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  // gridDim.y is limited to 65535 rows per launch
  for (int64_t r0 = 0; r0 < rows; r0 += 65535) {
    const int64_t n = rows - r0 < 65535 ? rows - r0 : 65535;
    const int st = launched(dflash2::launch_topk(logits + r0 * ld, n, V, ld, vals + r0 * kK,
                                                 idx + r0 * kK, h->err, h->num_sms, as_stream(stream)));
    if (st != DFLASH2_OK) return st;
  }
  return DFLASH2_OK;
}

size_t dflash2_pair_scores_workspace(const dflash2_handle* h, int64_t B, int64_t L, int64_t d) {
  if (bad_handle(h) || B <= 0 || L <= 0 || d <= 0 || d % 64 != 0) return 0;
  return dflash2::gate_workspace_bytes(B, L, d, h->num_sms);
}

int dflash2_pair_scores(dflash2_handle* h, const int32_t* cand_idx, const float* cand_val,
                        const int32_t* last_verified, const uint16_t* hs, const uint16_t* W_H,
                        const float* b_H, const uint16_t* A, const uint16_t* Bt, int64_t B,
                        int64_t L, int64_t d, int64_t V, float* gate, float* S, void* workspace,
                        size_t ws_bytes, void* stream) {
  const NvtxRange range("dflash2_pair_scores");
  if (bad_handle(h) || B < 0 || L < 0 || d <= 0 || V <= 0) return DFLASH2_ERR_INVALID_ARG;
  if (L > kMaxL || d % 64 != 0 || V >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (B == 0 || L == 0) return DFLASH2_OK;
  if (!cand_idx || !cand_val || !last_verified || !hs || !W_H || !A || !Bt || !gate || !S)
    return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(hs, 16) || !aligned(W_H, 16) || !aligned(A, 16) || !aligned(Bt, 16) ||
      !aligned(gate, 16) || !aligned(S, 16) || !aligned(cand_idx, 4) || !aligned(cand_val, 4) ||
      !aligned(last_verified, 4) || (b_H && !aligned(b_H, 4)) || (workspace && !aligned(workspace, 256)))
    return DFLASH2_ERR_MISALIGNED;
  if (workspace == nullptr || ws_bytes < dflash2::gate_workspace_bytes(B, L, d, h->num_sms))
    return DFLASH2_ERR_WORKSPACE;
  cudaStream_t s = as_stream(stream);
  if (const int st = wrong_device(h)) return st;
  const int st = launched(dflash2::launch_gate(hs, W_H, b_H, B * L, d, gate, workspace, h->err, h->num_sms, s));
  if (st != DFLASH2_OK) return st;
  return launched(dflash2::launch_pair_scores(cand_idx, cand_val, last_verified, static_cast<const float*>(workspace),
                                              b_H, gate, d, A, Bt, B, L, V, S, h->err, h->num_sms, s));
}

int dflash2_walk(dflash2_handle* h, const float* S, const int32_t* cand_idx, int64_t B, int64_t L,
                 float temperature, uint64_t seed, uint64_t offset, int32_t* draft_tok,
                 int32_t* draft_slot, float* draft_q, void* stream) {
  const NvtxRange range("dflash2_walk");
  if (bad_handle(h) || B < 0 || L < 0) return DFLASH2_ERR_INVALID_ARG;
  if (L > kMaxL || B >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (!(temperature == temperature)) return DFLASH2_ERR_INVALID_ARG;   // NaN
  if (B == 0 || L == 0) return DFLASH2_OK;
  if (!S || !cand_idx || !draft_tok || !draft_slot) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(S, 16) || !aligned(cand_idx, 4) || !aligned(draft_tok, 4) || !aligned(draft_slot, 4) ||
      (draft_q && !aligned(draft_q, 4)))
    return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_walk(S, cand_idx, B, L, temperature, seed, offset, draft_tok,
                                       draft_slot, draft_q, h->err, as_stream(stream)));
}

int dflash2_walk_viterbi(dflash2_handle* h, const float* S, const int32_t* cand_idx, int64_t B, int64_t L,
                         int32_t* draft_tok, int32_t* draft_slot, float* score, void* stream) {
  const NvtxRange range("dflash2_walk_viterbi");
  if (bad_handle(h) || B < 0 || L < 0) return DFLASH2_ERR_INVALID_ARG;
  if (L > kMaxL || B >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (B == 0 || L == 0) return DFLASH2_OK;
  if (!S || !cand_idx || !draft_tok || !draft_slot) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(S, 16) || !aligned(cand_idx, 4) || !aligned(draft_tok, 4) || !aligned(draft_slot, 4) ||
      (score && !aligned(score, 4)))
    return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_walk_viterbi(S, cand_idx, B, L, draft_tok, draft_slot, score, h->err,
                                                   as_stream(stream)));
}

int dflash2_selector_eval(dflash2_handle* h, const int32_t* gt, const int32_t* cand_idx, int64_t B, int64_t L,
                          int32_t* accept1, int32_t* accept16, int64_t* counts, void* stream) {
  const NvtxRange range("dflash2_selector_eval");
  if (bad_handle(h) || B < 0 || L < 0) return DFLASH2_ERR_INVALID_ARG;
  if (L > kMaxL || B >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (L == 0) return DFLASH2_OK;
  if (!counts || (B > 0 && (!gt || !cand_idx || !accept1 || !accept16))) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(counts, 8) || (B > 0 && (!aligned(gt, 4) || !aligned(cand_idx, 4) || !aligned(accept1, 4) ||
                                        !aligned(accept16, 4))))
    return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_selector_eval(gt, cand_idx, B, L, accept1, accept16, counts, h->num_sms,
                                                    as_stream(stream)));
}

size_t dflash2_conv2tap_workspace(const dflash2_handle* h, int64_t B, int64_t L, int64_t d) {
  if (bad_handle(h) || B <= 0 || L <= 0 || d <= 0 || d % 64 != 0) return 0;
  return dflash2::conv_workspace_bytes(B, L, d, h->num_sms);
}

int dflash2_conv2tap(dflash2_handle* h, const uint16_t* x, const uint16_t* x_prev,
                     const uint16_t* hs, const uint16_t* k0, const uint16_t* k1,
                     const uint16_t* W_c, const float* b_c, int64_t B, int64_t L, int64_t d,
                     void* y, int y_is_fp32, void* workspace, size_t ws_bytes, void* stream) {
  const NvtxRange range("dflash2_conv2tap");
  if (bad_handle(h) || B < 0 || L < 0 || d <= 0) return DFLASH2_ERR_INVALID_ARG;
  if (d % 64 != 0 || L > kMaxL || B > 65535) return DFLASH2_ERR_UNSUPPORTED;
  if (B == 0 || L == 0) return DFLASH2_OK;
  if (!x || !x_prev || !k0 || !k1 || !W_c || !y) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x_prev, 16) || (hs && !aligned(hs, 16)) || !aligned(k0, 16) ||
      !aligned(k1, 16) || !aligned(W_c, 16) || !aligned(y, 16) || (b_c && !aligned(b_c, 4)) ||
      (workspace && !aligned(workspace, 256)))
    return DFLASH2_ERR_MISALIGNED;
  if (workspace == nullptr || ws_bytes < dflash2::conv_workspace_bytes(B, L, d, h->num_sms))
    return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_conv2tap(x, x_prev, hs, k0, k1, W_c, b_c, B, L, d, y, y_is_fp32, workspace,
                                           h->err, h->num_sms, as_stream(stream)));
}

size_t dflash2_gemm_conv2tap_workspace(const dflash2_handle* h, int64_t B, int64_t L, int64_t d) {
  if (bad_handle(h) || B <= 0 || L <= 0 || d <= 0) return 0;
  return dflash2::gemm_conv_workspace_bytes(B, L, d);
}

int dflash2_gemm_conv2tap(dflash2_handle* h, const uint16_t* A, const uint16_t* W, const uint16_t* x_prev,
                          const uint16_t* hs, const uint16_t* k0, const uint16_t* k1, const uint16_t* W_c,
                          const float* b_c, int64_t B, int64_t L, int64_t K, int64_t d, float* c_work,
                          size_t c_bytes, void* y, int y_is_fp32, void* stream) {
  const NvtxRange range("dflash2_gemm_conv2tap");
  if (bad_handle(h) || B < 0 || L < 0 || K <= 0 || d <= 0) return DFLASH2_ERR_INVALID_ARG;
  if (d % 64 != 0 || K % 64 != 0 || L > kMaxL || B * L >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (B == 0 || L == 0) return DFLASH2_OK;
  if (!A || !W || !x_prev || !hs || !k0 || !k1 || !W_c || !c_work || !y) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(A, 16) || !aligned(W, 16) || !aligned(x_prev, 16) || !aligned(hs, 16) || !aligned(k0, 16) ||
      !aligned(k1, 16) || !aligned(W_c, 16) || !aligned(c_work, 16) || !aligned(y, 16) || (b_c && !aligned(b_c, 4)))
    return DFLASH2_ERR_MISALIGNED;
  if (c_bytes < dflash2::gemm_conv_workspace_bytes(B, L, d)) return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_gemm_conv2tap(A, W, x_prev, hs, k0, k1, W_c, b_c, B, L, K, d, c_work, y, y_is_fp32,
                                                h->err, h->num_sms, as_stream(stream)));
}

size_t dflash2_verify_workspace(const dflash2_handle* h, int64_t B, int64_t L, int64_t V) {
  if (bad_handle(h) || B <= 0 || L < 0 || L > kMaxL || V <= 0 || V > dflash2::verify_max_vocab()) return 0;
  return dflash2::verify_workspace_bytes(B, L, V);
}

int dflash2_verify(dflash2_handle* h, const uint16_t* target, int64_t ld, const int32_t* draft_tok,
                   const int32_t* draft_slot, const float* draft_q, const int32_t* cand_idx,
                   int64_t B, int64_t L, int64_t V, float temperature, uint64_t seed,
                   uint64_t offset, int32_t* accept_len, int32_t* out_tok, void* workspace,
                   size_t ws_bytes, void* stream) {
  const NvtxRange range("dflash2_verify");
  if (bad_handle(h) || B < 0 || L < 0 || V <= 0 || ld < V) return DFLASH2_ERR_INVALID_ARG;
  if (L > kMaxL || V > dflash2::verify_max_vocab()) return DFLASH2_ERR_UNSUPPORTED;
  if (!(temperature == temperature)) return DFLASH2_ERR_INVALID_ARG;
  if (B == 0) return DFLASH2_OK;
  const bool sampled = temperature > 0.0f;
  // an empty block (L = 0) reads no draft: only the bonus row is decided
  if (!target || (L > 0 && !draft_tok) || !accept_len || !out_tok) return DFLASH2_ERR_INVALID_ARG;
  if (sampled && L > 0 && (!draft_slot || !draft_q || !cand_idx)) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(target, 16) || (ld % 8) != 0 || !aligned(draft_tok, 4) || !aligned(accept_len, 4) ||
      !aligned(out_tok, 4) || (draft_slot && !aligned(draft_slot, 4)) ||
      (draft_q && !aligned(draft_q, 4)) || (cand_idx && !aligned(cand_idx, 4)) ||
      (workspace && !aligned(workspace, 256)))
    return DFLASH2_ERR_MISALIGNED;
  if (workspace == nullptr || ws_bytes < dflash2::verify_workspace_bytes(B, L, V)) return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_verify(target, ld, draft_tok, draft_slot, draft_q, cand_idx, B, L, V,
                                         temperature, seed, offset, accept_len, out_tok, workspace, h->err,
                                         h->num_sms, as_stream(stream)));
}

size_t dflash2_lmhead_topk_workspace(const dflash2_handle* h, int64_t M, int64_t V, int64_t d) {
  if (bad_handle(h) || M <= 0 || V <= 0 || d <= 0) return 0;
  return dflash2::lmhead_workspace_bytes(M, V, d, h->num_sms);
}

int dflash2_lmhead_topk(dflash2_handle* h, const uint16_t* hidden, const uint16_t* W, int64_t M,
                        int64_t V, int64_t d, float* vals, int32_t* idx, void* workspace,
                        size_t ws_bytes, void* stream) {
  const NvtxRange range("dflash2_lmhead_topk");
  if (bad_handle(h) || M < 0 || V < 0 || d <= 0) return DFLASH2_ERR_INVALID_ARG;
  if (d % 64 != 0 || V < kK || V >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (M == 0) return DFLASH2_OK;
  if (!hidden || !W || !vals || !idx) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(vals, 4) || !aligned(idx, 4) ||
      (workspace && !aligned(workspace, 256)))
    return DFLASH2_ERR_MISALIGNED;
  if (workspace == nullptr || ws_bytes < dflash2::lmhead_workspace_bytes(M, V, d, h->num_sms))
    return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_lmhead_topk(hidden, W, M, V, d, vals, idx, workspace, h->num_sms,
                                              h->err, as_stream(stream)));
}

int dflash2_lmhead_topk_gate(dflash2_handle* h, const uint16_t* hidden, const uint16_t* W, const uint16_t* W_H,
                             const float* b_H, int64_t M, int64_t V, int64_t d, float* vals, int32_t* idx,
                             float* gate, void* workspace, size_t ws_bytes, void* stream) {
  const NvtxRange range("dflash2_lmhead_topk_gate");
  if (bad_handle(h) || M < 0 || V < 0 || d <= 0) return DFLASH2_ERR_INVALID_ARG;
  if (d % 64 != 0 || V < kK || V >= (int64_t(1) << 31) - 256) return DFLASH2_ERR_UNSUPPORTED;
  if (M == 0) return DFLASH2_OK;
  if (!hidden || !W || !W_H || !vals || !idx || !gate) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(W_H, 16) || !aligned(vals, 4) || !aligned(idx, 4) ||
      !aligned(gate, 16) || (b_H && !aligned(b_H, 4)) || (workspace && !aligned(workspace, 256)))
    return DFLASH2_ERR_MISALIGNED;
  if (workspace == nullptr || ws_bytes < dflash2::lmhead_workspace_bytes(M, V, d, h->num_sms))
    return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_lmhead_topk_gate(hidden, W, W_H, b_H, M, V, d, vals, idx, gate, workspace,
                                                   h->num_sms, h->err, as_stream(stream)));
}

size_t dflash2_pair_scores_proj_workspace(const dflash2_handle* h, int64_t B, int64_t L) {
  if (bad_handle(h) || B <= 0 || L <= 0 || L > kMaxL) return 0;
  return dflash2::proj_workspace_bytes(B, L);
}

int dflash2_pair_scores_proj(dflash2_handle* h, const int32_t* cand_idx, const float* cand_val,
                             const int32_t* last_verified, const float* gate, const uint16_t* E,
                             const uint16_t* W_A, const uint16_t* W_B, int64_t B, int64_t L, int64_t d, int64_t V,
                             float* P, size_t P_bytes, float* S, void* stream) {
  const NvtxRange range("dflash2_pair_scores_proj");
  if (bad_handle(h) || B < 0 || L < 0 || d <= 0 || V <= 0) return DFLASH2_ERR_INVALID_ARG;
  if (d % 64 != 0 || L > kMaxL || V >= (int64_t(1) << 31) || B * L >= (int64_t(1) << 26))
    return DFLASH2_ERR_UNSUPPORTED;
  if (B == 0 || L == 0) return DFLASH2_OK;
  if (!cand_idx || !cand_val || !last_verified || !gate || !E || !W_A || !W_B || !P || !S)
    return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(cand_idx, 4) || !aligned(cand_val, 4) || !aligned(last_verified, 4) || !aligned(gate, 16) ||
      !aligned(E, 16) || !aligned(W_A, 16) || !aligned(W_B, 16) || !aligned(P, 16) || !aligned(S, 4))
    return DFLASH2_ERR_MISALIGNED;
  if (P_bytes < dflash2::proj_workspace_bytes(B, L)) return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_pair_scores_proj(cand_idx, cand_val, last_verified, gate, E, W_A, W_B, B, L, d,
                                                   V, P, S, h->num_sms, h->err, as_stream(stream)));
}

int dflash2_selftest_wait_timeout(dflash2_handle* h, uint64_t limit_ns, uint32_t* words, void* stream) {
  const NvtxRange range("dflash2_selftest_wait_timeout");
  if (bad_handle(h) || words == nullptr || limit_ns == 0 || limit_ns > dflash2::kWaitLimitNs)
    return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(words, 4)) return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  return launched(dflash2::launch_wait_timeout_selftest(words, limit_ns, h->err, words + 1, as_stream(stream)));
}

int dflash2_lmhead_topk_noalloc(dflash2_handle* h, const uint16_t* hidden, const uint16_t* W, int64_t M,
                                int64_t V, int64_t d, float* vals, int32_t* idx, void* stream) {
  const NvtxRange range("dflash2_lmhead_topk_noalloc");
  if (bad_handle(h) || M < 0 || V < 0 || d <= 0) return DFLASH2_ERR_INVALID_ARG;
  if (d % 64 != 0 || V < kK || V >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
  if (M == 0) return DFLASH2_OK;
  if (!hidden || !W || !vals || !idx) return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(vals, 4) || !aligned(idx, 4))
    return DFLASH2_ERR_MISALIGNED;
  if (dflash2::lmhead_workspace_bytes(M, V, d, h->num_sms) > dflash2::kLmheadNoAllocScratchBytes)
    return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  void* scratch = nullptr;
  if (dflash2::lmhead_noalloc_scratch(h->device, &scratch) != cudaSuccess) return DFLASH2_ERR_CUDA;
  return launched(dflash2::launch_lmhead_topk(hidden, W, M, V, d, vals, idx, scratch, h->num_sms, h->err,
                                              as_stream(stream)));
}

size_t dflash2_tree_attention_workspace(const dflash2_handle* h, int64_t B, int64_t T, int64_t heads,
                                        int64_t kv_heads, int64_t head_dim) {
  if (bad_handle(h) || B <= 0 || T <= 0 || T > dflash2::kMaxNodes || kv_heads <= 0 || heads <= 0 ||
      heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return dflash2::tree_attn_workspace_bytes(B, T, heads, kv_heads, head_dim, h->num_sms);
}

int dflash2_tree_attention(dflash2_handle* h, const uint16_t* q, int64_t q_batch_stride, int64_t q_token_stride,
                           int64_t q_head_stride, const dflash2_kv_cache* cache, const int32_t* cache_len,
                           const uint16_t* k_new, const uint16_t* v_new, int64_t new_batch_stride,
                           int64_t new_token_stride, int64_t new_head_stride, const uint64_t* tree_mask, int64_t B,
                           int64_t T, int64_t heads, float scale, uint16_t* out, float* lse, void* workspace,
                           size_t ws_bytes, void* stream) {
  const NvtxRange range("dflash2_tree_attention");
  if (bad_handle(h)) return DFLASH2_ERR_INVALID_ARG;
  dflash2::AttnArgs a;
  if (const int st = check_attention(q, {q_batch_stride, q_token_stride, q_head_stride}, cache, cache_len, k_new, v_new,
                                     {new_batch_stride, new_token_stride, new_head_stride}, tree_mask, B, T, heads, scale,
                                     out, lse, workspace, &a))
    return st;
  if (B == 0 || T == 0) return DFLASH2_OK;
  if (ws_bytes < dflash2::tree_attn_workspace_bytes(B, T, heads, cache->heads, cache->head_dim, h->num_sms) ||
      workspace == nullptr)
    return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  a.err = h->err;
  return launched(dflash2::launch_tree_attn(a, cache->head_dim, workspace, h->num_sms, as_stream(stream)));
}

size_t dflash2_prefix_attention_workspace(const dflash2_handle* h, int64_t B, int64_t T, int64_t heads,
                                          int64_t kv_heads, int64_t head_dim) {
  if (bad_handle(h) || B <= 0 || B > 65535 || T <= 0 || T > dflash2::kMaxNodes || kv_heads <= 0 || heads <= 0 ||
      kv_heads > kMaxKvHeads || heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return dflash2::prefix_attn_workspace_bytes(B, T, heads, kv_heads, head_dim, h->num_sms);
}

int dflash2_prefix_attention(dflash2_handle* h, const uint16_t* q, int64_t q_batch_stride, int64_t q_token_stride,
                             int64_t q_head_stride, const dflash2_kv_cache* cache, const int32_t* cache_len,
                             const int32_t* prefix_len, const int32_t* prefix_start, int64_t groups,
                             const uint16_t* k_new, const uint16_t* v_new, int64_t new_batch_stride,
                             int64_t new_token_stride, int64_t new_head_stride, const uint64_t* tree_mask, int64_t B,
                             int64_t T, int64_t heads, float scale, uint16_t* out, float* lse, void* workspace,
                             size_t ws_bytes, void* stream) {
  const NvtxRange range("dflash2_prefix_attention");
  if (bad_handle(h) || groups < 0 || groups > B || (groups > 1 && !prefix_start) || (groups > 0 && !prefix_len))
    return DFLASH2_ERR_INVALID_ARG;
  dflash2::PrefixArgs x;
  dflash2::AttnArgs& a = x.attn;
  if (const int st = check_attention(q, {q_batch_stride, q_token_stride, q_head_stride}, cache, cache_len, k_new, v_new,
                                     {new_batch_stride, new_token_stride, new_head_stride}, tree_mask, B, T, heads, scale,
                                     out, lse, workspace, &a))
    return st;
  if (B == 0 || T == 0) return DFLASH2_OK;
  if (!aligned(prefix_len, 4) || !aligned(prefix_start, 4)) return DFLASH2_ERR_MISALIGNED;
  if (ws_bytes < dflash2::prefix_attn_workspace_bytes(B, T, heads, cache->heads, cache->head_dim, h->num_sms) ||
      workspace == nullptr)
    return DFLASH2_ERR_WORKSPACE;
  if (const int st = wrong_device(h)) return st;
  x.start = prefix_start;
  x.len = prefix_len;
  x.groups = static_cast<int32_t>(groups);
  a.err = h->err;
  return launched(dflash2::launch_prefix_attn(x, cache->head_dim, workspace, h->num_sms, as_stream(stream)));
}

int dflash2_cache_commit(dflash2_handle* h, const uint16_t* k_new, const uint16_t* v_new, int64_t new_batch_stride,
                         int64_t new_token_stride, int64_t new_head_stride, const dflash2_kv_cache* cache,
                         const int32_t* cache_len, const int32_t* count, const int32_t* path, int64_t B, int64_t T,
                         float* scores, int64_t scores_ld, int32_t* new_len, void* stream) {
  const NvtxRange range("dflash2_cache_commit");
  if (bad_handle(h) || B < 0 || T < 0 || (scores && scores_ld < 0)) return DFLASH2_ERR_INVALID_ARG;
  if (T > dflash2::kMaxNodes || B > 65535) return DFLASH2_ERR_UNSUPPORTED;
  dflash2::CommitArgs a;
  if (const int st = view_cache(cache, B, &a.cache)) return st;
  if (B == 0) return DFLASH2_OK;
  if (!cache_len || !new_len || (T > 0 && (!k_new || !v_new))) return DFLASH2_ERR_INVALID_ARG;
  // one CTA of a sequence writes its new length while others may still read these
  if (overlap(new_len, B, cache_len, B) || overlap(new_len, B, count, B)) return DFLASH2_ERR_INVALID_ARG;
  RowStrides ns = {new_batch_stride, new_token_stride, new_head_stride};
  if (const int st = check_rows(&ns, B, T, cache->heads, cache->head_dim)) return st;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(cache_len, 4) || !aligned(count, 4) ||
      !aligned(path, 4) || !aligned(scores, 4) || !aligned(new_len, 4))
    return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  a.k_new = k_new;
  a.v_new = v_new;
  a.new_b = ns.b, a.new_t = ns.t, a.new_h = ns.h;
  a.cache_len = cache_len;
  a.count = count;
  a.path = path;
  a.B = B;
  a.T = static_cast<int32_t>(T);
  a.scores = scores;
  a.scores_ld = scores_ld;
  a.new_len = new_len;
  a.err = h->err;
  return launched(dflash2::launch_cache_commit(a, cache->head_dim, as_stream(stream)));
}

int dflash2_cache_scores(dflash2_handle* h, const uint16_t* q, int64_t q_batch_stride, int64_t q_token_stride,
                         int64_t q_head_stride, const float* lse, const dflash2_kv_cache* cache,
                         const int32_t* cache_len, const int32_t* count, const int32_t* path, int64_t B, int64_t T,
                         int64_t heads, float scale, float* scores, int64_t scores_ld, void* stream) {
  const NvtxRange range("dflash2_cache_scores");
  if (bad_handle(h) || scores_ld < 0) return DFLASH2_ERR_INVALID_ARG;
  if (const int st = check_queries(B, T, heads, cache, scale)) return st;
  dflash2::ScoresArgs a;
  if (const int st = view_cache(cache, B, &a.cache)) return st;
  if (B == 0 || T == 0) return DFLASH2_OK;
  if (dflash2::tree_attn_units(B, 1, 1, cache->heads, a.cache.capacity) >= (int64_t(1) << 31))
    return DFLASH2_ERR_UNSUPPORTED;
  if (!q || !lse || !cache_len || !scores) return DFLASH2_ERR_INVALID_ARG;
  RowStrides qs = {q_batch_stride, q_token_stride, q_head_stride};
  if (const int st = check_rows(&qs, B, T, heads, cache->head_dim)) return st;
  if (!aligned(q, 16) || !aligned(lse, 4) || !aligned(cache_len, 4) || !aligned(count, 4) || !aligned(path, 4) ||
      !aligned(scores, 4))
    return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  a.q = q;
  a.q_b = qs.b, a.q_t = qs.t, a.q_h = qs.h;
  a.lse = lse;
  a.cache_len = cache_len;
  a.count = count;
  a.path = path;
  a.B = B;
  a.T = static_cast<int32_t>(T);
  a.heads = static_cast<int32_t>(heads);
  a.group = static_cast<int32_t>(heads / cache->heads);
  a.scale = scale;
  a.scores = scores;
  a.scores_ld = scores_ld;
  a.err = h->err;
  return launched(dflash2::launch_cache_scores(a, cache->head_dim, h->num_sms, as_stream(stream)));
}

int dflash2_cache_evict(dflash2_handle* h, const float* scores, int64_t scores_ld, const dflash2_kv_cache* cache,
                        const int32_t* cache_len, const dflash2_kv_cache* dst, int64_t B, int64_t keep,
                        int64_t recent, int32_t* kept, int32_t* new_len, float* dst_scores, int64_t dst_ld,
                        void* stream) {
  const NvtxRange range("dflash2_cache_evict");
  if (bad_handle(h) || B < 0 || scores_ld < 0 || keep < 1 || recent < 0 || recent > keep ||
      (dst_scores && dst_ld < keep))
    return DFLASH2_ERR_INVALID_ARG;
  dflash2::EvictArgs a;
  if (const int st = view_cache(cache, B, &a.cache)) return st;
  if (const int st = view_cache(dst, B, &a.dst)) return st;
  if (cache->heads != dst->heads || cache->head_dim != dst->head_dim) return DFLASH2_ERR_INVALID_ARG;
  if (B > 65535 || B * cache->heads >= (int64_t(1) << 24) ||
      B * cache->heads * (keep / 16 + 1) >= (int64_t(1) << 31))
    return DFLASH2_ERR_UNSUPPORTED;
  if (B == 0) return DFLASH2_OK;
  if (keep > a.dst.capacity || !scores || !cache_len || !kept || !new_len || overlap(new_len, B, cache_len, B) ||
      overlap(dst_scores, B * cache->heads * dflash2::imin64(dst_ld, kMaxElements), scores,
              B * cache->heads * dflash2::imin64(scores_ld, kMaxElements)))
    return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(scores, 4) || !aligned(cache_len, 4) || !aligned(kept, 4) || !aligned(new_len, 4) ||
      !aligned(dst_scores, 4))
    return DFLASH2_ERR_MISALIGNED;
  if (const int st = wrong_device(h)) return st;
  a.scores = scores;
  a.scores_ld = scores_ld;
  a.cache_len = cache_len;
  a.B = B;
  a.keep = static_cast<int32_t>(keep);
  a.recent = static_cast<int32_t>(recent);
  a.kept = kept;
  a.new_len = new_len;
  a.dst_scores = dst_scores;
  a.dst_ld = dst_ld;
  a.err = h->err;
  return launched(dflash2::launch_cache_evict(a, cache->head_dim, h->num_sms, as_stream(stream)));
}

}  // extern "C"
