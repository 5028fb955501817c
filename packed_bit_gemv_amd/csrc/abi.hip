// C ABI of libpackedbitgemv: argument validation (before any HIP call),
// error mapping and dispatch to the gfx950 launchers.
#include "packed_bit_gemv.h"
#include "pbg_internal.hpp"

namespace {

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool bad_nk(int64_t n, int64_t k) { return n < 1 || n > PBG_MAX_N || k < 1 || k > PBG_MAX_K; }

bool bad_m(int64_t m) { return m < 1 || m > PBG_MAX_M; }

bool bad_ffn(int64_t d_model, int64_t d_ff) {
  return d_model < 8 || d_model > PBG_FFN_MAX_MODEL || d_model % 8 != 0 || bad_nk(d_ff, d_model);
}

// Rows of the 8-bit path: m x k within the limits of one launch and of an exact int32 sum.
bool bad_rows(int64_t m, int64_t k) { return m < 1 || m > PBG_MAX_ROWS || k < 1 || k > PBG_I8_MAX_K; }

bool bad_outputs(int64_t m, int64_t n) { return n < 1 || n > PBG_MAX_N || m * n > PBG_MAX_OUTPUTS; }

// The paged cache and the requests of a step.
bool bad_pages(int64_t pages, int64_t page_size) {
  return page_size < 1 || page_size > PBG_MAX_PAGE || (page_size & (page_size - 1)) != 0 || pages < 1 ||
         pages > 0x7FFFFFFFLL || pages * page_size >= 1LL << 40;
}

bool bad_table(int64_t requests, int64_t table_width, int64_t page_size) {
  return requests < 1 || requests > PBG_MAX_REQUESTS || table_width < 1 || table_width > (1LL << 30) / page_size;
}

// Heads of a step's m rows; the elements of a key head's page stay below 2^31.
bool bad_heads(int64_t m, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  return m < 1 || m > PBG_MAX_ROWS || heads < 1 || heads > PBG_MAX_HEADS || kv_heads < 1 || heads % kv_heads != 0 ||
         head_dim < 8 || head_dim > PBG_MAX_HEAD_DIM || head_dim % 8 != 0 || m * (heads + 2 * kv_heads) > 1LL << 26;
}

// True when earlier work on this thread left a HIP error pending. Such an
// error is the caller's: it is left in place (not cleared) and the call
// enqueues nothing. hipErrorNotReady from a completion query is a status,
// not a failure, and is cleared so that the launch check below sees only
// this call's errors.
bool pending_error() {
  const hipError_t e = hipPeekAtLastError();
  if (e == hipSuccess) return false;
  if (e == hipErrorNotReady) {
    (void)hipGetLastError();
    return false;
  }
  return true;
}

int finish(hipError_t launch_status) {
  if (launch_status != hipSuccess) return PBG_ERR_HIP;
  return hipGetLastError() == hipSuccess ? PBG_OK : PBG_ERR_HIP;
}

}  // namespace

extern "C" {

int pbg_abi_version(void) { return PBG_ABI_VERSION; }

const char* pbg_strerror(int code) {
  switch (code) {
    case PBG_OK: return "ok";
    case PBG_ERR_NULL: return "a required pointer is NULL";
    case PBG_ERR_SHAPE: return "n, k or m out of range";
    case PBG_ERR_ALIGN: return "a pointer lacks its required alignment";
    case PBG_ERR_CODE: return "pack input held a value outside {-1, 0, +1}";
    case PBG_ERR_HIP: return "a HIP launch or copy failed";
    case PBG_ERR_VALUE: return "a scalar argument is out of range";
    case PBG_ERR_WORKSPACE: return "workspace smaller than the call needs";
    default: return "unknown error code";
  }
}

int64_t pbg_words_per_row(int64_t k) { return pbg::words_per_row(k); }

int pack_ternary(const int8_t* codes, int64_t n, int64_t k, uint32_t* packed, int32_t* row_sum, int64_t* stats,
                 int64_t* stats_host, hipStream_t stream) {
  if (!codes || !packed || !row_sum || !stats) return PBG_ERR_NULL;
  if (bad_nk(n, k)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(row_sum, 4) || misaligned(stats, 8)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  int rc = finish(pbg::launch_pack(codes, n, k, packed, row_sum, stats, stream));
  if (rc != PBG_OK || !stats_host) return rc;
  if (hipMemcpyAsync(stats_host, stats, 4 * sizeof(int64_t), hipMemcpyDeviceToHost, stream) != hipSuccess)
    return PBG_ERR_HIP;
  if (hipStreamSynchronize(stream) != hipSuccess) return PBG_ERR_HIP;
  return stats_host[3] > 0 ? PBG_ERR_CODE : PBG_OK;
}

int64_t pbg_words_per_row3(int64_t k) { return pbg::words_per_row3(k); }

int pack_ternary3(const int8_t* codes, int64_t n, int64_t k, uint32_t* packed, int32_t* row_sum, int64_t* stats,
                  int64_t* stats_host, hipStream_t stream) {
  if (!codes || !packed || !row_sum || !stats) return PBG_ERR_NULL;
  if (bad_nk(n, k)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(row_sum, 4) || misaligned(stats, 8)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  int rc = finish(pbg::launch_pack3(codes, n, k, packed, row_sum, stats, stream));
  if (rc != PBG_OK || !stats_host) return rc;
  if (hipMemcpyAsync(stats_host, stats, 6 * sizeof(int64_t), hipMemcpyDeviceToHost, stream) != hipSuccess)
    return PBG_ERR_HIP;
  if (hipStreamSynchronize(stream) != hipSuccess) return PBG_ERR_HIP;
  return stats_host[5] > 0 ? PBG_ERR_CODE : PBG_OK;
}

int ternary3_gemv(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const uint16_t* x, float* y,
                  hipStream_t stream) {
  if (!packed || !scale || !x || !y) return PBG_ERR_NULL;
  if (bad_nk(n, k)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(y, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ternary3_gemv(packed, scale, n, k, x, y, stream));
}

int ternary3_gemm_small(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const uint16_t* x,
                        int64_t m, float* y, hipStream_t stream) {
  if (!packed || !scale || !x || !y) return PBG_ERR_NULL;
  if (bad_nk(n, k) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(y, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ternary3_gemm_small(packed, scale, n, k, x, static_cast<int>(m), y, stream));
}

int ternary_gemv(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const uint16_t* x, float* y,
                 hipStream_t stream) {
  if (!packed || !scale || !x || !y) return PBG_ERR_NULL;
  if (bad_nk(n, k)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(y, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ternary_gemv(packed, scale, n, k, x, y, stream));
}

int ternary_gemm_small(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const uint16_t* x,
                       int64_t m, float* y, hipStream_t stream) {
  if (!packed || !scale || !x || !y) return PBG_ERR_NULL;
  if (bad_nk(n, k) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(y, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ternary_gemm_small(packed, scale, n, k, x, static_cast<int>(m), y, stream));
}

int64_t pbg_splitk_workspace_bytes(int64_t n, int64_t k) {
  if (bad_nk(n, k)) return 0;
  return pbg::splitk_workspace_bytes(n, k);
}

int ternary_gemm_splitk(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const uint16_t* x,
                        int64_t m, float* y, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!packed || !scale || !x || !y || !workspace) return PBG_ERR_NULL;
  if (bad_nk(n, k) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(y, 4) ||
      misaligned(workspace, 256))
    return PBG_ERR_ALIGN;
  if (workspace_bytes < pbg::splitk_workspace_bytes(n, k)) return PBG_ERR_WORKSPACE;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ternary_gemm_splitk(packed, scale, n, k, x, static_cast<int>(m), y, workspace,
                                                workspace_bytes, stream));
}

int int8_head_gemv(const int8_t* w, const float* scale, int64_t n, int64_t k, const uint16_t* x, int64_t m,
                   float* y, hipStream_t stream) {
  if (!w || !scale || !x || !y) return PBG_ERR_NULL;
  if (bad_nk(n, k) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(w, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(y, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_int8_head(w, scale, n, k, x, static_cast<int>(m), y, stream));
}

int int8_head_argmax(const int8_t* w, const float* scale, int64_t n, int64_t k, const uint16_t* x, int64_t m,
                     uint64_t* keys, int32_t* token, float* logit, hipStream_t stream) {
  if (!w || !scale || !x || !keys || !token) return PBG_ERR_NULL;
  if (bad_nk(n, k) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(w, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(keys, 8) || misaligned(token, 4) ||
      misaligned(logit, 4))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_int8_head_argmax(w, scale, n, k, x, static_cast<int>(m),
                                             reinterpret_cast<unsigned long long*>(keys), token, logit, stream));
}

int int8_head_argmax_noalloc(const int8_t* w, const float* scale, int64_t n, int64_t k, const uint16_t* x,
                             int64_t m, int32_t* token, float* logit, hipStream_t stream) {
  if (!w || !scale || !x || !token) return PBG_ERR_NULL;
  if (bad_nk(n, k) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(w, 16) || misaligned(scale, 4) || misaligned(x, 2) || misaligned(token, 4) || misaligned(logit, 4))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_int8_head_argmax_noalloc(w, scale, n, k, x, static_cast<int>(m), token, logit, stream));
}

int int8_embedding_gather(const int8_t* table, const float* scale, int64_t n, int64_t k, const int32_t* tokens,
                          int64_t m, float* out, hipStream_t stream) {
  if (!table || !scale || !tokens || !out) return PBG_ERR_NULL;
  if (bad_nk(n, k) || m < 1 || m > PBG_MAX_N || pbg::embedding_blocks(m, k) > (1LL << 23)) return PBG_ERR_SHAPE;
  if (misaligned(scale, 4) || misaligned(tokens, 4) || misaligned(out, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_embedding_gather(table, scale, n, k, tokens, m, out, stream));
}

int64_t pbg_q8_row_bytes(int64_t k) { return pbg::q8_row_bytes(k); }

int add_rmsnorm(const float* x, const float* residual, const float* weight, float eps, int64_t m, int64_t k,
                float* residual_out, uint16_t* h, int8_t* q, float* q_scale, hipStream_t stream) {
  if (!x || !weight || (!h && !q) || (q == nullptr) != (q_scale == nullptr)) return PBG_ERR_NULL;
  if (bad_rows(m, k)) return PBG_ERR_SHAPE;
  if (misaligned(x, 4) || misaligned(residual, 4) || misaligned(weight, 4) || misaligned(residual_out, 4) ||
      misaligned(h, 2) || misaligned(q, 16) || misaligned(q_scale, 4))
    return PBG_ERR_ALIGN;
  if (!(eps > 0.0f && eps < __builtin_inff())) return PBG_ERR_VALUE;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_add_rmsnorm(x, residual, weight, eps, m, k, residual_out, h, q, q_scale, stream));
}

int quantize_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* q, float* q_scale, hipStream_t stream) {
  if (!x || !q || !q_scale) return PBG_ERR_NULL;
  if (bad_rows(m, k)) return PBG_ERR_SHAPE;
  if (misaligned(x, 2) || misaligned(q, 16) || misaligned(q_scale, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_quantize_rows(x, m, k, q, q_scale, stream));
}

int ternary_gemm_i8(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const int8_t* q,
                    const float* q_scale, int64_t m, float* y, hipStream_t stream) {
  if (!packed || !scale || !q || !q_scale || !y) return PBG_ERR_NULL;
  if (bad_rows(m, k) || bad_outputs(m, n)) return PBG_ERR_SHAPE;
  if (misaligned(packed, 16) || misaligned(scale, 4) || misaligned(q, 16) || misaligned(q_scale, 4) ||
      misaligned(y, 4))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ternary_gemm_i8(packed, scale, n, k, q, q_scale, m, y, stream));
}

int ternary_swiglu_gate_up_i8(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                              const float* up_scale, int64_t d_model, int64_t d_ff, const int8_t* q,
                              const float* q_scale, int64_t m, uint16_t* h, hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !q || !q_scale || !h) return PBG_ERR_NULL;
  if (bad_rows(m, d_model) || bad_outputs(m, d_ff)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(gate_scale, 4) ||
      misaligned(up_scale, 4) || misaligned(q, 16) || misaligned(q_scale, 4) || misaligned(h, 2))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_swiglu_gate_up_i8(gate_packed, gate_scale, up_packed, up_scale, d_model, d_ff, q, q_scale,
                                              m, h, stream));
}

int64_t pbg_lora_workspace_bytes(int64_t m, int64_t rank) {
  if (m < 1 || m > PBG_MAX_ROWS || rank < 1 || rank > PBG_LORA_MAX_RANK) return 0;
  return pbg::lora_workspace_bytes(m, static_cast<int>(rank));
}

int lora_add(const float* y, const uint16_t* x, const int32_t* ids, const uint16_t* a, const uint16_t* b,
             const float* scale, int64_t m, int64_t n, int64_t k, int64_t adapters, int64_t rank, float* out,
             void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!y || !x || !ids || !a || !b || !scale || !out || !workspace) return PBG_ERR_NULL;
  if (bad_rows(m, k) || bad_outputs(m, n) || adapters < 1 || adapters > PBG_LORA_MAX_ADAPTERS || rank < 1 ||
      rank > PBG_LORA_MAX_RANK)
    return PBG_ERR_SHAPE;
  if (misaligned(y, 4) || misaligned(x, 2) || misaligned(ids, 4) || misaligned(a, 2) || misaligned(b, 2) ||
      misaligned(scale, 4) || misaligned(out, 4) || misaligned(workspace, 16))
    return PBG_ERR_ALIGN;
  if (workspace_bytes < pbg_lora_workspace_bytes(m, rank)) return PBG_ERR_WORKSPACE;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_lora_add(y, x, ids, a, b, scale, m, n, k, static_cast<int>(adapters),
                                     static_cast<int>(rank), out, workspace, stream));
}

int pbg_stream_read(const void* src, int64_t bytes, uint32_t* sink, hipStream_t stream) {
  if (!src || !sink) return PBG_ERR_NULL;
  if (bytes < 16 || bytes > PBG_STREAM_READ_MAX_BYTES || bytes % 16 != 0) return PBG_ERR_SHAPE;
  if (misaligned(src, 16) || misaligned(sink, 4)) return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_stream_read(src, bytes, sink, stream));
}

int ternary_swiglu_gate_up(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                           const float* up_scale, int64_t d_model, int64_t d_ff, const uint16_t* x, uint16_t* h,
                           hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !x || !h) return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(gate_scale, 4) ||
      misaligned(up_scale, 4) || misaligned(x, 16) || misaligned(h, 16))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_swiglu_gate_up(gate_packed, gate_scale, up_packed, up_scale, d_model, d_ff, x, h, stream));
}

int ternary_ffn_swiglu(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                       const float* up_scale, const uint32_t* down_packed, const float* down_scale, int64_t d_model,
                       int64_t d_ff, const uint16_t* x, uint16_t* h, float* y, hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !down_packed || !down_scale || !x || !h || !y)
    return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(down_packed, 16) ||
      misaligned(gate_scale, 4) || misaligned(up_scale, 4) || misaligned(down_scale, 4) || misaligned(x, 16) ||
      misaligned(h, 16) || misaligned(y, 4))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ffn_swiglu(gate_packed, gate_scale, up_packed, up_scale, down_packed, down_scale, d_model,
                                       d_ff, x, h, y, stream));
}

int ternary_swiglu_gate_up_small(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                                 const float* up_scale, int64_t d_model, int64_t d_ff, const uint16_t* x, int64_t m,
                                 uint16_t* h, hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !x || !h) return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(gate_scale, 4) ||
      misaligned(up_scale, 4) || misaligned(x, 16) || misaligned(h, 16))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_swiglu_gate_up_small(gate_packed, gate_scale, up_packed, up_scale, d_model, d_ff, x,
                                                 static_cast<int>(m), h, stream));
}

int ternary_ffn_swiglu_small(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                             const float* up_scale, const uint32_t* down_packed, const float* down_scale,
                             int64_t d_model, int64_t d_ff, const uint16_t* x, int64_t m, uint16_t* h, float* y,
                             hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !down_packed || !down_scale || !x || !h || !y)
    return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(down_packed, 16) ||
      misaligned(gate_scale, 4) || misaligned(up_scale, 4) || misaligned(down_scale, 4) || misaligned(x, 16) ||
      misaligned(h, 16) || misaligned(y, 4))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ffn_swiglu_small(gate_packed, gate_scale, up_packed, up_scale, down_packed, down_scale,
                                             d_model, d_ff, x, static_cast<int>(m), h, y, stream));
}

int ternary3_swiglu_gate_up(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                            const float* up_scale, int64_t d_model, int64_t d_ff, const uint16_t* x, uint16_t* h,
                            hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !x || !h) return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(gate_scale, 4) ||
      misaligned(up_scale, 4) || misaligned(x, 16) || misaligned(h, 16))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_swiglu3_gate_up(gate_packed, gate_scale, up_packed, up_scale, d_model, d_ff, x, h, stream));
}

int ternary3_ffn_swiglu(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                        const float* up_scale, const uint32_t* down_packed, const float* down_scale, int64_t d_model,
                        int64_t d_ff, const uint16_t* x, uint16_t* h, float* y, hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !down_packed || !down_scale || !x || !h || !y)
    return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(down_packed, 16) ||
      misaligned(gate_scale, 4) || misaligned(up_scale, 4) || misaligned(down_scale, 4) || misaligned(x, 16) ||
      misaligned(h, 16) || misaligned(y, 4))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ffn3_swiglu(gate_packed, gate_scale, up_packed, up_scale, down_packed, down_scale, d_model,
                                        d_ff, x, h, y, stream));
}

int ternary3_swiglu_gate_up_small(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                                  const float* up_scale, int64_t d_model, int64_t d_ff, const uint16_t* x, int64_t m,
                                  uint16_t* h, hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !x || !h) return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(gate_scale, 4) ||
      misaligned(up_scale, 4) || misaligned(x, 16) || misaligned(h, 16))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_swiglu3_gate_up_small(gate_packed, gate_scale, up_packed, up_scale, d_model, d_ff, x,
                                                  static_cast<int>(m), h, stream));
}

int ternary3_ffn_swiglu_small(const uint32_t* gate_packed, const float* gate_scale, const uint32_t* up_packed,
                              const float* up_scale, const uint32_t* down_packed, const float* down_scale,
                              int64_t d_model, int64_t d_ff, const uint16_t* x, int64_t m, uint16_t* h, float* y,
                              hipStream_t stream) {
  if (!gate_packed || !gate_scale || !up_packed || !up_scale || !down_packed || !down_scale || !x || !h || !y)
    return PBG_ERR_NULL;
  if (bad_ffn(d_model, d_ff) || bad_m(m)) return PBG_ERR_SHAPE;
  if (misaligned(gate_packed, 16) || misaligned(up_packed, 16) || misaligned(down_packed, 16) ||
      misaligned(gate_scale, 4) || misaligned(up_scale, 4) || misaligned(down_scale, 4) || misaligned(x, 16) ||
      misaligned(h, 16) || misaligned(y, 4))
    return PBG_ERR_ALIGN;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_ffn3_swiglu_small(gate_packed, gate_scale, up_packed, up_scale, down_packed, down_scale,
                                              d_model, d_ff, x, static_cast<int>(m), h, y, stream));
}

int cache_plan(const int32_t* lengths, const int32_t* added, int64_t requests, int32_t* table, int64_t table_width,
               const int32_t* free_pages, int64_t free_capacity, const int32_t* free_count, int64_t pages,
               int64_t page_size, const int32_t* parents, int64_t m, int32_t* row_start, int32_t* request,
               int32_t* position, int64_t* slot, uint64_t* ancestors, int32_t* free_left, hipStream_t stream) {
  if (!lengths || !added || !table || !free_pages || !free_count || !row_start || !request || !position || !slot ||
      !free_left)
    return PBG_ERR_NULL;
  if (m < 1 || m > PBG_MAX_ROWS || bad_pages(pages, page_size) || bad_table(requests, table_width, page_size) ||
      free_capacity < 1 || free_capacity > 0x7FFFFFFFLL)
    return PBG_ERR_SHAPE;
  if (misaligned(lengths, 4) || misaligned(added, 4) || misaligned(table, 4) || misaligned(free_pages, 4) ||
      misaligned(free_count, 4) || misaligned(parents, 4) || misaligned(row_start, 4) || misaligned(request, 4) ||
      misaligned(position, 4) || misaligned(slot, 8) || misaligned(ancestors, 8) || misaligned(free_left, 4))
    return PBG_ERR_ALIGN;
  if (free_left == free_count) return PBG_ERR_VALUE;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_cache_plan(lengths, added, requests, table, table_width, free_pages, free_capacity,
                                       free_count, pages, page_size, parents, m, row_start, request, position, slot,
                                       ancestors, free_left, stream));
}

int rotary_qkv(const float* qkv, const int32_t* position, const int64_t* slot, const double* inv_freq,
               const float* q_weight, const float* k_weight, float eps, float amplitude, int interleaved, int64_t m,
               int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t rotary_dim, uint16_t* q, uint16_t* k_cache,
               uint16_t* v_cache, int64_t pages, int64_t page_size, hipStream_t stream) {
  if (!qkv || !position || !slot || !q || !k_cache || !v_cache) return PBG_ERR_NULL;
  if (bad_heads(m, heads, kv_heads, head_dim) || rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 8 != 0 ||
      bad_pages(pages, page_size))
    return PBG_ERR_SHAPE;
  if ((inv_freq == nullptr) != (rotary_dim == 0)) return PBG_ERR_NULL;
  if (misaligned(qkv, 4) || misaligned(position, 4) || misaligned(slot, 8) || misaligned(inv_freq, 8) ||
      misaligned(q_weight, 4) || misaligned(k_weight, 4) || misaligned(q, 16) || misaligned(k_cache, 16) ||
      misaligned(v_cache, 16))
    return PBG_ERR_ALIGN;
  if (!(eps > 0.0f) || !(eps < __builtin_inff()) || !(amplitude > -__builtin_inff()) || !(amplitude < __builtin_inff()))
    return PBG_ERR_VALUE;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_rotary_qkv(qkv, position, slot, inv_freq, q_weight, k_weight, eps, amplitude,
                                       interleaved != 0, m, static_cast<int>(heads), static_cast<int>(kv_heads),
                                       static_cast<int>(head_dim), static_cast<int>(rotary_dim), q, k_cache, v_cache,
                                       pages, page_size, stream));
}

int64_t pbg_attention_workspace_bytes(int64_t heads, int64_t kv_heads, int64_t head_dim) {
  return bad_heads(1, heads, kv_heads, head_dim) ? 0 : pbg::attention_workspace_bytes(static_cast<int>(head_dim));
}

int tree_attention(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache, int64_t pages,
                   int64_t page_size, const int32_t* table, int64_t table_width, const int32_t* lengths,
                   const int32_t* row_start, int64_t requests, const uint64_t* ancestors, int64_t m, int64_t heads,
                   int64_t kv_heads, int64_t head_dim, float scale, uint16_t* out, void* workspace,
                   int64_t workspace_bytes, hipStream_t stream) {
  if (!q || !k_cache || !v_cache || !table || !lengths || !row_start || !out || !workspace) return PBG_ERR_NULL;
  if (bad_heads(m, heads, kv_heads, head_dim) || bad_pages(pages, page_size) || page_size < PBG_ATTENTION_MIN_PAGE ||
      bad_table(requests, table_width, page_size))
    return PBG_ERR_SHAPE;
  if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(table, 4) ||
      misaligned(lengths, 4) || misaligned(row_start, 4) || misaligned(ancestors, 8) || misaligned(out, 16) ||
      misaligned(workspace, 16))
    return PBG_ERR_ALIGN;
  // the kernels multiply by scale * log2(e)
  if (!(scale > 0.0f) || !(scale < 0x1p127f)) return PBG_ERR_VALUE;
  if (workspace_bytes < pbg::attention_workspace_bytes(static_cast<int>(head_dim))) return PBG_ERR_WORKSPACE;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_tree_attention(q, k_cache, v_cache, pages, page_size, table, table_width, lengths,
                                           row_start, requests, ancestors, m, static_cast<int>(heads),
                                           static_cast<int>(kv_heads), static_cast<int>(head_dim), scale, out,
                                           workspace, stream));
}

int penalize_logits(const float* logits, const int32_t* request, const int32_t* tokens, int64_t tokens_width,
                    const int32_t* prompt_length, const int32_t* length, const float* repetition,
                    const float* frequency, const float* presence, int64_t requests, const int32_t* drafts,
                    const int32_t* row_start, const uint64_t* ancestors, const int32_t* bias_start,
                    const int32_t* bias_token, const float* bias_value, int64_t bias_entries, const uint32_t* grammar,
                    const int32_t* grammar_row, int64_t states, int64_t m, int64_t n, float* out, int32_t* token,
                    float* top, uint64_t* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!logits || !request || !tokens || !prompt_length || !length || !repetition || !frequency || !presence || !out)
    return PBG_ERR_NULL;
  const bool has_drafts = drafts != nullptr, has_bias = bias_start != nullptr, has_grammar = grammar != nullptr;
  if ((row_start != nullptr) != has_drafts || (ancestors != nullptr) != has_drafts ||
      (bias_token != nullptr) != has_bias || (bias_value != nullptr) != has_bias ||
      (grammar_row != nullptr) != has_grammar || (token != nullptr) != (top != nullptr) || (token && !workspace))
    return PBG_ERR_NULL;
  if (m < 1 || m > PBG_MAX_ROWS || n < 1 || n > PBG_MAX_N || m * n > PBG_MAX_LOGITS || requests < 1 ||
      requests > PBG_MAX_REQUESTS || tokens_width < 1 || tokens_width > 1LL << 24 ||
      (has_bias && (bias_entries < 1 || bias_entries > 0x7FFFFFFFLL)) ||
      (has_grammar && (states < 1 || states > 0x7FFFFFFFLL)))
    return PBG_ERR_SHAPE;
  if (misaligned(logits, 4) || misaligned(request, 4) || misaligned(tokens, 4) || misaligned(prompt_length, 4) ||
      misaligned(length, 4) || misaligned(repetition, 4) || misaligned(frequency, 4) || misaligned(presence, 4) ||
      misaligned(drafts, 4) || misaligned(row_start, 4) || misaligned(ancestors, 8) || misaligned(bias_start, 4) ||
      misaligned(bias_token, 4) || misaligned(bias_value, 4) || misaligned(grammar, 4) || misaligned(grammar_row, 4) ||
      misaligned(out, 4) || misaligned(token, 4) || misaligned(top, 4) || misaligned(workspace, 8))
    return PBG_ERR_ALIGN;
  if (token && workspace_bytes < 8 * m * ((n + PBG_LOGITS_SLICE - 1) / PBG_LOGITS_SLICE)) return PBG_ERR_WORKSPACE;
  if (pending_error()) return PBG_ERR_HIP;
  return finish(pbg::launch_penalize_logits(logits, request, tokens, tokens_width, prompt_length, length, repetition,
                                            frequency, presence, requests, drafts, row_start, ancestors, bias_start,
                                            bias_token, bias_value, bias_entries, grammar, grammar_row, states, m, n,
                                            out, token, top, workspace, stream));
}

}  // extern "C"
