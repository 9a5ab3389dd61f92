// kda_attn_api.cu -- the extern "C" entry points of the full attention and its
// paged cache: argument validation, workspace sizes and the choice of path.
// Declarations and contracts are in include/kda.h.
#include "kda_attn_tc.cuh"

namespace kda {
namespace {

bool head_dim_ok(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }
bool dtype_ok(kda_dtype_t t) { return t == KDA_F32 || t == KDA_BF16; }
bool page_ok(int32_t p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }
bool misaligned(const void* ws) { return (reinterpret_cast<uintptr_t>(ws) & 255) != 0; }
kda_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

int shift_of(int32_t page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

kda_status_t validate_heads(int32_t H, int32_t Hkv, int32_t D, kda_dtype_t dt) {
  if (H < 1 || Hkv < 1 || H % Hkv != 0) return KDA_ERR_INVALID_ARG;
  if (!dtype_ok(dt)) return KDA_ERR_INVALID_ARG;
  // key heads are the y dimension of the kernels' grids
  if (!head_dim_ok(D) || H / Hkv > KDA_ATTN_MAX_GROUP || Hkv > 65535) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// token indices are int32 coordinates in the kernels' copies and grids
bool tokens_ok(int64_t T) { return T < ((int64_t)1 << 30); }
// so are the positions of a row
bool positions_ok(int32_t max_pages, int32_t page_size) {
  return (int64_t)max_pages * page_size < ((int64_t)1 << 31) - 1024;
}

kda_status_t validate(const kda_attn_prefill_args* a) {
  if (!a || a->num_seqs < 1 || a->total_tokens < 0 || !a->cu_seqlens) return KDA_ERR_INVALID_ARG;
  const kda_status_t st = validate_heads(a->num_heads, a->num_kv_heads, a->head_dim, a->in_dtype);
  if (st != KDA_OK) return st;
  if (a->total_tokens > 0 && (!a->q || !a->k || !a->v || !a->o)) return KDA_ERR_INVALID_ARG;
  return tokens_ok(a->total_tokens) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status_t validate(const kda_attn_paged_args* a) {
  if (!a || a->num_seqs < 1 || a->total_tokens < 0 || !a->cu_seqlens) return KDA_ERR_INVALID_ARG;
  const kda_status_t st = validate_heads(a->num_heads, a->num_kv_heads, a->head_dim, a->in_dtype);
  if (st != KDA_OK) return st;
  if (a->num_pages < 0 || a->num_rows < 0 || a->max_pages < 0 || a->max_seqlen < 0) return KDA_ERR_INVALID_ARG;
  if (!page_ok(a->page_size)) return KDA_ERR_UNSUPPORTED;
  if (!a->rows && a->num_rows < a->num_seqs) return KDA_ERR_INVALID_ARG;
  if (a->total_tokens > 0 && (!a->q || !a->o || !a->kv_lens || !a->block_table || !a->k_cache || !a->v_cache))
    return KDA_ERR_INVALID_ARG;
  if (!positions_ok(a->max_pages, a->page_size)) return KDA_ERR_UNSUPPORTED;
  return tokens_ok(a->total_tokens) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

AttnParams params(const kda_attn_prefill_args* a) {
  AttnParams p{};
  p.num_seqs = a->num_seqs;
  p.H = a->num_heads;
  p.Hkv = a->num_kv_heads;
  p.G = p.H / p.Hkv;
  p.D = a->head_dim;
  p.total_tokens = a->total_tokens;
  p.max_seqlen = a->total_tokens;
  p.cu_seqlens = a->cu_seqlens;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.o = a->o;
  p.scale = a->scale;
  p.status = a->status;
  p.dt = a->in_dtype;
  return p;
}

AttnParams params(const kda_attn_paged_args* a) {
  AttnParams p{};
  p.num_seqs = a->num_seqs;
  p.H = a->num_heads;
  p.Hkv = a->num_kv_heads;
  p.G = p.H / p.Hkv;
  p.D = a->head_dim;
  p.total_tokens = a->total_tokens;
  p.max_seqlen = a->max_seqlen > 0 && a->max_seqlen < a->total_tokens ? a->max_seqlen : a->total_tokens;
  p.cu_seqlens = a->cu_seqlens;
  p.q = a->q;
  p.k = a->k_cache;
  p.v = a->v_cache;
  p.o = a->o;
  p.scale = a->scale;
  p.num_pages = a->num_pages;
  p.page_shift = shift_of(a->page_size);
  p.max_pages = a->max_pages;
  p.num_rows = a->num_rows;
  p.block_table = a->block_table;
  p.kv_lens = a->kv_lens;
  p.rows = a->rows;
  p.status = a->status;
  p.dt = a->in_dtype;
  return p;
}

// The path of a call: few rows a request (few_rows) on the streaming kernel,
// more on the tensor cores' row tiles (two a CTA; one for heads of 256 channels
// and fp32), fp32 heads of 256 channels on the streaming kernel again, and what
// none of them takes (odd alignment, a scale that is not positive) on the CUDA
// cores.
enum class AttnPath { kRows, kTc, kTc1, kSimt };
AttnPath attn_path(const AttnParams& p) {
  if (few_rows(p) && attn_rows_fits(p)) return AttnPath::kRows;
  if (attn_tc_fits(p)) return AttnPath::kTc;
  if (attn_tc1_fits(p)) return AttnPath::kTc1;
  return attn_rows_fits(p) ? AttnPath::kRows : AttnPath::kSimt;
}
size_t attn_workspace(const AttnParams& p) {
  switch (attn_path(p)) {
    case AttnPath::kRows: return attn_rows_workspace(p);
    case AttnPath::kTc: return attn_tc_workspace(p);
    case AttnPath::kTc1: return attn_tc1_workspace(p);
    case AttnPath::kSimt: break;
  }
  return 256;
}

kda_status_t run_attn(const AttnParams& p, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || ws_bytes < attn_workspace(p) || misaligned(ws)) return KDA_ERR_WORKSPACE;
  if (p.total_tokens == 0) return KDA_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (attn_path(p)) {
    case AttnPath::kRows: return from_cuda(launch_attn_rows(p, ws, s));
    case AttnPath::kTc: return from_cuda(launch_attn_tc(p, ws, s));
    case AttnPath::kTc1: return from_cuda(launch_attn_tc1(p, ws, s));
    case AttnPath::kSimt: break;
  }
  return from_cuda(launch_attn_simt(p, s));
}

kda_status_t validate(const kda_kv_plan_args* a) {
  if (!a || a->num_seqs < 1 || a->total_tokens < 0 || !a->cu_seqlens) return KDA_ERR_INVALID_ARG;
  if (a->num_pages < 0 || a->num_rows < 0 || a->max_pages < 0) return KDA_ERR_INVALID_ARG;
  if (!page_ok(a->page_size) || !tokens_ok(a->total_tokens) || !positions_ok(a->max_pages, a->page_size))
    return KDA_ERR_UNSUPPORTED;
  if (!a->rows && a->num_rows < a->num_seqs) return KDA_ERR_INVALID_ARG;
  if (!a->free_count_in || !a->free_count_out) return KDA_ERR_INVALID_ARG;
  if (a->num_rows > 0 && (!a->kv_lens_in || !a->kv_lens_out)) return KDA_ERR_INVALID_ARG;
  if (a->num_rows > 0 && a->max_pages > 0 && !a->block_table) return KDA_ERR_INVALID_ARG;
  if (a->num_pages > 0 && !a->free_pages) return KDA_ERR_INVALID_ARG;
  if (a->total_tokens > 0 && !a->slot_map) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status_t validate(const kda_kv_release_args* a) {
  if (!a || a->num_release < 0) return KDA_ERR_INVALID_ARG;
  if (a->num_pages < 0 || a->num_rows < 0 || a->max_pages < 0) return KDA_ERR_INVALID_ARG;
  if (!page_ok(a->page_size) || !positions_ok(a->max_pages, a->page_size)) return KDA_ERR_UNSUPPORTED;
  if (a->num_release > 0 && (!a->rows || !a->free_count)) return KDA_ERR_INVALID_ARG;
  if (a->num_rows > 0 && !a->kv_lens) return KDA_ERR_INVALID_ARG;
  if (a->num_rows > 0 && a->max_pages > 0 && !a->block_table) return KDA_ERR_INVALID_ARG;
  if (a->num_pages > 0 && !a->free_pages) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_attn_prefill_workspace_size(const kda_attn_prefill_args* a) {
  return validate(a) == KDA_OK ? attn_workspace(params(a)) : 0;
}

kda_status_t kda_attn_prefill(const kda_attn_prefill_args* a, void* ws, size_t ws_bytes, void* stream) {
  const kda_status_t st = validate(a);
  return st != KDA_OK ? st : run_attn(params(a), ws, ws_bytes, stream);
}

size_t kda_attn_paged_workspace_size(const kda_attn_paged_args* a) {
  return validate(a) == KDA_OK ? attn_workspace(params(a)) : 0;
}

kda_status_t kda_attn_paged(const kda_attn_paged_args* a, void* ws, size_t ws_bytes, void* stream) {
  const kda_status_t st = validate(a);
  return st != KDA_OK ? st : run_attn(params(a), ws, ws_bytes, stream);
}

size_t kda_kv_plan_workspace_size(const kda_kv_plan_args* a) {
  return validate(a) == KDA_OK ? kv_plan_workspace(a->num_seqs, a->num_rows) : 0;
}

kda_status_t kda_kv_plan(const kda_kv_plan_args* a, void* ws, size_t ws_bytes, void* stream) {
  const kda_status_t st = validate(a);
  if (st != KDA_OK) return st;
  if (!ws || ws_bytes < kv_plan_workspace(a->num_seqs, a->num_rows) || misaligned(ws)) return KDA_ERR_WORKSPACE;
  return from_cuda(launch_kv_plan(*a, ws, static_cast<cudaStream_t>(stream)));
}

size_t kda_kv_release_workspace_size(const kda_kv_release_args* a) {
  return validate(a) == KDA_OK ? kv_plan_workspace(0, a->num_rows) : 0;
}

kda_status_t kda_kv_release(const kda_kv_release_args* a, void* ws, size_t ws_bytes, void* stream) {
  const kda_status_t st = validate(a);
  if (st != KDA_OK) return st;
  if (!ws || ws_bytes < kv_plan_workspace(0, a->num_rows) || misaligned(ws)) return KDA_ERR_WORKSPACE;
  return from_cuda(launch_kv_release(*a, ws, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_kv_write(const kda_kv_write_args* a, void* stream) {
  if (!a || a->total_tokens < 0 || a->num_kv_heads < 1 || a->num_slots < 0) return KDA_ERR_INVALID_ARG;
  if (!dtype_ok(a->in_dtype)) return KDA_ERR_INVALID_ARG;
  if (!head_dim_ok(a->head_dim)) return KDA_ERR_UNSUPPORTED;
  if (a->total_tokens == 0) return KDA_OK;
  if (!a->k || !a->v || !a->slot_map) return KDA_ERR_INVALID_ARG;
  if (a->num_slots > 0 && (!a->k_cache || !a->v_cache)) return KDA_ERR_INVALID_ARG;
  return from_cuda(launch_kv_write(*a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
