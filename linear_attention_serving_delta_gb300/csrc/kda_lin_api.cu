// kda_lin_api.cu -- the extern "C" entry points of the linear attention with a
// decay for each head: argument validation, workspace sizes and the choice of
// path.  Declarations and contracts are in include/kda.h.
#include <algorithm>

#include "kda_lin.cuh"

namespace kda {
namespace {

bool width_ok(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }
bool misaligned(const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) != 0; }
kda_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// What all four argument blocks have (a call without tokens may lack its gates)
template <typename A>
kda_status_t validate_heads(const A* a, int64_t tokens) {
  if (a->num_heads < 1 || a->num_key_heads < 1 || a->num_heads % a->num_key_heads != 0) return KDA_ERR_INVALID_ARG;
  if (a->in_dtype != KDA_F32 && a->in_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (a->num_states < 0 || (tokens > 0 && !a->g && !a->slope)) return KDA_ERR_INVALID_ARG;
  // heads are the y dimension of the kernels' grids
  return width_ok(a->dk) && width_ok(a->dv) && a->num_heads <= 65535 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}
// states are read and written 16 bytes at a time
kda_status_t validate_states(const void* in, const void* out, const int32_t* slots, int64_t n, int32_t num_states) {
  if (!in && !out) return KDA_OK;
  if (!slots && num_states < n) return KDA_ERR_INVALID_ARG;
  return misaligned(in, 16) || misaligned(out, 16) ? KDA_ERR_INVALID_ARG : KDA_OK;
}
// token indices are int32 coordinates in the kernels' copies and grids
bool tokens_ok(int64_t T) { return T < ((int64_t)1 << 30); }

kda_status_t validate(const kda_lin_prefill_args* a) {
  if (!a || a->num_seqs < 1 || a->total_tokens < 0 || !a->cu_seqlens) return KDA_ERR_INVALID_ARG;
  kda_status_t st = validate_heads(a, a->total_tokens);
  if (st != KDA_OK) return st;
  st = validate_states(a->initial_state, a->final_state, a->state_slots, a->num_seqs, a->num_states);
  if (st != KDA_OK) return st;
  if (a->total_tokens > 0 && (!a->q || !a->k || !a->v || !a->o)) return KDA_ERR_INVALID_ARG;
  return tokens_ok(a->total_tokens) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status_t validate(const kda_lin_decode_args* a) {
  if (!a || a->batch < 0) return KDA_ERR_INVALID_ARG;
  const kda_status_t st = validate_heads(a, a->batch);
  if (st != KDA_OK) return st;
  if (a->batch == 0) return KDA_OK;
  if (!a->q || !a->k || !a->v || !a->o || !a->state || !a->state_out) return KDA_ERR_INVALID_ARG;
  return validate_states(a->state, a->state_out, a->state_slots, a->batch, a->num_states);
}

template <typename A>
kda_status_t validate_tree(const A* a) {
  if (a->num_seqs < 1 || a->total_tokens < 0 || !a->cu_seqlens || a->max_seqlen < 0) return KDA_ERR_INVALID_ARG;
  const kda_status_t st = validate_heads(a, a->total_tokens);
  if (st != KDA_OK) return st;
  if (a->max_seqlen > KDA_LIN_MAX_DRAFT || !tokens_ok(a->total_tokens)) return KDA_ERR_UNSUPPORTED;
  if (!a->state || (a->total_tokens > 0 && (!a->k || !a->v))) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}
kda_status_t validate(const kda_lin_draft_args* a) {
  if (!a) return KDA_ERR_INVALID_ARG;
  const kda_status_t st = validate_tree(a);
  if (st != KDA_OK) return st;
  if (a->total_tokens > 0 && (!a->q || !a->o)) return KDA_ERR_INVALID_ARG;
  return validate_states(a->state, nullptr, a->state_slots, a->num_seqs, a->num_states);
}
kda_status_t validate(const kda_lin_commit_args* a) {
  if (!a) return KDA_ERR_INVALID_ARG;
  const kda_status_t st = validate_tree(a);
  if (st != KDA_OK) return st;
  if (!a->last || !a->state_out) return KDA_ERR_INVALID_ARG;
  return validate_states(a->state, a->state_out, a->state_slots, a->num_seqs, a->num_states);
}

template <typename A>
LinParams common(const A* a) {
  LinParams p{};
  p.H = a->num_heads;
  p.Hk = a->num_key_heads;
  p.R = p.H / p.Hk;
  p.dk = a->dk;
  p.dv = a->dv;
  p.k = a->k;
  p.v = a->v;
  p.g = a->g;
  p.slope = a->slope;
  p.num_states = a->num_states;
  p.slots = a->state_slots;
  p.status = a->status;
  p.dt = a->in_dtype;
  return p;
}
LinParams params(const kda_lin_prefill_args* a) {
  LinParams p = common(a);
  p.num_seqs = a->num_seqs;
  p.total_tokens = p.max_seqlen = a->total_tokens;
  p.cu_seqlens = a->cu_seqlens;
  p.q = a->q;
  p.scale = a->scale;
  p.state_in = a->initial_state;
  p.state_out = a->final_state;
  // without states of its own a call needs no rows for its slots
  if (!p.state_in && !p.state_out) p.num_states = INT32_MAX;
  p.o = a->o;
  return p;
}
LinParams params(const kda_lin_decode_args* a) {
  LinParams p = common(a);
  p.num_seqs = a->batch;
  p.total_tokens = a->batch;
  p.max_seqlen = 1;
  p.q = a->q;
  p.scale = a->scale;
  p.state_in = a->state;
  p.state_out = a->state_out;
  p.o = a->o;
  return p;
}
template <typename A>
LinParams tree_params(const A* a) {
  LinParams p = common(a);
  p.num_seqs = a->num_seqs;
  p.total_tokens = a->total_tokens;
  p.max_seqlen = a->max_seqlen > 0 ? a->max_seqlen : KDA_LIN_MAX_DRAFT;
  p.cu_seqlens = a->cu_seqlens;
  p.parents = a->parents;
  p.state_in = a->state;
  return p;
}

// Enough for either path: a call's pointers may be aligned otherwise than those that the
// size was asked with
size_t prefill_workspace(const LinParams& p) {
  return p.dt == KDA_BF16 ? std::max(lin_tc_workspace(p), lin_simt_workspace(p)) : lin_simt_workspace(p);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_lin_prefill_workspace_size(const kda_lin_prefill_args* a) {
  if (validate(a) != KDA_OK) return 0;
  return prefill_workspace(params(a));
}

kda_status_t kda_lin_prefill(const kda_lin_prefill_args* a, void* ws, size_t ws_bytes, void* stream) {
  const kda_status_t st = validate(a);
  if (st != KDA_OK) return st;
  const LinParams p = params(a);
  const bool tc = lin_tc_fits(p);
  if (!ws || ws_bytes < prefill_workspace(p) || misaligned(ws, 256)) return KDA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(tc ? launch_lin_tc(p, ws, s) : launch_lin_simt(p, ws, s));
}

kda_status_t kda_lin_decode(const kda_lin_decode_args* a, void* stream) {
  const kda_status_t st = validate(a);
  if (st != KDA_OK || a->batch == 0) return st;
  return from_cuda(launch_lin_decode(params(a), static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_lin_draft(const kda_lin_draft_args* a, void* stream) {
  const kda_status_t st = validate(a);
  if (st != KDA_OK || a->total_tokens == 0) return st;
  LinParams p = tree_params(a);
  p.q = a->q;
  p.scale = a->scale;
  p.o = a->o;
  return from_cuda(launch_lin_draft(p, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_lin_commit(const kda_lin_commit_args* a, void* stream) {
  const kda_status_t st = validate(a);
  if (st != KDA_OK) return st;
  LinParams p = tree_params(a);
  p.last = a->last;
  p.state_out = a->state_out;
  return from_cuda(launch_lin_commit(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
