// kda_attn.cuh -- what the full-attention kernels and the paged cache's
// kernels share: parameter blocks, the checks of device-side lengths and
// rows, and the launchers.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// Status flags of the attention and cache calls beside those of kda_common.cuh
enum : int32_t {
  kFlagBadCache = 32,     // a malformed row, length, page or slot
  kFlagNoPages = 64,      // the free list ran out
  kFlagLongSequence = 128 // a sequence longer than max_seqlen
};

__device__ __forceinline__ void attn_flag(int32_t* status, int32_t f) {
  if (status) atomicOr(status, f);
}

// Both attention calls.  block_table null: k, v are packed as q is (whole
// prompts); otherwise they are the caches.
struct AttnParams {
  int32_t num_seqs, H, Hkv, G, D;  // G = H / Hkv
  int64_t total_tokens;
  int64_t max_seqlen;
  const int64_t* cu_seqlens;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float scale;
  int32_t num_pages, page_shift, max_pages, num_rows;
  const int32_t* block_table;
  const int64_t* kv_lens;
  const int32_t* rows;
  int32_t* status;
  kda_dtype_t dt;
};

// One sequence of a call: its new tokens [tok0, tok0 + len) and the kv_len
// positions they attend (new ones included); token i stands at position
// kv_len - len + i.  len = 0: nothing to do (empty, skipped or malformed).
struct AttnSeq {
  int64_t tok0;
  int64_t kv_len;
  int32_t len;
  int32_t row;
  int32_t flag;  // what was malformed, or 0
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int32_t s) {
  AttnSeq r;
  r.tok0 = p.cu_seqlens[s];
  const int64_t end = p.cu_seqlens[s + 1];
  r.len = 0;
  r.row = s;
  r.kv_len = end - r.tok0;
  r.flag = 0;
  if (r.tok0 < 0 || end < r.tok0 || end > p.total_tokens || (s == 0 && r.tok0 != 0)) {
    r.flag = kFlagBadSeqlens;
    return r;
  }
  const int64_t len = end - r.tok0;
  if (len > p.max_seqlen) {
    r.flag = kFlagLongSequence;
    return r;
  }
  if (p.block_table) {
    r.row = p.rows ? p.rows[s] : s;
    if (r.row < 0) return r;
    if (r.row >= p.num_rows) {
      r.flag = kFlagBadCache;
      return r;
    }
    r.kv_len = p.kv_lens[r.row];
    if (r.kv_len < 0 || r.kv_len > ((int64_t)p.max_pages << p.page_shift)) {
      r.flag = kFlagBadCache;
      return r;
    }
  }
  r.len = (int32_t)len;
  return r;
}

// The plain CUDA-core kernel: every dtype, head size and alignment
cudaError_t launch_attn_simt(const AttnParams& p, cudaStream_t stream);

cudaError_t launch_kv_plan(const kda_kv_plan_args& a, void* ws, cudaStream_t stream);
cudaError_t launch_kv_release(const kda_kv_release_args& a, void* ws, cudaStream_t stream);
cudaError_t launch_kv_write(const kda_kv_write_args& a, cudaStream_t stream);
size_t kv_plan_workspace(int64_t num_seqs, int64_t num_rows);

}  // namespace kda
