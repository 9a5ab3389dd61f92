// kda_lin.cuh -- what the kernels of the linear attention with a decay for each
// head share: parameter block, the checks of device-side offsets and slots, and
// the decay logarithms.
#pragma once

#include "kda_attn.cuh"

namespace kda {

// All four calls; the fields that a call lacks are null or zero.
struct LinParams {
  int32_t num_seqs, H, Hk, R;  // R = H / Hk
  int32_t dk, dv;
  int64_t total_tokens;
  int64_t max_seqlen;          // draft and commit; otherwise total_tokens
  const int64_t* cu_seqlens;   // null: sequence s is token s (decode)
  const void* q;
  const void* k;
  const void* v;
  const void* g;               // null: softplus(g) counts as 1
  const float* slope;          // null: 1
  float scale;
  const float* state_in;       // null: zeros
  float* state_out;            // null: not kept
  int32_t num_states;
  const int32_t* slots;
  const int32_t* parents;
  const int32_t* last;
  void* o;
  int32_t* status;
  kda_dtype_t dt;
};

// A sequence of a call: tokens [tok0, tok0 + len), its row of the states.
// ok false: malformed (flag says how) or skipped.
struct LinSeq {
  int64_t tok0;
  int64_t len;
  int32_t slot;
  int32_t flag;
  bool ok;
};

__device__ __forceinline__ LinSeq lin_seq(const LinParams& p, int32_t s) {
  LinSeq r;
  r.flag = 0;
  r.ok = false;
  r.slot = p.slots ? p.slots[s] : s;  // (beside the offsets: one wait for all three)
  if (p.cu_seqlens) {
    r.tok0 = p.cu_seqlens[s];
    const int64_t end = p.cu_seqlens[s + 1];
    if (r.tok0 < 0 || end < r.tok0 || end > p.total_tokens || (s == 0 && r.tok0 != 0)) {
      r.flag = kFlagBadSeqlens;
      return r;
    }
    r.len = end - r.tok0;
    if (r.len > p.max_seqlen) {
      r.flag = kFlagLongSequence;
      return r;
    }
  } else {
    r.tok0 = s;
    r.len = 1;
  }
  if (p.slots) {
    if (r.slot < 0) return r;
    if (r.slot >= p.num_states) {
      r.flag = kFlagBadCache;
      return r;
    }
  }
  r.ok = true;
  return r;
}

// SMs of a GB300, which grids are sized by.  On a part with fewer of them results are the
// same, in more waves.
constexpr int kLinSms = 152;

constexpr float kLinLog2e = 1.4426950408889634f;
// An alpha below 2^-kLinMaxDecay counts as 0 (so the sums of logarithms stay finite)
constexpr float kLinMaxDecay = 1024.f;

// The gate of token t, head h, and log2 alpha of it
template <typename T>
__device__ __forceinline__ float lin_gate(const LinParams& p, int64_t t, int h) {
  return p.g ? ld_in(static_cast<const T*>(p.g), t * p.H + h) : 0.f;
}
__device__ __forceinline__ float lin_log2_alpha(const LinParams& p, float gate, int h) {
  float x = p.g ? log_alpha_of(gate) : -1.f;
  if (p.slope) x *= p.slope[h];
  x *= kLinLog2e;
  return x < -kLinMaxDecay ? -kLinMaxDecay : x;  // (a NaN stays)
}
template <typename T>
__device__ __forceinline__ float lin_log2_alpha(const LinParams& p, int64_t t, int h) {
  return lin_log2_alpha(p, lin_gate<T>(p, t, h), h);
}

// A sum of logarithms kept as a whole number and a fraction of at most a half,
// each fp32: differences of far sums keep the precision of their fractions
// (2^-25), which one fp32 sum of a few hundred would lose to cancellation.
struct LogSum {
  float i, f;
};
__device__ __forceinline__ LogSum log_sum(float x) {
  const float r = rintf(x);
  return LogSum{r, x - r};
}
__device__ __forceinline__ LogSum operator+(LogSum a, LogSum b) {
  const float f = a.f + b.f, r = rintf(f);
  return LogSum{a.i + b.i + r, f - r};
}
// a - b as one number
__device__ __forceinline__ float log_diff(LogSum a, LogSum b) { return (a.i - b.i) + (a.f - b.f); }

// A factor alpha = 2^x as it is applied to a state: from a half up as 1 + m, so
// that a decay close to 1 keeps its distance from it (a constant one rounded to
// fp32, off by up to 2^-25 every token, would drift by that times the tokens remembered).
struct LinDecay {
  float m;
  bool near_one;
};
__device__ __forceinline__ LinDecay lin_decay(float x) {
  LinDecay d;
  d.near_one = x > -1.f;
  d.m = d.near_one ? expm1f(x * 0.6931471805599453f) : exp2f(x);
  return d;
}

bool lin_tc_fits(const LinParams& p);
size_t lin_tc_workspace(const LinParams& p);
cudaError_t launch_lin_tc(const LinParams& p, void* ws, cudaStream_t stream);

// Prompts token by token on the CUDA cores: every type, size and alignment
size_t lin_simt_workspace(const LinParams& p);
cudaError_t launch_lin_simt(const LinParams& p, void* ws, cudaStream_t stream);

cudaError_t launch_lin_decode(const LinParams& p, cudaStream_t stream);
cudaError_t launch_lin_draft(const LinParams& p, cudaStream_t stream);
cudaError_t launch_lin_commit(const LinParams& p, cudaStream_t stream);

}  // namespace kda
