// kda_lin_state.cu -- the states of the linear attention with a decay for each
// head: one token a row (decode), the states advanced along accepted tokens
// (commit), drafted tokens over the states as they are (draft).  Formulas in
// include/kda.h.
//
// Decode and commit read every state once and write it once and do little
// else, so they are bound by HBM: a CTA takes one (row, head) -- or a slice
// of 16,384 elements of a wide one -- with 16-byte loads straight into
// registers, all issued before anything waits, and writes them back from there.
#include "kda_lin.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDraft = KDA_LIN_MAX_DRAFT;

// A CTA's slice of a state: DK x DVS elements, a float4 of VPT for each thread
template <int DK, int DV>
struct Tile {
  static constexpr int DVS = DK * DV > 16384 ? 16384 / DK : DV;  // columns
  static constexpr int QPR = DVS / 4;                            // float4 of a row
  static constexpr int NT = DK * QPR < kThreads ? DK * QPR : kThreads;
  static constexpr int NRG = NT / QPR;                           // rows that the threads cover at once
  static constexpr int VPT = DK / NRG;
  static_assert(NT % QPR == 0 && DK % NRG == 0, "threads tile the slice");
};

__device__ __forceinline__ float4 fma4(float a, float4 x, float4 y) {
  return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
}
__device__ __forceinline__ float4 mul4(float a, float4 x) { return make_float4(a * x.x, a * x.y, a * x.z, a * x.w); }
template <int N>
__device__ __forceinline__ void decay_all(LinDecay a, float4 (&s)[N]) {
  if (a.near_one) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = fma4(a.m, s[i], s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = mul4(a.m, s[i]);
  }
}

// ------------------------------------------------------------------ decode
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(Tile<DK, DV>::NT) lin_decode(const LinParams p) {
  using L = Tile<DK, DV>;
  __shared__ float sq[DK], sk[DK];
  __shared__ __align__(16) float sv[L::DVS];
  __shared__ __align__(16) float part[L::NRG][L::DVS];
  const int tid = threadIdx.x, row = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * L::DVS;
  const LinSeq seq = lin_seq(p, row);
  if (seq.flag && tid == 0 && h == 0 && c0 == 0) attn_flag(p.status, seq.flag);
  if (!seq.ok) return;
  const int cq = tid % L::QPR, rg = tid / L::QPR;
  const int64_t at = ((int64_t)seq.slot * p.H + h) * DK * DV + c0 + 4 * cq;
  float4 s[L::VPT];
#pragma unroll
  for (int i = 0; i < L::VPT; ++i) s[i] = *reinterpret_cast<const float4*>(p.state_in + at + (int64_t)(rg + i * L::NRG) * DV);
  const int64_t tk = ((int64_t)row * p.Hk + h / p.R) * DK, tv = ((int64_t)row * p.H + h) * DV + c0;
  for (int i = tid; i < DK; i += L::NT) {
    sq[i] = ld_in(static_cast<const T*>(p.q), tk + i);
    sk[i] = ld_in(static_cast<const T*>(p.k), tk + i);
  }
  for (int i = tid; i < L::DVS; i += L::NT) sv[i] = ld_in(static_cast<const T*>(p.v), tv + i);
  const LinDecay a = lin_decay(lin_log2_alpha<T>(p, row, h));
  __syncthreads();
  decay_all(a, s);
  const float4 v4 = *reinterpret_cast<const float4*>(sv + 4 * cq);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < L::VPT; ++i) {
    const int r = rg + i * L::NRG;
    s[i] = fma4(sk[r], v4, s[i]);
    y = fma4(sq[r], s[i], y);
    *reinterpret_cast<float4*>(p.state_out + at + (int64_t)r * DV) = s[i];
  }
  *reinterpret_cast<float4*>(&part[rg][4 * cq]) = y;
  __syncthreads();
  for (int c = tid; c < L::DVS; c += L::NT) {
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < L::NRG; ++r) x += part[r][c];
    st_out(static_cast<T*>(p.o), tv + c, x * p.scale);
  }
}

// ------------------------------------------------------------------ trees
// The parents of a request's tokens in shared memory; false (for the whole
// CTA) if one is malformed.
__device__ __forceinline__ bool load_parents(const LinParams& p, const LinSeq& seq, int8_t* par) {
  bool good = true;
  for (int i = threadIdx.x; i < (int)seq.len; i += blockDim.x) {
    const int x = p.parents ? p.parents[seq.tok0 + i] : i - 1;
    good = good && x >= -1 && x < i;
    par[i] = (int8_t)x;
  }
  return __syncthreads_and(good) != 0;
}

// Commit.  Token j of the path contributes 2^{G_a - G_j} k_j v_j^T, G_a - G_j
// being the sum of log2 alpha over what follows j on the path: taken from the
// accepted token upwards, so that no difference of far sums appears.
constexpr int kBatch = 16;  // tokens of the path in shared memory at a time

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(Tile<DK, DV>::NT) lin_commit(const LinParams p) {
  using L = Tile<DK, DV>;
  constexpr int kB = DK == 256 ? kBatch / 2 : kBatch;
  __shared__ float sk[kB][DK];
  __shared__ __align__(16) float sv[kB][L::DVS];
  __shared__ float la[kMaxDraft], w[kMaxDraft];
  __shared__ int8_t par[kMaxDraft], path[kMaxDraft];
  __shared__ int32_t n_path;
  __shared__ LinDecay decay;
  const int tid = threadIdx.x, h = blockIdx.y, c0 = blockIdx.z * L::DVS;
  const LinSeq seq = lin_seq(p, blockIdx.x);
  const bool first = tid == 0 && h == 0 && c0 == 0;
  if (seq.flag && first) attn_flag(p.status, seq.flag);
  if (!seq.ok) return;
  const int a = p.last[blockIdx.x];
  const bool good = load_parents(p, seq, par) && a >= -1 && a < seq.len;
  if (!good) {
    if (first) attn_flag(p.status, kFlagBadCache);
    return;
  }
  if (a < 0 && p.state_in == p.state_out) return;
  const int cq = tid % L::QPR, rg = tid / L::QPR;
  const int64_t at = ((int64_t)seq.slot * p.H + h) * DK * DV + c0 + 4 * cq;
  float4 s[L::VPT];
#pragma unroll
  for (int i = 0; i < L::VPT; ++i) s[i] = *reinterpret_cast<const float4*>(p.state_in + at + (int64_t)(rg + i * L::NRG) * DV);
  for (int i = tid; i <= a; i += L::NT) la[i] = lin_log2_alpha<T>(p, seq.tok0 + i, h);
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    float sum = 0.f;
    for (int j = a; j >= 0; j = par[j]) {
      path[n] = (int8_t)j;
      w[n++] = exp2f(sum);
      sum += la[j];
    }
    n_path = n;
    decay = lin_decay(sum);
  }
  __syncthreads();
  const int n = n_path;
  if (n > 0) decay_all(decay, s);
  for (int b = n - 1; b >= 0; b -= kB) {  // from the root on
    const int m = min(kB, b + 1);
    for (int i = tid; i < m * DK; i += L::NT) {
      const int j = i / DK, d = i % DK;
      sk[j][d] = w[b - j] * ld_in(static_cast<const T*>(p.k), ((seq.tok0 + path[b - j]) * p.Hk + h / p.R) * DK + d);
    }
    for (int i = tid; i < m * L::DVS; i += L::NT) {
      const int j = i / L::DVS, c = i % L::DVS;
      sv[j][c] = ld_in(static_cast<const T*>(p.v), ((seq.tok0 + path[b - j]) * p.H + h) * DV + c0 + c);
    }
    __syncthreads();
    for (int j = 0; j < m; ++j) {
      const float4 v4 = *reinterpret_cast<const float4*>(&sv[j][4 * cq]);
#pragma unroll
      for (int i = 0; i < L::VPT; ++i) s[i] = fma4(sk[j][rg + i * L::NRG], v4, s[i]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < L::VPT; ++i) *reinterpret_cast<float4*>(p.state_out + at + (int64_t)(rg + i * L::NRG) * DV) = s[i];
}

// Draft.  A CTA per (request, head, 32 columns): the columns of the state in
// shared memory, a warp per token, lane = column.
template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) lin_draft(const LinParams p) {
  constexpr int kCols = 32;
  __shared__ float S[DK][kCols];
  __shared__ LogSum G[kMaxDraft];
  __shared__ float la[kMaxDraft];
  __shared__ int8_t par[kMaxDraft];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, c0 = blockIdx.z * kCols, cols = min(kCols, p.dv - c0);
  const LinSeq seq = lin_seq(p, blockIdx.x);
  const bool first = tid == 0 && h == 0 && c0 == 0;
  if (seq.flag && first) attn_flag(p.status, seq.flag);
  if (!seq.ok || seq.len == 0) return;
  if (!load_parents(p, seq, par)) {
    if (first) attn_flag(p.status, kFlagBadCache);
    return;
  }
  const int n = (int)seq.len;
  const int64_t at = ((int64_t)seq.slot * p.H + h) * DK * p.dv + c0 + lane;
  for (int d = warp; d < DK; d += kThreads / 32) S[d][lane] = lane < cols ? p.state_in[at + (int64_t)d * p.dv] : 0.f;
  if (tid < n) la[tid] = lin_log2_alpha<T>(p, seq.tok0 + tid, h);
  __syncthreads();
  if (tid == 0)
    for (int i = 0; i < n; ++i) {
      const LogSum own = log_sum(la[i]);
      G[i] = par[i] < 0 ? own : G[par[i]] + own;
    }
  __syncthreads();
  const T* k = static_cast<const T*>(p.k);
  const T* v = static_cast<const T*>(p.v);
  for (int i = warp; i < n; i += kThreads / 32) {
    float q[(DK + 31) / 32];
#pragma unroll
    for (int u = 0; u < (DK + 31) / 32; ++u)
      q[u] = 32 * u + lane < DK ? ld_in(static_cast<const T*>(p.q), ((seq.tok0 + i) * p.Hk + h / p.R) * DK + 32 * u + lane) : 0.f;
    float y = 0.f;
#pragma unroll
    for (int d = 0; d < DK; ++d) y = fmaf(__shfl_sync(0xffffffffu, q[d / 32], d % 32), S[d][lane], y);
    y *= exp2f(G[i].i + G[i].f);
    for (int j = i; j >= 0; j = par[j]) {
      float x = 0.f;
#pragma unroll
      for (int u = 0; u < (DK + 31) / 32; ++u)
        if (32 * u + lane < DK) x = fmaf(q[u], ld_in(k, ((seq.tok0 + j) * p.Hk + h / p.R) * DK + 32 * u + lane), x);
      x = warp_sum(x) * exp2f(log_diff(G[i], G[j]));
      if (lane < cols) y = fmaf(x, ld_in(v, ((seq.tok0 + j) * p.H + h) * p.dv + c0 + lane), y);
    }
    if (lane < cols) st_out(static_cast<T*>(p.o), ((seq.tok0 + i) * p.H + h) * p.dv + c0 + lane, y * p.scale);
  }
}

// ------------------------------------------------------------------ launches
template <typename T, int DK, int DV, bool kCommit>
cudaError_t launch_state(const LinParams& p, cudaStream_t stream) {
  using L = Tile<DK, DV>;
  const dim3 grid((unsigned)p.num_seqs, (unsigned)p.H, DV / L::DVS);
  if (kCommit) lin_commit<T, DK, DV><<<grid, L::NT, 0, stream>>>(p);
  else lin_decode<T, DK, DV><<<grid, L::NT, 0, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, int DK, bool kCommit>
cudaError_t launch_dv(const LinParams& p, cudaStream_t stream) {
  switch (p.dv) {
    case 16: return launch_state<T, DK, 16, kCommit>(p, stream);
    case 32: return launch_state<T, DK, 32, kCommit>(p, stream);
    case 64: return launch_state<T, DK, 64, kCommit>(p, stream);
    case 128: return launch_state<T, DK, 128, kCommit>(p, stream);
    case 256: return launch_state<T, DK, 256, kCommit>(p, stream);
  }
  return cudaErrorInvalidValue;
}
template <typename T, bool kCommit>
cudaError_t launch_dk(const LinParams& p, cudaStream_t stream) {
  switch (p.dk) {
    case 16: return launch_dv<T, 16, kCommit>(p, stream);
    case 32: return launch_dv<T, 32, kCommit>(p, stream);
    case 64: return launch_dv<T, 64, kCommit>(p, stream);
    case 128: return launch_dv<T, 128, kCommit>(p, stream);
    case 256: return launch_dv<T, 256, kCommit>(p, stream);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_draft_t(const LinParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.num_seqs, (unsigned)p.H, (unsigned)((p.dv + 31) / 32));
  switch (p.dk) {
    case 16: lin_draft<T, 16><<<grid, kThreads, 0, stream>>>(p); break;
    case 32: lin_draft<T, 32><<<grid, kThreads, 0, stream>>>(p); break;
    case 64: lin_draft<T, 64><<<grid, kThreads, 0, stream>>>(p); break;
    case 128: lin_draft<T, 128><<<grid, kThreads, 0, stream>>>(p); break;
    case 256: lin_draft<T, 256><<<grid, kThreads, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_decode(const LinParams& p, cudaStream_t stream) {
  return p.dt == KDA_BF16 ? launch_dk<__nv_bfloat16, false>(p, stream) : launch_dk<float, false>(p, stream);
}
cudaError_t launch_lin_commit(const LinParams& p, cudaStream_t stream) {
  return p.dt == KDA_BF16 ? launch_dk<__nv_bfloat16, true>(p, stream) : launch_dk<float, true>(p, stream);
}
cudaError_t launch_lin_draft(const LinParams& p, cudaStream_t stream) {
  return p.dt == KDA_BF16 ? launch_draft_t<__nv_bfloat16>(p, stream) : launch_draft_t<float>(p, stream);
}

}  // namespace kda
