// kda_lin_simt.cu -- linear attention with a decay for each head over packed
// prompts, token by token on the fp32 CUDA cores: every type, size and
// alignment the ABI takes.
//
//   S = alpha_t S + k_t v_t^T,   o_t = scale S^T q_t
//
// A CTA runs one chain: a sequence, or a segment of one (kda_lin_plan.cu), of a
// head and 32 or 64 columns of the state.  Lane = column; the eight warps share the key
// channels, DK / 8 of the state in each thread's registers.  Tokens go through
// shared memory a few at a time, the next ones on their way in registers; each warp
// leaves its part of their o there, and the parts are added up in warp order.
//
// Bound by instructions: three fused operations on every element of the state a token,
// which no tensor core does to fp32 precision at a better rate.  Two prompts of 500 to
// 1,500 tokens, 8 heads of 64 x 64: 217 us as one chain a sequence and 32 columns, 67 in
// segments of 32 tokens and up, 53 with two columns a lane (an element of k or q
// from shared memory serves both), 47 with segments in steps of 16 tokens.
#include <algorithm>

#include "kda_lin_tc.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = 8;

// Columns of a lane: a key's or query's element from shared memory serves both (256
// key channels leave no registers for two)
int cols_of(const LinParams& p) { return p.dk == 256 ? 1 : (p.dv > 32 ? 2 : 1); }

// kFirst: the first pass over segments, most of which leave their end states alone
template <typename T, int DK, int NC, bool kFirst>
__global__ void __launch_bounds__(kThreads, 3) lin_simt(const LinParams p, const LinPlan a, const bool planned) {
  constexpr int R = DK / kWarps, kCols = 32 * NC;      // key channels of a thread, columns of the CTA
  constexpr int kTok = DK > 64 ? 8 : 16;               // tokens of a block: 48 KB hold them
  constexpr int kQK = kTok * DK / kThreads, kV = kTok * kCols / kThreads;  // a thread's share
  static_assert(kQK * kThreads == kTok * DK && kV * kThreads == kTok * kCols, "whole shares");
  __shared__ __align__(16) float sq[kTok][DK], sk[kTok][DK];
  __shared__ __align__(16) float sv[kTok][kCols], so[kWarps][kTok][kCols];
  __shared__ LinDecay sa[kTok];
  __shared__ float sl[kTok];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, c0 = blockIdx.z * kCols, cols = min(kCols, p.dv - c0);
  LinItem it{};
  if (planned) {
    if ((int)blockIdx.x >= (kFirst ? a.head->locals : a.head->items)) return;
    it = (kFirst ? a.locals : a.items)[blockIdx.x];
  } else {
    const LinSeq seq = lin_seq(p, blockIdx.x);
    if (seq.flag && tid == 0 && h == 0 && c0 == 0) attn_flag(p.status, seq.flag);
    if (!seq.ok) return;
    const int row = -2 - seq.slot;
    it = LinItem{(int32_t)seq.tok0, (int32_t)seq.len, h, 0, p.state_in ? row : -1, p.state_out ? row : -1, 0, 1};
  }
  const bool local = kFirst && !it.outputs;
  // element i of the thread's columns: lane + 32 i
  float S[R][NC];
  auto state_at = [&](int32_t place) {
    return ((int64_t)(place >= 0 ? place : -2 - place) * p.H + h) * DK * p.dv + (int64_t)warp * R * p.dv + c0 + lane;
  };
  auto put_state = [&](float* to) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (lane + 32 * j < cols) to[(int64_t)i * p.dv + 32 * j] = S[i][j];
  };
  {
    const float* from = it.from == -1 ? nullptr : (it.from >= 0 ? a.states : p.state_in) + state_at(it.from);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < NC; ++j) S[i][j] = from && lane + 32 * j < cols ? from[(int64_t)i * p.dv + 32 * j] : 0.f;
  }
  // the next block of tokens, in registers: element u of a thread is kThreads on
  const int64_t row_k = (int64_t)p.Hk * DK, row_v = (int64_t)p.H * p.dv;
  const int tk = tid / DK, tv = tid / kCols, cv = tid % kCols;
  const int64_t at_k = ((int64_t)it.tok0 + tk) * row_k + (int64_t)(h / p.R) * DK + tid % DK;
  const int64_t at_v = ((int64_t)it.tok0 + tv) * row_v + (int64_t)h * p.dv + c0 + cv;
  const T* q = static_cast<const T*>(p.q) + at_k;
  const T* k = static_cast<const T*>(p.k) + at_k;
  const T* v = static_cast<const T*>(p.v) + at_v;
  T* o = static_cast<T*>(p.o) + at_v;
  float rq[kQK], rk[kQK], rv[kV], rg = 0.f;
  auto fetch = [&](int t0) {
    const int n = it.len - t0;
#pragma unroll
    for (int u = 0; u < kQK; ++u) {
      const int t = u * (kThreads / DK);
      if (tk + t >= n) continue;
      if (!local) rq[u] = ld_in(q, (t0 + t) * row_k);
      rk[u] = ld_in(k, (t0 + t) * row_k);
    }
#pragma unroll
    for (int u = 0; u < kV; ++u) {
      const int t = u * (kThreads / kCols);
      rv[u] = tv + t < n && cv < cols ? ld_in(v, (t0 + t) * row_v) : 0.f;
    }
    if (tid < min(n, kTok)) rg = lin_gate<T>(p, (int64_t)it.tok0 + t0 + tid, h);
  };
  LogSum sum{0.f, 0.f};  // log2 of the chain's decay, in the first thread
  if (it.len > 0) fetch(0);
  for (int t0 = 0; t0 < it.len; t0 += kTok) {
    const int n = min(kTok, it.len - t0);
#pragma unroll
    for (int u = 0; u < kQK; ++u) {
      if (!local) (&sq[0][0])[tid + u * kThreads] = rq[u];
      (&sk[0][0])[tid + u * kThreads] = rk[u];
    }
#pragma unroll
    for (int u = 0; u < kV; ++u) (&sv[0][0])[tid + u * kThreads] = rv[u];
    if (tid < n) {
      const float l = lin_log2_alpha(p, rg, h);
      sa[tid] = lin_decay(l);
      sl[tid] = l;
    }
    __syncthreads();
    if (t0 + kTok < it.len) fetch(t0 + kTok);
    if (local && tid == 0)
      for (int t = 0; t < n; ++t) sum = sum + log_sum(sl[t]);
#pragma unroll 2
    for (int t = 0; t < n; ++t) {
      const LinDecay d = sa[t];
      float x[NC], y[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) x[j] = sv[t][lane + 32 * j], y[j] = 0.f;
      if (d.near_one) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < NC; ++j) S[i][j] = fmaf(d.m, S[i][j], fmaf(sk[t][warp * R + i], x[j], S[i][j]));
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < NC; ++j) S[i][j] = fmaf(d.m, S[i][j], sk[t][warp * R + i] * x[j]);
      }
      if (local) continue;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j) y[j] = fmaf(sq[t][warp * R + i], S[i][j], y[j]);
#pragma unroll
      for (int j = 0; j < NC; ++j) so[warp][t][lane + 32 * j] = y[j];
    }
    __syncthreads();
    if (local) continue;
#pragma unroll
    for (int u = 0; u < kV; ++u) {
      const int t = u * (kThreads / kCols);
      if (tv + t >= n || cv >= cols) continue;
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) y += so[w][tv + t][cv];
      st_out(o, (t0 + t) * row_v, y * p.scale);
    }
  }
  if (it.to != -1) put_state((it.to >= 0 ? a.states : p.state_out) + state_at(it.to));
  if (local && c0 == 0 && tid == 0) a.logs[(int64_t)it.to * p.H + h] = sum.i + sum.f;
}

// Three CTAs an SM (chains for four, with registers for two: 108 us where three with
// registers for three took 87), in segments of 32 tokens and up (of 128 and up: 87 us where
// these took 70) in steps of 16 (of 32: 55 us where these took 47)
LinShare share(const LinParams& p) {
  const int cols = 32 * cols_of(p);
  return LinShare{(p.dv + cols - 1) / cols, kLinSimtSlots, 16, 2, 8, 32, false};
}

template <typename T, int DK, int NC>
cudaError_t launch_nc(const LinParams& p, void* ws, cudaStream_t stream) {
  const LinShare sh = share(p);
  const LinLayout L = lin_layout(p, sh);
  const LinPlan plan = lin_plan_of(p, sh, L, ws);
  auto run = [&](auto kernel, int64_t x, bool planned) {
    return launch_maybe_dependent(true, kernel, dim3((unsigned)x, (unsigned)p.H, (unsigned)sh.tiles), dim3(kThreads), 0,
                                  stream, p, plan, planned);
  };
  if (!L.may_split) return run(lin_simt<T, DK, NC, false>, p.num_seqs, false);
  const int64_t chains = sh.slots / ((int64_t)p.H * sh.tiles);  // of cut sequences, at most, in either pass
  cudaError_t e = launch_lin_plan(p, plan, stream);
  if (e == cudaSuccess) e = run(lin_simt<T, DK, NC, true>, chains, true);
  if (e == cudaSuccess) e = launch_lin_combine(p, plan, stream);
  return e != cudaSuccess ? e : run(lin_simt<T, DK, NC, false>, p.num_seqs + chains, true);
}

template <typename T, int DK>
cudaError_t launch_dk(const LinParams& p, void* ws, cudaStream_t stream) {
  if constexpr (DK < 256)
    if (cols_of(p) == 2) return launch_nc<T, DK, 2>(p, ws, stream);
  return launch_nc<T, DK, 1>(p, ws, stream);
}

template <typename T>
cudaError_t launch_t(const LinParams& p, void* ws, cudaStream_t stream) {
  switch (p.dk) {
    case 16: return launch_dk<T, 16>(p, ws, stream);
    case 32: return launch_dk<T, 32>(p, ws, stream);
    case 64: return launch_dk<T, 64>(p, ws, stream);
    case 128: return launch_dk<T, 128>(p, ws, stream);
    case 256: return launch_dk<T, 256>(p, ws, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t lin_simt_workspace(const LinParams& p) { return lin_layout(p, share(p)).total; }
cudaError_t launch_lin_simt(const LinParams& p, void* ws, cudaStream_t stream) {
  return p.dt == KDA_BF16 ? launch_t<__nv_bfloat16>(p, ws, stream) : launch_t<float>(p, ws, stream);
}

}  // namespace kda
