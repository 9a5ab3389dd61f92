// kda_lin_simt.cu -- linear attention with a decay for each head over packed
// prompts, token by token on the fp32 CUDA cores: every type, size and
// alignment the ABI takes.
//
//   S = alpha_t S + k_t v_t^T,   o_t = scale S^T q_t
//
// A CTA runs one (sequence, head, 32 columns of the state).  Lane = column; the
// eight warps share the key channels, DK / 8 of the state in each thread's
// registers.  Tokens go through shared memory a few at a time; each warp
// leaves its part of their o there, and the parts are added up in warp order.
// Bound by the chain: three operations on every element of the state a token.
#include "kda_lin.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kCols = 32;

template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) lin_simt(const LinParams p) {
  constexpr int R = DK / kWarps;             // key channels of a thread
  constexpr int kTok = DK == 256 ? 8 : 16;  // tokens of a block: 48 KB hold them
  __shared__ float sq[kTok][DK], sk[kTok][DK], sv[kTok][kCols];
  __shared__ LinDecay sa[kTok];
  __shared__ float so[kWarps][kTok][kCols];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * kCols, cols = min(kCols, p.dv - c0);
  const LinSeq seq = lin_seq(p, s);
  if (seq.flag && tid == 0 && h == 0 && c0 == 0) attn_flag(p.status, seq.flag);
  if (!seq.ok) return;
  const T* q = static_cast<const T*>(p.q);
  const T* k = static_cast<const T*>(p.k);
  const T* v = static_cast<const T*>(p.v);
  T* o = static_cast<T*>(p.o);
  const int64_t at = ((int64_t)seq.slot * p.H + h) * DK * p.dv + c0 + lane;
  float S[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    S[i] = p.state_in && lane < cols ? p.state_in[at + (int64_t)(warp * R + i) * p.dv] : 0.f;
  for (int64_t t0 = 0; t0 < seq.len; t0 += kTok) {
    const int n = (int)min((int64_t)kTok, seq.len - t0);
    const int64_t tok = seq.tok0 + t0;
    for (int i = tid; i < n * DK; i += kThreads) {
      const int t = i / DK, d = i % DK;
      const int64_t x = ((tok + t) * p.Hk + h / p.R) * DK + d;
      sq[t][d] = ld_in(q, x);
      sk[t][d] = ld_in(k, x);
    }
    for (int i = tid; i < n * kCols; i += kThreads) {
      const int t = i / kCols, c = i % kCols;
      sv[t][c] = c < cols ? ld_in(v, ((tok + t) * p.H + h) * p.dv + c0 + c) : 0.f;
    }
    if (tid < n) sa[tid] = lin_decay(lin_log2_alpha<T>(p, tok + tid, h));
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const LinDecay a = sa[t];
      const float x = sv[t][lane];
      float y = 0.f;
      if (a.near_one) {
#pragma unroll
        for (int i = 0; i < R; ++i) S[i] = fmaf(a.m, S[i], S[i]);
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i) S[i] *= a.m;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        S[i] = fmaf(sk[t][warp * R + i], x, S[i]);
        y = fmaf(sq[t][warp * R + i], S[i], y);
      }
      so[warp][t][lane] = y;
    }
    __syncthreads();
    for (int i = tid; i < n * kCols; i += kThreads) {
      const int t = i / kCols, c = i % kCols;
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) y += so[w][t][c];
      if (c < cols) st_out(o, ((tok + t) * p.H + h) * p.dv + c0 + c, y * p.scale);
    }
  }
  if (p.state_out && lane < cols)
#pragma unroll
    for (int i = 0; i < R; ++i) p.state_out[at + (int64_t)(warp * R + i) * p.dv] = S[i];
}

template <typename T>
cudaError_t launch_t(const LinParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.num_seqs, (unsigned)p.H, (unsigned)((p.dv + kCols - 1) / kCols));
  switch (p.dk) {
    case 16: lin_simt<T, 16><<<grid, kThreads, 0, stream>>>(p); break;
    case 32: lin_simt<T, 32><<<grid, kThreads, 0, stream>>>(p); break;
    case 64: lin_simt<T, 64><<<grid, kThreads, 0, stream>>>(p); break;
    case 128: lin_simt<T, 128><<<grid, kThreads, 0, stream>>>(p); break;
    case 256: lin_simt<T, 256><<<grid, kThreads, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_simt(const LinParams& p, cudaStream_t stream) {
  return p.dt == KDA_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace kda
