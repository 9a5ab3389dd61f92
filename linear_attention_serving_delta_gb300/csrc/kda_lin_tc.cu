// kda_lin_tc.cu -- linear attention with a decay for each head over packed
// prompts on the tcgen05 tensor cores: bf16, states in fp32.
//
// Chunks of C = 128 tokens, with G_i = sum_{m <= i} log2 alpha_m within a chunk:
//
//   P = Q K^T                          tcgen05
//   P~_ij = 2^{G_i - G_j} P_ij, j <= i rounded to bf16, into P's columns of TMEM
//   O = 2^{G_i} (Q S) + P~ V           tcgen05, S rounded to bf16 for this alone
//   S <- 2^{G_C} S + K~^T V            K~_j = 2^{G_C - G_j} k_j in two bf16 parts
//
// K~ = hi + lo leaves out less than 2^-16 of a term, so states keep fp32's
// precision to about 1e-6 in norm (hi alone: 1e-3); the product starts from zero in each
// chunk and is added to S in registers, rounded to nearest (the tensor cores'
// own accumulation cuts, a bias that grows with the chunks).  All exponents
// are <= 0 and taken as differences before the exponential.
//
// A CTA runs one chain: a sequence (or a segment of one) of a head and DV columns
// of its state, chunk after chunk.  Warps 0-3: P~ and the outputs, a thread a
// row.  Warps 4-11: the state, DV / 2 columns of a row in a thread's registers; they
// also look through V and make K~ in place: hi over K, lo over Q, which the
// products before have read.  Warp 12 copies, 13 issues the MMAs, 14 sums the gates.
//
// Bytes of a chunk at 128 x 128: 128 KB, 2.9 us of an SM's share of HBM; the chain
// through the state (Q S, K~, K~^T V, S) takes about half of that.
//
// Values that are not finite.  P~ is exactly 0 at later tokens, which would
// still turn their infinities and NaN into NaN: V's are taken out in shared
// memory, and a channel is NaN in o from that token on, and in the state.  Rows
// of V and K~ behind the sequence are zeroed.
#include <cstddef>

#include "kda_lin_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int C = kLinChunk;
constexpr int kThreads = 480;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBlock = C * 128;  // bytes of 64 channels of a tile

template <int DK, int DV>
struct Shape {
  static constexpr int MB = DK > 128 ? DK / 128 : 1;       // row tiles of the state
  static constexpr uint32_t kQK = DK / 64 * kBlock, kVb = DV / 64 * kBlock;
  static constexpr uint32_t kSop = DK * DV * 2;            // the state as an operand
  static constexpr uint32_t kStage = 2 * kQK + kVb;
  static constexpr int kStages = (int)((229376 - kSop) / kStage) < 4 ? (int)((229376 - kSop) / kStage) : 4;
  static constexpr uint32_t kK = kStages * kQK;            // Q first
  static constexpr uint32_t kV = 2 * kStages * kQK;
  static constexpr uint32_t kS = kStages * kStage;
  static constexpr uint32_t kTail = kS + kSop;
  static constexpr uint32_t kBytes = kTail + 3072;
  static constexpr int kSCols = MB == 1 ? DV / 2 : DV;     // columns of a state thread
  // TMEM columns
  static constexpr int tP = 0, tOI = C, tOA = C + DV, tKV = C + 2 * DV;
  static_assert(tKV + MB * DV <= (int)kTmemCols && kStages >= 1 && kBytes <= 232448, "fits an SM");
};

struct Tail {
  uint64_t qk_full[4], v_full[4], empty[4];
  uint64_t p_full, qs_done, o_full, kv_full;               // committed by the MMA warp
  uint64_t s_ready, p_ready, v_ready, k_ready, o_free, g_full, g_free, meet, drain;
  uint32_t dead, tmem;
  uint32_t poisoned;      // some channel's nan_from is set
  float total;            // log2 of the chunk's decay
  float block_total[4];   // and of its blocks of 32 tokens
  // (the outputs read these two four at a time)
  alignas(16) float g32[C];     // sum of log2 alpha from the start of the token's block of 32
  alignas(16) float to_end[C];  // 2^ of the sum over what follows it in its block
  float w[C];             // 2^{G_C - G_j}
  int32_t nan_from[128];  // first token of the chain with a value that is not finite, per channel
};
static_assert(sizeof(Tail) <= 3072 && offsetof(Tail, g32) % 16 == 0 && offsetof(Tail, to_end) % 16 == 0, "tail block");

struct Chain {
  int32_t tok0, len, head, tile, from, to;
  bool any;
};

// The CTA's i-th chain, for every role alike
__device__ __forceinline__ bool chain_at(const LinParams& p, const LinTcArgs& a, int i, Chain* ch) {
  if (a.items) {
    const int64_t w = nth_item(i);
    if (w >= *a.num_items) return false;
    const LinItem it = a.items[w];
    *ch = Chain{it.tok0, it.len, it.head, it.tile, it.from, it.to, true};
    return true;
  }
  if (i > 0) return false;
  const int per = p.H * a.tiles, s = (int)(blockIdx.x / per), r = (int)(blockIdx.x % per);
  const LinSeq seq = lin_seq(p, s);
  if (seq.flag && r == 0 && threadIdx.x == 0) attn_flag(p.status, seq.flag);
  const int row = -2 - seq.slot;
  *ch = Chain{(int32_t)seq.tok0, (int32_t)seq.len, r / a.tiles, r % a.tiles, p.state_in ? row : -1,
              p.state_out ? row : -1, seq.ok};
  return seq.ok;
}
// A state of the pool or the workspace
__device__ __forceinline__ int64_t state_at(const LinParams& p, int32_t place, int head) {
  return ((int64_t)(place >= 0 ? place : -2 - place) * p.H + head) * p.dk * p.dv;
}

// ------------------------------------------------------------------ copies
template <int DK, int DV, bool kLocal>
__device__ void copy_role(const LinParams& p, const LinTcArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                          const CUtensorMap* mv, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  Ring<S::kStages> ring;
  uint32_t n = 0;
  bool ok = true;
  Chain ch;
  for (int i = 0; ok && chain_at(p, a, i, &ch); ++i) {
    const int kh = ch.head / p.R;
    for (int t = 0; t < ch.len; t += C) {
      if (!(ok = wait_or_dead(&b->empty[ring.st], ring.ph ^ 1, &b->dead))) break;
      mbar_arrive_expect_tx(&b->qk_full[ring.st], kLocal ? S::kQK : 2 * S::kQK);
#pragma unroll
      for (int c = 0; c < DK / 64; ++c) {
        if (!kLocal) tma_3d(sm + ring.st * S::kQK + c * kBlock, mq, 64 * c, kh, ch.tok0 + t, &b->qk_full[ring.st]);
        tma_3d(sm + S::kK + ring.st * S::kQK + c * kBlock, mk, 64 * c, kh, ch.tok0 + t, &b->qk_full[ring.st]);
      }
      mbar_arrive_expect_tx(&b->v_full[ring.st], S::kVb);
#pragma unroll
      for (int c = 0; c < DV / 64; ++c)
        tma_3d(sm + S::kV + ring.st * S::kVb + c * kBlock, mv, ch.tile * DV + 64 * c, ch.head, ch.tok0 + t,
               &b->v_full[ring.st]);
      ring.next();
      ++n;
    }
  }
  // no copy of its own is in flight when a CTA that gave up exits
  if (!ok)
    for (uint32_t k = n > S::kStages ? n - S::kStages : 0; k < n; ++k) {
      mbar_wait(&b->qk_full[k % S::kStages], (k / S::kStages) & 1, kWaitLimitNs);
      mbar_wait(&b->v_full[k % S::kStages], (k / S::kStages) & 1, kWaitLimitNs);
    }
}

// ------------------------------------------------------------------ MMAs
template <int DK, int DV, bool kLocal>
__device__ void mma_role(const LinParams& p, const LinTcArgs& a, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  const uint32_t tmem = __shfl_sync(0xffffffffu, b->tmem, 0);
  constexpr uint32_t id_qk = idesc_bf16(C, C), id_n = idesc_bf16(C, DV, 0, 1), id_kv = idesc_bf16(C, DV, 1, 1);
  // K-major Q and K; channels of Q and K as rows of K~^T; V and S by rows of the contraction
  const uint64_t q0 = sdesc_sw128(smem_u32(sm), 16, 1024), k0 = sdesc_sw128(smem_u32(sm + S::kK), 16, 1024),
                 lo0 = sdesc_sw128(smem_u32(sm), kBlock, 1024), hi0 = sdesc_sw128(smem_u32(sm + S::kK), kBlock, 1024),
                 v0 = sdesc_sw128(smem_u32(sm + S::kV), kBlock, 1024),
                 s0 = sdesc_sw128(smem_u32(sm + S::kS), DK * 128, 1024);
  const bool issue = elect_one();
  Ring<S::kStages> ring;
  uint32_t n = 0, ns = 0;
  uint32_t* dead = &b->dead;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_dead(bar, parity, dead)) != 0;
  };
  bool ok = true;
  Chain ch;
  for (int i = 0; ok && chain_at(p, a, i, &ch); ++i) {
    bool has = ch.from != -1;  // a state to read o from
    for (int t = 0; t < ch.len; t += C, ++n, has = true) {
      const uint64_t qd = q0 + (uint64_t)(ring.st * (S::kQK >> 4)), kd = k0 + (uint64_t)(ring.st * (S::kQK >> 4)),
                     vd = v0 + (uint64_t)(ring.st * (S::kVb >> 4));
      if (!(ok = wait(&b->qk_full[ring.st], ring.ph))) break;
      if (!kLocal) {
        fence_after_sync();
        if (issue) {
#pragma unroll
          for (int s = 0; s < DK / 16; ++s) {
            const uint32_t off = ((s / 4) * kBlock + (s % 4) * 32) >> 4;
            mma_bf16(tmem + S::tP, qd + off, kd + off, id_qk, s > 0);
          }
          mma_commit(&b->p_full);
        }
        // the outputs of the chunk before have been read
        if (n > 0 && !(ok = wait(&b->o_free, (n - 1) & 1))) break;
        if (has) {
          if (!(ok = wait(&b->s_ready, ns & 1))) break;
          ++ns;
          fence_after_sync();
          if (issue) {
#pragma unroll
            for (int s = 0; s < DK / 16; ++s)
              mma_bf16(tmem + S::tOI, qd + (((s / 4) * kBlock + (s % 4) * 32) >> 4), s0 + (uint64_t)(s * (2048 >> 4)),
                       id_n, s > 0);
          }
        }
        if (issue) mma_commit(&b->qs_done);
        if (!(ok = wait(&b->v_ready, n & 1)) || !(ok = wait(&b->p_ready, n & 1))) break;
        fence_after_sync();
        if (issue) {
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16_ts(tmem + S::tOA, tmem + S::tP + s * 8, vd + (uint64_t)(s * (2048 >> 4)), id_n, s > 0);
          mma_commit(&b->o_full);
        }
      } else {
        if (!(ok = wait(&b->v_ready, n & 1))) break;
      }
      if (!(ok = wait(&b->k_ready, n & 1))) break;
      fence_after_sync();
      if (issue) {
        const uint64_t hd = hi0 + (uint64_t)(ring.st * (S::kQK >> 4)), ld = lo0 + (uint64_t)(ring.st * (S::kQK >> 4));
#pragma unroll
        for (int m = 0; m < S::MB; ++m)
#pragma unroll
          for (int s = 0; s < C / 16; ++s) {
            const uint32_t off = (2 * m * kBlock + s * 2048) >> 4;
            mma_bf16(tmem + S::tKV + m * DV, ld + off, vd + (uint64_t)(s * (2048 >> 4)), id_kv, s > 0);
            mma_bf16(tmem + S::tKV + m * DV, hd + off, vd + (uint64_t)(s * (2048 >> 4)), id_kv, 1);
          }
        mma_commit(&b->kv_full);
        mma_commit(&b->empty[ring.st]);
      }
      ring.next();
    }
  }
  // no MMA and no arrival of one is left in flight
  if (issue) mma_commit(&b->drain);
  mbar_wait(&b->drain, 0, kWaitLimitNs);
}

// ------------------------------------------------------------------ gates
// A warp, four neighbouring tokens a lane; the logits of the next chunk are
// read before this one's sums are waited for.
template <bool kLocal>
__device__ void gate_role(const LinParams& p, const LinTcArgs& a, Tail* b) {
  const int lane = threadIdx.x & 31;
  uint32_t n = 0;
  Chain ch;
  for (int i = 0; chain_at(p, a, i, &ch); ++i) {
    float x[4];
    auto fetch = [&](int t) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        x[u] = t + 4 * lane + u < ch.len ? lin_log2_alpha<__nv_bfloat16>(p, (int64_t)ch.tok0 + t + 4 * lane + u, ch.head)
                                         : 0.f;
    };
    if (ch.len > 0) fetch(0);
    for (int t = 0; t < ch.len; t += C, ++n) {
      LogSum g[4];
      g[0] = log_sum(x[0]);
#pragma unroll
      for (int u = 1; u < 4; ++u) g[u] = g[u - 1] + log_sum(x[u]);
      LogSum before = g[3];  // of the lanes up to this one, then of those before it
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const LogSum y{__shfl_up_sync(0xffffffffu, before.i, o), __shfl_up_sync(0xffffffffu, before.f, o)};
        if (lane >= o) before = y + before;
      }
      auto from = [&](int src) {
        return LogSum{__shfl_sync(0xffffffffu, before.i, src), __shfl_sync(0xffffffffu, before.f, src)};
      };
      const LogSum end = from(lane | 7), all = from(31), prev = from(lane > 0 ? lane - 1 : 0),
                   start = from(lane >= 8 ? (lane & ~7) - 1 : 0);
      const bool first = lane == 0, first_block = lane < 8;
      if (t + C < ch.len) fetch(t + C);
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->g_free, (n & 1) ^ 1, &b->dead))) return;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const LogSum G = first ? g[u] : prev + g[u];
        const int j = 4 * lane + u;
        b->g32[j] = first_block ? G.i + G.f : log_diff(G, start);
        b->to_end[j] = exp2f(log_diff(end, G));
        b->w[j] = exp2f(log_diff(all, G));
      }
      if ((lane & 7) == 7) b->block_total[lane >> 3] = first_block ? end.i + end.f : log_diff(end, start);
      if (lane == 31) b->total = all.i + all.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->g_full);
    }
  }
}

// ------------------------------------------------------------------ outputs
template <int DK, int DV>
__device__ void out_role(const LinParams& p, const LinTcArgs& a, Tail* b) {
  using S = Shape<DK, DV>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = 32 * warp + lane;
  const uint32_t lanes = (uint32_t)(32 * warp) << 16, tp = b->tmem + lanes + S::tP;
  uint32_t* dead = &b->dead;
  uint32_t n = 0;
  Chain ch;
  for (int i = 0; chain_at(p, a, i, &ch); ++i) {
    bool has = ch.from != -1;
    for (int t = 0; t < ch.len; t += C, ++n, has = true) {
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->g_full, n & 1, dead))) return;
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->p_full, n & 1, dead))) return;
      fence_after_sync();
      const float gi = b->g32[row];
      // 2^{G_i - G_j}: within the row's own block of 32 tokens from the difference,
      // for an earlier block as 2^{G_i - G_e} 2^{G_e - G_j}, e the block's last token
      float since = gi;  // from the end of block c to the row
      float back[4];
#pragma unroll
      for (int c = 3; c >= 0; --c) {
        if (c >= warp) {
          back[c] = 0.f;
        } else {
          back[c] = exp2_fast(since);
          since += b->block_total[c];
        }
      }
      const float from_start = exp2f(since);  // 2^{G_i}
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
        if (c <= warp) {
          float s[32];
          tmem_ld32(tp + 32 * c, s);
          tmem_ld_wait();
          if (c < warp) {
#pragma unroll
            for (int u = 0; u < 32; u += 4) {
              const float4 e = *reinterpret_cast<const float4*>(&b->to_end[32 * c + u]);
              pk[u / 2] = pack2(s[u] * (back[c] * e.x), s[u + 1] * (back[c] * e.y));
              pk[u / 2 + 1] = pack2(s[u + 2] * (back[c] * e.z), s[u + 3] * (back[c] * e.w));
            }
          } else {
#pragma unroll
            for (int u = 0; u < 32; u += 4) {
              const float4 g = *reinterpret_cast<const float4*>(&b->g32[32 * c + u]);
              const float y0 = u <= lane ? s[u] * exp2_fast(gi - g.x) : 0.f,
                          y1 = u + 1 <= lane ? s[u + 1] * exp2_fast(gi - g.y) : 0.f,
                          y2 = u + 2 <= lane ? s[u + 2] * exp2_fast(gi - g.z) : 0.f,
                          y3 = u + 3 <= lane ? s[u + 3] * exp2_fast(gi - g.w) : 0.f;
              pk[u / 2] = pack2(y0, y1);
              pk[u / 2 + 1] = pack2(y2, y3);
            }
          }
        } else {
#pragma unroll
          for (int u = 0; u < 16; ++u) pk[u] = 0;
        }
        tmem_st16(tp + 16 * c, reinterpret_cast<const float*>(pk));
      }
      tmem_st_wait();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&b->p_ready);
        mbar_arrive(&b->g_free);
      }
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->o_full, n & 1, dead))) return;
      fence_after_sync();
      const bool mine = t + row < ch.len;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) +
                         ((int64_t)(ch.tok0 + t + row) * p.H + ch.head) * p.dv + ch.tile * DV;
      const bool poisoned = *reinterpret_cast<volatile uint32_t*>(&b->poisoned) != 0;
      const int width = min(DV, p.dv - ch.tile * DV);
#pragma unroll 1
      for (int c = 0; c < width; c += 32) {
        float x[32];
        tmem_ld32(tp + (S::tOA - S::tP) + c, x);
        if (has) {
          float y[32];
          tmem_ld32(tp + (S::tOI - S::tP) + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 32; ++u) x[u] = fmaf(from_start, y[u], x[u]);
        } else {
          tmem_ld_wait();
        }
        if (poisoned)
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if (reinterpret_cast<const volatile int32_t*>(b->nan_from)[c + u] <= t + row) x[u] = NAN;
        if (mine) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) pk[u] = pack2(x[2 * u] * p.scale, x[2 * u + 1] * p.scale);
          st_32b(o + c, pk, a.o_wide);
          if (c + 16 < width) st_32b(o + c + 16, pk + 8, a.o_wide);
        }
        __syncwarp();
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->o_free);
    }
  }
}

// ------------------------------------------------------------------ the state
template <int DK, int DV, bool kLocal>
__device__ void state_role(const LinParams& p, const LinTcArgs& a, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  constexpr int N = S::kSCols;
  const int x = threadIdx.x - 128, lane = x & 31, quarter = (x >> 5) & 3, half = x >> 7;
  // the state: row d, columns [col, col + N)
  const int d = 32 * quarter + lane + (S::MB > 1 ? 128 * half : 0), col = S::MB > 1 ? 0 : half * N;
  const bool holds = d < DK;
  const uint32_t kv = b->tmem + ((uint32_t)(32 * quarter) << 16) + S::tKV + half * N;
  // copies: row r of a tile, half of its 16-byte pieces
  const int r = x & 127;
  uint32_t* dead = &b->dead;
  uint32_t n = 0, met = 0;
  Ring<S::kStages> ring;
  // the state's threads meet (a wait with a limit, as all others)
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->meet);
    return __all_sync(0xffffffffu, wait_or_dead(&b->meet, met++ & 1, dead)) != 0;
  };
  Chain ch;
  for (int i = 0; chain_at(p, a, i, &ch); ++i) {
    float s[N];
    const int c0 = ch.tile * DV + col;  // of the head's columns
    const bool mine = holds && d < p.dk;
    {
      const float* from = ch.from == -1 ? nullptr : (ch.from >= 0 ? a.states : p.state_in) + state_at(p, ch.from, ch.head);
#pragma unroll
      for (int u = 0; u < N; u += 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from && mine && c0 + u < p.dv) y = *reinterpret_cast<const float4*>(from + (int64_t)d * p.dv + c0 + u);
        s[u] = y.x;
        s[u + 1] = y.y;
        s[u + 2] = y.z;
        s[u + 3] = y.w;
      }
    }
    // what was noted in the chain before is dropped once its last outputs are written
    if (!meet()) return;
    if (!kLocal && n > 0 && *reinterpret_cast<volatile uint32_t*>(&b->poisoned) &&
        !__all_sync(0xffffffffu, wait_or_dead(&b->o_free, (n - 1) & 1, dead)))
      return;
    if (!meet()) return;
    if (x < DV) b->nan_from[x] = INT32_MAX;
    if (x == 0) b->poisoned = 0;
    if (!meet()) return;
    LinDecay decay{0.f, true};
    bool has = ch.from != -1;
    // S <- decay S + K~^T V of the chunk before, which ended at token t
    auto advance = [&](int t) -> bool {
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->kv_full, (n - 1) & 1, dead))) return false;
      fence_after_sync();
      if (holds) {
#pragma unroll
        for (int c = 0; c < N; c += 32) {
          float y[32];
          tmem_ld32(kv + c, y);
          tmem_ld_wait();
          if (decay.near_one) {
#pragma unroll
            for (int u = 0; u < 32; ++u) s[c + u] = fmaf(decay.m, s[c + u], s[c + u]) + y[u];
          } else {
#pragma unroll
            for (int u = 0; u < 32; ++u) s[c + u] = fmaf(decay.m, s[c + u], y[u]);
          }
        }
        if (*reinterpret_cast<volatile uint32_t*>(&b->poisoned))
#pragma unroll
          for (int u = 0; u < N; ++u)
            if (reinterpret_cast<volatile int32_t*>(b->nan_from)[col + u] < t) s[u] = NAN;
      }
      fence_before_sync();
      return true;
    };
    for (int t = 0; t < ch.len; t += C, ++n, has = true) {
      const int live = min(C, ch.len - t);
      // V: rows behind the sequence to zero, values that are not finite out
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->v_full[ring.st], ring.ph, dead))) return;
      {
        char* vt = sm + S::kV + ring.st * S::kVb;
        constexpr int P = DV / 16;
        if (r >= live) {
#pragma unroll
          for (int c = 0; c < P; ++c) *reinterpret_cast<uint4*>(vt + sw_off(r, half * P + c, kBlock)) = make_uint4(0, 0, 0, 0);
        } else {
          uint32_t seen = 0;
#pragma unroll
          for (int c = 0; c < P; ++c) seen |= exponents_full(*reinterpret_cast<const uint4*>(vt + sw_off(r, half * P + c, kBlock)));
          if (seen & 0x80008000u) {
#pragma unroll 1
            for (int c = 0; c < P; ++c) {
              uint4* at = reinterpret_cast<uint4*>(vt + sw_off(r, half * P + c, kBlock));
              const uint4 y = *at;
              const uint32_t bad = nonfinite8(y);
              if (!bad) continue;
              for (int e = 0; e < 8; ++e)
                if (bad >> e & 1) atomicMin_block(&b->nan_from[8 * (half * P + c) + e], t + r);
              *at = make_uint4(finite_only(y.x), finite_only(y.y), finite_only(y.z), finite_only(y.w));
            }
            *reinterpret_cast<volatile uint32_t*>(&b->poisoned) = 1;
          }
        }
      }
      fence_async_smem();
      // the state after the chunk before, also as an operand
      if (t > 0 && !advance(t)) return;
      __syncwarp();
      // (behind kv_full, so that the MMA warp has passed the arrival of the chunk before)
      if (lane == 0) mbar_arrive(&b->v_ready);
      if (!kLocal && has) {
        if (holds) {
          char* st = sm + S::kS;
#pragma unroll
          for (int u = 0; u < N; u += 8)
            *reinterpret_cast<uint4*>(st + sw_off(d, (col + u) / 8, DK * 128)) =
                make_uint4(pack2(s[u], s[u + 1]), pack2(s[u + 2], s[u + 3]), pack2(s[u + 4], s[u + 5]), pack2(s[u + 6], s[u + 7]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->s_ready);
      }
      // K~
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->g_full, n & 1, dead))) return;
      const float w = b->w[r];
      decay = lin_decay(b->total);
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->qk_full[ring.st], ring.ph, dead))) return;
      if (!kLocal && !__all_sync(0xffffffffu, wait_or_dead(&b->qs_done, n & 1, dead))) return;
      fence_after_sync();
      {
        char *lo = sm + ring.st * S::kQK, *hi = sm + S::kK + ring.st * S::kQK;
        constexpr int P = DK / 16;
#pragma unroll 4
        for (int c = 0; c < P; ++c) {
          const uint32_t off = sw_off(r, half * P + c, kBlock);
          uint4 h4 = make_uint4(0, 0, 0, 0), l4 = h4;
          if (r < live) {
            const uint4 k4 = *reinterpret_cast<const uint4*>(hi + off);
            auto part = [&](uint32_t k2, uint32_t* h2, uint32_t* l2) {
              const float k0 = bf_lo(k2), k1 = bf_hi(k2);
              *h2 = pack2(k0 * w, k1 * w);
              *l2 = pack2(fmaf(k0, w, -bf_lo(*h2)), fmaf(k1, w, -bf_hi(*h2)));
            };
            part(k4.x, &h4.x, &l4.x);
            part(k4.y, &h4.y, &l4.y);
            part(k4.z, &h4.z, &l4.z);
            part(k4.w, &h4.w, &l4.w);
          }
          *reinterpret_cast<uint4*>(hi + off) = h4;
          *reinterpret_cast<uint4*>(lo + off) = l4;
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&b->k_ready);
        mbar_arrive(&b->g_free);
      }
      ring.next();
    }
    if (ch.len > 0 && !advance(ch.len)) return;
    if (ch.to != -1 && mine) {
      float* to = (ch.to >= 0 ? a.states : p.state_out) + state_at(p, ch.to, ch.head) + (int64_t)d * p.dv + c0;
#pragma unroll
      for (int u = 0; u < N; u += 4)
        if (c0 + u < p.dv) *reinterpret_cast<float4*>(to + u) = make_float4(s[u], s[u + 1], s[u + 2], s[u + 3]);
    }
  }
}

template <int DK, int DV, bool kLocal>
__global__ void __launch_bounds__(kThreads, 1)
    lin_tc(const LinParams p, const LinTcArgs a, const __grid_constant__ CUtensorMap mq,
           const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Shape<DK, DV>;
  extern __shared__ __align__(1024) char sm[];
  Tail* b = reinterpret_cast<Tail*>(sm + S::kTail);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&b->qk_full[s], 1);
      mbar_init(&b->v_full[s], 1);
      mbar_init(&b->empty[s], 1);
    }
    for (uint64_t* x : {&b->p_full, &b->qs_done, &b->o_full, &b->kv_full, &b->g_full, &b->drain}) mbar_init(x, 1);
    for (uint64_t* x : {&b->s_ready, &b->v_ready, &b->k_ready, &b->meet}) mbar_init(x, 8);
    mbar_init(&b->p_ready, 4);
    mbar_init(&b->o_free, 4);
    mbar_init(&b->g_free, kLocal ? 8 : 12);
    b->dead = 0;
    mbar_init_fence();
  }
  if (threadIdx.x == 32) {
    if (!kLocal) prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
  }
  if (warp == 13) tmem_alloc(&b->tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  pdl_wait();  // the plan, or what came before
  if (warp < 4) {
    if (!kLocal) out_role<DK, DV>(p, a, b);
  } else if (warp < 12) {
    state_role<DK, DV, kLocal>(p, a, sm, b);
  } else if (warp == 12) {
    if ((threadIdx.x & 31) == 0) copy_role<DK, DV, kLocal>(p, a, &mq, &mk, &mv, sm, b);
  } else if (warp == 13) {
    mma_role<DK, DV, kLocal>(p, a, sm, b);
  } else {
    gate_role<kLocal>(p, a, b);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && b->dead) attn_flag(p.status, kFlagTimeout);
  if (warp == 13) tmem_dealloc(b->tmem, kTmemCols);
}

// ------------------------------------------------------------------ host
// Column tiles: 128 wide, 64 where the keys are 256 or the values no wider
int tile_width(const LinParams& p) { return p.dk > 128 || p.dv <= 64 ? 64 : 128; }

bool lin_map(CUtensorMap* m, const void* base, int64_t tokens, int heads, int d) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * heads};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)C}, elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV>
cudaError_t launch_shape(const LinParams& p, void* ws, cudaStream_t stream) {
  using S = Shape<DK, DV>;
  CUtensorMap mq, mk, mv;
  if (!lin_map(&mq, p.q, p.total_tokens, p.Hk, p.dk) || !lin_map(&mk, p.k, p.total_tokens, p.Hk, p.dk) ||
      !lin_map(&mv, p.v, p.total_tokens, p.H, p.dv))
    return cudaErrorInvalidValue;
  LinTcArgs a{};
  a.tiles = (p.dv + DV - 1) / DV;
  a.o_wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
  cudaError_t e =
      cudaFuncSetAttribute(lin_tc<DK, DV, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t chains = (int64_t)p.num_seqs * p.H * a.tiles;
  return launch_maybe_dependent(true, lin_tc<DK, DV, false>, dim3((unsigned)chains), dim3(kThreads), (size_t)S::kBytes,
                                stream, p, a, mq, mk, mv);
}

}  // namespace

// bf16 with what the tensor maps need: 16-byte aligned bases; some token
bool lin_tc_fits(const LinParams& p) {
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  return p.dt == KDA_BF16 && p.total_tokens > 0 && al16(p.q) && al16(p.k) && al16(p.v) && al16(p.o) &&
         (int64_t)p.num_seqs * p.H * 4 < INT32_MAX;
}
size_t lin_tc_workspace(const LinParams&) { return 256; }
cudaError_t launch_lin_tc(const LinParams& p, void* ws, cudaStream_t stream) {
  const int w = tile_width(p);
  if (p.dk > 128) return launch_shape<256, 64>(p, ws, stream);
  if (p.dk > 64) return w == 64 ? launch_shape<128, 64>(p, ws, stream) : launch_shape<128, 128>(p, ws, stream);
  return w == 64 ? launch_shape<64, 64>(p, ws, stream) : launch_shape<64, 128>(p, ws, stream);
}

}  // namespace kda
