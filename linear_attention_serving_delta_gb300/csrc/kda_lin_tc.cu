// kda_lin_tc.cu -- linear attention with a decay for each head over packed
// prompts on the tcgen05 tensor cores: bf16, states in fp32.
//
// Chunks of C = 128 tokens, with G_i = sum_{m <= i} log2 alpha_m within a chunk:
//
//   P = Q K^T                          tcgen05
//   P~_ij = 2^{M - G_j} P_ij, j <= i   rounded to bf16, into P's columns of TMEM
//   O = 2^{G_i - M} (Q 2^M S + P~ V)   tcgen05, P~ from TMEM; 2^M S rounded to bf16 for this alone
//   S <- 2^{G_C} S + K~^T V            K~_j = 2^{G_C - G_j} k_j in three bf16 parts, A from TMEM
//
// That is for a weak chunk, |G| <= 64, with M the middle of the G: no factor is above 2^33, and
// one of them is left to the epilogue.  In a strong one P~_ij = 2^{G_i - G_j} P_ij, the
// difference taken before the exponential (over whole blocks of 32 tokens as a product of two
// factors <= 1), and the queries are multiplied by theirs, Q~_i = 2^{G_i} q_i in bf16 beside P~.
//
// Three parts of K~ leave out less than 2^-25 of a term, so states keep fp32's
// precision (two: 2.3e-6 in norm, one: 1e-3); the product starts from zero in each
// chunk and is added to S in registers, rounded to nearest (the tensor cores'
// own accumulation cuts, a bias that grows with the chunks).
//
// A CTA runs one chain: a sequence (or a segment of one) of a head and DV columns
// of its state, chunk after chunk.  Warp 0 copies, 1 issues the products of the
// outputs, 2 those of the state (the lowest warps, which the schedulers prefer: all
// others wait for what these do).  Warps 4-7 look through V and make P~, a thread a
// row.  Warps 8-11: the outputs.  Warps 12-19: the state, DV / 2 columns of a row in
// a thread's registers, and K~, whose transposition ldmatrix and the 16-lane stores
// to TMEM make.  The gates' sums of each (chunk, head) are a record in the workspace
// (kda_lin_tc.cuh), made before: as a role of their own they took the longest.
//
// What it takes (a copy reaches 6.8 TB/s): 8,192 tokens of 32 heads of 128 x 128 in
// 124 us, of which the plan 11, the first pass 46, the joining of its states 8 and the second
// pass 67, each traced by itself; eight prompts of 1,024 to 32,768 tokens in 1.39 ms, 4.1 TB/s.
// An SM does a chunk in 3.9 to 4.6 us there, against 2.9 of HBM for its 128 KB at an
// SM's share; what is beyond that is 256 chains that 152 SMs cannot share evenly.  (Of
// these the third part of K~ takes 15 us and 80 us, 2^M 1.5 and 18.)  64 columns a chain take
// 3.5 us a chunk all the same: then a chunk's chain of waits -- products, state, operand, products, outputs --
// bounds it, one chain an SM.
//
// Roles run side by side on the schedulers' small instruction caches: unrolled ones of
// 140 KB together issued an instruction in 6 to 10 cycles.  What waits for shared
// memory or TMEM is unrolled as far as its latency asks, the rest is not.
//
// Shared memory is what an SM runs short of: its copies, the MMAs' operands and the
// threads' accesses are 480 KB a chunk at 128 x 128 (3,750 cycles at 128 bytes each)
// beside the 5,500 that HBM takes for the chunk's 128 KB.  Hence A from TMEM wherever
// a thread has to rewrite the operand anyway, and the outputs go through the value
// tile, which is needed again last.
//
// Values that are not finite.  P~ is exactly 0 at later tokens, which would
// still turn their infinities and NaN into NaN: V's are taken out in shared
// memory, and a channel is NaN in o from that token on, and in the state.  Rows
// of V and K~ behind the sequence are zeroed.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "kda_lin_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int C = kLinChunk;
constexpr int kThreads = 640;
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
  static constexpr uint32_t kBytes = kTail + 3 * 1024;
  static constexpr int kSCols = MB == 1 ? DV / 2 : DV;     // columns of a state thread
  // K~ goes through TMEM a half or a quarter of a chunk of one row tile at a time, in two
  // places where there is room: one is made while the other is multiplied
  static constexpr int kTok = DK <= 128 && DV <= 64 ? C / 2 : C / 4, kPhases = C / kTok * MB, kKBuf = MB == 1 ? 2 : 1;
  static constexpr int kKStep = 24, kKPlace = kTok / 16 * kKStep;  // TMEM columns of 16 tokens' three parts, of a place
  // TMEM columns: P (P~ over its first half, Q~ over its second or behind it), O, K~^T V, K~
  static constexpr int tP = 0, tQ = DK <= 128 ? 64 : C, tO = DK <= 128 ? C : C + DK / 2, tKV = tO + DV,
                       tK = tKV + MB * DV;
  static_assert(tK + kKBuf * kKPlace <= (int)kTmemCols && kStages >= 1 && kBytes <= 232448, "fits an SM");
};

struct Tail {
  uint64_t q_full[4], k_full[4], v_full[4], v_ready[4], q_empty[4], k_empty[4], v_done[4], v_empty[4];
  uint64_t p_full, o_full, kv_full[2];                     // committed by the MMA warps
  uint64_t s_ready[2], p_ready, k_ready[2], o_free[2], g_full[2], g_free[2], drain[2];  // [2]: chunks in turn, k_ready phases
  uint32_t dead, tmem;
  int32_t poisoned;       // the CTA's chain that nan_from speaks of, -1: none so far
  int32_t scaled_q;       // the chunk is strong, for the MMAs
  LinItem only;           // the CTA's chain where there is no plan
  int32_t num_items, local;  // local: the CTA's chain leaves its end state alone
  alignas(16) LinGateHead gates[2];  // the records of two chunks
  // per channel the first token with a value that is not finite in the latest chain
  // that had one, counted through the CTA's chunks
  uint32_t nan_from[128];
};
static_assert(sizeof(Tail) <= 3 * 1024 && offsetof(Tail, gates) % 16 == 0, "tail block");

// The CTA's i-th chain, for every role alike
__device__ __forceinline__ bool chain_at(const LinParams& p, const LinTcArgs& a, const Tail* b, int i, LinItem* ch) {
  if (!a.items) {
    *ch = b->only;
    return i == 0 && ch->len >= 0;
  }
  const uint32_t g = gridDim.x, c = blockIdx.x, w = (uint32_t)i * g + ((i & 1) ? g - 1 - c : c);  // (see nth_item)
  if (w >= (uint32_t)b->num_items) return false;
  const uint32_t per = (uint32_t)(p.H * a.tiles), pair = w / per, r = w - pair * per;
  *ch = a.items[pair];
  ch->head = (int32_t)(r >> a.tile_shift);
  ch->tile = (int32_t)(r & ((1u << a.tile_shift) - 1));
  return true;
}
// Without a plan CTA b takes chain b of sequence, head, tile (len -1: skipped)
__device__ __forceinline__ LinItem own_chain(const LinParams& p, const LinTcArgs& a, int64_t* sum) {
  const int per = p.H * a.tiles, s = (int)(blockIdx.x / per), r = (int)(blockIdx.x % per);
  const LinSeq seq = lin_seq(p, s);
  const int64_t rec = seq_records(p, s, kThreads, sum), chunks = (seq.len + C - 1) / C;
  // (sequences that overlap between malformed ones may have more chunks than there are records)
  const bool ok = seq.ok && rec + chunks <= a.max_records;
  const int32_t flag = seq.ok && !ok ? kFlagBadSeqlens : seq.flag;
  if (flag && r == 0 && threadIdx.x == 0) attn_flag(p.status, flag);
  const int row = -2 - seq.slot;
  return LinItem{(int32_t)seq.tok0, ok ? (int32_t)seq.len : -1, r / a.tiles, r % a.tiles, p.state_in ? row : -1,
                 p.state_out ? row : -1, (int32_t)rec, 1};
}
// Waits for `parity` of `bar`, for a second of an SM's fastest clock at most; false, with
// *dead set, once that is over.  Few instructions, as 20 warps do it (a time limit of
// try_wait's own makes the compiler sleep between polls, and wake late).
constexpr uint32_t kWaitClocks = 2070000000u;
__device__ __forceinline__ bool mbar_hold(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 t, u;\n\t"
      "mov.u32 t, %%clock;\n"
      "WAIT_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE_%=;\n\t"
      "mov.u32 u, %%clock;\n\t"
      "sub.u32 u, u, t;\n\t"
      "setp.lt.u32 q, u, %3;\n\t"
      "@q bra WAIT_%=;\n"
      "DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity), "n"(kWaitClocks)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  if (mbar_hold(bar, parity)) return true;
  *reinterpret_cast<volatile uint32_t*>(dead) = 1;
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  if (__all_sync(0xffffffffu, mbar_hold(bar, parity))) return true;
  *reinterpret_cast<volatile uint32_t*>(dead) = 1;
  return false;
}
// Whether token `token` >= 0 of a chain has one before or at it; n: the CTA's chunks before the chain
__device__ __forceinline__ bool nan_at(const Tail* b, int channel, uint32_t n, int token) {
  const uint32_t x = reinterpret_cast<const volatile uint32_t*>(b->nan_from)[channel];
  return x >= n * C && x <= n * C + (uint32_t)token;
}
__device__ __noinline__ void nan_note(Tail* b, int channel, uint32_t n, int token) {
  uint32_t *at = &b->nan_from[channel], x = *reinterpret_cast<volatile uint32_t*>(at);
  while (x < n * C || x > n * C + (uint32_t)token) {
    const uint32_t y = atomicCAS_block(at, x, n * C + (uint32_t)token);
    if (y == x) break;
    x = y;
  }
}
// A state of the pool or the workspace
__device__ __forceinline__ int64_t state_at(const LinParams& p, int32_t place, int head) {
  return ((int64_t)(place >= 0 ? place : -2 - place) * p.H + head) * p.dk * p.dv;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ uint32_t pack2(float2 x) { return tc::pack2(x.x, x.y); }

// Four 8 x 8 blocks of bf16, transposed: the thread gets column l / 4, rows 2 (l % 4) and + 1 of each
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 lanes of TMEM, N blocks of four 32-bit columns: of each block the thread gives
// column l % 4 of lanes l / 4 and l / 4 + 8
template <int N>
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t* v) {
  static_assert(N == 2 || N == 4, "blocks");
  if constexpr (N == 4)
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  else
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(m), "r"(x), "r"(y),
               "r"(z), "r"(smem_u32(src))
               : "memory");
}
// ------------------------------------------------------------------ copies
template <int DK, int DV, bool kLocal>
__device__ void copy_role(const LinParams& p, const LinTcArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                          const CUtensorMap* mv, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  Ring<S::kStages> ring;
  uint32_t n = 0, nv = 0, nq = 0, ng = 0;  // copies of K, V, Q and gates under way
  bool ok = true;
  LinItem ch;
  for (int i = 0; ok && chain_at(p, a, b, i, &ch); ++i) {
    const int kh = ch.head / p.R;
    for (int t = 0; t < ch.len; t += C) {
      const uint32_t st = ring.st, g = ng & 1;
      if (!(ok = thread_wait(&b->g_free[g], ((ng >> 1) & 1) ^ 1, &b->dead))) break;
      mbar_arrive_expect_tx(&b->g_full[g], sizeof(LinGateHead));
      bulk_g2s(&b->gates[g], &a.records[((int64_t)ch.rec + t / C) * p.H + ch.head].head, sizeof(LinGateHead), &b->g_full[g]);
      ++ng;
      if (!(ok = thread_wait(&b->k_empty[st], ring.ph ^ 1, &b->dead))) break;
      mbar_arrive_expect_tx(&b->k_full[st], S::kQK);
#pragma unroll
      for (int c = 0; c < DK / 64; ++c)
        tma_3d(sm + S::kK + st * S::kQK + c * kBlock, mk, 64 * c, kh, ch.tok0 + t, &b->k_full[st]);
      ++n;
      if (!(ok = thread_wait(&b->v_empty[st], ring.ph ^ 1, &b->dead))) break;
      mbar_arrive_expect_tx(&b->v_full[st], S::kVb);
#pragma unroll
      for (int c = 0; c < DV / 64; ++c)
        tma_3d(sm + S::kV + st * S::kVb + c * kBlock, mv, ch.tile * DV + 64 * c, ch.head, ch.tok0 + t, &b->v_full[st]);
      ++nv;
      if (!kLocal) {
        if (!(ok = thread_wait(&b->q_empty[st], ring.ph ^ 1, &b->dead))) break;
        mbar_arrive_expect_tx(&b->q_full[st], S::kQK);
#pragma unroll
        for (int c = 0; c < DK / 64; ++c)
          tma_3d(sm + st * S::kQK + c * kBlock, mq, 64 * c, kh, ch.tok0 + t, &b->q_full[st]);
        ++nq;
      }
      ring.next();
    }
  }
  // no copy of its own is in flight when a CTA that gave up exits
  if (!ok) {
    auto drain = [&](uint64_t* full, uint32_t count, uint32_t stages) {
      for (uint32_t k = count > stages ? count - stages : 0; k < count; ++k)
        mbar_wait(&full[k % stages], (k / stages) & 1, kWaitLimitNs);
    };
    drain(b->k_full, n, S::kStages);
    drain(b->v_full, nv, S::kStages);
    drain(b->q_full, nq, S::kStages);
    drain(b->g_full, ng, 2);
  }
}

// ------------------------------------------------------------------ MMAs
// The products of the outputs: Q K^T, then P~ V and Q~ S over it.  P's columns take
// the next chunk once both have been issued: an issuer's MMAs execute in order.
template <int DK, int DV>
__device__ void mma_out_role(const LinParams& p, const LinTcArgs& a, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  const uint32_t tmem = __shfl_sync(0xffffffffu, b->tmem, 0);
  constexpr uint32_t id_qk = idesc_bf16(C, C), id_n = idesc_bf16(C, DV, 0, 1);
  // K-major Q and K; V and S by rows of the contraction
  const uint64_t q0 = sdesc_sw128(smem_u32(sm), 16, 1024), k0 = sdesc_sw128(smem_u32(sm + S::kK), 16, 1024),
                 v0 = sdesc_sw128(smem_u32(sm + S::kV), kBlock, 1024),
                 s0 = sdesc_sw128(smem_u32(sm + S::kS), DK * 128, 1024);
  const bool issue = elect_one();
  uint32_t n = 0;
  Ring<S::kStages> ring;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait(bar, parity, &b->dead);
  };
  bool ok = true;
  LinItem ch;
  for (int i = 0; ok && chain_at(p, a, b, i, &ch); ++i) {
    for (int t = 0; t < ch.len; t += C, ++n) {
      if (!(ok = wait(&b->k_full[ring.st], ring.ph)) || !(ok = wait(&b->q_full[ring.st], ring.ph))) break;
      fence_after_sync();
      if (issue) {
        const uint64_t qd = q0 + (uint64_t)(ring.st * (S::kQK >> 4)), kd = k0 + (uint64_t)(ring.st * (S::kQK >> 4));
#pragma unroll 1
        for (int s = 0; s < DK / 16; ++s) {
          const uint32_t off = ((s / 4) * kBlock + (s % 4) * 32) >> 4;
          mma_bf16(tmem + S::tP, qd + off, kd + off, id_qk, s > 0);
        }
        mma_commit(&b->p_full);
        mma_commit(&b->k_empty[ring.st]);
      }
      // the outputs of the chunk before have been read
      if (n > 0 && !(ok = wait(&b->o_free[(n - 1) & 1], ((n - 1) >> 1) & 1))) break;
      if (!(ok = wait(&b->v_ready[ring.st], ring.ph)) || !(ok = wait(&b->p_ready, n & 1))) break;
      fence_after_sync();
      if (issue) {
        const uint64_t vd = v0 + (uint64_t)(ring.st * (S::kVb >> 4));
#pragma unroll 1
        for (int s = 0; s < C / 16; ++s)
          mma_bf16_ts(tmem + S::tO, tmem + S::tP + s * 8, vd + (uint64_t)(s * (2048 >> 4)), id_n, s > 0);
        mma_commit(&b->v_done[ring.st]);
      }
      if (!(ok = wait(&b->s_ready[n & 1], (n >> 1) & 1))) break;
      fence_after_sync();
      if (issue) {
        if (t > 0 || ch.from != -1) {
          const bool scaled = *reinterpret_cast<volatile int32_t*>(&b->scaled_q) != 0;
          const uint64_t qd = q0 + (uint64_t)(ring.st * (S::kQK >> 4));
#pragma unroll 1
          for (int s = 0; s < DK / 16; ++s) {
            const uint64_t sd = s0 + (uint64_t)(s * (2048 >> 4));
            if (scaled) mma_bf16_ts(tmem + S::tO, tmem + S::tQ + s * 8, sd, id_n, 1);
            else mma_bf16(tmem + S::tO, qd + (((s / 4) * kBlock + (s % 4) * 32) >> 4), sd, id_n, 1);
          }
        }
        mma_commit(&b->o_full);
        mma_commit(&b->q_empty[ring.st]);
      }
      ring.next();
    }
  }
  // no MMA and no arrival of one is left in flight
  if (issue) mma_commit(&b->drain[0]);
  mbar_wait(&b->drain[0], 0, kWaitLimitNs);
}

// Those of the state: K~^T V from zero, the parts of K~ in turn, smallest first
template <int DK, int DV, bool kLocal>
__device__ void mma_state_role(const LinParams& p, const LinTcArgs& a, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  const uint32_t tmem = __shfl_sync(0xffffffffu, b->tmem, 0);
  constexpr uint32_t id_n = idesc_bf16(C, DV, 0, 1);
  const uint64_t v0 = sdesc_sw128(smem_u32(sm + S::kV), kBlock, 1024);
  const bool issue = elect_one();
  uint32_t n = 0;  // phases
  Ring<S::kStages> ring;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait(bar, parity, &b->dead);
  };
  bool ok = true;
  LinItem ch;
  for (int i = 0; ok && chain_at(p, a, b, i, &ch); ++i) {
    for (int t = 0; ok && t < ch.len; t += C) {
      const uint64_t vd = v0 + (uint64_t)(ring.st * (S::kVb >> 4));
      if (!(ok = wait(&b->v_ready[ring.st], ring.ph))) break;
#pragma unroll 1
      for (int ph = 0; ph < S::kPhases; ++ph, ++n) {
        if (!(ok = wait(&b->k_ready[n & 1], (n >> 1) & 1))) break;
        fence_after_sync();
        if (issue) {
          constexpr int kPer = C / S::kTok;
          const int tok = ph % kPer * S::kTok;
          const uint32_t buf = tmem + S::tK + (n & (S::kKBuf - 1)) * S::kKPlace;
#pragma unroll 1
          for (int s = 0; s < S::kTok / 16; ++s) {
            const uint64_t vs = vd + (uint64_t)((tok / 16 + s) * (2048 >> 4));
            const uint32_t to = tmem + S::tKV + ph / kPer * DV;
            mma_bf16_ts(to, buf + s * S::kKStep + 16, vs, id_n, tok > 0 || s > 0);
            mma_bf16_ts(to, buf + s * S::kKStep + 8, vs, id_n, 1);
            mma_bf16_ts(to, buf + s * S::kKStep, vs, id_n, 1);
          }
          mma_commit(&b->kv_full[n & 1]);
          if (ph + 1 == S::kPhases) mma_commit(kLocal ? &b->v_empty[ring.st] : &b->v_done[ring.st]);
        }
      }
      ring.next();
    }
  }
  if (issue) mma_commit(&b->drain[1]);
  mbar_wait(&b->drain[1], 0, kWaitLimitNs);
}

// ------------------------------------------------------------------ values, P~ and Q~
// V before the products read it: rows behind the sequence to zero, values that are
// not finite out (r: the thread's row of the tile).
// These are noted once nothing of an earlier chain asks for its own.
template <int DK, int DV, bool kLocal>
__device__ __forceinline__ bool look_through(char* vt, int r, int live, int chain, int token, uint32_t n, Tail* b) {
  using S = Shape<DK, DV>;
  constexpr int P = DV / 8;
  uint32_t seen = 0;
  if (r >= live) {
#pragma unroll 1
    for (int c = 0; c < P; ++c) *reinterpret_cast<uint4*>(vt + sw_off(r, c, kBlock)) = make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll 4
    for (int c = 0; c < P; ++c) seen |= exponents_full(*reinterpret_cast<const uint4*>(vt + sw_off(r, c, kBlock)));
  }
  if (__any_sync(0xffffffffu, (seen & 0x80008000u) != 0)) {
    // A note of this chain may take the place of one of an earlier chain: not before all that
    // asks for that is over, the outputs of the chunk before being read and the states' warps
    // being in this chunk.  A wait by parity holds only where the phase before is known to be
    // over and the next one is not.  p_full of the chunk before (weight_role) says so of s_ready
    // two chunks back and of o_free three back, hence two barriers of each in turn; s_ready of
    // the chunk before then says so of k_ready.  (A CTA whose chain leaves its end state alone
    // has no earlier one.)
    if (!kLocal) {
      const uint32_t m = n - 1;
      if (n > 0 && (!warp_wait(&b->o_free[m & 1], (m >> 1) & 1, &b->dead) ||
                    !warp_wait(&b->s_ready[m & 1], (m >> 1) & 1, &b->dead)))
        return false;
      if (!warp_wait(&b->k_ready[0], (n * S::kPhases >> 1) & 1, &b->dead)) return false;
    }
    if (seen & 0x80008000u) {
#pragma unroll 1
      for (int c = 0; c < P; ++c) {
        uint4* at = reinterpret_cast<uint4*>(vt + sw_off(r, c, kBlock));
        const uint4 z = *at;
        const uint32_t bad = nonfinite8(z);
#pragma unroll 1
        for (int e = 0; e < 8; ++e)
          if (bad >> e & 1)
            nan_note(b, 8 * c + e, n - token / C, token);
        *at = make_uint4(finite_only(z.x), finite_only(z.y), finite_only(z.z), finite_only(z.w));
      }
      *reinterpret_cast<volatile int32_t*>(&b->poisoned) = chain;
    }
  }
  return true;
}

template <int DK, int DV, bool kLocal>
__device__ void weight_role(const LinParams& p, const LinTcArgs& a, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  const int warp = (threadIdx.x >> 5) - 4, lane = threadIdx.x & 31, row = 32 * warp + lane;
  const uint32_t lanes = b->tmem + ((uint32_t)(32 * warp) << 16), tp = lanes + S::tP;
  uint32_t* dead = &b->dead;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait(bar, parity, dead);
  };
  uint32_t n = 0;
  Ring<S::kStages> ring;
  LinItem ch;
  for (int i = 0; chain_at(p, a, b, i, &ch); ++i) {
    for (int t = 0; t < ch.len; t += C, ++n) {
      if (!wait(&b->v_full[ring.st], ring.ph)) return;
      if (!look_through<DK, DV, kLocal>(sm + S::kV + ring.st * S::kVb, row, min(C, ch.len - t), i, t + row, n, b)) return;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->v_ready[ring.st]);
      if (kLocal) {
        ring.next();
        continue;
      }
      const LinGateHead& gh = b->gates[n & 1];
      if (!wait(&b->g_full[n & 1], (n >> 1) & 1) || !wait(&b->p_full, n & 1)) return;
      fence_after_sync();
      const bool strong = gh.strong != 0;
      if (row == 0) b->scaled_q = strong;
      if (!strong) {
        // 2^{M - G_j} P_ij for j <= i; 64 columns at a time, over columns that have been read
#pragma unroll 1
        for (int c = 0; c < C; c += 64) {
          uint32_t pk[32];
          if (c <= 32 * warp) {
            float x[64];
            tmem_ld32(tp + c, x);
            tmem_ld32(tp + c + 32, x + 32);
            tmem_ld_wait();
            const int last = row - c;
#pragma unroll
            for (int u = 0; u < 64; u += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&gh.col[c + u]);
              const float2 y = mul2(make_float2(x[u], x[u + 1]), make_float2(f.x, f.y)),
                           z = mul2(make_float2(x[u + 2], x[u + 3]), make_float2(f.z, f.w));
              pk[u / 2] = tc::pack2(last >= u ? y.x : 0.f, last >= u + 1 ? y.y : 0.f);
              pk[u / 2 + 1] = tc::pack2(last >= u + 2 ? z.x : 0.f, last >= u + 3 ? z.y : 0.f);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 32; ++u) pk[u] = 0;
          }
          tmem_st32(tp + c / 2, pk);
        }
      } else {
        // 2^{G_i - G_j}.  For an earlier block of 32 tokens as 2^{G_i - G_e} 2^{G_e - G_j},
        // e the block's last token
        const float* g32 = a.records[((int64_t)ch.rec + t / C) * p.H + ch.head].row;
        const float gi = g32[row];
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) pk[u] = 0;
          if (c <= warp) {
            float since = gi;
#pragma unroll 1
            for (int y = c + 1; y < warp; ++y) since += gh.block[y];
            const float back = exp2_fast(since);
            float x[32];
            tmem_ld32(tp + 32 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 32; u += 2) {
              float f[2];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int j = 32 * c + u + z;
                f[z] = c < warp ? back * gh.col[j] : exp2_fast(gi - g32[j]);
                x[u + z] = j <= row ? x[u + z] * f[z] : 0.f;
              }
              pk[u / 2] = tc::pack2(x[u], x[u + 1]);
            }
          }
          tmem_st16(tp + 16 * c, reinterpret_cast<const float*>(pk));
        }
        // 2^{G_i} q_i
        if (!wait(&b->q_full[ring.st], ring.ph)) return;
        const char* qt = sm + ring.st * S::kQK;
        float since = gi;
#pragma unroll 1
        for (int y = 0; y < warp; ++y) since += gh.block[y];
        const float f = exp2f(since);
        const float2 f2 = make_float2(f, f);
        auto part = [&](uint32_t q2) { return pack2(mul2(make_float2(bf_lo(q2), bf_hi(q2)), f2)); };
#pragma unroll 1
        for (int c = 0; c < DK / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(qt + sw_off(row, 4 * c + u, kBlock));
            pk[4 * u] = part(q4.x);
            pk[4 * u + 1] = part(q4.y);
            pk[4 * u + 2] = part(q4.z);
            pk[4 * u + 3] = part(q4.w);
          }
          tmem_st16(lanes + S::tQ + 16 * c, reinterpret_cast<const float*>(pk));
        }
      }
      tmem_st_wait();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&b->p_ready);
        mbar_arrive(&b->g_free[n & 1]);
      }
      ring.next();
    }
  }
}

// ------------------------------------------------------------------ outputs
template <int DK, int DV>
__device__ void out_role(const LinParams& p, const LinTcArgs& a, const CUtensorMap* mo, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  const int warp = (threadIdx.x >> 5) - 8, lane = threadIdx.x & 31, row = 32 * warp + lane;
  const uint32_t to = b->tmem + ((uint32_t)(32 * warp) << 16) + S::tO;
  uint32_t n = 0;
  Ring<S::kStages> ring;
  LinItem ch;
  for (int i = 0; chain_at(p, a, b, i, &ch); ++i) {
    const int width = min(DV, p.dv - ch.tile * DV);
    const int64_t stride = (int64_t)p.H * p.dv;
    const LinGates* rec = a.records + (int64_t)ch.rec * p.H + ch.head;
    for (int t = 0; t < ch.len; t += C, rec += p.H) {
      const float own = rec->row[row];
      const int32_t strong = rec->head.strong;
      char* vt = sm + S::kV + ring.st * S::kVb;
      if (!warp_wait(&b->o_full, n & 1, &b->dead)) return;
      fence_after_sync();
      const int live = min(C, ch.len - t) - 32 * warp;  // rows of the warp that are tokens
      const bool poisoned = __any_sync(0xffffffffu, *reinterpret_cast<volatile int32_t*>(&b->poisoned) == i);
      const float f = p.scale * (strong ? 1.f : own);
      const float2 f2 = make_float2(f, f);
      // Through the warp's rows of the value tile, once no product reads it any more
      if (!warp_wait(&b->v_done[ring.st], ring.ph, &b->dead)) return;
#pragma unroll 1
      for (int c = 0; c < DV; c += 64) {
        float x[64];
        tmem_ld32(to + c, x);
        tmem_ld32(to + c + 32, x + 32);
        tmem_ld_wait();
        if (c + 64 == DV && !poisoned) {
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->o_free[n & 1]);
        }
#pragma unroll
        for (int u = 0; u < 64; u += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) pk[z] = pack2(mul2(make_float2(x[u + 2 * z], x[u + 2 * z + 1]), f2));
          *reinterpret_cast<uint4*>(vt + sw_off(row, (c + u) / 8, kBlock)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      if (poisoned) {
#pragma unroll 1
        for (int u = 0; u < DV; ++u)
          if (nan_at(b, u, n - t / C, t + row))
            *reinterpret_cast<uint16_t*>(vt + sw_off(row, u / 8, kBlock) + 2 * (u % 8)) = 0x7fff;
        // (only now: then the next chunk's notes may take the place of these)
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->o_free[n & 1]);
      }
      fence_async_smem();
      __syncwarp();
      if (live >= 32) {
        // 32 rows of 64 channels a copy (stores of the threads took 2,700 cycles a chunk)
        if (lane == 0) {
#pragma unroll
          for (int c = 0; c < DV; c += 64)
            if (c < width)
              tma_store_3d(mo, vt + c / 64 * kBlock + warp * 4096, ch.tile * DV + c, ch.head, ch.tok0 + t + 32 * warp);
          bulk_commit();
          bulk_wait_read_all();
        }
      } else {
        const int piece = lane & 7, r0 = lane >> 3;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) +
                           ((int64_t)(ch.tok0 + t + 32 * warp + r0) * p.H + ch.head) * p.dv + ch.tile * DV + 8 * piece;
#pragma unroll 1
        for (int r = r0; r < live; r += 4, o += 4 * stride)
#pragma unroll
          for (int c = 0; c < DV; c += 64)
            if (c + 8 * piece < width)
              *reinterpret_cast<uint4*>(o + c) =
                  *reinterpret_cast<const uint4*>(vt + sw_off(32 * warp + r, c / 8 + piece, kBlock));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->v_empty[ring.st]);
      ring.next();
      ++n;
    }
  }
  if (lane == 0) bulk_wait_all();
}

// ------------------------------------------------------------------ the state
template <int DK, int DV, bool kLocal>
__device__ void state_role(const LinParams& p, const LinTcArgs& a, char* sm, Tail* b) {
  using S = Shape<DK, DV>;
  constexpr int N = S::kSCols;
  constexpr int TH = S::kTok / 2;  // tokens of K~ that a warp makes at a time, of 32 channels
  const int x = threadIdx.x - 384, lane = x & 31, quarter = (x >> 5) & 3, half = x >> 7;
  // the state: row d, columns [col, col + N)
  const int d = 32 * quarter + lane + (S::MB > 1 ? 128 * half : 0), col = S::MB > 1 ? 0 : half * N;
  const bool holds = d < DK;
  const uint32_t lanes = b->tmem + ((uint32_t)(32 * quarter) << 16), kv = lanes + S::tKV + half * N;
  uint32_t* dead = &b->dead;
  uint32_t n = 0;
  Ring<S::kStages> ring;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait(bar, parity, dead);
  };
  LinItem ch;
  for (int i = 0; chain_at(p, a, b, i, &ch); ++i) {
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
    LinDecay decay{0.f, true};
    // S <- decay S + K~^T V of the chunk before
    auto advance = [&]() -> bool {
      if (!wait(&b->kv_full[1], ((n * S::kPhases - 1) >> 1) & 1)) return false;
      fence_after_sync();
      if (holds) {
        const float one = decay.near_one ? 1.f : 0.f;
        const float2 m = make_float2(decay.m, decay.m), keep = make_float2(one, one);
#pragma unroll
        for (int c = 0; c < N; c += 32) {
          float y[32];
          tmem_ld32(kv + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 32; u += 2) {
            const float2 old = make_float2(s[c + u], s[c + u + 1]);
            const float2 z = fma2(keep, old, fma2(m, old, make_float2(y[u], y[u + 1])));
            s[c + u] = z.x;
            s[c + u + 1] = z.y;
          }
        }
      }
      fence_before_sync();
      return true;
    };
    for (int t = 0; t < ch.len; t += C, ++n) {
      const int live = min(C, ch.len - t);
      const bool has = t > 0 || ch.from != -1;
      LinDecay next;
      float lift;
      // K~ of a phase: 32 channels and TH tokens, transposed on the way to TMEM
      auto make_k = [&](int ph) {
        const int m = ph / (C / S::kTok), tok0 = ph % (C / S::kTok) * S::kTok + half * TH;
        const uint32_t kt = smem_u32(sm + S::kK + ring.st * S::kQK);
        if (32 * quarter < DK) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int ch0 = 128 * m + 32 * quarter + 16 * g;
#pragma unroll
            for (int c = 0; c < TH / 16; ++c) {
              // the tokens' keys, then the parts of K~: largest, middle, smallest
              uint32_t part[12], *key = part + 8;
              ldsm4t(key, kt + sw_off(tok0 + 16 * c + (lane & 7) + (lane >> 4) * 8, ch0 / 8 + ((lane >> 3) & 1), kBlock));
              if (live < C)  // rows behind the sequence
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const int y = tok0 + 16 * c + (u >> 1) * 8 + 2 * (lane & 3);
                  if (y >= live) key[u] = 0;
                  else if (y + 1 >= live) key[u] &= 0xffffu;
                }
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float2 w =
                    *reinterpret_cast<const float2*>(&b->gates[n & 1].w[tok0 + 16 * c + (u >> 1) * 8 + 2 * (lane & 3)]);
                const float2 f = mul2(make_float2(bf_lo(key[u]), bf_hi(key[u])), w), minus = make_float2(-1.f, -1.f);
                part[u] = pack2(f);
                const float2 rest = fma2(make_float2(bf_lo(part[u]), bf_hi(part[u])), minus, f);
                part[4 + u] = pack2(rest);
                part[8 + u] = pack2(fma2(make_float2(bf_lo(part[4 + u]), bf_hi(part[4 + u])), minus, rest));
              }
              const uint32_t at = lanes + ((uint32_t)(16 * g) << 16) + S::tK + (ph & (S::kKBuf - 1)) * S::kKPlace +
                                  (half * (TH / 16) + c) * S::kKStep;
              tmem_st_16x128<4>(at, part);
              tmem_st_16x128<2>(at + 16, part + 8);
            }
          }
          tmem_st_wait();
        }
        fence_before_sync();
      };
      auto gates = [&]() -> bool {
        if (!wait(&b->g_full[n & 1], (n >> 1) & 1) || !wait(&b->k_full[ring.st], ring.ph)) return false;
        next = lin_decay(b->gates[n & 1].total);
        lift = b->gates[n & 1].lift;
        return true;
      };
      // with two places the first quarter of K~ beside the product of the chunk before, else behind it
      if (S::kKBuf == 2) {
        if (!gates()) return;
        if (t > 0 && !wait(&b->kv_full[0], ((n * S::kPhases - 2) >> 1) & 1)) return;
        fence_after_sync();
        make_k(0);
        if (t > 0 && !advance()) return;
      } else {
        if (t > 0 && !advance()) return;
        if (!gates()) return;
        make_k(0);
      }
      decay = next;
#pragma unroll 1
      for (int ph = 0;;) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->k_ready[ph & 1]);
        if (++ph == S::kPhases) break;
        // its place, once multiplied (the second quarter's was the chunk before's last, which the state has)
        if (ph >= S::kKBuf) {
          if (!wait(&b->kv_full[(ph - S::kKBuf) & 1], ((n * S::kPhases + ph - S::kKBuf) >> 1) & 1)) return;
          fence_after_sync();
        }
        make_k(ph);
      }
      if (lane == 0) {
        mbar_arrive(&b->k_empty[ring.st]);
        mbar_arrive(&b->g_free[n & 1]);
      }
      // the state as an operand, once the product with the one before is done
      if (!kLocal) {
        if (n > 0 && !wait(&b->o_full, (n - 1) & 1)) return;
        if (has && holds) {
          char* st = sm + S::kS;
          const float2 lift2 = make_float2(lift, lift);
#pragma unroll
          for (int u = 0; u < N; u += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) pk[z] = pack2(mul2(make_float2(s[u + 2 * z], s[u + 2 * z + 1]), lift2));
            *reinterpret_cast<uint4*>(st + sw_off(d, (col + u) / 8, DK * 128)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          // (nothing of the chain precedes its first chunk)
          if (t > 0 && *reinterpret_cast<volatile int32_t*>(&b->poisoned) == i)
#pragma unroll 1
            for (int u = 0; u < N; ++u)
              if (nan_at(b, col + u, n - t / C, t - 1))
                *reinterpret_cast<uint16_t*>(st + sw_off(d, (col + u) / 8, DK * 128) + 2 * (u % 8)) = 0x7fff;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->s_ready[n & 1]);
      }
      ring.next();
    }
    if (ch.len > 0 && !advance()) return;
    if (ch.to != -1 && mine) {
      float* to = (ch.to >= 0 ? a.states : p.state_out) + state_at(p, ch.to, ch.head) + (int64_t)d * p.dv + c0;
#pragma unroll
      for (int u = 0; u < N; u += 4)
        if (c0 + u < p.dv) *reinterpret_cast<float4*>(to + u) = make_float4(s[u], s[u + 1], s[u + 2], s[u + 3]);
      if (ch.len > 0 && *reinterpret_cast<volatile int32_t*>(&b->poisoned) == i)
#pragma unroll 1
        for (int u = 0; u < N; ++u)
          if (c0 + u < p.dv && nan_at(b, col + u, n - (ch.len + C - 1) / C, ch.len - 1)) to[u] = NAN;
    }
  }
}

// kFirst: the first pass over segments, a chain a CTA, most of which leave their end states alone
template <int DK, int DV, bool kFirst>
__global__ void __launch_bounds__(kThreads, 1)
    lin_tc(const LinParams p, const LinTcArgs a, const __grid_constant__ CUtensorMap mq,
           const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
           const __grid_constant__ CUtensorMap mo) {
  using S = Shape<DK, DV>;
  extern __shared__ __align__(1024) char sm[];
  Tail* b = reinterpret_cast<Tail*>(sm + S::kTail);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      for (uint64_t* x : {&b->q_full[s], &b->k_full[s], &b->v_full[s]}) mbar_init(x, 1);
      mbar_init(&b->v_ready[s], 4);
      mbar_init(&b->q_empty[s], 1);
      mbar_init(&b->v_done[s], 2);
    }
    for (uint64_t* x : {&b->p_full, &b->o_full, &b->kv_full[0], &b->kv_full[1], &b->drain[0], &b->drain[1],
                        &b->g_full[0], &b->g_full[1]})
      mbar_init(x, 1);
    for (uint64_t* x : {&b->s_ready[0], &b->s_ready[1], &b->k_ready[0], &b->k_ready[1]}) mbar_init(x, 8);
    for (uint64_t* x : {&b->p_ready, &b->o_free[0], &b->o_free[1]}) mbar_init(x, 4);
    b->dead = 0;
    b->poisoned = -1;
    b->local = 0;
  }
  if (threadIdx.x == 32) {
    prefetch_map(&mq);
    prefetch_map(&mo);
    prefetch_map(&mk);
    prefetch_map(&mv);
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + 128) b->nan_from[threadIdx.x - 64] = ~0u;
  if (warp == 1) tmem_alloc(&b->tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  pdl_wait();  // the plan, or what came before
  if (a.items) {
    if (threadIdx.x == 0) {
      const int32_t per = p.H * a.tiles, n = *a.num_items * per;  // (lin_tc_fits)
      b->num_items = n;
      if (kFirst && (int)blockIdx.x < n) b->local = !a.items[blockIdx.x / per].outputs;
    }
  } else {
    // a chain of the CTA's own, and its records (the tiles of a head all make them, alike)
    const LinItem own = own_chain(p, a, reinterpret_cast<int64_t*>(sm));
    if (threadIdx.x == 0) b->only = own;
    for (int c = warp; c * C < own.len; c += kThreads / 32)
      make_gates(p, own.tok0, own.len, c * C, own.head, &a.records[((int64_t)own.rec + c) * p.H + own.head]);
    fence_proxy_async_global();
  }
  if (threadIdx.x == 0) {
    // what is not free for others before all who read it are done with it
    const bool local = kFirst && b->local;
    for (int s = 0; s < 4; ++s) {
      mbar_init(&b->k_empty[s], local ? 8 : 9);
      mbar_init(&b->v_empty[s], local ? 1 : 4);
    }
    for (uint64_t* x : {&b->g_free[0], &b->g_free[1]}) mbar_init(x, local ? 8 : 12);
    mbar_init_fence();
  }
  __syncthreads();
  // registers: 96 a thread at launch (640 x 96 = 61,440); 128 x (48 + 104 + 88 + 2 x 120)
  auto roles = [&](auto kind) {
    constexpr bool kLocal = decltype(kind)::value;
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
      if (warp == 0) {
        if ((threadIdx.x & 31) == 0) copy_role<DK, DV, kLocal>(p, a, &mq, &mk, &mv, sm, b);
      } else if (warp == 1) {
        if (!kLocal) mma_out_role<DK, DV>(p, a, sm, b);
      } else if (warp == 2) {
        mma_state_role<DK, DV, kLocal>(p, a, sm, b);
      }
    } else if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
      weight_role<DK, DV, kLocal>(p, a, sm, b);
    } else if (warp < 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
      if (!kLocal) out_role<DK, DV>(p, a, &mo, sm, b);
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
      state_role<DK, DV, kLocal>(p, a, sm, b);
    }
  };
  if (kFirst && b->local) roles(std::true_type{});
  else roles(std::false_type{});
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && b->dead) attn_flag(p.status, kFlagTimeout);
  if (warp == 1) tmem_dealloc(b->tmem, kTmemCols);
}

// ------------------------------------------------------------------ host
bool lin_map(CUtensorMap* m, const void* base, int64_t tokens, int heads, int d, int box_tokens) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * heads};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_tokens}, elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV>
cudaError_t launch_shape(const LinParams& p, void* ws, cudaStream_t stream) {
  using S = Shape<DK, DV>;
  CUtensorMap mq, mk, mv, mo;
  if (!lin_map(&mq, p.q, p.total_tokens, p.Hk, p.dk, C) || !lin_map(&mk, p.k, p.total_tokens, p.Hk, p.dk, C) ||
      !lin_map(&mv, p.v, p.total_tokens, p.H, p.dv, C) || !lin_map(&mo, p.o, p.total_tokens, p.H, p.dv, 32))
    return cudaErrorInvalidValue;
  char* w = static_cast<char*>(ws);
  const LinShare sh = lin_tc_share(p);
  const LinLayout L = lin_layout(p, sh);
  LinTcArgs a{};
  a.tiles = (p.dv + DV - 1) / DV;
  a.tile_shift = a.tiles == 4 ? 2 : a.tiles - 1;
  a.records = reinterpret_cast<LinGates*>(w + L.records);
  a.max_records = lin_max_records(p);
  auto run = [&](auto kernel, int64_t ctas) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
    if (e != cudaSuccess) return e;
    return launch_maybe_dependent(true, kernel, dim3((unsigned)ctas), dim3(kThreads), (size_t)S::kBytes, stream, p, a, mq,
                                  mk, mv, mo);
  };
  const int64_t per = (int64_t)p.H * a.tiles;
  if (L.direct) return run(lin_tc<DK, DV, false>, p.num_seqs * per);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const LinPlan plan = lin_plan_of(p, sh, L, ws);
  a.states = plan.states;
  if ((e = launch_lin_plan(p, plan, stream)) != cudaSuccess) return e;
  if (L.may_split) {
    a.items = plan.locals;
    a.num_items = &plan.head->locals;
    if ((e = run(lin_tc<DK, DV, true>, sh.slots / per * per)) != cudaSuccess) return e;
    if ((e = launch_lin_combine(p, plan, stream)) != cudaSuccess) return e;
  }
  a.items = plan.items;
  a.num_items = &plan.head->items;
  return run(lin_tc<DK, DV, false>, std::min<int64_t>(sms, (p.num_seqs + sh.slots / per) * per));
}

}  // namespace

// bf16 with what the tensor maps need: 16-byte aligned bases; some token
bool lin_tc_fits(const LinParams& p) {
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  return p.dt == KDA_BF16 && p.total_tokens > 0 && al16(p.q) && al16(p.k) && al16(p.v) && al16(p.o) &&
         (int64_t)p.num_seqs * p.H * 4 < INT32_MAX;
}
size_t lin_tc_workspace(const LinParams& p) { return lin_layout(p, lin_tc_share(p)).total; }
cudaError_t launch_lin_tc(const LinParams& p, void* ws, cudaStream_t stream) {
  const int w = lin_tile_width(p);
  if (p.dk > 128) return launch_shape<256, 64>(p, ws, stream);
  if (p.dk > 64) return w == 64 ? launch_shape<128, 64>(p, ws, stream) : launch_shape<128, 128>(p, ws, stream);
  return w == 64 ? launch_shape<64, 64>(p, ws, stream) : launch_shape<64, 128>(p, ws, stream);
}

}  // namespace kda
