// kda_lin_tc.cuh -- what the tensor-core prompts of the linear attention with a decay
// for each head share: work items, gate records, workspace.
#pragma once

#include "kda_attn_tc.cuh"
#include "kda_lin.cuh"

namespace kda {

constexpr int kLinChunk = 128;  // tokens of a chunk: the rows of a tensor-core tile

// One chain: tokens [tok0, tok0 + len) of a head's columns [tile * DV, ...).
// from, to: the state it starts from and leaves, a place of the workspace's
// states (>= 0), row -2 - x of the pool (<= -2), or none (-1).  rec: its first record.
// outputs: whether the first pass makes its outputs too.  A plan holds one for all heads
// and tiles.
struct LinItem {
  int32_t tok0, len, head, tile, from, to, rec, outputs;
};

// A sequence cut into segments, whose start states are at place, place + 1, ...
struct LinSplit {
  int32_t place, segments, rec, chunks;
};
// Segment i of n chunks cut into k: its first chunk.  The first segment is shorter, `first`
// tenths of another: the first pass makes its outputs too.
__host__ __device__ __forceinline__ int32_t lin_cut(int32_t n, int32_t k, int32_t i, int32_t first) {
  if (k == 1 || i == 0) return i == 0 ? 0 : n;
  int32_t a = n * first / (10 * (k - 1) + first);
  a = a > 1 ? a : 1;
  const int32_t rest = n - a, each = rest / (k - 1), more = rest - each * (k - 1);  // `more` have one more
  return a + (i - 1) * each + (i - 1 < more ? i - 1 : more);
}
// The chains of either pass that n chunks in segments of m give
__host__ __device__ __forceinline__ int32_t lin_chains(int32_t n, int32_t m, int32_t first) {
  if (n <= m) return 1;
  int32_t a = (int32_t)((int64_t)m * first / 10);
  a = a > 1 ? a : 1;
  return n - a > m ? (n - a - 1) / m + 1 : 1;
}

struct LinHead {
  int32_t items, locals, splits;  // entries of the lists, for one head and tile
};
// The CTAs that chains are shared out to: one an SM on the tensor cores, three on the CUDA cores
constexpr int kLinTcSlots = kLinSms, kLinSimtSlots = 3 * kLinSms;
// Segments of one sequence at most: one for each CTA of the second pass, and the first
constexpr int kLinMostSegments = kLinSimtSlots + 1;
// The fewest chunks of a segment.  One prompt of 8,192 tokens, 8 heads of 128 x 128: 86 us,
// where 16 take 121 and 4 take 70; 16 heads of 64 x 64 and 16,384 tokens: 100, 104 and 100
constexpr int kLinMinSegment = 8;
// A chunk without its outputs takes 2.3 us where one with them takes 3.9
constexpr int kLinFirst = 6;
// Up to how many tokens of a call a chain each needs no plan.  One prompt of 2,048 tokens, 32
// heads of 128 x 128: 68 us where a plan and segments take 82; of 4,096: 126 and 88.  (Two
// of 2,048 would take 70 where they take 88, but the host knows their sum alone)
constexpr int kLinDirectTokens = 2048;

// The gates of a chunk of one head, with G_i the sum of log2 alpha up to token i.  A
// chunk is weak while |G| <= kLinWeak: weights are then split as 2^{G_i - M} 2^{M - G_j}, with
// M the middle of the G, a whole number, so that neither factor is above 2^33 (2^{-G_j} by itself
// would take products from 2^64 on out of fp32) and M scales without rounding.
constexpr float kLinWeak = 64.f;
struct LinGateHead {
  float w[kLinChunk];    // 2^{G_C - G_j}
  // weak: 2^{M - G_j}; strong: 2^ of the sum over what follows the token in its block of 32
  float col[kLinChunk];
  float total;           // G_C
  int32_t strong;
  float lift;            // weak: 2^M; strong: 1
  int32_t pad;
  float block[4];        // the sums over the blocks of 32
};
struct LinGates {
  LinGateHead head;
  float row[kLinChunk];  // weak: 2^{G_i - M}; strong: the sum from the block's start on
};
static_assert(sizeof(LinGateHead) % 16 == 0 && sizeof(LinGates) % 16 == 0, "bulk copies");

struct LinTcArgs {
  const LinItem* items;    // null: CTA b takes chain b of sequence, head, tile
  const int32_t* num_items;
  float* states;           // [places][H][dk][dv]
  LinGates* records;       // [max_records][H]
  int64_t max_records;
  int32_t tiles;           // column tiles of a head: 1, 2 or 4
  int32_t tile_shift;
};

// What the plan leaves in the workspace
struct LinPlan {
  LinHead* head;
  int32_t* seq_rec;        // [N] a sequence's first record, or -1: skipped
  LinItem* items;          // costliest first
  LinItem* locals;         // the first pass's segments
  LinSplit* splits;
  int32_t tiles;           // column tiles of a head
  int32_t slots;           // CTAs that the chains are shared out to
  int32_t chunk;           // tokens of a chunk
  int32_t min_segment;     // fewest chunks of a segment
  int32_t first;           // of lin_cut
  int64_t max_records;
  int32_t may_split;
  float* states;           // [places][H][dk][dv] start states of segments
  // log2 of the decay of the segment before a place: from the records, or [places][H]
  LinGates* records;
  float* logs;
};

// How a path plans: its column tiles, CTAs, tokens of a chunk, shortest segment in
// chunks, the share of the first one, up to how many tokens its chains need no plan,
// whether it has gate records
struct LinShare {
  int32_t tiles, slots, chunk, min_segment, first, direct_tokens;
  bool records;
};
struct LinLayout {
  size_t head, seq_rec, items, locals, splits, states, records, logs, total;
  int64_t places;
  bool direct, may_split;
};
int lin_tile_width(const LinParams& p);
LinShare lin_tc_share(const LinParams& p);
LinLayout lin_layout(const LinParams& p, const LinShare& sh);
LinPlan lin_plan_of(const LinParams& p, const LinShare& sh, const LinLayout& L, void* ws);
cudaError_t launch_lin_plan(const LinParams& p, const LinPlan& a, cudaStream_t stream);
cudaError_t launch_lin_combine(const LinParams& p, const LinPlan& a, cudaStream_t stream);

// Chunks of all sequences of a well-formed call, at most
inline int64_t lin_max_records(const LinParams& p, int chunk = kLinChunk) { return p.total_tokens / chunk + p.num_seqs; }

// The chunks of the valid sequences before s, for the whole block (sum: shared, free before and after)
__device__ __forceinline__ int64_t seq_records(const LinParams& p, int s, int threads, int64_t* sum) {
  unsigned long long* at = reinterpret_cast<unsigned long long*>(sum);
  if (threadIdx.x == 0) *at = 0;
  __syncthreads();
  long long x = 0;
  for (int y = threadIdx.x; y < s; y += threads) {
    const LinSeq q = lin_seq(p, y);
    if (q.ok) x += (q.len + kLinChunk - 1) / kLinChunk;
  }
  if (x) atomicAdd_block(at, (unsigned long long)x);
  __syncthreads();
  const int64_t r = (int64_t)*at;
  tc::fence_async_smem();
  __syncthreads();
  return r;
}

// The record of the chunk at token t of a sequence of len tokens from tok0 on, by a
// warp, four neighbouring tokens a lane (bf16 gates).
__device__ __forceinline__ void make_gates(const LinParams& p, int64_t tok0, int len, int t, int head, LinGates* out) {
  const int lane = threadIdx.x & 31;
  LogSum G[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int x = t + 4 * lane + u;
    const LogSum la = log_sum(x < len ? lin_log2_alpha<__nv_bfloat16>(p, tok0 + x, head) : 0.f);
    G[u] = u == 0 ? la : G[u - 1] + la;
  }
  // within the lane's block of 32 tokens, then over the blocks
  LogSum upto = G[3];
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const LogSum y{__shfl_up_sync(0xffffffffu, upto.i, o), __shfl_up_sync(0xffffffffu, upto.f, o)};
    if ((lane & 7) >= o) upto = y + upto;
  }
  auto from = [&](LogSum v, int src) {
    return LogSum{__shfl_sync(0xffffffffu, v.i, src), __shfl_sync(0xffffffffu, v.f, src)};
  };
  const LogSum prev = from(upto, lane > 0 ? lane - 1 : 0), t0 = from(upto, 7), t1 = from(upto, 15),
               t2 = from(upto, 23), t3 = from(upto, 31), end = from(upto, lane | 7);
  LogSum before{0.f, 0.f};
  if (lane >= 8) before = t0;
  if (lane >= 16) before = before + t1;
  if (lane >= 24) before = before + t2;
  const LogSum all = (t0 + t1) + (t2 + t3);
  LogSum from_start[4];
  float w[4], col[4], row[4], low = 0.f;
  bool far = false;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if ((lane & 7) != 0) G[u] = prev + G[u];
    const LogSum x = from_start[u] = before + G[u];
    w[u] = exp2f(log_diff(all, x));
    // (a NaN is not far, nor the lowest: it leaves the tokens before it as they are)
    far |= fabsf(x.i + x.f) > kLinWeak;
    low = fminf(low, x.i + x.f);
  }
  const bool strong = __any_sync(0xffffffffu, far);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
  const float mid = strong ? 0.f : rintf(0.5f * low);
  // 2^n for whole n (NaN: 1, beside a factor that is NaN)
  auto octaves = [](float n) { return __int_as_float(((int)n + 127) << 23); };
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const LogSum x = from_start[u];
    col[u] = strong ? exp2f(log_diff(end, G[u])) : exp2f(-x.f) * octaves(mid - x.i);
    row[u] = strong ? G[u].i + G[u].f : exp2f(x.f) * octaves(x.i - mid);
  }
  reinterpret_cast<float4*>(out->head.w)[lane] = make_float4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<float4*>(out->head.col)[lane] = make_float4(col[0], col[1], col[2], col[3]);
  reinterpret_cast<float4*>(out->row)[lane] = make_float4(row[0], row[1], row[2], row[3]);
  if (lane == 0) {
    out->head.total = all.i + all.f;
    out->head.strong = strong;
    out->head.lift = octaves(mid);
  }
  if ((lane & 7) == 7) out->head.block[lane >> 3] = end.i + end.f;
}

}  // namespace kda
