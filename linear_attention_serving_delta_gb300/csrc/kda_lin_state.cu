// kda_lin_state.cu -- the states of the linear attention with a decay for each
// head: one token a row (decode), the states advanced along accepted tokens
// (commit), drafted tokens over the states as they are (draft).  Formulas in
// include/kda.h.
//
// Decode and commit are bound by HBM: they read every state once, write it once and do
// little else.  A CTA takes one (row, head), or a slice of a wide one, with 16-byte loads
// straight into registers, all issued before anything waits, and writes them back from
// there.  256 rows of 32 heads of 128 x 128: 158 us, 6.85 TB/s, what a copy reaches; one row
// 3.3 us, a launch.  The commit of 64 trees of 8 tokens takes 51 us, 5.3 TB/s (the path comes
// between its reads and its writes).  Their draft, which only reads, takes 36 us, 4.2 TB/s, and
// is bound by the loads that four CTAs an SM keep in flight (DRAM 50% busy); fp32 drafts go
// token by token and are bound by instructions (64 chains of 8 tokens, 16 heads of 128 x 128:
// 72 us, where bf16 takes 21).
#include "kda_lin.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDraft = KDA_LIN_MAX_DRAFT;

// A CTA's slice of a state: DK x DVS elements, a float4 of VPT for each thread
// (narrow: at most 32 columns, for calls too small to fill the GPU otherwise)
template <int DK, int DV, bool kNarrow = false, int kElems = 16384>
struct Tile {
  static constexpr int kWide = DK * DV > kElems ? kElems / DK : DV;
  static constexpr int DVS = kNarrow && kWide > 32 ? 32 : kWide;  // columns
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
template <typename T, int DK, int DV, bool kNarrow>
__global__ void __launch_bounds__(Tile<DK, DV, kNarrow>::NT) lin_decode(const LinParams p) {
  using L = Tile<DK, DV, kNarrow>;
  __shared__ float sq[DK], sk[DK];
  __shared__ __align__(16) float sv[L::DVS];
  __shared__ __align__(16) float part[L::NRG][L::DVS];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, row = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * L::DVS;
  const LinSeq seq = lin_seq(p, row);
  if (seq.flag && tid == 0 && h == 0 && c0 == 0) attn_flag(p.status, seq.flag);
  if (!seq.ok) return;
  const int cq = tid % L::QPR, rg = tid / L::QPR;
  const int64_t at = ((int64_t)seq.slot * p.H + h) * DK * DV + c0 + 4 * cq;
  float4 s[L::VPT];
#pragma unroll
  for (int i = 0; i < L::VPT; ++i)
    s[i] = *reinterpret_cast<const float4*>(p.state_in + at + (int64_t)(rg + i * L::NRG) * DV);
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
// accepted token upwards, so that no difference of far sums appears.  Every warp
// walks the path for itself, with the tokens' logarithms in its lanes; the keys
// and values of the first kBatch tokens are on their way beside the state, whether
// on the path or not (a wait for them behind the walk took a quarter of the time).
constexpr int kBatch = 16;  // tokens in shared memory at a time

// (slices of 32 KB: with 64 KB the state left too few registers for the rest)
template <int DK, int DV>
using CommitTile = Tile<DK, DV, false, 8192>;
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(CommitTile<DK, DV>::NT, 4) lin_commit(const LinParams p) {
  using L = CommitTile<DK, DV>;
  constexpr int kB = DK == 256 ? kBatch / 2 : kBatch;
  __shared__ float sk[kB][DK];
  __shared__ __align__(16) float sv[kB][L::DVS];
  __shared__ float la[kMaxDraft];
  __shared__ int8_t par[kMaxDraft];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, h = blockIdx.y, c0 = blockIdx.z * L::DVS;
  const int a = p.last[blockIdx.x];
  const LinSeq seq = lin_seq(p, blockIdx.x);
  const bool first = tid == 0 && h == 0 && c0 == 0;
  if (seq.flag && first) attn_flag(p.status, seq.flag);
  if (!seq.ok) return;
  const int n = (int)seq.len;
  static_assert(L::NT >= kMaxDraft, "a thread a token");
  int parent = tid - 1;
  float gate = 0.f;
  if (tid < n) {
    if (p.parents) parent = p.parents[seq.tok0 + tid];
    gate = lin_gate<T>(p, seq.tok0 + tid, h);
  }
  const int cq = tid % L::QPR, rg = tid / L::QPR;
  const int64_t at = ((int64_t)seq.slot * p.H + h) * DK * DV + c0 + 4 * cq;
  float4 s[L::VPT];
  const bool moves = a >= -1 && a < n && !(a < 0 && p.state_in == p.state_out);
  if (moves)
#pragma unroll
    for (int i = 0; i < L::VPT; ++i)
      s[i] = *reinterpret_cast<const float4*>(p.state_in + at + (int64_t)(rg + i * L::NRG) * DV);
  auto fetch = [&](int b) {  // tokens b .. b + kB - 1 up to the accepted one
    const int m = min(kB, a + 1 - b);
    for (int i = tid; i < m * DK; i += L::NT)
      sk[i / DK][i % DK] = ld_in(static_cast<const T*>(p.k), ((seq.tok0 + b + i / DK) * p.Hk + h / p.R) * DK + i % DK);
    for (int i = tid; i < m * L::DVS; i += L::NT)
      sv[i / L::DVS][i % L::DVS] =
          ld_in(static_cast<const T*>(p.v), ((seq.tok0 + b + i / L::DVS) * p.H + h) * DV + c0 + i % L::DVS);
  };
  if (moves) fetch(0);
  if (tid < n) {
    la[tid] = lin_log2_alpha(p, gate, h);
    par[tid] = (int8_t)parent;
  }
  if (!__syncthreads_and(parent >= -1 && parent < tid || tid >= n) || a < -1 || a >= n) {
    if (first) attn_flag(p.status, kFlagBadCache);
    return;
  }
  if (!moves) return;
  // the path, and of the lane's tokens (lane, lane + 32) the sum over what follows them
  const float l0 = lane <= a ? la[lane] : 0.f, l1 = lane + 32 <= a ? la[lane + 32] : 0.f;
  unsigned long long path = 0;
  float sum = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll 1
  for (int j = a; j >= 0; j = par[j]) {
    path |= 1ull << j;
    if (lane == j) w0 = sum;
    if (lane + 32 == j) w1 = sum;
    sum += __shfl_sync(0xffffffffu, j < 32 ? l0 : l1, j & 31);
  }
  w0 = exp2f(w0);
  w1 = exp2f(w1);
  if (a >= 0) decay_all(lin_decay(sum), s);
  for (int b = 0; b <= a; b += kB) {
    if (b > 0) {
      if (!(path >> b & ((1ull << kB) - 1))) continue;
      __syncthreads();
      fetch(b);
      __syncthreads();
    }
#pragma unroll 1
    for (unsigned long long left = path >> b & ((1ull << kB) - 1); left; left &= left - 1) {
      const int j = __ffsll((long long)left) - 1;
      const float w = __shfl_sync(0xffffffffu, b + j < 32 ? w0 : w1, (b + j) & 31);
      const float4 v4 = mul4(w, *reinterpret_cast<const float4*>(&sv[j][4 * cq]));
#pragma unroll
      for (int i = 0; i < L::VPT; ++i) s[i] = fma4(sk[j][rg + i * L::NRG], v4, s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < L::VPT; ++i) *reinterpret_cast<float4*>(p.state_out + at + (int64_t)(rg + i * L::NRG) * DV) = s[i];
}

// Draft, bf16.  A CTA per (request, head), a warp per 32 columns of the state, on
// mma.sync: up to MT tiles of 16 tokens as rows, so a 128-row tcgen05 tile would be
// mostly padding, and the state is read once either way -- the kernel is bound by it.
//
// A product's contraction may run over its index in any order, so the fragments take
// whole 16-byte loads: of a block of 16 key channels the thread's four slots are
// channels 4 (l % 4) + 0..3, and of a warp's 32 columns column n of tile j is 4 n + j.
// States are rounded to bf16 on the way; o = 2^{G_i} (Q S) in fp32, then + (weights) V
// with the weights 2^{G_i - G_j} q.k of the token's path, 0 elsewhere, rounded to
// bf16.  Values that are not finite are taken out before they meet a weight of 0
// and make NaN of their channel in the tokens whose path holds them.
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ bool finite2(uint32_t w) { return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u; }

// Ancestors (itself included) and sums of log2 alpha along the path of every token
struct Tree {
  unsigned long long path[kMaxDraft];
  LogSum G[kMaxDraft];
  int8_t par[kMaxDraft];
};
constexpr int kPer = kMaxDraft / 32;  // tokens of a thread, at most
// What a tree is made from, on its way beside the other loads
struct TreeIn {
  int32_t parent[kPer];
  float gate[kPer];
};
template <typename T>
__device__ __forceinline__ TreeIn tree_in(const LinParams& p, const LinSeq& seq, int h) {
  TreeIn in;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = threadIdx.x + u * blockDim.x;
    if (i >= seq.len) continue;
    in.parent[u] = p.parents ? p.parents[seq.tok0 + i] : i - 1;
    in.gate[u] = lin_gate<T>(p, seq.tok0 + i, h);
  }
  return in;
}
// By doubling: after round r a token knows the 2^r nearest of its path.  For the whole
// CTA; false if a parent is malformed.
__device__ __forceinline__ bool make_tree(const LinParams& p, const LinSeq& seq, const TreeIn& in, int h, Tree* t) {
  const int n = (int)seq.len;
  bool good = true;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = threadIdx.x + u * blockDim.x;
    if (i >= n) continue;
    good = good && in.parent[u] >= -1 && in.parent[u] < i;
    t->par[i] = (int8_t)in.parent[u];
    t->path[i] = 1ull << i;
    t->G[i] = log_sum(lin_log2_alpha(p, in.gate[u], h));
  }
  if (!__syncthreads_and(good)) return false;
  for (int d = 1; d < n; d *= 2) {
    unsigned long long path[kPer];
    LogSum G[kPer];
    int8_t up[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = threadIdx.x + u * blockDim.x;
      if (i >= n) continue;
      const int y = t->par[i];
      path[u] = t->path[i];
      G[u] = t->G[i];
      up[u] = (int8_t)y;
      if (y >= 0) {
        path[u] |= t->path[y];
        G[u] = G[u] + t->G[y];
        up[u] = t->par[y];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = threadIdx.x + u * blockDim.x;
      if (i >= n) continue;
      t->path[i] = path[u];
      t->G[i] = G[u];
      t->par[i] = up[u];
    }
    __syncthreads();
  }
  return true;
}

// 16 bytes from global to shared memory, or zeros
__device__ __forceinline__ void copy16(void* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
               "r"(there ? 16 : 0)
               : "memory");
}

// Rows of queries, keys and values in shared memory are 32 bytes apart beyond their own
// bytes: the fragments' 8-byte reads of eight rows then fall on different banks.
constexpr int kRowPad = 16;  // elements

// MT tiles of 16 tokens in MT / MW groups of warps, which all read the state: for calls too
// small to fill the GPU, where the products one after the other are what takes the time.
template <int DK, int MT, int MW>
__global__ void __launch_bounds__(256, DK <= 128 && MW == 1 ? 2 : 1)
    lin_draft_mma(const LinParams p) {
  using T = __nv_bfloat16;
  constexpr int KB = DK / 16, NB = KB < 4 ? KB : 4;
  extern __shared__ __align__(16) char dyn[];
  __shared__ Tree tree;
  __shared__ unsigned long long bad[256];  // tokens whose value is not finite, per column
  __shared__ int32_t any_bad;
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kGroups = MT / MW;
  const int lane = threadIdx.x & 31, wide = (p.dv + 31) / 32, gi = lane >> 2, ti = lane & 3;
  const int warp = (threadIdx.x >> 5) % wide, group = (threadIdx.x >> 5) / wide;
  // a warp's tile u: every second row of groups backwards, as later tiles have more to add up
  auto tile_of = [&](int u) { return u * kGroups + (u & 1 ? kGroups - 1 - group : group); };
  const int h = blockIdx.y, cb = 32 * warp + 4 * gi, co = 32 * warp + 8 * ti;  // columns: of loads, of outputs
  const LinSeq seq = lin_seq(p, blockIdx.x);
  const bool first = threadIdx.x == 0 && h == 0;
  if (seq.flag && first) attn_flag(p.status, seq.flag);
  if (!seq.ok || seq.len == 0) return;
  const int n = (int)seq.len, mt = (n + 15) / 16;
  constexpr int kPitch = DK + kRowPad;
  const int pv = p.dv + kRowPad;
  T *sq = reinterpret_cast<T*>(dyn), *sk = sq + 16 * MT * kPitch, *sv = sk + 16 * MT * kPitch;
  const float* S = p.state_in + ((int64_t)seq.slot * p.H + h) * DK * p.dv + cb;
  float4 s[NB][4];
  auto load = [&](int k0) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[b][e] = cb < p.dv && tile_of(0) < mt
                      ? *reinterpret_cast<const float4*>(S + (int64_t)(16 * (k0 + b) + 4 * ti + e) * p.dv)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load(0);
  // queries, keys and values of the request, rows behind it zero, 16 bytes at a time and
  // without a wait in between: what a call's loads wait for one after the other, a CTA
  // waits for with its state half loaded
  for (int i = threadIdx.x; i < 16 * mt * (DK / 8); i += blockDim.x) {
    const int t = i / (DK / 8), c = i % (DK / 8) * 8;
    const int64_t at = t < n ? ((seq.tok0 + t) * p.Hk + h / p.R) * DK + c : 0;
    copy16(sq + t * kPitch + c, static_cast<const T*>(p.q) + at, t < n);
    copy16(sk + t * kPitch + c, static_cast<const T*>(p.k) + at, t < n);
  }
  for (int i = threadIdx.x; i < 16 * mt * (p.dv / 8); i += blockDim.x) {
    const int t = i / (p.dv / 8), c = i % (p.dv / 8) * 8;
    const int64_t at = t < n ? ((seq.tok0 + t) * p.H + h) * p.dv + c : 0;
    copy16(sv + t * pv + c, static_cast<const T*>(p.v) + at, t < n);
  }
  const TreeIn in = tree_in<T>(p, seq, h);
  for (int i = threadIdx.x; i < p.dv; i += blockDim.x) bad[i] = 0;
  if (threadIdx.x == 0) any_bad = 0;
  if (!make_tree(p, seq, in, h, &tree)) {
    if (first) attn_flag(p.status, kFlagBadCache);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int i = threadIdx.x; i < 16 * mt * (p.dv / 8); i += blockDim.x) {  // (the thread's own copies)
    const int t = i / (p.dv / 8), c = i % (p.dv / 8) * 8;
    uint4* at = reinterpret_cast<uint4*>(sv + t * pv + c);
    const uint4 x = *at;
    if (finite2(x.x) && finite2(x.y) && finite2(x.z) && finite2(x.w)) continue;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t ones = e & 1 ? 0x7f800000u : 0x7f80u;
      if ((w[e / 2] & ones) != ones) continue;
      atomicOr(&bad[c + e], 1ull << t);
      w[e / 2] &= e & 1 ? 0xffffu : 0xffff0000u;
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
    any_bad = 1;
  }
  __syncthreads();
  const bool found = any_bad != 0;
  // four channels of a token's query or key
  auto four = [&](const T* x, int tok, int kb) {
    return *reinterpret_cast<const uint2*>(x + tok * kPitch + 16 * kb + 4 * ti);
  };
  float acc[MW][4][4];
#pragma unroll
  for (int u = 0; u < MW; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[u][j][e] = 0.f;
#pragma unroll
  for (int k0 = 0; k0 < KB; k0 += NB) {
    uint32_t b0[NB][4], b1[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      b0[b][0] = pack2(s[b][0].x, s[b][1].x);
      b1[b][0] = pack2(s[b][2].x, s[b][3].x);
      b0[b][1] = pack2(s[b][0].y, s[b][1].y);
      b1[b][1] = pack2(s[b][2].y, s[b][3].y);
      b0[b][2] = pack2(s[b][0].z, s[b][1].z);
      b1[b][2] = pack2(s[b][2].z, s[b][3].z);
      b0[b][3] = pack2(s[b][0].w, s[b][1].w);
      b1[b][3] = pack2(s[b][2].w, s[b][3].w);
    }
    if (k0 + NB < KB) load(k0 + NB);  // beside this part's products
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < MW; ++u) {
        const int m = tile_of(u);
        if (m >= mt) continue;
        const uint2 x = four(sq, 16 * m + gi, k0 + b), y = four(sq, 16 * m + gi + 8, k0 + b);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[u][j], x.x, y.x, x.y, y.y, b0[b][j], b1[b][j]);
      }
  }
#pragma unroll
  for (int um = 0; um < MW; ++um) {
    const int m = tile_of(um);
    if (m >= mt) continue;
    const int r0 = 16 * m + gi, r1 = r0 + 8;  // the thread's two tokens
    const LogSum none{0.f, 0.f};
    const LogSum g0 = r0 < n ? tree.G[r0] : none, g1 = r1 < n ? tree.G[r1] : none;
    const unsigned long long p0 = r0 < n ? tree.path[r0] : 0, p1 = r1 < n ? tree.path[r1] : 0;
    {
      const float f0 = exp2f(g0.i + g0.f), f1 = exp2f(g1.i + g1.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[um][j][0] *= f0;
        acc[um][j][1] *= f0;
        acc[um][j][2] *= f1;
        acc[um][j][3] *= f1;
      }
    }
    // sixteen earlier tokens at a time: their weights are the next product's fragments
#pragma unroll 1
    for (int t = 0; t <= m; ++t) {
      float w[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[u][e] = 0.f;
#pragma unroll 4
      for (int kb = 0; kb < KB; ++kb) {
        const uint2 x = four(sq, r0, kb), y = four(sq, r1, kb);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint2 z = four(sk, 16 * t + 8 * u + gi, kb);
          mma16816(w[u], x.x, y.x, x.y, y.y, z.x, z.y);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * t + 8 * u + 2 * ti + (e & 1);
          const bool on = ((e < 2 ? p0 : p1) >> j & 1) != 0;
          w[u][e] = on ? w[u][e] * exp2f(log_diff(e < 2 ? g0 : g1, tree.G[j])) : 0.f;
        }
      // V: rows 2 ti, + 1, + 8, + 9 of the sixteen, the thread's four columns
      uint2 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = cb < p.dv ? *reinterpret_cast<const uint2*>(sv + (16 * t + 2 * ti + (e & 1) + 8 * (e >> 1)) * pv + cb)
                         : make_uint2(0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t pick = j & 1 ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(j < 2 ? v[0].x : v[0].y, j < 2 ? v[1].x : v[1].y, pick),
                       b1 = __byte_perm(j < 2 ? v[2].x : v[2].y, j < 2 ? v[3].x : v[3].y, pick);
        mma16816(acc[um][j], pack2(w[0][0], w[0][1]), pack2(w[0][2], w[0][3]), pack2(w[1][0], w[1][1]),
                 pack2(w[1][2], w[1][3]), b0, b1);
      }
    }
    // columns co .. co + 7 of the two tokens: n = 2 ti of the tiles, then n = 2 ti + 1
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = r ? r1 : r0;
      if (i >= n || co >= p.dv) continue;
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = acc[um][j][2 * r] * p.scale;
        x[4 + j] = acc[um][j][2 * r + 1] * p.scale;
      }
      if (found)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (bad[co + j] & (r ? p1 : p0)) x[j] = NAN;
      *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + ((seq.tok0 + i) * p.H + h) * p.dv + co) =
          make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    }
  }
}

// Draft in fp32, and where the tensors are not aligned.  A CTA per (request, head, 32
// columns): the columns of the state in shared memory, a warp per token, lane = column.
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
      q[u] = 32 * u + lane < DK
                 ? ld_in(static_cast<const T*>(p.q), ((seq.tok0 + i) * p.Hk + h / p.R) * DK + 32 * u + lane)
                 : 0.f;
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
// Launched as the dependents of what is before them on the stream, as the cache's calls are
template <typename T, int DK, int DV, bool kCommit>
cudaError_t launch_state(const LinParams& p, cudaStream_t stream) {
  using L = Tile<DK, DV>;
  using N = Tile<DK, DV, true>;
  const dim3 grid((unsigned)p.num_seqs, (unsigned)p.H, DV / L::DVS), narrow(grid.x, grid.y, DV / N::DVS);
  if (kCommit) {
    using M = CommitTile<DK, DV>;
    return launch_maybe_dependent(true, lin_commit<T, DK, DV>, dim3(grid.x, grid.y, DV / M::DVS), dim3(M::NT), 0, stream, p);
  }
  // fewer CTAs than SMs (one row of 32 heads of 128 x 128: 6.1 us in whole states)
  if (N::DVS < L::DVS && (int64_t)grid.x * grid.y * grid.z < kLinSms)
    return launch_maybe_dependent(true, lin_decode<T, DK, DV, true>, narrow, dim3(N::NT), 0, stream, p);
  return launch_maybe_dependent(true, lin_decode<T, DK, DV, false>, grid, dim3(L::NT), 0, stream, p);
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

template <int DK>
cudaError_t launch_draft_mma(const LinParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.num_seqs, (unsigned)p.H);
  const int wide = (p.dv + 31) / 32;
  auto run = [&](auto kernel, int tokens, int groups) {
    const int threads = 32 * wide * groups;
    const size_t smem = (size_t)tokens * (2 * (DK + kRowPad) + p.dv + kRowPad) * sizeof(__nv_bfloat16);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e != cudaSuccess ? e : launch_maybe_dependent(true, kernel, grid, dim3(threads), smem, stream, p);
  };
  if (p.max_seqlen <= 16) return run(lin_draft_mma<DK, 1, 1>, 16, 1);
  // as many groups as eight warps allow while the CTAs are at most two an SM: nine trees of
  // 60 tokens, 32 heads of 128 x 64 21.9 -> 14.4 us, but 64 trees and 128 x 128 131 -> 168
  const bool split = (int64_t)p.num_seqs * p.H <= 2 * kLinSms;
  if (p.max_seqlen <= 32)
    return split && wide <= 4 ? run(lin_draft_mma<DK, 2, 1>, 32, 2) : run(lin_draft_mma<DK, 2, 2>, 32, 1);
  if (split && wide <= 2) return run(lin_draft_mma<DK, 4, 1>, 64, 4);
  return split && wide <= 4 ? run(lin_draft_mma<DK, 4, 2>, 64, 2) : run(lin_draft_mma<DK, 4, 4>, 64, 1);
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
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  if (p.dt == KDA_BF16 && al16(p.q) && al16(p.k) && al16(p.v) && al16(p.o)) {
    switch (p.dk) {
      case 16: return launch_draft_mma<16>(p, stream);
      case 32: return launch_draft_mma<32>(p, stream);
      case 64: return launch_draft_mma<64>(p, stream);
      case 128: return launch_draft_mma<128>(p, stream);
      case 256: return launch_draft_mma<256>(p, stream);
    }
  }
  return p.dt == KDA_BF16 ? launch_draft_t<__nv_bfloat16>(p, stream) : launch_draft_t<float>(p, stream);
}

}  // namespace kda
