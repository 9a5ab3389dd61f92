// kda_attn_rows.cu -- attention by blocks of at most 16 rows (32 in fp32): single tokens (or
// a few) over the paged cache in both types, all of fp32 with heads of 256
// channels, and calls of at most 32 rows a key head in fp32 or with 256 channels.
//
// A block's rows are those of one key head: row = token * gb + head, with gb
// = min(G, 16 or 32) of its G query heads and as many tokens (a power of two) as fit
// a block.  For single tokens that reads every cached key and value once and
// does little with them, so the kernel is a stream: bf16 is bound by HBM, fp32
// by the splitting of its operands and six products for each.
//
// The key tiles of all blocks form one line of work, sequence after sequence,
// head after head, and every CTA of a grid that fills the GPU takes an equal
// stretch of it, whatever the lengths.  A block inside one stretch is finished
// there; one that crosses stretches leaves its parts (unnormalised output,
// running maximum m and sum l, fp32) for attn_rows_join, which adds them in
// line order:  M = max m_k,  o = sum 2^(m_k - M) O_k / sum 2^(m_k - M) l_k.
//
// In a CTA one warp copies tiles into a ring (tensor-map copies, a box per
// page, 128-byte swizzle) and four warps each take a quarter of a tile's keys
// with softmax statistics of their own, joined at the end of a block.  bf16:
// 16 keys a warp on mma.sync (a 128-row tcgen05 tile would be 7/8 padding for
// single tokens, and the tensor cores wait for memory either way); the
// weights are rounded to bf16, as P V's operand.  fp32: the same with every
// operand in three bf16 parts.
//
// Measured on GB300, 32 query heads over 8 of 128 channels, bf16: one token each
// of 256 requests over 64..8191 keys 630..646 us (6.6..6.7 TB/s, the measured copy
// rate), one token over 131,072 keys 92 us (5.8 TB/s).  fp32, 64 requests over
// 64..8191 keys: 0.75 ms with 128 channels (2.6 TB/s), 1.79 ms with 256 (2.2 TB/s);
// one prompt of 4096 tokens with 256 channels 17.1 ms (16 TFLOP/s).
#include <algorithm>

#include "kda_attn_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kWarps = 4;                      // consumers
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxRows = 32;                   // most rows of a block (16, or 32 in fp32)
constexpr int kMinTiles = 1;                   // shortest stretch of a CTA
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazyLog2 = 8.f;  // how far the maximum may rise before O is rescaled

template <typename T, int DP, int R>
struct Shape {
  static constexpr int KT = sizeof(T) == 2 || DP <= 128 ? 64 : 32;  // keys of a tile
  static constexpr int NB = DP * (int)sizeof(T) / 128;     // 128-byte blocks of a row
  static constexpr uint32_t kBlock = KT * 128;
  static constexpr uint32_t kKV = 2 * NB * kBlock;         // K, then V; also the joining warps' scratch
  static constexpr uint32_t kQBlock = R * 128;      // bf16: q of a pair, with its first tile
  static constexpr uint32_t kStage = kKV + (sizeof(T) == 2 ? NB * kQBlock : 0);
  static constexpr int CTAS = kKV <= 32768 ? 2 : 1;
  static constexpr int kStages = kKV <= 8192 ? 8 : kKV <= 16384 ? 5 : 3;
  static constexpr uint32_t kQ = kStages * kStage;         // fp32: the pair's q rows, plain
  static constexpr uint32_t kQPlane = (DP + 63) / 64 * kQBlock;  // fp32: a bf16 part of q (split3)
  static constexpr uint32_t kTail = kQ + (sizeof(T) == 2 ? 0 : 3 * kQPlane);
  static constexpr uint32_t kBytes = kTail + 2048 + 1024;  // barriers; slack to align the base
};
template <typename T, int DP, int R>
constexpr bool shape_ok() {
  using S = Shape<T, DP, R>;
  return S::kKV >= kWarps * R * DP * 4                                  // the warps' outputs fit a stage
         && S::CTAS * (S::kBytes + 1024) <= 233472 && S::kBytes <= 232448;
}

// A tile in the ring, for its consumers
struct Tile {
  int32_t tok0, head0;  // packed token and query head of the block's first row
  int32_t rows, gb;     // rows of the block, query heads of a token in it
  int32_t pos0, end;    // position of its first token; keys its last one attends
  int32_t x0;           // position of the tile's first key
  int32_t first, last;  // of the block in this stretch
  int32_t slot;         // at the last tile: where the part goes, or -1 (the block is whole)
  int32_t base;         // first packed token of the sequence, or its row of the block table
  int32_t kvh;          // key head
};

// The non-finite values taken out of a block's V: the positions past its first
// token's that had some, and for those that all of its rows attend the channels
// with +inf, -inf and NaN, a bit each
struct Poison {
  int32_t from, to;
  uint32_t seen;
  uint32_t bits[3][8];
};
constexpr int kPoisonWords = sizeof(Poison) / 4;
__device__ __forceinline__ int32_t no_poison(int word) { return word == 0 ? INT32_MAX : word == 1 ? -1 : 0; }

struct Tail {
  uint64_t full[8], empty[8];
  uint64_t join[2];
  uint32_t dead;
  uint32_t pad;
  Tile tile[8];
  float2 ml[kWarps][kMaxRows];
  int64_t sum[kWarps + 1];
  int64_t found;   // where in its sequence's tiles the stretch starts
  int32_t found_at;
  Poison poison[3];  // of the CTA's k-th block, in turn
  AttnSeq found_seq;
};
static_assert(sizeof(Tail) <= 2048, "tail block");

struct RowsJoin {
  int32_t parts;  // 0: nothing to join
  int32_t tok0, head0, rows, gb;
};
struct RowsArgs {
  RowsJoin* joins;   // [grid]
  float2* ml;        // [2 grid][kMaxRows]
  float* o;          // [2 grid][kMaxRows][DP]
  int32_t box_shift; // log2 of the positions per copy
  int32_t q_shift;   // log2 of a block's tokens
  int32_t parts;     // blocks of a token's G heads
};

// a / b for a >= 0, b > 0: the quick way where both are small
__device__ __noinline__ int64_t div_large(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t div_any(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : div_large(a, b);
}

// The blocks of a sequence for one head (part): n of them, block i with
// tiles(i) = max(1, ceil((pos + (i + 1) q) / KT)) key tiles, q = 2^q_shift
// tokens each, pos the position of the first token.  (The last block may count
// a tile without keys; a block without keys still writes its zeros.)  With R =
// KT / q and d = floor((pos + KT - 1) / q) + 1 that is max(1, floor((d + i) / R)),
// and sum_{j < n} floor(j / R) = R t (t - 1) / 2 + t (n - t R) for t = floor(n / R).
template <int KT>
struct Blocks {
  int64_t n, d;
  int rs;  // log2 R
  __device__ __forceinline__ Blocks(const AttnSeq& s, int q_shift) {
    n = ((int64_t)s.len + (1 << q_shift) - 1) >> q_shift;
    d = ((s.kv_len - s.len + KT - 1) >> q_shift) + 1;
    rs = 31 - __clz(KT) - q_shift;
  }
  __device__ __forceinline__ int tiles(int64_t i) const { return (int)max((int64_t)1, (d + i) >> rs); }
  __device__ __forceinline__ int64_t sum(int64_t m) const {
    const int64_t t = m >> rs;
    return (t * (t - 1) / 2 << rs) + t * (m - (t << rs));
  }
  __device__ __forceinline__ int64_t ones() const {  // blocks before the formula passes 1
    return min(n, max((int64_t)0, ((int64_t)1 << rs) - d));
  }
  __device__ __forceinline__ int64_t total() const { return n == 1 ? tiles(0) : ones() + sum(d + n) - sum(d + ones()); }
  // the block that holds tile r of the head, and r's index in it
  __device__ void find(int64_t r, int64_t* block, int* tile) const {
    if (n == 1) {
      *block = 0;
      *tile = (int)r;
      return;
    }
    const int64_t o = ones();
    if (r < o) {
      *block = r;
      *tile = 0;
      return;
    }
    const int64_t y = r - o + sum(d + o);
    // largest t with R t (t - 1) / 2 <= y
    int64_t t = (int64_t)((1.f + sqrtf(1.f + 8.f * (float)y / (float)(1 << rs))) * 0.5f);
    if (t < 1) t = 1;
    while ((t * (t - 1) / 2 << rs) > y) --t;
    while ((t * (t + 1) / 2 << rs) <= y) ++t;
    const int64_t z = y - (t * (t - 1) / 2 << rs), m = div_any(z, t);
    *block = (t << rs) + m - d;
    *tile = (int)(z - m * t);
  }
};

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same over 8 keys, and by the number of keys
__device__ __forceinline__ void mma1688(float* d, const uint32_t* a, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(b0));
}
template <int NT>
__device__ __forceinline__ void mma_keys(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (NT == 2) mma16816(d, a, b0, b1);
  else mma1688(d, a, b0);
}
// Non-finite values among keys [key0, key0 + n) of a V tile (x0: position of the
// tile's first key) become zeros and are noted in ps (pos0: the last position that
// all rows attend).  The block's outputs get them back when they are written.
template <typename T, int NB>
__device__ __noinline__ void take_out(char* vs, uint32_t block, int key0, int n, int x0, int pos0, Poison* ps, int lane) {
  constexpr int E = 16 / (int)sizeof(T);
  int lo = INT32_MAX, hi = -1;
#pragma unroll 1
  for (int i = lane; i < n * NB * 8; i += 32) {
    const int r = key0 + i / (NB * 8);
    uint4* at = reinterpret_cast<uint4*>(vs + sw_off(r, i % (NB * 8), block));
    const uint4 x = *at;
    uint4 y;
    if constexpr (sizeof(T) == 2) {
      y = make_uint4(finite_only(x.x), finite_only(x.y), finite_only(x.z), finite_only(x.w));
    } else {
      auto keep = [](uint32_t v) { return (v & 0x7f800000u) == 0x7f800000u ? 0u : v; };
      y = make_uint4(keep(x.x), keep(x.y), keep(x.z), keep(x.w));
    }
    if (x.x == y.x && x.y == y.y && x.z == y.z && x.w == y.w) continue;
    *at = y;
    if (x0 + r > pos0) {
      lo = min(lo, x0 + r);
      hi = max(hi, x0 + r);
    } else {
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float f = E == 4 ? __uint_as_float(w[e & 3]) : e & 1 ? bf_hi(w[e / 2 & 3]) : bf_lo(w[e / 2 & 3]);
        const int ch = i % (NB * 8) * E + e;
        if ((__float_as_uint(f) & 0x7f800000u) == 0x7f800000u)
          atomicOr_block(&ps->bits[poison_kind(f)][ch >> 5], 1u << (ch & 31));
      }
    }
    *reinterpret_cast<volatile uint32_t*>(&ps->seen) = 1;
  }
  if (hi >= 0) {
    atomicMin_block(&ps->from, lo);
    atomicMax_block(&ps->to, hi);
  }
}

// Channels c.. of one row's output with what was taken out of its block's V given
// back (slow path); last: the last position that the row attends.
template <typename T>
__device__ __noinline__ float4 put_back(float4 x, const Poison& ps, const T* v, int64_t stride, const int32_t* pages,
                                        int num_pages, int shift, int last, int c, int D) {
  float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int ch = c + u;
    if (ch >= D) break;
    auto bit = [&](int kind) { return (ps.bits[kind][ch >> 5] >> (ch & 31) & 1) != 0; };
    const float z = poison_value(bit(0), bit(1), bit(2)) +
                    poison_of(v + ch, stride, pages, num_pages, shift, ps.from, min(ps.to, last));
    if (z != 0.f) y[u] += z;  // a NaN already there stays
  }
  return make_float4(y[0], y[1], y[2], y[3]);
}

// One quarter-tile's work and its running state, bf16
template <int DP>
struct RowsBf16 {
  static constexpr int kRows = 16;
  using S = Shape<__nv_bfloat16, DP, kRows>;
  static constexpr int NK = DP / 16, NV = DP / 8;
  uint32_t q[NK][4];
  float o[NV][4], m[2], l[2];

  __device__ void start(const char* stage, float*, int lane) {
    const uint32_t qs = smem_u32(stage + S::kKV);
#pragma unroll
    for (int k = 0; k < NK; ++k)
      ldsm4(q[k], qs + sw_off((lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4), S::kQBlock));
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[v][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  __device__ void step(char* stage, const float*, const Tile& t, float sc, Poison* ps, int warp, int lane) {
    const int x0 = t.x0 + 16 * warp;  // this warp's keys
    if (x0 >= t.end) return;
    const uint32_t ks = smem_u32(stage);
    char* vs = stage + S::NB * S::kBlock;
    const int live = min(16, t.end - x0);
    bool poison = false;
    const bool masked = x0 + 15 > t.pos0;
    if (masked) {
      // rows of V behind the block's last key to zero; non-finite values that some row may not attend
      for (int i = lane; i < 16 * S::NB * 8; i += 32) {
        const int r = i / (S::NB * 8), c = i % (S::NB * 8);
        uint4* x = reinterpret_cast<uint4*>(vs + sw_off(16 * warp + r, c, S::kBlock));
        if (r >= live) *x = make_uint4(0, 0, 0, 0);
        else if (t.rows > t.gb) {
          const uint4 y = *x;
          poison |= ((((y.x & 0x7f807f80u) + 0x00800080u) | ((y.y & 0x7f807f80u) + 0x00800080u) |
                      ((y.z & 0x7f807f80u) + 0x00800080u) | ((y.w & 0x7f807f80u) + 0x00800080u)) & 0x80008000u) != 0;
        }
      }
      poison = __any_sync(0xffffffffu, poison);
    }
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      uint32_t b[4];
      ldsm4(b, ks + sw_off(16 * warp + (lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1), S::kBlock));
      mma16816(s[0], q[k], b[0], b[1]);
      mma16816(s[1], q[k], b[2], b[3]);
    }
    const int r0 = lane >> 2, c0 = 2 * (lane & 3);
    int limit[2];
    if (masked) {
#pragma unroll
      for (int h = 0; h < 2; ++h) limit[h] = min(t.end - 1, t.pos0 + (r0 + 8 * h) / t.gb) - x0;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * n + c0 + (e & 1) > limit[e >> 1]) s[n][e] = -INFINITY;
    }
    float x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      x[h] = fmaxf(x[h], __shfl_xor_sync(0xffffffffu, x[h], 1));
      x[h] = sc * fmaxf(x[h], __shfl_xor_sync(0xffffffffu, x[h], 2));
    }
    bool move[2], scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      move[h] = x[h] > m[h] + kLazyLog2 || (m[h] == -INFINITY && x[h] > m[h]);
      scale[h] = move[h] && m[h] != -INFINITY;
    }
    if (__any_sync(0xffffffffu, scale[0] || scale[1])) {
      const float f0 = scale[0] ? exp2_fast(m[0] - x[0]) : 1.f, f1 = scale[1] ? exp2_fast(m[1] - x[1]) : 1.f;
      l[0] *= f0;
      l[1] *= f1;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        o[v][0] *= f0;
        o[v][1] *= f0;
        o[v][2] *= f1;
        o[v][3] *= f1;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (move[h]) m[h] = x[h];
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2_fast(fmaf(s[n][e], sc, -ref[e >> 1]));
        l[e >> 1] += s[n][e];
      }
    if (masked && poison) take_out<__nv_bfloat16, S::NB>(vs, S::kBlock, 16 * warp, 16, t.x0, t.pos0, ps, lane);
    __syncwarp();  // V's zeroed rows
    const uint32_t a[4] = {pack2(s[0][0], s[0][1]), pack2(s[0][2], s[0][3]), pack2(s[1][0], s[1][1]),
                           pack2(s[1][2], s[1][3])};
    const uint32_t va = smem_u32(vs);
#pragma unroll
    for (int v = 0; v < NV; v += 2) {
      uint32_t b[4];
      ldsm4t(b, va + sw_off(16 * warp + (lane & 15), v + (lane >> 4), S::kBlock));
      mma16816(o[v], a, b[0], b[1]);
      mma16816(o[v + 1], a, b[2], b[3]);
    }
  }

  // m and l of the warp's rows; then its output times f[row half] into scratch [16][DP]
  __device__ void stats(float2* ml, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if ((lane & 3) == 0) ml[(lane >> 2) + 8 * h] = make_float2(m[h], l[h]);
    }
  }
  __device__ void put(float* scratch, const float2 (*ml)[kMaxRows], int rows, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      if (r >= rows) continue;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][r].x);
      const float f = exp2_fast(m[h] - (M == -INFINITY ? 0.f : M));
#pragma unroll
      for (int v = 0; v < NV; ++v)
        *reinterpret_cast<float2*>(scratch + r * DP + 8 * v + 2 * (lane & 3)) =
            make_float2(o[v][2 * h] * f, o[v][2 * h + 1] * f);
    }
  }
};

// The same in fp32 on the same instructions: every operand is split into three
// bf16 parts (split3) and a product takes the six pairs that matter, h h, h m,
// m h, h l, l h and m m; what is left out is below 2^-22 of it, as an fp32
// rounding or two.  KW keys a warp; MT tiles of 16 rows, which share the
// splitting of K and V (more work than the products).
template <int DP, int KW, int MT>
struct RowsF32 {
  static constexpr int kRows = 16 * MT;
  using S = Shape<float, DP, kRows>;
  static_assert(KW * kWarps == S::KT, "a warp's share of a tile");
  static constexpr int NK = DP / 16, NV = DP / 8, NT = KW / 8;
  float o[MT][NV][4], m[MT][2], l[MT][2];

  __device__ void start(const char*, float*, int) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][v][e] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
  }
  // the block's q rows, split, by all consumers; rows it does not have are zeros
  static __device__ void load_q(const AttnParams& p, const Tile& t, float* qs, int tid) {
    const float* q = static_cast<const float*>(p.q);
    char* base = reinterpret_cast<char*>(qs);
#pragma unroll 4
    for (int i = tid; i < kRows * DP / 2; i += 32 * kWarps) {
      const int r = i / (DP / 2), c = 2 * (i % (DP / 2));
      float2 x = make_float2(0.f, 0.f);
      if (r < t.rows && c < p.D)
        x = *reinterpret_cast<const float2*>(q + ((int64_t)(t.tok0 + r / t.gb) * p.H + t.head0 + r % t.gb) * p.D + c);
      const Split y = split3(x.x, x.y);
      const uint32_t off = sw_off(r, c >> 3, S::kQBlock) + (c & 7) * 2;
      *reinterpret_cast<uint32_t*>(base + off) = y.h;
      *reinterpret_cast<uint32_t*>(base + S::kQPlane + off) = y.m;
      *reinterpret_cast<uint32_t*>(base + 2 * S::kQPlane + off) = y.l;
    }
  }

  __device__ void step(char* stage, const float* qs, const Tile& t, float sc, Poison* ps, int warp, int lane) {
    const int x0 = t.x0 + KW * warp;  // this warp's keys
    if (x0 >= t.end) return;
    char* vs = stage + S::NB * S::kBlock;
    const int live = min(KW, t.end - x0);
    bool poison = false;
    const bool masked = x0 + KW - 1 > t.pos0;
    // rows of V behind the block's last key to zero; non-finite values are
    // looked for in every tile (split, they would meet parts that are 0)
    if (live < KW) {
      for (int i = live * S::NB * 8 + lane; i < KW * S::NB * 8; i += 32)
        *reinterpret_cast<uint4*>(vs + sw_off(KW * warp + i / (S::NB * 8), i % (S::NB * 8), S::kBlock)) =
            make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    uint32_t seen = 0;
#pragma unroll 8
    for (int i = lane; i < KW * S::NB * 8; i += 32) {
      const uint4 y = *reinterpret_cast<const uint4*>(vs + sw_off(KW * warp + i / (S::NB * 8), i % (S::NB * 8), S::kBlock));
      seen |= ((y.x & 0x7f800000u) + 0x00800000u) | ((y.y & 0x7f800000u) + 0x00800000u) |
              ((y.z & 0x7f800000u) + 0x00800000u) | ((y.w & 0x7f800000u) + 0x00800000u);
    }
    poison = (seen & 0x80000000u) != 0;
    poison = __any_sync(0xffffffffu, poison);
    const int r0 = lane >> 2, q2 = lane & 3;
    // h h apart from the smaller products, and (one key tile of 8) even from odd
    // steps: products that follow one another are of different sums
    constexpr int KS = MT * NT == 1 ? 2 : 1;
    float s[MT][NT][4], sh[KS][MT][NT][4], sx[KS][2][MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int z = 0; z < KS; ++z) sh[z][i][n][e] = sx[z][0][i][n][e] = sx[z][1][i][n][e] = 0.f;
    const uint32_t qa = smem_u32(qs);
#pragma unroll (MT == 1 ? 4 / KS : 1)
    for (int k0 = 0; k0 < NK; k0 += KS) {
#pragma unroll
      for (int z = 0; z < KS; ++z) {
        const int k = k0 + z;
        uint32_t ah[MT][4], am[MT][4], al[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint32_t off = sw_off(16 * i + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4), S::kQBlock);
          ldsm4(ah[i], qa + off);
          ldsm4(am[i], qa + S::kQPlane + off);
          ldsm4(al[i], qa + 2 * S::kQPlane + off);
        }
        Split b0[NT], b1[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int row = KW * warp + 8 * n + r0;
          const float2 x = *reinterpret_cast<const float2*>(stage + sw_off(row, 4 * k + (q2 >> 1), S::kBlock) + (q2 & 1) * 8);
          const float2 y = *reinterpret_cast<const float2*>(stage + sw_off(row, 4 * k + 2 + (q2 >> 1), S::kBlock) + (q2 & 1) * 8);
          b0[n] = split3(x.x, x.y);
          b1[n] = split3(y.x, y.y);
        }
#pragma unroll
        for (int r = 0; r < 3; ++r)
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (r == 0) mma16816(sx[z][0][i][n], ah[i], b0[n].l, b1[n].l);
              if (r == 1) mma16816(sx[z][0][i][n], al[i], b0[n].h, b1[n].h);
              if (r == 2) mma16816(sx[z][0][i][n], am[i], b0[n].m, b1[n].m);
              if (r == 0) mma16816(sh[z][i][n], ah[i], b0[n].h, b1[n].h);
              if (r == 1) mma16816(sx[z][1][i][n], ah[i], b0[n].m, b1[n].m);
              if (r == 2) mma16816(sx[z][1][i][n], am[i], b0[n].h, b1[n].h);
            }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][n][e] = (sx[0][0][i][n][e] + sx[0][1][i][n][e]) + sh[0][i][n][e];
          if (KS == 2) s[i][n][e] += (sx[KS - 1][0][i][n][e] + sx[KS - 1][1][i][n][e]) + sh[KS - 1][i][n][e];
        }
    int limit[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      limit[i][0] = limit[i][1] = KW - 1;
      if (masked) {
#pragma unroll
        for (int h = 0; h < 2; ++h) limit[i][h] = min(t.end - 1, t.pos0 + (16 * i + r0 + 8 * h) / t.gb) - x0;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * n + 2 * q2 + (e & 1) > limit[i][e >> 1]) s[i][n][e] = -INFINITY;
      }
      float x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[h] = fmaxf(s[i][0][2 * h], s[i][0][2 * h + 1]);
        if (NT == 2) x[h] = fmaxf(x[h], fmaxf(s[i][NT - 1][2 * h], s[i][NT - 1][2 * h + 1]));
        x[h] = fmaxf(x[h], __shfl_xor_sync(0xffffffffu, x[h], 1));
        x[h] = sc * fmaxf(x[h], __shfl_xor_sync(0xffffffffu, x[h], 2));
      }
      if (__any_sync(0xffffffffu, x[0] > m[i][0] || x[1] > m[i][1])) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(x[h] > m[i][h])) x[h] = m[i][h];
          const float f = m[i][h] == -INFINITY ? 1.f : exp2f(m[i][h] - x[h]);
          m[i][h] = x[h];
          l[i][h] *= f;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            o[i][v][2 * h] *= f;
            o[i][v][2 * h + 1] *= f;
          }
        }
      }
      const float ref[2] = {m[i][0] == -INFINITY ? 0.f : m[i][0], m[i][1] == -INFINITY ? 0.f : m[i][1]};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][n][e] = exp2f(fmaf(s[i][n][e], sc, -ref[e >> 1]));
          l[i][e >> 1] += s[i][n][e];
        }
    }
    if (poison) take_out<float, S::NB>(vs, S::kBlock, KW * warp, KW, t.x0, t.pos0, ps, lane);
    __syncwarp();  // V's zeroed rows
    uint32_t ah[MT][2 * NT], am[MT][2 * NT], al[MT][2 * NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int z = 0; z < 2 * NT; ++z) {
        const Split y = split3(s[i][z >> 1][2 * (z & 1)], s[i][z >> 1][2 * (z & 1) + 1]);
        ah[i][z] = y.h;
        am[i][z] = y.m;
        al[i][z] = y.l;
      }
    // VG groups of 8 channels at a time: products that follow one another are
    // of different sums (one after the other on one sum, their latency would rule)
    constexpr int VG = 4 / MT;
#pragma unroll
    for (int v = 0; v < NV; v += VG) {
      Split b0[VG], b1[VG];
#pragma unroll
      for (int g = 0; g < VG; ++g) {
        // keys 2 q2, + 1 (, + 8, + 9) of channel 8 (v + g) + r0
        float y[2 * NT];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i)
          y[i] = *reinterpret_cast<const float*>(
              vs + sw_off(KW * warp + 2 * q2 + (i & 1) + 8 * (i >> 1), 2 * (v + g) + (r0 >> 2), S::kBlock) + (r0 & 3) * 4);
        b0[g] = split3(y[0], y[1]);
        b1[g] = split3(y[2 * NT - 2], y[2 * NT - 1]);
      }
      // from zero, and added rounded to nearest: the tensor cores' own
      // accumulation cuts, a bias that grows with the tiles
      float y4[MT][VG][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int g = 0; g < VG; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) y4[i][g][e] = 0.f;
#pragma unroll
      for (int z = 0; z < 6; ++z)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int g = 0; g < VG; ++g) {
            const uint32_t* x = z == 1 ? al[i] : z == 2 || z == 4 ? am[i] : ah[i];
            const uint32_t c0 = z == 0 ? b0[g].l : z == 2 || z == 3 ? b0[g].m : b0[g].h;
            const uint32_t c1 = z == 0 ? b1[g].l : z == 2 || z == 3 ? b1[g].m : b1[g].h;
            mma_keys<NT>(y4[i][g], x, c0, c1);
          }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int g = 0; g < VG; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][v + g][e] += y4[i][g][e];
    }
  }
  __device__ void stats(float2* ml, int lane) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[i][h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if ((lane & 3) == 0) ml[16 * i + (lane >> 2) + 8 * h] = make_float2(m[i][h], x);
      }
  }
  __device__ void put(float* scratch, const float2 (*ml)[kMaxRows], int rows, int lane) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * i + (lane >> 2) + 8 * h;
        if (r >= rows) continue;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][r].x);
        const float f = exp2f(m[i][h] - (M == -INFINITY ? 0.f : M));
#pragma unroll
        for (int v = 0; v < NV; ++v)
          *reinterpret_cast<float2*>(scratch + r * DP + 8 * v + 2 * (lane & 3)) =
              make_float2(o[i][v][2 * h] * f, o[i][v][2 * h + 1] * f);
      }
  }
};

template <typename T, int DP, typename Work>
__global__ void __launch_bounds__(kThreads, Shape<T, DP, Work::kRows>::CTAS)
    attn_rows(const AttnParams p, const RowsArgs a, const __grid_constant__ CUtensorMap mq,
              const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Shape<T, DP, Work::kRows>;
  static_assert(shape_ok<T, DP, Work::kRows>(), "shared memory");
  constexpr int R = Work::kRows;
  constexpr int KT = S::KT;
  extern __shared__ char raw[];
  char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Tail* b = reinterpret_cast<Tail*>(sm + S::kTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&b->full[s], 1);
      mbar_init(&b->empty[s], kWarps);
    }
    mbar_init(&b->join[0], kWarps);
    mbar_init(&b->join[1], kWarps);
    b->dead = 0;
    mbar_init_fence();
  }
  if (tid < 3 * kPoisonWords) reinterpret_cast<int32_t*>(b->poison)[tid] = no_poison(tid % kPoisonWords);
  if (tid == 32) {
    prefetch_map(&mk);
    prefetch_map(&mv);
    if (sizeof(T) == 2) prefetch_map(&mq);
  }
  pdl_wait();
  pdl_launch_dependents();  // the join's launch overlaps the work (it waits for the end of it)

  // the line of work: its length, this CTA's stretch, and where that starts
  int64_t u0 = 0, u1 = 0, per = 0;
  const bool one = p.num_seqs <= kThreads;  // the batch in one go: its tiles are counted once
  for (int pass = 0; pass < 2; ++pass) {
    int64_t before = 0;
    for (int base = 0; base < p.num_seqs; base += kThreads) {
      const int s = base + tid;
      int64_t n = 0;
      AttnSeq q{};
      if (s < p.num_seqs) {
        q = attn_seq(p, s);
        if (pass == 0 && q.flag && blockIdx.x == 0) attn_flag(p.status, q.flag);
        if (q.len > 0) n = Blocks<KT>(q, a.q_shift).total() * p.Hkv * a.parts;
      }
      int64_t x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) b->sum[warp] = x;
      __syncthreads();
      int64_t total = 0;
#pragma unroll
      for (int w = 0; w <= kWarps; ++w) {
        if (w < warp) x += b->sum[w];
        total += b->sum[w];
      }
      if (pass == 0 && one) {
        const int64_t share = div_any(total + gridDim.x - 1, gridDim.x);
        per = share > kMinTiles ? share : kMinTiles;
        u0 = min(total, per * blockIdx.x);
        u1 = min(total, u0 + per);
      }
      if ((pass == 1 || one) && n > 0 && u0 >= before + x - n && u0 < before + x) {
        b->found = u0 - (before + x - n);
        b->found_at = s;
        b->found_seq = q;
      }
      before += total;
      if (pass == 1 && u0 < before) break;
    }
    if (pass == 0 && !one) {
      const int64_t share = div_any(before + gridDim.x - 1, gridDim.x);
      per = share > kMinTiles ? share : kMinTiles;
      u0 = min(before, per * blockIdx.x);
      u1 = min(before, u0 + per);
    }
    if (u0 == u1) {
      if (tid == 0) a.joins[blockIdx.x].parts = 0;
      return;
    }
    if (one) break;
  }
  __syncthreads();
  const int64_t first_off = b->found;

  if (warp == kWarps) {
    // ---- copies
    int base = b->found_at, cur = 0;  // sequences behind the first: 32 at a time, one a lane
    AttnSeq mine{};
    auto fetch = [&](int at) {
      base = at;
      mine = AttnSeq{};
      if (at + lane < p.num_seqs) mine = attn_seq(p, at + lane);
    };
    AttnSeq sq = b->found_seq;
    auto seq = [&] {
      sq.tok0 = __shfl_sync(0xffffffffu, mine.tok0, cur);
      sq.len = __shfl_sync(0xffffffffu, mine.len, cur);
      sq.kv_len = __shfl_sync(0xffffffffu, mine.kv_len, cur);
      sq.row = __shfl_sync(0xffffffffu, mine.row, cur);
    };
    Blocks<KT> bl(sq, a.q_shift);
    const int64_t per_head = bl.total();
    int head = (int)div_any(first_off, per_head), tile;  // head: key head * parts + part
    int64_t block;
    bl.find(first_off - head * per_head, &block, &tile);
    int n = bl.tiles(block);
    bool seg_first = true;
    int seg_tile0 = tile;
    bool ok = true;
    uint32_t k = 0;
    if (lane == 0) a.joins[blockIdx.x].parts = 0;
    const uint32_t box_bytes = 128u << a.box_shift;
    const int box = 1 << a.box_shift, qt = 1 << a.q_shift, gmax = min(p.G, R);
    for (int64_t u = u0; u < u1 && ok; ++u, ++k) {
      const int kvh = a.parts == 1 ? head : head / a.parts, part = a.parts == 1 ? 0 : head - kvh * a.parts;
      const int t0 = (int)block << a.q_shift, ntok = min(qt, sq.len - t0);
      const int pos0 = (int)sq.kv_len - sq.len + t0, end = max(0, min((int)sq.kv_len, pos0 + ntok));
      const int x0 = tile * KT;
      const int nb = max(0, min(KT >> a.box_shift, (end - x0 + box - 1) >> a.box_shift));
      const int x = x0 + (lane << a.box_shift);
      int c2 = (int)sq.tok0 + x, c3 = 0;
      if (p.block_table) {
        int page = p.num_pages;
        if (lane < nb) {
          page = p.block_table[(int64_t)sq.row * p.max_pages + (x >> p.page_shift)];
          if (page < 0 || page >= p.num_pages) {
            attn_flag(p.status, kFlagBadCache);
            page = p.num_pages;  // outside the map: filled with zeros
          }
        }
        c2 = x & ((1 << p.page_shift) - 1);
        c3 = page;
      }
      const uint32_t st = k % S::kStages;
      ok = __all_sync(0xffffffffu, wait_or_dead(&b->empty[st], ((k / S::kStages) & 1) ^ 1, &b->dead));
      if (!ok) break;
      char* dst = sm + st * S::kStage;
      const bool last = u + 1 == u1 || tile + 1 == n;
      if (lane == 0) {
        Tile t;
        t.tok0 = (int)sq.tok0 + t0;
        t.head0 = kvh * p.G + part * R;
        t.gb = a.parts == 1 ? p.G : min(R, p.G - part * R);
        t.rows = ntok * t.gb;
        t.pos0 = pos0;
        t.end = end;
        t.x0 = x0;
        t.base = p.block_table ? sq.row : (int)sq.tok0;
        t.kvh = kvh;
        t.first = seg_first;
        t.last = last;
        t.slot = -1;
        if (last && (seg_tile0 > 0 || tile + 1 < n)) {
          t.slot = 2 * (int)blockIdx.x + (seg_tile0 == 0);
          if (seg_tile0 == 0)  // the block starts here: its other parts are the next stretches' first ones
            a.joins[blockIdx.x] = RowsJoin{(int)div_any(u - tile + n - 1, per) - (int)blockIdx.x + 1, t.tok0, t.head0, t.rows, t.gb};
        }
        b->tile[st] = t;
        const uint32_t bytes = (uint32_t)nb * box_bytes * 2 * S::NB +
                               (sizeof(T) == 2 && seg_first ? (uint32_t)(qt * gmax) * 128u * S::NB : 0u);
        mbar_arrive_expect_tx(&b->full[st], bytes);
        if (sizeof(T) == 2 && seg_first)
#pragma unroll
          for (int c = 0; c < S::NB; ++c)
            tma_3d(dst + S::kKV + c * S::kQBlock, &mq, c * (128 / (int)sizeof(T)), t.head0, t.tok0, &b->full[st]);
      }
      __syncwarp();
      if (lane < nb)
#pragma unroll
        for (int c = 0; c < S::NB; ++c) {
          const int ch = c * (128 / (int)sizeof(T));
          tma_4d(dst + c * S::kBlock + lane * box_bytes, &mk, ch, kvh, c2, c3, &b->full[st]);
          tma_4d(dst + (S::NB + c) * S::kBlock + lane * box_bytes, &mv, ch, kvh, c2, c3, &b->full[st]);
        }
      if (k == 0) fetch(base);  // (the first sequence again, and those behind it)
      // the next tile of the line
      seg_first = last;
      if (++tile == n) {
        tile = 0;
        if (++block == bl.n) {
          block = 0;
          if (++head == p.Hkv * a.parts) {
            head = 0;
            if (u + 1 < u1) {
              do {
                if (++cur == 32) {
                  cur = 0;
                  fetch(base + 32);
                }
                seq();
              } while (sq.len == 0 && base + cur < p.num_seqs);
              bl = Blocks<KT>(sq, a.q_shift);
            }
          }
        }
        n = bl.tiles(block);
      }
      if (seg_first) seg_tile0 = tile;
    }
    if (!ok)  // no copy in flight when a CTA that gave up exits
      for (uint32_t i = k > (uint32_t)S::kStages ? k - S::kStages : 0; i < k; ++i)
        mbar_wait(&b->full[i % S::kStages], (i / S::kStages) & 1, kWaitLimitNs);
  } else {
    // ---- scores, softmax, output
    Work w;
    float* qs = reinterpret_cast<float*>(sm + S::kQ);
    const float sc = p.scale * kLog2e;
    uint32_t joins = 0;
    int block = 0;  // of the blocks of the stretch, modulo 3
    uint32_t k = 0;
    for (int64_t u = u0; u < u1; ++u, ++k) {
      const uint32_t st = k % S::kStages;
      char* stage = sm + st * S::kStage;
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->full[st], (k / S::kStages) & 1, &b->dead))) break;
      const Tile t = b->tile[st];
      if (t.first) {
        if constexpr (sizeof(T) == 4) {
          // (the last pair's readers of qs are done: they met at its join)
          Work::load_q(p, t, qs, tid);
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->join[0]);
          if (!__all_sync(0xffffffffu, wait_or_dead(&b->join[0], joins & 1, &b->dead))) break;
          if (lane == 0) mbar_arrive(&b->join[1]);
          if (!__all_sync(0xffffffffu, wait_or_dead(&b->join[1], joins & 1, &b->dead))) break;
          ++joins;
        }
        w.start(stage, qs, lane);
      }
      w.step(stage, qs, t, sc, &b->poison[block], warp, lane);
      if (t.last) {
        const int rows = t.rows;
        w.stats(b->ml[warp], lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->join[0]);
        if (!__all_sync(0xffffffffu, wait_or_dead(&b->join[0], joins & 1, &b->dead))) break;
        // every warp is done with this stage's K and V: it holds the outputs now
        float* scratch = reinterpret_cast<float*>(stage);
        w.put(scratch + warp * R * DP, b->ml, rows, lane);
        // each row's M and l over the warps, before another pair's replace them;
        // a thread's output quads are STEPS pieces of the [R][DP] tile
        constexpr int VEC = DP / 4, STEPS = R * VEC / (32 * kWarps);
        float M[STEPS], L[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const int r = (i * 32 * kWarps + tid) / VEC;
          M[i] = -INFINITY;
          L[i] = 0.f;
          if (r >= rows) continue;
#pragma unroll
          for (int z = 0; z < kWarps; ++z) M[i] = fmaxf(M[i], b->ml[z][r].x);
#pragma unroll
          for (int z = 0; z < kWarps; ++z)
            L[i] += exp2f(b->ml[z][r].x - (M[i] == -INFINITY ? 0.f : M[i])) * b->ml[z][r].y;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->join[1]);
        if (!__all_sync(0xffffffffu, wait_or_dead(&b->join[1], joins & 1, &b->dead))) break;
        ++joins;
        T* out = static_cast<T*>(p.o);
        const Poison* ps = &b->poison[block];
        const bool poisoned = *reinterpret_cast<const volatile uint32_t*>(&ps->seen) != 0;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const int e = i * 32 * kWarps + tid, r = e / VEC, c = (e % VEC) * 4;
          if (r >= rows) continue;
          float4 x = *reinterpret_cast<const float4*>(scratch + r * DP + c);
#pragma unroll
          for (int z = 1; z < kWarps; ++z) {
            const float4 y = *reinterpret_cast<const float4*>(scratch + (z * R + r) * DP + c);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
          }
          if (poisoned) {
            const int64_t stride = (int64_t)p.Hkv * p.D;
            x = put_back(x, *ps, static_cast<const T*>(p.v) + (int64_t)t.kvh * p.D + (p.block_table ? 0 : t.base * stride),
                         stride, p.block_table ? p.block_table + (int64_t)t.base * p.max_pages : nullptr, p.num_pages,
                         p.page_shift, min(t.end - 1, t.pos0 + r / t.gb), c, p.D);
          }
          if (t.slot >= 0) {
            *reinterpret_cast<float4*>(a.o + ((int64_t)t.slot * kMaxRows + r) * DP + c) = x;
            if (c == 0) a.ml[t.slot * kMaxRows + r] = make_float2(M[i], L[i]);
          } else if (c < p.D) {
            const int64_t at =
                ((int64_t)(t.tok0 + r / t.gb) * p.H + t.head0 + r % t.gb) * p.D + c;
            const float f = L[i] == 0.f ? 0.f : 1.f / L[i];
            if constexpr (sizeof(T) == 2)
              *reinterpret_cast<uint2*>(out + at) = make_uint2(pack2(x.x * f, x.y * f), pack2(x.z * f, x.w * f));
            else
              *reinterpret_cast<float4*>(out + at) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
          }
        }
        // the word of the block after next is free: all warps are past the block
        // before this one, and none starts that one before this thread's next join
        const int next = block == 0 ? 2 : block - 1;
        if (tid < kPoisonWords) reinterpret_cast<int32_t*>(&b->poison[next])[tid] = no_poison(tid);
        block = block == 2 ? 0 : block + 1;
      }
      // generic accesses of the stage before the copies that refill it
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->empty[st]);
    }
  }
  __syncthreads();
  if (tid == 0 && b->dead) attn_flag(p.status, kFlagTimeout);
}

// The blocks that cross stretches: parts 2 c + 1, 2 (c + 1), 2 (c + 2), .. of
// stretch c.  A CTA per row at a time, the parts dealt to its warps, which are
// then added in their order.
constexpr int kJoinWarps = 8, kJoinRows = 16;
template <typename T, int DP>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_rows_join(const AttnParams p, const RowsArgs a) {
  __shared__ float sm_o[kJoinWarps][DP];
  __shared__ float sm_l[kJoinWarps];
  pdl_wait();
  const RowsJoin jn = a.joins[blockIdx.x];
  if (jn.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int V = DP / 32;
  const int s0 = 2 * (int)blockIdx.x;
  for (int r = blockIdx.y; r < jn.rows; r += gridDim.y) {
    auto slot = [&](int k) { return (k == 0 ? s0 + 1 : s0 + 2 * k) * kMaxRows + r; };
    float M = -INFINITY;
    for (int k = lane; k < jn.parts; k += 32) M = fmaxf(M, a.ml[slot(k)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;
    float l = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
#pragma unroll 4
    for (int k = warp; k < jn.parts; k += kJoinWarps) {
      const float2 ml = a.ml[slot(k)];
      const float f = exp2f(ml.x - M);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = fmaf(f, a.o[(int64_t)slot(k) * DP + 32 * v + lane], o[v]);
    }
    __syncthreads();  // the row before is written
#pragma unroll
    for (int v = 0; v < V; ++v) sm_o[warp][32 * v + lane] = o[v];
    if (lane == 0) sm_l[warp] = l;
    __syncthreads();
    const int64_t at = ((int64_t)(jn.tok0 + r / jn.gb) * p.H + jn.head0 + r % jn.gb) * p.D;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) sum += sm_l[w];
    for (int c = threadIdx.x; c < p.D; c += 32 * kJoinWarps) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) x += sm_o[w][c];
      st_out(static_cast<T*>(p.o), at + c, sum == 0.f ? 0.f : x / sum);
    }
  }
}

// ------------------------------------------------------------------ host
constexpr int kMaxGrid = 2 * 192;  // two CTAs on each of up to 192 SMs

int padded(const AttnParams& p) {
  const int low = p.dt == KDA_BF16 ? 64 : 32;
  return p.D < low ? low : p.D;
}

// Tokens of a block, log2: as many as its rows hold and a sequence may have
int block_shift(const AttnParams& p, int rows) {
  int s = 0;
  while ((2 << s) * p.G <= rows && (1 << s) < p.max_seqlen) ++s;
  return s;
}

template <typename T, int DP, typename Work>
cudaError_t launch_w(const AttnParams& p, char* w, cudaStream_t stream) {
  constexpr int R = Work::kRows;
  using S = Shape<T, DP, R>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  auto kernel = attn_rows<T, DP, Work>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
  if (e != cudaSuccess) return e;
  // no more CTAs than stretches of kMinTiles that the longest rows could fill
  const int64_t keys = p.block_table ? (int64_t)p.max_pages << p.page_shift : p.total_tokens;
  const int64_t blocks = ((p.total_tokens >> block_shift(p, R)) + p.num_seqs) * ((p.G + R - 1) / R) * p.Hkv;
  const int64_t most = blocks < kMaxGrid * kMinTiles ? (blocks * (keys / S::KT + 2) + kMinTiles - 1) / kMinTiles : kMaxGrid;
  int grid = sms * S::CTAS < kMaxGrid ? sms * S::CTAS : kMaxGrid;
  if (most < grid) grid = (int)most;
  RowsArgs a{};
  a.joins = reinterpret_cast<RowsJoin*>(w);
  a.ml = reinterpret_cast<float2*>(w + align_up(sizeof(RowsJoin) * kMaxGrid, 256));
  a.o = reinterpret_cast<float*>(a.ml + 2 * kMaxGrid * kMaxRows);
  constexpr int kt_shift = S::KT == 64 ? 6 : 5;
  a.box_shift = p.block_table && p.page_shift < kt_shift ? p.page_shift : kt_shift;
  a.q_shift = block_shift(p, R);
  a.parts = (p.G + R - 1) / R;
  const int heads = p.G < R ? p.G : R;
  CUtensorMap mq, mk, mv;
  if (!attn_map(&mq, p, p.q, true, heads, 1 << a.q_shift) || !attn_map(&mk, p, p.k, false, 1, 1 << a.box_shift) ||
      !attn_map(&mv, p, p.v, false, 1, 1 << a.box_shift))
    return cudaErrorInvalidValue;
  e = launch_maybe_dependent(true, kernel, dim3((unsigned)grid), dim3(kThreads), (size_t)S::kBytes, stream, p, a, mq, mk,
                             mv);
  if (e != cudaSuccess) return e;
  return launch_maybe_dependent(true, attn_rows_join<T, DP>,
                                dim3((unsigned)grid, (unsigned)std::min(heads << a.q_shift, kJoinRows)),
                                dim3(32 * kJoinWarps), 0, stream, p, a);
}

// fp32: 32 rows where a sequence has them, else 16
template <int DP>
cudaError_t launch_f32(const AttnParams& p, char* w, cudaStream_t stream) {
  if (p.max_seqlen * p.G > 16) return launch_w<float, DP, RowsF32<DP, 16, 2>>(p, w, stream);
  return launch_w<float, DP, RowsF32<DP, 16, 1>>(p, w, stream);
}

}  // namespace

// Single tokens, or as few as 16 rows hold, over the cache (more rows go to the
// tensor cores' 128-row tiles first, where they have a form for the type and head
// size); all of fp32 and of 256 channels that none of them takes.  A positive
// finite scale (the running maximum is taken before the scaling), 16-byte aligned
// bases for the tensor maps.
bool attn_rows_fits(const AttnParams& p) {
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  return (few_rows(p) || p.dt == KDA_F32 || p.D == 256) && p.scale > 0.f && p.scale <= 3.4e38f && al16(p.q) && al16(p.k) &&
         al16(p.v) && al16(p.o) && (!p.block_table || p.num_pages > 0);
}
size_t attn_rows_workspace(const AttnParams& p) {
  return align_up(sizeof(RowsJoin) * kMaxGrid, 256) + 2 * kMaxGrid * kMaxRows * (sizeof(float2) + padded(p) * 4);
}
cudaError_t launch_attn_rows(const AttnParams& p, void* ws, cudaStream_t stream) {
  char* w = static_cast<char*>(ws);
  if (p.dt == KDA_BF16) {
    switch (padded(p)) {
      case 64: return launch_w<__nv_bfloat16, 64, RowsBf16<64>>(p, w, stream);
      case 128: return launch_w<__nv_bfloat16, 128, RowsBf16<128>>(p, w, stream);
      default: return launch_w<__nv_bfloat16, 256, RowsBf16<256>>(p, w, stream);
    }
  }
  switch (padded(p)) {
    case 32: return launch_f32<32>(p, w, stream);
    case 64: return launch_f32<64>(p, w, stream);
    case 128: return launch_f32<128>(p, w, stream);
    default: return launch_w<float, 256, RowsF32<256, 8, 1>>(p, w, stream);
  }
}

}  // namespace kda
