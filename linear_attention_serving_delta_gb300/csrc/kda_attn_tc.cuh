// kda_attn_tc.cuh -- plan records and PTX helpers of the tensor-core attention
// and of the attention of a few rows.
//
// Shared-memory operands here are 128-byte swizzled: a tile is stored in
// blocks of 64 channels, each [rows][64] bf16 with rows of 128 bytes whose
// eight 16-byte pieces are permuted by row % 8 (what a tensor-map copy with
// CU_TENSOR_MAP_SWIZZLE_128B writes).  As a K-major operand (Q, K) the 8-row
// groups are 1024 bytes apart and 16 channels are 32 bytes; as an MN-major
// one (V, whose tokens are the contraction) the 64-channel blocks are the
// leading stride, and 16 tokens are 2048 bytes.
#pragma once

#include <type_traits>

#include "kda_attn.cuh"
#include "kda_tc.cuh"

namespace kda {

// Over the cache, requests of up to kTinyRows rows a key head take the streaming
// kernel's blocks, and so do a few blocks of rows over short tables: a 128-row
// tile's chain of steps would take longer (163 requests of 1..40 tokens over
// tables of 320 positions 38 us, 48 on the row tiles; 100 requests of 32 rows over
// 960 positions 73 and 58).
constexpr int kTinyRows = 16, kShortRows = 64, kShortKeys = 512;
// Requests of up to this many rows a key head take blocks of 16 or 32 rows where
// a CTA would have one row tile only (fp32, 20 rows of 7 requests: 23 us, 34 on
// the row tiles)
constexpr int kFewRows = 32;
constexpr int kRowTile = 128;  // rows of a row tile
// The SMs the cut into pieces is sized for, the pieces an SM gets (a chunk of 512
// tokens over 32k keys beside eight requests: one 328 us, two 277, three 297,
// four 300), and the fewest key tiles a piece has
constexpr int kSplitSms = 152;
constexpr int kPiecesPerSm = 2;
constexpr int kMinPiece = 4;
// Rows of up to this many positions are not worth cutting in a small call
constexpr int kSelfPlanKeys = 2048;

// One unit of work (for each key head): ntok tokens from packed token tok0 on,
// the first at position pos0, over the key tiles [kt0, kt1) of a sequence of
// kv_len positions.  base: the sequence's first packed token (prompts) or its
// row of the block table.  slot >= 0: a piece, its partial result's place.
struct AttnItem {
  int32_t tok0, ntok, base, pos0, kv_len, kt0, kt1, slot;
};
struct AttnJoin {
  int32_t tok0, ntok, slot, pieces;
};
struct AttnHead {
  int32_t items, joins;
};
struct TcArgs {
  AttnHead* head;
  int64_t* seq_begin;   // [N] first tile of each sequence
  AttnItem* items;
  int64_t max_items;    // tiles the workspace has room for
  int32_t row_tiles;    // row tiles of an item
  int32_t tpt;          // tokens of a row tile
  int32_t kt_shift;     // log2 of a key tile's positions
  int32_t box_shift;    // log2 of the positions per copy
  int32_t self_plan;    // every CTA finds its one item
  int32_t o_wide;       // o is 32-byte aligned
  int32_t split_sms;    // > 0: items may be cut into pieces
  AttnJoin* joins;
  float2* part_ml;      // [pieces][Hkv][row_tiles * 128] (m, l)
  float* part_o;        // [pieces][Hkv][row_tiles * 128][DP]
};

struct TcLayout {
  size_t head, seq_begin, items, joins, ml, o, total;
  int64_t max_items, max_pieces;
  bool split, self_plan;
};

// Tile `tile` (of row_tiles x tpt tokens) of sequence s, over all of its keys
__device__ __forceinline__ AttnItem make_item(const AttnParams& p, const TcArgs& a, const AttnSeq& s, int64_t tile) {
  const int tpi = a.row_tiles * a.tpt;
  AttnItem it;
  it.tok0 = (int32_t)(s.tok0 + tile * tpi);
  it.ntok = (int32_t)min((int64_t)tpi, s.len - tile * tpi);
  it.base = p.block_table ? s.row : (int32_t)s.tok0;
  it.pos0 = (int32_t)(s.kv_len - s.len + tile * tpi);
  it.kv_len = (int32_t)s.kv_len;
  it.kt0 = 0;
  it.kt1 = (max(0, min(it.kv_len, it.pos0 + it.ntok)) + (1 << a.kt_shift) - 1) >> a.kt_shift;
  it.slot = -1;
  return it;
}
__device__ __forceinline__ const AttnItem& item_at(const TcArgs& a, int64_t w, int Hkv) {
  return a.items[a.self_plan ? w : w / Hkv];
}

// The CTA's i-th item: items go round the CTAs back and forth, so that the
// sorted costs even out.
__device__ __forceinline__ int64_t nth_item(int i) {
  const int64_t g = gridDim.x, c = blockIdx.x;
  return (int64_t)i * g + ((i & 1) ? g - 1 - c : c);
}

// A stage of a ring and its phase
template <int N>
struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1;
    }
  }
};

// Key tile x0.. of K or V for the whole warp, a box a lane: c2, c3 are the
// box's coordinates in the map, n how many boxes hold positions.
struct Boxes {
  int c2, c3, n;
};
__device__ __forceinline__ Boxes boxes_of(const AttnParams& p, const AttnItem& it, int x0, int keys, int shift, int lane) {
  Boxes r;
  r.n = min(keys >> shift, (it.kv_len - x0 + (1 << shift) - 1) >> shift);
  const int x = x0 + (lane << shift);
  r.c2 = it.base + x;
  r.c3 = 0;
  if (p.block_table) {
    int page = p.num_pages;
    if (lane < r.n) {
      page = p.block_table[(int64_t)it.base * p.max_pages + (x >> p.page_shift)];
      if (page < 0 || page >= p.num_pages) {
        attn_flag(p.status, kFlagBadCache);
        page = p.num_pages;  // outside the map: filled with zeros
      }
    }
    r.c2 = x & ((1 << p.page_shift) - 1);
    r.c3 = page;
  }
  return r;
}

struct OwnPlan {
  uint32_t own;     // this CTA has an item; 0 at the start
  int32_t sum[12];  // of the warps
};
// Small calls plan for themselves: no more items than CTAs, so the order does
// not matter and CTA w needs item w alone, which the thread of its sequence
// leaves in the workspace.  Returns whether there is one (for every thread).
template <int THREADS>
__device__ bool plan_own_item(const AttnParams& p, const TcArgs& a, OwnPlan* b) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tpi = a.row_tiles * a.tpt;
  const int64_t want = blockIdx.x / p.Hkv;
  int64_t before = 0;
  for (int base = 0; base < p.num_seqs; base += THREADS) {
    const int s = base + tid;
    AttnSeq q{};
    int n = 0;
    if (s < p.num_seqs) {
      q = attn_seq(p, s);
      if (q.flag && blockIdx.x == 0) attn_flag(p.status, q.flag);
      n = (q.len + tpi - 1) / tpi;
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) b->sum[warp] = x;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) x += b->sum[w];
      total += b->sum[w];
    }
    const int64_t first = before + x - n;
    if (n > 0 && want >= first && want < first + n) {
      a.items[blockIdx.x] = make_item(p, a, q, want - first);
      b->own = 1;
    }
    before += total;
    __syncthreads();
  }
  return *reinterpret_cast<volatile uint32_t*>(&b->own) != 0;
}

// The non-finite values taken out of V tiles come back at the output (slow
// path).  What a channel of a row gets: an infinity, or NaN where both signs or
// a NaN meet; 0 for none.
__device__ __forceinline__ float poison_value(bool pos, bool neg, bool nan) {
  return nan || (pos && neg) ? NAN : pos ? INFINITY : neg ? -INFINITY : 0.f;
}
// The kind of a non-finite value, as an index of a row of bits: +inf, -inf, NaN
__device__ __forceinline__ int poison_kind(float x) { return x != x ? 2 : x < 0.f ? 1 : 0; }
// From the cache itself, over the positions from..limit: those that some rows of
// a tile may attend and others may not, no more than its tokens (a longer way,
// one load after the other, would outlast the CTA's other waits).
template <typename T>
static __device__ __noinline__ float poison_of(const T* v, int64_t stride, const int32_t* pages, int num_pages, int shift,
                                        int from, int limit) {
  bool pos = false, neg = false, nan = false;
  for (int x = from; x <= limit; ++x) {
    int64_t at = x;
    if (pages) {
      const int32_t page = pages[x >> shift];
      if (page < 0 || page >= num_pages) continue;
      at = ((int64_t)page << shift) + (x & ((1 << shift) - 1));
    }
    const float y = ld_in(v, at * stride);
    pos |= y == INFINITY;
    neg |= y == -INFINITY;
    nan |= y != y;
    if (nan || (pos && neg)) break;
  }
  return poison_value(pos, neg, nan);
}

namespace tc {

// descriptor of a 128-byte swizzled operand (see above)
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return sdesc(saddr, lbo, sbo) | ((uint64_t)2 << 61);
}

// D[tmem] (+)= A[tmem] * B[smem], A bf16 in 32-bit columns of two
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 32 columns of 32-bit data (see tmem_ld16 / tmem_st16)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for `parity` of `bar`; false once any wait of the CTA has expired
// (kWaitLimitNs), so that the roles end together.
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_or_dead_slow(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_done(bar, parity)) return true;
    if ((it & 63) == 0) {
      if (*reinterpret_cast<volatile uint32_t*>(dead)) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        *reinterpret_cast<volatile uint32_t*>(dead) = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_or_dead(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  if (mbar_done(bar, parity)) return true;
  if (mbar_done(bar, parity)) return true;  // (each suspends for a while)
  return wait_or_dead_slow(bar, parity, dead);
}

// Tensor-map copies into shared memory, completion counted in bytes on `bar`.
// The innermost coordinate is a multiple of 64 bf16 here (TMA wants 16 bytes).
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* m, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// 2^x with the hardware approximation (relative error about 2^-22), 0 below 2^-126
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 operations per instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// two floats to bf16, `lo` in the low half
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 32 bytes to global memory, in one store (a whole sector) where p is 32-byte aligned
__device__ __forceinline__ void st_32b(void* p, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
// two bf16, each zeroed if it is infinite or NaN
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// which of eight bf16 are infinite or NaN, a bit each
__device__ __forceinline__ uint32_t nonfinite8(uint4 x) {
  auto two = [](uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 1u : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 2u : 0u);
  };
  return two(x.x) | two(x.y) << 2 | two(x.z) << 4 | two(x.w) << 6;
}
// Non-finite bf16 values among the 16-byte pieces [from, live) of the `blocks`
// swizzled blocks of a V tile (`bytes` apart, 64 channels each) become zeros, and
// their channels' bits of `words` are set: the whole warp, where the search found some.
__device__ __forceinline__ void take_out_bf16(char* tile, uint32_t bytes, int blocks, int from, int live,
                                              uint32_t* words) {
  for (int c = 0; c < blocks; ++c) {
    uint4* blk = reinterpret_cast<uint4*>(tile + c * bytes);
#pragma unroll 1
    for (int v = from + (threadIdx.x & 31); v < live; v += 32) {
      const uint4 x = blk[v];
      const uint32_t bad = nonfinite8(x);
      if (!bad) continue;
      const int piece = (v & 7) ^ ((v >> 3) & 7);
      atomicOr_block(&words[2 * c + (piece >> 2)], bad << (8 * (piece & 3)));
      blk[v] = make_uint4(finite_only(x.x), finite_only(x.y), finite_only(x.z), finite_only(x.w));
    }
  }
}
// the search: bits 15 and 31 tell whether one of eight bf16 has an exponent of all
// ones (which carries into the sign's place)
__device__ __forceinline__ uint32_t exponents_full(uint4 x) {
  return ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
         ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
}

// byte offset of 16-byte piece c of row r in swizzled blocks of `block` bytes
__device__ __forceinline__ uint32_t sw_off(int r, int c, uint32_t block) {
  return (uint32_t)(c >> 3) * block + (uint32_t)r * 128u + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// x = h + m + l to fp32 precision, each part bf16: h is x cut to 8 bits (so it
// never overflows), m and l round what is left, |x - h - m - l| <= 2^-23 |x|.
// An infinity or NaN stays in h alone.  Two values at a time.
struct Split {
  uint32_t h, m, l;
};
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ Split split3(float x, float y) {
  Split s;
  const uint32_t bx = __float_as_uint(x) & 0xffff0000u, by = __float_as_uint(y) & 0xffff0000u;
  s.h = (bx >> 16) | by;
  // (a NaN whose payload the cut loses would turn into an infinity)
  if (x != x) s.h |= 0x7fffu;
  if (y != y) s.h |= 0x7fff0000u;
  float rx = x - __uint_as_float(bx), ry = y - __uint_as_float(by);
  rx = rx == rx ? rx : 0.f;
  ry = ry == ry ? ry : 0.f;
  s.m = pack2(rx, ry);
  s.l = pack2(rx - bf_lo(s.m), ry - bf_hi(s.m));
  return s;
}

}  // namespace tc

// Workspace, arguments and launches of the plan and of the joining of pieces.
// row_tiles: of an item; dp: padded channels; kt_shift: log2 of a key tile.
inline bool few_rows(const AttnParams& p) {
  const int64_t rows = p.max_seqlen * p.G;
  return p.block_table &&
         (rows <= kTinyRows || (rows <= kShortRows && ((int64_t)p.max_pages << p.page_shift) <= kShortKeys));
}

TcLayout tc_layout(const AttnParams& p, int row_tiles, int dp);
TcArgs tc_args(const AttnParams& p, const TcLayout& L, int row_tiles, int kt_shift, void* ws);
cudaError_t launch_attn_plan(const AttnParams& p, const TcArgs& a, cudaStream_t stream);
cudaError_t launch_attn_join(const AttnParams& p, const TcArgs& a, int dp, int sms, cudaStream_t stream);

// Tensor map of q, or of K or V as [pages][positions][Hkv][D] (packed: one page
// of all tokens), box {128 bytes of channels, `heads`, `box` positions (, 1
// page)}, 128-byte swizzle; what lies outside reads as zeros.
bool attn_map(CUtensorMap* m, const AttnParams& p, const void* base, bool q, int heads, int box);

bool attn_tc_fits(const AttnParams& p);
size_t attn_tc_workspace(const AttnParams& p);
cudaError_t launch_attn_tc(const AttnParams& p, void* ws, cudaStream_t stream);

bool attn_tc1_fits(const AttnParams& p);
size_t attn_tc1_workspace(const AttnParams& p);
cudaError_t launch_attn_tc1(const AttnParams& p, void* ws, cudaStream_t stream);

bool attn_rows_fits(const AttnParams& p);
size_t attn_rows_workspace(const AttnParams& p);
cudaError_t launch_attn_rows(const AttnParams& p, void* ws, cudaStream_t stream);

}  // namespace kda
