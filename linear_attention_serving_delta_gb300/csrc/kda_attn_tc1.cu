// kda_attn_tc1.cu -- the tensor-core attention with one row tile per CTA: bf16
// heads of 256 channels (whose output fills half of TMEM), and fp32 heads of up
// to 128, whose operands are split into three bf16 parts.
//
// The items, softmax and masks are those of kda_attn_tc.cu; key tiles are 64
// positions.  With one row tile the tensor core is kept busy by S of the next
// key tile, issued before P of this one is waited for, in a second buffer:
//
//   S(j+1) = Q K(j+1)^T   while  P(j) = 2^(x - m)   then  O += P(j) V(j)
//
// fp32: x = h + m + l with bf16 parts (split3), and a product of two operands
// takes the six pairs h h, h m, m h, h l, l h, m m, what is left out being below
// 2^-22 of it.  A warpgroup splits K and V tiles from a staging ring into the
// operands' layout beside the products, the softmax threads split P.
//
// Bound by a chain, not by a unit.  bf16: one warpgroup's TMEM loads, maximum,
// exponentials and TMEM stores of a key tile.  fp32: P V of a tile, its addition
// to the sum, P of the next tile and its P V, one after the other (one P, one V
// and one buffer of what P V gives fit).
//
// Measured on GB300, one prompt of 4096 tokens, 32 query heads over 8: bf16 of
// 256 channels 229 us (1.20 PFLOP/s, the tensor pipe 51% busy), fp32 of 128
// channels 1.02 ms (134 TFLOP/s, 0.81 PFLOP/s of bf16 products, the tensor pipe 34%).
#include "kda_attn_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kKeys = 64;   // positions of a key tile
constexpr int kKeyShift = 6;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazyLog2 = 8.f;
constexpr uint32_t kTmemCols = 512;

template <int NP, int DP>
struct Shape {
  static constexpr int NB = DP / 64;                           // 64-channel blocks of an operand
  static constexpr uint32_t kQBlock = kRowTile * 128;
  static constexpr uint32_t kQPlane = NB * kQBlock;
  static constexpr uint32_t kKBlock = kKeys * 128;
  static constexpr uint32_t kPlane = NB * kKBlock;             // one part of a K or V tile
  static constexpr uint32_t kOperand = NP * kPlane;
  static constexpr int kKStages = NP == 1 ? 2 : DP == 64 ? 2 : 1, kVStages = NP == 1 ? 3 : DP == 64 ? 2 : 1;
  // fp32: tiles arrive as halves of 32 positions, 32 channels to a block
  static constexpr int kHalfKeys = 32, kHalfBlocks = DP / 32;
  static constexpr uint32_t kHalfBlock = kHalfKeys * 128;
  static constexpr uint32_t kHalf = kHalfBlocks * kHalfBlock;
  static constexpr int kHalfStages = NP == 1 ? 0 : DP == 64 ? 6 : 2;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = NP * kQPlane;
  static constexpr uint32_t kV = kK + kKStages * kOperand;
  static constexpr uint32_t kStaging = kV + kVStages * kOperand;
  static constexpr uint32_t kBars = kStaging + kHalfStages * kHalf;
  static constexpr uint32_t kBytes = kBars + 1024;
  static_assert(kBytes <= 232448, "shared memory");
  // TMEM columns: two S, (fp32) P's three parts, what P V gives, (fp32) the sum of it
  static constexpr uint32_t kS = 0, kP = 2 * kKeys, kO = NP == 1 ? 2 * kKeys : 2 * kKeys + 3 * (kKeys / 2),
                            kSum = kO + DP;
  static_assert(kO + (NP == 1 ? 1 : 2) * DP <= kTmemCols, "TMEM");
  static constexpr int kSplitWarps = NP == 1 ? 0 : 4;
  static constexpr int kThreads = 32 * (4 + 3 + kSplitWarps);  // softmax; copies of Q and K, of V, MMAs; splitting
};

// s_full, p_full and pv_done have a barrier for each of the two buffers: the
// softmax may be a tile ahead of P V, and a parity tells two phases apart, not
// three.
struct Bars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], h_full[8], h_empty[8];
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done[2], fix, drain;
  uint32_t dead, tmem;
  OwnPlan plan;
  // the CTA's k-th item with key tiles (index k % 8): the positions past its first
  // token's whose non-finite values were taken out of V, and their channels, a bit
  // each; (fp32) three more rows of bits for the positions that all of its rows
  // attend, the channels with +inf, -inf and NaN there
  int32_t poison_from[8], poison_to[8];
  uint32_t poison_seen[8], poison[8][16];
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

struct Geo {
  int rows, n, kt0;
  int fix_from;  // first key tile with a position some row may not attend, or past the sequence
};
__device__ __forceinline__ Geo geometry(const AttnItem& it, int G) {
  Geo g;
  g.rows = it.ntok * G;
  g.kt0 = it.kt0;
  g.n = it.kt1 - it.kt0;
  g.fix_from = it.pos0 + 1 <= 0 ? 0 : (it.pos0 + 1) / kKeys;
  return g;
}

template <int NP, int DP>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  return __all_sync(0xffffffffu, wait_or_dead(bar, parity, dead)) != 0;
}

// Boxes of one head's positions into blocks of `block` bytes, NBLK blocks of
// 128 bytes of channels (`per` channels each)
template <int NBLK>
__device__ __forceinline__ void copy_boxes(const CUtensorMap* m, char* dst, uint32_t block, int per, const Boxes& bx,
                                           int shift, int h, int lane, uint64_t* bar) {
  const uint32_t box_bytes = 128u << shift;
  if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)max(bx.n, 0) * box_bytes * NBLK);
  __syncwarp();
  if (lane < bx.n)
#pragma unroll
    for (int c = 0; c < NBLK; ++c) tma_4d(dst + c * block + lane * box_bytes, m, per * c, h, bx.c2, bx.c3, bar);
}

// ------------------------------------------------------------------ copies, bf16
template <int DP>
__device__ void load_k_bf16(const AttnParams& p, const TcArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                            char* sm, Bars* b, int64_t total) {
  using S = Shape<1, DP>;
  const int lane = threadIdx.x & 31;
  Ring<S::kKStages> ring;
  uint32_t n = 0, nq = 0;
  bool ok = true;
  for (int i = 0; ok; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) break;
    const AttnItem it = item_at(a, w, p.Hkv);
    const int h = (int)(w % p.Hkv);
    const Geo g = geometry(it, p.G);
    if (g.n <= 0) continue;
    if (!(ok = warp_wait<1, DP>(&b->q_empty, (nq & 1) ^ 1, &b->dead))) break;
    if (lane == 0) {
      mbar_arrive_expect_tx(&b->q_full, (uint32_t)(a.tpt * p.G) * 128u * S::NB);
#pragma unroll
      for (int c = 0; c < S::NB; ++c) tma_3d(sm + S::kQ + c * S::kQBlock, mq, 64 * c, h * p.G, it.tok0, &b->q_full);
    }
    ++nq;
    for (int j = 0; j < g.n; ++j) {
      const Boxes bx = boxes_of(p, it, (g.kt0 + j) * kKeys, kKeys, a.box_shift, lane);
      if (!(ok = warp_wait<1, DP>(&b->k_empty[ring.st], ring.ph ^ 1, &b->dead))) break;
      copy_boxes<S::NB>(mk, sm + S::kK + ring.st * S::kOperand, S::kKBlock, 64, bx, a.box_shift, h, lane,
                        &b->k_full[ring.st]);
      ring.next();
      ++n;
    }
  }
  if (!ok) {  // no copy of its own is in flight when a CTA that gave up exits
    for (uint32_t k = n > S::kKStages ? n - S::kKStages : 0; k < n; ++k)
      mbar_wait(&b->k_full[k % S::kKStages], (k / S::kKStages) & 1, kWaitLimitNs);
    if (nq > 0) mbar_wait(&b->q_full, (nq - 1) & 1, kWaitLimitNs);
  }
}

// (out of line: 4096 tokens of 256 channels 229 us, 236 with it in the loop)
static __device__ __noinline__ void take_out_of(char* tile, uint32_t bytes, int blocks, int from, int live,
                                                uint32_t* words) {
  take_out_bf16(tile, bytes, blocks, from, live, words);
}

template <int DP>
__device__ void load_v_bf16(const AttnParams& p, const TcArgs& a, const CUtensorMap* mv, char* sm, Bars* b,
                            int64_t total) {
  using S = Shape<1, DP>;
  const int lane = threadIdx.x & 31;
  Ring<S::kVStages> ring;
  uint32_t n = 0, nfix = 0, busy = 0;
  bool ok = true;
  for (int i = 0; ok; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) break;
    const AttnItem it = item_at(a, w, p.Hkv);
    const int h = (int)(w % p.Hkv);
    const Geo g = geometry(it, p.G);
    if (g.n <= 0) continue;
    const int slot = busy++ & 7;
    if (lane == 0) b->poison_to[slot] = -1, b->poison_seen[slot] = 0;
    if (lane < 8) b->poison[slot][lane] = 0;  // (before the copies' __syncwarp)
    for (int j = 0; j < g.n; ++j) {
      const int kt = g.kt0 + j, x0 = kt * kKeys;
      const bool fix = kt >= g.fix_from;
      const Boxes bx = boxes_of(p, it, x0, kKeys, a.box_shift, lane);
      char* dst = sm + S::kV + ring.st * S::kOperand;
      if (!(ok = warp_wait<1, DP>(&b->v_empty[ring.st], ring.ph ^ 1, &b->dead))) break;
      copy_boxes<S::NB>(mv, dst, S::kKBlock, 64, bx, a.box_shift, h, lane, fix ? &b->fix : &b->v_full[ring.st]);
      if (fix) {
        ok = warp_wait<1, DP>(&b->fix, nfix & 1, &b->dead);
        ++nfix;
        if (!ok) break;
        // in 16-byte pieces of a block: the rows some row may not attend, and the
        // first that none may (a sequence's later tokens stand there too)
        const int from = max(0, it.pos0 + 1 - x0) * 8,
                  live = min(kKeys, min(it.kv_len, it.pos0 + it.ntok) - x0) * 8;
        uint32_t seen = 0;
#pragma unroll
        for (int c = 0; c < S::NB; ++c) {
          uint4* blk = reinterpret_cast<uint4*>(dst + c * S::kKBlock);
#pragma unroll 4
          for (int v = from + lane; v < live; v += 32) seen |= exponents_full(blk[v]);
          for (int v = live + lane; v < kKeys * 8; v += 32) blk[v] = make_uint4(0, 0, 0, 0);
        }
        const bool bad = __any_sync(0xffffffffu, (seen & 0x80008000u) != 0);
        if (bad) take_out_of(dst, S::kKBlock, S::NB, from, live, b->poison[slot]);
        if (bad && lane == 0) {
          if (b->poison_to[slot] < 0) b->poison_from[slot] = max(x0, it.pos0 + 1);
          b->poison_to[slot] = x0 + kKeys - 1;
          b->poison_seen[slot] = 1;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->v_full[ring.st]);
      }
      ring.next();
      ++n;
    }
  }
  if (!ok) {
    for (uint32_t k = n > S::kVStages ? n - S::kVStages : 0; k < n; ++k)
      mbar_wait(&b->v_full[k % S::kVStages], (k / S::kVStages) & 1, kWaitLimitNs);
    if (nfix > 0) mbar_wait(&b->fix, (nfix - 1) & 1, kWaitLimitNs);
  }
}

// ------------------------------------------------------------------ copies and splitting, fp32
// The order in which an item's tiles are taken: K 0, then K j + 1 and V j for
// each j (the order of their MMAs).  f(tile of K or V, which) until it says no.
template <typename F>
__device__ __forceinline__ bool tiles_in_order(int n, F f) {
  if (!f(0, false)) return false;
  for (int j = 0; j < n; ++j) {
    if (j + 1 < n && !f(j + 1, false)) return false;
    if (!f(j, true)) return false;
  }
  return true;
}

template <int DP>
__device__ void load_f32(const AttnParams& p, const TcArgs& a, const CUtensorMap* mk, const CUtensorMap* mv, char* sm,
                         Bars* b, int64_t total) {
  using S = Shape<3, DP>;
  const int lane = threadIdx.x & 31;
  Ring<S::kHalfStages> ring;
  uint32_t n = 0;
  bool ok = true;
  const int shift = min(a.box_shift, 5);
  for (int i = 0; ok; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) break;
    const AttnItem it = item_at(a, w, p.Hkv);
    const int h = (int)(w % p.Hkv);
    const Geo g = geometry(it, p.G);
    if (g.n <= 0) continue;
    ok = tiles_in_order(g.n, [&](int j, bool v) {
      for (int half = 0; half < 2; ++half) {
        const int x0 = (g.kt0 + j) * kKeys + half * S::kHalfKeys;
        const Boxes bx = boxes_of(p, it, x0, S::kHalfKeys, shift, lane);
        if (!warp_wait<3, DP>(&b->h_empty[ring.st], ring.ph ^ 1, &b->dead)) return false;
        copy_boxes<S::kHalfBlocks>(v ? mv : mk, sm + S::kStaging + ring.st * S::kHalf, S::kHalfBlock, 32, bx, shift, h,
                                   lane, &b->h_full[ring.st]);
        ring.next();
        ++n;
      }
      return true;
    });
  }
  if (!ok)
    for (uint32_t k = n > (uint32_t)S::kHalfStages ? n - S::kHalfStages : 0; k < n; ++k)
      mbar_wait(&b->h_full[k % S::kHalfStages], (k / S::kHalfStages) & 1, kWaitLimitNs);
}

// The non-finite values of half a tile of fp32 V, noted by the thread that took them
// out (slow path): rows below `live` of the staged half from position x0 on; pos0: the
// last position that all rows attend.
template <int DP>
static __device__ __noinline__ void note_poison(Bars* b, int slot, const char* in, int tid, int x0, int live, int pos0) {
  using S = Shape<3, DP>;
#pragma unroll 1
  for (int z = tid; z < S::kHalfKeys * DP / 8; z += 128) {
    const int r = z % S::kHalfKeys, x = x0 + r;
    if (r >= live) continue;
#pragma unroll 1
    for (int u = 0; u < 8; ++u) {
      const int ch = z / S::kHalfKeys * 8 + u;
      const float y = *reinterpret_cast<const float*>(in + sw_off(r, ch >> 2, S::kHalfBlock) + (ch & 3) * 4);
      if ((__float_as_uint(y) & 0x7f800000u) != 0x7f800000u) continue;
      *reinterpret_cast<volatile uint32_t*>(&b->poison_seen[slot]) = 1;
      if (x <= pos0) {
        atomicOr_block(&b->poison[slot][4 + 4 * poison_kind(y) + (ch >> 5)], 1u << (ch & 31));
      } else {
        atomicOr_block(&b->poison[slot][ch >> 5], 1u << (ch & 31));
        atomicMin_block(&b->poison_from[slot], x);
        atomicMax_block(&b->poison_to[slot], x);
      }
    }
  }
}

// The four splitting warps: Q's rows, then the tiles, from fp32 into three
// bf16 operands.  V: zeros behind the sequence, non-finite values taken out.
template <int DP>
__device__ void split_role(const AttnParams& p, const TcArgs& a, char* sm, Bars* b, int64_t total, int tid) {
  using S = Shape<3, DP>;
  const int lane = tid & 31;
  Ring<S::kHalfStages> ring;
  Ring<S::kKStages> kr;
  Ring<S::kVStages> vr;
  uint32_t nq = 0, busy = 0;
  for (int i = 0;; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) return;
    const AttnItem it = item_at(a, w, p.Hkv);
    const int h = (int)(w % p.Hkv);
    const Geo g = geometry(it, p.G);
    if (g.n <= 0) continue;
    // The word of a later item is made ready here: the staging ring keeps the
    // warps within two items of one another, so it is long before its use.
    const int slot = busy & 7;
    if (tid == 0) {
      b->poison_from[(busy + 3) & 7] = INT32_MAX;
      b->poison_to[(busy + 3) & 7] = -1;
      b->poison_seen[(busy + 3) & 7] = 0;
    }
    if (tid < 16) b->poison[(busy + 3) & 7][tid] = 0;
    ++busy;
    if (!warp_wait<3, DP>(&b->q_empty, (nq & 1) ^ 1, &b->dead)) return;
    ++nq;
    const float* q = static_cast<const float*>(p.q);
    constexpr int C8 = DP / 8;  // a thread takes eight channels of a row
#pragma unroll 2
    for (int z = tid; z < kRowTile * C8; z += 128) {
      const int r = z / C8, c = 8 * (z % C8);
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (r < g.rows && c < p.D) {
        const float* src = q + ((int64_t)(it.tok0 + r / p.G) * p.H + (int64_t)h * p.G + r % p.G) * p.D + c;
        const float4 y0 = reinterpret_cast<const float4*>(src)[0], y1 = reinterpret_cast<const float4*>(src)[1];
        x[0] = y0.x; x[1] = y0.y; x[2] = y0.z; x[3] = y0.w;
        x[4] = y1.x; x[5] = y1.y; x[6] = y1.z; x[7] = y1.w;
      }
      Split s[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] = split3(x[2 * u], x[2 * u + 1]);
      char* dst = sm + S::kQ + sw_off(r, c >> 3, S::kQBlock);
      *reinterpret_cast<uint4*>(dst) = make_uint4(s[0].h, s[1].h, s[2].h, s[3].h);
      *reinterpret_cast<uint4*>(dst + S::kQPlane) = make_uint4(s[0].m, s[1].m, s[2].m, s[3].m);
      *reinterpret_cast<uint4*>(dst + 2 * S::kQPlane) = make_uint4(s[0].l, s[1].l, s[2].l, s[3].l);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->q_full);
    const bool ok = tiles_in_order(g.n, [&](int j, bool v) {
      uint64_t* empty = v ? &b->v_empty[vr.st] : &b->k_empty[kr.st];
      uint64_t* full = v ? &b->v_full[vr.st] : &b->k_full[kr.st];
      if (!warp_wait<3, DP>(empty, (v ? vr.ph : kr.ph) ^ 1, &b->dead)) return false;
      char* out = sm + (v ? S::kV + vr.st * S::kOperand : S::kK + kr.st * S::kOperand);
      for (int half = 0; half < 2; ++half) {
        const int x0 = (g.kt0 + j) * kKeys + half * S::kHalfKeys;
        if (!warp_wait<3, DP>(&b->h_full[ring.st], ring.ph, &b->dead)) return false;
        const char* in = sm + S::kStaging + ring.st * S::kHalf;
        const int live = it.kv_len - x0;
        int seen = 0;
#pragma unroll 2
        for (int z = tid; z < S::kHalfKeys * C8; z += 128) {
          // lanes along the rows: 16-byte pieces of eight swizzled rows meet no bank twice
          const int r = z % S::kHalfKeys, c = z / S::kHalfKeys;
          float x[8];
          const float4 y0 = *reinterpret_cast<const float4*>(in + sw_off(r, 2 * c, S::kHalfBlock));
          const float4 y1 = *reinterpret_cast<const float4*>(in + sw_off(r, 2 * c + 1, S::kHalfBlock));
          x[0] = y0.x; x[1] = y0.y; x[2] = y0.z; x[3] = y0.w;
          x[4] = y1.x; x[5] = y1.y; x[6] = y1.z; x[7] = y1.w;
          if (v) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              if (r >= live) x[u] = 0.f;
              if ((__float_as_uint(x[u]) & 0x7f800000u) == 0x7f800000u) {
                x[u] = 0.f;
                seen = 1;
              }
            }
          }
          Split s[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) s[u] = split3(x[2 * u], x[2 * u + 1]);
          char* dst = out + sw_off(half * S::kHalfKeys + r, c, S::kKBlock);
          *reinterpret_cast<uint4*>(dst) = make_uint4(s[0].h, s[1].h, s[2].h, s[3].h);
          *reinterpret_cast<uint4*>(dst + S::kPlane) = make_uint4(s[0].m, s[1].m, s[2].m, s[3].m);
          *reinterpret_cast<uint4*>(dst + 2 * S::kPlane) = make_uint4(s[0].l, s[1].l, s[2].l, s[3].l);
        }
        if (seen) note_poison<DP>(b, slot, in, tid, x0, live, it.pos0);
        fence_async_smem();  // reads of the staging before its next copy, writes before the MMAs
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->h_empty[ring.st]);
        ring.next();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
      if (v) vr.next();
      else kr.next();
      return true;
    });
    if (!ok) return;
  }
}

// ------------------------------------------------------------------ MMAs
template <int NP, int DP>
__device__ void mma_role(const AttnParams& p, const TcArgs& a, char* sm, Bars* b, int64_t total) {
  using S = Shape<NP, DP>;
  const uint32_t tmem = __shfl_sync(0xffffffffu, b->tmem, 0);
  constexpr uint32_t id_qk = idesc_bf16(kRowTile, kKeys), id_pv = idesc_bf16(kRowTile, DP, 0, 1);
  const uint64_t q0 = sdesc_sw128(smem_u32(sm + S::kQ), 16, 1024), k0 = sdesc_sw128(smem_u32(sm + S::kK), 16, 1024),
                 v0 = sdesc_sw128(smem_u32(sm + S::kV), S::kKBlock, 1024);
  // the pairs of parts of a product, the smallest first
  constexpr int kPairs = NP == 1 ? 1 : 6;
  constexpr int pa[6] = {0, 2, 1, 0, 1, 0}, pb[6] = {2, 0, 1, 1, 0, 0};
  const bool issue = elect_one();
  Ring<S::kKStages> kr;
  Ring<S::kVStages> vr;
  uint32_t nq = 0, np = 0;
  uint32_t* dead = &b->dead;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_dead(bar, parity, dead)) != 0;
  };
  auto commit = [&](uint64_t* bar) {
    if (issue) mma_commit(bar);
  };
  auto qk = [&](int buf) {
    const uint64_t kd = k0 + (uint64_t)(kr.st * (S::kOperand >> 4));
    if (issue) {
#pragma unroll
      for (int z = 0; z < kPairs; ++z) {
        const int x = NP == 1 ? 0 : pa[z], y = NP == 1 ? 0 : pb[z];
#pragma unroll
        for (int s = 0; s < DP / 16; ++s)
          mma_bf16(tmem + S::kS + buf * kKeys,
                   q0 + ((x * S::kQPlane + (s / 4) * S::kQBlock + (s % 4) * 32) >> 4),
                   kd + ((y * S::kPlane + (s / 4) * S::kKBlock + (s % 4) * 32) >> 4), id_qk, z > 0 || s > 0);
      }
      mma_commit(&b->s_full[buf]);
      mma_commit(&b->k_empty[kr.st]);
    }
    kr.next();
  };
  auto pv = [&](int buf, bool first) {
    const uint64_t vd = v0 + (uint64_t)(vr.st * (S::kOperand >> 4));
    const uint32_t tp = tmem + (NP == 1 ? S::kS + buf * kKeys : S::kP);
    if (issue) {
#pragma unroll
      for (int z = 0; z < kPairs; ++z) {
        const int x = NP == 1 ? 0 : pa[z], y = NP == 1 ? 0 : pb[z];
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)
          mma_bf16_ts(tmem + S::kO, tp + x * (kKeys / 2) + s * 8, vd + ((y * S::kPlane + s * 2048) >> 4), id_pv,
                      !first || z > 0 || s > 0);
      }
      mma_commit(&b->v_empty[vr.st]);
      mma_commit(&b->pv_done[buf]);
    }
    vr.next();
  };
  bool ok = true;
  for (int i = 0; ok; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) break;
    const AttnItem it = item_at(a, w, p.Hkv);
    const Geo g = geometry(it, p.G);
    if (g.n <= 0) continue;
    if (!(ok = wait(&b->q_full, nq & 1))) break;
    ++nq;
    if (!(ok = wait(&b->k_full[kr.st], kr.ph))) break;
    fence_after_sync();
    // (S and P of the last item are done with: its last P V was waited for by its softmax)
    qk(np & 1);
    if (g.n == 1) commit(&b->q_empty);
    for (int j = 0; j < g.n; ++j) {
      if (j + 1 < g.n) {
        if (!(ok = wait(&b->k_full[kr.st], kr.ph))) break;
        fence_after_sync();
        qk((np + 1) & 1);
        if (j + 2 == g.n) commit(&b->q_empty);
      }
      if (!(ok = wait(&b->v_full[vr.st], vr.ph))) break;
      if (!(ok = wait(&b->p_full[np & 1], (np >> 1) & 1))) break;
      fence_after_sync();
      pv(np & 1, NP == 3 || j == 0);
      ++np;
    }
  }
  // no MMA and no arrival of one is left in flight
  commit(&b->drain);
  mbar_wait(&b->drain, 0, kWaitLimitNs);
}

// ------------------------------------------------------------------ softmax and outputs
template <int NP, int DP>
__device__ void softmax_role(const AttnParams& p, const TcArgs& a, Bars* b, int64_t total) {
  using S = Shape<NP, DP>;
  using T = typename std::conditional<NP == 1, __nv_bfloat16, float>::type;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x;
  uint32_t* dead = &b->dead;
  const uint32_t base = b->tmem + ((uint32_t)(warp * 32) << 16);
  const float sc = p.scale * kLog2e;
  uint32_t np = 0, busy_items = 0;
  // P V of the CTA's k-th key tile is done
  auto pv_wait = [&](uint32_t k) {
    const bool ok = __all_sync(0xffffffffu, wait_or_dead(&b->pv_done[k & 1], (k >> 1) & 1, dead));
    fence_after_sync();
    return ok;
  };
  for (int i = 0;; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) return;
    const AttnItem it = item_at(a, w, p.Hkv);
    const int h = (int)(w % p.Hkv);
    const Geo g = geometry(it, p.G);
    const int slot = busy_items & 7, n = max(g.n, 0);
    busy_items += n > 0;
    const int tok = row / p.G;
    const int limit = it.pos0 + tok;
    const bool busy = warp * 32 < g.rows;  // a warp without rows only keeps step
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j, ++np) {
      const int buf = np & 1;
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->s_full[buf], (np >> 1) & 1, dead))) return;
      fence_after_sync();
      if (busy) {
        float s[kKeys];
        tmem_ld32(base + S::kS + buf * kKeys, s);
        tmem_ld32(base + S::kS + buf * kKeys + 32, s + 32);
        tmem_ld_wait();
        const int kt = g.kt0 + j;
        if (kt >= g.fix_from) {
          const int last = min(limit, it.kv_len - 1) - kt * kKeys;
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c] = c <= last ? s[c] : -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kKeys; c += 4)
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], s[c + u]);
        const float x = sc * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        float sum[2] = {0.f, 0.f};
        if constexpr (NP == 1) {
          // the reference moves with the first finite maximum, then only past the threshold
          const bool move = x > m + kLazyLog2 || (m == -INFINITY && x > m);
          const bool scale_o = move && m != -INFINITY;
          if (__any_sync(0xffffffffu, scale_o)) {
            // O as P V of the tile before leaves it
            if (!pv_wait(np - 1)) return;
            const float f = scale_o ? exp2_fast(m - x) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
              float o[32];
              tmem_ld32(base + S::kO + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 32; ++u) o[u] *= f;
              tmem_st32(base + S::kO + c, reinterpret_cast<const uint32_t*>(o));
            }
          }
          if (move) m = x;
          const float ref = m == -INFINITY ? 0.f : m;
          uint32_t pk[kKeys / 2];
#pragma unroll
          for (int u = 0; u < kKeys / 2; ++u) {
            const float e0 = exp2_fast(fmaf(s[2 * u], sc, -ref)), e1 = exp2_fast(fmaf(s[2 * u + 1], sc, -ref));
            sum[u & 1] += e0 + e1;
            pk[u] = pack2(e0, e1);
          }
          tmem_st32(base + S::kS + buf * kKeys, pk);
        } else {
          const float mn = x > m ? x : m, ref = mn == -INFINITY ? 0.f : mn;
          const float f = m == -INFINITY ? 1.f : exp2f(m - mn);
          m = mn;
          l *= f;
#pragma unroll
          for (int u = 0; u < kKeys; ++u) {
            s[u] = exp2f(fmaf(s[u], sc, -ref));
            sum[u & 1] += s[u];
          }
          if (j > 0) {
            // what P V gave for the tile before, added up rounded to nearest: the
            // tensor core's own accumulation cuts, a bias that grows with the keys
            if (!pv_wait(np - 1)) return;
#pragma unroll 1
            for (int c = 0; c < DP; c += 16) {
              float o[16], y[16];
              tmem_ld16(base + S::kO + c, y);
              if (j > 1) tmem_ld16(base + S::kSum + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] = (j > 1 ? o[u] + y[u] : y[u]) * f;
              tmem_st16(base + S::kSum + c, o);
            }
          }
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t ph[16], pm[16], pl[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const Split y = split3(s[c + 2 * u], s[c + 2 * u + 1]);
              ph[u] = y.h;
              pm[u] = y.m;
              pl[u] = y.l;
            }
            const uint32_t to = base + S::kP + c / 2;
            tmem_st16(to, reinterpret_cast<const float*>(ph));
            tmem_st16(to + kKeys / 2, reinterpret_cast<const float*>(pm));
            tmem_st16(to + kKeys, reinterpret_cast<const float*>(pl));
          }
        }
        l += sum[0] + sum[1];
        tmem_st_wait();
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->p_full[buf]);
    }
    // o = O / l, or the piece's O with its m and l
    if (n > 0 && !pv_wait(np - 1)) return;
    if (busy) {
      const bool poison = n > 0 && *reinterpret_cast<volatile uint32_t*>(&b->poison_seen[slot]) != 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int gq = row - tok * p.G;
      const bool live = row < g.rows;
      const int64_t orow = ((int64_t)(it.tok0 + tok) * p.H + (int64_t)h * p.G + gq) * p.D;
      const int64_t prow = it.slot < 0 ? 0 : ((int64_t)it.slot * p.Hkv + h) * kRowTile + row;
#pragma unroll 1
      for (int c = 0; c < DP; c += 32) {
        float x[32];
        if (n > 0) {
          tmem_ld32(base + S::kO + c, x);
          tmem_ld_wait();
          if (NP == 3 && n > 1) {
            float y[32];
            tmem_ld32(base + S::kSum + c, y);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 32; ++u) x[u] += y[u];
          }
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) x[u] = 0.f;
        }
        if (live && c < p.D) {
          const float f = it.slot < 0 ? inv : 1.f;
#pragma unroll
          for (int u = 0; u < 32; ++u) x[u] *= f;
          if (poison) {
            const volatile uint32_t* bits = b->poison[slot] + (c >> 5);
            const uint32_t some = bits[0];  // channels with such values that some rows attend
            uint32_t all[3] = {0, 0, 0};    // and that all rows do
            if (NP == 3)
#pragma unroll
              for (int z = 0; z < 3; ++z) all[z] = bits[4 + 4 * z];
            const int from = *reinterpret_cast<volatile int32_t*>(&b->poison_from[slot]),
                      to = min(*reinterpret_cast<volatile int32_t*>(&b->poison_to[slot]),
                               min(limit, min(it.kv_len, it.kt1 * kKeys) - 1));
            const int64_t stride = (int64_t)p.Hkv * p.D;
            const T* v = static_cast<const T*>(p.v) + (int64_t)h * p.D + c + (p.block_table ? 0 : it.base * stride);
            const int32_t* pages = p.block_table ? p.block_table + (int64_t)it.base * p.max_pages : nullptr;
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              float z = poison_value(all[0] >> u & 1, all[1] >> u & 1, all[2] >> u & 1);
              if (some >> u & 1) z += poison_of(v + u, stride, pages, p.num_pages, p.page_shift, from, to);
              if (z != 0.f) x[u] += z;  // a NaN already there stays
            }
          }
          if (it.slot >= 0) {
            float* part = a.part_o + prow * DP + c;
#pragma unroll
            for (int u = 0; u < 32; u += 8) st_32b(part + u, reinterpret_cast<const uint32_t*>(x + u), true);
          } else if constexpr (NP == 1) {
            uint32_t pk[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) pk[u] = pack2(x[2 * u], x[2 * u + 1]);
            T* o = static_cast<T*>(p.o) + orow + c;
#pragma unroll
            for (int u = 0; u < 16; u += 8)
              if (c + 2 * u < p.D) st_32b(o + 2 * u, pk + u, a.o_wide);
          } else {
            T* o = static_cast<T*>(p.o) + orow + c;
#pragma unroll
            for (int u = 0; u < 32; u += 8)
              if (c + u < p.D) st_32b(o + u, reinterpret_cast<const uint32_t*>(x + u), a.o_wide);
          }
        }
        __syncwarp();
      }
      if (live && it.slot >= 0) a.part_ml[prow] = make_float2(m, l);
    }
    // these reads of O come before the arrival that lets the next item's P V write it
    fence_before_sync();
  }
}

template <int NP, int DP>
__global__ void __launch_bounds__(Shape<NP, DP>::kThreads, 1)
    attn_tc1(const AttnParams p, const TcArgs a, const __grid_constant__ CUtensorMap mq,
             const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Shape<NP, DP>;
  extern __shared__ __align__(1024) char sm[];
  Bars* b = reinterpret_cast<Bars*>(sm + S::kBars);
  const int warp = threadIdx.x >> 5;
  constexpr uint32_t kFill = NP == 1 ? 1 : 4;  // arrivals that fill an operand: a copy's, or the splitting warps'
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&b->k_full[s], kFill);
      mbar_init(&b->k_empty[s], 1);
      mbar_init(&b->v_full[s], kFill);
      mbar_init(&b->v_empty[s], 1);
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(&b->h_full[s], 1);
      mbar_init(&b->h_empty[s], 4);
    }
    mbar_init(&b->q_full, kFill);
    mbar_init(&b->q_empty, 1);
    mbar_init(&b->s_full[0], 1);
    mbar_init(&b->s_full[1], 1);
    mbar_init(&b->p_full[0], 4);
    mbar_init(&b->p_full[1], 4);
    mbar_init(&b->pv_done[0], 1);
    mbar_init(&b->pv_done[1], 1);
    mbar_init(&b->fix, 1);
    mbar_init(&b->drain, 1);
    for (int s = 0; s < 8; ++s) {
      b->poison_from[s] = INT32_MAX;
      b->poison_to[s] = -1;
      b->poison_seen[s] = 0;
    }
    b->dead = 0;
    b->plan.own = 0;
    mbar_init_fence();
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + 8 * 16) (&b->poison[0][0])[threadIdx.x - 64] = 0;
  if (threadIdx.x == 32) {
    if (NP == 1) prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
  }
  if (warp == 5) tmem_alloc(&b->tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  pdl_wait();  // the plan, or what came before
  const int64_t total = a.self_plan ? (plan_own_item<S::kThreads>(p, a, &b->plan) ? blockIdx.x + 1 : 0)
                                    : (int64_t)a.head->items * p.Hkv;
  if (warp < 4) softmax_role<NP, DP>(p, a, b, total);
  else if (warp == 5) mma_role<NP, DP>(p, a, sm, b, total);
  else if constexpr (NP == 1) {
    if (warp == 4) load_k_bf16<DP>(p, a, &mq, &mk, sm, b, total);
    else load_v_bf16<DP>(p, a, &mv, sm, b, total);
  } else {
    if (warp == 4) load_f32<DP>(p, a, &mk, &mv, sm, b, total);
    else if (warp >= 7) split_role<DP>(p, a, sm, b, total, threadIdx.x - 32 * 7);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && b->dead) attn_flag(p.status, kFlagTimeout);
  if (warp == 5) tmem_dealloc(b->tmem, kTmemCols);
}

template <int NP, int DP>
cudaError_t launch_np(const AttnParams& p, void* ws, cudaStream_t stream) {
  using S = Shape<NP, DP>;
  const TcLayout L = tc_layout(p, 1, DP);
  TcArgs a = tc_args(p, L, 1, kKeyShift, ws);
  const int box = 1 << (NP == 1 || a.box_shift < 5 ? a.box_shift : 5);
  CUtensorMap mq, mk, mv;
  if (!attn_map(&mq, p, p.q, true, p.G, a.tpt) || !attn_map(&mk, p, p.k, false, 1, box) ||
      !attn_map(&mv, p, p.v, false, 1, box))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  auto kernel = attn_tc1<NP, DP>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
  a.self_plan = L.self_plan && L.max_items * p.Hkv <= sms;
  if (e == cudaSuccess && !a.self_plan) e = launch_attn_plan(p, a, stream);
  if (e != cudaSuccess) return e;
  const int64_t most = (L.max_items + L.max_pieces) * p.Hkv;
  e = launch_maybe_dependent(true, kernel, dim3((unsigned)(most < sms ? most : sms)), dim3(S::kThreads),
                             (size_t)S::kBytes, stream, p, a, mq, mk, mv);
  return e != cudaSuccess || !L.split ? e : launch_attn_join(p, a, DP, sms, stream);
}

}  // namespace

// bf16 heads of 256 channels and fp32 heads of up to 128, where a request may
// have more rows than the streaming kernel's blocks hold (it takes the others);
// otherwise as attn_tc_fits.
bool attn_tc1_fits(const AttnParams& p) {
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  const bool shape = p.dt == KDA_BF16 ? p.D == 256 : p.D <= 128;
  return shape && p.max_seqlen * p.G > kFewRows && p.scale > 0.f && p.scale <= 3.4e38f && al16(p.q) && al16(p.k) &&
         al16(p.v) && al16(p.o) && (!p.block_table || p.num_pages > 0);
}
size_t attn_tc1_workspace(const AttnParams& p) {
  return tc_layout(p, 1, p.dt == KDA_BF16 ? 256 : p.D <= 64 ? 64 : 128).total;
}
cudaError_t launch_attn_tc1(const AttnParams& p, void* ws, cudaStream_t stream) {
  if (p.dt == KDA_BF16) return launch_np<1, 256>(p, ws, stream);
  return p.D <= 64 ? launch_np<3, 64>(p, ws, stream) : launch_np<3, 128>(p, ws, stream);
}

}  // namespace kda
