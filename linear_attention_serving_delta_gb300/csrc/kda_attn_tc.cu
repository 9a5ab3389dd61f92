// kda_attn_tc.cu -- causal attention with grouped heads on the tcgen05 tensor
// cores: bf16, heads of up to 128 channels, packed prompts or the paged cache.
//
// Rows.  The rows of a key head's G query heads are packed, row = token * G +
// head, so that one pass over K and V serves them all.  An item is two row
// tiles of 128 rows (floor(128 / G) tokens each) of one (sequence, key head),
// or a piece of its keys; a persistent CTA per SM takes items, the costliest
// first (attn_plan_kernel sorts them).
//
// Per key tile of 128 positions and row tile, with the logits in base 2,
// x = (scale / ln 2) q.k:
//
//   S = Q K^T            tcgen05, fp32 in TMEM
//   m' = max(m, max x)   l = l 2^(m - m') + sum 2^(x - m')     one thread a row
//   P = 2^(x - m')       rounded to bf16, into S's columns of TMEM
//   O = O 2^(m - m') + P V   tcgen05, A from TMEM
//
// The reference m of a row follows its maximum only once weights taken against
// the old one would pass 2^kLazyLog2 (the same relative rounding): most tiles
// need no rescaling pass over O, and of their first half not even the maximum.
// o = O / l at the end, so the choice changes no result beyond rounding.
//
// Warps: 0-3 and 4-7 hold the softmax of the two row tiles (thread = row =
// TMEM lane), 9 and 10 issue the MMAs of one row tile each, 8 copies Q and K, 11
// V.  While one tile's softmax runs, the tensor core works on the other tile.
// The MMAs of a row tile are issued by one thread and execute in issue order, so S of
// the next key tile may be issued right behind the P V that reads P from the
// same columns.
//
// Masked places.  Logits past a row's position are replaced by -inf before
// they are used, so K may hold anything there.  V meets weights of exactly 0,
// which would still turn infinities and NaN into NaN: a key tile that ends
// behind the sequence has its remaining V rows zeroed in shared memory, and
// in a tile with positions that some row of the item may not attend,
// non-finite values of V are zeroed too; the epilogue then puts them back
// into the rows that do attend them (a slow path no finite input takes).
//
// Bound by the tensor core and by the softmax between S and P V.  Measured on
// GB300: one prompt of 8192 tokens, 32 query heads over 8 of 128 channels, 355 us
// call after call (1.55 PFLOP/s), 328 us with pauses (1.68, the tensor pipe 74%
// busy); 182k tokens of 8 prompts 24.5 ms (1.44 PFLOP/s under the power cap).
#include "kda_attn_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kTile = 128;       // rows of a row tile, positions of a key tile
constexpr int kThreads = 384;    // two softmax warpgroups; copies and MMAs
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFirst = kTile / 2;  // positions of P handed over first
constexpr float kLazyLog2 = 8.f;
constexpr float kLazySum = 256.f;  // 2^kLazyLog2
constexpr uint32_t kTmemCols = 512;

template <int DP>
struct Shape {
  static constexpr int NH = DP / 64;                        // 128-byte column blocks of a tile
  static constexpr uint32_t kBlock = kTile * 128;           // bytes of one block
  static constexpr uint32_t kTileBytes = NH * kBlock;
  // V's ring is one deeper: some of its tiles are put right in place before use
  static constexpr int kKStages = DP == 128 ? 2 : 4, kVStages = DP == 128 ? 3 : 4;
  static constexpr uint32_t kQ = 0;                         // two row tiles
  static constexpr uint32_t kK = 2 * kTileBytes;
  static constexpr uint32_t kV = kK + kKStages * kTileBytes;
  static constexpr uint32_t kBars = kV + kVStages * kTileBytes;
  static constexpr uint32_t kBytes = kBars + 512;
};

struct Bars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2];
  uint64_t fix, drain[2];
  uint32_t dead;      // a wait expired: every role winds down
  OwnPlan plan;
  uint32_t turn;      // held by the MMA warp whose burst is being issued
  uint32_t tmem;
  // the CTA's k-th item with key tiles: the channels in which non-finite values
  // were taken out of its V tiles, a bit each (index k % 8; V's ring lets the copies
  // begin at most five such items ahead of the epilogue)
  uint32_t poison[8][4];
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// What every role derives from an item
struct Geo {
  int rows[2];   // valid rows of each row tile
  int n[2];      // key tiles of each
  int nmax;
  int kt0;       // first key tile
  int fix_from;  // first key tile with a position some row may not attend, or past the sequence
};
__device__ __forceinline__ Geo geometry(const AttnItem& it, int G, int tpt) {
  Geo g;
  g.kt0 = it.kt0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int tok = min(tpt, max(0, it.ntok - t * tpt));
    g.rows[t] = tok * G;
    const int end = tok > 0 ? max(0, min(it.kv_len, it.pos0 + t * tpt + tok)) : 0;
    g.n[t] = max(0, min(it.kt1, (end + kTile - 1) / kTile) - it.kt0);
  }
  g.nmax = max(g.n[0], g.n[1]);
  const int first = it.pos0 + 1;
  g.fix_from = first <= 0 ? 0 : first / kTile;
  return g;
}

// ------------------------------------------------------------------ copies
template <int DP>
__device__ __forceinline__ void copy_boxes(const CUtensorMap* m, char* dst, const Boxes& bx, int shift, int h, int lane,
                                           uint64_t* bar) {
  using S = Shape<DP>;
  const uint32_t box_bytes = 128u << shift;
  if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)bx.n * box_bytes * S::NH);
  __syncwarp();
  if (lane < bx.n)
#pragma unroll
    for (int c = 0; c < S::NH; ++c) tma_4d(dst + c * S::kBlock + lane * box_bytes, m, 64 * c, h, bx.c2, bx.c3, bar);
}

// Q's row tiles and K
template <int DP>
__device__ void load_k_role(const AttnParams& p, const TcArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                            char* sm, Bars* b, int64_t total, int tpt) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  Ring<S::kKStages> ring;
  uint32_t n = 0, nq[2] = {0, 0};
  bool ok = true;
  for (int i = 0; ok; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) break;
    const AttnItem it = item_at(a, w, p.Hkv);
    const int h = (int)(w % p.Hkv);
    const Geo g = geometry(it, p.G, tpt);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (g.n[t] == 0 || !ok) continue;
      ok = __all_sync(0xffffffffu, wait_or_dead(&b->q_empty[t], (nq[t] & 1) ^ 1, &b->dead));
      if (!ok) continue;
      if (lane == 0) {
        mbar_arrive_expect_tx(&b->q_full[t], (uint32_t)(tpt * p.G) * 128u * S::NH);
#pragma unroll
        for (int c = 0; c < S::NH; ++c)
          tma_3d(sm + S::kQ + t * S::kTileBytes + c * S::kBlock, mq, 64 * c, h * p.G, it.tok0 + t * tpt,
                 &b->q_full[t]);
      }
      ++nq[t];
    }
    for (int j = 0; j < g.nmax && ok; ++j) {
      const Boxes bx = boxes_of(p, it, (g.kt0 + j) * kTile, kTile, a.box_shift, lane);
      ok = __all_sync(0xffffffffu, wait_or_dead(&b->k_empty[ring.st], ring.ph ^ 1, &b->dead));
      if (!ok) break;
      copy_boxes<DP>(mk, sm + S::kK + ring.st * S::kTileBytes, bx, a.box_shift, h, lane, &b->k_full[ring.st]);
      ring.next();
      ++n;
    }
  }
  // no copy of its own is in flight when a CTA that gave up exits
  if (!ok) {
    for (uint32_t k = n > S::kKStages ? n - S::kKStages : 0; k < n; ++k)
      mbar_wait(&b->k_full[k % S::kKStages], (k / S::kKStages) & 1, kWaitLimitNs);
    for (int t = 0; t < 2; ++t)
      if (nq[t] > 0) mbar_wait(&b->q_full[t], (nq[t] - 1) & 1, kWaitLimitNs);
  }
}

// V, and what has to be put right in it
template <int DP>
__device__ void load_v_role(const AttnParams& p, const TcArgs& a, const CUtensorMap* mv, char* sm, Bars* b,
                            int64_t total, int tpt) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  Ring<S::kVStages> ring;
  uint32_t n = 0, nfix = 0, busy_items = 0;
  bool ok = true;
  for (int i = 0; ok; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) break;
    const AttnItem it = item_at(a, w, p.Hkv);
    const int h = (int)(w % p.Hkv);
    const Geo g = geometry(it, p.G, tpt);
    if (g.nmax == 0) continue;
    uint32_t* poison = b->poison[busy_items++ & 7];
    if (lane < 4) poison[lane] = 0;  // (before the copies' __syncwarp)
    for (int j = 0; j < g.nmax; ++j) {
      const int kt = g.kt0 + j, x0 = kt * kTile;
      const bool fix = kt >= g.fix_from;
      const Boxes bx = boxes_of(p, it, x0, kTile, a.box_shift, lane);
      char* dst = sm + S::kV + ring.st * S::kTileBytes;
      ok = __all_sync(0xffffffffu, wait_or_dead(&b->v_empty[ring.st], ring.ph ^ 1, &b->dead));
      if (!ok) break;
      copy_boxes<DP>(mv, dst, bx, a.box_shift, h, lane, fix ? &b->fix : &b->v_full[ring.st]);
      if (fix) {
        // in place: rows behind the sequence to zero, non-finite values out
        ok = __all_sync(0xffffffffu, wait_or_dead(&b->fix, nfix & 1, &b->dead));
        ++nfix;
        if (!ok) break;
        // in 16-byte pieces of a block: the rows some row may not attend, the end of the sequence
        // (an item holds two tokens where its sequence does: one of a single token is the sequence's last)
        const int from = max(0, it.pos0 + 1 - x0) * 8, live = min(kTile, it.kv_len - x0) * 8;
        uint32_t seen = 0;
#pragma unroll
        for (int c = 0; c < S::NH; ++c) {
          uint4* blk = reinterpret_cast<uint4*>(dst + c * S::kBlock);
          if (it.ntok > 1) {
#pragma unroll 8
            for (int v = from + lane; v < live; v += 32) seen |= exponents_full(blk[v]);
          }
          for (int v = live + lane; v < kTile * 8; v += 32) blk[v] = make_uint4(0, 0, 0, 0);
        }
        if (__any_sync(0xffffffffu, (seen & 0x80008000u) != 0))
          take_out_bf16(dst, S::kBlock, S::NH, from, live, poison);
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

// ------------------------------------------------------------------ MMAs
// A warp for each row tile: what one waits for, the other's MMAs cover (a wait
// behind S's MMAs costs the tensor core 50-100 cycles when one warp issues
// both tiles' work).  The whole warp walks the items, so that descriptors stay
// in uniform registers; one lane issues.
template <int DP>
__device__ void mma_role(const AttnParams& p, const TcArgs& a, char* sm, Bars* b, int64_t total, int tpt, int t) {
  using S = Shape<DP>;
  const uint32_t tmem = __shfl_sync(0xffffffffu, b->tmem, 0);
  const uint32_t ts = tmem + t * kTile, to = tmem + 2 * kTile + t * DP;
  constexpr uint32_t id_qk = idesc_bf16(kTile, kTile), id_pv = idesc_bf16(kTile, DP, 0, 1);
  const uint64_t qd = sdesc_sw128(smem_u32(sm + S::kQ + t * S::kTileBytes), 16, 1024),
                 k0 = sdesc_sw128(smem_u32(sm + S::kK), 16, 1024),
                 v0 = sdesc_sw128(smem_u32(sm + S::kV), S::kBlock, 1024);
  const bool issue = elect_one();
  Ring<S::kKStages> kr;
  Ring<S::kVStages> vr;
  uint32_t nq = 0, np = 0;
  uint32_t* dead = &b->dead;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_dead(bar, parity, dead)) != 0;
  };
  // this row tile's share of a stage is done: with its MMAs, or at once
  auto release = [&](uint64_t* empty, bool used) {
    if (issue) {
      if (used) mma_commit(empty);
      else mbar_arrive(empty);
    }
  };
  auto give = [&] {
    if (issue) atomicExch_block(&b->turn, 0u);
  };
  auto qk = [&](uint32_t stage, bool held) {
    const uint64_t kd = k0 + (uint64_t)(stage * (S::kTileBytes >> 4));
    if (issue) {
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        const uint32_t off = ((s / 4) * S::kBlock + (s % 4) * 32) >> 4;
        mma_bf16(ts, qd + off, kd + off, id_qk, s > 0);
      }
      if (held) give();
      mma_commit(&b->s_full[t]);
    }
  };
  // P V over the first kFirst positions of the key tile, or the others
  auto pv = [&](uint32_t stage, bool rest, bool first) {
    const uint64_t vd = v0 + (uint64_t)(stage * (S::kTileBytes >> 4));
    if (issue) {
      if (!rest) {
#pragma unroll
        for (int s = 0; s < kFirst / 16; ++s)
          mma_bf16_ts(to, ts + s * 8, vd + s * (2048 >> 4), id_pv, !first || s > 0);
      } else {
#pragma unroll
        for (int s = kFirst / 16; s < kTile / 16; ++s) mma_bf16_ts(to, ts + s * 8, vd + s * (2048 >> 4), id_pv, 1);
      }
    }
  };
  // One row tile's burst (P V, then S of the next key tile) at a time: bursts
  // that interleave end together, and so do the softmaxes behind them, each
  // slower for the other (8192 tokens, 32 heads of 128: 368 us, 418 without).
  // If the holder waits for P's second half and gives up, so does the other.
  auto take = [&] {
    bool mine = true;
    if (issue) {
      uint64_t t0 = 0;
      for (uint32_t it = 0; atomicCAS_block(&b->turn, 0u, 1u) != 0u; ++it) {
        if (it == 0) t0 = globaltimer_ns();
        else if ((it & 63) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
          *reinterpret_cast<volatile uint32_t*>(dead) = 1;
          mine = false;
          break;
        }
      }
    }
    return __all_sync(0xffffffffu, mine) != 0;
  };
  bool ok = true;
  for (int i = 0; ok; ++i) {
    const int64_t w = nth_item(i);
    if (w >= total) break;
    const AttnItem it = item_at(a, w, p.Hkv);
    const Geo g = geometry(it, p.G, tpt);
    const int n = t == 0 ? g.n[0] : g.n[1];
    if (g.nmax == 0) continue;
    if (!(ok = wait(&b->k_full[kr.st], kr.ph))) break;
    if (n > 0) {
      if (!(ok = wait(&b->q_full[t], nq & 1))) break;
      ++nq;
      fence_after_sync();
      qk(kr.st, false);
      if (n == 1 && issue) mma_commit(&b->q_empty[t]);
    }
    release(&b->k_empty[kr.st], n > 0);
    kr.next();
    for (int j = 0; j < g.nmax; ++j) {
      if (!(ok = wait(&b->v_full[vr.st], vr.ph))) break;
      const bool more = j + 1 < g.nmax;
      if (more && !(ok = wait(&b->k_full[kr.st], kr.ph))) break;
      if (j < n) {
        if (!(ok = wait(&b->p_half[t], np & 1))) break;
        if (!(ok = take())) break;
        fence_after_sync();
        pv(vr.st, false, j == 0);
        if (!(ok = wait(&b->p_full[t], np & 1))) break;
        ++np;
        fence_after_sync();
        pv(vr.st, true, false);
        if (j + 1 < n) {
          release(&b->v_empty[vr.st], true);
          qk(kr.st, true);
          if (j + 2 == n && issue) mma_commit(&b->q_empty[t]);
        } else {
          give();
          if (issue) mma_commit(&b->o_full[t]);
          release(&b->v_empty[vr.st], true);
        }
      } else {
        release(&b->v_empty[vr.st], false);
      }
      vr.next();
      if (more) {
        release(&b->k_empty[kr.st], j + 1 < n);
        kr.next();
      }
    }
  }
  // no MMA and no arrival of one is left in flight
  if (issue) mma_commit(&b->drain[t]);
  mbar_wait(&b->drain[t], 0, kWaitLimitNs);
}

// ------------------------------------------------------------------ softmax and outputs
template <int DP>
__device__ void softmax_role(const AttnParams& p, const TcArgs& a, Bars* b, int64_t total, int tpt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = warp >> 2, row = (warp & 3) * 32 + lane;
  uint32_t* dead = &b->dead;
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_col = b->tmem + lanes + t * kTile, o_col = b->tmem + lanes + 2 * kTile + t * DP;
  const float sc = p.scale * kLog2e;
  uint32_t ns = 0, no = 0, busy_items = 0;
  AttnItem ahead{};  // the next item, read during the one before
  int h_ahead = 0;
  auto fetch = [&](int64_t w) {
    if (w < total) {
      ahead = item_at(a, w, p.Hkv);
      h_ahead = (int)(w % p.Hkv);
    }
  };
  fetch(nth_item(0));
  for (int i = 0;; ++i) {
    if (nth_item(i) >= total) return;
    const AttnItem it = ahead;
    const int h = h_ahead;
    fetch(nth_item(i + 1));
    const Geo g = geometry(it, p.G, tpt);
    const int rows = g.rows[t], n = g.n[t];
    const uint32_t* poisoned = b->poison[busy_items & 7];
    busy_items += g.nmax > 0;
    if (rows == 0) continue;
    const int tok = row / p.G;  // within the row tile
    const int limit = it.pos0 + t * tpt + tok;
    const int mask_from = it.pos0 + t * tpt + 1 <= 0 ? 0 : (it.pos0 + t * tpt + 1) / kTile;
    const bool busy = (warp & 3) * 32 < rows;  // a warp without rows only keeps step
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->s_full[t], ns & 1, dead))) return;
      ++ns;
      fence_after_sync();
      if (busy) {
        float s[kTile];
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tmem_ld32(s_col + c, s + c);
        tmem_ld_wait();
        const int kt = g.kt0 + j;
        if (kt >= mask_from) {
          const int last = min(limit, it.kv_len - 1) - kt * kTile;
#pragma unroll
          for (int c = 0; c < kTile; ++c) s[c] = c <= last ? s[c] : -INFINITY;
        }
        // The first half's weights against the old reference, beside the
        // maximum of the second half.  If their sum, or that maximum, has
        // risen too far for some row of the warp, they are taken again (the
        // first tile, and seldom after), and the reference of that row moves: of
        // no other one, which may be another token's, or none's with whatever
        // shared memory held for its query.
        uint32_t pk[kFirst / 2];
        float2 sum[2];
        sum[0] = sum[1] = make_float2(0.f, 0.f);
        auto weight = [&](const float* y, int u, float2 sc2, float2 ref2) {
          float2 e = fma2(make_float2(y[2 * u], y[2 * u + 1]), sc2, ref2);
          e.x = exp2_fast(e.x);
          e.y = exp2_fast(e.y);
          sum[u & 1] = add2(sum[u & 1], e);
          pk[u] = pack2(e.x, e.y);
        };
        const float2 sc2 = make_float2(sc, sc);
        float2 ref2 = make_float2(-m, -m);
        if (m == -INFINITY) ref2 = make_float2(0.f, 0.f);
        float mx[4] = {s[kFirst], s[kFirst + 1], s[kFirst + 2], s[kFirst + 3]};
#pragma unroll
        for (int u = 0; u < kFirst / 2; ++u) {
          weight(s, u, sc2, ref2);
          mx[u & 3] = fmaxf(mx[u & 3], fmaxf(s[kFirst + 2 * u], s[kFirst + 2 * u + 1]));
        }
        const float x2 = sc * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float s1 = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        // (a sum that is no number, or an infinite one, asks for the maximum too)
        const bool far = !(s1 <= kLazySum) || x2 > m + kLazyLog2 || m == -INFINITY;
        if (__any_sync(0xffffffffu, far)) {
#pragma unroll
          for (int u = 0; u < kFirst / 2; ++u) mx[u & 3] = fmaxf(mx[u & 3], fmaxf(s[2 * u], s[2 * u + 1]));
          const float x = sc * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool move = far && x > m;
          const bool scale_o = move && m != -INFINITY;
          if (__any_sync(0xffffffffu, scale_o)) {
            const float f = scale_o ? exp2_fast(m - x) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
              float o[32];
              tmem_ld32(o_col + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 32; ++u) o[u] *= f;
              tmem_st32(o_col + c, reinterpret_cast<const uint32_t*>(o));
            }
          }
          if (move) {
            m = x;
            ref2 = make_float2(-m, -m);
          }
          sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
          for (int u = 0; u < kFirst / 2; ++u) weight(s, u, sc2, ref2);
        }
        tmem_st32(s_col, pk);
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->p_half[t]);
#pragma unroll
        for (int u = 0; u < (kTile - kFirst) / 2; ++u) weight(s + kFirst, u, sc2, ref2);
        tmem_st32(s_col + 32, pk);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_st_wait();
      } else {
        if (lane == 0) mbar_arrive(&b->p_half[t]);
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->p_full[t]);
    }
    // o = O / l, or the piece's O with its m and l
    if (n > 0) {
      if (!__all_sync(0xffffffffu, wait_or_dead(&b->o_full[t], no & 1, dead))) return;
      ++no;
      fence_after_sync();
    }
    if (!busy) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int gq = row - tok * p.G;
    const bool mine = row < rows;
    const int64_t orow = ((int64_t)(it.tok0 + t * tpt + tok) * p.H + (int64_t)h * p.G + gq) * p.D;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + orow;
    const int64_t prow = it.slot < 0 ? 0 : ((int64_t)it.slot * p.Hkv + h) * (2 * kTile) + t * kTile + row;
#pragma unroll 1
    for (int c = 0; c < DP; c += 32) {
      float x[32];
      if (n > 0) {
        tmem_ld32(o_col + c, x);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] = 0.f;
      }
      if (mine && c < p.D) {
        const float f = it.slot < 0 ? inv : 1.f;
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] *= f;
        const uint32_t poison = n > 0 ? reinterpret_cast<const volatile uint32_t*>(poisoned)[c >> 5] : 0;
        if (poison) {
          const int from = max(g.kt0 * kTile, it.pos0 + 1), to = min(limit, min(it.kv_len, it.kt1 * kTile) - 1);
          const int64_t stride = (int64_t)p.Hkv * p.D;
          const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + (int64_t)h * p.D + c +
                                   (p.block_table ? 0 : it.base * stride);
          const int32_t* pages = p.block_table ? p.block_table + (int64_t)it.base * p.max_pages : nullptr;
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            if (!(poison >> u & 1)) continue;
            const float y = poison_of(v + u, stride, pages, p.num_pages, p.page_shift, from, to);
            if (y != 0.f) x[u] += y;  // a NaN already there stays
          }
        }
        if (it.slot < 0) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) pk[u] = pack2(x[2 * u], x[2 * u + 1]);
#pragma unroll
          for (int u = 0; u < 16; u += 8)
            if (c + 2 * u < p.D) st_32b(o + c + 2 * u, pk + u, a.o_wide);
        } else {
          float* part = a.part_o + prow * DP + c;
#pragma unroll
          for (int u = 0; u < 32; u += 4) *reinterpret_cast<float4*>(part + u) = make_float4(x[u], x[u + 1], x[u + 2], x[u + 3]);
        }
      }
      __syncwarp();
    }
    if (mine && it.slot >= 0) a.part_ml[prow] = make_float2(m, l);
    // these reads of O come before the arrival that lets the next item's P V write it
    fence_before_sync();
  }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc(const AttnParams p, const TcArgs a, const __grid_constant__ CUtensorMap mq,
            const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Shape<DP>;
  extern __shared__ __align__(1024) char sm[];
  Bars* b = reinterpret_cast<Bars*>(sm + S::kBars);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&b->k_full[s], 1);
      mbar_init(&b->k_empty[s], 2);
      mbar_init(&b->v_full[s], 1);
      mbar_init(&b->v_empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&b->drain[t], 1);
      mbar_init(&b->q_full[t], 1);
      mbar_init(&b->q_empty[t], 1);
      mbar_init(&b->s_full[t], 1);
      mbar_init(&b->p_half[t], 4);
      mbar_init(&b->p_full[t], 4);
      mbar_init(&b->o_full[t], 1);
    }
    mbar_init(&b->fix, 1);
    b->dead = 0;
    b->plan.own = 0;
    b->turn = 0;
    mbar_init_fence();
  }
  if (threadIdx.x == 32) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
  }
  if (warp == 9) tmem_alloc(&b->tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  pdl_wait();  // the plan, or what came before
  const int tpt = kTile / p.G;
  const int64_t total =
      a.self_plan ? (plan_own_item<kThreads>(p, a, &b->plan) ? blockIdx.x + 1 : 0) : (int64_t)a.head->items * p.Hkv;
  // registers: 168 a thread at launch (384 x 168 = 64,512); a softmax thread
  // holds a row of 128 logits: 2 x 128 x 208 + 128 x 80 = 63,488
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax_role<DP>(p, a, b, total, tpt);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 8) load_k_role<DP>(p, a, &mq, &mk, sm, b, total, tpt);
    else if (warp == 11) load_v_role<DP>(p, a, &mv, sm, b, total, tpt);
    else mma_role<DP>(p, a, sm, b, total, tpt, warp - 9);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && b->dead) attn_flag(p.status, kFlagTimeout);
  if (warp == 9) tmem_dealloc(b->tmem, kTmemCols);
}

// ------------------------------------------------------------------ host
constexpr int kKeyShift = 7;  // log2 of kTile
int padded(int D) { return D <= 64 ? 64 : 128; }

template <int DP>
cudaError_t launch_dp(const AttnParams& p, const TcLayout& L, void* ws, cudaStream_t stream) {
  using S = Shape<DP>;
  TcArgs a = tc_args(p, L, 2, kKeyShift, ws);
  CUtensorMap mq, mk, mv;
  if (!attn_map(&mq, p, p.q, true, p.G, a.tpt) || !attn_map(&mk, p, p.k, false, 1, 1 << a.box_shift) ||
      !attn_map(&mv, p, p.v, false, 1, 1 << a.box_shift))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_tc<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t most = (L.max_items + L.max_pieces) * p.Hkv;
  a.self_plan = L.self_plan && L.max_items * p.Hkv <= sms;
  if (a.self_plan)
    return launch_maybe_dependent(true, attn_tc<DP>, dim3((unsigned)(L.max_items * p.Hkv)), dim3(kThreads),
                                  (size_t)S::kBytes, stream, p, a, mq, mk, mv);
  e = launch_attn_plan(p, a, stream);
  if (e != cudaSuccess) return e;
  e = launch_maybe_dependent(true, attn_tc<DP>, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads),
                             (size_t)S::kBytes, stream, p, a, mq, mk, mv);
  return e != cudaSuccess || !L.split ? e : launch_attn_join(p, a, DP, sms, stream);
}

}  // namespace

// bf16, up to 128 channels (narrower heads run zero-padded to 64 or 128 by the
// copies), a positive finite scale (the running maximum is taken before the
// scaling), and what the tensor maps need: 16-byte aligned bases and indices
// inside int32.  Everything else runs on the CUDA cores.
bool attn_tc_fits(const AttnParams& p) {
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  return p.dt == KDA_BF16 && p.D <= 128 && p.scale > 0.f && p.scale <= 3.4e38f && al16(p.q) && al16(p.k) &&
         al16(p.v) && al16(p.o) && (!p.block_table || p.num_pages > 0);
}
size_t attn_tc_workspace(const AttnParams& p) { return tc_layout(p, 2, padded(p.D)).total; }
cudaError_t launch_attn_tc(const AttnParams& p, void* ws, cudaStream_t stream) {
  const TcLayout L = tc_layout(p, 2, padded(p.D));
  return p.D <= 64 ? launch_dp<64>(p, L, ws, stream) : launch_dp<128>(p, L, ws, stream);
}

}  // namespace kda
