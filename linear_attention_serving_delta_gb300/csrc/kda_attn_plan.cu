// kda_attn_plan.cu -- the plan of the tensor-core attention (items from the
// device-side lengths, costliest first, long ones cut into pieces), the
// joining of the pieces, its workspace and its tensor maps.
#include "kda_attn_tc.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 2560;
constexpr int kPlanSeqs = 640;

// costs up to 255 keep their own bucket, larger ones their seven leading bits
__device__ __forceinline__ int bucket_of(int cost) {
  if (cost < 256) return cost;
  const int e = 31 - __clz(cost) - 7;
  return (e << 7) + (cost >> e);
}

__device__ int64_t plan_scan(int64_t x, int64_t* part, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t y = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    part[lane] = y;
  }
  __syncthreads();
  if (warp > 0) x += part[warp - 1];
  *total = part[31];
  __syncthreads();
  return x;
}

// One CTA: the items of the call from the device-side lengths, sorted by
// their key tiles, costliest first.  When they are too few to fill the GPU
// (split_sms > 0) an item's key tiles are cut into pieces of about equal
// share, and the list of what to join is left for attn_join.
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const AttnParams p, const TcArgs a) {
  __shared__ int64_t part[32];
  __shared__ int hist[kBuckets];
  __shared__ unsigned long long cost_sum;
  __shared__ AttnSeq sm_seq[kPlanSeqs];       // the sequences, for batches of up to kPlanSeqs
  __shared__ int32_t sm_begin[kPlanSeqs];
  const int tid = threadIdx.x, tpi = a.row_tiles * a.tpt;
  const bool near = p.num_seqs <= kPlanSeqs;
  pdl_launch_dependents();
  pdl_wait();
  for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
  if (tid == 0) cost_sum = 0;
  // the sequences' tiles and their prefix sums
  int64_t n_tiles = 0;
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int s = base + tid;
    int64_t n = 0, total;
    AttnSeq q{};
    if (s < p.num_seqs) {
      q = attn_seq(p, s);
      if (q.flag) attn_flag(p.status, q.flag);
      n = ((int64_t)q.len + tpi - 1) / tpi;
    }
    const int64_t end = plan_scan(n, part, &total);
    if (s < p.num_seqs) {
      if (near) {
        sm_seq[s] = q;
        sm_begin[s] = (int32_t)min(n_tiles + end - n, (int64_t)INT32_MAX);  // (past max_items: not looked up)
      } else {
        a.seq_begin[s] = n_tiles + end - n;
      }
    }
    n_tiles += total;
  }
  n_tiles = min(n_tiles, a.max_items);
  __syncthreads();
  auto tile_item = [&](int64_t x) {
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((near ? (int64_t)sm_begin[mid] : a.seq_begin[mid]) <= x) lo = mid; else hi = mid - 1;
    }
    return near ? make_item(p, a, sm_seq[lo], x - sm_begin[lo])
                : make_item(p, a, attn_seq(p, lo), x - a.seq_begin[lo]);
  };
  const bool split = a.split_sms > 0 && n_tiles * p.Hkv < 2 * (int64_t)a.split_sms;
  int piece = INT32_MAX;
  if (split) {
    unsigned long long c = 0;
    for (int64_t x = tid; x < n_tiles; x += kPlanThreads) c += (unsigned long long)tile_item(x).kt1;
    if (c) atomicAdd(&cost_sum, c);
    __syncthreads();
    const int64_t parts = (int64_t)kPiecesPerSm * a.split_sms;
    const int64_t share = ((int64_t)cost_sum * p.Hkv + parts - 1) / parts;
    piece = (int)max((int64_t)kMinPiece, share);
  }
  // pieces of an item: how many, and each one's key tiles
  // (to the nearest; the CTAs need not come out even: 64 like items of 258 key
  // tiles give 320 pieces, three for some of 152 CTAs and two for the others)
  auto pieces = [&](const AttnItem& it) { return split ? max(1, (int)(((int64_t)it.kt1 * 2 + piece) / (2 * (int64_t)piece))) : 1; };
  for (int64_t x = tid; x < n_tiles; x += kPlanThreads) {
    const AttnItem it = tile_item(x);
    const int np = pieces(it);
    for (int k = 0; k < np; ++k) {
      const int64_t k0 = (int64_t)it.kt1 * k / np, k1 = (int64_t)it.kt1 * (k + 1) / np;
      atomicAdd(&hist[bucket_of((int)(k1 - k0))], 1);
    }
  }
  __syncthreads();
  // hist[b] becomes the first place of bucket b: costlier buckets go first.
  // A thread sums kBuckets / kPlanThreads neighbours.
  constexpr int kPer = (kBuckets + kPlanThreads - 1) / kPlanThreads;
  int mine[kPer];
  int64_t n = 0, total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int bkt = kBuckets - 1 - (tid * kPer + i);
    mine[i] = bkt >= 0 ? hist[bkt] : 0;
    n += mine[i];
  }
  int64_t at = plan_scan(n, part, &total) - n;
  const int64_t items = total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int bkt = kBuckets - 1 - (tid * kPer + i);
    if (bkt >= 0) hist[bkt] = (int)at;
    at += mine[i];
  }
  __syncthreads();
  int64_t slots = 0, joins = 0;
  for (int64_t base = 0; base < n_tiles; base += kPlanThreads) {
    const int64_t x = base + tid;
    AttnItem it{};
    int np = 0;
    if (x < n_tiles) {
      it = tile_item(x);
      np = pieces(it);
    }
    int64_t slot0 = 0, join = 0;
    if (split) {  // partial results in tile order, whatever the order of the atomics below
      const int64_t cut = np > 1 ? np : 0;
      slot0 = slots + plan_scan(cut, part, &total) - cut;
      slots += total;
      const int64_t one = np > 1;
      join = joins + plan_scan(one, part, &total) - one;
      joins += total;
    }
    if (np > 1) a.joins[join] = AttnJoin{it.tok0, it.ntok, (int32_t)slot0, np};
    const int kt1 = it.kt1;
    for (int k = 0; k < np; ++k) {
      it.kt0 = (int)((int64_t)kt1 * k / np);
      it.kt1 = (int)((int64_t)kt1 * (k + 1) / np);
      it.slot = np > 1 ? (int32_t)(slot0 + k) : -1;
      a.items[atomicAdd(&hist[bucket_of(it.kt1 - it.kt0)], 1)] = it;
    }
  }
  if (tid == 0) {
    a.head->items = (int32_t)items;
    a.head->joins = (int32_t)joins;
  }
}

// The pieces of a cut item joined: with M = max m_k, o = sum 2^(m_k - M) O_k /
// sum 2^(m_k - M) l_k, in piece order.  A warp per row.
template <typename T, int DP>
__global__ void __launch_bounds__(256) attn_join(const AttnParams p, const TcArgs a) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = a.row_tiles * kRowTile;
  const int64_t work = (int64_t)a.head->joins * p.Hkv * (rows / 8);
  constexpr int V = DP / 32;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int64_t pair = w / (rows / 8);
    const AttnJoin jn = a.joins[pair / p.Hkv];
    const int h = (int)(pair % p.Hkv), r = (int)(w % (rows / 8)) * 8 + warp;
    const int t = r / kRowTile, row = r % kRowTile, tok = t * a.tpt + row / p.G;
    if (row >= a.tpt * p.G || tok >= jn.ntok) continue;
    auto at = [&](int k) { return ((int64_t)(jn.slot + k) * p.Hkv + h) * rows + r; };
    float M = -INFINITY;
    for (int k = lane; k < jn.pieces; k += 32) M = fmaxf(M, a.part_ml[at(k)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;
    float l = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
#pragma unroll 2
    for (int k = 0; k < jn.pieces; ++k) {
      const float2 ml = a.part_ml[at(k)];
      const float f = exp2f(ml.x - M);
      l += f * ml.y;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = fmaf(f, a.part_o[at(k) * DP + v * 32 + lane], o[v]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t out = ((int64_t)(jn.tok0 + tok) * p.H + (int64_t)h * p.G + row % p.G) * p.D;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane < p.D) st_out(static_cast<T*>(p.o), out + v * 32 + lane, o[v] * inv);
  }
}

template <typename T>
cudaError_t join_t(const AttnParams& p, const TcArgs& a, int dp, dim3 grid, cudaStream_t stream) {
  auto kernel = dp == 64 ? attn_join<T, 64> : dp == 128 ? attn_join<T, 128> : attn_join<T, 256>;
  return launch_maybe_dependent(true, kernel, grid, dim3(256), 0, stream, p, a);
}

}  // namespace

TcLayout tc_layout(const AttnParams& p, int row_tiles, int dp) {
  TcLayout L{};
  const int tpi = row_tiles * (kRowTile / p.G);
  L.max_items = (p.total_tokens + tpi - 1) / tpi + p.num_seqs;
  // pieces only where the whole batch cannot fill the GPU: at most two per SM
  // are whole items, and the cuts add kPiecesPerSm
  L.split = p.block_table && (p.total_tokens + tpi - 1) / tpi * p.Hkv < 2 * kSplitSms;
  // a call whose items cannot outnumber the SMs plans for itself, unless long
  // key ranges are better cut
  const int64_t keys = p.block_table ? (int64_t)p.max_pages << p.page_shift : p.total_tokens;
  L.self_plan = L.max_items * p.Hkv <= kSplitSms && (!L.split || keys <= kSelfPlanKeys);
  if (L.self_plan) L.split = false;
  L.max_pieces = L.split ? (2 + kPiecesPerSm) * (int64_t)kSplitSms / p.Hkv + 1 : 0;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.head = take(sizeof(AttnHead));
  L.seq_begin = take(sizeof(int64_t) * p.num_seqs);
  L.items = take(sizeof(AttnItem) * (size_t)(L.self_plan ? L.max_items * p.Hkv : L.max_items + L.max_pieces));
  if (L.split) {
    L.joins = take(sizeof(AttnJoin) * (size_t)(2 * kSplitSms));
    const size_t rows = (size_t)L.max_pieces * p.Hkv * row_tiles * kRowTile;
    L.ml = take(rows * sizeof(float2));
    L.o = take(rows * dp * sizeof(float));
  }
  L.total = off;
  return L;
}

TcArgs tc_args(const AttnParams& p, const TcLayout& L, int row_tiles, int kt_shift, void* ws) {
  char* w = static_cast<char*>(ws);
  TcArgs a{};
  a.head = reinterpret_cast<AttnHead*>(w + L.head);
  a.seq_begin = reinterpret_cast<int64_t*>(w + L.seq_begin);
  a.items = reinterpret_cast<AttnItem*>(w + L.items);
  a.max_items = L.max_items;
  a.row_tiles = row_tiles;
  a.tpt = kRowTile / p.G;
  a.kt_shift = kt_shift;
  a.box_shift = p.block_table && p.page_shift < kt_shift ? p.page_shift : kt_shift;
  a.o_wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
  if (L.split) {
    a.split_sms = kSplitSms;
    a.joins = reinterpret_cast<AttnJoin*>(w + L.joins);
    a.part_ml = reinterpret_cast<float2*>(w + L.ml);
    a.part_o = reinterpret_cast<float*>(w + L.o);
  }
  return a;
}

cudaError_t launch_attn_plan(const AttnParams& p, const TcArgs& a, cudaStream_t stream) {
  return launch_maybe_dependent(true, attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p, a);
}
cudaError_t launch_attn_join(const AttnParams& p, const TcArgs& a, int dp, int sms, cudaStream_t stream) {
  const dim3 grid((unsigned)(16 * sms));
  return p.dt == KDA_BF16 ? join_t<__nv_bfloat16>(p, a, dp, grid, stream) : join_t<float>(p, a, dp, grid, stream);
}

bool attn_map(CUtensorMap* m, const AttnParams& p, const void* base, bool q, int heads, int box) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const bool half = p.dt == KDA_BF16, paged = !q && p.block_table;
  const cuuint64_t es = half ? 2 : 4, page = paged ? (cuuint64_t)1 << p.page_shift : (cuuint64_t)p.total_tokens;
  const cuuint64_t nh = q ? p.H : p.Hkv, row = nh * p.D * es;
  const cuuint64_t dims[4] = {(cuuint64_t)p.D, nh, page, paged ? (cuuint64_t)p.num_pages : 1};
  const cuuint64_t strides[3] = {p.D * es, row, row * page};
  const cuuint32_t bx[4] = {(cuuint32_t)(128 / es), (cuuint32_t)heads, (cuuint32_t)box, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return enc(m, half ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, q ? 3 : 4,
             const_cast<void*>(base), dims, strides, bx, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kda
