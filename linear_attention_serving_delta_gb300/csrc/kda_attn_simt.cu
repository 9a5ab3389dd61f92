// kda_attn_simt.cu -- causal attention with grouped heads on fp32 CUDA cores,
// over packed prompts or the paged cache: every dtype, head size and
// alignment the ABI takes.
//
// A CTA takes kRows rows of one (sequence, key head).  The rows of a key
// head's G query heads are packed, row = token * G + head, so one pass over K
// and V serves them all.  It walks the keys in tiles of BN and keeps, per
// row, the running maximum m of the logits and the sum l of 2^(x - m) with
// x = scale q.k / ln 2; a tile that raises m scales l and the accumulated
// output by 2^(m_old - m_new).  At the end o = acc / l.
//
// Bound by the FMA units: 16 x 16 threads, each a 4 x (BN / 16) patch of the
// scores and 4 x (D / 16) of the output, so an operand read from shared
// memory feeds 4 or more FMAs.
#include <type_traits>

#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kRows = 64;
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// Tile `idx` of the call, counted over the sequences' tiles of `per` tokens:
// its sequence, and the tile's index in it.  Executed by the whole block.
struct TileRef {
  int32_t seq;
  int64_t tile;
};
__device__ TileRef find_tile(const AttnParams& p, int64_t idx, int per, int64_t* sh) {
  // sh: 16 int64 in shared memory
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t before = 0;
  for (int base = 0; base < p.num_seqs; base += kThreads) {
    const int s = base + tid;
    int64_t n = 0;
    if (s < p.num_seqs) n = ((int64_t)attn_seq(p, s).len + per - 1) / per;
    int64_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = x;
    if (tid == 0) sh[8] = -1;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) x += sh[w];
      total += sh[w];
    }
    const int64_t begin = before + x - n;
    if (n > 0 && idx >= begin && idx < begin + n) {
      sh[8] = s;
      sh[9] = idx - begin;
    }
    __syncthreads();
    if (sh[8] >= 0) return TileRef{(int32_t)sh[8], sh[9]};
    before += total;
  }
  return TileRef{-1, 0};
}

template <typename T, int D>
struct SimtShape {
  static constexpr int BN = D == 256 ? 32 : 64;
  static constexpr int LD = kRows + 4;  // row stride of the transposed tiles, floats
  static constexpr int LK = BN + 4;
  static constexpr int Q = 0;                    // [D][LD]
  static constexpr int K = Q + D * LD;           // [D][LK]
  static constexpr int V = K + D * LK;           // [BN][D]
  static constexpr int P = V + BN * D;           // [BN][LD]
  static constexpr int FLOATS = P + BN * LD;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_simt(AttnParams p) {
  using S = SimtShape<T, D>;
  constexpr int BN = S::BN, NC = BN / 16, DC = D / 16;
  extern __shared__ float sm[];
  __shared__ int64_t sh[16];
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int G = p.G, per = kRows / G > 0 ? kRows / G : 1;
  // (G > kRows: a tile is kRows of one token's G rows)
  const int parts = (G + kRows - 1) / kRows;
  const int part = blockIdx.x % parts;
  if (blockIdx.x == 0 && blockIdx.y == 0)  // flags of malformed sequences, which have no tiles
    for (int s = tid; s < p.num_seqs; s += kThreads) {
      const int32_t flag = attn_seq(p, s).flag;
      if (flag) attn_flag(p.status, flag);
    }
  const TileRef ref = find_tile(p, blockIdx.x / parts, per, sh);
  if (ref.seq < 0) return;
  const AttnSeq sq = attn_seq(p, ref.seq);
  const int64_t t0 = ref.tile * per;
  const int ntok = (int)min((int64_t)per, sq.len - t0);
  const int nrows = min(kRows, ntok * G - part * kRows);  // rows of this tile
  const int kvh = blockIdx.y;
  const T* q = static_cast<const T*>(p.q);
  const T* k = static_cast<const T*>(p.k);
  const T* v = static_cast<const T*>(p.v);

  // packed row r of the tile: token and query head
  auto row_off = [&](int r) -> int64_t {
    const int x = r + part * kRows, t = x / G, g = x - t * G;
    return ((sq.tok0 + t0 + t) * p.H + (int64_t)kvh * G + g) * D;
  };
  for (int i = tid; i < kRows * D; i += kThreads) {
    const int r = i / D, d = i - r * D;
    sm[S::Q + d * S::LD + r] = r < nrows ? ld_in(q, row_off(r) + d) : 0.f;
  }
  const float sc = p.scale * kLog2e;
  // position of the tile's first token, and the last position of its last
  const int64_t pos0 = sq.kv_len - sq.len + t0;
  const int64_t kv_end = min(sq.kv_len, pos0 + ntok);
  int64_t limit[4];  // last position each of this thread's rows attends
#pragma unroll
  for (int i = 0; i < 4; ++i) limit[i] = pos0 + min(4 * ty + i + part * kRows, ntok * G - 1) / G;
  float m[4], l[4], acc[4][DC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DC; ++c) acc[i][c] = 0.f;
  }
  for (int64_t j0 = 0; j0 < kv_end; j0 += BN) {
    __syncthreads();
    const int nk = (int)min((int64_t)BN, kv_end - j0);
    for (int i = tid; i < BN * D; i += kThreads) {
      const int j = i / D, d = i - j * D;
      float kx = 0.f, vx = 0.f;
      if (j < nk) {
        int64_t at = sq.tok0 + j0 + j;
        bool ok = true;
        if (p.block_table) {
          const int64_t x = j0 + j;
          const int32_t page = p.block_table[(int64_t)sq.row * p.max_pages + (x >> p.page_shift)];
          ok = page >= 0 && page < p.num_pages;
          at = ((int64_t)page << p.page_shift) + (x & (((int64_t)1 << p.page_shift) - 1));
          if (!ok) attn_flag(p.status, kFlagBadCache);
        }
        if (ok) {
          at = (at * p.Hkv + kvh) * D + d;
          kx = ld_in(k, at);
          vx = ld_in(v, at);
        }
      }
      sm[S::K + d * S::LK + j] = kx;
      sm[S::V + j * D + d] = vx;
    }
    __syncthreads();
    float s[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) s[i][c] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; ++d) {
      const float4 a = *reinterpret_cast<const float4*>(&sm[S::Q + d * S::LD + 4 * ty]);
      const float av[4] = {a.x, a.y, a.z, a.w};
      float b[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) b[c] = sm[S::K + d * S::LK + NC * tx + c];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) s[i][c] = fmaf(av[i], b[c], s[i][c]);
    }
    const bool masked = j0 + BN > pos0;  // some row of the tile may not attend some key of it
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        s[i][c] *= sc;
        if (masked && j0 + NC * tx + c > limit[i]) s[i][c] = -INFINITY;
        mx = fmaxf(mx, s[i][c]);
        if (s[i][c] != s[i][c]) mx = s[i][c];  // a NaN logit makes its row NaN
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, mx, o);
        mx = (mx != mx || y != y) ? NAN : fmaxf(mx, y);
      }
      const float mn = (m[i] != m[i] || mx != mx) ? NAN : fmaxf(m[i], mx);
      const float ref_m = mn == -INFINITY ? 0.f : mn;  // a row with nothing to attend yet
      const float f = exp2f(m[i] - ref_m);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float e = (masked && j0 + NC * tx + c > limit[i]) ? 0.f : exp2f(s[i][c] - ref_m);
        sum += e;
        sm[S::P + (NC * tx + c) * S::LD + 4 * ty + i] = e;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[i] = l[i] * f + sum;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < DC; ++c) acc[i][c] *= f;
    }
    __syncthreads();
    auto add = [&](auto mask_tag) {
      constexpr bool kMask = decltype(mask_tag)::value;
#pragma unroll 2
      for (int j = 0; j < nk; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(&sm[S::P + j * S::LD + 4 * ty]);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const float x = sm[S::V + j * D + 16 * c + tx];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            // a masked key's value stays out even where it is not finite
            if (!kMask || j0 + j <= limit[i]) acc[i][c] = fmaf(av[i], x, acc[i][c]);
        }
      }
    };
    if (masked) add(std::true_type{});
    else add(std::false_type{});
  }
  T* o = static_cast<T*>(p.o);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= nrows) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
    for (int c = 0; c < DC; ++c) st_out(o, row_off(r) + 16 * c + tx, acc[i][c] * inv);
  }
}

template <typename T, int D>
cudaError_t launch_d(const AttnParams& p, cudaStream_t stream) {
  const int per = kRows / p.G > 0 ? kRows / p.G : 1, parts = (p.G + kRows - 1) / kRows;
  const int64_t tiles = ((p.total_tokens + per - 1) / per + p.num_seqs) * parts;
  const size_t smem = SimtShape<T, D>::FLOATS * sizeof(float);
  auto kernel = attn_simt<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)tiles, (unsigned)p.Hkv), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const AttnParams& p, cudaStream_t stream) {
  switch (p.D) {
    case 16: return launch_d<T, 16>(p, stream);
    case 32: return launch_d<T, 32>(p, stream);
    case 64: return launch_d<T, 64>(p, stream);
    case 128: return launch_d<T, 128>(p, stream);
    case 256: return launch_d<T, 256>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attn_simt(const AttnParams& p, cudaStream_t stream) {
  return p.dt == KDA_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace kda
