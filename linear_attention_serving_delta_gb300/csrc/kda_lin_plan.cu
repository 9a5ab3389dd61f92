// kda_lin_plan.cu -- what comes before the chains of the tensor-core prompts of the
// linear attention with a decay for each head: the plan (chains from the
// device-side lengths, costliest first, long ones cut into segments), the gate
// records, and the start states of the segments.
//
// A chain is a walk over its chunks, and a call with few sequences and heads has
// fewer chains than the GPU has SMs.  Then sequences are cut into segments of equal
// length: a first pass leaves the end state of every segment but the last one,
// B_i, from zeros (the first from the initial state); with the decay D_i of a
// segment its start state follows as
//
//   S_0 = S,   S_1 = B_0,   S_{i+1} = D_i S_i + B_i
//
// (the recurrence is affine in S, and its linear part one factor), and a
// second pass gives the outputs of all segments side by side.  Keys and values are
// read twice, from L2 where the call's fit it.
#include <algorithm>

#include "kda_lin_tc.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 2560;

// lengths up to 255 chunks keep their own bucket, longer ones their seven leading bits
__device__ __forceinline__ int bucket_of(int n) {
  if (n < 256) return n;
  const int e = 31 - __clz(n) - 7;
  return min(kBuckets - 1, (e << 7) + (n >> e));
}

// Inclusive sum over the block; *total: of all
__device__ int64_t scan(int64_t x, int64_t* part, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int64_t y = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  *total = __shfl_sync(0xffffffffu, y, 31);
  const int64_t before = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return warp > 0 ? x + before : x;
}

__global__ void __launch_bounds__(kPlanThreads) lin_plan(const LinParams p, const LinPlan a) {
  __shared__ int64_t part[32];
  __shared__ int32_t hist[kBuckets];
  const int tid = threadIdx.x, per = p.H * a.tiles;
  pdl_launch_dependents();
  pdl_wait();
  for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
  // chunks and records
  auto chunks_of = [](const LinSeq& q) { return (int32_t)((q.len + kLinChunk - 1) / kLinChunk); };
  int64_t chunks = 0, active = 0, total;
  int32_t mine_n = 0;  // the thread's first sequence, for the search below
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int s = base + tid;
    LinSeq q{};
    if (s < p.num_seqs) q = lin_seq(p, s);
    const int32_t n = q.ok ? chunks_of(q) : 0;
    const int64_t rec = chunks + scan(n, part, &total) - n;
    chunks += total;
    // (sequences that overlap between malformed ones may have more chunks than there are records)
    if (q.ok && rec + n > a.max_records) {
      q.ok = false;
      q.flag = kFlagBadSeqlens;
    }
    if (q.flag) attn_flag(p.status, q.flag);
    if (s < p.num_seqs) a.seq_rec[s] = q.ok ? (int32_t)rec : -1;
    active += __syncthreads_count(q.ok);
    if (base == 0) mine_n = q.ok ? max(n, 1) : 0;
  }
  // chunks of a segment: the least with which all chains fit the CTAs at once, or where
  // there are more chains than CTAs twice a CTA's share, so that only what would
  // outlast the others is cut
  int32_t limit = INT32_MAX;
  if (a.may_split && chunks > 0) {
    if (active * per <= kLinSlots) {
      int64_t lo = kLinMinSegment, hi = chunks > kLinMinSegment ? chunks : kLinMinSegment;
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        int64_t x = (mine_n + mid - 1) / mid;
        for (int s = tid + kPlanThreads; s < p.num_seqs; s += kPlanThreads)
          if (a.seq_rec[s] >= 0) x += max((int64_t)1, (chunks_of(lin_seq(p, s)) + mid - 1) / mid);
        scan(x, part, &total);
        if (total * per <= kLinSlots) hi = mid;
        else lo = mid + 1;
      }
      limit = (int32_t)min(lo, (int64_t)INT32_MAX);
    } else {
      limit = (int32_t)min(max((int64_t)kLinMinSegment, (2 * chunks * per + kLinSlots - 1) / kLinSlots), (int64_t)INT32_MAX);
    }
  }
  auto segments_of = [&](int32_t n) { return n > limit ? (n - 1) / limit + 1 : 1; };
  __syncthreads();
  for (int s = tid; s < p.num_seqs; s += kPlanThreads) {
    if (a.seq_rec[s] < 0) continue;
    const int32_t n = chunks_of(lin_seq(p, s)), k = segments_of(n);
    for (int i = 0; i < k; ++i) atomicAdd(&hist[bucket_of(lin_cut(n, k, i + 1) - lin_cut(n, k, i))], 1);
  }
  __syncthreads();
  // hist[b] becomes the first place of bucket b: longer ones first
  constexpr int kPer = (kBuckets + kPlanThreads - 1) / kPlanThreads;
  int32_t mine[kPer];
  int64_t n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = kBuckets - 1 - (tid * kPer + i);
    mine[i] = b >= 0 ? hist[b] : 0;
    n += mine[i];
  }
  int64_t at = scan(n, part, &total) - n;
  const int64_t items = total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = kBuckets - 1 - (tid * kPer + i);
    if (b >= 0) hist[b] = (int32_t)at;
    at += mine[i];
  }
  __syncthreads();
  int64_t places = 0, splits = 0, locals = 0;
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int s = base + tid;
    LinSeq q{};
    int32_t n_s = 0, k = 0, rec = -1;
    if (s < p.num_seqs && (rec = a.seq_rec[s]) >= 0) {
      q = lin_seq(p, s);
      n_s = chunks_of(q);
      k = segments_of(n_s);
    }
    const bool cut = k > 1;
    const int64_t place = places + scan(cut ? k : 0, part, &total) - (cut ? k : 0);
    places += total;
    const int64_t split = splits + scan(cut, part, &total) - cut;
    splits += total;
    const int64_t local = locals + scan(cut ? k - 1 : 0, part, &total) - (cut ? k - 1 : 0);
    locals += total;
    const int32_t row = -2 - q.slot, from = p.state_in ? row : -1, to = p.state_out ? row : -1;
    if (cut) a.splits[split] = LinSplit{(int32_t)place, k, rec, n_s};
    for (int i = 0; i < k; ++i) {
      const int32_t c0 = lin_cut(n_s, k, i), c1 = lin_cut(n_s, k, i + 1);
      LinItem it{};
      it.tok0 = (int32_t)q.tok0 + c0 * kLinChunk;
      it.len = (int32_t)min((int64_t)(c1 - c0) * kLinChunk, q.len - (int64_t)c0 * kLinChunk);
      it.rec = rec + c0;
      it.copy = -1;
      // (the first segment starts from a copy: the last one may write the pool in place meanwhile)
      it.from = !cut || (i == 0 && !p.state_in) ? from : (int32_t)place + i;
      it.to = i + 1 == k ? to : -1;
      a.items[atomicAdd(&hist[bucket_of(c1 - c0)], 1)] = it;
      if (i + 1 < k) {
        it.from = i == 0 ? from : -1;
        it.copy = i == 0 && p.state_in ? (int32_t)place : -1;
        it.to = (int32_t)place + i + 1;
        a.locals[local + i] = it;
      }
    }
  }
  if (tid == 0) {
    a.head->items = (int32_t)(items * per);
    a.head->locals = (int32_t)(locals * per);
    a.head->splits = (int32_t)splits;
  }
}

// A CTA per chunk and eight heads, a warp each
__global__ void __launch_bounds__(256) lin_gates(const LinParams p, const LinPlan a, LinGates* records) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t x = blockIdx.x;
  // the last sequence whose records start at or before x (skipped ones: found by those before them)
  int lo = 0, hi = p.num_seqs - 1, found = -1;
  while (lo <= hi) {
    int mid = (lo + hi) >> 1, y = mid;
    while (y >= lo && a.seq_rec[y] < 0) --y;
    if (y < lo) {
      lo = mid + 1;
      continue;
    }
    if (a.seq_rec[y] <= x) {
      found = y;
      lo = mid + 1;
    } else {
      hi = y - 1;
    }
  }
  if (found < 0) return;
  const LinSeq q = lin_seq(p, found);
  const int64_t c = x - a.seq_rec[found];
  if (c * kLinChunk >= q.len) return;
  const int h = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (h < p.H) make_gates(p, q.tok0, (int)q.len, (int)(c * kLinChunk), h, &records[x * p.H + h]);
}

// Start states of segments 2, 3, ...: a thread four elements
__global__ void __launch_bounds__(256) lin_combine(const LinParams p, const LinPlan a, const LinGates* records,
                                                   float* states) {
  __shared__ float decay[kLinSlots + 2];
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y;
  const int64_t size = (int64_t)p.dk * p.dv, e = ((int64_t)blockIdx.z * 256 + threadIdx.x) * 4;
  for (int x = blockIdx.x; x < a.head->splits; x += gridDim.x) {
    const LinSplit sp = a.splits[x];
    __syncthreads();
    // log2 of each segment's decay, a warp a segment
    for (int i = 1 + (threadIdx.x >> 5); i < sp.segments - 1; i += 8) {
      LogSum g{0.f, 0.f};
      for (int c = lin_cut(sp.chunks, sp.segments, i) + (threadIdx.x & 31); c < lin_cut(sp.chunks, sp.segments, i + 1); c += 32)
        g = g + log_sum(records[((int64_t)sp.rec + c) * p.H + h].head.total);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        g = g + LogSum{__shfl_xor_sync(0xffffffffu, g.i, o), __shfl_xor_sync(0xffffffffu, g.f, o)};
      if ((threadIdx.x & 31) == 0) decay[i] = g.i + g.f;
    }
    __syncthreads();
    if (e >= size) continue;
    float4* at = reinterpret_cast<float4*>(states + ((int64_t)sp.place * p.H + h) * size + e);
    const int64_t step = (int64_t)p.H * size / 4;
    float4 s = at[step];
    for (int i = 2; i < sp.segments; ++i) {
      const LinDecay d = lin_decay(decay[i - 1]);
      const float one = d.near_one ? 1.f : 0.f;
      float4 y = at[i * step];
      y.x = fmaf(one, s.x, fmaf(d.m, s.x, y.x));
      y.y = fmaf(one, s.y, fmaf(d.m, s.y, y.y));
      y.z = fmaf(one, s.z, fmaf(d.m, s.z, y.z));
      y.w = fmaf(one, s.w, fmaf(d.m, s.w, y.w));
      at[i * step] = s = y;
    }
  }
}

}  // namespace

// Column tiles: 128 wide, 64 where the keys are 256 or the values no wider
int lin_tile_width(const LinParams& p) { return p.dk > 128 || p.dv <= 64 ? 64 : 128; }

LinLayout lin_layout(const LinParams& p) {
  LinLayout L{};
  const int w = lin_tile_width(p);
  const int64_t per = (int64_t)p.H * ((p.dv + w - 1) / w), chunks = lin_max_records(p);
  // Short prompts that the CTAs hold at once need no plan: a chain each, which makes its
  // gates itself
  L.direct = p.total_tokens <= kLinDirectTokens && p.num_seqs * per <= 2 * kLinSlots;
  // with more than half as many chains a sequence as CTAs no cut would fit
  L.may_split = !L.direct && 2 * per <= kLinSlots && p.total_tokens > kLinMinSegment * kLinChunk;
  L.places = L.may_split ? kLinSlots / per + 2 : 0;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  if (!L.direct) {
    L.head = take(sizeof(LinHead));
    L.seq_rec = take(sizeof(int32_t) * (size_t)p.num_seqs);
    L.items = take(sizeof(LinItem) * (size_t)(p.num_seqs + L.places));
    L.locals = take(sizeof(LinItem) * (size_t)L.places);
    L.splits = take(sizeof(LinSplit) * (size_t)L.places);
    L.states = take(sizeof(float) * (size_t)L.places * p.H * p.dk * p.dv);
  }
  L.records = take(sizeof(LinGates) * (size_t)chunks * p.H);
  L.total = off;
  return L;
}

cudaError_t launch_lin_plan(const LinParams& p, const LinPlan& a, cudaStream_t stream) {
  return launch_maybe_dependent(true, lin_plan, dim3(1), dim3(kPlanThreads), 0, stream, p, a);
}
cudaError_t launch_lin_gates(const LinParams& p, const LinPlan& a, LinGates* records, cudaStream_t stream) {
  return launch_maybe_dependent(true, lin_gates, dim3((unsigned)a.max_records, (unsigned)((p.H + 7) / 8)), dim3(256), 0, stream, p, a, records);
}
cudaError_t launch_lin_combine(const LinParams& p, const LinPlan& a, const LinGates* records, float* states,
                               cudaStream_t stream) {
  const int64_t size = (int64_t)p.dk * p.dv;
  const dim3 grid((unsigned)std::max(1, kLinSlots / (2 * p.H)), (unsigned)p.H, (unsigned)((size + 1023) / 1024));
  return launch_maybe_dependent(true, lin_combine, grid, dim3(256), 0, stream, p, a, records, states);
}

}  // namespace kda
