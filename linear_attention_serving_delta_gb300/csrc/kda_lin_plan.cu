// kda_lin_plan.cu -- what comes before the chains of the linear attention with a decay
// for each head over prompts: the plan (chains from the device-side lengths,
// costliest first, long ones cut into segments), the gate records of the tensor-core
// path, and the start states of the segments.
//
// A chain is a walk over its chunks, and a call with few sequences and heads has
// fewer chains than the GPU has SMs.  Then sequences are cut into segments: a first pass
// leaves the end state B_i of every segment but the last one, of the first segment from the
// initial state and with its outputs, of the others from zeros and without; with the
// decay D_i of a segment the start states follow as
//
//   S_1 = B_0,   S_{i+1} = D_i S_i + B_i
//
// (the recurrence is affine in S, and its linear part one factor), and a
// second pass gives the outputs of the other segments side by side.  So k segments are
// k - 1 chains of either pass, and the first is as much shorter as its outputs take longer.
// Keys and values of those between the first and the last are read twice, from L2 where
// the call's fit it.  One block plans, in about 11 us: lengths, scans over the block,
// and a search for the length of the segments that tries 32 at a time (one after the
// other took 4 us more, and writing a prompt's segments by one thread 6 us).
#include <algorithm>

#include "kda_lin_tc.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 2560;

// A sequence as its segments need it
struct LinMine {
  int32_t tok0, len, rec, place, local, row;
};

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

// Sequence base + thread, with its chunks and its first record, and *before moved on by all of them
struct LinCounted {
  LinSeq seq;
  int32_t chunks;
  int64_t rec;
};
__device__ LinCounted count_chunks(const LinParams& p, const LinPlan& a, int base, int64_t* part, int64_t* before) {
  const int s = base + threadIdx.x;
  LinCounted c{};
  if (s < p.num_seqs) c.seq = lin_seq(p, s);
  c.chunks = c.seq.ok ? (int32_t)((c.seq.len + a.chunk - 1) / a.chunk) : 0;
  int64_t total;
  c.rec = *before + scan(c.chunks, part, &total) - c.chunks;
  *before += total;
  // (sequences that overlap between malformed ones may have more chunks than there are records)
  if (c.seq.ok && c.rec + c.chunks > a.max_records) {
    c.seq.ok = false;
    c.seq.flag = kFlagBadSeqlens;
  }
  return c;
}

// The gate records of a CTA: of some chunks where there are fewer than 32 heads, a warp
// each, otherwise of one chunk and 32 heads.  It counts the chunks for itself, so that it
// runs beside the plan.
__device__ __forceinline__ int gate_chunks(int H) { return H < 32 ? 32 / H : 1; }
__device__ void gates_role(const LinParams& p, const LinPlan& a, int64_t x0, int h0, int64_t* part) {
  __shared__ LinMine of[32];  // the chunks' tokens
  const int mine = gate_chunks(p.H), warp = threadIdx.x >> 5;
  if (threadIdx.x < 32) of[threadIdx.x].len = 0;
  int64_t before = 0;
  for (int base = 0; base < p.num_seqs && before <= x0 + mine - 1; base += kPlanThreads) {
    const LinCounted c = count_chunks(p, a, base, part, &before);
    if (!c.seq.ok) continue;
    for (int64_t x = max(x0, c.rec); x < min(x0 + mine, c.rec + c.chunks); ++x)
      of[x - x0] = LinMine{(int32_t)c.seq.tok0, (int32_t)c.seq.len, (int32_t)(x - c.rec), 0, 0, 0};
  }
  __syncthreads();
  const int c = p.H < 32 ? warp / p.H : 0, h = p.H < 32 ? warp % p.H : h0 + warp;
  if (c >= mine || h >= p.H || of[c].len == 0) return;
  make_gates(p, of[c].tok0, of[c].len, of[c].rec * kLinChunk, h, &a.records[(x0 + c) * p.H + h]);
}

// Block 0 plans, the others make the gate records
__global__ void __launch_bounds__(kPlanThreads) lin_plan(const LinParams p, const LinPlan a) {
  __shared__ int64_t part[32];
  __shared__ int32_t hist[kBuckets];
  __shared__ LinMine mine_of[kPlanThreads];
  __shared__ int32_t first_n[kPlanThreads];  // chunks of the first sequences, for the search
  const int tid = threadIdx.x, per = p.H * a.tiles;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x > 0) {
    gates_role(p, a, (int64_t)(blockIdx.x - 1) * gate_chunks(p.H), blockIdx.y * 32, part);
    return;
  }
  if (blockIdx.y > 0) return;
  for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
  // chunks and records
  auto chunks_of = [&](const LinSeq& q) { return (int32_t)((q.len + a.chunk - 1) / a.chunk); };
  int64_t chunks = 0, active = 0, total;
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int s = base + tid;
    const LinCounted c = count_chunks(p, a, base, part, &chunks);
    const LinSeq& q = c.seq;
    if (q.flag) attn_flag(p.status, q.flag);
    if (s < p.num_seqs) a.seq_rec[s] = q.ok ? (int32_t)c.rec : -1;
    if (base == 0) first_n[tid] = q.ok ? max(c.chunks, 1) : 0;
    active += __syncthreads_count(q.ok);
  }
  // chunks of a segment: the least with which all chains fit the CTAs at once, or where
  // there are more chains than CTAs twice a CTA's share, so that only what would
  // outlast the others is cut
  int32_t limit = INT32_MAX;
  if (a.may_split && chunks > 0) {
    if (active * per <= a.slots) {
      // 32 candidates at once, a warp each; the first that fits ends a round
      const int lane = tid & 31, warp = tid >> 5;
      int64_t lo = a.min_segment, hi = chunks > a.min_segment ? chunks : a.min_segment;
      while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, mid = lo + warp * step;
        const int32_t m = (int32_t)min(mid, hi);
        int64_t x = 0;
        for (int s = lane; s < p.num_seqs; s += 32) {
          int32_t n = s < kPlanThreads ? first_n[s] : 0;
          if (s >= kPlanThreads && a.seq_rec[s] >= 0) n = max(chunks_of(lin_seq(p, s)), 1);
          x += n > 0 ? lin_chains(n, m, a.first) : 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) part[warp] = x * per <= a.slots;
        __syncthreads();
        const int fit = __ffs(__ballot_sync(0xffffffffu, part[lane] != 0)) - 1;
        __syncthreads();
        if (fit != 0) lo = min(hi, lo + (fit < 0 ? 31 : fit - 1) * step + 1);
        if (fit >= 0) hi = fit == 0 ? lo : min(hi, lo - 1 + step);
      }
      limit = (int32_t)min(lo, (int64_t)INT32_MAX);
    } else {
      limit = (int32_t)min(max((int64_t)a.min_segment, (2 * chunks * per + a.slots - 1) / a.slots), (int64_t)INT32_MAX);
    }
  }
  auto segments_of = [&](int32_t n) { return n > limit ? lin_chains(n, limit, a.first) + 1 : 1; };
  __syncthreads();
  // A thread a sequence; the segments of one that is cut by all lanes of its warp
  auto each_segment = [&](int32_t n, int32_t k, auto one) {
    if (k == 1) one(tid & 31, n, 1, 0);
    for (uint32_t cut = __ballot_sync(0xffffffffu, k > 1); cut; cut &= cut - 1) {
      const int from = __ffs(cut) - 1;
      const int32_t n_of = __shfl_sync(0xffffffffu, n, from), k_of = __shfl_sync(0xffffffffu, k, from);
      for (int i = tid & 31; i < k_of; i += 32) one(from, n_of, k_of, i);
    }
  };
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int s = base + tid;
    const bool ok = s < p.num_seqs && a.seq_rec[s] >= 0;
    const int32_t n = ok ? chunks_of(lin_seq(p, s)) : 0;
    each_segment(n, ok ? segments_of(n) : 0, [&](int, int32_t n, int32_t k, int32_t i) {
      if (k > 1 && i == 0) return;  // (the first pass has done it)
      atomicAdd(&hist[bucket_of(lin_cut(n, k, i + 1, a.first) - lin_cut(n, k, i, a.first))], 1);
    });
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
  int64_t before = 0;
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
    // sequences cut and their segments before this one, in one sum
    const int64_t both = cut ? ((int64_t)1 << 32) + k : 0, sum = before + scan(both, part, &total) - both;
    before += total;
    const int64_t split = sum >> 32, place = sum & 0xffffffff, local = place - split;
    if (cut) a.splits[split] = LinSplit{(int32_t)place, k, rec, n_s};
    mine_of[tid] = LinMine{(int32_t)q.tok0, (int32_t)q.len, rec, (int32_t)place, (int32_t)local, -2 - q.slot};
    __syncwarp();
    each_segment(n_s, k, [&](int lane, int32_t n, int32_t k, int32_t i) {
      const LinMine m = mine_of[(tid & ~31) + lane];
      const int32_t c0 = lin_cut(n, k, i, a.first), c1 = lin_cut(n, k, i + 1, a.first);
      const int32_t from = p.state_in ? m.row : -1, to = p.state_out ? m.row : -1;
      LinItem it{};
      it.tok0 = m.tok0 + c0 * a.chunk;
      it.len = min((c1 - c0) * a.chunk, m.len - c0 * a.chunk);
      it.rec = m.rec + c0;
      it.outputs = 1;
      if (k == 1 || i > 0) {
        it.from = k == 1 ? from : m.place + i;
        it.to = i + 1 == k ? to : -1;
        a.items[atomicAdd(&hist[bucket_of(c1 - c0)], 1)] = it;
      }
      if (i + 1 < k) {
        it.from = i == 0 ? from : -1;
        it.to = m.place + i + 1;
        it.outputs = i == 0;
        a.locals[m.local + i] = it;
      }
    });
    __syncwarp();
  }
  if (tid == 0) {
    a.head->items = (int32_t)items;
    a.head->locals = (int32_t)((before & 0xffffffff) - (before >> 32));
    a.head->splits = (int32_t)(before >> 32);
  }
}

// Start states of segments 2, 3, ...: a thread four elements
__global__ void __launch_bounds__(256) lin_combine(const LinParams p, const LinPlan a) {
  __shared__ LinDecay decay[kLinMostSegments];
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y;
  const int64_t size = (int64_t)p.dk * p.dv, e = ((int64_t)blockIdx.z * 256 + threadIdx.x) * 4;
  for (int x = blockIdx.x; x < a.head->splits; x += gridDim.x) {
    const LinSplit sp = a.splits[x];
    __syncthreads();
    // each segment's decay: from the first pass, or from the records, a warp a segment
    if (a.logs)
      for (int i = 1 + threadIdx.x; i < sp.segments - 1; i += 256)
        decay[i] = lin_decay(a.logs[((int64_t)sp.place + i + 1) * p.H + h]);
    for (int i = 1 + (threadIdx.x >> 5); !a.logs && i < sp.segments - 1; i += 8) {
      LogSum g{0.f, 0.f};
      for (int c = lin_cut(sp.chunks, sp.segments, i, a.first) + (threadIdx.x & 31);
           c < lin_cut(sp.chunks, sp.segments, i + 1, a.first); c += 32)
        g = g + log_sum(a.records[((int64_t)sp.rec + c) * p.H + h].head.total);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        g = g + LogSum{__shfl_xor_sync(0xffffffffu, g.i, o), __shfl_xor_sync(0xffffffffu, g.f, o)};
      if ((threadIdx.x & 31) == 0) decay[i] = lin_decay(g.i + g.f);
    }
    __syncthreads();
    if (e >= size) continue;
    float4* at = reinterpret_cast<float4*>(a.states + ((int64_t)sp.place * p.H + h) * size + e);
    const int64_t step = (int64_t)p.H * size / 4;
    float4 s = at[step];
    // (eight loads at a time: one after the other they would be a chain of waits)
    constexpr int kAhead = 8;
    for (int i0 = 2; i0 < sp.segments; i0 += kAhead) {
      float4 y[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u < sp.segments) y[u] = at[(i0 + u) * step];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (i0 + u >= sp.segments) break;
        const LinDecay d = decay[i0 + u - 1];
        const float one = d.near_one ? 1.f : 0.f;
        y[u].x = fmaf(one, s.x, fmaf(d.m, s.x, y[u].x));
        y[u].y = fmaf(one, s.y, fmaf(d.m, s.y, y[u].y));
        y[u].z = fmaf(one, s.z, fmaf(d.m, s.z, y[u].z));
        y[u].w = fmaf(one, s.w, fmaf(d.m, s.w, y[u].w));
        at[(i0 + u) * step] = s = y[u];
      }
    }
  }
}

}  // namespace

// Column tiles: 128 wide, 64 where the keys are 256 or the values no wider
int lin_tile_width(const LinParams& p) { return p.dk > 128 || p.dv <= 64 ? 64 : 128; }

LinShare lin_tc_share(const LinParams& p) {
  const int w = lin_tile_width(p);
  return LinShare{(p.dv + w - 1) / w, kLinTcSlots, kLinChunk, kLinMinSegment, kLinFirst, kLinDirectTokens, true};
}

LinLayout lin_layout(const LinParams& p, const LinShare& sh) {
  LinLayout L{};
  const int64_t per = (int64_t)p.H * sh.tiles, chunks = lin_max_records(p, sh.chunk);
  // Short prompts that the CTAs hold at once need no plan: a chain each, which makes its
  // gates itself
  L.direct = p.total_tokens <= sh.direct_tokens && p.num_seqs * per <= 2 * sh.slots;
  // with more than half as many chains a sequence as CTAs no cut would fit
  L.may_split = !L.direct && 2 * per <= sh.slots && p.total_tokens > sh.min_segment * sh.chunk;
  // (a segment more than chains of a pass for each sequence that is cut)
  L.places = L.may_split ? 2 * (sh.slots / per) + 2 : 0;
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
    if (!sh.records) L.logs = take(sizeof(float) * (size_t)L.places * p.H);
  }
  if (sh.records) L.records = take(sizeof(LinGates) * (size_t)chunks * p.H);
  L.total = off > 0 ? off : 256;
  return L;
}

LinPlan lin_plan_of(const LinParams& p, const LinShare& sh, const LinLayout& L, void* ws) {
  char* w = static_cast<char*>(ws);
  LinPlan a{};
  a.head = reinterpret_cast<LinHead*>(w + L.head);
  a.seq_rec = reinterpret_cast<int32_t*>(w + L.seq_rec);
  a.items = reinterpret_cast<LinItem*>(w + L.items);
  a.locals = reinterpret_cast<LinItem*>(w + L.locals);
  a.splits = reinterpret_cast<LinSplit*>(w + L.splits);
  a.tiles = sh.tiles;
  a.slots = sh.slots;
  a.min_segment = sh.min_segment;
  a.first = sh.first;
  a.chunk = sh.chunk;
  a.max_records = lin_max_records(p, sh.chunk);
  a.may_split = L.may_split;
  a.states = reinterpret_cast<float*>(w + L.states);
  a.records = sh.records ? reinterpret_cast<LinGates*>(w + L.records) : nullptr;
  a.logs = sh.records ? nullptr : reinterpret_cast<float*>(w + L.logs);
  return a;
}

cudaError_t launch_lin_plan(const LinParams& p, const LinPlan& a, cudaStream_t stream) {
  dim3 grid(1);
  if (a.records) {
    const int64_t each = p.H < 32 ? 32 / p.H : 1;
    grid = dim3((unsigned)(1 + (a.max_records + each - 1) / each), (unsigned)((p.H + 31) / 32));
  }
  return launch_maybe_dependent(true, lin_plan, grid, dim3(kPlanThreads), 0, stream, p, a);
}
cudaError_t launch_lin_combine(const LinParams& p, const LinPlan& a, cudaStream_t stream) {
  const int64_t size = (int64_t)p.dk * p.dv;
  const dim3 grid((unsigned)std::max(1, a.slots / (2 * p.H * a.tiles)), (unsigned)p.H, (unsigned)((size + 1023) / 1024));
  return launch_maybe_dependent(true, lin_combine, grid, dim3(256), 0, stream, p, a);
}

}  // namespace kda
