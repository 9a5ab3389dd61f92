// kda_kv.cu -- the paged cache's bookkeeping on the GPU: block tables and slot
// maps from request lengths, pages back to the free list, and the write of
// new keys and values into their slots.  Formulas in include/kda.h.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int64_t kNoPlan = -1;
// The first request that names a row is found in shared memory for pools of up
// to this many rows, in the workspace beyond.
constexpr int kSharedRows = 4096;
// A batch of up to kOneLaunchTokens tokens of up to kPlanThreads requests takes
// its slots in the planning CTA itself, from shared memory: one launch, where a
// second one costs more than the CTA's few passes.
constexpr int64_t kOneLaunchTokens = 4096;

// What the planning CTA leaves for the slot map, in the workspace
struct KvWs {
  int32_t* owner;   // [num_rows] the first request of the batch that names the row
  int64_t* first;   // [N] e_s, or kNoPlan for a skipped or refused request
  int64_t* ctx;     // [N] positions cached before the call
  int32_t* count;   // [2] pages on the free list before the call; requests before malformed cu_seqlens
};

KvWs kv_ws(void* ws, int64_t n) {
  KvWs w;
  char* c = static_cast<char*>(ws);
  w.count = reinterpret_cast<int32_t*>(c);
  w.first = reinterpret_cast<int64_t*>(c + 256);
  w.ctx = w.first + n;
  w.owner = reinterpret_cast<int32_t*>(w.ctx + n);
  return w;
}

// Inclusive sum over the block's threads; *total gets the sum of all.  `part`
// is shared, 32 entries, and free again at the next barrier.
__device__ int64_t block_scan(int64_t x, int64_t* part, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int64_t y = lane < warps ? part[lane] : 0;  // every warp adds up the warps before it
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  *total = __shfl_sync(0xffffffffu, y, 31);
  const int64_t before = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
  return warp > 0 ? x + before : x;
}

__device__ __forceinline__ int64_t ceil_shift(int64_t x, int s) { return (x + ((int64_t)1 << s) - 1) >> s; }

// owner[r] = the first entry of rows[0..n) that is r, for every r named there
__device__ void find_owners(const int32_t* rows, int32_t n, int32_t num_rows, int32_t* owner) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int32_t r = rows[i];
    if (r >= 0 && r < num_rows) owner[r] = INT32_MAX;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int32_t r = rows[i];
    if (r >= 0 && r < num_rows) atomicMin(&owner[r], i);
  }
  __syncthreads();
}

// The slot of new token t of request s (and, at a page's first token, the
// page's table entry); c: cached before, first: e_s
__device__ int64_t plan_slot(const kda_kv_plan_args& a, int shift, int64_t count, int64_t t, int32_t s, int64_t b,
                             int64_t c, int64_t first) {
  const int32_t r = a.rows ? a.rows[s] : s;
  const int64_t pos = c + (t - b), have = ceil_shift(c, shift), j = pos >> shift;
  const int64_t off = pos & (((int64_t)1 << shift) - 1);
  int32_t* entry = a.block_table + (int64_t)r * a.max_pages + j;
  int32_t page;
  if (j >= have) {
    page = a.free_pages[count - 1 - (first + (j - have))];
    if (off == 0) *entry = page;
  } else {
    page = *entry;
  }
  if (page >= 0 && page < a.num_pages) return ((int64_t)page << shift) + off;
  attn_flag(a.status, kFlagBadCache);
  return -1;
}

// One CTA: the pages each request needs, their prefix sum over the batch, and
// which requests the free list can serve.  Bound by its chain of dependent
// global loads (row, length, page), a few microseconds whatever the batch (256
// requests with their slots: 3.5 us; 6.1 as a plain launch, 7.7 with the owners
// and the slots' inputs in global memory).
// kSlots: it goes on to the slots (one request a thread at most).
template <bool kSlots>
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(kda_kv_plan_args a, KvWs w, int shift) {
  __shared__ int64_t part[2][32];
  __shared__ int64_t sm_cu[kSlots ? kPlanThreads + 1 : 1], sm_first[kSlots ? kPlanThreads : 1],
      sm_ctx[kSlots ? kPlanThreads : 1];
  __shared__ int32_t sm_good;  // requests before the first with malformed cu_seqlens
  extern __shared__ int32_t sm_owner[];
  const int tid = threadIdx.x, threads = blockDim.x;
  if (tid == 0) sm_good = a.num_seqs;
  __syncthreads();
  pdl_wait();
  int32_t count = *a.free_count_in;
  int32_t* owner = a.num_rows <= kSharedRows ? sm_owner : w.owner;
  if (a.rows) find_owners(a.rows, a.num_seqs, a.num_rows, owner);
  if (count < 0 || count > a.num_pages) {
    if (tid == 0) attn_flag(a.status, kFlagBadCache);
    count = 0;
  }
  int64_t before = 0, served = 0;
  for (int base = 0; base < a.num_seqs; base += threads) {
    const int s = base + tid;
    int64_t need = 0, c = 0, len = 0, b = 0;
    int32_t r = -1;
    bool ok = false;
    if (s < a.num_seqs) {
      r = a.rows ? a.rows[s] : s;
      b = a.cu_seqlens[s];
      const int64_t e = a.cu_seqlens[s + 1];
      len = e - b;
      if (r >= a.num_rows || (r >= 0 && a.rows && owner[r] != s)) {
        attn_flag(a.status, kFlagBadCache);
        r = -1;  // no row of the pool; the owner's length stays as the owner leaves it
      }
      if (b < 0 || e < b || e > a.total_tokens || (s == 0 && b != 0)) {
        attn_flag(a.status, kFlagBadSeqlens);
        atomicMin(&sm_good, s);
      } else if (r >= 0) {
        c = a.kv_lens_in[r];
        const int64_t most = (int64_t)a.max_pages << shift;
        ok = c >= 0 && c <= most && len <= most - c;  // (c + len may pass 64 bits)
        if (!ok) attn_flag(a.status, kFlagBadCache);
      }
      if (ok) need = ceil_shift(c + len, shift) - ceil_shift(c, shift);
      if (kSlots) {
        sm_cu[s] = b;
        if (s + 1 == a.num_seqs) sm_cu[s + 1] = e;
      }
    }
    int64_t total, all;
    const int64_t end = before + block_scan(need, part[0], &total);
    if (s < a.num_seqs) {
      // behind malformed offsets a token's request cannot be told (what these
      // requests need stands behind all that is served in the prefix sum)
      if (s >= *reinterpret_cast<volatile int32_t*>(&sm_good)) ok = false;
      if (ok && need > 0 && end > count) {
        ok = false;
        attn_flag(a.status, kFlagNoPages);
      }
      const int64_t first = ok ? end - need : kNoPlan;
      if (kSlots) {
        sm_first[s] = first;
        sm_ctx[s] = c;
      } else {
        w.first[s] = first;
        w.ctx[s] = c;
      }
      if (ok) a.kv_lens_out[r] = c + len;
      else if (r >= 0 && a.kv_lens_out != a.kv_lens_in) a.kv_lens_out[r] = a.kv_lens_in[r];
    }
    block_scan(ok ? need : 0, part[1], &all);
    before += total;
    served += all;
    if (base + threads < a.num_seqs) __syncthreads();  // `part` again
  }
  if (tid == 0) {
    *a.free_count_out = count - (int32_t)served;
    if (!kSlots) {
      w.count[0] = count;
      w.count[1] = sm_good;
    }
  }
  if constexpr (kSlots) {
    __syncthreads();
    const int32_t good = sm_good;
    for (int64_t t = tid; t < a.total_tokens; t += threads) {
      // the request of the token: a decode batch has one token each
      int32_t s = t < good && sm_cu[t] == t && sm_cu[t + 1] > t ? (int32_t)t : seq_of_token(sm_cu, good, t);
      const int64_t b = sm_cu[s], first = sm_first[s];
      a.slot_map[t] = t >= b && t < sm_cu[s + 1] && first != kNoPlan
                          ? plan_slot(a, shift, count, t, s, b, sm_ctx[s], first)
                          : -1;
    }
  }
}

__global__ void __launch_bounds__(256) kv_slots_kernel(kda_kv_plan_args a, KvWs w, int shift) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  if (t >= a.total_tokens) return;
  const int32_t s = seq_of_token(a.cu_seqlens, w.count[1], t);
  const int64_t b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
  const int64_t first = w.first[s];
  a.slot_map[t] = t >= b && t < e && first != kNoPlan ? plan_slot(a, shift, w.count[0], t, s, b, w.ctx[s], first) : -1;
}

// One CTA: the pages each row gives back and their prefix sum, then the pages
// themselves, spread over the threads whichever row they come from (64 rows of
// 2,048 pages: 98 us, 448 with a thread for each row; one row of 8,192: 18 and 324).
__global__ void __launch_bounds__(kPlanThreads) kv_release_kernel(kda_kv_release_args a, KvWs w, int shift) {
  constexpr int kAhead = 4;  // pages of a thread in flight
  __shared__ int64_t part[2][32];
  __shared__ int64_t sm_end[kPlanThreads];  // pages of this pass's rows up to and with each
  __shared__ int32_t sm_row[kPlanThreads];
  extern __shared__ int32_t sm_owner[];
  const int tid = threadIdx.x;
  pdl_wait();
  int64_t count = *a.free_count;
  int32_t* owner = a.num_rows <= kSharedRows ? sm_owner : w.owner;
  __syncthreads();
  if (count < 0 || count > a.num_pages) {
    if (tid == 0) attn_flag(a.status, kFlagBadCache);
    return;
  }
  find_owners(a.rows, a.num_release, a.num_rows, owner);
  for (int base = 0; base < a.num_release; base += kPlanThreads) {
    const int i = base + tid;
    int64_t n = 0;
    int32_t r = -1;
    if (i < a.num_release) {
      r = a.rows[i];
      if (r >= a.num_rows) {
        attn_flag(a.status, kFlagBadCache);
        r = -1;
      } else if (r >= 0 && owner[r] == i) {
        const int64_t len = a.kv_lens[r];
        if (len < 0 || len > ((int64_t)a.max_pages << shift)) {
          attn_flag(a.status, kFlagBadCache);
          r = -1;
        } else {
          n = ceil_shift(len, shift);
        }
      } else {
        r = -1;
      }
    }
    int64_t total;
    block_scan(n, part[0], &total);
    if (count + total > a.num_pages) {  // (an over-full list: row by row, a row that does not fit is passed over)
      sm_end[tid] = n;
      __syncthreads();
      if (tid == 0) {
        int64_t at = count;
        for (int x = 0; x < kPlanThreads; ++x) {
          if (at + sm_end[x] > a.num_pages) sm_end[x] = -1;
          else at += sm_end[x];
        }
      }
      __syncthreads();
      if (sm_end[tid] < 0) {
        attn_flag(a.status, kFlagBadCache);
        r = -1;
        n = 0;
      }
      __syncthreads();  // sm_end again
    }
    if (r >= 0) a.kv_lens[r] = 0;
    sm_end[tid] = block_scan(n, part[1], &total);
    sm_row[tid] = r;
    __syncthreads();
    for (int64_t x0 = tid; x0 < total; x0 += kAhead * kPlanThreads) {
      int32_t page[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t x = x0 + u * kPlanThreads;
        if (x >= total) break;
        int lo = 0, hi = kPlanThreads - 1;  // the first row whose pages end past x
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (sm_end[mid] > x) hi = mid; else lo = mid + 1;
        }
        const int64_t j = x - (lo > 0 ? sm_end[lo - 1] : 0);
        page[u] = a.block_table[(int64_t)sm_row[lo] * a.max_pages + j];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t x = x0 + u * kPlanThreads;
        if (x < total) a.free_pages[count + x] = page[u];
      }
    }
    count += total;
    __syncthreads();  // the shared arrays again
  }
  if (tid == 0) *a.free_count = (int32_t)count;
}

// One warp per token: the row of k, then that of v, in units of V.  Moves
// every byte once; bound by HBM on large batches (110,353 tokens of 8 x 128
// bf16: 138 us, 6.6 TB/s, 98% of the measured copy rate), by latency on a
// decode's (256 tokens: 2.9 us, 4.1 as a plain launch).
template <typename V>
__global__ void __launch_bounds__(256) kv_write_kernel(kda_kv_write_args a, int64_t row_units) {
  const int64_t warps = (int64_t)gridDim.x * 8;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < a.total_tokens; t += warps) {
    const int64_t slot = a.slot_map[t];
    if (slot < 0) continue;
    if (slot >= a.num_slots) {
      if (lane == 0) attn_flag(a.status, kFlagBadCache);
      continue;
    }
    const V* k = static_cast<const V*>(a.k) + t * row_units;
    const V* v = static_cast<const V*>(a.v) + t * row_units;
    V* kc = static_cast<V*>(a.k_cache) + slot * row_units;
    V* vc = static_cast<V*>(a.v_cache) + slot * row_units;
#pragma unroll 4
    for (int64_t i = lane; i < row_units; i += 32) {
      const V x = k[i], y = v[i];
      kc[i] = x;
      vc[i] = y;
    }
  }
}

int shift_of(int32_t page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

size_t owner_bytes(int32_t rows) { return rows <= kSharedRows ? (size_t)rows * sizeof(int32_t) : 0; }

}  // namespace

size_t kv_plan_workspace(int64_t n, int64_t rows) {
  return align_up(256 + (size_t)n * 16 + (size_t)rows * 4, 256);
}

cudaError_t launch_kv_plan(const kda_kv_plan_args& a, void* ws, cudaStream_t stream) {
  const KvWs w = kv_ws(ws, a.num_seqs);
  const int shift = shift_of(a.page_size);
  const bool one = a.total_tokens <= kOneLaunchTokens && a.num_seqs <= kPlanThreads;
  const int64_t most = one && a.total_tokens > a.num_seqs ? a.total_tokens : a.num_seqs;
  const int threads = most >= kPlanThreads ? kPlanThreads : (int)(most + 31) / 32 * 32;
  // (each of these as the programmatic dependent of what precedes it: its launch overlaps that one's end)
  const cudaError_t e = launch_maybe_dependent(true, one ? kv_plan_kernel<true> : kv_plan_kernel<false>, dim3(1),
                                               dim3(threads), owner_bytes(a.num_rows), stream, a, w, shift);
  if (e != cudaSuccess || one || a.total_tokens == 0) return e;
  return launch_maybe_dependent(true, kv_slots_kernel, dim3((unsigned)((a.total_tokens + 255) / 256)), dim3(256), 0,
                                stream, a, w, shift);
}

cudaError_t launch_kv_release(const kda_kv_release_args& a, void* ws, cudaStream_t stream) {
  if (a.num_release == 0) return cudaSuccess;
  return launch_maybe_dependent(true, kv_release_kernel, dim3(1), dim3(kPlanThreads), owner_bytes(a.num_rows), stream, a,
                                kv_ws(ws, 0), shift_of(a.page_size));
}

cudaError_t launch_kv_write(const kda_kv_write_args& a, cudaStream_t stream) {
  if (a.total_tokens == 0) return cudaSuccess;
  const int64_t bytes = (int64_t)a.num_kv_heads * a.head_dim * (a.in_dtype == KDA_BF16 ? 2 : 4);
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                        reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache);
  int64_t ctas = (a.total_tokens + 7) / 8;
  if (ctas > 152 * 8) ctas = 152 * 8;
  // rows are multiples of 32 bytes (16 channels of 2 bytes); an unaligned base takes 2-byte units
  const bool wide = (all & 15) == 0;
  return launch_maybe_dependent(true, wide ? kv_write_kernel<uint4> : kv_write_kernel<uint16_t>, dim3((unsigned)ctas),
                                dim3(256), 0, stream, a, bytes / (wide ? 16 : 2));
}

}  // namespace kda
