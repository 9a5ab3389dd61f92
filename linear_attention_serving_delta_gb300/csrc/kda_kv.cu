// kda_kv.cu -- the paged cache's bookkeeping on the GPU: block tables and slot
// maps from request lengths, pages back to the free list, and the write of
// new keys and values into their slots.  Formulas in include/kda.h.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int64_t kNoPlan = -1;

// What the planning kernel leaves for the slot map
struct KvWs {
  int32_t* owner;   // [num_rows] the first request of the batch that names the row
  int64_t* first;   // [N] e_s, or kNoPlan for a skipped or refused request
  int64_t* ctx;     // [N] positions cached before the call
  int32_t* count;   // [1] pages on the free list before the call
};

__host__ __device__ KvWs kv_ws(void* ws, int64_t n, int64_t rows) {
  KvWs w;
  char* c = static_cast<char*>(ws);
  w.count = reinterpret_cast<int32_t*>(c);
  w.first = reinterpret_cast<int64_t*>(c + 256);
  w.ctx = w.first + n;
  w.owner = reinterpret_cast<int32_t*>(w.ctx + n);
  (void)rows;
  return w;
}

// Inclusive sum over the block's threads (kPlanThreads of them); *total gets
// the sum of all.  `part` is shared, 32 entries.
__device__ int64_t block_scan(int64_t x, int64_t* part, int64_t* total) {
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

__device__ __forceinline__ int64_t ceil_shift(int64_t x, int s) { return (x + ((int64_t)1 << s) - 1) >> s; }

// The slot of new token t (and, at a page's first token, the page's table entry)
__device__ void plan_token(const kda_kv_plan_args& a, const KvWs& w, int shift, int64_t t) {
  const int32_t s = seq_of_token(a.cu_seqlens, a.num_seqs, t);
  const int64_t b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
  int64_t slot = -1;
  const int64_t first = w.first[s];
  if (t >= b && t < e && first != kNoPlan) {
    const int32_t r = a.rows ? a.rows[s] : s;
    const int64_t c = w.ctx[s], pos = c + (t - b);
    const int64_t have = ceil_shift(c, shift), j = pos >> shift;
    const int64_t off = pos & (((int64_t)1 << shift) - 1);
    int32_t* entry = a.block_table + (int64_t)r * a.max_pages + j;
    int32_t page;
    if (j >= have) {
      page = a.free_pages[*w.count - 1 - (first + (j - have))];
      if (off == 0) *entry = page;
    } else {
      page = *entry;
    }
    if (page >= 0 && page < a.num_pages) slot = ((int64_t)page << shift) + off;
    else attn_flag(a.status, kFlagBadCache);
  }
  a.slot_map[t] = slot;
}

// One CTA: the pages each request needs, their prefix sum over the batch, and
// which requests the free list can serve.  Bound by its chain of dependent
// global loads (row, length, owner), a few microseconds whatever the batch.
// With `tokens` it goes on to the slots (small batches: one launch).
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(kda_kv_plan_args a, KvWs w, int shift, int tokens) {
  __shared__ int64_t part[32];
  const int tid = threadIdx.x;
  int32_t count = *a.free_count_in;
  if (count < 0 || count > a.num_pages) {
    if (tid == 0) attn_flag(a.status, kFlagBadCache);
    count = 0;
  }
  // the first request that names a row owns it
  if (a.rows) {
    for (int s = tid; s < a.num_seqs; s += kPlanThreads) {
      const int32_t r = a.rows[s];
      if (r >= 0 && r < a.num_rows) w.owner[r] = INT32_MAX;
    }
    __syncthreads();
    for (int s = tid; s < a.num_seqs; s += kPlanThreads) {
      const int32_t r = a.rows[s];
      if (r >= 0 && r < a.num_rows) atomicMin(&w.owner[r], s);
    }
    __syncthreads();
  }
  int64_t before = 0, served = 0;
  for (int base = 0; base < a.num_seqs; base += kPlanThreads) {
    const int s = base + tid;
    int64_t need = 0, c = 0, len = 0;
    int32_t r = -1;
    bool ok = false;
    if (s < a.num_seqs) {
      r = a.rows ? a.rows[s] : s;
      const int64_t b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
      len = e - b;
      if (b < 0 || e < b || e > a.total_tokens || (s == 0 && b != 0)) {
        attn_flag(a.status, kFlagBadSeqlens);
      } else if (r >= a.num_rows || (r >= 0 && a.rows && *(volatile int32_t*)&w.owner[r] != s)) {
        attn_flag(a.status, kFlagBadCache);
        r = -1;  // the owner's length stays as the owner leaves it
      } else if (r >= 0) {
        c = a.kv_lens_in[r];
        ok = c >= 0 && c + len <= ((int64_t)a.max_pages << shift) && c + len >= c;
        if (!ok) attn_flag(a.status, kFlagBadCache);
      }
      if (ok) need = ceil_shift(c + len, shift) - ceil_shift(c, shift);
    }
    int64_t total;
    const int64_t end = before + block_scan(need, part, &total);
    if (s < a.num_seqs) {
      if (ok && need > 0 && end > count) {
        ok = false;
        attn_flag(a.status, kFlagNoPages);
      }
      w.first[s] = ok ? end - need : kNoPlan;
      w.ctx[s] = c;
      if (ok) a.kv_lens_out[r] = c + len;
      else if (r >= 0 && a.kv_lens_out != a.kv_lens_in) a.kv_lens_out[r] = a.kv_lens_in[r];
    }
    // the served ones that need pages come first among those that do
    block_scan(ok ? need : 0, part, &total);
    served += total;
    int64_t all;
    block_scan(need, part, &all);
    before += all;
  }
  if (tid == 0) {
    *w.count = count;
    *a.free_count_out = count - (int32_t)served;
  }
  if (!tokens) return;
  __syncthreads();
  for (int64_t t = tid; t < a.total_tokens; t += kPlanThreads) plan_token(a, w, shift, t);
}

__global__ void __launch_bounds__(256) kv_slots_kernel(kda_kv_plan_args a, KvWs w, int shift) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  if (t < a.total_tokens) plan_token(a, w, shift, t);
}

__global__ void __launch_bounds__(kPlanThreads) kv_release_kernel(kda_kv_release_args a, KvWs w, int shift) {
  __shared__ int64_t part[32];
  const int tid = threadIdx.x;
  int64_t count = *a.free_count;
  __syncthreads();
  if (count < 0 || count > a.num_pages) {
    if (tid == 0) attn_flag(a.status, kFlagBadCache);
    return;
  }
  for (int i = tid; i < a.num_release; i += kPlanThreads) {
    const int32_t r = a.rows[i];
    if (r >= 0 && r < a.num_rows) w.owner[r] = INT32_MAX;
  }
  __syncthreads();
  for (int i = tid; i < a.num_release; i += kPlanThreads) {
    const int32_t r = a.rows[i];
    if (r >= 0 && r < a.num_rows) atomicMin(&w.owner[r], i);
  }
  __syncthreads();
  for (int base = 0; base < a.num_release; base += kPlanThreads) {
    const int i = base + tid;
    int64_t n = 0;
    int32_t r = -1;
    if (i < a.num_release) {
      r = a.rows[i];
      if (r >= a.num_rows) {
        attn_flag(a.status, kFlagBadCache);
        r = -1;
      } else if (r >= 0 && *(volatile int32_t*)&w.owner[r] == i) {
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
    int64_t at = count + block_scan(n, part, &total) - n;
    if (n > 0 && at + n > a.num_pages) {
      attn_flag(a.status, kFlagBadCache);
      r = -1;
      n = 0;
    }
    if (r >= 0) {
      a.kv_lens[r] = 0;
      for (int64_t j = 0; j < n; ++j) a.free_pages[at + j] = a.block_table[(int64_t)r * a.max_pages + j];
    }
    block_scan(n, part, &total);
    count += total;
  }
  if (tid == 0) *a.free_count = (int32_t)count;
}

// One warp per token: the row of k, then that of v, in units of V.  Moves
// every byte once; bound by HBM on large batches, by latency on a decode's.
template <typename V>
__global__ void __launch_bounds__(256) kv_write_kernel(kda_kv_write_args a, int64_t row_units) {
  const int64_t warps = (int64_t)gridDim.x * 8;
  const int lane = threadIdx.x & 31;
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

// Batches up to this many tokens take their slots in the planning CTA itself:
// one launch, where a second one costs more than the CTA's few passes.
constexpr int64_t kOneLaunchTokens = 4096;

}  // namespace

size_t kv_plan_workspace(int64_t n, int64_t rows) {
  return align_up(256 + (size_t)n * 16 + (size_t)rows * 4, 256);
}

cudaError_t launch_kv_plan(const kda_kv_plan_args& a, void* ws, cudaStream_t stream) {
  const KvWs w = kv_ws(ws, a.num_seqs, a.num_rows);
  const int shift = shift_of(a.page_size);
  const int one = a.total_tokens <= kOneLaunchTokens;
  kv_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, w, shift, one);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || one) return e;
  return launch_maybe_dependent(true, kv_slots_kernel, dim3((unsigned)((a.total_tokens + 255) / 256)), dim3(256), 0,
                                stream, a, w, shift);
}

cudaError_t launch_kv_release(const kda_kv_release_args& a, void* ws, cudaStream_t stream) {
  if (a.num_release == 0) return cudaSuccess;
  kv_release_kernel<<<1, kPlanThreads, 0, stream>>>(a, kv_ws(ws, 0, a.num_rows), shift_of(a.page_size));
  return cudaGetLastError();
}

cudaError_t launch_kv_write(const kda_kv_write_args& a, cudaStream_t stream) {
  if (a.total_tokens == 0) return cudaSuccess;
  const int64_t bytes = (int64_t)a.num_kv_heads * a.head_dim * (a.in_dtype == KDA_BF16 ? 2 : 4);
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                        reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache);
  int64_t ctas = (a.total_tokens + 7) / 8;
  if (ctas > 152 * 8) ctas = 152 * 8;
  // rows are multiples of 32 bytes (16 channels of 2 bytes); an unaligned base takes 2-byte units
  if ((all & 15) == 0)
    kv_write_kernel<uint4><<<(unsigned)ctas, 256, 0, stream>>>(a, bytes / 16);
  else
    kv_write_kernel<uint16_t><<<(unsigned)ctas, 256, 0, stream>>>(a, bytes / 2);
  return cudaGetLastError();
}

}  // namespace kda
