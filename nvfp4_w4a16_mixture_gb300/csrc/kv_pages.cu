// Pages of the paged KV cache: copies of whole or part-filled pages, and the
// plan of a compaction.
//
// Copy: bytes only.  A (pair, K or V, slot, head) row is 256 contiguous
// bytes, 16 threads x 16 bytes.
// Plan: three kernels.  mark sets the bit of every page in use; rank scans
// the bitmap (one CTA): the live count, each word's number of live pages
// below it, and the pairs; rename writes the new table.  All in integers, so
// the result does not depend on the order of the atomics.
#include "attn.cuh"

namespace flint {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const KvCopyArgs a) {
  SpanGuard<kSpanKvCopy> span_guard;
  pdl_wait();  // the pairs and the pages are earlier kernels' output
  pdl_launch_dependents();
  int n = a.num_moves;
  if (a.count) n = min(n, ldg_cg_i32(a.count));
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int src = ldg_cg_i32(a.moves + 2 * (long long)i), dst = ldg_cg_i32(a.moves + 2 * (long long)i + 1);
    if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
      if (threadIdx.x == 0) attn_error(a.status);
      continue;
    }
    int slots = a.block_size;
    if (a.tokens) {
      const int t = ldg_cg_i32(a.tokens + i);
      if ((t < 0 || t > slots) && threadIdx.x == 0) attn_error(a.status);
      slots = min(max(t, 0), slots);
    }
    for (int r = threadIdx.x / 16; r < slots * a.nkv; r += kCopyThreads / 16) {
      const long long at = (long long)(r / a.nkv) * a.s_slot + (long long)(r % a.nkv) * a.s_head + 8 * (threadIdx.x % 16);
      const uint4 kv = ldg_cg_v4(a.k + src * a.s_block + at);
      const uint4 vv = ldg_cg_v4(a.v + src * a.s_block + at);
      *reinterpret_cast<uint4*>(a.k + dst * a.s_block + at) = kv;
      *reinterpret_cast<uint4*>(a.v + dst * a.s_block + at) = vv;
    }
  }
}

// Pages of sequence b (its length taken into the table's reach).
FLINT_DEV int seq_pages(const KvPlanArgs& a, int b) {
  const int n = ldg_cg_i32(a.seq_lens + b);
  const long long most = (long long)a.max_blocks * a.block_size;
  if (n < 0 || n > most) {
    attn_error(a.status);
    return n < 0 ? 0 : a.max_blocks;
  }
  return (int)(((long long)n + a.block_size - 1) / a.block_size);
}

__global__ void __launch_bounds__(256) kv_mark_kernel(const KvPlanArgs a) {
  SpanGuard<kSpanKvPlan> span_guard;
  pdl_wait();
  pdl_launch_dependents();
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int used = seq_pages(a, b);
    for (int i = threadIdx.x; i < used; i += 256) {
      const int p = ldg_cg_i32(a.block_table + (long long)b * a.table_stride + i);
      if (p < 0 || p >= a.num_blocks)
        attn_error(a.status);
      else
        atomicOr(a.live + (p >> 5), 1u << (p & 31));
    }
  }
}

FLINT_DEV uint32_t ldg_cg_u32(const uint32_t* p) { return (uint32_t)ldg_cg_i32(reinterpret_cast<const int*>(p)); }

// Sum over the CTA's threads below this one; total in *all.
FLINT_DEV int scan_cta(int v, int* warps, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warps[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    warps[lane] = w;
  }
  __syncthreads();
  const int r = x - v + (warp ? warps[warp - 1] : 0);
  *all = warps[31];
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(kPlanThreads) kv_rank_kernel(const KvPlanArgs a) {
  SpanGuard<kSpanKvPlan> span_guard;
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int warps[32];
  const int words = (a.num_blocks + 31) / 32;
  int live = 0;
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x;
    int all;
    const int below = scan_cta(w < words ? __popc(ldg_cg_u32(a.live + w)) : 0, warps, &all);
    if (w < words) a.rank[w] = live + below;
    live += all;
  }
  // `rank[w]` was written by this very thread
  int above = 0;  // live pages at or above `live` = unused pages below it
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x;
    int c = 0;
    if (w < words) {
      const uint32_t bits = ldg_cg_u32(a.live + w);
      const int p0 = 32 * w;
      const uint32_t ge = p0 >= live ? ~0u : (live - p0 >= 32 ? 0u : ~0u << (live - p0));
      c = __popc(bits & ge);
    }
    int all;
    scan_cta(c, warps, &all);
    above += all;
  }
  const int low = live - above;  // live pages below `live`
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x;
    if (w >= words) continue;
    const uint32_t bits = ldg_cg_u32(a.live + w);
    int rank = a.rank[w];
    for (int i = 0; i < 32 && 32 * w + i < a.num_blocks; ++i) {
      const int p = 32 * w + i;
      const bool on = (bits >> i) & 1u;
      if (on && p >= live) a.moves[2 * (long long)(rank - low)] = p;
      if (!on && p < live) a.moves[2 * (long long)(p - rank) + 1] = p;
      rank += on;
    }
  }
  for (int i = 2 * above + threadIdx.x; i < a.num_blocks / 2 * 2; i += kPlanThreads) a.moves[i] = -1;
  if (threadIdx.x == 0) {
    a.counts[0] = live;
    a.counts[1] = above;
  }
}

__global__ void __launch_bounds__(256) kv_rename_kernel(const KvPlanArgs a) {
  SpanGuard<kSpanKvPlan> span_guard;
  pdl_wait();
  pdl_launch_dependents();
  const int live = ldg_cg_i32(a.counts), low = live - ldg_cg_i32(a.counts + 1);
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int used = seq_pages(a, b);
    for (int i = threadIdx.x; i < a.max_blocks; i += 256) {
      int p = -1;
      if (i < used) {
        p = ldg_cg_i32(a.block_table + (long long)b * a.table_stride + i);
        if (p < 0 || p >= a.num_blocks) {
          p = -1;
        } else if (p >= live) {
          const int rank = ldg_cg_i32(a.rank + (p >> 5)) + __popc(ldg_cg_u32(a.live + (p >> 5)) & ((1u << (p & 31)) - 1));
          p = ldg_cg_i32(a.moves + 2 * (long long)(rank - low) + 1);
        }
      }
      a.new_table[(long long)b * a.max_blocks + i] = p;
    }
  }
}

__global__ void __launch_bounds__(256) kv_clear_kernel(const KvPlanArgs a) {
  SpanGuard<kSpanKvPlan> span_guard;
  pdl_wait();
  pdl_launch_dependents();
  const int words = (a.num_blocks + 31) / 32;
  for (int w = blockIdx.x * 256 + threadIdx.x; w < words; w += gridDim.x * 256) a.live[w] = 0;
}

template <class Args>
cudaError_t launch_pdl(const void* fn, unsigned grid, unsigned block, const Args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  Args aa = a;
  void* args[] = {&aa};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_kv_copy(const KvCopyArgs& a, cudaStream_t st) {
  int sms = 0;
  cudaError_t err = device_sms(&sms);
  if (err != cudaSuccess) return err;
  const int grid = a.num_moves < 8 * sms ? a.num_moves : 8 * sms;
  return launch_pdl(reinterpret_cast<const void*>(kv_copy_kernel), (unsigned)grid, kCopyThreads, a, st);
}

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t st) {
  int sms = 0;
  cudaError_t err = device_sms(&sms);
  if (err != cudaSuccess) return err;
  const unsigned rows = (unsigned)(a.B < 4 * sms ? (a.B < 1 ? 1 : a.B) : 4 * sms);
  const int words = (a.num_blocks + 31) / 32;
  const unsigned clear = (unsigned)((words + 255) / 256 < sms ? (words + 255) / 256 : sms);
  err = launch_pdl(reinterpret_cast<const void*>(kv_mark_kernel), rows, 256, a, st);
  if (err == cudaSuccess) err = launch_pdl(reinterpret_cast<const void*>(kv_rank_kernel), 1, kPlanThreads, a, st);
  if (err == cudaSuccess) err = launch_pdl(reinterpret_cast<const void*>(kv_rename_kernel), rows, 256, a, st);
  if (err == cudaSuccess) err = launch_pdl(reinterpret_cast<const void*>(kv_clear_kernel), clear, 256, a, st);
  return err;
}

FLINT_SPAN_SETTER(kv_pages)

}  // namespace flint
