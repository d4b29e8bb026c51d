// Pages of the paged KV cache: copies of whole or part-filled pages, and the
// plan of a compaction.
//
// Copy: bytes only.  A (pair, K or V, slot, head) row is 256 contiguous
// bytes, 16 threads x 16 bytes; a CTA takes 64 rows of a pair's keys and
// values at a time, eight 16-byte loads of each thread under way before the
// first store, and asks for the next pair's page ids meanwhile.  8 CTAs an SM
// share the items.  4360 pages of 16 slots and 4 heads: 46 us, 6.1 TB/s read
// and written (a plain copy reaches 6.8); with 4 CTAs an SM 50, with a CTA per
// item 60, with half the loads under way 47, with a quarter 56.
// Plan: two kernels.  The first sets the bit of every page in use, and its
// last CTA scans the bitmap: the live count, each word's number of live pages
// below it, and the pairs; it leaves a copy of the bitmap for the second and
// the bitmap itself cleared for the next call.  The second writes the new
// table and fills up the list of pairs.  All in integers, so the result does
// not depend on the order of the atomics.  48 sequences in a pool of 24000
// pages: 11 us, a chain of latencies (lengths and entries, atomics, the last
// CTA's scan, its list, the second kernel's look-ups).
#include "attn.cuh"

namespace flint {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kRowStep = kCopyThreads / 16;      // rows that the CTA's threads cover at once
constexpr int kRowsPer = 4;                      // rows of a thread
constexpr int kCopyRows = kRowStep * kRowsPer;   // rows of an item
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const KvCopyArgs a) {
  SpanGuard<kSpanKvCopy> span_guard;
  pdl_wait();  // the pairs and the pages are earlier kernels' output
  pdl_launch_dependents();
  int n = a.num_moves;
  if (a.count) n = min(n, ldg_cg_i32(a.count));
  const int rows = a.block_size * a.nkv;
  const int parts = (rows + kCopyRows - 1) / kCopyRows;  // per pair
  const int step_slot = kRowStep / a.nkv, step_head = kRowStep % a.nkv;
  const long long items = (long long)max(n, 0) * parts;
  struct Move {
    int src, dst, tokens;
  };
  auto ask = [&](long long item) {
    Move m = {0, 0, 0};
    if (item < items) {
      const long long i = item / parts;
      m.src = ldg_cg_i32(a.moves + 2 * i);
      m.dst = ldg_cg_i32(a.moves + 2 * i + 1);
      m.tokens = a.tokens ? ldg_cg_i32(a.tokens + i) : a.block_size;
    }
    return m;
  };
  Move next = ask(blockIdx.x);
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const Move m = next;
    next = ask(item + gridDim.x);
    const bool bad = m.src < 0 || m.src >= a.num_blocks || m.dst < 0 || m.dst >= a.num_blocks;
    if ((bad || m.tokens < 0 || m.tokens > a.block_size) && threadIdx.x == 0) attn_error(a.status);
    if (bad) continue;
    const int end = min(max(m.tokens, 0), a.block_size) * a.nkv;  // rows to copy
    int r = (int)(item % parts) * kCopyRows + (int)threadIdx.x / 16;
    int slot = r / a.nkv, head = r - slot * a.nkv;
    const long long src = m.src * a.s_block, to = m.dst * a.s_block - src;
    long long at[kRowsPer];
    uint4 kv[kRowsPer], vv[kRowsPer];
#pragma unroll
    for (int x = 0; x < kRowsPer; ++x) {
      at[x] = r < end ? src + slot * a.s_slot + head * a.s_head + 8 * ((int)threadIdx.x % 16) : -1;
      if (at[x] >= 0) {
        kv[x] = ldg_cg_v4(a.k + at[x]);
        vv[x] = ldg_cg_v4(a.v + at[x]);
      }
      r += kRowStep;
      slot += step_slot;
      head += step_head;
      if (head >= a.nkv) {
        head -= a.nkv;
        ++slot;
      }
    }
#pragma unroll
    for (int x = 0; x < kRowsPer; ++x)
      if (at[x] >= 0) {
        *reinterpret_cast<uint4*>(a.k + at[x] + to) = kv[x];
        *reinterpret_cast<uint4*>(a.v + at[x] + to) = vv[x];
      }
  }
}

// Pages of a sequence of n keys, n taken into the table's reach.
FLINT_DEV int seq_pages(const KvPlanArgs& a, int n) {
  const long long most = (long long)a.max_blocks * a.block_size;
  if (n < 0 || n > most) {
    attn_error(a.status);
    return n < 0 ? 0 : a.max_blocks;
  }
  return (int)(((long long)n + a.block_size - 1) / a.block_size);
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

// The used pages' bits; then, in the CTA that comes last, the ranks and pairs.
__global__ void __launch_bounds__(kPlanThreads) kv_mark_kernel(const KvPlanArgs a) {
  SpanGuard<kSpanKvPlan> span_guard;
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int warps[32];
  __shared__ int s_last;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    // (the first entries are asked for together with the length)
    const int* row = a.block_table + (long long)b * a.table_stride;
    int p = (int)threadIdx.x < a.max_blocks ? ldg_cg_i32(row + threadIdx.x) : 0;
    const int used = seq_pages(a, ldg_cg_i32(a.seq_lens + b));
    for (int i = threadIdx.x; i < used; i += kPlanThreads) {
      if (i >= kPlanThreads) p = ldg_cg_i32(row + i);
      if (p < 0 || p >= a.num_blocks)
        attn_error(a.status);
      else
        atomicOr(a.live + (p >> 5), 1u << (p & 31));
    }
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int last = atomicAdd(a.done, 1) == (int)gridDim.x - 1;
    if (last) *a.done = 0;
    s_last = last;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  const int words = (a.num_blocks + 31) / 32;
  int live = 0;
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x;
    const uint32_t bits = w < words ? ldg_cg_u32(a.live + w) : 0u;
    int all;
    const int below = scan_cta(__popc(bits), warps, &all);
    if (w < words) {
      a.rank[w] = live + below;
      a.bits[w] = bits;
      a.live[w] = 0u;
    }
    live += all;
  }
  // live pages below `live`: what its word's rank and lower bits say
  __shared__ int s_low;
  if (threadIdx.x == 0) s_low = live;  // (all pages are live)
  __syncthreads();
  if (live < a.num_blocks && (live >> 5) % kPlanThreads == (int)threadIdx.x)  // the thread that wrote that word
    s_low = a.rank[live >> 5] + __popc(a.bits[live >> 5] & ((1u << (live & 31)) - 1u));
  __syncthreads();
  const int low = s_low;
  // A warp takes a word's pages at once, lane = page, so that its store fills
  // whole lines: the ranks of neighbouring pages are neighbours in the list.
  const int lane = threadIdx.x & 31;
  const uint32_t lower = (1u << lane) - 1u;
  for (int w0 = (int)threadIdx.x & ~31; w0 < words; w0 += kPlanThreads) {
    const int n = min(32, words - w0);
    const int ranks = lane < n ? a.rank[w0 + lane] : 0;
    const uint32_t bitss = lane < n ? a.bits[w0 + lane] : 0u;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const uint32_t bits = __shfl_sync(0xffffffffu, bitss, j);
      const int used_below = __shfl_sync(0xffffffffu, ranks, j) + __popc(bits & lower);
      const int p = 32 * (w0 + j) + lane;
      const bool used = (bits >> lane) & 1u, high = p >= live;
      // used, to be moved: a pair's first; unused, to be filled: its second
      if (used == high && p < a.num_blocks) a.moves[2 * (long long)(high ? used_below - low : p - used_below) + !high] = p;
    }
  }
  if (threadIdx.x == 0) {
    a.counts[0] = live;
    a.counts[1] = live - low;
  }
}

constexpr int kRenameThreads = 512;
__global__ void __launch_bounds__(kRenameThreads) kv_rename_kernel(const KvPlanArgs a) {
  SpanGuard<kSpanKvPlan> span_guard;
  pdl_wait();
  pdl_launch_dependents();
  const int live = ldg_cg_i32(a.counts), above = ldg_cg_i32(a.counts + 1), low = live - above;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int* row = a.block_table + (long long)b * a.table_stride;
    const int n = ldg_cg_i32(a.seq_lens + b);
    int at = (int)threadIdx.x < a.max_blocks ? ldg_cg_i32(row + threadIdx.x) : 0;
    const int used = seq_pages(a, n);
    for (int i = threadIdx.x; i < a.max_blocks; i += kRenameThreads) {
      int p = -1;
      if (i < used) {
        p = i < kRenameThreads ? at : ldg_cg_i32(row + i);
        if (p < 0 || p >= a.num_blocks) {
          p = -1;
        } else if (p >= live) {
          const int rank = ldg_cg_i32(a.rank + (p >> 5)) + __popc(ldg_cg_u32(a.bits + (p >> 5)) & ((1u << (p & 31)) - 1));
          p = ldg_cg_i32(a.moves + 2 * (long long)(rank - low) + 1);
        }
      }
      a.new_table[(long long)b * a.max_blocks + i] = p;
    }
  }
  const long long end = a.num_blocks / 2 * 2;  // (of the list's ints)
  for (long long i = 2ll * above + blockIdx.x * kRenameThreads + threadIdx.x; i < end;
       i += (long long)gridDim.x * kRenameThreads) a.moves[i] = -1;
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
  const long long parts = ((long long)a.block_size * a.nkv + kCopyRows - 1) / kCopyRows;
  const long long items = a.num_moves * parts, most = 8ll * sms;
  return launch_pdl(reinterpret_cast<const void*>(kv_copy_kernel), (unsigned)(items < most ? items : most),
                    kCopyThreads, a, st);
}

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t st) {
  int sms = 0;
  cudaError_t err = device_sms(&sms);
  if (err != cudaSuccess) return err;
  const int rows = a.B < 1 ? 1 : a.B;
  err = launch_pdl(reinterpret_cast<const void*>(kv_mark_kernel), (unsigned)(rows < sms ? rows : sms), kPlanThreads, a, st);
  if (err != cudaSuccess) return err;
  return launch_pdl(reinterpret_cast<const void*>(kv_rename_kernel), (unsigned)(rows < 4 * sms ? rows : 4 * sms),
                    kRenameThreads, a, st);
}

FLINT_SPAN_SETTER(kv_pages)

}  // namespace flint
