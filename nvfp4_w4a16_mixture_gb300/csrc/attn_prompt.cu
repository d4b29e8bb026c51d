// Causal attention of packed prompts over the paged cache, on the tensor
// cores (flint_attn_prompt where its rows fill 128-row tiles).
//
// Rows: as in attn_rows.cu, packed row r of a sequence and kv head is token
// r / G, head r % G, so the keys are loaded once for the G query heads of a
// group and a causal border crosses few tokens.  A unit is up to 256 packed
// rows (two tiles of 128) of one (sequence, kv head) and the 128-key tiles
// that they see.
//
// Per key tile j and row tile t: S_t = Q_t K_j^T (128 x 128, fp32 in TMEM),
// P = 2^(S c - m) in registers, rounded to bf16 and written over S's columns,
// O_t += P V_j (P from TMEM, V as an N-contiguous operand).  P's rounding to
// bf16 is the type of the second product's tensor-core operand; the row sums
// take the unrounded fp32 values.  m is a running reference in units of log2:
// it moves (and O and the sum are rescaled) only when some score exceeds it
// by more than 8, so P stays below 2^8 and O is seldom touched.
//
// One CTA per SM, 12 warps (two idle, there to make up the third warpgroup
// whose registers the softmax takes over):
//   warps 0-3, 4-7: softmax of row tile 0, 1 (thread = row): Q into swizzled
//     shared memory, then per key tile S from TMEM, P back, and at the
//     unit's end O to the output;
//   warp 8: MMA issue.  Order S_0(0) S_1(0), then per j: PV_0(j) S_0(j+1)
//     PV_1(j) S_1(j+1): while one tile's softmax runs, the other's products
//     do;
//   warp 9: TMA of the key and value tiles (a ring of five 32 KB stages), as
//     boxes of gcd(page, 128) rows, the pages looked up one per lane.
// Shared memory: Q 2 x 32 KB, ring 5 x 32 KB.  TMEM: S_0, S_1, O_0, O_1, 128
// columns each.
//
// Work split: a plan kernel lays all units on a line by their weight (key
// tiles x row tiles + a fixed part) and cuts it into equal pieces, one per
// CTA.  A unit cut by a border is shared: each CTA writes its part (O
// unnormalised, m, l) to the workspace, and the one that finishes last joins
// the parts in CTA order, so the result does not depend on which one that is.
//
// Keys past a sequence's end or on a page outside the cache: their scores
// become -inf and their V rows are zeroed in shared memory before the product
// (whatever the slots hold).  Every wait is bounded (FLINT_ERR_TIMEOUT in the
// status word on expiry).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn.cuh"
#include "tc.cuh"

namespace flint {
namespace {

constexpr int kTile = 128;                 // rows of a row tile; keys of a key tile
constexpr int kUnitRows = 2 * kTile;
constexpr int kHalf = kTile * 128;         // 128 rows x 64 bf16
constexpr int kStageBytes = 2 * kHalf;
constexpr int kStages = 5;
constexpr int kOffRing = 2 * kStageBytes;  // after Q_0, Q_1
constexpr int kOffCtl = kOffRing + kStages * kStageBytes;
constexpr int kWarpMma = 8, kWarpLoad = 9;
constexpr int kThreads = 384;              // three warpgroups
// Registers per thread: 168 at launch (65536 / 384, in eights); the two
// softmax warpgroups take what the third gives up: 2 * 216 + 72 = 3 * 168.
constexpr int kRegsLaunch = 168, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kRegsLaunch, "setmaxnreg.inc would wait for ever");
constexpr int kInfo = 8;                   // key-tile records in flight
constexpr int kUnitWeight = 3;             // a unit's fixed part, in tile products
constexpr int kMinWeight = 8;              // least work of a CTA
constexpr float kLazy = 8.0f;
constexpr unsigned long long kWaitNs = 200ull * 1000 * 1000;
constexpr uint32_t kSuspendNs = 50000;
constexpr int kPartFloats = kUnitRows * (kHeadDim + 2);

struct TileInfo {
  int keys;         // valid keys of the tile (from its start)
  uint32_t bad[4];  // boxes on a page outside the cache
};
struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_free[2], wg[2];
  uint32_t tmem;
  int abort;
  int last[2];
  TileInfo info[kInfo];
};
constexpr size_t kSmem = (size_t)kOffCtl + sizeof(Ctl) + 1024;

// Called by a whole warp, with one answer for all its lanes.
FLINT_DEV bool wait_lane(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  if (mbar_test_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  for (;;) {
    if (*abort) return false;
    if (mbar_try_wait(bar, parity, kSuspendNs)) return true;
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitNs) {
      *abort = 1;
      atomicCAS(status, 0, FLINT_ERR_TIMEOUT);
      return false;
    }
  }
}

FLINT_DEV bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, wait_lane(bar, parity, abort, status));
}

struct Args {
  AttnArgs a;
  PromptWs w;
  int box, box_log2;  // rows of a TMA box: gcd(block_size, 128)
};
struct Maps {
  CUtensorMap k, v;  // {128, heads, slots, pages}, box {64, 1, box, 1}
};

// ---------------------------------------------------------------- the plan
// Entry: up to 256 packed rows of a sequence (all kv heads).
struct Entry {
  int b, lo, n, keys;     // sequence, its first q row, its q rows, its keys
  int r0, rows, tiles, mul;  // packed rows, key tiles seen, row tiles at work
};
FLINT_DEV long long weight(const Entry& e) { return (long long)e.tiles * e.mul + kUnitWeight; }

FLINT_DEV Entry load_entry(const PromptWs& w, int i) {
  const uint4 x = ldg_cg_v4(w.entries + 2 * (long long)i), y = ldg_cg_v4(w.entries + 2 * (long long)i + 1);
  Entry e;
  e.b = (int)x.x; e.lo = (int)x.y; e.n = (int)x.z; e.keys = (int)x.w;
  e.r0 = (int)y.x; e.rows = (int)y.y; e.tiles = (int)y.z; e.mul = (int)y.w;
  return e;
}

FLINT_DEV long long scan_cta64(long long v, long long* warps, long long* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = warps[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    warps[lane] = w;
  }
  __syncthreads();
  const long long r = x - v + (warp ? warps[warp - 1] : 0);
  *all = warps[31];
  __syncthreads();
  return r;
}

// One CTA: entries of all sequences, their weights' prefix sums, and the
// first unit of each of the main kernel's CTAs.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const Args p, int ctas) {
  SpanGuard<kSpanAttnPrompt> span_guard;
  pdl_wait();
  pdl_launch_dependents();
  __shared__ long long warps[32];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, G = a.nq / a.nkv;
  long long n_entries = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int lo = 0, n = 0;
    if (b < a.B) seq_rows(a, b, lo, n);
    long long all;
    const long long mine = b < a.B ? ((long long)n * G + kUnitRows - 1) / kUnitRows : 0;
    const long long at = n_entries + scan_cta64(mine, warps, &all);
    if (b < a.B) p.w.first[b] = (int)at;
    n_entries += all;
  }
  if (tid == 0) p.w.first[a.B] = (int)n_entries;
  __syncthreads();
  // a warp per sequence writes its entries (overlapping pieces of a bad cu_q
  // could outgrow the table: cut off there)
  const long long most = (long long)a.T * G / kUnitRows + a.B;
  if (n_entries > most) {
    if (tid == 0) attn_error(a.status);
    n_entries = most;
  }
  for (int b = tid >> 5; b < a.B; b += kPlanThreads / 32) {
    int lo, n;
    seq_rows(a, b, lo, n);
    const int keys = seq_keys(a, b);
    const int e0 = ldg_cg_i32(p.w.first + b), e1 = min((long long)ldg_cg_i32(p.w.first + b + 1), n_entries);
    for (int e = e0 + (tid & 31); e < e1; e += 32) {
      const int r0 = (e - e0) * kUnitRows, rows = min(kUnitRows, n * G - r0);
      const int seen = max(0, min(keys, keys - n + (r0 + rows - 1) / G + 1));  // by its last row
      p.w.entries[2 * (long long)e] = make_int4(b, lo, n, keys);
      p.w.entries[2 * (long long)e + 1] =
          make_int4(r0, rows, (seen + kTile - 1) / kTile, rows > kTile ? 2 : 1);
    }
  }
  __syncthreads();
  long long total = 0;
  for (long long e0 = 0; e0 < n_entries; e0 += kPlanThreads) {
    const long long e = e0 + tid;
    long long all;
    const long long at = total + scan_cta64(e < n_entries ? weight(load_entry(p.w, (int)e)) * a.nkv : 0, warps, &all);
    if (e < n_entries) p.w.prefix[e] = at;
    total += all;
  }
  if (tid == 0) p.w.prefix[n_entries] = total;
  __syncthreads();
  const long long n_cta = total == 0 ? 0 : max(1ll, min((long long)ctas, total / kMinWeight));
  if (tid == 0) {
    p.w.head[0] = total;
    p.w.head[1] = n_cta;
  }
  // CTA c's piece begins at floor(c total / n_cta); entry e writes those inside it
  for (long long e = tid; e < n_entries; e += kPlanThreads) {
    const Entry x = load_entry(p.w, (int)e);
    const long long w = weight(x), at = p.w.prefix[e], end = at + w * a.nkv;
    for (long long c = (at * n_cta + total - 1) / total; c < n_cta; ++c) {
      const long long pos = c * total / n_cta;
      if (pos >= end) break;
      if (pos < at) continue;
      p.w.starts[c] = make_int4((int)e, (int)((pos - at) / w), (int)((pos - at) % w), 0);
    }
  }
}

// ------------------------------------------------------------- the pieces
// One CTA's walk along its piece: the same in every role.
struct Walk {
  const PromptWs* w;
  int nkv;
  long long total, ctas, rem;
  int cta, i, h, off;
  Entry e;
  // the current step
  int t0, t1;          // key tiles
  int c_first, c_last; // CTAs that share the unit
};

FLINT_DEV bool walk_start(Walk& k, const Args& p) {
  k.w = &p.w;
  k.nkv = p.a.nkv;
  k.cta = blockIdx.x;
  const uint4 hd = ldg_cg_v4(p.w.head);
  k.total = (long long)hd.x | ((long long)hd.y << 32);
  k.ctas = (long long)hd.z | ((long long)hd.w << 32);
  if (k.cta >= k.ctas) return false;
  const long long at = k.cta * k.total / k.ctas;
  k.rem = (k.cta + 1) * k.total / k.ctas - at;
  const uint4 s = ldg_cg_v4(p.w.starts + k.cta);
  k.i = (int)s.x; k.h = (int)s.y; k.off = (int)s.z;
  k.e = load_entry(p.w, k.i);
  return true;
}

// The next part of a unit in this CTA's piece; false at its end.
FLINT_DEV bool walk_next(Walk& k, Entry& u, int& h) {
  while (k.rem > 0) {
    const int wgt = (int)weight(k.e);
    const int take = (int)min((long long)(wgt - k.off), k.rem);
    const int real = max(1, k.e.tiles * k.e.mul);
    const bool at_work = k.off < real;
    if (at_work) {
      u = k.e;
      h = k.h;
      k.t0 = min(k.off / k.e.mul, k.e.tiles);
      k.t1 = min((k.off + take) / k.e.mul, k.e.tiles);
      k.c_first = k.c_last = k.cta;
      if (k.off > 0 || take < real) {  // CTA of position x: floor(((x + 1) ctas - 1) / total)
        const long long at = __ldcg(k.w->prefix + k.i) + (long long)k.h * wgt;
        k.c_first = (int)(((at + 1) * k.ctas - 1) / k.total);
        k.c_last = (int)(((at + real) * k.ctas - 1) / k.total);
      }
    }
    k.rem -= take;
    k.off += take;
    if (k.off == wgt) {
      k.off = 0;
      if (++k.h == k.nkv) {
        k.h = 0;
        ++k.i;
        if (k.rem > 0) k.e = load_entry(*k.w, k.i);
      }
    }
    if (at_work) return true;
  }
  return false;
}

FLINT_DEV uint32_t pack2(float a, float b) {
  __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&r);
}

// A finished row's 32 columns from c0 on, scaled, to bf16.
FLINT_DEV void store_cols(uint16_t* dst, const float* o, float inv) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    *reinterpret_cast<uint4*>(dst + i) =
        make_uint4(pack2(o[i] * inv, o[i + 1] * inv), pack2(o[i + 2] * inv, o[i + 3] * inv),
                   pack2(o[i + 4] * inv, o[i + 5] * inv), pack2(o[i + 6] * inv, o[i + 7] * inv));
}

// -------------------------------------------------------------- the softmax
FLINT_DEV void softmax_role(const Args& p, Ctl& C, uint8_t* smem, uint32_t tmem, int t) {
  const AttnArgs& a = p.a;
  const int G = a.nq / a.nkv;
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = 32 * warp + lane;  // of the tile
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t tS = tmem + lanes + (uint32_t)(kTile * t);
  const uint32_t tO = tmem + lanes + (uint32_t)(2 * kTile + kTile * t);
  uint8_t* sq = smem + t * kStageBytes;
  const float c = a.scale * 1.4426950408889634f;
  volatile int* abort = &C.abort;
  uint32_t n_s = 0, n_o = 0, n_wg = 0;  // phases done: s_full, o_full, wg
  int n_tile = 0;                       // key tiles of the CTA so far
  Walk k;
  Entry u;
  int h;
  if (!walk_start(k, p)) return;
  while (!*abort && walk_next(k, u, h)) {
    const int nt = k.t1 - k.t0;
    if (u.rows <= kTile * t) {  // the unit has one row tile
      n_tile += nt;
      continue;
    }
    if (nt > 0) {
      // Q_t: 16 lanes per row
      const int ch = lane & 15;
#pragma unroll
      for (int i0 = 0; i0 < 16; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 32 * warp + 2 * (i0 + i) + (lane >> 4), R = kTile * t + r;
          const int q = u.r0 + R, token = q / G, head = h * G + q - token * G;
          v[i] = R < u.rows ? ldg_cg_v4(a.q + (long long)(u.lo + token) * a.q_stride + (long long)head * kHeadDim + 8 * ch)
                            : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 32 * warp + 2 * (i0 + i) + (lane >> 4);
          *reinterpret_cast<uint4*>(sq + (ch >> 3) * kHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v[i];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&C.q_full[t]);
    }
    const int R = kTile * t + row, q = u.r0 + R;
    const bool valid = R < u.rows;
    const int lim = u.keys - u.n + q / G;  // last key that the row sees
    const int lim0 = u.keys - u.n + (u.r0 + kTile * t + 32 * warp) / G;  // the warp's first row
    float m = neg_inf(), l = 0.0f;
    bool ok = true;
    for (int j = k.t0; j < k.t1; ++j, ++n_tile) {
      if (!wait(&C.s_full[t], n_s & 1, abort, a.status)) { ok = false; break; }
      ++n_s;
      tc::fence_after_sync();
      uint32_t s[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tc::tmem_ld32_async(tS + 32 * i, s[i]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 4; ++i) tc::tmem_regs_ready(s[i]);
      const TileInfo& info = C.info[n_tile % kInfo];
      const int keys = info.keys;
      const bool bad = (info.bad[0] | info.bad[1] | info.bad[2] | info.bad[3]) != 0;
      if (keys < kTile || j * kTile + kTile - 1 > lim0) {
        const int vis = min(keys, lim - j * kTile + 1);
#pragma unroll
        for (int i = 0; i < kTile; ++i)
          if (i >= vis) s[i >> 5][i & 31] = 0xff800000u;
      }
      if (bad) {
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
          const int box = i >> p.box_log2;
          if ((info.bad[box >> 5] >> (box & 31)) & 1u) s[i >> 5][i & 31] = 0xff800000u;
        }
      }
      float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
      for (int i = 0; i < kTile; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i >> 5][i & 31]));
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
      const bool raise = mt > m + kLazy;
      if (j > k.t0 && __any_sync(0xffffffffu, raise)) {
        // S(j) was issued after PV(j - 1) and has completed, so O is stable
        const float to = fmaxf(m, mt);
        const float r = m == to ? 1.0f : ex2(m - to);
        m = to;
        l *= r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[32];
          tc::tmem_ld32(tO + 32 * i, o);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * r);
          tc::tmem_st32(tO + 32 * i, o);
        }
      } else if (j == k.t0) {
        m = mt;
      }
      const float neg = m == neg_inf() ? 0.0f : -m;
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float e = ex2(fmaf(__uint_as_float(s[i][x]), c, neg));
          sum[x & 3] += e;
          s[i][x] = __float_as_uint(e);
        }
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      uint32_t pk[2][32];
#pragma unroll
      for (int i = 0; i < 64; ++i)
        pk[i >> 5][i & 31] = pack2(__uint_as_float(s[i >> 4][(2 * i) & 31]), __uint_as_float(s[i >> 4][(2 * i + 1) & 31]));
      tc::tmem_st32(tS, pk[0]);
      tc::tmem_st32(tS + 32, pk[1]);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&C.p_full[t]);
    }
    if (!ok) break;
    if (nt > 0) {
      if (!wait(&C.o_full[t], n_o & 1, abort, a.status)) break;
      ++n_o;
      tc::fence_after_sync();
    }
    const int token = q / G, head = h * G + q - token * G;
    const long long orow = (long long)(u.lo + token) * a.nq + head;
    uint16_t* dst = a.out + orow * kHeadDim;
    const bool whole = k.c_first == k.c_last;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    float* part = p.w.parts + (size_t)(2 * k.cta + (k.cta == k.c_first)) * kPartFloats;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t o[32];
      if (nt > 0) {
        tc::tmem_ld32(tO + 32 * i, o);
      } else {
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = 0;
      }
      if (whole) {
        if (valid) store_cols(dst + 32 * i, reinterpret_cast<const float*>(o), inv);
      } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          *reinterpret_cast<uint4*>(part + ((size_t)(8 * i + x) * kUnitRows + R) * 4) =
              make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
      }
    }
    if (nt > 0) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&C.o_free[t]);
    }
    if (whole) {
      if (valid && a.lse) a.lse[orow] = l == 0.0f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
      continue;
    }
    part[kHeadDim * kUnitRows + R] = m;
    part[(kHeadDim + 1) * kUnitRows + R] = l;
    // the last of the unit's CTAs joins the parts
    __threadfence();
    __syncwarp();
    if (lane == 0) mbar_arrive(&C.wg[t]);
    if (!wait(&C.wg[t], n_wg & 1, abort, a.status)) break;
    ++n_wg;
    if (warp == 0 && lane == 0) {
      __threadfence();
      int* cnt = p.w.count + 2 * k.c_first + t;
      const int last = atomicAdd(cnt, 1) == k.c_last - k.c_first;
      if (last) *cnt = 0;
      C.last[t] = last;
      __threadfence();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&C.wg[t]);
    if (!wait(&C.wg[t], n_wg & 1, abort, a.status)) break;
    ++n_wg;
    if (!*reinterpret_cast<volatile int*>(&C.last[t])) continue;
    __threadfence();
    m = neg_inf();
    for (int x = k.c_first; x <= k.c_last; ++x)
      m = fmaxf(m, __ldcg(p.w.parts + (size_t)(2 * x + (x == k.c_first)) * kPartFloats + kHeadDim * kUnitRows + R));
    l = 0.0f;
    float o[4][32];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < 32; ++x) o[i][x] = 0.0f;
    for (int x = k.c_first; x <= k.c_last; ++x) {
      const float* pp = p.w.parts + (size_t)(2 * x + (x == k.c_first)) * kPartFloats;
      const float pm = __ldcg(pp + kHeadDim * kUnitRows + R), pl = __ldcg(pp + (kHeadDim + 1) * kUnitRows + R);
      const float f = pm == neg_inf() ? (pl == 0.0f ? 0.0f : 1.0f) : ex2(pm - m);
      l += f * pl;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(pp) + (size_t)i * kUnitRows + R);
        o[i >> 3][4 * (i & 7)] += f * v.x;
        o[i >> 3][4 * (i & 7) + 1] += f * v.y;
        o[i >> 3][4 * (i & 7) + 2] += f * v.z;
        o[i >> 3][4 * (i & 7) + 3] += f * v.w;
      }
    }
    if (valid) {
      const float iv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int i = 0; i < 4; ++i) store_cols(dst + 32 * i, o[i], iv);
      if (a.lse) a.lse[orow] = l == 0.0f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
}

// ------------------------------------------------------------------ the MMAs
FLINT_DEV void mma_role(const Args& p, Ctl& C, uint8_t* smem, uint32_t tmem) {
  const int lane = threadIdx.x & 31;
  volatile int* abort = &C.abort;
  int* status = p.a.status;
  const uint32_t idS = tc::idesc_bf16(kTile, kTile), idO = idS | tc::kIdescBMajorN;
  uint32_t it = 0, n_q[2] = {0, 0}, n_p[2] = {0, 0}, n_o[2] = {0, 0};
  int n_tile = 0;
  Walk k;
  Entry u;
  int h;
  if (!walk_start(k, p)) return;
  auto stage_wait = [&](uint32_t i) { return wait(&C.full[i % kStages], (i / kStages) & 1, abort, status); };
  auto issue_s = [&](int t, uint32_t i) {  // S_t = Q_t K^T, K in ring slot i
    if (lane == 0) {
      const uint64_t dq = tc::desc_sw128(smem + t * kStageBytes);
      const uint64_t dk = tc::desc_sw128(smem + kOffRing + (i % kStages) * kStageBytes);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint64_t o = (uint64_t)((kk >> 2) * (kHalf >> 4) + 2 * (kk & 3));
        tc::mma_bf16(tmem + (uint32_t)(kTile * t), dq + o, dk + o, idS, kk > 0);
      }
      mbar_arrive(&C.s_full[t]);  // orders the tile's record before the softmax's reads
      tc::commit(&C.s_full[t]);
    }
    __syncwarp();
  };
  while (!*abort && walk_next(k, u, h)) {
    const int nt = k.t1 - k.t0;
    if (nt == 0) continue;
    const int tiles = u.rows > kTile ? 2 : 1;
    // ring slots: it + 2 j is K_j, it + 2 j + 1 is V_j
    bool ok = stage_wait(it);
    for (int t = 0; ok && t < tiles; ++t) {
      ok = wait(&C.q_full[t], n_q[t] & 1, abort, status);
      if (!ok) break;
      ++n_q[t];
      tc::fence_after_sync();
      issue_s(t, it);
    }
    if (!ok) break;
    if (lane == 0) tc::commit(&C.empty[it % kStages]);
    __syncwarp();
    for (int j = 0; j < nt; ++j) {
      const uint32_t iv = it + 2 * j + 1, ik = it + 2 * j + 2;
      ok = stage_wait(iv);
      if (!ok) break;
      uint8_t* sv = smem + kOffRing + (iv % kStages) * kStageBytes;
      const TileInfo& info = C.info[(n_tile + j) % kInfo];
      if (info.keys < kTile || (info.bad[0] | info.bad[1] | info.bad[2] | info.bad[3]) != 0) {
        // V rows that were not loaded, or past the sequence's end: zeros
        for (int r = 0; r < kTile; ++r) {
          const int box = r >> p.box_log2;
          if (r >= info.keys || ((info.bad[box >> 5] >> (box & 31)) & 1u))
            *reinterpret_cast<uint2*>(sv + (lane >> 4) * kHalf + r * 128 + (lane & 15) * 8) = make_uint2(0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (j + 1 < nt) {
        ok = stage_wait(ik);
        if (!ok) break;
      }
      for (int t = 0; t < tiles; ++t) {
        ok = wait(&C.p_full[t], n_p[t] & 1, abort, status);
        if (!ok) break;
        ++n_p[t];
        if (j == 0) {  // O_t of the CTA's previous unit has been read
          if (n_o[t] > 0) ok = wait(&C.o_free[t], (n_o[t] - 1) & 1, abort, status);
          if (!ok) break;
          ++n_o[t];
        }
        tc::fence_after_sync();
        if (lane == 0) {
          const uint64_t dv = tc::desc_sw128_mn(sv, kHalf);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16_ta(tmem + (uint32_t)(2 * kTile + kTile * t), tmem + (uint32_t)(kTile * t + 8 * kk),
                            dv + (uint64_t)(kk * (2048 >> 4)), idO, j > 0 || kk > 0);
          if (j + 1 == nt) tc::commit(&C.o_full[t]);
        }
        __syncwarp();
        if (j + 1 < nt) issue_s(t, ik);
      }
      if (!ok) break;
      if (lane == 0) {
        tc::commit(&C.empty[iv % kStages]);
        if (j + 1 < nt) tc::commit(&C.empty[ik % kStages]);
      }
      __syncwarp();
    }
    if (!ok) break;
    it += 2 * nt;
    n_tile += nt;
  }
}

// ------------------------------------------------------------------ the loads
FLINT_DEV void load_role(const Args& p, const Maps& maps, Ctl& C, uint8_t* smem) {
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &C.abort;
  const int boxes = kTile / p.box;  // per tile: one lane each up to 32
  uint32_t it = 0;
  int n_tile = 0;
  bool ok = true;
  Walk k;
  Entry u;
  int h;
  if (!walk_start(k, p)) return;
  while (ok && !*abort && walk_next(k, u, h)) {
    for (int j = k.t0; ok && j < k.t1; ++j, ++n_tile) {
      const int key0 = j * kTile, keys = min(kTile, u.keys - key0);
      // pages of this lane's boxes (lane + 32 x)
      int page[4], slot[4];
      uint32_t good[4];
      TileInfo info;
      info.keys = keys;
      int n_good = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int box = lane + 32 * x, first = box * p.box;
        const bool want = box < boxes && first < keys;
        page[x] = 0;
        slot[x] = 0;
        bool in = false;
        if (want) {
          const int pos = key0 + first, blk = pos / a.block_size;
          slot[x] = pos - blk * a.block_size;
          page[x] = ldg_cg_i32(a.block_table + (long long)u.b * a.table_stride + blk);
          in = page[x] >= 0 && page[x] < a.num_blocks;
          if (!in) attn_error(a.status);
        }
        good[x] = __ballot_sync(0xffffffffu, in);
        info.bad[x] = __ballot_sync(0xffffffffu, want && !in);
        n_good += __popc(good[x]);
      }
      const uint32_t bytes = (uint32_t)(n_good * p.box * 2 * 128);
      for (int kv = 0; kv < 2; ++kv, ++it) {
        const int s = it % kStages;
        if (it >= (uint32_t)kStages) ok = wait(&C.empty[s], ((it / kStages) - 1) & 1, abort, a.status);
        if (!ok) break;
        if (lane == 0) {
          if (kv == 0) C.info[n_tile % kInfo] = info;
          mbar_arrive_expect_tx(&C.full[s], bytes);
        }
        __syncwarp();
        uint8_t* st = smem + kOffRing + s * kStageBytes;
        const CUtensorMap* map = kv ? &maps.v : &maps.k;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if ((good[x] >> lane) & 1u) {
            uint8_t* dst = st + (lane + 32 * x) * p.box * 128;
            tc::tma_load_4d(dst, map, 0, h, slot[x], page[x], &C.full[s]);
            tc::tma_load_4d(dst + kHalf, map, 64, h, slot[x], page[x], &C.full[s]);
          }
        }
        __syncwarp();
      }
    }
  }
  if (*abort) {  // no copy may land after the block has exited
    const uint32_t n = it < (uint32_t)kStages ? it : (uint32_t)kStages;
    for (uint32_t i = it - n; i < it; ++i) {
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_test_wait(&C.full[i % kStages], (i / kStages) & 1) && globaltimer_ns() - t0 < kWaitNs) {
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ Args p, const __grid_constant__ Maps maps) {
  SpanGuard<kSpanAttnPrompt> span_guard;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Ctl& C = *reinterpret_cast<Ctl*>(smem + kOffCtl);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&C.full[i], 1);
      mbar_init(&C.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&C.q_full[t], 4);
      mbar_init(&C.s_full[t], 2);
      mbar_init(&C.p_full[t], 4);
      mbar_init(&C.o_full[t], 1);
      mbar_init(&C.o_free[t], 4);
      mbar_init(&C.wg[t], 4);
    }
    C.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tc::tmem_alloc(&C.tmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = C.tmem;
  pdl_wait();  // the plan, q and the cache's newest rows are earlier kernels' output
  pdl_launch_dependents();
  if (warp < kWarpMma) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_role(p, C, smem, tmem, warp >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kWarpMma)
      mma_role(p, C, smem, tmem);
    else if (warp == kWarpLoad)
      load_role(p, maps, C, smem);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// --------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

int box_rows(int page) {
  int b = 1;
  while (b < kTile && page % (2 * b) == 0) b *= 2;
  return b;
}

bool make_map(CUtensorMap* m, const AttnArgs& a, const uint16_t* base, int box) {
  auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {kHeadDim, (cuuint64_t)a.nkv, (cuuint64_t)a.block_size, (cuuint64_t)a.num_blocks};
  // the stride of an extent of 1 is never used, but has to be a valid one
  const cuuint64_t strides[3] = {(cuuint64_t)(a.nkv > 1 ? a.s_head * 2 : 256),
                                 (cuuint64_t)(a.block_size > 1 ? a.s_slot * 2 : 256),
                                 (cuuint64_t)(a.num_blocks > 1 ? a.s_block * 2 : 256)};
  for (cuuint64_t s : strides)
    if (s == 0 || s >= (1ull << 40)) return false;
  const cuuint32_t bx[4] = {64, 1, (cuuint32_t)box, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

PromptWs prompt_ws(void* base, int T, int B, int nq, int nkv) {
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = kAttnData;
  auto take = [&](size_t n) {
    uint8_t* p = b + off;
    off += (n + 255) / 256 * 256;
    return p;
  };
  const size_t entries = (size_t)T * (nq / nkv) / kUnitRows + B;
  PromptWs w;
  static_assert(kAttnPromptCounters + 2 * kPromptCtas * sizeof(int) <= kAttnData, "counters overlap");
  w.count = reinterpret_cast<int*>(b + kAttnPromptCounters);
  w.parts = reinterpret_cast<float*>(take((size_t)2 * kPromptCtas * kPartFloats * sizeof(float)));
  w.starts = reinterpret_cast<int4*>(take((kPromptCtas + 1) * sizeof(int4)));
  w.head = reinterpret_cast<long long*>(take(2 * sizeof(long long)));
  w.first = reinterpret_cast<int*>(take((size_t)(B + 1) * sizeof(int)));
  w.entries = reinterpret_cast<int4*>(take(entries * 2 * sizeof(int4)));
  w.prefix = reinterpret_cast<long long*>(take((entries + 1) * sizeof(long long)));
  w.total = off;
  return w;
}

cudaError_t launch_attn_prompt(const AttnArgs& a, const PromptWs& w, cudaStream_t st) {
  Args p;
  p.a = a;
  p.w = w;
  p.box = box_rows(a.block_size);
  for (p.box_log2 = 0; (1 << p.box_log2) < p.box;) ++p.box_log2;
  Maps maps;
  if (!make_map(&maps.k, a, a.k, p.box) || !make_map(&maps.v, a, a.v, p.box)) return cudaErrorNotSupported;
  int sms = 0;
  cudaError_t err = device_sms(&sms);
  if (err != cudaSuccess) return err;
  int ctas = sms < kPromptCtas ? sms : kPromptCtas;
  const void* fn = reinterpret_cast<const void*>(attn_prompt_kernel);
  static std::atomic<bool> allowed[64], checked;
  err = allow_smem(fn, (int)kSmem, allowed);
  if (err != cudaSuccess) return err;
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa;
    err = cudaFuncGetAttributes(&fa, fn);
    if (err != cudaSuccess) return err;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split needs them
    checked.store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  void* plan_args[] = {&p, &ctas};
  err = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(attn_plan_kernel), plan_args);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  void* args[] = {&p, &maps};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

FLINT_SPAN_SETTER(attn_prompt)

}  // namespace flint
