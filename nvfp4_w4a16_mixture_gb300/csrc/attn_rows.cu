// Attention of one new token per sequence over the paged cache
// (flint_attn_decode).
//
// The rows of one sequence and kv head are the query heads of its group (G
// heads per kv head), so one pass over the keys serves the whole group.  A
// unit is up to 8 NT rows of one (sequence, kv head) and all its keys, in
// tiles of 128: 16 keys for each of the CTA's 8 warps.
//
// Per 16 keys a warp forms S^T = K Q^T and O^T += V^T P on mma.sync
// m16n8k16 with the keys (then the head's dims) as the 16-row operand and 8
// rows as the 8 columns, so a group of 8 heads wastes nothing.  The
// bytes that a lane's operand registers need are the lane's own 16-byte
// pieces of the cache:
//  - K: lane (g, t) = (lane / 4, lane % 4) takes dims 32 i + 8 t .. + 7 of
//    keys g and g + 8; the four words are the operands of two k-steps (Q is
//    loaded with the same permutation of the dims, and a sum does not depend
//    on their order);
//  - V: lane (g, t) takes dims 8 g .. + 7 and 64 + 8 g .. + 7 of keys 2t,
//    2t + 1, 2t + 8, 2t + 9; a byte permutation pairs two keys' values of one
//    dim, and dim 8 g + j (64 + 8 g + j) is row g (g + 8) of tile j.
// So each lane copies its own pieces ahead of use (cp.async into a ring of
// kDepth chunks of 8 KB per warp) and reads back only what it wrote: no
// barrier in the loop, and the ring runs on across units.
// P's accumulator layout (row = key) becomes the operand layout (row = packed
// row) by movmatrix.  P enters as hi + lo, two bf16 values (relative error
// 2^-18): a single bf16 would double the output's squared rounding error, and
// the kernel waits for the cache's bytes, not for these products.
//
// Softmax, in units of log2: x = s * scale * log2(e); a running reference m
// that is only moved (and sums and outputs rescaled) when some x exceeds it
// by more than 8, so that p = 2^(x - m) stays below 2^8; sums in fp32.
//
// Work split: all units lie on a line by their weight (tiles + a fixed part)
// and each CTA (one per SM) takes an equal piece of it, found from the
// lengths by one scan at the kernel's start.  A unit cut by a border is
// shared: its CTAs write their parts (O unnormalised, m, l) to the workspace
// and the one that finishes last joins them in CTA order, so the result does
// not depend on which one that is.
#include "attn.cuh"

namespace flint {
namespace {

constexpr int kRowsWarps = 8;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr int kTileKeys = 16 * kRowsWarps;
constexpr int kUnitWeight = 2;  // a unit's fixed part, in tiles (2.3 us beside 1 us for a tile of 64 KB)
constexpr int kMinWeight = 1;   // least work of a CTA
constexpr int kChunkBytes = 16 * kHeadDim * 2 * 2;  // 16 keys' K and V
constexpr float kLazy = 8.0f;

struct Args {
  AttnArgs a;
  RowsWs w;
};

FLINT_DEV uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// {lo = bf16(a), hi = bf16(b)}
FLINT_DEV uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&r);
}

// One part of a unit: rows r0 .. of the group of kv head h, sequence b, key
// tiles [t0, t1).
struct Part {
  int b, h, r0, rows;
  int keys;             // of the sequence
  int t0, t1;
  int c_first, c_last;  // CTAs that share the unit
};

// A walk along the CTA's piece of the line.
template <int NT>
struct Walk {
  long long total, ctas, rem;
  long long at;  // position of the sequence's first unit
  int b, unit, off;
  int keys, tiles, units;  // of the sequence; units is the same for all

  FLINT_DEV void sequence(const AttnArgs& a) {
    keys = seq_keys(a, b);
    tiles = (keys + kTileKeys - 1) / kTileKeys;
  }
  FLINT_DEV bool next(const AttnArgs& a, Part& p) {
    while (rem > 0) {
      if (unit == units) {
        at += (long long)units * (tiles + kUnitWeight);
        ++b;
        unit = 0;
        sequence(a);
        continue;
      }
      const int w = tiles + kUnitWeight;
      const int take = (int)min((long long)(w - off), rem);
      const int real = max(1, tiles);
      const bool at_work = off < real;
      if (at_work) {
        const int G = a.nq / a.nkv;
        p.b = b;
        p.h = unit % a.nkv;
        p.r0 = unit / a.nkv * 8 * NT;
        p.rows = min(8 * NT, G - p.r0);
        p.keys = keys;
        p.t0 = min(off, tiles);
        p.t1 = min(off + take, tiles);
        p.c_first = p.c_last = blockIdx.x;
        if (off > 0 || take < real) {  // CTA of position x: floor(((x + 1) ctas - 1) / total)
          const long long u0 = at + (long long)unit * w;
          p.c_first = (int)(((u0 + 1) * ctas - 1) / total);
          p.c_last = (int)(((u0 + real) * ctas - 1) / total);
        }
      }
      rem -= take;
      off += take;
      if (off == w) {
        off = 0;
        ++unit;
      }
      if (at_work) return true;
    }
    return false;
  }
};

template <int NT>
struct Acc {
  float o[NT][8][4];  // tile j: {dim 8g+j, 64+8g+j} x rows 2t, 2t+1 of 8-row tile nt
  float m[NT][2], l[NT][2];
};

// Query head of row r of the part.
FLINT_DEV int head_of(const AttnArgs& a, const Part& u, int r) { return u.h * (a.nq / a.nkv) + u.r0 + r; }

// The warps' parts of 8 NT rows, joined in warp order.
template <int NT>
struct Parts {
  float o[kRowsWarps][8 * NT][kHeadDim];
  float m[kRowsWarps][8 * NT], l[kRowsWarps][8 * NT];
  int start[3];
  int last;
  long long pos[2];
  long long scan[kRowsWarps];
};
template <int NT>
constexpr int kDepth = NT == 1 ? 3 : 2;  // what shared memory holds beside Parts
template <int NT>
constexpr size_t kRing = (size_t)kDepth<NT> * kRowsWarps * kChunkBytes;
template <int NT>
constexpr size_t kSmem = kRing<NT> + sizeof(Parts<NT>);
template <int NT>
constexpr int kPartFloats = 8 * NT * (kHeadDim + 2);

template <int NT>
FLINT_DEV void store_part(Parts<NT>& P, const Acc<NT>& A) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      float l = A.l[nt][f];
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      const int r = 8 * nt + 2 * t + f;
      if (g == 0) {
        P.m[warp][r] = A.m[nt][f];
        P.l[warp][r] = l;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 4)
          *reinterpret_cast<float4*>(&P.o[warp][r][64 * i + 8 * g + j]) =
              make_float4(A.o[nt][j][2 * i + f], A.o[nt][j + 1][2 * i + f], A.o[nt][j + 2][2 * i + f],
                          A.o[nt][j + 3][2 * i + f]);
    }
}

// Weight of a part with reference pm and sum pl against the joint reference m.
FLINT_DEV float part_factor(float pm, float pl, float m) {
  return pm == neg_inf() ? (pl == 0.0f ? 0.0f : 1.0f) : ex2(pm - m);
}

// Four dims of a finished row: o / l in bf16 (zeros where no key had any
// weight), and its lse.
FLINT_DEV void write_row(const AttnArgs& a, const Part& u, int r, int d4, float4 o, float m, float l) {
  const long long row = (long long)u.b * a.nq + head_of(a, u, r);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint2 w;
  w.x = pack_bf16(o.x * inv, o.y * inv);
  w.y = pack_bf16(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(a.out + row * kHeadDim + 4 * d4) = w;
  if (a.lse && d4 == 0) a.lse[row] = l == 0.0f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
}

// This CTA's piece of the line: [pos, end) of total, and the unit it starts in.
template <int NT>
FLINT_DEV bool find_piece(const AttnArgs& a, Parts<NT>& P, Walk<NT>& k) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // two rounds over the sequences: the total, then the start (one round where
  // all sequences fit the CTA's threads)
  long long total = 0, pos = -1, end = 0;
  k.units = (a.nq / a.nkv + 8 * NT - 1) / (8 * NT) * a.nkv;
  for (int round = 0; round < 2; ++round) {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kRowsThreads) {
      const int b = b0 + tid;
      long long w = 0;
      int tiles = 0;
      if (b < a.B) {
        tiles = (seq_keys(a, b) + kTileKeys - 1) / kTileKeys;
        w = (long long)k.units * (tiles + kUnitWeight);
      }
      long long x = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();
      if (lane == 31) P.scan[warp] = x;
      __syncthreads();
      long long below = base;
#pragma unroll
      for (int i = 0; i < kRowsWarps; ++i) {
        if (i < warp) below += P.scan[i];
        base += P.scan[i];
      }
      const long long first = below + x - w;
      if (round == 0 && b0 + kRowsThreads >= a.B) {
        total = base;
        const long long ctas = total == 0 ? 0 : max(1ll, min((long long)gridDim.x, total / kMinWeight));
        k.total = total;
        k.ctas = ctas;
        if ((long long)blockIdx.x >= ctas) return false;
        pos = blockIdx.x * total / ctas;
        end = (blockIdx.x + 1) * total / ctas;
      }
      if (pos >= first && pos < first + w) {
        P.start[0] = b;
        P.start[1] = (int)((pos - first) / (tiles + kUnitWeight));
        P.start[2] = (int)((pos - first) % (tiles + kUnitWeight));
        P.pos[0] = first;
      }
    }
    if (a.B <= kRowsThreads) break;
  }
  __syncthreads();
  k.rem = end - pos;
  k.b = P.start[0];
  k.unit = P.start[1];
  k.off = P.start[2];
  k.at = P.pos[0];
  k.sequence(a);
  return true;
}

// GS: keys that lie at one stride (4 where pages have a multiple of 4 slots,
// else 1), so a look-up of the page table by all lanes serves 2 * GS chunks.
template <int NT, int GS>
__global__ void __launch_bounds__(kRowsThreads, 1) attn_rows_kernel(const __grid_constant__ Args args) {
  SpanGuard<kSpanAttnRows> span_guard;
  pdl_wait();  // q and the cache's newest rows are the previous kernel's output
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint8_t smem[];
  Parts<NT>& P = *reinterpret_cast<Parts<NT>*>(smem + kRing<NT>);
  const AttnArgs& a = args.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float c = a.scale * 1.4426950408889634f;

  Walk<NT> comp;
  if (!find_piece(a, P, comp)) return;

  // ---- the fetch side: a walk of its own, ahead of the products
  constexpr int kPer = 16 / GS, kChunks = 32 / kPer;  // look-ups per chunk, chunks per look-up
  Walk<NT> fwalk = comp;
  Part f = {};
  int ftile = 0, fpos = 0;    // next tile to fetch, its place in the look-up
  long long cur = -1, nxt = -1;  // element offsets of GS keys each, -1: none
  uint32_t cur_ok = 0;        // which of them are there
  bool fmore = true;
  auto chunk_key = [&](int tile) { return tile * kTileKeys + 16 * warp; };
  auto look_up = [&](int tile) {
    const int at = tile + lane / kPer, key = chunk_key(at) + lane % kPer * GS;
    return at < f.t1 && key < f.keys ? key_offset(a, f.b, key) : -1ll;
  };
  auto to_chunk = [&]() {  // on to this warp's next chunk, over the units
    if (ftile < f.t1 && chunk_key(ftile) < f.keys) {
      if (++fpos < kChunks) return;
      cur = nxt;
      nxt = look_up(ftile + kChunks);
    } else {
      do {
        fmore = fwalk.next(a, f);
        ftile = f.t0;
      } while (fmore && (ftile >= f.t1 || chunk_key(ftile) >= f.keys));
      if (!fmore) return;
      cur = look_up(ftile);
      nxt = look_up(ftile + kChunks);
    }
    fpos = 0;
    cur_ok = __ballot_sync(0xffffffffu, cur >= 0);
  };
  uint4* ring = reinterpret_cast<uint4*>(smem) + (size_t)warp * kDepth<NT> * (kChunkBytes / 16) + lane;
  auto fetch = [&](int slot) -> uint32_t {  // fills a slot; which of its GS-key groups are there
    uint32_t there = 0;
    if (fmore) {
      const uint32_t dst = smem_addr(ring + slot * (kChunkBytes / 16));
      const int left = f.keys - chunk_key(ftile), l0 = fpos * kPer;  // keys from the chunk's first on
      there = (cur_ok >> l0) & ((1u << kPer) - 1u);
      const uint16_t* kb = a.k + (long long)f.h * a.s_head + 8 * t;
      const uint16_t* vb = a.v + (long long)f.h * a.s_head + 8 * g;
      auto place = [&](int key, long long o) { return o + (GS > 1 ? (long long)(key % GS) * a.s_slot : 0ll); };
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = g + 8 * e;
        const long long o = __shfl_sync(0xffffffffu, cur, l0 + key / GS);
        const bool ok = o >= 0 && key < left;
        const uint16_t* src = kb + (ok ? place(key, o) : 0ll);
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16_or_zero(dst + 512 * (4 * e + i), src + 32 * i, ok);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = 2 * t + 8 * e;
        const long long o0 = __shfl_sync(0xffffffffu, cur, l0 + key / GS);
        const long long o1 = GS > 1 ? o0 : __shfl_sync(0xffffffffu, cur, l0 + key + 1);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const long long o = d ? o1 : o0;
          const bool ok = o >= 0 && key + d < left;
          const uint16_t* src = vb + (ok ? place(key + d, o) : 0ll);
#pragma unroll
          for (int i = 0; i < 2; ++i) cp_async16_or_zero(dst + 512 * (8 + 2 * (2 * e + d) + i), src + 64 * i, ok);
        }
      }
      ++ftile;
      to_chunk();
    }
    cp_async_commit();
    return there;
  };
  to_chunk();
  uint32_t there[kDepth<NT>];
#pragma unroll
  for (int i = 0; i < kDepth<NT>; ++i) there[i] = fetch(i);
  int slot = 0;

  Part u;
  while (comp.next(a, u)) {
    if (u.t0 >= u.t1) {  // a sequence without keys
      for (int i = threadIdx.x; i < u.rows * 32; i += kRowsThreads)
        write_row(a, u, i >> 5, i & 31, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f, 0.0f);
      continue;
    }
    // ---- Q of the unit's rows
    uint4 qf[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool ok = 8 * nt + g < u.rows;
      const uint16_t* p = a.q + (long long)u.b * a.q_stride + (long long)head_of(a, u, 8 * nt + g) * kHeadDim + 8 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[nt][i] = ok ? ldg_cg_v4(p + 32 * i) : make_uint4(0, 0, 0, 0);
    }
    Acc<NT> A;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) A.o[nt][j][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        A.m[nt][e] = neg_inf();
        A.l[nt][e] = 0.0f;
      }
    }
    for (int tile = u.t0; tile < u.t1 && chunk_key(tile) < u.keys; ++tile) {
      const int key0 = chunk_key(tile);
      cp_async_wait_group<kDepth<NT> - 1>();
      const uint4* src = ring + slot * (kChunkBytes / 16);
      const uint32_t ok = there[0];
      float s[NT][4];
      {
        uint4 kr[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) kr[e][i] = src[32 * (4 * e + i)];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_bf16_16816(s[nt], kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, qf[nt][i].x, qf[nt][i].y);
            mma_bf16_16816(s[nt], kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, qf[nt][i].z, qf[nt][i].w);
          }
        }
      }
      uint4 vr[4][2];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i) vr[e][i] = src[32 * (8 + 2 * e + i)];
      // s[nt][2 e + i]: key g + 8 e, row 2t + i
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = g + 8 * (i >> 1);
          if (!((ok >> (kk / GS)) & 1u) || key0 + kk >= u.keys) s[nt][i] = neg_inf();
          raise |= s[nt][i] * c > A.m[nt][i & 1] + kLazy;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[nt][e], s[nt][2 + e]) * c;
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            m = fmaxf(m, A.m[nt][e]);
            const float r = A.m[nt][e] == m ? 1.0f : ex2(A.m[nt][e] - m);
            A.m[nt][e] = m;
            A.l[nt][e] *= r;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              A.o[nt][j][e] *= r;
              A.o[nt][j][2 + e] *= r;
            }
          }
      }
      uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = A.m[nt][i & 1];
          p[i] = ex2(fmaf(s[nt][i], c, m == neg_inf() ? 0.0f : -m));
          A.l[nt][i & 1] += p[i];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t hi = pack_bf16(p[2 * e], p[2 * e + 1]);
          const uint32_t lo = pack_bf16(p[2 * e] - __uint_as_float(hi << 16),
                                        p[2 * e + 1] - __uint_as_float(hi & 0xffff0000u));
          bh[nt][e] = movmatrix(hi);
          bl[nt][e] = movmatrix(lo);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        uint32_t av[4];
#pragma unroll
        for (int e = 0; e < 2; ++e)    // keys 2t, 2t + 1 (+ 8 e)
#pragma unroll
          for (int i = 0; i < 2; ++i)  // dims 8g + j, 64 + 8g + j
            av[2 * e + i] = __byte_perm(reinterpret_cast<const uint32_t*>(&vr[2 * e][i])[j >> 1],
                                        reinterpret_cast<const uint32_t*>(&vr[2 * e + 1][i])[j >> 1], sel);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16_16816(A.o[nt][j], av[0], av[1], av[2], av[3], bh[nt][0], bh[nt][1]);
          mma_bf16_16816(A.o[nt][j], av[0], av[1], av[2], av[3], bl[nt][0], bl[nt][1]);
        }
      }
      // the slot's pieces are in registers: fill it again
#pragma unroll
      for (int i = 0; i + 1 < kDepth<NT>; ++i) there[i] = there[i + 1];
      there[kDepth<NT> - 1] = fetch(slot);
      slot = slot + 1 == kDepth<NT> ? 0 : slot + 1;
    }
    // ---- the unit's end in this CTA
    store_part<NT>(P, A);
    __syncthreads();
    const bool whole = u.c_first == u.c_last;
    float* part = args.w.parts + (size_t)(2 * blockIdx.x + ((int)blockIdx.x == u.c_first)) * kPartFloats<NT>;
    for (int i = threadIdx.x; i < u.rows * 32; i += kRowsThreads) {
      const int r = i >> 5, d4 = i & 31;
      float m = neg_inf();
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) m = fmaxf(m, P.m[w][r]);
      float l = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float x = part_factor(P.m[w][r], P.l[w][r], m);
        const float4 v = *reinterpret_cast<const float4*>(&P.o[w][r][4 * d4]);
        l += x * P.l[w][r];
        o.x += x * v.x;
        o.y += x * v.y;
        o.z += x * v.z;
        o.w += x * v.w;
      }
      if (whole) {
        write_row(a, u, r, d4, o, m, l);
      } else {
        *reinterpret_cast<float4*>(part + r * kHeadDim + 4 * d4) = o;
        if (d4 == 0) {
          part[8 * NT * kHeadDim + r] = m;
          part[8 * NT * (kHeadDim + 1) + r] = l;
        }
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();
        int* cnt = args.w.count + u.c_first;
        const int last = atomicAdd(cnt, 1) == u.c_last - u.c_first;
        if (last) *cnt = 0;
        P.last = last;
        __threadfence();
      }
      __syncthreads();
      if (P.last) {
        // a warp per row: the parts' references and sums one per lane, then
        // their outputs, several loads under way
        const int n = u.c_last - u.c_first + 1;
        auto part_at = [&](int i) {
          const int x = u.c_first + i;
          return args.w.parts + (size_t)(2 * x + (i == 0)) * kPartFloats<NT>;
        };
        for (int r = warp; r < u.rows; r += kRowsWarps) {
          float m = neg_inf();
          for (int i = lane; i < n; i += 32) m = fmaxf(m, __ldcg(part_at(i) + 8 * NT * kHeadDim + r));
#pragma unroll
          for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          float l = 0.0f;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int i0 = 0; i0 < n; i0 += 32) {
            float y = 0.0f, yl = 0.0f;
            if (i0 + lane < n) {
              const float pl = __ldcg(part_at(i0 + lane) + 8 * NT * (kHeadDim + 1) + r);
              y = part_factor(__ldcg(part_at(i0 + lane) + 8 * NT * kHeadDim + r), pl, m);
              yl = y * pl;
            }
            const int here = min(32, n - i0);
#pragma unroll 8
            for (int i = 0; i < here; ++i) {
              const float f = __shfl_sync(0xffffffffu, y, i);
              l += __shfl_sync(0xffffffffu, yl, i);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(part_at(i0 + i) + r * kHeadDim + 4 * lane));
              o.x += f * v.x;
              o.y += f * v.y;
              o.z += f * v.z;
              o.w += f * v.w;
            }
          }
          write_row(a, u, r, lane, o, m, l);
        }
      }
    }
    __syncthreads();  // Parts is free again
  }
  cp_async_wait_all();
}

template <int NT, int GS>
cudaError_t launch_nt(const AttnArgs& a, const RowsWs& w, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(attn_rows_kernel<NT, GS>);
  static std::atomic<bool> allowed[64];
  cudaError_t err = allow_smem(fn, (int)kSmem<NT>, allowed);
  if (err != cudaSuccess) return err;
  int sms = 0;
  err = device_sms(&sms);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms < kRowsCtas ? sms : kRowsCtas));
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = kSmem<NT>;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  Args p;
  p.a = a;
  p.w = w;
  void* args[] = {&p};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

RowsWs rows_ws(void* base) {
  static_assert(kAttnRowsCounters + kRowsCtas * sizeof(int) <= kAttnPromptCounters, "counters overlap");
  uint8_t* b = static_cast<uint8_t*>(base);
  RowsWs w;
  w.count = reinterpret_cast<int*>(b + kAttnRowsCounters);
  w.parts = reinterpret_cast<float*>(b + kAttnData);
  w.total = kAttnData + (size_t)2 * kRowsCtas * kPartFloats<2> * sizeof(float);
  return w;
}

cudaError_t launch_attn_rows(const AttnArgs& a, const RowsWs& w, cudaStream_t st) {
  // 8 rows per unit where a group fits them, else 16 (the keys are read once
  // per unit)
  const bool small = a.nq / a.nkv <= 8;
  if (a.block_size % 4 == 0) return small ? launch_nt<1, 4>(a, w, st) : launch_nt<2, 4>(a, w, st);
  return small ? launch_nt<1, 1>(a, w, st) : launch_nt<2, 1>(a, w, st);
}

FLINT_SPAN_SETTER(attn_rows)

}  // namespace flint
