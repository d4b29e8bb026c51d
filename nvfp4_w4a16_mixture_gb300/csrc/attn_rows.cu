// Attention of few query rows over the paged cache (flint_attn_decode, and
// flint_attn_prompt until its rows fill tensor-core tiles).
//
// The rows of one sequence and kv head are its tokens' query heads packed
// together: packed row r is token r / G, head r % G of the group (G query
// heads per kv head), so one pass over the keys serves the whole group.  A
// CTA takes 8 NT packed rows of one (sequence, kv head) and all the keys they
// see; its 8 warps take 16 keys each in turn.
//
// Per 16 keys a warp forms S^T = K Q^T and O^T += V^T P on mma.sync
// m16n8k16 with the keys (then the head's dims) as the 16-row operand and 8
// packed rows as the 8 columns, so a group of 8 heads wastes nothing.  Keys
// and values go from global memory straight into operand registers:
//  - K: lane (g, t) = (lane / 4, lane % 4) loads dims 32 i + 8 t .. + 7 of
//    keys g and g + 8; its four words are the operands of two k-steps (Q is
//    loaded with the same permutation of the dims, and a sum does not depend
//    on their order);
//  - V: lane (g, t) loads dims 8 g .. + 7 and 64 + 8 g .. + 7 of keys 2t,
//    2t + 1, 2t + 8, 2t + 9; a byte permutation pairs two keys' values of one
//    dim, and dim 8 g + j (64 + 8 g + j) is row g (g + 8) of tile j.
// P's accumulator layout (row = key) becomes the operand layout (row = packed
// row) by movmatrix.  P enters as hi + lo, two bf16 values (relative error
// 2^-18): a single bf16 would double the output's squared rounding error, and
// the kernel waits for the cache's bytes, not for these products.
//
// Softmax, in units of log2: x = s * scale * log2(e); a running reference m
// that is only moved (and sums and outputs rescaled) when some x exceeds it
// by more than 8, so that p = 2^(x - m) stays below 2^8; sums in fp32.
#include "attn.cuh"

namespace flint {
namespace {

constexpr int kRowsWarps = 8;
constexpr float kLazy = 8.0f;

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

// Packed rows of one unit: rows r0 .. of sequence b's q rows, kv head h.
struct Unit {
  int b, h, r0;
  int rows;  // valid packed rows of the unit (at most 8 NT)
  int lo;    // first q row of the sequence
  int n;     // its q rows
  int keys;  // its keys
};

template <int NT>
struct Acc {
  float o[NT][8][4];  // tile j: {dim 8g+j, 64+8g+j} x packed rows 2t, 2t+1 of 8-row tile nt
  float m[NT][2], l[NT][2];
};

// Token row (of q) and query head of packed row r.
FLINT_DEV void row_of(const AttnArgs& a, const Unit& u, int r, int& token, int& head) {
  const int G = a.nq / a.nkv, R = u.r0 + r;
  token = R / G;
  head = u.h * G + R % G;
}

// Keys [k0, k1) of the unit into acc, 16 at a time: chunk i of this warp is
// keys k0 + 16 (warp + kRowsWarps * i) ..
template <int NT>
FLINT_DEV void attend(const AttnArgs& a, const Unit& u, int k0, int k1, Acc<NT>& A) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float c = a.scale * 1.4426950408889634f;
  uint4 qf[NT][4];
  int lim[NT][2];  // last key that packed rows 2t, 2t + 1 see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    int token, head;
    row_of(a, u, 8 * nt + g, token, head);
    const bool ok = 8 * nt + g < u.rows;
    const uint16_t* p = a.q + (long long)(u.lo + token) * a.q_stride + (long long)head * kHeadDim + 8 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) qf[nt][i] = ok ? ldg_cg_v4(p + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      row_of(a, u, 8 * nt + 2 * t + e, token, head);
      lim[nt][e] = u.keys - u.n + token;
    }
  }
  const uint16_t* kb = a.k + (long long)u.h * a.s_head;
  const uint16_t* vb = a.v + (long long)u.h * a.s_head;
  auto offset = [&](int key) { return key < k1 ? key_offset(a, u.b, key) : -1ll; };
  int key0 = k0 + 16 * warp;
  long long off = offset(key0 + (lane & 15));
  long long off_next = offset(key0 + 16 * kRowsWarps + (lane & 15));
  uint4 kr[2][4], vr[4][2];
  bool kok[2], kok_next[2];
  auto load_k = [&](long long o, bool (&ok)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long ko = __shfl_sync(0xffffffffu, o, g + 8 * e);
      ok[e] = ko >= 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) kr[e][i] = ok[e] ? ldg_cg_v4(kb + ko + 32 * i + 8 * t) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_v = [&](long long o) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long vo = __shfl_sync(0xffffffffu, o, 2 * t + (e & 1) + 8 * (e >> 1));
#pragma unroll
      for (int i = 0; i < 2; ++i) vr[e][i] = vo >= 0 ? ldg_cg_v4(vb + vo + 64 * i + 8 * g) : make_uint4(0, 0, 0, 0);
    }
  };
  if (key0 >= k1) return;
  load_k(off, kok);
  load_v(off);
  while (key0 < k1) {
    const bool more = key0 + 16 * kRowsWarps < k1;
    float s[NT][4];
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
    kok_next[0] = kok_next[1] = false;
    if (more) load_k(off_next, kok_next);
    // s[nt][2 e + f]: key g + 8 e, packed row 2t + f
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + g + 8 * (i >> 1);
        if (!kok[i >> 1] || key > lim[nt][i & 1]) s[nt][i] = neg_inf();
        raise |= s[nt][i] * c > A.m[nt][i & 1] + kLazy;
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float m = fmaxf(s[nt][f], s[nt][2 + f]) * c;
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          m = fmaxf(m, A.m[nt][f]);
          const float r = A.m[nt][f] == m ? 1.0f : ex2(A.m[nt][f] - m);
          A.m[nt][f] = m;
          A.l[nt][f] *= r;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            A.o[nt][j][f] *= r;
            A.o[nt][j][2 + f] *= r;
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
    if (more) load_v(off_next);
    kok[0] = kok_next[0];
    kok[1] = kok_next[1];
    key0 += 16 * kRowsWarps;
    off_next = offset(key0 + 16 * kRowsWarps + (lane & 15));
  }
}

// The warps' parts of 8 NT rows, joined in warp order.
template <int NT>
struct Parts {
  float o[kRowsWarps][8 * NT][kHeadDim];
  float m[kRowsWarps][8 * NT], l[kRowsWarps][8 * NT];
};

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

// Four dims of a finished row: o / l in bf16 (zeros where no key had any
// weight), and its lse.
FLINT_DEV void write_row(const AttnArgs& a, const Unit& u, int r, int d4, float4 o, float m, float l) {
  int token, head;
  row_of(a, u, r, token, head);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint2 w;
  w.x = pack_bf16(o.x * inv, o.y * inv);
  w.y = pack_bf16(o.z * inv, o.w * inv);
  const long long row = u.lo + token;
  *reinterpret_cast<uint2*>(a.out + (row * a.nq + head) * kHeadDim + 4 * d4) = w;
  if (a.lse && d4 == 0) a.lse[row * a.nq + head] = l == 0.0f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
}

template <int NT>
__global__ void __launch_bounds__(kRowsWarps * 32) attn_rows_kernel(const AttnArgs a) {
  SpanGuard<kSpanAttnRows> span_guard;
  pdl_wait();  // q and the cache's newest rows are the previous kernel's output
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint8_t smem[];
  Parts<NT>& P = *reinterpret_cast<Parts<NT>*>(smem);
  const int G = a.nq / a.nkv;
  // sequence and row tile of this CTA
  Unit u;
  u.h = blockIdx.y;
  int tile = blockIdx.x;
  for (u.b = 0; u.b < a.B; ++u.b) {
    seq_rows(a, u.b, u.lo, u.n);
    const long long tiles = ((long long)u.n * G + 8 * NT - 1) / (8 * NT);
    if (tile < tiles) break;
    tile -= (int)tiles;
  }
  if (u.b >= a.B) return;
  u.r0 = tile * 8 * NT;
  u.rows = min(8 * NT, u.n * G - u.r0);
  u.keys = seq_keys(a, u.b);
  const int last = u.keys - u.n + (u.r0 + u.rows - 1) / G;  // last key of the last row
  Acc<NT> A;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) A.o[nt][j][e] = 0.0f;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      A.m[nt][f] = neg_inf();
      A.l[nt][f] = 0.0f;
    }
  }
  attend<NT>(a, u, 0, min(u.keys, last + 1), A);
  store_part<NT>(P, A);
  __syncthreads();
  for (int i = threadIdx.x; i < u.rows * 32; i += kRowsWarps * 32) {
    const int r = i >> 5, d4 = i & 31;
    float m = neg_inf();
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) m = fmaxf(m, P.m[w][r]);
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) {
      const float f = P.m[w][r] == neg_inf() ? (P.l[w][r] == 0.0f ? 0.0f : 1.0f) : ex2(P.m[w][r] - m);
      const float4 v = *reinterpret_cast<const float4*>(&P.o[w][r][4 * d4]);
      l += f * P.l[w][r];
      o.x += f * v.x;
      o.y += f * v.y;
      o.z += f * v.z;
      o.w += f * v.w;
    }
    write_row(a, u, r, d4, o, m, l);
  }
}

template <int NT>
cudaError_t launch_nt(const AttnArgs& a, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(attn_rows_kernel<NT>);
  cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Parts<NT>));
  if (err != cudaSuccess) return err;
  const long long G = a.nq / a.nkv;
  // tiles of all sequences: at most one ragged tile each
  const long long tiles = a.cu_q ? (long long)a.T * G / (8 * NT) + a.B : a.B * ((G + 8 * NT - 1) / (8 * NT));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)a.nkv);
  cfg.blockDim = dim3(kRowsWarps * 32);
  cfg.dynamicSmemBytes = sizeof(Parts<NT>);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  AttnArgs aa = a;
  void* args[] = {&aa};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t st) {
  // 8 packed rows per CTA where a token's group fits them, else 16 (the keys
  // are read once per CTA)
  const bool small = !a.cu_q && a.nq / a.nkv <= 8;
  return small ? launch_nt<1>(a, st) : launch_nt<2>(a, st);
}

FLINT_SPAN_SETTER(attn_rows)

}  // namespace flint
