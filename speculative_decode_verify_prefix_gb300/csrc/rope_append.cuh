// Rotary positions of queries and keys, alone or on the way of the keys and
// values into a cache: a pool of rows (rope_kernel) or blocks of e4m3 rows with
// a scale of their own (rope_block_kernel).
//
// A head's first R elements are R / 2 pairs; pair i of a row at position p turns
// by the angle p f_i:  (a, b) -> A (a cos - b sin, b cos + a sin).  Pairs are
// (i, i + R / 2), or (2 i, 2 i + 1) when interleaved.  Elements from R on stay.
//
// Angles.  A 32-bit product p f_i is off by more than a radian at far positions.
// The frequency in turns, f / 2 pi, is taken once per thread in 64 bits and
// written as a fraction of 2^64; p times it, in 64-bit integers, wraps at whole
// turns by itself, so the phase is exact but for the frequency's own 2^-53.  One
// table of (A cos, A sin) per CTA serves all heads of its tokens.
//
// All of it is bound by memory: a thread takes 16 elements of one head of one
// row, the two 16-byte loads whose pairs belong together.
#pragma once
#include "verify_kernel.cuh"

namespace vsk {
namespace rp {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;   // rope_kernel: tokens of a CTA
constexpr int kMaxBlock = 128;   // rows of a block at most
constexpr float kTop = 448.f;    // the largest e4m3 value
constexpr int kMinExp = -40, kMaxExp = 40;  // powers of two a block's scale takes

struct View {
  unsigned char* p;
  long long s0, s1;  // bytes
};

struct RopeParams {
  View q, k, v, qo, ko;  // qo, ko: where the rotated rows go (ko.p may be null)
  const void* pos;
  int pos64;
  const float* freq;
  float size;
  long long n;
  int h_q, h_kv, rot, inter;
  unsigned* err;
  // caches: rows [pool], their place (rope_kernel) or blocks (rope_block_kernel)
  View kc, vc;
  long long pool;
  const void* loc;
  int loc64;
  float k_scale, v_scale;
  int tokens, heads;  // rope_kernel: tokens and heads of a CTA
  // blocks
  float* ks;
  float* vs;
  long long ks_s0, vs_s0;
  const int* qo_ptr;
  const int* lens;
  const int* bt;
  long long bt_s0;
  int bt_cols, block, B;
  long long n_blocks;
};

using RopeFn = void (*)(const RopeParams);

// The frequency as a fraction of 2^64 turns per position.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  double t = static_cast<double>(f) * 0.15915494309189535;  // 1 / 2 pi
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}
// (A cos, A sin) of a position; a frequency that is no number gives none.
__device__ __forceinline__ float2 turn(unsigned long long f, long long pos, float size) {
  const long long phase = static_cast<long long>(f * static_cast<unsigned long long>(pos));
  const float half = __ll2float_rn(phase) * 1.0842021724855044e-19f;  // 2^-63: half turns in [-1, 1]
  float s, c;
  sincospif(half, &s, &c);
  return make_float2(size * c, size * s);
}
__device__ __forceinline__ long long index_at(const void* p, int wide, long long i) {
  return wide ? __ldg(static_cast<const long long*>(p) + i) : static_cast<long long>(__ldg(static_cast<const int*>(p) + i));
}

// Table of tokens [t0, t0 + n): entry (i, pair).
__device__ __forceinline__ void fill_table(const RopeParams& p, float2* cs, long long t0, int n) {
  const int pairs = p.rot >> 1;
  const int step = kThreads / pairs;  // tokens a pass (rot <= 256: at least two)
  const int pair = threadIdx.x % pairs, first = threadIdx.x / pairs;
  if (first < step && first < n) {
    const float f = __ldg(p.freq + pair);
    const unsigned long long turns = turns_of(f);
    const float size = isfinite(f) ? p.size : __int_as_float(0x7FC00000);
    for (int i = first; i < n; i += step) cs[i * pairs + pair] = turn(turns, index_at(p.pos, p.pos64, t0 + i), size);
  }
}

// 16 elements of a head: two runs of 8 at element offsets o1 and o2, and the
// table entries of their pairs (null: they stay).
struct Item {
  int o1, o2;
  const float2* cs;
};
__device__ __forceinline__ Item item_at(const RopeParams& p, const float2* row, int c) {
  Item it;
  const bool turned = 16 * c < p.rot;
  const bool split = turned && !p.inter;
  it.o1 = split ? 8 * c : 16 * c;
  it.o2 = split ? (p.rot >> 1) + 8 * c : 16 * c + 8;
  it.cs = turned ? row + 8 * c : nullptr;
  return it;
}
struct F16 {
  float a[8], b[8];
};
__device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
  const float2 f0 = unpack_bf16(w.x), f1 = unpack_bf16(w.y), f2 = unpack_bf16(w.z), f3 = unpack_bf16(w.w);
  x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y, x[4] = f2.x, x[5] = f2.y, x[6] = f3.x, x[7] = f3.y;
}
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void rotate(const RopeParams& p, const float2* cs, F16& x) {
  if (cs == nullptr) return;
  const float4* t4 = reinterpret_cast<const float4*>(cs);
  float2 t[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w = t4[i];
    t[2 * i] = make_float2(w.x, w.y);
    t[2 * i + 1] = make_float2(w.z, w.w);
  }
  if (p.inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x.a[2 * i], b = x.a[2 * i + 1], c = x.b[2 * i], d = x.b[2 * i + 1];
      x.a[2 * i] = a * t[i].x - b * t[i].y;
      x.a[2 * i + 1] = b * t[i].x + a * t[i].y;
      x.b[2 * i] = c * t[4 + i].x - d * t[4 + i].y;
      x.b[2 * i + 1] = d * t[4 + i].x + c * t[4 + i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x.a[i], b = x.b[i];
      x.a[i] = a * t[i].x - b * t[i].y;
      x.b[i] = b * t[i].x + a * t[i].y;
    }
  }
}

// Eight values under scale s as e4m3 codes: round to nearest even of x / s in 32
// bits, saturating.  A power of two divides exactly as its reciprocal multiplies.
__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x007FFFFFu) == 0u; }
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float inv, bool pow2) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = pow2 ? x[i] * inv : __fdiv_rn(x[i], s);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint4 ld16(const unsigned char* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(unsigned char* p, const uint4& w) { *reinterpret_cast<uint4*>(p) = w; }
__device__ __forceinline__ void st8(unsigned char* p, const uint2& w) { *reinterpret_cast<uint2*>(p) = w; }

}  // namespace rp

// Rows of q and k rotated; POOL 1 / 2: rotated k and v also stored to the rows
// `loc` of a bf16 / e4m3 pool.  A CTA takes p.tokens tokens of p.heads heads (of
// the h_q + h_kv, or h_q + 2 h_kv, of a row).
template <int D, int POOL>
__global__ void __launch_bounds__(rp::kThreads) rope_kernel(const __grid_constant__ rp::RopeParams p) {
  using namespace rp;
  constexpr int CH = D / 16;              // items of a head
  constexpr int SLOTS = kThreads / CH;    // heads in flight
  __shared__ __align__(16) float2 cs[kMaxTokens * 128];
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tokens), p.n - t0));
  const int total = p.h_q + (POOL ? 2 : 1) * p.h_kv;
  const int h0 = blockIdx.y * p.heads, nh = min(p.heads, total - h0);
  fill_table(p, cs, t0, nt);
  __syncthreads();
  const int c = threadIdx.x % CH;
  for (int r = threadIdx.x / CH; r < nt * nh; r += SLOTS) {
    const int i = r / nh, h = h0 + r % nh;
    const long long t = t0 + i;
    const Item it = item_at(p, cs + i * (p.rot >> 1), c);
    const int kind = h < p.h_q ? 0 : h < p.h_q + p.h_kv ? 1 : 2;  // q, k, v
    const int hh = kind == 0 ? h : kind == 1 ? h - p.h_q : h - p.h_q - p.h_kv;
    const View& in = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const unsigned char* src = in.p + t * in.s0 + hh * in.s1;
    F16 x;
    widen(ld16(src + 2 * it.o1), x.a);
    widen(ld16(src + 2 * it.o2), x.b);
    if (kind < 2) {
      rotate(p, it.cs, x);
      const View& out = kind == 0 ? p.qo : p.ko;
      if (out.p) {
        unsigned char* dst = out.p + t * out.s0 + hh * out.s1;
        st16(dst + 2 * it.o1, narrow(x.a));
        st16(dst + 2 * it.o2, narrow(x.b));
      }
    }
    if constexpr (POOL != 0) {
      if (kind > 0) {
        const long long row = index_at(p.loc, p.loc64, t);
        if (row >= 0 && row < p.pool) {
          const View& cache = kind == 1 ? p.kc : p.vc;
          const float s = kind == 1 ? p.k_scale : p.v_scale;
          unsigned char* dst = cache.p + row * cache.s0 + hh * cache.s1;
          const bool pow2 = is_pow2(s) && s > 1e-30f && s < 1e30f;
          const float inv = __frcp_rn(s);
          if constexpr (POOL == 2) {
            st8(dst + it.o1, codes8(x.a, s, inv, pow2));
            st8(dst + it.o2, codes8(x.b, s, inv, pow2));
          } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              x.a[u] = pow2 ? x.a[u] * inv : __fdiv_rn(x.a[u], s);
              x.b[u] = pow2 ? x.b[u] * inv : __fdiv_rn(x.b[u], s);
            }
            st16(dst + 2 * it.o1, narrow(x.a));
            st16(dst + 2 * it.o2, narrow(x.b));
          }
        } else if (row != -1 && hh == 0 && c == 0) {
          atomicOr(p.err, kErrBadIndex);
        }
      }
    }
  }
}

// The same into a cache of e4m3 blocks.  Unit u of the grid is a block that the
// call adds rows to (sequence after sequence); its CTAs (grid y) share its heads.
// A warp takes K or V of one head: the largest magnitude of the new rows gives
// the scale, a power of two, so that e4m3 loses nothing to it but at the lower
// end of its range; if the block holds earlier rows its scale never falls, and
// where it grows they are rounded again under the new one.
template <int D>
__global__ void __launch_bounds__(rp::kThreads) rope_block_kernel(const __grid_constant__ rp::RopeParams p) {
  using namespace rp;
  constexpr int CH = D / 16, RPI = 32 / CH;  // items of a head; rows of a warp's pass
  constexpr int NW = kThreads / 32;
  extern __shared__ __align__(16) float2 cs_dyn[];
  __shared__ long long scan[NW];
  __shared__ long long found_base;
  __shared__ int found_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // rows, and rows of the first block that are there already, of a sequence
  auto seq = [&](int b, int& row0, int& n, int& len, bool& held) -> int {  // its blocks
    const int a = __ldg(p.qo_ptr + b), e = __ldg(p.qo_ptr + b + 1);
    const bool ok = a >= 0 && e >= a && e <= p.n;
    row0 = ok ? a : 0;
    n = ok ? e - a : 0;
    len = __ldg(p.lens + b);
    held = len >= 0 && static_cast<long long>(len) + n <= static_cast<long long>(p.bt_cols) * p.block;
    if (blockIdx.x == 0 && blockIdx.y == 0 && (!ok || !held)) atomicOr(p.err, !ok ? kErrBadQoIndptr : kErrBadKvIndptr);
    if (!held) len = 0;
    return n == 0 ? 0 : static_cast<int>((static_cast<long long>(len % p.block) + n - 1) / p.block) + 1;
  };
  if (tid == 0) found_b = -1;
  int row0, n, len;
  bool held;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
  long long mine = 0;
  for (int b = lo; b < hi; ++b) mine += seq(b, row0, n, len, held);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long at = incl - mine;
  for (int w = 0; w < warp; ++w) at += scan[w];
  const long long unit = blockIdx.x;
  if (unit >= at && unit < at + mine) {
    for (int b = lo; b < hi; ++b) {
      const int k = seq(b, row0, n, len, held);
      if (unit < at + k) {
        found_b = b;
        found_base = unit - at;
        break;
      }
      at += k;
    }
  }
  __syncthreads();
  if (found_b < 0) return;  // uniform: fewer blocks than the host allowed for
  const int b = found_b;
  seq(b, row0, n, len, held);
  // block `found_base` of the sequence's new ones: rows [off, off + nt) of it
  const long long head = found_base * p.block - len % p.block;  // new rows before the block (negative: none)
  const int off = head < 0 ? static_cast<int>(-head) : 0;
  const long long done = head < 0 ? 0 : head;
  const int nt = static_cast<int>(min(static_cast<long long>(p.block - off), n - done));
  const long long t0 = row0 + done;
  long long page = -1;
  if (held) {
    const long long col = len / p.block + found_base;
    page = __ldg(p.bt + b * p.bt_s0 + col);
    if (page < 0 || page >= p.n_blocks) {
      page = -1;
      if (tid == 0 && blockIdx.y == 0) atomicOr(p.err, kErrBadIndex);
    }
  }
  fill_table(p, cs_dyn, t0, nt);
  __syncthreads();
  const int pairs = p.rot >> 1;
  const int c = lane % CH, sub = lane / CH;
  // ---- keys and values: a warp per (head, K or V) ----
  for (int task = blockIdx.y * NW + warp; task < 2 * p.h_kv; task += NW * gridDim.y) {
    const int h = task >> 1;
    const bool isv = task & 1;
    const View& in = isv ? p.v : p.k;
    const View& cache = isv ? p.vc : p.kc;
    const unsigned char* src = in.p + t0 * in.s0 + h * in.s1;
    auto load = [&](int i, Item& it, F16& x) {
      it = item_at(p, cs_dyn + i * pairs, c);
      const unsigned char* r = src + i * in.s0;
      widen(ld16(r + 2 * it.o1), x.a);
      widen(ld16(r + 2 * it.o2), x.b);
      if (!isv) rotate(p, it.cs, x);
    };
    float s = 1.f, old = 1.f;
    if (page >= 0) {
      float top = 0.f;  // of the finite values
      for (int i = sub; i < nt; i += RPI) {
        Item it;
        F16 x;
        load(i, it, x);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float a = fabsf(x.a[u]), d = fabsf(x.b[u]);
          top = fmaxf(top, a < INFINITY ? a : 0.f);
          top = fmaxf(top, d < INFINITY ? d : 0.f);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // the smallest 2^e with top <= 448 2^e = 1.75 2^(8 + e)
      const unsigned bits = __float_as_uint(top);
      int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
      e = max(kMinExp, min(kMaxExp, e));
      const float need = __int_as_float((127 + e) << 23);
      float* sp = (isv ? p.vs + page * p.vs_s0 : p.ks + page * p.ks_s0) + h;
      if (off > 0) {
        old = *sp;
        s = fmaxf(old, need);
      } else {
        s = need;
      }
      if (off > 0 && s != old) {
        const float by = __fdiv_rn(old, s);
        for (int i = sub; i < off; i += RPI) {
          unsigned char* r = cache.p + (page * p.block + i) * cache.s0 + h * cache.s1 + 16 * c;
          const uint4 w = ld16(r);
          const uint32_t in4[4] = {w.x, w.y, w.z, w.w};
          uint32_t out4[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t y = 0;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t h2 = e4m3x2_to_f16x2(static_cast<unsigned short>(in4[u] >> (16 * z)));
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
              y |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f.x * by, f.y * by), __NV_SATFINITE, __NV_E4M3))
                   << (16 * z);
            }
            out4[u] = y;
          }
          st16(r, make_uint4(out4[0], out4[1], out4[2], out4[3]));
        }
      }
      __syncwarp();  // every lane has read the old scale
      if (lane == 0) *sp = s;
    }
    if (page < 0 && (isv || p.ko.p == nullptr)) continue;
    const bool pow2 = is_pow2(s);
    const float inv = __frcp_rn(s);
    for (int i = sub; i < nt; i += RPI) {
      Item it;
      F16 x;
      load(i, it, x);
      if (!isv && p.ko.p) {
        unsigned char* dst = p.ko.p + (t0 + i) * p.ko.s0 + h * p.ko.s1;
        st16(dst + 2 * it.o1, narrow(x.a));
        st16(dst + 2 * it.o2, narrow(x.b));
      }
      if (page >= 0) {
        unsigned char* dst = cache.p + (page * p.block + off + i) * cache.s0 + h * cache.s1;
        st8(dst + it.o1, codes8(x.a, s, inv, pow2));
        st8(dst + it.o2, codes8(x.b, s, inv, pow2));
      }
    }
  }
  // ---- queries ----
  const int slots = kThreads / CH * gridDim.y;
  for (int r = (blockIdx.y * kThreads + tid) / CH; r < nt * p.h_q; r += slots) {
    const int i = r / p.h_q, h = r % p.h_q;
    const Item it = item_at(p, cs_dyn + i * pairs, tid % CH);
    const unsigned char* src = p.q.p + (t0 + i) * p.q.s0 + h * p.q.s1;
    F16 x;
    widen(ld16(src + 2 * it.o1), x.a);
    widen(ld16(src + 2 * it.o2), x.b);
    rotate(p, it.cs, x);
    unsigned char* dst = p.qo.p + (t0 + i) * p.qo.s0 + h * p.qo.s1;
    st16(dst + 2 * it.o1, narrow(x.a));
    st16(dst + 2 * it.o2, narrow(x.b));
  }
}

rp::RopeFn kernel_rope(int D, int pool);   // pool 0 none, 1 bf16, 2 e4m3
rp::RopeFn kernel_rope_block(int D);

}  // namespace vsk
