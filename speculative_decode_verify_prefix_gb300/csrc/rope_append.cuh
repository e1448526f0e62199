// Rotary positions of queries and keys, alone or on the way of the keys and
// values into a cache: a pool of rows (rope_kernel) or blocks of e4m3 rows with
// a scale of their own (rope_block_kernel).
//
// A head's first R elements are R / 2 pairs; pair i of a row at position p turns
// by the angle p f_i:  (a, b) -> A (a cos - b sin, b cos + a sin).  Pairs are
// (i, i + R / 2), or (2 i, 2 i + 1) when interleaved.  Elements from R on stay.
//
// Angles.  A 32-bit product p f_i is off by more than a radian at far positions.
// The frequency in turns, f / 2 pi, is a fraction of 2^64 here; p times it, in 64-bit
// integers, wraps at whole turns by itself, so the phase is off by p 2^-64 of a turn
// and what a 64-bit 2^64 / 2 pi leaves, p f 2^-62.  One table of (A cos, A sin) per CTA
// serves all heads of its tokens.
//
// All of it but the blocks' keys and values is bound by memory: a thread takes 16
// elements of one head of one row, the two 16-byte loads whose pairs belong together.
// 21,716 rows of 32/8 heads of 128 take 70 us rotated (445 MB, 6.3 TB/s), a plain copy of
// as many bytes 68.5 (6.5); with K and V stored to a pool 93 (579 MB, 6.2).
#pragma once
#include "verify_kernel.cuh"

namespace vsk {
namespace rp {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;    // rope_kernel: tokens of a CTA
constexpr int kMaxBlock = 128;   // rows of a block at most
constexpr int kBlockThreads = 256;  // rope_block_kernel
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
  int warps;  // of a (block, head, K or V): a power of two
  int units, parts;  // blocks at most, CTAs of one
  int turn;          // CTAs from one of keys and values to the next
  long long n_blocks;
};

using RopeFn = void (*)(const RopeParams);

// The frequency as a fraction of 2^64 turns per position: f = m 2^-s times 2^64 / 2 pi.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  constexpr unsigned long long C = 0x28BE60DB9391054Aull;  // 2^64 / 2 pi
  const unsigned bits = __float_as_uint(f);
  const int e = static_cast<int>(bits >> 23 & 255u), s = 150 - max(e, 1);
  const unsigned long long m = (bits & 0x007FFFFFu) | (e ? 0x00800000u : 0u);
  const unsigned long long lo = m * C, hi = __umul64hi(m, C);  // hi < 2^24
  unsigned long long x;
  if (s >= 64)
    x = s < 128 ? hi >> (s - 64) : 0ull;
  else if (s > 0)
    x = hi << (64 - s) | lo >> s;
  else
    x = s > -64 ? lo << -s : 0ull;
  return bits >> 31 ? 0ull - x : x;
}
// (A cos, A sin) of a position; a frequency that is no number gives none.  The upper
// 32 bits of the phase, less the nearest quarter turn, leave an angle r of at most
// pi / 4; Taylor's series to r^9 and r^8 end within 3e-8.
__device__ __forceinline__ float2 turn(unsigned long long f, long long pos, float size) {
  const unsigned phase = static_cast<unsigned>(f * static_cast<unsigned long long>(pos) >> 32);
  const unsigned q = (phase + 0x20000000u) >> 30;
  const float r = static_cast<float>(static_cast<int>(phase - (q << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = r * r;
  float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f), c = fmaf(z, 1.f / 40320.f, -1.f / 720.f);
  s = fmaf(s, z, 1.f / 120.f);
  c = fmaf(c, z, 1.f / 24.f);
  s = fmaf(s, z, -1.f / 6.f);
  c = fmaf(c, z, -0.5f);
  s = fmaf(s * z, r, r);
  c = fmaf(c, z, 1.f);
  const float a = q & 1 ? s : c, b = q & 1 ? c : s;  // a quarter turn: (cos, sin) -> (-sin, cos)
  const float as = __uint_as_float(__float_as_uint(size) ^ ((q + 1u) << 30 & 0x80000000u));
  const float bs = __uint_as_float(__float_as_uint(size) ^ (q << 30 & 0x80000000u));
  return make_float2(as * a, bs * b);
}
__device__ __forceinline__ long long index_at(const void* p, int wide, long long i) {
  return wide ? __ldg(static_cast<const long long*>(p) + i) : static_cast<long long>(__ldg(static_cast<const int*>(p) + i));
}

// Table of tokens [t0, t0 + n).  A thread reads the eight entries of pairs 8 c ..
// 8 c + 7 in four pieces of two: piece k of all c lies together, so that the lanes
// of a head read side by side (with a thread's entries together four lanes meet in a
// bank: 21,716 rows, 32/8 heads of 128, 86 us, so 76).
template <int NT>
__device__ __forceinline__ void fill_table(const RopeParams& p, float2* cs, long long t0, int n) {
  const int pairs = p.rot >> 1;
  const int step = NT / pairs;  // tokens a pass (rot <= 256: at least two)
  const int pair = threadIdx.x % pairs, first = threadIdx.x / pairs;
  if (first < step && first < n) {
    const float f = __ldg(p.freq + pair);
    const int at = ((pair & 7) >> 1) * (pairs >> 2) + (pair >> 3) * 2 + (pair & 1);
    const unsigned long long turns = turns_of(f);
    const float size = isfinite(f) ? p.size : __int_as_float(0x7FC00000);
    for (int i = first; i < n; i += step) cs[i * pairs + at] = turn(turns, index_at(p.pos, p.pos64, t0 + i), size);
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
  it.cs = turned ? row + 2 * c : nullptr;
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
  float2 t[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w = *reinterpret_cast<const float4*>(cs + i * (p.rot >> 3));
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

// Values under scale s: the 32-bit quotients x / s.  A power of two divides exactly
// as its reciprocal multiplies (one branch for all of them, not 16 divisions beside
// 16 products).
struct Under {
  float s, inv;
  bool exact;
  __device__ __forceinline__ explicit Under(float scale) : s(scale), inv(1.f / scale) {
    exact = (__float_as_uint(s) & 0x007FFFFFu) == 0u && s > 1e-30f && s < 1e30f;
  }
  __device__ __forceinline__ void operator()(F16& x) const {
    if (exact) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x.a[i] *= inv;
        x.b[i] *= inv;
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {  // (rotating through the first place: one copy of the division)
        const float a = __fdiv_rn(x.a[0], s), b = __fdiv_rn(x.b[0], s);
#pragma unroll
        for (int k = 0; k < 7; ++k) {
          x.a[k] = x.a[k + 1];
          x.b[k] = x.b[k + 1];
        }
        x.a[7] = a;
        x.b[7] = b;
      }
    }
  }
};
// Eight values as e4m3 codes: to nearest even, saturating.
__device__ __forceinline__ uint2 codes8(const float (&y)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

// Four codes under a scale `by` times larger.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float by) {
  uint32_t y = 0;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const uint32_t h2 = e4m3x2_to_f16x2(static_cast<unsigned short>(w >> (16 * z)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    y |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f.x * by, f.y * by), __NV_SATFINITE, __NV_E4M3)) << (16 * z);
  }
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint4 ld16(const unsigned char* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(unsigned char* p, const uint4& w) { *reinterpret_cast<uint4*>(p) = w; }
__device__ __forceinline__ void st8(unsigned char* p, const uint2& w) { *reinterpret_cast<uint2*>(p) = w; }

}  // namespace rp

// Heads [h0, h0 + nh) of rows [t0, t0 + nt): q and k rotated; POOL 1 / 2: rotated k
// and v also stored to the rows `loc` of a bf16 / e4m3 pool.  Rows whose bit of
// `mask` is not set are left alone.  A thread's next item is on its way while it works
// on one, the first while `table` fills the table (which ends with a barrier and gives
// the mask).
template <int D, int POOL, int NT, bool Q_ONLY, typename Table>
__device__ __forceinline__ void rotate_rows(const rp::RopeParams& p, const float2* cs, long long t0, int nt, int h0, int nh,
                                            Table table) {
  using namespace rp;
  constexpr int CH = D / 16;        // items of a head
  constexpr int SLOTS = NT / CH;    // heads in flight
  const int c = threadIdx.x % CH;
  const Item it = item_at(p, cs, c);
  const int gap = it.o2 - it.o1;
  // (row, head) of an item; SLOTS items on, without dividing again
  struct At {
    int i, h;
  };
  const int di = SLOTS / nh, dh = SLOTS % nh;
  auto on = [&](At& a) {
    a.i += di;
    a.h += dh;
    if (a.h >= nh) {
      a.h -= nh;
      ++a.i;
    }
  };
  struct Row {
    At a;
    uint4 w1, w2;
  } next = {};
  auto kind_of = [&](int h) { return Q_ONLY || h < p.h_q ? 0 : h < p.h_q + p.h_kv ? 1 : 2; };  // q, k, v
  auto head_of = [&](int h, int kind) { return kind == 0 ? h : kind == 1 ? h - p.h_q : h - p.h_q - p.h_kv; };
  auto place = [&](const View& v, int i, int hh) { return v.p + (t0 + i) * v.s0 + hh * v.s1; };
  auto fetch = [&] {
    const int h = h0 + next.a.h, kind = kind_of(h);
    const unsigned char* src = place(kind == 0 ? p.q : kind == 1 ? p.k : p.v, next.a.i, head_of(h, kind)) + 2 * it.o1;
    next.w1 = ld16(src);
    next.w2 = ld16(src + 2 * gap);
  };
  next.a.i = static_cast<int>(threadIdx.x) / CH / nh;
  next.a.h = static_cast<int>(threadIdx.x) / CH % nh;
  if (next.a.i < nt) fetch();
  const unsigned mask = table();
  while (next.a.i < nt) {
    const Row now = next;
    on(next.a);
    if (next.a.i < nt) fetch();
    const int i = now.a.i;
    if ((mask >> i & 1u) == 0u) continue;
    const int h = h0 + now.a.h, kind = kind_of(h), hh = head_of(h, kind);
    F16 x;
    widen(now.w1, x.a);
    widen(now.w2, x.b);
    if (kind < 2) {
      if (it.cs) rotate(p, it.cs + i * (p.rot >> 1), x);
      const View& out = kind == 0 ? p.qo : p.ko;
      if (out.p) {
        unsigned char* dst = place(out, i, hh) + 2 * it.o1;
        st16(dst, narrow(x.a));
        st16(dst + 2 * gap, narrow(x.b));
      }
    }
    if constexpr (POOL != 0) {
      if (kind > 0) {
        const long long row = index_at(p.loc, p.loc64, t0 + i);
        if (row >= 0 && row < p.pool) {
          const View& cache = kind == 1 ? p.kc : p.vc;
          unsigned char* dst = cache.p + row * cache.s0 + hh * cache.s1;
          Under(kind == 1 ? p.k_scale : p.v_scale)(x);
          if constexpr (POOL == 2) {
            st8(dst + it.o1, codes8(x.a));
            st8(dst + it.o2, codes8(x.b));
          } else {
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

// A CTA takes p.tokens tokens of p.heads heads (of the h_q + h_kv, or h_q + 2 h_kv,
// of a row).  Without a pool five CTAs fit an SM (21,716 rows, 32/8 heads of 128: four
// 73.3 us, five 70.8, six 72.6); with one the fifth costs spills (94, so 96).
template <int D, int POOL>
__global__ void __launch_bounds__(rp::kThreads, POOL == 0 ? 5 : 4) rope_kernel(const __grid_constant__ rp::RopeParams p) {
  using namespace rp;
  __shared__ __align__(16) float2 cs[kMaxTokens * 128];
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tokens), p.n - t0));
  const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.h_q + (POOL ? 2 : 1) * p.h_kv - h0);
  rotate_rows<D, POOL, kThreads, false>(p, cs, t0, nt, h0, nh, [&] {
    fill_table<kThreads>(p, cs, t0, nt);
    __syncthreads();
    return ~0u;
  });
}

// The same into a cache of e4m3 blocks.  p.units * p.parts of the CTAs take keys
// and values: unit u is a block that the call adds rows to (sequence after sequence),
// whose heads p.parts CTAs share.  p.warps warps take K or V of one head, a thread
// 16 elements of a row, which it rotates and holds: the largest magnitude of the new
// rows gives the scale, a power of two, so that e4m3 loses nothing to it but at the
// lower end of its range; if the block holds earlier rows its scale never falls, and
// where it grows they are rounded again under the new one.  Of a block's parts some have
// keys alone, some values alone: those need no table of angles.
// The other CTAs take the queries as rope_kernel does: they are most of the bytes, and
// need none of this.
// 21,716 rows, 32/8 heads of 128, blocks of 64: 103 us, 5.2 TB/s, of which keys and
// values alone 60 at 3.0: instructions and latency (without loads and stores 41, of
// which 10 to find the blocks and 14 for the tables).
template <int D>
__global__ void __launch_bounds__(rp::kBlockThreads, 4) rope_block_kernel(const __grid_constant__ rp::RopeParams p) {
  using namespace rp;
  constexpr int CH = D / 16, RPI = 32 / CH;  // items of a head; rows of a warp's pass
  constexpr int NT = kBlockThreads, NW = NT / 32;
  __shared__ unsigned tops[2][NW];
  extern __shared__ __align__(16) float2 cs_dyn[];
  __shared__ int scan[NW];
  __shared__ int found[6];  // sequence (-1: none), its block, rows: seq's answers
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // every p.turn-th CTA is one of keys and values, as long as there are any: the two
  // kinds run side by side, latency beside bandwidth
  const int group_of = static_cast<int>(blockIdx.x) / p.turn, kv_ctas = p.units * p.parts;
  const int kv = group_of * p.turn == static_cast<int>(blockIdx.x) && group_of < kv_ctas ? group_of : -1;
  if (kv < 0) {
    // ---- queries ----
    const int x = static_cast<int>(blockIdx.x) - min(group_of + 1, kv_ctas), per_tile = (p.h_q + p.heads - 1) / p.heads;
    const long long t0 = static_cast<long long>(x / per_tile) * p.tokens;
    const int nt = static_cast<int>(min(static_cast<long long>(p.tokens), p.n - t0));
    const int h0 = x % per_tile * p.heads;
    if (tid == 0) tops[0][0] = 0u;
    __syncthreads();
    rotate_rows<D, 0, NT, true>(p, cs_dyn, t0, nt, h0, min(p.heads, p.h_q - h0), [&] {
      // rows that belong to a sequence
      for (int b = tid; b < p.B; b += NT) {
        const int a = __ldg(p.qo_ptr + b), e = __ldg(p.qo_ptr + b + 1);
        if (a < 0 || e < a || e > p.n) continue;
        const int from = static_cast<int>(max(a - t0, 0LL)), to = static_cast<int>(min(e - t0, static_cast<long long>(nt)));
        if (from < to) atomicOr(&tops[0][0], ((1u << (to - from)) - 1u) << from);
      }
      fill_table<NT>(p, cs_dyn, t0, nt);
      __syncthreads();
      return tops[0][0];
    });
    return;
  }
  const int unit = kv / p.parts, member = kv % p.parts;
  // rows, and rows of the first block that are there already, of a sequence
  auto seq = [&](int b, int& row0, int& n, int& len, bool& held) -> int {  // its blocks
    const int a = __ldg(p.qo_ptr + b), e = __ldg(p.qo_ptr + b + 1);
    const bool ok = a >= 0 && e >= a && e <= p.n;
    row0 = ok ? a : 0;
    n = ok ? e - a : 0;
    len = __ldg(p.lens + b);
    held = len >= 0 && static_cast<long long>(len) + n <= static_cast<long long>(p.bt_cols) * p.block;
    if (kv == 0 && (!ok || !held)) atomicOr(p.err, !ok ? kErrBadQoIndptr : kErrBadKvIndptr);
    if (!held) len = 0;
    return n == 0 ? 0 : (len % p.block + n - 1) / p.block + 1;
  };
  if (tid == 0) found[0] = -1;
  int row0, n, len;
  bool held;
  const int per = (p.B + NT - 1) / NT;
  const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
  int mine = 0;
  for (int b = lo; b < hi; ++b) mine += seq(b, row0, n, len, held);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int at0 = incl - mine;
  for (int w = 0; w < warp; ++w) at0 += scan[w];
  if (unit >= at0 && unit < at0 + mine) {
    for (int b = lo; b < hi; ++b) {
      const int k = per > 1 ? seq(b, row0, n, len, held) : mine;
      if (unit < at0 + k) {
        found[0] = b;
        found[1] = unit - at0;
        found[2] = row0;
        found[3] = n;
        found[4] = len;
        found[5] = held;
        break;
      }
      at0 += k;
    }
  }
  __syncthreads();
  const int b = found[0], found_base = found[1];
  if (b < 0) return;  // uniform: fewer blocks than the host allowed for
  row0 = found[2];
  n = found[3];
  len = found[4];
  held = found[5] != 0;
  // block `found_base` of the sequence's new ones: rows [off, off + nt) of it
  const long long head = static_cast<long long>(found_base) * p.block - len % p.block;  // new rows before it (negative: none)
  const int off = head < 0 ? static_cast<int>(-head) : 0;
  const int done = head < 0 ? 0 : static_cast<int>(head);
  const int nt = min(p.block - off, n - done);
  const long long t0 = row0 + done;
  const int found_page = held ? __ldg(p.bt + b * p.bt_s0 + len / p.block + found_base) : -1;  // asked for, not waited for
  const int pairs = p.rot >> 1;
  const int c = lane % CH;
  const Item it = item_at(p, cs_dyn, c);
  const int wt = p.warps, groups = NW / wt, group = warp / wt, part = warp % wt;
  // this thread's row of the new ones, and again `chunk` rows on (more rows than the
  // warps hold are read twice)
  const int first = part * RPI + lane / CH, chunk = wt * RPI;
  const int last = (nt - 1) / chunk * chunk;
  // tasks: K of every head, then V of every head; this CTA's [.., tasks), its groups by turns
  const int each = (2 * p.h_kv + p.parts - 1) / p.parts, tasks = min(2 * p.h_kv, (member + 1) * each);
  int task = member * each + group;
  uint4 n1, n2;  // the next task's row
  float next_old = 0.f;
  auto fetch = [&](int which, int at, uint4& a, uint4& b2) {
    const View& in = which >= p.h_kv ? p.v : p.k;
    a = b2 = make_uint4(0u, 0u, 0u, 0u);
    if (at + first < nt) {
      const unsigned char* src = in.p + (t0 + at + first) * in.s0 + (which >= p.h_kv ? which - p.h_kv : which) * in.s1;
      a = ld16(src + 2 * it.o1);
      b2 = ld16(src + 2 * it.o2);
    }
  };
  auto scale_of = [&](long long page, int which) -> float* {
    return which >= p.h_kv ? p.vs + page * p.vs_s0 + (which - p.h_kv) : p.ks + page * p.ks_s0 + which;
  };
  if (task < tasks) fetch(task, 0, n1, n2);
  if (member * each < p.h_kv) fill_table<NT>(p, cs_dyn, t0, nt);  // (V alone needs none) while the first loads are on their way
  const long long page = found_page >= 0 && found_page < p.n_blocks ? found_page : -1;
  if (held && page < 0 && tid == 0 && member == 0) atomicOr(p.err, kErrBadIndex);
  const bool grows = page >= 0 && off > 0;
  if (grows && task < tasks) next_old = *scale_of(page, task);
  __syncthreads();
  int turn_of = 0;
  for (; task < tasks; task += groups, turn_of ^= 1) {
    const bool isv = task >= p.h_kv;
    const int h = isv ? task - p.h_kv : task;
    const float old = next_old;
    F16 x;
    auto take = [&](int at, const uint4& a, const uint4& b2) {
      widen(a, x.a);
      widen(b2, x.b);
      if (!isv && it.cs && at + first < nt) rotate(p, it.cs + (at + first) * pairs, x);
    };
    take(0, n1, n2);
    if (task + groups < tasks) {  // while this one is worked on
      fetch(task + groups, 0, n1, n2);
      if (grows) next_old = *scale_of(page, task + groups);
    }
    float s = 1.f;
    if (page >= 0) {
      unsigned most = 0;  // bits of the largest finite magnitude
      for (int at = 0;;) {
        float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e & 3] = max3(m[e & 3], fabsf(x.a[e]), fabsf(x.b[e]));
        unsigned top = __float_as_uint(max3(max3(m[0], m[1], m[2]), m[3], 0.f));
        if (top >= 0x7F800000u) {  // rare: infinities and NaN do not count
          top = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const unsigned a = __float_as_uint(x.a[e]) & 0x7FFFFFFFu, d = __float_as_uint(x.b[e]) & 0x7FFFFFFFu;
            top = max(top, max(a < 0x7F800000u ? a : 0u, d < 0x7F800000u ? d : 0u));
          }
        }
        most = max(most, top);
        if (at == last) break;
        at += chunk;
        uint4 a, b2;
        fetch(task, at, a, b2);
        take(at, a, b2);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (wt > 1) {
        if (lane == 0) tops[turn_of][warp] = most;
        named_bar_sync(1 + group, 32 * wt);  // (everyone has read the old scale, too)
        most = __reduce_max_sync(0xffffffffu, tops[turn_of][group * wt + (lane & (wt - 1))]);
      }
      // the smallest 2^e with the maximum <= 448 2^e = 1.75 2^(8 + e)
      int e = static_cast<int>(most >> 23) - 127 - 8 + ((most & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
      e = max(kMinExp, min(kMaxExp, e));
      s = __int_as_float((127 + e) << 23);
      if (off > 0) {
        s = fmaxf(old, s);
        if (s != old) {
          const View& cache = isv ? p.vc : p.kc;
          const float by = __fdiv_rn(old, s);
          for (int i = first; i < off; i += chunk) {
            unsigned char* r = cache.p + (page * p.block + i) * cache.s0 + h * cache.s1 + 16 * c;
            const uint4 w = ld16(r);
            st16(r, make_uint4(rescaled(w.x, by), rescaled(w.y, by), rescaled(w.z, by), rescaled(w.w, by)));
          }
        }
      }
      __syncwarp();  // every lane has read the old scale
      if (part == 0 && lane == 0) *scale_of(page, task) = s;
    }
    const Under under(s);
    // (with a block the last rows are in hand, without one the first)
    for (int at = page >= 0 ? last : 0;;) {
      const int i = at + first;
      if (i < nt) {
        if (!isv && p.ko.p) {
          unsigned char* dst = p.ko.p + (t0 + i) * p.ko.s0 + h * p.ko.s1;
          st16(dst + 2 * it.o1, narrow(x.a));
          st16(dst + 2 * it.o2, narrow(x.b));
        }
        if (page >= 0) {
          const View& cache = isv ? p.vc : p.kc;
          unsigned char* dst = cache.p + (page * p.block + off + i) * cache.s0 + h * cache.s1;
          under(x);
          st8(dst + it.o1, codes8(x.a));
          st8(dst + it.o2, codes8(x.b));
        }
      }
      at = page >= 0 ? at - chunk : at + chunk;
      if (at < 0 || at >= nt) break;
      uint4 a, b2;
      fetch(task, at, a, b2);
      take(at, a, b2);
    }
  }
}

rp::RopeFn kernel_rope(int D, int pool);   // pool 0 none, 1 bf16, 2 e4m3
rp::RopeFn kernel_rope_block(int D);

}  // namespace vsk
