// verify_splitkv_mass: the attention weight that every prefix key receives
// from a verify call's draft rows.
//
//   mass[h][kv0 + j] = mass_in[h][kv0 + j] + sum over the rows r of KV head h
//                      of 2^(x_rj - lse_r),   x_rj = q_r . k_j sm_scale k_scale log2 e
//   lse_r = log2 of the sum of 2^x over the row's prefix keys and its drafts t <= i
//
// A key's weight needs its row's lse, which needs every key: two passes over
// the scores, of which only the first should read K.  One thread-block cluster
// owns one (sequence, KV head); each of its CTAs takes a slice of the keys,
// computes their scores once and keeps them in shared memory (32-bit, R x 4
// bytes a key), then the CTAs exchange their rows' maxima and sums through
// distributed shared memory and turn the kept scores into weights.  K is read
// once as long as a slice's scores fit (1,536 keys a CTA at 16 rows
// of head_dim 128, 320 at 64 rows, 96 at 128); of a longer slice all but the last
// chunk is loaded and computed again.
//
// Bound by the K stream.  Each warp loads 8-key groups straight into the
// registers of the mma.sync B operand: lane (g, j) of the fragment needs key
// g's elements at four positions of every 16-wide k step, and which positions
// those are is free as long as the queries use the same ones, so the lane
// takes 16 consecutive bytes (4 lanes: 64 bytes of a row) and no shuffle,
// ldmatrix or staging buffer is needed.  The next stage's loads are in flight
// while one is multiplied (deeper queues cost registers: the serving batch
// 1354 us with three stages, 1213 with two; a ring filled by cp.async 1211
// against 1072).  e4m3 keys are widened to f16 (exact) and meet queries scaled
// by a power of two so that the largest finite one lies in [2^14, 2^15)
// (elements more than 2^29 smaller than it lose bits).
//
// Measured: 64 sequences of 8,192 to 32,768 keys, 32/8 heads of 128, 4 drafts,
// bf16: 1,064 us, 2.7 TB/s of keys over the call (a fifth of them, in the 43
// sequences longer than their 12 CTAs' scores, is loaded twice) and about 4 while
// keys load; nothing loads while a CTA sweeps its scores, exchanges and weighs.
// With 64 packed rows 16 sequences of 8,192 keys take 530 us, with 128 1,520:
// short chunks, most keys loaded twice.
//
// The sum over a head's rows runs in row order and every key has one writer:
// the result does not depend on scheduling.
#pragma once
#include <cooperative_groups.h>

#include "verify_kernel.cuh"

namespace vsk {
namespace km {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 128;
constexpr int kSmem = 110 * 1024;  // two CTAs per SM
constexpr unsigned kNoRow = 0xFFFFFFFFu;

struct MassParams {
  Params v;                 // the flat call: q, ke, kb, qo, kvp, kvi, scales
  const float* in; long long in_s0;
  float* out;      long long out_s0;
  int h_kv, MT, cap, pitch;  // keys of a chunk (a multiple of 32), floats between score rows
  int x_off, i_off, s_off;   // shared memory: the CTAs' row sums, pool rows, scores (queries at 0)
};
using MassFn = void (*)(const MassParams);

// 8-key groups of a stage, 16-byte loads of a lane per key row, stages in flight.
// A stage takes 16 registers a lane (32 at 512-byte rows); DEPTH - 1 of them are
// loading while one is multiplied.
template <int D, bool FP8>
struct Geo {
  static constexpr int ROWB = D * (FP8 ? 1 : 2);
  static constexpr int NL = ROWB / 64;                      // loads per key row
  static constexpr int NB = NL >= 4 ? 1 : 4 / NL;           // groups per stage
  static constexpr int KEYS = 8 * NB;
  static constexpr int DEPTH = 2;
  static constexpr int KS = D / 16;                         // k steps
  static constexpr int QCH = D / 8;                         // 16-byte chunks of a query row in shared memory
};

// 16 bytes of a key row; the lanes of a row take its 64-byte pieces one after
// the other, so L2 is asked for all of it (ROWB bytes or 256) at the first, and
// L1 keeps what the first brought (bypassing it measured 30 % slower)
template <int ROWB>
__device__ __forceinline__ uint4 ld_row(const void* a) {
  uint4 v;
  if constexpr (ROWB >= 256)
    asm volatile("ld.global.nc.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(a));
  else
    asm volatile("ld.global.nc.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(a));
  return v;
}

}  // namespace km

// QREG: one 16-row tile whose query fragments stay in registers (head_dim <= 128)
template <int D, bool FP8, bool QREG>
__global__ void __launch_bounds__(km::kThreads, 2) mass_kernel(const __grid_constant__ km::MassParams mp) {
  using namespace km;
  using G = km::Geo<D, FP8>;
  namespace cg = cooperative_groups;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float row_m[kMaxRows], row_l[kMaxRows], row_lse[kMaxRows];
  __shared__ unsigned q_max;
  const Params& p = mp.v;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j4 = lane & 3;
  const long long seg = blockIdx.x / C;
  const int b = static_cast<int>(seg / mp.h_kv), h = static_cast<int>(seg % mp.h_kv);
  const float NEG_INF = -INFINITY;

  int P;
  long long kv0;
  const bool seq_ok = seq_info(p, b, P, kv0);
  const int qa = __ldg(p.qo + b), qe = __ldg(p.qo + b + 1);
  const bool q_ok = qa >= 0 && qe - qa == p.L && static_cast<long long>(qa) + p.L <= p.n_rows;
  if (rank == 0 && h == 0 && tid == 0) {
    if (!seq_ok) atomicOr(p.err, kErrBadKvIndptr);
    if (!q_ok) atomicOr(p.err, kErrBadQoIndptr);
  }
  if (P == 0) return;  // the whole cluster: no key, nothing to write
  cluster.barrier_arrive();  // completes once every CTA runs: its shared memory may then be written
  const long long s_b = q_ok ? qa : static_cast<long long>(b) * p.L;
  const int per = (P + C * 32 - 1) / (C * 32) * 32;
  const int lo = static_cast<int>(min(static_cast<long long>(P), static_cast<long long>(rank) * per));
  const int hi = min(P, lo + per);

  // ---- queries into shared memory, 16-byte chunk c of row r at chunk c ^ (r & 7) ----
  unsigned char* qs = smem;
  float* sc = reinterpret_cast<float*>(smem + mp.s_off);
  if (tid == 0) q_max = 0u;
  __syncthreads();
  const int rows_pad = 16 * mp.MT;
  {
    unsigned mx = 0;
    for (int i = tid; i < rows_pad * G::QCH; i += kThreads) {
      const int r = i / G::QCH, c = i % G::QCH;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (r < p.R) {
        const __nv_bfloat16* src =
            p.q + (s_b + r / p.gq) * p.q_s0 + static_cast<long long>(h * p.gq + r % p.gq) * p.q_s1 + c * 8;
        x = make_uint4(ld_u32(src), ld_u32(src + 2), ld_u32(src + 4), ld_u32(src + 6));
      }
      if constexpr (FP8) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) mx = max(mx, finite_mag_bf16x2(w[u]));
      }
      *reinterpret_cast<uint4*>(qs + r * (D * 2) + ((c ^ (r & 7)) << 4)) = x;
    }
    if constexpr (FP8) {
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) atomicMax(&q_max, mx);
    }
  }
  for (int r = tid; r < kMaxRows; r += kThreads) {
    row_m[r] = NEG_INF;
    row_l[r] = 0.f;
  }
  __syncthreads();

  // ---- rank 0: the drafts' part of every row's sum (t <= i) ----
  if (rank == 0) {
    constexpr int DE = D / 8;
    const int part = lane & 7, tt = lane >> 3;
    for (int r = warp; r < p.R; r += kWarps) {
      const int i = r / p.gq;
      float m = NEG_INF, l = 0.f;
      for (int t0 = 0; t0 <= i; t0 += 4) {
        const int t = t0 + tt;
        float x = 0.f;
        if (t <= i) {
          const __nv_bfloat16* kr = p.ke + (s_b + t) * p.ke_s0 + static_cast<long long>(h) * p.ke_s1 + part * DE;
#pragma unroll
          for (int u = 0; u < DE / 2; ++u) {
            const int d = part * DE + 2 * u;
            const float2 kv = unpack_bf16(ld_u32(kr + 2 * u));
            const float2 qv = unpack_bf16(*reinterpret_cast<const uint32_t*>(
                qs + r * (D * 2) + (((d >> 3) ^ (r & 7)) << 4) + (d & 7) * 2));
            x = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, x));
          }
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x = t <= i ? x * p.dscale2 : NEG_INF;
        float mx = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mn = fmaxf(m, mx), ms = mn == NEG_INF ? 0.f : mn;
        float e = exp2f(x - ms);
        e += __shfl_xor_sync(0xffffffffu, e, 8);
        e += __shfl_xor_sync(0xffffffffu, e, 16);
        l = l * exp2f(m - ms) + e;
        m = mn;
      }
      if (lane == 0) {
        row_m[r] = m;
        row_l[r] = l;
      }
    }
  }

  // ---- e4m3 keys: the queries as scaled f16 ----
  float scale2 = p.scale2;
  if constexpr (FP8) {
    __syncthreads();  // the draft part read the bf16 queries
    const unsigned mx = q_max;
    int sh = mx == 0u ? 0 : 14 - (static_cast<int>(mx >> 7) - 127);  // the largest |q| 2^sh lies in [2^14, 2^15)
    sh = max(-120, min(120, sh));
    const float up = __int_as_float((127 + sh) << 23);
    scale2 *= __int_as_float((127 - sh) << 23);
    for (int i = tid; i < rows_pad * (D / 2); i += kThreads) {
      uint32_t* w = reinterpret_cast<uint32_t*>(qs) + i;
      const float2 f = unpack_bf16(*w);
      *w = pack_f16(f.x * up, f.y * up);
    }
    __syncthreads();
  }

  // Elements of lane j4 in load i of a key row: bytes 64 i + 16 j4 .. + 15, so
  // bf16: k steps 2 i and 2 i + 1 take elements 32 i + 8 j4 + {0, 1 | 2, 3} and + {4, 5 | 6, 7};
  // e4m3: k steps 4 i .. 4 i + 3 take elements 64 i + 16 j4 + 4 s + {0, 1 | 2, 3}.
  auto q_frag = [&](int mt, int ks, uint32_t (&a)[4]) {
    int d;
    if constexpr (FP8)
      d = 64 * (ks >> 2) + 16 * j4 + 4 * (ks & 3);
    else
      d = 32 * (ks >> 1) + 8 * j4 + 4 * (ks & 1);
    const int r = 16 * mt + g;  // rows g and g + 8 have the same r & 7
    const unsigned char* q0 = qs + r * (D * 2) + (((d >> 3) ^ (r & 7)) << 4) + (d & 7) * 2;
    const uint2 x = *reinterpret_cast<const uint2*>(q0);
    const uint2 y = *reinterpret_cast<const uint2*>(q0 + 8 * D * 2);
    a[0] = x.x;
    a[1] = y.x;
    a[2] = x.y;
    a[3] = y.y;
  };
  uint32_t qf[QREG ? G::KS : 1][4];
  if constexpr (QREG) {
#pragma unroll
    for (int ks = 0; ks < G::KS; ++ks) q_frag(0, ks, qf[ks]);
  }

  const unsigned char* kbase = p.kb + static_cast<long long>(h) * p.kb_s1;
  struct Stage {
    uint4 k[G::NB][G::NL];
    unsigned ok;  // bit n: key g of group n is in the chunk and its index in the pool
  };
  unsigned* idx = reinterpret_cast<unsigned*>(smem + mp.i_off);  // pool rows of the chunk's keys, kNoRow: none
  // (a key without a row loads row 0, and its scores become -inf: a load under a
  // condition would be waited for where the two cases meet)
  auto load_k = [&](int at, Stage& s) {
    s.ok = 0u;
#pragma unroll
    for (int n = 0; n < G::NB; ++n) {
      const unsigned loc = idx[at + 8 * n + g];
      const bool ok = loc != kNoRow;
      s.ok |= ok ? 1u << n : 0u;
      const unsigned char* src = kbase + static_cast<long long>(ok ? loc : 0u) * p.kb_s0 + 16 * j4;
#pragma unroll
      for (int i = 0; i < G::NL; ++i) s.k[n][i] = ld_row<G::ROWB>(src + 64 * i);
    }
  };
  // scores of one stage into sc[row][key of the chunk]
  auto multiply = [&](const Stage& s, int at0) {
#pragma unroll 1
    for (int mt = 0; mt < (QREG ? 1 : mp.MT); ++mt) {
      // (two chains of products where the stage is one group)
      constexpr int NC = G::NB == 1 ? 2 : 1;
      float acc[G::NB * NC][4];
#pragma unroll
      for (int n = 0; n < G::NB * NC; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < G::KS; ++ks) {
        uint32_t a[4];
        if constexpr (QREG) {
#pragma unroll
          for (int u = 0; u < 4; ++u) a[u] = qf[ks][u];
        } else {
          q_frag(mt, ks, a);
        }
#pragma unroll
        for (int n = 0; n < G::NB; ++n) {
          if constexpr (FP8) {
            const uint4& w = s.k[n][ks >> 2];
            const uint32_t x = (ks & 3) == 0 ? w.x : (ks & 3) == 1 ? w.y : (ks & 3) == 2 ? w.z : w.w;
            mma_f16(acc[n * NC + ks % NC], a, e4m3x2_to_f16x2(static_cast<unsigned short>(x & 0xFFFFu)),
                    e4m3x2_to_f16x2(static_cast<unsigned short>(x >> 16)));
          } else {
            const uint4& w = s.k[n][ks >> 1];
            mma_bf16(acc[n * NC + ks % NC], a, (ks & 1) ? w.z : w.x, (ks & 1) ? w.w : w.y);
          }
        }
      }
      if constexpr (NC == 2) {
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[0][u] += acc[1][u];
      }
#pragma unroll
      for (int n = 0; n < G::NB; ++n) {
        // columns 2 j4 and 2 j4 + 1 of the group: their keys' validity sits in lanes 8 j4 and 8 j4 + 4
        const bool v0 = (__shfl_sync(0xffffffffu, s.ok, 8 * j4) >> n) & 1u;
        const bool v1 = (__shfl_sync(0xffffffffu, s.ok, 8 * j4 + 4) >> n) & 1u;
        const int at = at0 + 8 * n + 2 * j4;
        const int r = 16 * mt + g;
        if (r < p.R)
          *reinterpret_cast<float2*>(sc + r * mp.pitch + at) =
              make_float2(v0 ? acc[n][0] * scale2 : NEG_INF, v1 ? acc[n][1] * scale2 : NEG_INF);
        if (r + 8 < p.R)
          *reinterpret_cast<float2*>(sc + (r + 8) * mp.pitch + at) =
              make_float2(v0 ? acc[n][2] * scale2 : NEG_INF, v1 ? acc[n][3] * scale2 : NEG_INF);
      }
    }
  };
  // scores of the chunk of n keys at c0: stages dealt to the warps in turn
  auto chunk = [&](int c0, int n) {
    constexpr int STEP = kWarps * G::KEYS;
    const int end = (n + G::KEYS - 1) / G::KEYS * G::KEYS;
    for (int i = tid; i < end; i += kThreads) {
      unsigned row = kNoRow;
      if (i < n) {
        const long long at = kv0 + c0 + i;
        const long long loc = p.idx64 ? __ldg(static_cast<const long long*>(p.kvi) + at)
                                      : static_cast<long long>(__ldg(static_cast<const int*>(p.kvi) + at));
        if (loc >= 0 && loc < p.pool)
          row = static_cast<unsigned>(loc);
        else
          atomicOr(p.err, kErrBadIndex);
      }
      idx[i] = row;
    }
    __syncthreads();
    int at = warp * G::KEYS;
    if (at < end) {
      Stage s[G::DEPTH];
#pragma unroll
      for (int u = 0; u < G::DEPTH - 1; ++u)
        if (at + u * STEP < end) load_k(at + u * STEP, s[u]);
#pragma unroll 1
      while (at < end) {
#pragma unroll
        for (int u = 0; u < G::DEPTH; ++u) {
          if (at < end) {
            if (at + (G::DEPTH - 1) * STEP < end) load_k(at + (G::DEPTH - 1) * STEP, s[(u + G::DEPTH - 1) % G::DEPTH]);
            multiply(s[u], at);
            at += STEP;
          }
        }
      }
    }
    __syncthreads();
  };
  // chunks of cap keys behind a first one of the rest, so that the scores kept
  // at the end are as many as fit
  const int n_chunks = (hi - lo + mp.cap - 1) / mp.cap;
  const int rest = hi - lo - (n_chunks - 1) * mp.cap;
  auto chunk_at = [&](int k) { return k == 0 ? lo : lo + rest + (k - 1) * mp.cap; };
  auto chunk_keys = [&](int k) { return k == 0 ? rest : mp.cap; };
  for (int k = 0; k < n_chunks; ++k) {
    const int n = chunk_keys(k);
    chunk(chunk_at(k), n);
    for (int r = warp; r < p.R; r += kWarps) {
      // keys past n, up to a multiple of 4, hold -inf
      const float4* x = reinterpret_cast<const float4*>(sc + r * mp.pitch);
      float m = NEG_INF, l = 0.f;
#pragma unroll 2
      for (int i = lane; 4 * i < n; i += 32) {
        const float4 v = x[i];
        const float mn = fmaxf(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)), m), ms = mn == NEG_INF ? 0.f : mn;
        l = l * fast_exp2(m - ms) + ((fast_exp2(v.x - ms) + fast_exp2(v.y - ms)) + (fast_exp2(v.z - ms) + fast_exp2(v.w - ms)));
        m = mn;
      }
      const float old = row_m[r];
      float mn = fmaxf(m, old);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      const float ms = mn == NEG_INF ? 0.f : mn;
      l *= fast_exp2(m - ms);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      __syncwarp();
      if (lane == 0) {
        row_l[r] = row_l[r] * fast_exp2(old - ms) + l;
        row_m[r] = mn;
      }
    }
    __syncthreads();  // the scores are done with
  }

  // ---- the rows' sums over the whole cluster: every CTA hands its own to all ----
  __syncthreads();
  cluster.barrier_wait();
  float2* xch = reinterpret_cast<float2*>(smem + mp.x_off);  // [C][R] (m, l)
  for (int i = tid; i < C * p.R; i += kThreads) {
    const int c = i / p.R, r = i % p.R;
    *cluster.map_shared_rank(xch + rank * p.R + r, c) = make_float2(row_m[r], row_l[r]);
  }
  cluster.sync();
  for (int r = tid; r < p.R; r += kThreads) {
    float m = NEG_INF, l = 0.f;
    for (int c = 0; c < C; ++c) m = fmaxf(m, xch[c * p.R + r].x);
    const float ms = m == NEG_INF ? 0.f : m;
    for (int c = 0; c < C; ++c) l += xch[c * p.R + r].y * exp2f(xch[c * p.R + r].x - ms);
    row_lse[r] = l == 0.f ? INFINITY : ms + log2f(l);  // a row with nothing visible gives no weight
  }
  __syncthreads();

  // ---- weights: the last chunk from the kept scores, the others computed again ----
  const float* in = mp.in ? mp.in + h * mp.in_s0 + kv0 : nullptr;
  float* out = mp.out + h * mp.out_s0 + kv0;
  for (int k = n_chunks - 1; k >= 0; --k) {
    const int c0 = chunk_at(k), n = chunk_keys(k);
    if (k < n_chunks - 1) {
      __syncthreads();
      chunk(c0, n);
    }
    for (int i = tid; i < n; i += kThreads) {
      float w = 0.f;
#pragma unroll 8
      for (int r = 0; r < p.R; ++r) w += fast_exp2(sc[r * mp.pitch + i] - row_lse[r]);
      out[c0 + i] = (in ? in[c0 + i] : 0.f) + w;
    }
  }
}

km::MassFn kernel_mass(int D, bool fp8, bool qreg);

}  // namespace vsk
