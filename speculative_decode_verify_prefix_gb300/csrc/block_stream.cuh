// Prefix stream of the verify call over an e4m3 cache whose blocks (pages) have
// a scale of their own for each KV head, one for K and one for V.
//
//   t_rj = s log2e ks_j <q_r, K_j> + log2 vs_j,  x_rj = 2^(t_rj - m_r),
//   l_r  = sum_j x_rj / vs_j,                     o_r  = sum_j x_rj V_j / l_r
// (K_j, V_j the stored codes' values, ks_j, vs_j the scales of key j's block):
// the running reference m_r is taken over the weights as V meets them, so that
// blocks of very different scales share one accumulator, and the row's sum
// takes the scale out again.
//
// Both products run on tcgen05 straight from the cache's bytes (kind::f8f6f4);
// nothing is widened.  What is not e4m3 is written as a sum of e4m3 terms:
//   queries  q 2^sh = hi + lo (bf16 has 8 significant bits, a term 4): exact, but that
//            elements more than 2^10 below the row's largest are off by up to 2^-17 of
//            that; along K of one accumulator, or 16 lanes apart;
//   weights  y = 2^6 x: the top 4 bits, the next 4 and the rest rounded to 4, as
//            three groups of rows of one M = 128 product under scales 1, 2^4,
//            2^8: 12 bits, and 2^-24 of the reference at the lower end.
// A tile is 128 keys of one KV head:
//   S[128][128 keys] = Q[128] x K^T   (all packed rows several times over: every
//                      warp finds them in its own lanes)
//   O[128][D]       += P[128][128 keys] x V    (rows 32 p + r: term p of row r)
//
// Roles (7 warps; two CTAs an SM at head_dim 64 and 128, one at 256):
//   warps 0-3  softmax: warp w the keys 32 w .. 32 w + 31 of all rows.
//   warps 4, 6 block table, TMA of boxes of up to 128 keys into the K and V rings, scales.
//   warp 5     tensor memory, MMAs.
// Up to eight KV heads are taken by a team of as many CTAs, each its own over the
// same keys: what lies side by side in memory is read at about the same time (8
// heads of 128, 64 sequences: 488 us with heads apart, 428 so; 32 single tokens 100,
// 91).  More than 32 packed rows are row tiles, a CTA each beside the others: the keys
// come from memory once (64 rows: 139 us with the tiles one after the other, 115 so).
// The tiles of all (sequence, head group) segments are laid end to end and every team
// takes an equal share; a segment's part of a share is a piece, whose partial (o, log2
// of its sum) block_combine_kernel folds: of CTA c and segment s, slot c + team * s.
// What bounds it: 64 sequences of 8,259 to 32,600 keys (8 heads of 128, 16 rows) take
// 420-428 us, 6.6-6.7 TB/s, memory; at head_dim 64 a tile's softmax outlasts its bytes
// (189 us for 829 MB), with 32 rows the chain of scores, softmax and weights (313 us for
// 1.66 GB).
// Every wait is bounded (one second); a CTA that gives up sets error bit 8.  Its loaders
// end their loops, the other roles go through their tiles without waiting, multiplying
// or arriving anywhere (the copies' barriers then still tell when those under way are
// done; what such a CTA writes to its partials is no result), then it waits for copies
// and MMAs in flight, frees the tensor memory and exits.  No barrier can run two phases
// ahead of a wait for it: each phase needs an arrival that follows the wait for the
// one before.
#pragma once
#include <type_traits>

#include "flash_tc.cuh"

namespace vsk {

enum : unsigned { kErrBadScale = 64u };

namespace bk {

constexpr int KT = 128;      // keys of a tile
constexpr int GK = 16;       // keys of a group (of one block, so under one scale; a TMA box takes 1, 2, 4 or 8)
constexpr int GT = KT / GK;  // groups of a tile
constexpr int kThreads = 224;
constexpr int kSm = 128;     // softmax threads
constexpr int kMeta = 8;     // tiles whose scales are kept (more than the ring holds)
constexpr float kThr = 2.f;  // log2 headroom before a reference is raised
constexpr int kUp = 6;       // y = 2^kUp x <= 2^(kUp + kThr) = 256
constexpr float kMaxQsc = 1.5474250491067253e26f;  // 2^87
constexpr float kMinScale = 9.094947017729282e-13f, kMaxScale = 1.099511627776e12f;  // 2^-40, 2^40

struct BkParams {
  const __nv_bfloat16* q;  long long q_s0, q_s1;
  const __nv_bfloat16* ke; long long ke_s0, ke_s1;
  const __nv_bfloat16* ve; long long ve_s0, ve_s1;
  __nv_bfloat16* o;        long long o_s0, o_s1;
  const int* qo;
  const int* bt;
  long long bt_s0;
  int bt_cols;
  const int* lens;
  const float* ks;
  const float* vs;
  long long ks_s0, vs_s0;
  long long n_blocks, n_rows;
  int block, bgroups;   // keys, groups of a block
  int box;              // groups of a TMA box: a power of two that divides bgroups, GT at most
  int B, L, gq, R, h_kv, rows;  // rows: of a partial (whole row tiles: R rounded up to 8, 16 or a multiple of 32)
  float scale2;         // softmax scale in base 2
  int team, n_hg, n_team;  // KV heads of a team, h_kv / team, teams
  int tiles;               // row tiles: CTAs of a head in a team
  const unsigned char* cmask;
  const void* mindptr;
  int mindptr64;
  long long n_mask;
  unsigned* err;
  float* plse;
  float* po;
};

using BkFn = void (*)(const BkParams, const CUtensorMap, const CUtensorMap);
using BkJoinFn = void (*)(const BkParams);

// Packed rows of a CTA: the smallest of 8, 16, 32 that holds them (32: in row
// tiles).  A warp finds NR rows 32 / NR times in its lanes and its lanes share the keys:
// with 32 rows for all 64 sequences of 16 rows take 467 us, so 428, 32 single tokens of 4
// rows 109, so 91.
__host__ __device__ constexpr int row_tile(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }

template <int D, int NR>
struct Geo {
  static constexpr int CB = D < 128 ? 64 : 128;     // bytes of a shared-memory row
  static constexpr int NB = D / CB;                 // column blocks of a K / V tile
  static constexpr int ENT = KT * D;                // K (or V) rows of a tile
  // Q: 128 rows.  16 rows fit a warp's lanes with both their terms (hi in the lower
  // half, lo in the upper); 32 have them one behind the other along K.
  static constexpr bool both = NR == 32;
  static constexpr int QW = both ? 2 * D : D;       // bytes of a row
  static constexpr int QCB = QW < 128 ? 64 : 128;   // bytes of its column blocks
  static constexpr int QB = 128 * QW;
  static constexpr int PB = 3 * NR * 128;           // P; the MMA reads 128 rows, of the others nobody takes the result
  static constexpr int NP = D == 128 && NR == 32 ? 1 : 2;  // its buffers
  static constexpr int per_sm = D == 256 ? 1 : 2;
  static constexpr int ctl = 3 * 1024;              // barriers, scales, exchanges
  static constexpr int room = (per_sm == 1 ? kSmemPerCTAMax : kSmemPerSM / 2 - kReservedPerCTA) - ctl - QB - NP * PB;
  static constexpr int entries = room / ENT < 10 ? room / ENT : 10;
  static constexpr int NK = entries / 2, NV = entries - NK;  // ring entries of K and of V (which stay longer)
  static constexpr int q_off = ctl;
  static constexpr int p_off = q_off + QB;
  static constexpr int ring_off = p_off + NP * PB;
  static constexpr int v_off = ring_off + NK * ENT;
  static constexpr int smem = v_off + NV * ENT;
  static constexpr int cols = D == 256 ? 512 : 256;  // S 128, O D
  static_assert(NK >= 2 && NV <= 5 && NK + 2 < kMeta, "ring");
  static_assert(QB >= PB, "a piece's terms meet where P and Q were");
  static_assert((NK + NV) * ENT >= 128 * 128, "the rows behind P are read from the ring");
  static_assert(q_off % 1024 == 0 && p_off % 1024 == 0 && PB % 1024 == 0 && ring_off % 1024 == 0, "swizzled layouts");
};

// control block
constexpr int kScanOff = 0;     // the warps' sums, then the CTA's first segment
constexpr int kBarOff = 128;
constexpr int kBKFull = 0, kBKEmpty = 5, kBVFull = 10, kBVEmpty = 15, kBSFull = 20, kBSEmpty = 21, kBPFull = 22,
              kBPEmpty = 24, kBQFull = 26, kBDone = 27, kBMeta = 28, kNumBars = kBMeta + kMeta;
constexpr int kTmemOff = kBarOff + 8 * kNumBars;
constexpr int kAbortOff = kTmemOff + 4;
constexpr int kQscOff = 448;    // [32] float: a row's score scale
constexpr int kRedOff = 576;    // [4][NR] float: maxima of a tile
constexpr int kSumOff = 1088;   // [4][NR] float: sums of a piece
constexpr int kMetaOff = 1600;  // [kMeta][GT] float4: ks, log2 vs, 1 / vs, keys that are there (+ 256: the tile lacks some)
static_assert(kAbortOff + 4 <= kQscOff && kRedOff + 512 <= kSumOff && kSumOff + 512 <= kMetaOff && kMetaOff + kMeta * GT * 16 <= 3 * 1024,
              "control block");

// Segments and their cut, the same in both kernels.
__device__ __forceinline__ bool prefix_len(const BkParams& p, int b, int& P) {
  const int n = __ldg(p.lens + b);
  const bool ok = n >= 0 && static_cast<long long>(n) <= static_cast<long long>(p.bt_cols) * p.block;
  P = ok ? n : 0;
  return ok;
}
__device__ __forceinline__ int seg_tiles(int P) { return P > 0 ? (P - 1) / KT + 1 : 1; }
__device__ __forceinline__ int share_of(const BkParams& p, int total) {  // (the host bounds the total)
  return (total - 1) / p.n_team + 1;
}
struct BSeg {
  int b, h, P, T;  // h: this CTA's head of the head group; T: tiles
  int off;         // its first tile among all
};
__device__ __forceinline__ void seg_load(const BkParams& p, BSeg& s) {
  prefix_len(p, s.b, s.P);
  s.T = seg_tiles(s.P);
}
__device__ __forceinline__ void seg_next(const BkParams& p, BSeg& s) {
  s.off += s.T;
  s.h += p.team;
  if (s.h >= p.h_kv) {
    s.h %= p.team;
    if (++s.b < p.B) seg_load(p, s);
  }
}
// The groups [g0, ge) of a segment's share, from a whole tile on; empty where the
// prefix is.
__device__ __forceinline__ void piece_of(const BSeg& s, int start, int end, int& g0, int& ge) {
  g0 = (max(start, s.off) - s.off) * GT;
  ge = static_cast<int>(min((static_cast<long long>(s.P) + GK - 1) / GK, static_cast<long long>(end - s.off) * GT));
}

// The CTA's share [start, end) of the tiles and the segment it begins in; all
// threads call it.  False: nothing to do.
__device__ __forceinline__ bool my_share(const BkParams& p, unsigned char* smem, int& start, int& end, BSeg& s) {
  int* scan = reinterpret_cast<int*>(smem + kScanOff);
  volatile int* found = scan + 8;  // sequence, its length, its first tile
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kThreads / 32;
  if (tid == 0) *found = -1;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
  int mine = 0;
  bool bad = false;
  int P = 0;  // the only one where a thread has one sequence: not loaded twice
  for (int b = lo; b < hi; ++b) {
    bad |= !prefix_len(p, b, P);
    mine += seg_tiles(P);
  }
  if (bad && blockIdx.x == 0) atomicOr(p.err, kErrBadKvIndptr);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int at = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) at += scan[w];
    all += scan[w];
  }
  const int total = all * p.n_hg, W = share_of(p, total);
  const int cta = static_cast<int>(blockIdx.x) / p.tiles, member = cta % p.team;
  if (static_cast<long long>(cta / p.team) * W >= total) return false;  // uniform
  start = cta / p.team * W;
  end = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(start) + W));
  if (start >= at * p.n_hg && start < (at + mine) * p.n_hg) {
    for (int b = lo; b < hi; ++b) {
      if (per > 1) prefix_len(p, b, P);
      const int T = seg_tiles(P);
      if (start < (at + T) * p.n_hg) {
        found[0] = b;
        found[1] = P;
        found[2] = at * p.n_hg;
        break;
      }
      at += T;
    }
  }
  __syncthreads();
  s.b = found[0];
  if (s.b < 0) return false;  // not reached: guards the walk
  s.P = found[1];
  s.T = seg_tiles(s.P);
  const int hg = (start - found[2]) / s.T;
  s.h = hg * p.team + member;
  s.off = found[2] + hg * s.T;
  return true;
}

// Groups 32 at a time (four tiles), piece after piece, for the loader.
struct BatchIt {
  BSeg s;
  int g, ge;
  bool valid;
  __device__ __forceinline__ void settle(const BkParams& p, int start, int end) {
    while (g >= ge) {
      seg_next(p, s);
      if (s.b >= p.B || s.off >= end) {
        valid = false;
        return;
      }
      piece_of(s, start, end, g, ge);
    }
  }
  __device__ __forceinline__ void first(const BkParams& p, const BSeg& s0, int start, int end) {
    s = s0;
    valid = true;
    piece_of(s, start, end, g, ge);
    settle(p, start, end);
  }
  __device__ __forceinline__ void next(const BkParams& p, int start, int end) {
    g += 32;
    settle(p, start, end);
  }
};

// Shared-memory matrix descriptor of rows of CB bytes in the CB-byte swizzle
// (version 1; layout 2: 128 bytes, 4: 64 bytes).
template <int CB>
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46) | (static_cast<uint64_t>(CB == 128 ? 2 : 4) << 61);
}
// fa::wait_all for two phases at once (a look takes some 150 cycles).
__device__ __forceinline__ bool wait_both(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, volatile int* abort_flag, unsigned* err) {
  const bool x = tr::test(a, pa), y = tr::test(b, pb);
  if (__all_sync(0xffffffffu, x && y)) return true;
  return fa::wait_all(a, pa, abort_flag, err) && fa::wait_all(b, pb, abort_flag, err);
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// The top 4 significant bits of y where e4m3 has them all (2^-6 and above), else 0.
__device__ __forceinline__ float top_bits(float y) {
  uint32_t there;
  asm("set.geu.u32.f32 %0, %1, 0f3C800000;" : "=r"(there) : "f"(y));  // (unordered: NaN stays NaN)
  return __uint_as_float(__float_as_uint(y) & 0xFFF00000u & there);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// The row tile's packed rows (row r = draft r / gq, query head h gq + r % gq;
// rows from R on are zero) into Q, as hi and lo terms, 128 / NR times (64 / NR), and
// their score scales; by the softmax warps, NR / 4 rows each.  First the loads alone.
template <int D, int NR>
struct Rows {
  static constexpr int W = D / 64;  // 32-bit words of a row per lane
  static constexpr int J = NR / 4;
  uint32_t v[J][W];
  __device__ __forceinline__ void fetch(const BkParams& p, const BSeg& s, int warp, int lane) {
    const int a = __ldg(p.qo + s.b), e = __ldg(p.qo + s.b + 1);
    const bool ok = a >= 0 && e - a == p.L && static_cast<long long>(a) + p.L <= p.n_rows;
    const long long first = ok ? a : static_cast<long long>(s.b) * p.L;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int r = static_cast<int>(blockIdx.x) % p.tiles * NR + J * warp + j;
      const bool live = r < p.R;
      const int rr = live ? r : 0;
      const __nv_bfloat16* src = p.q + (first + rr / p.gq) * p.q_s0 + static_cast<long long>(s.h * p.gq + rr % p.gq) * p.q_s1;
#pragma unroll
      for (int w = 0; w < W; ++w) v[j][w] = live ? ld_u32(src + 2 * (W * lane + w)) : 0u;
    }
  }
};
template <int D, int NR>
__device__ __forceinline__ void put_rows(const BkParams& p, Rows<D, NR>& rows, unsigned char* smem, int warp, int lane) {
  using G = Geo<D, NR>;
  constexpr int W = Rows<D, NR>::W, J = Rows<D, NR>::J;
  uint32_t (&v)[J][W] = rows.v;
  float* qsc = reinterpret_cast<float*>(smem + kQscOff);
  unsigned most[J], all = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    most[j] = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) most[j] = max(most[j], mag_bf16x2(v[j][w]));
    most[j] = __reduce_max_sync(0xffffffffu, most[j]);
    all = max(all, most[j]);
  }
  if (all >= kBf16Inf) {
    // e4m3 has no infinity; an infinite query makes its row's softmax NaN, as NaN does
#pragma unroll
    for (int j = 0; j < J; ++j) {
      most[j] = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        most[j] = max(most[j], finite_mag_bf16x2(v[j][w]));
        v[j][w] = inf_to_nan_bf16x2(v[j][w]);
      }
      most[j] = __reduce_max_sync(0xffffffffu, most[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int row = J * warp + j;
    const unsigned mx = most[j];
    // the row's largest |q| 2^sh lies in [128, 256)
    const int sh = mx == 0 ? 0 : max(-120, min(120, 7 - (static_cast<int>(mx >> 7) - 127)));
    const float up = __int_as_float((127 + sh) << 23);
    // capped, so that with the largest block scale it is still finite and a product of 0 a
    // score of 0; where the cap holds, scores are equal or at least 2^29 apart all the same
    if (lane == 0) qsc[row] = fminf(p.scale2 * __int_as_float((127 - sh) << 23), kMaxQsc);
    uint32_t hi[(W + 1) / 2] = {}, lo[(W + 1) / 2] = {};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 f = unpack_bf16(v[j][w]);
      const float x0 = f.x * up, x1 = f.y * up;
      const unsigned short h = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hh = e4m3x2_to_f16x2(h);
      const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hh));
      const unsigned short l = __nv_cvt_float2_to_fp8x2(make_float2(x0 - hf.x, x1 - hf.y), __NV_SATFINITE, __NV_E4M3);
      hi[w >> 1] |= static_cast<uint32_t>(h) << (16 * (w & 1));
      lo[w >> 1] |= static_cast<uint32_t>(l) << (16 * (w & 1));
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t* x = t ? lo : hi;
      // NR 32: byte t D + .. of row `row`, four times; else row `row` of each 16 (or
      // twice 8) rows, hi and lo in turn
      const int at = (G::both ? t * D : 0) + 2 * W * lane;
#pragma unroll
      for (int k = 0; k < (G::both ? 4 : 64 / NR); ++k) {
        const int qr = G::both ? 32 * k + row : 32 * (k * NR / 16) + 16 * t + k * NR % 16 + row;
        constexpr int CB = G::QCB;
        const int swz = CB == 128 ? qr & 7 : (qr >> 1) & 3;
        unsigned char* d = smem + G::q_off + at / CB * (128 * CB) + qr * CB + (((at % CB >> 4) ^ swz) << 4) + (at & 15);
        if constexpr (W == 1)
          *reinterpret_cast<unsigned short*>(d) = static_cast<unsigned short>(x[0]);
        else if constexpr (W == 2)
          *reinterpret_cast<uint32_t*>(d) = x[0];
        else
          *reinterpret_cast<uint2*>(d) = make_uint2(x[0], x[1]);
      }
    }
  }
}

}  // namespace bk

template <int D, int NR>
__global__ void __launch_bounds__(bk::kThreads, bk::Geo<D, NR>::per_sm)
    block_stream_kernel(const __grid_constant__ bk::BkParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using namespace bk;
  using tc::idesc, tc::mbar_arrive, tc::mbar_init, tc::mma_commit, tc::mma_f8_ss, tc::fence_proxy_async;
  using tc::tc_fence_after, tc::tc_fence_before, tc::tmem_ld, tc::tmem_st, tc::tmem_wait_st;
  using G = bk::Geo<D, NR>;
  constexpr int NK = G::NK, NV = G::NV, CB = G::CB, ENT = G::ENT, NP = G::NP;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int start, end;
  BSeg seg0;
  if (!my_share(p, smem, start, end, seg0)) return;  // uniform
  if ((smem_u32(smem) & 1023u) != 0u) {  // the swizzled layouts need it; dynamic shared memory starts so
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  const uint32_t k_s = smem_u32(smem + G::ring_off), v_s = smem_u32(smem + G::v_off);
  // what the first tile needs from memory is asked for before the set-up
  Rows<D, NR> rows;
  BatchIt cur;
  int page = -1;
  auto page_of_group = [&](const BatchIt& it) -> int {  // block of group `lane` of a batch
    const int gi = it.g + lane;
    return it.valid && gi < it.ge ? __ldg(p.bt + static_cast<long long>(it.s.b) * p.bt_s0 + gi / p.bgroups) : -1;
  };
  if (warp < 4) {
    rows.fetch(p, seg0, warp, lane);
  } else if (warp != 5) {
    cur.first(p, seg0, start, end);
    page = page_of_group(cur);
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < NK; ++i) {
      mbar_init(bar(kBKFull + i), 1);
      mbar_init(bar(kBKEmpty + i), 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(bar(kBVFull + i), 1);
      mbar_init(bar(kBVEmpty + i), 1);
    }
    mbar_init(bar(kBSFull), 1);
    mbar_init(bar(kBSEmpty), 4);
    for (int i = 0; i < NP; ++i) {
      mbar_init(bar(kBPFull + i), 4);
      mbar_init(bar(kBPEmpty + i), 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(bar(kBMeta + i), 1);
    mbar_init(bar(kBQFull), 4);
    mbar_init(bar(kBDone), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem + kTmemOff)),
                 "r"(G::cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kTmemOff);
  const uint32_t tS = tmem, tO = tmem + KT;

  if (warp == 4 || warp == 6) {
    // ================================ loaders ================================
    // Warp 4 brings K, warp 6 V and the scales.  Each goes on by itself: a K entry is
    // free once its scores are done, a V entry only when its weights have met it; and a
    // tile costs a warp some hundred cycles (one for both, 64 of 8k..16k keys at
    // head_dim 64: 229 us, so 192).
    const bool isv = warp == 6;
    const CUtensorMap* map = isv ? &vmap : &kmap;
    const uint32_t n_ent = isv ? NV : NK, ring = isv ? v_s : k_s;
    const int full0 = isv ? kBVFull : kBKFull, empty0 = isv ? kBVEmpty : kBKEmpty;
    float4* meta = reinterpret_cast<float4*>(smem + kMetaOff);
    BatchIt ahead;
    int page2 = -1;
    float ks = 1.f, vs = 1.f, ks2 = 1.f, vs2 = 1.f;
    auto scales = [&](int pg, int h, float& k, float& v) {
      k = v = 1.f;
      if (isv && pg >= 0 && pg < p.n_blocks) {
        k = __ldg(p.ks + pg * p.ks_s0 + h);
        v = __ldg(p.vs + pg * p.vs_s0 + h);
      }
    };
    scales(page, cur.s.h, ks, vs);
    uint32_t u = 0, issued = 0;
    uint32_t st = 0, par = 1;
    bool alive = true;
#pragma unroll 1
    while (cur.valid && alive) {
      const int gi = cur.g + lane;
      const bool in = gi < cur.ge, ok = in && page >= 0 && page < p.n_blocks;
      if (in && !ok && isv) atomicOr(p.err, kErrBadIndex);
      const int keys = ok ? min(GK, cur.s.P - gi * GK) : 0;
      const int row = ok ? page * p.block + gi % p.bgroups * GK : -1;
      const int tiles = (min(32, cur.ge - cur.g) + GT - 1) / GT;
      float4 mine;
#pragma unroll 1
      for (int j = 0; j < tiles; ++j, ++u) {
        // V's entry waits for the weights of a tile before; the scales are asked for with
        // the first tile's scores
        const bool late = isv && u < n_ent;
        auto tell = [&] {
          if (j == 0) {
            // a scale that is no positive finite number in the range gives NaN
            const bool good = ks >= kMinScale && ks <= kMaxScale && vs >= kMinScale && vs <= kMaxScale;
            if (!good) atomicOr(p.err, kErrBadScale);
            const float nan = __int_as_float(0x7FC00000);
            mine = make_float4(good ? ks : nan, good ? log2f(vs) : nan, good ? 1.f / vs : nan, __int_as_float(keys));
          }
          const bool lacks = __any_sync(0xffffffffu, (lane >> 3) == j && keys < GK);
          if ((lane >> 3) == j) {
            float4 x = mine;
            if (lacks) x.w = __int_as_float(keys + 256);
            meta[(u % kMeta) * GT + (lane & 7)] = x;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBMeta + u % kMeta));
        };
        if (isv && !late) tell();
        alive = fa::wait_all(bar(empty0 + st), par, abort_flag, p.err);
        if (!alive) break;
        int at[GT];  // first rows in the cache
#pragma unroll
        for (int i = 0; i < GT; ++i) at[i] = __shfl_sync(0xffffffffu, row, GT * j + i);
        // one lane copies all boxes (lanes that each copy one are taken one after the
        // other, some 130 cycles each)
        if (fa::elect_one()) {
          uint32_t n = 0;
#pragma unroll
          for (int i = 0; i < GT; ++i) n += (i & (p.box - 1)) == 0 && at[i] >= 0;
          expect(bar(full0 + st), n * p.box * (GK * D));
#pragma unroll
          for (int i = 0; i < GT; ++i)
            if ((i & (p.box - 1)) == 0 && at[i] >= 0)
#pragma unroll
              for (int c = 0; c < G::NB; ++c)
                fa::tma_load_box(ring + st * ENT + c * (KT * CB) + i * (GK * CB), map, bar(full0 + st), c * CB, cur.s.h, at[i]);
        }
        __syncwarp();
        if (late) tell();  // the first entries are free: copies first
        issued = u + 1;
        if (j == 0) {  // the next batch's blocks, while this one's tiles are on their way
          ahead = cur;
          ahead.next(p, start, end);
          page2 = page_of_group(ahead);
        }
        if (++st == n_ent) {
          st = 0;
          par ^= 1u;
        }
      }
      if (!alive) break;
      scales(page2, ahead.valid ? ahead.s.h : 0, ks2, vs2);
      cur = ahead;
      page = page2;
      ks = ks2;
      vs = vs2;
    }
    // block_combine_kernel's CTAs may start (they wait for this grid themselves)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the copies end before the CTA does (in a CTA that gave up, nobody else waits for them)
    for (uint32_t k = 1; k <= n_ent && k <= issued; ++k)
      fa::wait_last(bar(full0 + (issued - k) % n_ent), ((issued - k) / n_ent) & 1u);
  } else if (warp == 5) {
    // ================================ MMAs ================================
    constexpr uint32_t idS = idesc(0, 0, 0, 0, 128, KT), idO = idesc(0, 0, 0, 1, 128, D);
    const uint64_t dq = desc<G::QCB>(smem_u32(smem + G::q_off), 16, 8 * G::QCB), dp = desc<128>(smem_u32(smem + G::p_off), 16, 1024);
    const uint64_t dk = desc<CB>(k_s, 16, 8 * CB), dv = desc<CB>(v_s, KT * CB, 8 * CB);
    uint32_t u = 0, piece = 0;
    bool pending = false, pfirst = false, alive = true;
    auto wait = [&](int i, uint32_t pi, int k, uint32_t pk) { alive = alive && wait_both(bar(i), pi, bar(k), pk, abort_flag, p.err); };
    auto weigh = [&](uint32_t w, bool first) {  // O += P V of tile w
      const uint32_t st = w % NV;
      wait(kBPFull + w % NP, (w / NP) & 1u, kBVFull + st, (w / NV) & 1u);
      tc_fence_after();
      if (alive && fa::elect_one()) {
        const uint64_t vd = dv + static_cast<uint64_t>((st * ENT) >> 4);
        const uint64_t pd = dp + static_cast<uint64_t>(((w % NP) * G::PB) >> 4);
#pragma unroll
        for (int k = 0; k < KT / 32; ++k)
          mma_f8_ss(tO, pd + static_cast<uint64_t>(2 * k), vd + static_cast<uint64_t>((k * 32 * CB) >> 4), idO, !(first && k == 0));
        mma_commit(bar(kBPEmpty + w % NP));
        mma_commit(bar(kBVEmpty + st));
      }
      __syncwarp();
    };
    BSeg s = seg0;
#pragma unroll 1
    while (s.b < p.B && s.off < end) {
      int g0, ge;
      piece_of(s, start, end, g0, ge);
      if (g0 < ge) {
        if (pending) {  // the piece before ends first: its partial precedes this piece's queries
          weigh(u - 1, pfirst);
          pending = false;
        }
        wait(kBQFull, piece & 1u, kBQFull, piece & 1u);
        ++piece;
#pragma unroll 1
        for (int g = g0; g < ge; g += GT, ++u) {
          const uint32_t st = u % NK;
          wait(kBKFull + st, (u / NK) & 1u, kBSEmpty, (u & 1u) ^ 1u);
          tc_fence_after();
          if (alive && fa::elect_one()) {
            const uint64_t kd = dk + static_cast<uint64_t>((st * ENT) >> 4);
#pragma unroll
            for (int t = 0; t < (G::both ? 2 : 1); ++t)
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                const int qb = t * D + 32 * k, kb = 32 * k;
                mma_f8_ss(tS, dq + static_cast<uint64_t>((qb / G::QCB * (128 * G::QCB) + qb % G::QCB) >> 4),
                          kd + static_cast<uint64_t>(((kb / CB) * (KT * CB) + kb % CB) >> 4), idS, t + k > 0);
              }
            mma_commit(bar(kBSFull));
            mma_commit(bar(kBKEmpty + st));
          }
          __syncwarp();
          if (pending) weigh(u - 1, pfirst);
          pending = true;
          pfirst = g == g0;
        }
      }
      seg_next(p, s);
    }
    if (pending) weigh(u - 1, pfirst);
    if (fa::elect_one()) mma_commit(bar(kBDone));
    __syncwarp();
    fa::wait_last(bar(kBDone), 0);
  } else {
    // ================================ softmax ================================
    // Thread (warp w, lane): row lane % NR, its KN = NR keys 32 w + NR (lane / NR) ..
    constexpr int KN = NR;              // keys of a thread
    constexpr int NG = KN > GK ? 2 : 1;  // their groups
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const float NEG_INF = -INFINITY;
    const int r = lane & (NR - 1), part = lane / NR;
    const int key0 = 32 * warp + KN * part;  // this thread's first key of a tile
    const float4* meta = reinterpret_cast<const float4*>(smem + kMetaOff);
    float* red = reinterpret_cast<float*>(smem + kRedOff);
    float* sums = reinterpret_cast<float*>(smem + kSumOff);
    const float* qscs = reinterpret_cast<const float*>(smem + kQscOff);
    uint32_t u = 0;
    bool alive = true;
    auto wait = [&](int i, uint32_t parity) { alive = alive && fa::wait_all(bar(i), parity, abort_flag, p.err); };
    auto arrive = [&](int i) {
      if (lane == 0 && alive) mbar_arrive(bar(i));
    };
    auto wait_weighed = [&](uint32_t v) {  // P V of tile v done (and so of those before)
      wait(kBPEmpty + v % NP, (v / NP) & 1u);
      tc_fence_after();
    };
    BSeg s = seg0;
#pragma unroll 1
    for (; s.b < p.B && s.off < end; seg_next(p, s)) {
      int g0, ge;
      piece_of(s, start, end, g0, ge);
      const long long slot = static_cast<int>(blockIdx.x) / p.tiles + static_cast<long long>(s.b) * p.h_kv + s.h / p.team * p.team;
      const int row0 = static_cast<int>(blockIdx.x) % p.tiles * NR;
      float* lse_p = p.plse + slot * p.rows + row0;
      float* o_p = p.po + (slot * p.rows + row0) * D;
      const int live = min(NR, p.R - row0);
      if (g0 >= ge) {  // no key: an empty partial
        if (tid < live) lse_p[tid] = NEG_INF;
        continue;
      }
      if (s.off > start) rows.fetch(p, s, warp, lane);  // (the first piece's are on their way)
      put_rows<D, NR>(p, rows, smem, warp, lane);
      fence_proxy_async();
      named_bar_sync(1, kSm);  // the rows' scales
      arrive(kBQFull);
      const float qsc = qscs[r];
      float m = NEG_INF, l = 0.f;
#pragma unroll 1
      for (int g = g0; g < ge; g += GT, ++u) {
        alive = alive && wait_both(bar(kBSFull), u & 1u, bar(kBMeta + u % kMeta), (u / kMeta) & 1u, abort_flag, p.err);
        tc_fence_after();
        float x[KN];
        {
          float y[32];
          tmem_ld<32>(tS + lanes + 32 * warp, y);
          tc_fence_before();
          __syncwarp();
          arrive(kBSEmpty);
          // with 16 rows or fewer the lower half of the lanes holds the hi terms' scores
          // of all 32 keys and the upper half the lo terms': each gets those of its keys
          // from lane ^ 16
          if constexpr (NR == 32) {
#pragma unroll
            for (int i = 0; i < KN; ++i) x[i] = y[i];
          } else if constexpr (NR == 16) {
#pragma unroll
            for (int i = 0; i < KN; ++i) {
              const float mine = part ? y[16 + i] : y[i], its = part ? y[i] : y[16 + i];
              x[i] = mine + __shfl_xor_sync(0xffffffffu, its, 16);
            }
          } else {
#pragma unroll
            for (int i = 0; i < KN; ++i) {
              const float lo = part & 1 ? y[8 + i] : y[i], hi = part & 1 ? y[24 + i] : y[16 + i];
              const float mine = part & 2 ? hi : lo, its = part & 2 ? lo : hi;
              x[i] = mine + __shfl_xor_sync(0xffffffffu, its, 16);
            }
          }
        }
        const float4* mt = meta + (u % kMeta) * GT + key0 / GK;
        float4 me[NG];
#pragma unroll
        for (int h = 0; h < NG; ++h) me[h] = mt[h];
#pragma unroll
        for (int i = 0; i < KN; i += 2) {
          const float c = qsc * me[i / GK].x;
          const float2 y = fa::fma2(make_float2(x[i], x[i + 1]), make_float2(c, c), make_float2(me[i / GK].y, me[i / GK].y));
          x[i] = y.x;
          x[i + 1] = y.y;
        }
        const bool lacks = __float_as_int(me[0].w) >= 256;
        if (lacks) {
#pragma unroll
          for (int i = 0; i < KN; ++i)
            if ((key0 & (GK - 1)) + (i & (GK - 1)) >= (__float_as_int(me[i / GK].w) & 255)) x[i] = NEG_INF;
        }
        float t2[2] = {NEG_INF, NEG_INF};
#pragma unroll
        for (int i = 0; i < KN; i += 2) t2[i >> 1 & 1] = fa::max3(t2[i >> 1 & 1], x[i], x[i + 1]);
        float tm = fmaxf(t2[0], t2[1]);
        // The reference stays while no row of the tile passes it by 2^kThr.
        if (g == g0 || tc::bar_red_or(1, kSm, tm > m + kThr)) {  // alike in the four warps
#pragma unroll
          for (int o = NR; o < 32; o *= 2) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
          if (lane < NR) red[warp * NR + lane] = tm;
          named_bar_sync(1, kSm);
          tm = fmaxf(fmaxf(red[r], red[NR + r]), fmaxf(red[2 * NR + r], red[3 * NR + r]));
          const float mn = fmaxf(m, tm);
          const float al = mn == NEG_INF ? 1.f : fast_exp2(m - mn);
          if (g > g0) {  // O holds the piece's earlier tiles
            wait_weighed(u - 1);
            if (32 * warp < 3 * NR) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld<32>(tO + lanes + c, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= al;
                tmem_st<32>(tO + lanes + c, o);
              }
              tmem_wait_st();
            }
          }
          l *= al;
          m = mn;
        }
        // (looked at here: the answer comes while the weights are computed)
        const bool is_free = u < NP || tr::test(bar(kBPEmpty + u % NP), ((u / NP) & 1u) ^ 1u);
        const float up = m == NEG_INF ? 0.f : static_cast<float>(kUp) - m;
        uint32_t w[3][KN / 4];
        float2 sum[NG];
#pragma unroll
        for (int h = 0; h < NG; ++h) sum[h] = make_float2(0.f, 0.f);
        const float2 up2 = make_float2(up, up), k16 = make_float2(16.f, 16.f), zero = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < KN / 4; ++i) {
          float2 t[3][2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 z = fa::add2(make_float2(x[4 * i + 2 * e], x[4 * i + 2 * e + 1]), up2);
            const float2 y = make_float2(fast_exp2(z.x), fast_exp2(z.y));
            sum[i / 4] = fa::add2(sum[i / 4], y);
            const float2 a = make_float2(top_bits(y.x), top_bits(y.y));
            const float2 r = fa::fma2(fa::add2(y, make_float2(-a.x, -a.y)), k16, zero);
            const float2 b = make_float2(top_bits(r.x), top_bits(r.y));
            t[0][e] = a;
            t[1][e] = b;
            t[2][e] = fa::fma2(fa::add2(r, make_float2(-b.x, -b.y)), k16, zero);
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) w[k][i] = e4m3x4(t[k][0].x, t[k][0].y, t[k][1].x, t[k][1].y);
        }
#pragma unroll
        for (int h = 0; h < NG; ++h) l = fmaf(sum[h].x + sum[h].y, me[h].z, l);
        if (!__all_sync(0xffffffffu, is_free)) wait_weighed(u - NP);  // the buffer's tile before
        unsigned char* pb = smem + G::p_off + (u % NP) * G::PB;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int pr = NR * k + r;
          unsigned char* at = pb + pr * 128;
          if constexpr (KN >= 16) {
#pragma unroll
            for (int h = 0; h < KN / 16; ++h)
              *reinterpret_cast<uint4*>(at + (((key0 / 16 + h) ^ (pr & 7)) << 4)) =
                  make_uint4(w[k][4 * h], w[k][4 * h + 1], w[k][4 * h + 2], w[k][4 * h + 3]);
          } else {
            *reinterpret_cast<uint2*>(at + (((key0 / 16) ^ (pr & 7)) << 4) + (key0 & 15)) = make_uint2(w[k][0], w[k][1]);
          }
        }
        if (lacks) {
          // V rows of keys that are not there: 0 times what lies there may be NaN
          const uint32_t st = u % NV;
          wait(kBVFull + st, (u / NV) & 1u);
          if ((tid & 15) >= (__float_as_int(meta[(u % kMeta) * GT + (tid >> 4)].w) & 255)) {
            unsigned char* v = smem + G::v_off + st * ENT + tid * CB;
#pragma unroll
            for (int c = 0; c < G::NB; ++c)
#pragma unroll
              for (int i = 0; i < CB; i += 16) *reinterpret_cast<uint4*>(v + c * (KT * CB) + i) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        arrive(kBPFull + u % NP);
      }
      // ---- the piece's partial: o = sum of the terms / l, log2 of the sum ----
#pragma unroll
      for (int o = NR; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane < NR) sums[warp * NR + lane] = l;
      wait_weighed(u - 1);
      named_bar_sync(1, kSm);
      const float lt = (sums[r] + sums[NR + r]) + (sums[2 * NR + r] + sums[3 * NR + r]);
      if (warp == 0 && lane < live) lse_p[lane] = lt == 0.f ? NEG_INF : m + (log2f(lt) - static_cast<float>(kUp));
      // the terms meet in shared memory, [3][NR rows][32 columns] at a time, by turns where
      // P and Q were: a warp that writes the next but one has seen all read this one
      constexpr int TPR = 128 / NR, CPT = 32 / TPR;  // threads of a row, columns of a thread
      const int orow = tid / TPR, oc = (tid % TPR) * CPT;
      const float lo = (sums[orow] + sums[NR + orow]) + (sums[2 * NR + orow] + sums[3 * NR + orow]);
      const float inv = lo == 0.f ? 0.f : 1.f / lo;
      const int pr = 32 * warp + lane;  // term pr / NR of row pr % NR
#pragma unroll 2
      for (int c = 0; c < D; c += 32) {
        unsigned char* stage = smem + (c & 32 ? G::q_off : G::p_off);
        if (32 * warp < 3 * NR) {
          float o[32];
          tmem_ld<32>(tO + lanes + c, o);
          if (pr < 3 * NR) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(stage + pr * 128 + ((i ^ (pr & 7)) << 4)) =
                  make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        named_bar_sync(1, kSm);
        if (orow < live) {
          // NR is a multiple of 8: the three terms' rows are swizzled alike
          using V = std::conditional_t<CPT == 2, float2, float4>;
          constexpr int VN = sizeof(V) / 4;
          float res[CPT];
#pragma unroll
          for (int i = 0; i < CPT; i += VN) {
            const unsigned char* at = stage + orow * 128 + ((((oc + i) >> 2) ^ (orow & 7)) << 4) + (oc & (4 - VN)) * 4;
            V term[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) term[k] = *reinterpret_cast<const V*>(at + k * (NR * 128));
            const float *a = reinterpret_cast<const float*>(&term[0]), *b = reinterpret_cast<const float*>(&term[1]),
                        *d = reinterpret_cast<const float*>(&term[2]);
#pragma unroll
            for (int e = 0; e < VN; ++e) res[i + e] = fmaf(d[e], 0.00390625f, fmaf(b[e], 0.0625f, a[e])) * inv;
          }
          float* out = o_p + orow * D + c + oc;
#pragma unroll
          for (int i = 0; i < CPT; i += 2) *reinterpret_cast<float2*>(out + i) = make_float2(res[i], res[i + 1]);
        }
      }
      named_bar_sync(1, kSm);  // P and Q are free
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::cols) : "memory");
  }
}

bk::BkFn kernel_block_stream_64(int nr);  // nr: rows of a CTA
bk::BkFn kernel_block_stream_128(int nr);  // nr: rows of a CTA
bk::BkFn kernel_block_stream_256(int nr);  // nr: rows of a CTA
bk::BkJoinFn kernel_block_combine_64(bool split);
bk::BkJoinFn kernel_block_combine_128(bool split);
bk::BkJoinFn kernel_block_combine_256(bool split);

}  // namespace vsk
