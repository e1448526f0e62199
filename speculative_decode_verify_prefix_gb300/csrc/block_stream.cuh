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
//   queries  q 2^sh = hi + lo exactly (bf16 has 8 significant bits, a term 4;
//            elements 2^17 below the row's largest lose bits that no score
//            shows), both terms along K of one accumulator;
//   weights  y = 2^6 x: the top 4 bits, the next 4 and the rest rounded to 4, as
//            three groups of rows of one M = 128 product under scales 1, 2^4,
//            2^8: 12 bits, and 2^-24 of the reference at the lower end.
// A tile is 128 keys of one KV head:
//   S[128][128 keys] = Q[128][hi | lo] x K^T   (up to 32 packed rows, four times:
//                      every warp then finds all rows in its own lanes)
//   O[128][D]       += P[128][128 keys] x V    (rows 32 p + r: term p of row r)
//
// Roles (6 warps; two CTAs an SM at head_dim 64 and 128, one at 256):
//   warps 0-3  softmax: thread (w, r) holds keys 32 w .. 32 w + 31 of row r.
//   warp 4     block table and scales, TMA of 16-key boxes into the ring.
//   warp 5     tensor memory, MMAs.
// The groups of 16 keys of all (sequence, KV head) segments are laid end to end
// and every CTA takes an equal share; a segment's part of a share is a piece,
// whose partial (o, log2 of its sum) block_combine_kernel folds.
// Every wait is bounded (one second); a CTA that gives up sets error bit 8,
// waits for its copies and MMAs in flight, frees its tensor memory and exits.
#pragma once
#include "flash_tc.cuh"

namespace vsk {

enum : unsigned { kErrBadScale = 64u };

namespace bk {

constexpr int KT = 128;      // keys of a tile
constexpr int GK = 16;       // keys of a group (one TMA box, one block's scale)
constexpr int GT = KT / GK;  // groups of a tile
constexpr int RT = 32;       // packed rows of a CTA
constexpr int kThreads = 192;
constexpr int kSm = 128;     // softmax threads
constexpr int kMeta = 8;     // tiles whose scales are kept (more than the ring holds)
constexpr float kThr = 2.f;  // log2 headroom before a reference is raised
constexpr int kUp = 6;       // y = 2^kUp x <= 2^(kUp + kThr) = 256
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
  int B, L, gq, R, h_kv, rows;  // rows: of a partial (RT row tiles of 32)
  float scale2;         // softmax scale in base 2
  int w_min;            // groups of a share at least
  int n_cta;
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

template <int D>
struct Geo {
  static constexpr int CB = D < 128 ? 64 : 128;     // bytes of a shared-memory row
  static constexpr int NB = D / CB;                 // column blocks of a K / V tile
  static constexpr int ENT = KT * D;                // K (or V) rows of a tile
  static constexpr int QB = 128 * 2 * D;            // Q: [hi | lo] in 128-byte column blocks
  static constexpr int PB = 96 * 128;               // P; the MMA reads 32 rows more, whose result nobody takes
  static constexpr int per_sm = D == 256 ? 1 : 2;
  static constexpr int ctl = 3072;                  // barriers, scales, exchanges
  static constexpr int room = (per_sm == 1 ? kSmemPerCTAMax : kSmemPerSM / 2 - kReservedPerCTA) - ctl - QB - PB;
  static constexpr int NS = room / (2 * ENT) < 5 ? room / (2 * ENT) : 5;  // stages
  static constexpr int q_off = ctl;
  static constexpr int p_off = q_off + QB;
  static constexpr int ring_off = p_off + PB;
  static constexpr int smem = ring_off + 2 * NS * ENT;
  static constexpr int cols = D == 256 ? 512 : 256;  // S 128, O D
  static_assert(NS >= 1 && NS + 2 < kMeta, "ring");
  static_assert(2 * ENT >= 32 * 128, "P's last rows are read from the ring");
};

// control block
constexpr int kScanOff = 0;    // 6 warps' sums, then the CTA's first segment
constexpr int kBarOff = 128;
constexpr int kBKFull = 0, kBKEmpty = 5, kBVFull = 10, kBVEmpty = 15, kBSFull = 20, kBSEmpty = 21, kBPFull = 22,
              kBPEmpty = 23, kBQFull = 24, kBDone = 25, kNumBars = 26;
constexpr int kTmemOff = kBarOff + 8 * kNumBars;
constexpr int kAbortOff = kTmemOff + 4;
constexpr int kQscOff = 352;   // [32] float: a row's score scale
constexpr int kMetaOff = 512;  // [kMeta][GT] float4: ks, log2 vs, 1 / vs, keys that are there (+ 256: the tile lacks some)
constexpr int kRedOff = 1536;  // [2][4][32] float: maxima of a tile
constexpr int kSumOff = 2560;  // [4][32] float: sums of a piece
static_assert(kAbortOff + 4 <= kQscOff && kMetaOff + kMeta * GT * 16 <= kRedOff && kRedOff + 1024 <= kSumOff, "control block");

// Segments and their cut, the same in both kernels.
struct Cut {
  long long total, W;
};
__device__ __forceinline__ bool prefix_len(const BkParams& p, int b, int& P) {
  const int n = __ldg(p.lens + b);
  const bool ok = n >= 0 && static_cast<long long>(n) <= static_cast<long long>(p.bt_cols) * p.block;
  P = ok ? n : 0;
  return ok;
}
__device__ __forceinline__ int seg_groups(int P) { return P > 0 ? static_cast<int>((static_cast<long long>(P) + GK - 1) / GK) : 1; }
__device__ __forceinline__ long long share_of(const BkParams& p, long long total) {
  long long W = (total + p.n_cta - 1) / p.n_cta;
  if (W < p.w_min) W = p.w_min;
  return W > GT ? (W + GT - 1) / GT * GT : W;
}
struct BSeg {
  int b, h, P, G;
  long long off;  // its first group among all
};
__device__ __forceinline__ void seg_load(const BkParams& p, BSeg& s) {
  prefix_len(p, s.b, s.P);
  s.G = seg_groups(s.P);
}
__device__ __forceinline__ void seg_next(const BkParams& p, BSeg& s) {
  s.off += s.G;
  if (++s.h == p.h_kv) {
    s.h = 0;
    if (++s.b < p.B) seg_load(p, s);
  }
}
// The real groups [g0, ge) of a segment in a share; empty where there are none.
__device__ __forceinline__ void piece_of(const BSeg& s, long long start, long long end, int& g0, int& ge) {
  g0 = static_cast<int>(max(start, s.off) - s.off);
  ge = s.P > 0 ? static_cast<int>(min(static_cast<long long>(s.G), end - s.off)) : 0;
}

// The CTA's share [start, end) of the groups and the segment it begins in; all
// threads call it.  False: nothing to do.
__device__ __forceinline__ bool my_share(const BkParams& p, unsigned char* smem, long long& start, long long& end, BSeg& s) {
  long long* scan = reinterpret_cast<long long*>(smem + kScanOff);
  volatile long long* base = scan + 8;
  volatile int* found = reinterpret_cast<volatile int*>(scan + 9);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kThreads / 32;
  if (tid == 0) *found = -1;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
  long long mine = 0;
  bool bad = false;
  for (int b = lo; b < hi; ++b) {
    int P;
    bad |= !prefix_len(p, b, P);
    mine += seg_groups(P);
  }
  if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, kErrBadKvIndptr);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long at = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) at += scan[w];
    all += scan[w];
  }
  const long long total = all * p.h_kv, W = share_of(p, total);
  start = blockIdx.x * W;
  if (start >= total) return false;  // uniform
  end = min(total, start + W);
  for (int b = lo; b < hi; ++b) {
    int P;
    prefix_len(p, b, P);
    const int G = seg_groups(P);
    if (start >= at * p.h_kv && start < (at + G) * p.h_kv) {
      *found = b;
      *base = at * p.h_kv;
    }
    at += G;
  }
  __syncthreads();
  s.b = *found;
  if (s.b < 0) return false;  // not reached: guards the walk
  seg_load(p, s);
  s.h = static_cast<int>((start - *base) / s.G);
  s.off = *base + static_cast<long long>(s.h) * s.G;
  return true;
}

// Groups 32 at a time (four tiles), piece after piece, for the loader.
struct BatchIt {
  BSeg s;
  int g, ge;
  bool valid;
  __device__ __forceinline__ void settle(const BkParams& p, long long start, long long end) {
    while (g >= ge) {
      seg_next(p, s);
      if (s.b >= p.B || s.off >= end) {
        valid = false;
        return;
      }
      piece_of(s, start, end, g, ge);
    }
  }
  __device__ __forceinline__ void first(const BkParams& p, const BSeg& s0, long long start, long long end) {
    s = s0;
    valid = true;
    piece_of(s, start, end, g, ge);
    settle(p, start, end);
  }
  __device__ __forceinline__ void next(const BkParams& p, long long start, long long end) {
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
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// The row tile's packed rows (row r = draft r / gq, query head h gq + r % gq;
// rows from R on are zero) into Q, as hi and lo terms, four times, and their
// score scales; by the softmax warps, eight rows each.
template <int D>
__device__ __forceinline__ void load_rows(const BkParams& p, const BSeg& s, unsigned char* smem, int warp, int lane) {
  constexpr int W = D / 64;  // 32-bit words of a row per lane
  const int a = __ldg(p.qo + s.b), e = __ldg(p.qo + s.b + 1);
  const bool ok = a >= 0 && e - a == p.L && static_cast<long long>(a) + p.L <= p.n_rows;
  const long long first = ok ? a : static_cast<long long>(s.b) * p.L;
  float* qsc = reinterpret_cast<float*>(smem + kQscOff);
  uint32_t v[8][W];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = static_cast<int>(blockIdx.y) * RT + 8 * warp + j;
    const bool live = r < p.R;
    const int rr = live ? r : 0;
    const __nv_bfloat16* src = p.q + (first + rr / p.gq) * p.q_s0 + static_cast<long long>(s.h * p.gq + rr % p.gq) * p.q_s1;
#pragma unroll
    for (int w = 0; w < W; ++w) v[j][w] = live ? ld_u32(src + 2 * (W * lane + w)) : 0u;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = 8 * warp + j;
    unsigned mx = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) mx = max(mx, mag_bf16x2(v[j][w]));
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (mx >= kBf16Inf) {
      // e4m3 has no infinity; an infinite query makes its row's softmax NaN, as NaN does
      mx = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        mx = max(mx, finite_mag_bf16x2(v[j][w]));
        v[j][w] = inf_to_nan_bf16x2(v[j][w]);
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
    }
    // the row's largest |q| 2^sh lies in [128, 256)
    const int sh = mx == 0 ? 0 : max(-120, min(120, 7 - (static_cast<int>(mx >> 7) - 127)));
    const float up = __int_as_float((127 + sh) << 23);
    if (lane == 0) qsc[row] = p.scale2 * __int_as_float((127 - sh) << 23);
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
      const int at = t * D + 2 * W * lane;  // byte of the row [hi | lo]
      unsigned char* d = smem + Geo<D>::q_off + (at >> 7) * (128 * 128) + row * 128 + ((((at & 127) >> 4) ^ (row & 7)) << 4) + (at & 15);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        unsigned char* dk = d + k * (32 * 128);
        if constexpr (W == 1)
          *reinterpret_cast<unsigned short*>(dk) = static_cast<unsigned short>(x[0]);
        else if constexpr (W == 2)
          *reinterpret_cast<uint32_t*>(dk) = x[0];
        else
          *reinterpret_cast<uint2*>(dk) = make_uint2(x[0], x[1]);
      }
    }
  }
}

}  // namespace bk

template <int D>
__global__ void __launch_bounds__(bk::kThreads, bk::Geo<D>::per_sm)
    block_stream_kernel(const __grid_constant__ bk::BkParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using namespace bk;
  using tc::idesc, tc::mbar_arrive, tc::mbar_init, tc::mma_commit, tc::mma_f8_ss, tc::fence_proxy_async;
  using tc::tc_fence_after, tc::tc_fence_before, tc::tmem_ld, tc::tmem_st, tc::tmem_wait_st;
  using G = bk::Geo<D>;
  constexpr int NS = G::NS, CB = G::CB, ENT = G::ENT;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // block_combine_kernel's CTAs may start (they wait for this grid themselves)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  long long start, end;
  BSeg seg0;
  if (!my_share(p, smem, start, end, seg0)) return;  // uniform
  if ((smem_u32(smem) & 1023u) != 0u) {  // the swizzled layouts need it; dynamic shared memory starts so
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  const uint32_t ring_s = smem_u32(smem + G::ring_off);
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(kBKFull + i), 2);  // the copies' bytes; the tile's scales
      mbar_init(bar(kBKEmpty + i), 1);
      mbar_init(bar(kBVFull + i), 1);
      mbar_init(bar(kBVEmpty + i), 1);
    }
    mbar_init(bar(kBSFull), 1);
    mbar_init(bar(kBSEmpty), 4);
    mbar_init(bar(kBPFull), 4);
    mbar_init(bar(kBPEmpty), 1);
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

  if (warp == 4) {
    // ================================ loader ================================
    float4* meta = reinterpret_cast<float4*>(smem + kMetaOff);
    BatchIt cur, ahead;
    // group `lane` of a batch: its first row in the cache, its keys, its scales
    auto fetch = [&](const BatchIt& it, int& row, int& keys, float& ks, float& vs) {
      row = 0;
      keys = 0;
      ks = vs = 1.f;
      const int gi = it.g + lane;
      if (!it.valid || gi >= it.ge) return;
      const int col = gi / p.bgroups;
      const long long page = __ldg(p.bt + static_cast<long long>(it.s.b) * p.bt_s0 + col);
      if (page < 0 || page >= p.n_blocks) {
        atomicOr(p.err, kErrBadIndex);
        return;
      }
      row = static_cast<int>(page * p.block) + (gi - col * p.bgroups) * GK;
      keys = min(GK, it.s.P - gi * GK);
      ks = __ldg(p.ks + page * p.ks_s0 + it.s.h);
      vs = __ldg(p.vs + page * p.vs_s0 + it.s.h);
    };
    cur.first(p, seg0, start, end);
    ahead = cur;
    int row, keys, row2, keys2;
    float ks, vs, ks2, vs2;
    fetch(cur, row, keys, ks, vs);
    uint32_t nk = 0, nv = 0;  // K and V tiles whose copies were issued
    uint32_t u = 0;
#pragma unroll 1
    while (cur.valid) {
      ahead.next(p, start, end);
      fetch(ahead, row2, keys2, ks2, vs2);
      const int tiles = (min(32, cur.ge - cur.g) + GT - 1) / GT;
#pragma unroll 1
      for (int j = 0; j < tiles; ++j, ++u) {
        const uint32_t st = u % NS, par = (u / NS) & 1u;
        const bool mine = (lane >> 3) == j;
        const unsigned there = __ballot_sync(0xffffffffu, mine && keys > 0);
        const bool lacks = __any_sync(0xffffffffu, mine && keys < GK);
        const uint32_t bytes = __popc(there) * (GK * D);
        const uint32_t kd = ring_s + st * (2 * ENT) + (lane & 7) * (GK * CB), vd = kd + ENT;
        if (fa::wait_all(bar(kBKEmpty + st), par ^ 1u, abort_flag, p.err)) {
          if (lane == 0) asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar(kBKFull + st)), "r"(bytes) : "memory");
          __syncwarp();
          if (mine && keys > 0)
#pragma unroll
            for (int c = 0; c < G::NB; ++c)
              fa::tma_load_box(kd + c * (KT * CB), &kmap, bar(kBKFull + st), c * CB, cur.s.h, row);
          nk = u + 1;
        }
        // the tile before the last kMeta's scales have been read: V of tile u - NS was multiplied after that
        if (fa::wait_all(bar(kBVEmpty + st), par ^ 1u, abort_flag, p.err)) {
          if (lane == 0) asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar(kBVFull + st)), "r"(bytes) : "memory");
          __syncwarp();
          if (mine && keys > 0)
#pragma unroll
            for (int c = 0; c < G::NB; ++c)
              fa::tma_load_box(vd + c * (KT * CB), &vmap, bar(kBVFull + st), c * CB, cur.s.h, row);
          nv = u + 1;
        }
        if (mine) {
          // a scale that is no positive finite number in the range gives NaN
          const bool good = ks >= kMinScale && ks <= kMaxScale && vs >= kMinScale && vs <= kMaxScale;
          if (!good) atomicOr(p.err, kErrBadScale);
          const float nan = __int_as_float(0x7FC00000);
          meta[(u % kMeta) * GT + (lane & 7)] =
              make_float4(good ? ks : nan, good ? log2f(vs) : nan, good ? 1.f / vs : nan, __int_as_float(keys + (lacks ? 256 : 0)));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBKFull + st));
      }
      cur = ahead;
      row = row2;
      keys = keys2;
      ks = ks2;
      vs = vs2;
    }
    // the copies end before the CTA does (in a CTA that gave up, nobody else waits for them)
    for (uint32_t k = 1; k <= NS; ++k) {
      if (k <= nk) fa::wait_last(bar(kBKFull + (nk - k) % NS), ((nk - k) / NS) & 1u);
      if (k <= nv) fa::wait_last(bar(kBVFull + (nv - k) % NS), ((nv - k) / NS) & 1u);
    }
  } else if (warp == 5) {
    // ================================ MMAs ================================
    constexpr uint32_t idS = idesc(0, 0, 0, 0, 128, KT), idO = idesc(0, 0, 0, 1, 128, D);
    const uint64_t dq = desc<128>(smem_u32(smem + G::q_off), 16, 1024), dp = desc<128>(smem_u32(smem + G::p_off), 16, 1024);
    const uint64_t dk = desc<CB>(ring_s, 16, 8 * CB), dv = desc<CB>(ring_s + ENT, KT * CB, 8 * CB);
    uint32_t u = 0, piece = 0;
    bool pending = false, pfirst = false;
    auto weigh = [&](uint32_t w, bool first) {  // O += P V of tile w
      const uint32_t st = w % NS;
      fa::wait_all(bar(kBPFull), w & 1u, abort_flag, p.err);
      fa::wait_all(bar(kBVFull + st), (w / NS) & 1u, abort_flag, p.err);
      tc_fence_after();
      if (fa::elect_one()) {
        const uint64_t vd = dv + static_cast<uint64_t>((st * (2 * ENT)) >> 4);
#pragma unroll
        for (int k = 0; k < KT / 32; ++k)
          mma_f8_ss(tO, dp + static_cast<uint64_t>(2 * k), vd + static_cast<uint64_t>((k * 32 * CB) >> 4), idO, !(first && k == 0));
        mma_commit(bar(kBPEmpty));
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
        fa::wait_all(bar(kBQFull), piece & 1u, abort_flag, p.err);
        ++piece;
#pragma unroll 1
        for (int g = g0; g < ge; g += GT, ++u) {
          const uint32_t st = u % NS;
          fa::wait_all(bar(kBKFull + st), (u / NS) & 1u, abort_flag, p.err);
          fa::wait_all(bar(kBSEmpty), (u & 1u) ^ 1u, abort_flag, p.err);
          tc_fence_after();
          if (fa::elect_one()) {
            const uint64_t kd = dk + static_cast<uint64_t>((st * (2 * ENT)) >> 4);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                const int qb = t * D + 32 * k, kb = 32 * k;
                mma_f8_ss(tS, dq + static_cast<uint64_t>(((qb >> 7) * (128 * 128) + (qb & 127)) >> 4),
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
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const float NEG_INF = -INFINITY;
    const float4* meta = reinterpret_cast<const float4*>(smem + kMetaOff);
    float* red = reinterpret_cast<float*>(smem + kRedOff);
    float* sums = reinterpret_cast<float*>(smem + kSumOff);
    const float* qscs = reinterpret_cast<const float*>(smem + kQscOff);
    uint32_t u = 0;
    BSeg s = seg0;
#pragma unroll 1
    for (; s.b < p.B && s.off < end; seg_next(p, s)) {
      int g0, ge;
      piece_of(s, start, end, g0, ge);
      const long long slot = blockIdx.x + static_cast<long long>(s.b) * p.h_kv + s.h;
      const int row0 = static_cast<int>(blockIdx.y) * RT;
      float* lse_p = p.plse + slot * p.rows + row0;
      float* o_p = p.po + (slot * p.rows + row0) * D;
      const int live = min(RT, p.R - row0);
      if (g0 >= ge) {  // no key: an empty partial
        if (tid < live) lse_p[tid] = NEG_INF;
        continue;
      }
      load_rows<D>(p, s, smem, warp, lane);
      fence_proxy_async();
      named_bar_sync(1, kSm);  // the rows' scales
      if (lane == 0) mbar_arrive(bar(kBQFull));
      const float qsc = qscs[lane];
      float m = NEG_INF, l = 0.f;
#pragma unroll 1
      for (int g = g0; g < ge; g += GT, ++u) {
        fa::wait_all(bar(kBSFull), u & 1u, abort_flag, p.err);
        tc_fence_after();
        float x[32];
        tmem_ld<32>(tS + lanes + 32 * warp, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBSEmpty));
        const float4 me[2] = {meta[(u % kMeta) * GT + 2 * warp], meta[(u % kMeta) * GT + 2 * warp + 1]};
        float tm = NEG_INF;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float c = qsc * me[h].x;
#pragma unroll
          for (int i = 0; i < 16; ++i) x[16 * h + i] = fmaf(x[16 * h + i], c, me[h].y);
        }
        const bool lacks = __float_as_int(me[0].w) >= 256;
        if (lacks) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int keys = __float_as_int(me[h].w) & 255;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i >= keys) x[16 * h + i] = NEG_INF;
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) tm = fmaxf(tm, x[i]);
        float* rd = red + (u & 1) * 128;
        rd[tid] = tm;
        named_bar_sync(1, kSm);
        tm = fmaxf(fmaxf(rd[lane], rd[32 + lane]), fmaxf(rd[64 + lane], rd[96 + lane]));  // alike in the four warps
        // P and O are free once the tile before is weighed
        if (g > g0) {
          fa::wait_all(bar(kBPEmpty), (u & 1u) ^ 1u, abort_flag, p.err);
          tc_fence_after();
        }
        if (__any_sync(0xffffffffu, tm > m + kThr)) {
          const float mn = fmaxf(m, tm);
          const float al = mn == NEG_INF ? 1.f : fast_exp2(m - mn);
          if (g > g0 && warp < 3) {
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
          l *= al;
          m = mn;
        }
        const float up = m == NEG_INF ? 0.f : static_cast<float>(kUp) - m;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sum = 0.f;
          uint32_t w[3][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float t[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = fast_exp2(x[16 * h + 4 * i + e] + up);
              sum += y;
              // the top 4 bits where e4m3 has them all (2^-6 and above), and what they leave
              const float a = y < 0.015625f ? 0.f : __uint_as_float(__float_as_uint(y) & 0xFFF00000u);
              const float z = (y - a) * 16.f;
              const float b = z < 0.015625f ? 0.f : __uint_as_float(__float_as_uint(z) & 0xFFF00000u);
              t[0][e] = a;
              t[1][e] = b;
              t[2][e] = (z - b) * 16.f;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) w[k][i] = e4m3x4(t[k][0], t[k][1], t[k][2], t[k][3]);
          }
          l = fmaf(sum, me[h].z, l);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint4*>(smem + G::p_off + (32 * k + lane) * 128 + (((2 * warp + h) ^ (lane & 7)) << 4)) =
                make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
        }
        if (lacks) {
          // V rows of keys that are not there: 0 times what lies there may be NaN
          const uint32_t st = u % NS;
          fa::wait_all(bar(kBVFull + st), (u / NS) & 1u, abort_flag, p.err);
          if ((tid & 15) >= (__float_as_int(meta[(u % kMeta) * GT + (tid >> 4)].w) & 255)) {
            unsigned char* v = smem + G::ring_off + st * (2 * ENT) + ENT + tid * CB;
#pragma unroll
            for (int c = 0; c < G::NB; ++c)
#pragma unroll
              for (int i = 0; i < CB; i += 16) *reinterpret_cast<uint4*>(v + c * (KT * CB) + i) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBPFull));
      }
      // ---- the piece's partial: o = sum of the terms / l, log2 of the sum ----
      sums[tid] = l;
      fa::wait_all(bar(kBPEmpty), (u & 1u) ^ 1u, abort_flag, p.err);
      tc_fence_after();
      unsigned char* stage = smem + G::p_off;  // [3 terms][32 rows][32 columns], P is free
      const int row = tid >> 2, quarter = tid & 3;
      named_bar_sync(1, kSm);
      const float lr = (sums[row] + sums[32 + row]) + (sums[64 + row] + sums[96 + row]);
      const float inv = lr == 0.f ? 0.f : 1.f / lr;
      if (warp == 0 && lane < live) {
        const float la = (sums[lane] + sums[32 + lane]) + (sums[64 + lane] + sums[96 + lane]);
        lse_p[lane] = la == 0.f ? NEG_INF : m + (log2f(la) - static_cast<float>(kUp));
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        if (warp < 3) {
          float o[32];
          tmem_ld<32>(tO + lanes + c, o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(stage + (warp * 32 + lane) * 128 + ((i ^ (lane & 7)) << 4)) =
                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        named_bar_sync(1, kSm);
        if (row < live) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const unsigned char* at = stage + row * 128 + (((2 * quarter + i) ^ (row & 7)) << 4);
            const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + 4096),
                         d = *reinterpret_cast<const float4*>(at + 8192);
            float4 r;
            r.x = fmaf(d.x, 0.00390625f, fmaf(b.x, 0.0625f, a.x)) * inv;
            r.y = fmaf(d.y, 0.00390625f, fmaf(b.y, 0.0625f, a.y)) * inv;
            r.z = fmaf(d.z, 0.00390625f, fmaf(b.z, 0.0625f, a.z)) * inv;
            r.w = fmaf(d.w, 0.00390625f, fmaf(b.w, 0.0625f, a.w)) * inv;
            *reinterpret_cast<float4*>(o_p + row * D + c + 8 * quarter + 4 * i) = r;
          }
        }
        named_bar_sync(1, kSm);
      }
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

bk::BkFn kernel_block_stream_64();
bk::BkFn kernel_block_stream_128();
bk::BkFn kernel_block_stream_256();
bk::BkJoinFn kernel_block_combine_64();
bk::BkJoinFn kernel_block_combine_128();
bk::BkJoinFn kernel_block_combine_256();

}  // namespace vsk
