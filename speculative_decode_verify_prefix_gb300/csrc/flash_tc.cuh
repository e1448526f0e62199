// Attention of many query rows over many keys on the tensor cores (tcgen05,
// accumulators in tensor memory), for two calls:
//   prompt_attn_fwd            whole prompts, causal, K / V rows contiguous
//   verify_splitkv_shared_fwd  every draft row of a batch over the prefix its
//                              sequences share, K / V rows gathered from the pool
//
// Mathematics.  Per query row, one pass over the keys in tiles of 128 with a
// running reference m and sum l (base 2, x = score * sm_scale * log2 e):
//   P = 2^(x - m),  l += sum P,  O += P V,   o = O / l
// m is raised (and O, l scaled by 2^(m_old - m_new)) only when a tile's maximum
// exceeds it by more than 8: until then P stays below 2^8, far from any
// limit of the 32-bit sums, and O in tensor memory need not be touched.
// Scores, m, l and O are 32-bit; P is rounded to bf16 because both operands of
// an MMA have one type and V is bf16 (relative error 2^-9, of the order of the
// output's own rounding; l sums the unrounded P).
//
// Rows.  The g = h_q / h_kv query heads of a KV head share its keys, so the
// packed row r of a query tile is (token r / g, head r % g): a 128-row tile
// holds 128 / g tokens (rounded down; spare rows are zero and never stored).  A
// CTA owns one block of NQ tiles of one KV head: two at head_dim 64 / 128
// (every K / V tile in shared memory feeds both, and the tensor core works on
// one tile while the softmax of the other runs), one at 256, whose O takes
// half of the 512 tensor-memory columns and whose scores are double-buffered
// instead.
//
// What bounds it: per 128-key tile and query tile 2 MMAs of 128 x 128 x D
// against 16,384 exponentials; both pipes are busy at once.
//
// Roles (16 warps; registers redistributed with setmaxnreg):
//   warps 0-3, 4-7   softmax of query tile 0 / 1 (thread = row; at head_dim 256
//                    warps 4-7 are idle): scores from tensor memory, P back
//                    over them (bf16, half the columns), rescale, epilogue
//   warp 8           issues the MMAs (one elected lane): S = Q K^T (both operands in
//                    shared memory), O += P V (P in tensor memory)
//   warps 12-15      bring K / V rows into a ring of 128-key entries (128 head
//                    dimensions each, K then V of a tile): contiguous rows by
//                    TMA, gathered ones with 16-byte cp.async; e4m3 rows are
//                    widened to bf16 (exact) in registers
// S of the next tile is issued behind PV of this one: the issuing order makes
// the overwrite of P by S safe.
//
// Shared memory operands are in the 128-byte swizzled canonical layouts, [64
// head-dim block][row][128 B]: Q and K K-major, V MN-major.
//
// Masked keys.  A key beyond the sequence, or with a bad index, is zero in
// shared memory, and its score is replaced by -inf, so nothing that sits in
// such rows reaches the result.  In a causal tile V rows that later tokens own
// are multiplied by P = 0, which is NaN for an infinite or NaN value: the
// loaders zero such values in the tiles on the diagonal and flag them, and the
// epilogue adds them to the rows that do see them.
//
// Every mbarrier wait is bounded (one second): a wait that gives up sets error
// bit 8 and the CTA drains, frees its tensor memory and exits.
#pragma once
#include <cuda.h>

#include "verify_kernel.cuh"
#include "verify_tr.cuh"

namespace vsk {
namespace fa {

using tc::cp_async_arrive_noinc;
using tc::fence_proxy_async;
using tc::idesc;
using tc::mbar_arrive;
using tc::mbar_init;
using tc::mma_commit;
using tc::mma_f16_ss;
using tc::sdesc;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_ld;
using tc::tmem_st;
using tc::tmem_wait_st;

constexpr int KT = 128;          // keys per tile
constexpr int kThreads = 512;
constexpr int kWarpMma = 8;
constexpr int kWarpLoad = 12;    // loader warps 12-15
constexpr int kLoadThreads = 128;
constexpr int kRegsSoftmax = 184, kRegsOther = 72;
static_assert(8 * 32 * (kRegsSoftmax + kRegsOther) <= 65536, "register shares exceed the launch's");
constexpr float kThr = 8.f;      // log2 headroom before the running reference is raised
constexpr int kMaxNE = 8;        // ring entries at most
constexpr int kMaskRing = 8;     // > the tiles loaders can run ahead of the softmax

enum Mode { kPrompt = 0, kSharedBf16 = 1, kSharedE4m3 = 2 };

// shared-memory map
constexpr int kBarOff = 0;
constexpr int kTmemOff = 512, kAbortOff = 516, kBadVOff = 520, kWorkOff = 528;  // kWorkOff: 4 x i32
constexpr int kMaskOff = 1024;   // [kMaskRing][4] key-validity words
constexpr int kDataOff = 2048;
// barriers
constexpr int kBFull = 0, kBEmpty = kMaxNE, kBQFull = 2 * kMaxNE, kBSFull = kBQFull + 2, kBPFull = kBSFull + 2,
              kBOFull = kBPFull + 4, kBMask = kBOFull + 2, kBDone = kBMask + kMaskRing, kNumBars = kBDone + 1;
static_assert(kBarOff + 8 * kNumBars <= kTmemOff, "barriers overlap");

template <int D>
struct Geo {
  static constexpr int NQ = D == 256 ? 1 : 2;      // query tiles per CTA
  static constexpr int ED = D < 128 ? D : 128;     // head dimensions of a ring entry
  static constexpr int NH = D / ED;                // entries of a K (or V) tile
  static constexpr int ENT = KT * ED * 2;
  static constexpr int QT = 128 * D * 2;           // one query tile
  static constexpr int NE = D == 64 ? 8 : 5;
  static constexpr int q_off = kDataOff;
  static constexpr int ring_off = q_off + NQ * QT;
  static constexpr int smem = ring_off + NE * ENT;
  static constexpr int col_o = 256;                // TMEM: S buffers at 0 and 128, O tile t at 256 + t D
  static_assert(smem <= 227 * 1024, "fits an SM");
  static_assert(2 * NH + 1 <= NE, "a tile's V and the next tile's K are held together");
};

struct FaParams {
  const __nv_bfloat16* q; long long q_s0, q_s1;
  const unsigned char* k; long long k_s0, k_s1;  // byte strides
  const unsigned char* v; long long v_s0, v_s1;
  __nv_bfloat16* o;       long long o_s0, o_s1;
  const int* qo;          // prompt: [B + 1]
  int B;
  long long n_rows;       // query rows (tokens)
  const void* idx;        // shared: pool rows of the keys
  int idx64;
  long long n_keys, pool;
  int h_kv, gq, tpb;      // tpb: tokens per query tile
  int n_split, split_tiles;  // shared: key ranges per row block, key tiles of one
  float scale2;           // > 0
  int qmode;              // queries enter as they are (0), negated (1) or as zeros (2): the sign of the scale
  int q16, o16;           // 16-byte accesses allowed
  int tma;                // prompt: K / V tiles come through the tensor maps
  float v_scale;
  unsigned* err;
  float* plse;            // shared: partials, one row block of NQ * 128 rows per CTA
  float* po;
};

using FaFn = void (*)(const FaParams, const CUtensorMap, const CUtensorMap);

// The MMA warp runs its loop converged; one elected lane issues each group of
// MMAs.  Addresses and descriptors are then the same for the whole warp and stay
// in uniform registers (in a branch of one lane around the whole loop every MMA
// first moves them there: 140 cycles an MMA instead of 64).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem, uint32_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          tmem),
      "r"(a), "l"(b), "r"(id), "r"(acc ? 1 : 0));
}

// 32 lanes x 32 columns, without the wait
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// wait for this thread's tcgen05.ld; the registers pass through so that no use
// of them can be scheduled before it
__device__ __forceinline__ void tmem_pass(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// 16-byte global -> shared copy through L2 only, zeros when !valid
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

// Two 32-bit operations in one instruction; the larger of three.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One [32 rows][64 head dimensions] box of a K / V tensor map into shared memory.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int head, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(bar), "r"(x), "r"(head), "r"(row)
      : "memory");
}
// A warp's 32 arrivals by one lane: 31, and one that also announces the bytes
// its copies will bring.
__device__ __forceinline__ void mbar_arrive_warp_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 31;" ::"r"(bar) : "memory");
}

// bf16 pair with infinities and NaN replaced by 0; bad: whether there were any
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w, bool& bad) {
  const bool lo = (w & 0x7F80u) == 0x7F80u, hi = (w & 0x7F800000u) == 0x7F800000u;
  bad |= lo | hi;
  return w & (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
}

}  // namespace fa

template <int D, int MODE>
__global__ void __launch_bounds__(fa::kThreads, 1) fa_kernel(const __grid_constant__ fa::FaParams p,
                                                             const __grid_constant__ CUtensorMap kmap,
                                                             const __grid_constant__ CUtensorMap vmap) {
  using namespace fa;
  using G = fa::Geo<D>;
  constexpr int NQ = G::NQ, NH = G::NH, NE = G::NE, ENT = G::ENT;
  constexpr bool PROMPT = MODE == kPrompt;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
  const float NEG_INF = -INFINITY;

  // ---- this CTA's work: row block (tokens [tok0, tok0 + NQ tpb) of rows [row0, row0 + n)), KV head, key tiles ----
  int* work = reinterpret_cast<int*>(smem + kWorkOff);
  const int bt = NQ * p.tpb;
  int head, split = 0;
  if constexpr (PROMPT) {
    head = static_cast<int>(blockIdx.x % p.h_kv);
    if (warp == 0) {
      // the sequence that holds row block blockIdx.x / h_kv: blocks are
      // numbered sequence by sequence, the last block of a sequence (its
      // longest key range) first
      long long want = blockIdx.x / p.h_kv;
      int found = -1, n_f = 0, a_f = 0, blk_f = 0;
      for (int b0 = 0; b0 < p.B && found < 0; b0 += 32) {
        const int b = b0 + lane;
        int a = 0, n = 0;
        if (b < p.B) {
          a = __ldg(p.qo + b);
          const int e = __ldg(p.qo + b + 1);
          n = (a >= 0 && e >= a && e <= p.n_rows) ? e - a : 0;
        }
        const int nb = n / bt + (n % bt != 0);
        int incl = nb;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += y;
        }
        const bool here = want >= incl - nb && want < incl;
        const unsigned m = __ballot_sync(0xffffffffu, here);
        if (m) {
          const int src = __ffs(m) - 1;
          found = b0 + src;
          n_f = __shfl_sync(0xffffffffu, n, src);
          a_f = __shfl_sync(0xffffffffu, a, src);
          const int last = __shfl_sync(0xffffffffu, incl, src) - 1;
          blk_f = last - static_cast<int>(want);
        } else {
          want -= __shfl_sync(0xffffffffu, incl, 31);
        }
      }
      if (lane == 0) {
        work[0] = found;
        work[1] = a_f;
        work[2] = n_f;
        work[3] = blk_f;
      }
    }
    if (blockIdx.x == 0 && warp == 1) {
      for (int b = lane; b < p.B; b += 32) {
        const int a = __ldg(p.qo + b), e = __ldg(p.qo + b + 1);
        if (!(a >= 0 && e >= a && e <= p.n_rows)) atomicOr(p.err, kErrBadQoIndptr);
      }
    }
    __syncthreads();
    if (work[0] < 0) return;  // uniform: the grid is an upper bound
  }
  long long row0;
  int n, tok0, j_first, n_tiles[2];
  if constexpr (PROMPT) {
    row0 = work[1];
    n = work[2];
    tok0 = work[3] * bt;
    j_first = 0;
  } else {
    split = static_cast<int>(blockIdx.x % p.n_split);
    const int u = static_cast<int>(blockIdx.x / p.n_split);
    head = u % p.h_kv;
    row0 = 0;
    n = static_cast<int>(p.n_rows);
    tok0 = (u / p.h_kv) * bt;
    j_first = split * p.split_tiles;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = tok0 + t * p.tpb;
    if (t >= NQ || first >= n) {
      n_tiles[t] = 0;
    } else if constexpr (PROMPT) {
      n_tiles[t] = (min(first + p.tpb, n) + KT - 1) / KT;
    } else {
      const long long tiles = (p.n_keys + KT - 1) / KT;
      n_tiles[t] = static_cast<int>(max(0LL, min(static_cast<long long>(p.split_tiles), tiles - j_first)));
    }
  }
  const int nt = max(n_tiles[0], n_tiles[1]);
  const int j_edge = PROMPT ? tok0 / KT : 0;  // prompt: first tile that holds keys some row of the block must not see

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  volatile int* bad_v = reinterpret_cast<volatile int*>(smem + kBadVOff);
  volatile unsigned* maskw = reinterpret_cast<volatile unsigned*>(smem + kMaskOff);
  const uint32_t q_s = smem_u32(smem + G::q_off), ring_s = smem_u32(smem + G::ring_off);
  if ((smem_u32(smem) & 1023u) != 0u) {  // the swizzled layouts need it; uniform
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    *bad_v = 0;
    for (int i = 0; i < NE; ++i) {
      mbar_init(bar(kBFull + i), kLoadThreads);
      mbar_init(bar(kBEmpty + i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kBQFull + t), 4);
      mbar_init(bar(kBSFull + t), 1);
      mbar_init(bar(kBPFull + 2 * t), 4);
      mbar_init(bar(kBPFull + 2 * t + 1), 4);
      mbar_init(bar(kBOFull + t), 1);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(bar(kBMask + i), 4);
    mbar_init(bar(kBDone), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem + kTmemOff)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kTmemOff);

  if (warp < 4 * NQ) {
    // ================================ softmax ================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, w = warp & 3, tw = tid & 127;
    const int first = tok0 + t * p.tpb;  // first token of the tile
    const int my_tiles = n_tiles[t];
    // ---- queries of the tile into shared memory ----
    {
      constexpr int CPR = D / 8;  // 16-byte chunks of a row
      unsigned char* qs = smem + G::q_off + t * G::QT;
#pragma unroll 4
      for (int i = 0; i < CPR; ++i) {
        const int ci = tw + 128 * i, r = ci / CPR, c = ci % CPR;
        const int tok = first + r / p.gq, g = r % p.gq;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < p.tpb * p.gq && tok < n && p.qmode != 2) {
          const __nv_bfloat16* src =
              p.q + (row0 + tok) * p.q_s0 + static_cast<long long>(head * p.gq + g) * p.q_s1 + c * 8;
          if (p.q16)
            x = __ldg(reinterpret_cast<const uint4*>(src));
          else
            x = make_uint4(ld_u32(src), ld_u32(src + 2), ld_u32(src + 4), ld_u32(src + 6));
          if (p.qmode == 1) {
            x.x ^= 0x80008000u;
            x.y ^= 0x80008000u;
            x.z ^= 0x80008000u;
            x.w ^= 0x80008000u;
          }
        }
        *reinterpret_cast<uint4*>(qs + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBQFull + t));
    }
    const int r = 32 * w + lane;  // this thread's packed row
    const int tok = min(first + r / p.gq, n - 1);
    const bool real = r < p.tpb * p.gq && first + r / p.gq < n;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * w) << 16);
    const uint32_t t_o = t_lane + G::col_o + t * D;
    const float sc = p.scale2;
    float mrun = NEG_INF, l = 0.f;
#pragma unroll 1
    for (int j = 0; j < my_tiles; ++j) {
      const int buf = NQ == 2 ? t : (j & 1);
      const uint32_t par = NQ == 2 ? (j & 1) : ((j >> 1) & 1);
      const uint32_t t_s = t_lane + buf * KT;
      tr::wait_warp(bar(kBSFull + buf), par, abort_flag, p.err);
      tc_fence_after();
      // Scores, then P, in halves of 64 keys: the second half is on its way
      // while the first one's maximum is taken, and the first half of P is
      // handed to the MMAs while the second is computed.
      uint32_t s[KT];
      bool masked;
      unsigned mw[4];
      if constexpr (PROMPT) {
        masked = (j + 1) * KT - 1 > first;
        const int lim = tok - j * KT;  // keys c <= lim are visible
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int n_vis = min(32, max(0, lim + 1 - 32 * u));
          mw[u] = n_vis == 32 ? 0xFFFFFFFFu : (1u << n_vis) - 1u;
        }
      } else {
        const int jm = j % kMaskRing;
        tr::wait_warp(bar(kBMask + jm), static_cast<uint32_t>((j / kMaskRing) & 1), abort_flag, p.err);
#pragma unroll
        for (int u = 0; u < 4; ++u) mw[u] = maskw[4 * jm + u];
        masked = (mw[0] & mw[1] & mw[2] & mw[3]) != 0xFFFFFFFFu;
      }
      float mx[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 0) {
          tmem_ld32_nw(t_s, s);
          tmem_ld32_nw(t_s + 32, s + 32);
        }
        tmem_wait_ld();
        tmem_pass(s + 64 * h);
        tmem_pass(s + 64 * h + 32);
        if (h == 0) {
          tmem_ld32_nw(t_s + 64, s + 64);
          tmem_ld32_nw(t_s + 96, s + 96);
        }
        if (masked) {  // -inf for masked keys
#pragma unroll
          for (int c = 64 * h; c < 64 * h + 64; ++c)
            s[c] = ((mw[c >> 5] >> (c & 31)) & 1u) ? s[c] : __float_as_uint(NEG_INF);
        }
#pragma unroll
        for (int c = 64 * h; c < 64 * h + 64; c += 2)
          mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
      }
      // ---- raise the reference when the tile's maximum passes it by more than kThr ----
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
      if (__any_sync(0xffffffffu, mt > mrun + kThr)) {
        const float mn = fmaxf(mrun, mt);
        const float al = mn == NEG_INF ? 1.f : fast_exp2(mrun - mn);
        if (j > 0) {
          tr::wait_warp(bar(kBOFull + t), static_cast<uint32_t>((j - 1) & 1), abort_flag, p.err);
          tc_fence_after();
#pragma unroll 1
          for (int cb = 0; cb < D / 8; ++cb) {
            float o[8];
            tmem_ld<8>(t_o + 8 * cb, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= al;
            tmem_st<8>(t_o + 8 * cb, o);
          }
        }
        l *= al;
        mrun = mn;
      }
      const float mref = mrun == NEG_INF ? 0.f : mrun;
      // ---- P over the scores' columns ----
      const float2 sc2 = make_float2(sc, sc), mn2 = make_float2(-mref, -mref);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int c = 64 * h + 2 * i;
          const float2 x = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, mn2);
          const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
          pk[i] = pack_bf16(p0, p1);
          s[c] = __float_as_uint(p0);
          s[c + 1] = __float_as_uint(p1);
        }
        tmem_st32(t_s + 32 * h, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBPFull + 2 * buf + h));
      }
      // ---- the row's sum, off the MMAs' way ----
      float2 l4[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int i = 0; i < KT / 2; ++i)
        l4[i & 3] = add2(l4[i & 3], make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])));
      l4[0] = add2(add2(l4[0], l4[1]), add2(l4[2], l4[3]));
      l += l4[0].x + l4[0].y;
    }
    // ---- epilogue ----
    if (my_tiles > 0) {
      // one query tile: the last scores are issued before the PV of the tile
      // before, so that phase has to be seen to complete first
      if (NQ == 1 && my_tiles > 1)
        tr::wait_warp(bar(kBOFull + t), static_cast<uint32_t>((my_tiles - 2) & 1), abort_flag, p.err);
      tr::wait_warp(bar(kBOFull + t), static_cast<uint32_t>((my_tiles - 1) & 1), abort_flag, p.err);
      tc_fence_after();
    }
    if constexpr (PROMPT) {
      named_bar_sync(1, kLoadThreads + 128 * NQ);  // the loaders are done: bad_v is final
      if (my_tiles > 0) {
        const float inv = 1.f / l;
        const bool fix = *bad_v != 0;
        __nv_bfloat16* orow =
            p.o + (row0 + tok) * p.o_s0 + static_cast<long long>(head * p.gq + r % p.gq) * p.o_s1;
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          float o[32];
          tmem_ld<32>(t_o + 32 * cb, o);
          if (!real) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= inv;
          if (fix) {
            // values the loaders zeroed, for the rows that see them
            for (int key = j_edge * KT; key <= tok; ++key) {
              const uint32_t* vr = reinterpret_cast<const uint32_t*>(
                  p.v + (row0 + key) * p.v_s0 + head * p.v_s1 + cb * 64);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t x = __ldg(vr + i);
                const float2 f = unpack_bf16(x);
                if ((x & 0x7F80u) == 0x7F80u) o[2 * i] += f.x;
                if ((x & 0x7F800000u) == 0x7F800000u) o[2 * i + 1] += f.y;
              }
            }
          }
          uint32_t y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
          uint32_t* dst = reinterpret_cast<uint32_t*>(orow + 32 * cb);
          if (p.o16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4*>(dst)[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[i] = y[i];
          }
        }
      }
    } else if (my_tiles > 0) {
      // partial of this key range: o v_scale / l and m + log2 l, -inf and 0 where no key was valid
      const long long prow = static_cast<long long>(blockIdx.x) * (NQ * 128) + t * 128 + r;
      const float inv = l > 0.f ? p.v_scale / l : 0.f;
      if (real) p.plse[prow] = l > 0.f ? mrun + log2f(l) : (l == 0.f ? NEG_INF : l);
      float* orow = p.po + prow * D;
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        float o[32];
        tmem_ld<32>(t_o + 32 * cb, o);
        if (!real) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(orow + 32 * cb + 4 * i) =
              make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
      }
    }
    tc_fence_before();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp >= kWarpMma) {
      if (warp == kWarpMma) {
        // ============================ MMA issue ============================
        constexpr uint32_t idS = idesc(1, 1, 0, 0, 128, KT);
        constexpr uint32_t idPV = idesc(1, 1, 0, 1, 128, G::ED);
        const uint64_t dq0 = sdesc(q_s, 16, 1024), dk0 = sdesc(ring_s, 16, 1024), dv0 = sdesc(ring_s, KT * 128, 1024);
        // entry of (tile j, K / V, half h): (2 j + kv) NH + h
        auto wait_full = [&](int e) {
          tr::wait_warp(bar(kBFull + e % NE), static_cast<uint32_t>((e / NE) & 1), abort_flag, p.err);
        };
        auto qk = [&](int t, int j) {
          const uint32_t dc = tmem + (NQ == 2 ? t : (j & 1)) * KT;
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const int slot = (2 * j * NH + h) % NE;
            const uint64_t qd = dq0 + static_cast<uint64_t>((t * G::QT + h * 2 * (128 * 128)) >> 4);
            const uint64_t kd = dk0 + static_cast<uint64_t>((slot * ENT) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < G::ED / 16; ++ks) {
                const uint64_t off = static_cast<uint64_t>(((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4);
                mma_f16_ss(dc, qd + off, kd + off, idS, h > 0 || ks > 0);
              }
            }
          }
          if (elect_one()) mma_commit(bar(kBSFull + (NQ == 2 ? t : (j & 1))));
        };
        auto pv = [&](int t, int j) {
          const int buf = NQ == 2 ? t : (j & 1);
          const uint32_t par = static_cast<uint32_t>(NQ == 2 ? (j & 1) : ((j >> 1) & 1));
          const uint32_t a = tmem + buf * KT;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            tr::wait_warp(bar(kBPFull + 2 * buf + half), par, abort_flag, p.err);
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              const int slot = ((2 * j + 1) * NH + h) % NE;
              const uint64_t vd = dv0 + static_cast<uint64_t>((slot * ENT) >> 4);
              if (elect_one()) {
#pragma unroll
                for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                  mma_f16_ts(tmem + G::col_o + t * D + h * G::ED, a + ks * 8, vd + static_cast<uint64_t>(ks * 128),
                             idPV, j > 0 || ks > 0);
              }
            }
          }
          if (elect_one()) mma_commit(bar(kBOFull + t));
        };
        auto acquire = [&](int j, int kv) {
#pragma unroll
          for (int h = 0; h < NH; ++h) wait_full((2 * j + kv) * NH + h);
          // rows that came by cp.async (stores and TMA need none here)
          if (MODE == kSharedBf16 || (PROMPT && !p.tma)) fence_proxy_async();
          tc_fence_after();
        };
        auto release = [&](int j, int kv) {
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (elect_one()) mma_commit(bar(kBEmpty + ((2 * j + kv) * NH + h) % NE));
        };
        if (nt > 0) {
#pragma unroll
          for (int t = 0; t < NQ; ++t) tr::wait_warp(bar(kBQFull + t), 0u, abort_flag, p.err);
          acquire(0, 0);
#pragma unroll
          for (int t = 0; t < NQ; ++t)
            if (n_tiles[t] > 0) qk(t, 0);
          release(0, 0);
          for (int j = 0; j < nt; ++j) {
            if constexpr (NQ == 1) {
              if (j + 1 < nt) {
                acquire(j + 1, 0);
                qk(0, j + 1);
                release(j + 1, 0);
              }
              acquire(j, 1);
              pv(0, j);
              release(j, 1);
            } else {
              acquire(j, 1);
#pragma unroll
              for (int t = 0; t < NQ; ++t) {
                if (j < n_tiles[t]) pv(t, j);
                if (t == NQ - 1) release(j, 1);
                if (j + 1 < nt && t == 0) acquire(j + 1, 0);
                if (j + 1 < n_tiles[t]) qk(t, j + 1);
                if (t == NQ - 1 && j + 1 < nt) release(j + 1, 0);
              }
            }
          }
        }
        if (elect_one()) mma_commit(bar(kBDone));
        tr::wait_warp(bar(kBDone), 0u, abort_flag, p.err);  // no arrival is pending when the CTA exits
      } else if (warp >= kWarpLoad) {
        // ================================ loaders ================================
        const int lw = warp - kWarpLoad;
        constexpr int CPK = G::ED / 8;        // 16-byte chunks of an entry's bf16 row
        constexpr int RPP = 32 / CPK;         // rows of a warp's pass
        constexpr int NP = 32 / RPP;          // passes over a warp's 32 rows
        const int cc = lane % CPK, rr = lane / CPK;
        auto slot_wait = [&](int e) {
          tr::wait_warp(bar(kBEmpty + e % NE), static_cast<uint32_t>(((e / NE) & 1) ^ 1), abort_flag, p.err);
        };
        auto dst_off = [&](int key, int c) -> uint32_t {
          return static_cast<uint32_t>((c >> 3) * (KT * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4));
        };
        auto load_idx = [&](int j) -> long long {
          const long long at = static_cast<long long>(j_first + j) * KT + 32 * lw + lane;
          if (j >= nt || at >= p.n_keys) return -2;
          return p.idx64 ? __ldg(static_cast<const long long*>(p.idx) + at)
                         : static_cast<long long>(__ldg(static_cast<const int*>(p.idx) + at));
        };
        long long loc_next = 0;
        if constexpr (!PROMPT) loc_next = load_idx(0);
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
          long long loc = 0;
          unsigned ok_mask = 0u;
          if constexpr (PROMPT) {
            loc = row0 + static_cast<long long>(j) * KT + 32 * lw + lane;
            ok_mask = __ballot_sync(0xffffffffu, j * KT + 32 * lw + lane < n);
          } else {
            loc = loc_next;
            loc_next = load_idx(j + 1);
            const bool ok = loc >= 0 && loc < p.pool;
            if (!ok && loc != -2) atomicOr(p.err, kErrBadIndex);
            ok_mask = __ballot_sync(0xffffffffu, ok);
          }
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const unsigned char* base = kv ? p.v + head * p.v_s1 : p.k + head * p.k_s1;
            const long long s0 = kv ? p.v_s0 : p.k_s0;
#pragma unroll 1
            for (int h = 0; h < NH; ++h) {
              const int e = (2 * j + kv) * NH + h;
              unsigned char* ent = smem + G::ring_off + (e % NE) * ENT;
              slot_wait(e);
              if (!PROMPT && kv == 0 && h == 0 && lane == 0) {
                maskw[4 * (j % kMaskRing) + lw] = ok_mask;
                mbar_arrive(bar(kBMask + j % kMaskRing));
              }
              if constexpr (MODE == kSharedE4m3) {
                // 16 e4m3 values a lane, two 16-byte bf16 chunks
                constexpr int LPR = CPK / 2, RP8 = 32 / LPR, NP8 = 32 / RP8;
                const int c8 = lane % LPR, r8 = lane / LPR;
                uint4 x[NP8];
#pragma unroll
                for (int i = 0; i < NP8; ++i) {
                  const int kl = i * RP8 + r8;
                  const long long lc = __shfl_sync(0xffffffffu, loc, kl);
                  x[i] = ((ok_mask >> kl) & 1u)
                             ? __ldg(reinterpret_cast<const uint4*>(base + lc * s0 + h * G::ED + c8 * 16))
                             : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < NP8; ++i) {
                  const int key = 32 * lw + i * RP8 + r8;
                  const uint32_t wv[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                  uint32_t y[8];
#pragma unroll
                  for (int u = 0; u < 4; ++u) {
                    y[2 * u] = e4m3x2_to_bf16x2(static_cast<unsigned short>(wv[u] & 0xFFFFu));
                    y[2 * u + 1] = e4m3x2_to_bf16x2(static_cast<unsigned short>(wv[u] >> 16));
                  }
                  *reinterpret_cast<uint4*>(ent + dst_off(key, 2 * c8)) = make_uint4(y[0], y[1], y[2], y[3]);
                  *reinterpret_cast<uint4*>(ent + dst_off(key, 2 * c8 + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
                }
                fence_proxy_async();
                mbar_arrive(bar(kBFull + e % NE));
              } else if (PROMPT && p.tma && (kv == 0 || j < j_edge)) {
                // keys past the sequence may come along: their scores are masked,
                // and V tiles that hold any take the next branch
                if (lane == 0) {
                  const uint32_t d0 = smem_u32(ent) + 32 * lw * 128, fb = bar(kBFull + e % NE);
                  mbar_arrive_warp_tx(fb, 32 * G::ED * 2);
#pragma unroll
                  for (int cb = 0; cb < G::ED / 64; ++cb)
                    tma_load_box(d0 + cb * (KT * 128), kv ? &vmap : &kmap, fb, h * G::ED + cb * 64, head,
                                 static_cast<int>(row0) + j * KT + 32 * lw);
                }
                __syncwarp();
              } else if (PROMPT && kv == 1 && j >= j_edge) {
                // V on the diagonal: values that are not finite become 0 here
                // and are added by the epilogue to the rows that see them
                bool bad = false;
#pragma unroll 1
                for (int i0 = 0; i0 < NP; i0 += 4) {
                  uint4 x[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int kl = (i0 + i) * RPP + rr;
                    const long long lc = __shfl_sync(0xffffffffu, loc, kl);
                    x[i] = ((ok_mask >> kl) & 1u)
                               ? __ldg(reinterpret_cast<const uint4*>(base + lc * s0 + h * G::ED * 2 + cc * 16))
                               : make_uint4(0u, 0u, 0u, 0u);
                  }
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int key = 32 * lw + (i0 + i) * RPP + rr;
                    x[i].x = finite_bf16x2(x[i].x, bad);
                    x[i].y = finite_bf16x2(x[i].y, bad);
                    x[i].z = finite_bf16x2(x[i].z, bad);
                    x[i].w = finite_bf16x2(x[i].w, bad);
                    *reinterpret_cast<uint4*>(ent + dst_off(key, cc)) = x[i];
                  }
                }
                if (bad) *bad_v = 1;
                fence_proxy_async();
                mbar_arrive(bar(kBFull + e % NE));
              } else {
                const uint32_t d0 = smem_u32(ent);
#pragma unroll 4
                for (int i = 0; i < NP; ++i) {
                  const int kl = i * RPP + rr;
                  const long long lc = __shfl_sync(0xffffffffu, loc, kl);
                  const bool ok = (ok_mask >> kl) & 1u;
                  const unsigned char* src = ok ? base + lc * s0 + h * G::ED * 2 + cc * 16 : base;
                  cp_async_16z(d0 + dst_off(32 * lw + kl, cc), src, ok);
                }
                cp_async_arrive_noinc(bar(kBFull + e % NE));
              }
            }
          }
        }
        cp_async_wait<0>();
        if constexpr (PROMPT)
          asm volatile("bar.arrive %0, %1;" ::"r"(1), "r"(kLoadThreads + 128 * NQ) : "memory");
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// flash_tc instances by head_dim and mode (fa::Mode)
fa::FaFn kernel_fa(int D, int mode);
fa::FaFn kernel_fa_64(int mode);
fa::FaFn kernel_fa_128(int mode);
fa::FaFn kernel_fa_256(int mode);

}  // namespace vsk
