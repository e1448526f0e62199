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
// Scores, m, l and O are 32-bit.  P is rounded to V's type, since both operands
// of an MMA have one: to bf16 for bf16 V (relative error 2^-8 at most, that of
// the output's own rounding), to f16 for e4m3 V (2^-11), which f16 holds exactly.
// f16 ends at 2^-24, so P is there 2^(x - m + 7): at most 2^15, and exact to
// 2^-11 down to 2^-21 of the reference.  l sums the unrounded P.
//
// Rows.  The g = h_q / h_kv query heads of a KV head share its keys, so the
// packed row r of a query tile is (token r / g, head r % g): a 128-row tile
// holds 128 / g tokens (rounded down; spare rows are never stored).  An item of
// work is one block of NQ tiles of one KV head: two at head_dim 64 / 128
// (every K / V tile in shared memory feeds both, and the tensor core works on
// one tile while the softmax of the other runs), one at 256, whose O takes
// half of the 512 tensor-memory columns and whose scores are double-buffered
// instead.
//
// What bounds it: per 128-key tile and query tile 2 MMAs of 128 x 128 x D
// against 16,384 exponentials; both pipes are busy at once, and each waits for
// the other at a tile's hand-overs.  Measured: four prompts, 21,716 tokens,
// 32/8 heads of 128, 678 us = 0.78 of the library matrix product's rate over 20
// calls on a cool GPU, 725 us in a long run, where the power cap lowers the
// clocks of both (0.79 of the product's rate there); at 64, where the
// exponentials of a tile outlast its MMAs, 592; three documents, 2,296 tokens,
// 16/2 heads of 256, 38 us (too few items to fill the SMs evenly; two prompts of
// 4,096 225 us); a prefix of 32,768 rows shared by 64 sequences of 4 drafts, 32/8
// of 128, 126 us at 45 % of the tensor pipe (each of the four row blocks of a KV
// head gathers the rows again, 4.2 TB/s in all).
//
// Items.  The CTAs (one per SM) stay, so that the next item's loads run under
// the end of this one.  Prompts: an item is a block of query tiles over all its
// keys; items are drawn from a counter, longest first, as their lengths differ.
// Shared prefix: every block reads all keys, so each CTA takes an equal share of
// the (block, key tile) pairs, in order; the pieces of a block are joined by the
// launch behind.
//
// Roles (registers redistributed with setmaxnreg):
//   warps 0-3, 4-7   softmax of query tile 0 / 1 (thread = row): scores from
//                    tensor memory, P back over them (bf16, half the columns),
//                    rescale, epilogue; at head_dim 256 warps 4-7 load instead
//   warp 8           issues the MMAs: S = Q K^T (both operands in shared memory),
//                    O += P V (P in tensor memory)
//   warp 9           draws the items
//   from 10 (prompts at head_dim 64 / 128, two warps) or 12 (four) on
//                    bring K / V rows into a ring of 128-key entries (128 head
//                    dimensions each, K then V of a tile): contiguous rows by
//                    TMA boxes, gathered bf16 rows by TMA gathers of four rows,
//                    either with 16-byte cp.async where base, strides or row
//                    numbers do not fit a tensor map; e4m3 rows are widened in
//                    registers (exact), K to the queries' bf16, V to P's f16
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
// bit 8 and the CTA's abort flag; no further tile is loaded then, and the CTA
// waits for its copies and products under way, frees its tensor memory and exits.
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
constexpr int kWarpMma = 8;
constexpr int kWarpSched = 9;
constexpr int kLoadArrivals = 128;  // of a ring entry: one per key
constexpr float kThr = 8.f;      // log2 headroom before the running reference is raised
constexpr int kMaxNE = 8;        // ring entries at most
constexpr int kMaskRing = 8;     // > the tiles loaders can run ahead of the softmax

enum Mode { kPrompt = 0, kSharedBf16 = 1, kSharedE4m3 = 2 };

constexpr float kPShift = 7.f;   // log2 of what f16 P are scaled by: 2^(kThr + kPShift) is below f16's largest

// Warps and registers.  The softmax warps hold a row of 128 scores and half a
// row of P, so they get what the launch's registers allow; where two warps
// suffice to load (TMA), the CTA is one warpgroup smaller.
template <int D, int MODE>
struct Cfg {
  static constexpr bool kWide = D == 256 || MODE != kPrompt;
  static constexpr int threads = kWide ? 512 : 384;
  static constexpr int warp_load = kWide ? 12 : 10;  // first loader warp
  static constexpr int n_load = kWide ? 4 : 2;       // loader warps (of a group), 4 / n_load 32-key groups of a tile each
  static constexpr int groups = D == 256 ? 2 : 1;    // groups of loader warps (head_dim 256: warps 4-7 too)
  static constexpr int regs_softmax = D == 256 ? 232 : kWide ? 184 : 216;
  // (head_dim 256, 72: loaders of e4m3 rows spill, 64 sequences behind 32,768 of
  // them 233 us for 219, three documents 41.4 for 40.3)
  static constexpr int regs_other = D == 256 ? 88 : 72;
  static constexpr int regs_launch = 65536 / threads / 8 * 8;
  static_assert((D == 256 ? regs_softmax + 3 * regs_other : 2 * regs_softmax + (threads / 128 - 2) * regs_other) <=
                    threads / 128 * regs_launch, "register shares exceed the launch's");
};

// shared-memory map
constexpr int kBarOff = 0;
constexpr int kTmemOff = 512, kAbortOff = 516;
constexpr int kWorkOff = 576;    // [2] Work
constexpr int kMaskOff = 1024;   // [kMaskRing][4] key-validity words
constexpr int kDataOff = 2048;
// barriers
constexpr int kBFull = 0, kBEmpty = kMaxNE, kBQFull = 2 * kMaxNE, kBQEmpty = kBQFull + 2, kBSFull = kBQEmpty + 2,
              kBPFull = kBSFull + 2, kBOFull = kBPFull + 4, kBOEmpty = kBOFull + 2, kBWFull = kBOEmpty + 2,
              kBWEmpty = kBWFull + 2, kBEdge = kBWEmpty + 2, kBMask = kBEdge + 2, kBDone = kBMask + kMaskRing,
              kNumBars = kBDone + 1;
static_assert(kBarOff + 8 * kNumBars <= kTmemOff, "barriers overlap");

// One item: a row block (query tiles of tokens [tok0, tok0 + NQ tpb) of the
// rows [row0, row0 + n)), a KV head and key tiles [j_first, j_first + nt).
struct Work {
  int n_tiles[2];   // key tiles of query tile 0 / 1 (-1: no more items)
  int head, tok0, n, j_first, j_edge;
  int bad_v;        // prompt: a V value on the diagonal was not finite
  long long row0, item;
};
static_assert(kWorkOff + 2 * sizeof(Work) <= kMaskOff, "work slots overlap");

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
  int n_items;            // items at most
  int* sched;             // next ticket beyond the grid's, CTAs done (both zero between calls)
  long long n_units, share;  // shared: row blocks x KV heads, key tiles per CTA
  float scale2;           // > 0
  int qmode;              // queries enter as they are (0), negated (1) or as zeros (2): the sign of the scale
  int q16, o16;           // 16-byte accesses allowed
  int tma, qtma;          // K / V tiles (bf16), query tiles come through the tensor maps
  float v_scale;
  unsigned* err;
  float* plse;            // shared: partials; piece of CTA c, unit u: NQ * 128 rows at (c + u)
  float* po;
};

using FaFn = void (*)(const FaParams, const CUtensorMap, const CUtensorMap, const CUtensorMap);

// The MMA warp runs its loop converged; one elected lane issues each group of
// MMAs.  Addresses and descriptors are then the same for the whole warp and stay
// in uniform registers (with one lane in a branch around the whole loop long
// prompts took 1155 us, so 1020).
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

// Wait of a whole warp for a phase, one second at most (a wait that gives up
// sets the abort flag and the error bit).  Every lane looks, and looks again at
// once: a suspended warp (try_wait) wakes some hundred cycles late, which the
// chain of scores, softmax and product pays several times a tile (long prompts
// 1129 us suspended, 676 us so); the clock is read only after many looks.
// False: the phase is not complete and the CTA gives up.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  unsigned long long t0 = 0;
  for (int looks = 0; !__all_sync(0xffffffffu, tr::test(bar, parity)); ++looks) {
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    if (looks == 65536) t0 = tc::global_ns();
    if (looks > 65536 && (looks & 1023) == 0 && __all_sync(0xffffffffu, tc::global_ns() - t0 > 1000000000ull)) {
      *abort_flag = 1;
      if ((threadIdx.x & 31) == 0) atomicOr(err, kErrTimeout);
      return false;
    }
  }
  return true;
}
// The wait before a CTA that gave up exits: a phase that completes by itself,
// one second at most, whatever the abort flag says.
__device__ __forceinline__ void wait_last(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = tc::global_ns();
  while (!__all_sync(0xffffffffu, tr::test(bar, parity)))
    if (__all_sync(0xffffffffu, tc::global_ns() - t0 > 1000000000ull)) return;
}
// Position in the ring: slot and the parity of its lap.
template <int NE>
struct Pos {
  uint32_t slot, par;
  __device__ __forceinline__ Pos ahead(uint32_t n) const {
    const uint32_t x = slot + n;
    return x >= NE ? Pos{x - NE, par ^ 1u} : Pos{x, par};
  }
};

// One box of a [rows][heads][head_dim] tensor map into shared memory ([32 rows]
// [64 head dimensions] of a K / V head, [tpb rows][g heads][64] of the queries).
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int head, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(bar), "r"(x), "r"(head), "r"(row)
      : "memory");
}
// Four rows of 64 elements, gathered by row number, into four consecutive 128-byte rows.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int r0, int r1,
                                            int r2, int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
      "%6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
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
__global__ void __launch_bounds__(fa::Cfg<D, MODE>::threads, 1) fa_kernel(const __grid_constant__ fa::FaParams p,
                                                             const __grid_constant__ CUtensorMap qmap,
                                                             const __grid_constant__ CUtensorMap kmap,
                                                             const __grid_constant__ CUtensorMap vmap) {
  using namespace fa;
  using G = fa::Geo<D>;
  using C = fa::Cfg<D, MODE>;
  constexpr int NQ = G::NQ, NH = G::NH, NE = G::NE, ENT = G::ENT;
  constexpr bool PROMPT = MODE == kPrompt, P16 = MODE == kSharedE4m3;  // P and V are f16, else bf16
  constexpr float p_up = P16 ? kPShift : 0.f;                          // log2 of the scale of P, l and O
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
  const float NEG_INF = -INFINITY;
  const int bt = NQ * p.tpb;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  volatile unsigned* maskw = reinterpret_cast<volatile unsigned*>(smem + kMaskOff);
  Work* work = reinterpret_cast<Work*>(smem + kWorkOff);
  const uint32_t q_s = smem_u32(smem + G::q_off), ring_s = smem_u32(smem + G::ring_off);
  if ((smem_u32(smem) & 1023u) != 0u) {  // the swizzled layouts need it; uniform over the grid
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < NE; ++i) {
      mbar_init(bar(kBFull + i), kLoadArrivals);
      mbar_init(bar(kBEmpty + i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kBQFull + t), p.qtma ? 1 : 4);
      mbar_init(bar(kBQEmpty + t), 1);
      mbar_init(bar(kBSFull + t), 1);
      mbar_init(bar(kBPFull + 2 * t), 4);
      mbar_init(bar(kBPFull + 2 * t + 1), 4);
      mbar_init(bar(kBOFull + t), 1);
      mbar_init(bar(kBOEmpty + t), 4);
      mbar_init(bar(kBWFull + t), 1);
      mbar_init(bar(kBWEmpty + t), 4 * NQ + 1 + C::n_load * C::groups);
      mbar_init(bar(kBEdge + t), C::n_load * C::groups);
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
  if (p.qtma && p.tpb * p.gq < 128) {
    // rows of the query tiles that no box fills
    const int rows = 128 - p.tpb * p.gq;
    for (int i = tid; i < NQ * (D / 64) * rows * 8; i += C::threads)
      *reinterpret_cast<uint4*>(smem + G::q_off + (i / (rows * 8)) * (128 * 128) + (128 - rows) * 128 +
                                (i % (rows * 8)) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
  }
  if (PROMPT && blockIdx.x == 0 && warp == kWarpSched) {
    for (int b = lane; b < p.B; b += 32) {
      const int a = __ldg(p.qo + b), e = __ldg(p.qo + b + 1);
      if (!(a >= 0 && e >= a && e <= p.n_rows)) atomicOr(p.err, kErrBadQoIndptr);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kTmemOff);

  // The item of round `it` for a role's warp: false when there is none left.
  auto take = [&](int it, const Work*& w) -> bool {
    wait_all(bar(kBWFull + (it & 1)), static_cast<uint32_t>((it >> 1) & 1), abort_flag, p.err);
    w = work + (it & 1);
    const int first = *const_cast<const volatile int*>(&w->n_tiles[0]);
    return !__any_sync(0xffffffffu, *abort_flag != 0) && first >= 0;
  };
  auto give_back = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBWEmpty + (it & 1)));
  };

  if (warp < 4 * NQ) {
    // ================================ softmax ================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::regs_softmax));
    const int t = warp >> 2, w = warp & 3, tw = tid & 127;
    const int r = 32 * w + lane;  // this thread's packed row of the tile
    const int r_tok = r / p.gq, r_head = r % p.gq;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * w) << 16);
    const uint32_t t_o = t_lane + G::col_o + t * D;
    const float sc = p.scale2;
    uint32_t g = 0;   // key tiles of this query tile so far
    uint32_t gm = 0;  // key tiles of the CTA so far (shared prefix: the mask ring's position)
#pragma unroll 1
    for (int it = 0;; ++it) {
      const Work* wk;
      if (!take(it, wk)) break;
      const int my_tiles = wk->n_tiles[t], n = wk->n, head = wk->head;
      const int first = wk->tok0 + t * p.tpb;  // first token of the tile
      const long long row0 = wk->row0;
      // ---- queries of the tile into shared memory (where no tensor map takes them) ----
      if (!p.qtma) {
        wait_all(bar(kBQEmpty + t), static_cast<uint32_t>((it & 1) ^ 1), abort_flag, p.err);
        constexpr int CPR = D / 8;  // 16-byte chunks of a row
        unsigned char* qs = smem + G::q_off + t * G::QT;
#pragma unroll 8
        for (int i = 0; i < CPR; ++i) {
          const int ci = tw + 128 * i, qr = ci / CPR, c = ci % CPR;
          const int qt = first + qr / p.gq, qh = qr % p.gq;
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (qr < p.tpb * p.gq && qt < n && p.qmode != 2) {
            const __nv_bfloat16* src =
                p.q + (row0 + qt) * p.q_s0 + static_cast<long long>(head * p.gq + qh) * p.q_s1 + c * 8;
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
          *reinterpret_cast<uint4*>(qs + (c >> 3) * (128 * 128) + qr * 128 + (((c & 7) ^ (qr & 7)) << 4)) = x;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBQFull + t));
      }
      const int tok = min(first + r_tok, n - 1);
      const bool real = r < p.tpb * p.gq && first + r_tok < n;
      float mrun = NEG_INF, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < my_tiles; ++j, ++g) {
        const int buf = NQ == 2 ? t : (g & 1);
        const uint32_t par = NQ == 2 ? (g & 1) : ((g >> 1) & 1);
        const uint32_t t_s = t_lane + buf * KT;
        wait_all(bar(kBSFull + buf), par, abort_flag, p.err);
        tc_fence_after();
        // Scores, then P, in halves of 64 keys.  The first half's P is computed
        // against the reference that the tiles before left, while the second
        // half's scores arrive and the tile's maximum is taken; only where that
        // maximum passes the reference by more than kThr is it done again.
        uint32_t s[KT];
        bool masked;
        unsigned mw[4];
        if constexpr (PROMPT) {
          masked = (j + 1) * KT - 1 > first;
          if (masked) {
            const int lim = tok - j * KT;  // keys c <= lim are visible
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int n_vis = min(32, max(0, lim + 1 - 32 * u));
              mw[u] = n_vis == 32 ? 0xFFFFFFFFu : (1u << n_vis) - 1u;
            }
          }
        } else {
          const uint32_t jm = (gm + j) % kMaskRing;
          wait_all(bar(kBMask + jm), ((gm + j) / kMaskRing) & 1, abort_flag, p.err);
#pragma unroll
          for (int u = 0; u < 4; ++u) mw[u] = maskw[4 * jm + u];
          masked = (mw[0] & mw[1] & mw[2] & mw[3]) != 0xFFFFFFFFu;
        }
        float mx[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
        const float2 sc2 = make_float2(sc, sc);
        uint32_t pk[32];
        float2 l2[2];
        auto probs = [&](int h, float mref) {  // pk and the sum of half h
          const float2 mn2 = make_float2(p_up - mref, p_up - mref);
          l2[0] = l2[1] = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int c = 64 * h + 2 * i;
            float2 x = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, mn2);
            x.x = fast_exp2(x.x);
            x.y = fast_exp2(x.y);
            l2[i & 1] = add2(l2[i & 1], x);
            pk[i] = P16 ? pack_f16(x.x, x.y) : pack_bf16(x.x, x.y);
          }
        };
        auto hide = [&](int h) {  // -inf for masked keys
#pragma unroll
          for (int c = 64 * h; c < 64 * h + 64; ++c)
            s[c] = ((mw[c >> 5] >> (c & 31)) & 1u) ? s[c] : __float_as_uint(NEG_INF);
        };
        auto top = [&](int h) {
#pragma unroll
          for (int c = 64 * h; c < 64 * h + 64; c += 2)
            mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        };
        tmem_ld32_nw(t_s, s);
        tmem_ld32_nw(t_s + 32, s + 32);
        tmem_wait_ld();
        tmem_pass(s);
        tmem_pass(s + 32);
        tmem_ld32_nw(t_s + 64, s + 64);
        tmem_ld32_nw(t_s + 96, s + 96);
        if (__builtin_expect(masked, 0)) hide(0);
        probs(0, mrun == NEG_INF ? 0.f : mrun);
        top(0);
        tmem_wait_ld();
        tmem_pass(s + 64);
        tmem_pass(s + 96);
        if (__builtin_expect(masked, 0)) hide(1);
        top(1);
        // ---- raise the reference when the tile's maximum passes it by more than kThr ----
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        if (__builtin_expect(__any_sync(0xffffffffu, mt > mrun + kThr), 0)) {
          const float mn = fmaxf(mrun, mt);
          const float al = mn == NEG_INF ? 1.f : fast_exp2(mrun - mn);
          if (j > 0) {
            wait_all(bar(kBOFull + t), (g - 1) & 1, abort_flag, p.err);
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
          probs(0, mrun == NEG_INF ? 0.f : mrun);
        }
        // ---- P over the scores' columns, half by half ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1) probs(1, mrun == NEG_INF ? 0.f : mrun);
          tmem_st32(t_s + 32 * h, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBPFull + 2 * buf + h));
          l2[0] = add2(l2[0], l2[1]);
          l += l2[0].x + l2[0].y;
        }
      }
      gm += max(wk->n_tiles[0], wk->n_tiles[1]);
      // ---- epilogue ----
      if (my_tiles > 0) {
        // one query tile: the last scores are issued before the PV of the tile
        // before, so that phase has to be seen to complete first
        if (NQ == 1 && my_tiles > 1) wait_all(bar(kBOFull + t), (g - 2) & 1, abort_flag, p.err);
        wait_all(bar(kBOFull + t), (g - 1) & 1, abort_flag, p.err);
        tc_fence_after();
      }
      if constexpr (PROMPT) {
        // the item's diagonal V tiles have been looked at
        wait_all(bar(kBEdge + (it & 1)), static_cast<uint32_t>((it >> 1) & 1), abort_flag, p.err);
        if (my_tiles > 0) {
          const float inv = 1.f / l;
          const bool fix = *const_cast<const volatile int*>(&wk->bad_v) != 0;
          const int key0 = wk->j_edge * KT;
          __nv_bfloat16* orow =
              p.o + (row0 + tok) * p.o_s0 + static_cast<long long>(head * p.gq + r_head) * p.o_s1;
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            float o[32];
            tmem_ld<32>(t_o + 32 * cb, o);
            if (!real) continue;
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= inv;
            if (fix) {
              // values the loaders zeroed, for the rows that see them
              for (int key = key0; key <= tok; ++key) {
                const uint32_t* vr =
                    reinterpret_cast<const uint32_t*>(p.v + (row0 + key) * p.v_s0 + head * p.v_s1 + cb * 64);
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
        // partial of this key range: o v_scale / l and m + log2 l (of l without the scale of P), -inf and 0
        // where no key was valid
        const long long prow = wk->item * (NQ * 128) + t * 128 + r;
        const float inv = l == 0.f ? 0.f : p.v_scale / l;
        if (real) p.plse[prow] = l == 0.f ? NEG_INF : mrun + (log2f(l) - p_up);
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
      __syncwarp();
      if (lane == 0 && my_tiles > 0) mbar_arrive(bar(kBOEmpty + t));
      give_back(it);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::regs_other));
    if (warp == kWarpSched) {
      // ============================ items of this CTA ============================
      // Prompts: the first is the CTA's number, the others are drawn from a
      // counter, so that long and short items even out; a sequence's row blocks
      // come last (longest key range) first.  Shared prefix: every CTA has the
      // same number of key tiles, cut where a row block's keys end.
      long long at = static_cast<long long>(blockIdx.x) * p.share;  // shared prefix: next tile of this CTA's share
      int n_piece = 0;
      // prompts: sequences [0, b_scan) have `before` row blocks, all behind this
      // CTA's tickets (they only grow)
      int b_scan = 0;
      long long before = 0;
#pragma unroll 1
      for (int it = 0;; ++it) {
        int ticket = static_cast<int>(blockIdx.x);
        if (PROMPT && it > 0) {
          if (lane == 0) ticket = static_cast<int>(gridDim.x) + atomicAdd(p.sched, 1);
          ticket = __shfl_sync(0xffffffffu, ticket, 0);
        }
        Work x;
        x.n_tiles[0] = x.n_tiles[1] = -1;
        x.bad_v = 0;
        x.item = ticket;
        if (ticket < p.n_items) {
          bool found = true;
          if constexpr (PROMPT) {
            x.head = ticket % p.h_kv;
            x.j_first = 0;
            found = false;
            while (b_scan < p.B && !found) {
              const long long want = ticket / p.h_kv - before;
              const int b = b_scan + lane;
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
              const unsigned m = __ballot_sync(0xffffffffu, want >= incl - nb && want < incl);
              if (m) {
                const int src = __ffs(m) - 1;
                found = true;
                x.n = __shfl_sync(0xffffffffu, n, src);
                x.row0 = __shfl_sync(0xffffffffu, a, src);
                x.tok0 = (__shfl_sync(0xffffffffu, incl, src) - 1 - static_cast<int>(want)) * bt;
              } else {
                before += __shfl_sync(0xffffffffu, incl, 31);
                b_scan += 32;
              }
            }
          } else {
            // piece `it` of this CTA's share of the row blocks' key tiles, laid end to end
            const long long tiles = (p.n_keys + KT - 1) / KT;
            const long long end = min(tiles * p.n_units, static_cast<long long>(blockIdx.x + 1) * p.share);
            found = at < end;
            const int u = static_cast<int>(at / tiles);
            x.head = u % p.h_kv;
            x.row0 = 0;
            x.n = static_cast<int>(p.n_rows);
            x.tok0 = (u / p.h_kv) * bt;
            x.j_first = static_cast<int>(at - u * tiles);
            x.item = static_cast<long long>(blockIdx.x) + u;
            n_piece = static_cast<int>(min(tiles - x.j_first, end - at));
            at += n_piece;
          }
          if (found) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int first = x.tok0 + t * p.tpb;
              if (t >= NQ || first >= x.n) {
                x.n_tiles[t] = 0;
              } else if constexpr (PROMPT) {
                x.n_tiles[t] = (min(first + p.tpb, x.n) + KT - 1) / KT;
              } else {
                x.n_tiles[t] = n_piece;
              }
            }
            x.j_edge = PROMPT ? x.tok0 / KT : 0;  // first tile with keys that some row of the block must not see
          }
        }
        // (a slot that is still in use is left as it is)
        if (!wait_all(bar(kBWEmpty + (it & 1)), static_cast<uint32_t>(((it >> 1) & 1) ^ 1), abort_flag, p.err)) break;
        if (lane == 0) {
          work[it & 1] = x;
          mbar_arrive(bar(kBWFull + (it & 1)));
        }
        __syncwarp();
        if (x.n_tiles[0] < 0 || __any_sync(0xffffffffu, *abort_flag != 0)) break;
      }
    } else if (warp == kWarpMma) {
      // ============================ MMA issue ============================
      const uint32_t tmem_u = __reduce_max_sync(0xffffffffu, tmem);
      constexpr uint32_t idS = idesc(1, 1, 0, 0, 128, KT);
      constexpr uint32_t idPV = idesc(P16 ? 0 : 1, P16 ? 0 : 1, 0, 1, 128, G::ED);
      const uint64_t dq0 = sdesc(q_s, 16, 1024), dk0 = sdesc(ring_s, 16, 1024), dv0 = sdesc(ring_s, KT * 128, 1024);
      using RP = Pos<NE>;
      RP kp{0u, 0u}, vp{NH, 0u};   // ring entries of the next K / V tile (NH each; at NQ = 1 of the next tile)
      uint32_t g[2] = {0u, 0u};    // key tiles per query tile so far
      uint32_t n_o[2] = {0u, 0u};  // items that gave the query tile any
      // S of query tile t against the K tile at kp; last: the K tile's entries
      // are free afterwards; q_free: the queries are
      auto qk = [&](int t, uint32_t gt, bool last, bool q_free) {
        const uint32_t buf = NQ == 2 ? t : (gt & 1);
        const uint32_t dc = tmem_u + buf * KT;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const uint32_t slot = kp.ahead(h).slot;
          const uint64_t qd = dq0 + static_cast<uint64_t>((t * G::QT + h * 2 * (128 * 128)) >> 4);
          const uint64_t kd = dk0 + static_cast<uint64_t>(slot * (ENT >> 4));
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < G::ED / 16; ++ks) {
              const uint64_t off = static_cast<uint64_t>(((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4);
              mma_f16_ss(dc, qd + off, kd + off, idS, h > 0 || ks > 0);
            }
            if (h == NH - 1) mma_commit(bar(kBSFull + buf));
            if (last) mma_commit(bar(kBEmpty + slot));
            if (h == NH - 1 && q_free) mma_commit(bar(kBQEmpty + t));
          }
        }
      };
      // O += P V of query tile t with the V tile at vp
      auto pv = [&](int t, uint32_t gt, bool first, bool last) {
        const uint32_t buf = NQ == 2 ? t : (gt & 1), par = NQ == 2 ? (gt & 1) : ((gt >> 1) & 1);
        const uint32_t a = tmem_u + buf * KT;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait_all(bar(kBPFull + 2 * buf + half), par, abort_flag, p.err);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const uint32_t slot = vp.ahead(h).slot;
            const uint64_t vd = dv0 + static_cast<uint64_t>(slot * (ENT >> 4));
            if (elect_one()) {
#pragma unroll
              for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                mma_f16_ts(tmem_u + G::col_o + t * D + h * G::ED, a + ks * 8, vd + static_cast<uint64_t>(ks * 128), idPV,
                           !first || ks > 0);
              if (half == 1 && h == NH - 1) mma_commit(bar(kBOFull + t));
              if (half == 1 && last) mma_commit(bar(kBEmpty + slot));
            }
          }
        }
      };
      auto acquire = [&](const RP& x) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const RP y = x.ahead(h);
          wait_all(bar(kBFull + y.slot), y.par, abort_flag, p.err);
        }
        // rows that came by cp.async (stores are fenced by their writers, TMA needs none)
        if (MODE == kSharedBf16 || (PROMPT && !p.tma)) fence_proxy_async();
        tc_fence_after();
      };
#pragma unroll 1
      for (int it = 0;; ++it) {
        const Work* wk;
        if (!take(it, wk)) break;
        // (through a warp reduction, whose result is a uniform register: the loop
        // and with it the descriptors' arithmetic are then uniform, too)
        const int n0 = __reduce_max_sync(0xffffffffu, wk->n_tiles[0]);
        const int n1 = __reduce_max_sync(0xffffffffu, wk->n_tiles[1]);
        give_back(it);
        const int nt = max(n0, n1);
#pragma unroll
        for (int t = 0; t < NQ; ++t) wait_all(bar(kBQFull + t), static_cast<uint32_t>(it & 1), abort_flag, p.err);
        tc_fence_after();
        if (nt > 0) {
          acquire(kp);
          if (n0 > 0) qk(0, g[0], NQ == 1 || n1 == 0, n0 == 1);
          if (NQ == 2 && n1 > 0) qk(1, g[1], true, n1 == 1);
          kp = kp.ahead(NQ == 1 ? NH : 2 * NH);
        }
        if (elect_one()) {
          if (n0 == 0) mma_commit(bar(kBQEmpty));
          if (NQ == 2 && n1 == 0) mma_commit(bar(kBQEmpty + 1));
        }
        // the rows of O of the item before have been read (a query tile without
        // keys has none, and its softmax warps say nothing)
        if (n0 > 0) wait_all(bar(kBOEmpty), (n_o[0]++ & 1) ^ 1, abort_flag, p.err);
        if (NQ == 2 && n1 > 0) wait_all(bar(kBOEmpty + 1), (n_o[1]++ & 1) ^ 1, abort_flag, p.err);
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
          const bool more = j + 1 < nt;
          if constexpr (NQ == 1) {
            if (more) {
              acquire(kp);
              qk(0, g[0] + 1, true, j + 2 == nt);
              kp = kp.ahead(NH);
            }
            vp = kp;
            acquire(vp);
            pv(0, g[0], j == 0, true);
            kp = kp.ahead(NH);
            ++g[0];
          } else {
            // (the tiles of a block have as many keys or the second one more)
            acquire(vp);
            if (j < n0) {
              pv(0, g[0], j == 0, j >= n1);
              ++g[0];
            }
            if (more) acquire(kp);
            if (j + 1 < n0) qk(0, g[0], j + 1 >= n1, j + 2 == n0);
            if (j < n1) {
              pv(1, g[1], j == 0, true);
              ++g[1];
            }
            if (j + 1 < n1) qk(1, g[1], true, j + 2 == n1);
            if (more) kp = kp.ahead(2 * NH);
            vp = vp.ahead(2 * NH);
          }
        }
      }
      if (elect_one()) mma_commit(bar(kBDone));
      wait_last(bar(kBDone), 0u);  // no product or arrival is pending when the CTA exits
    } else if (warp >= C::warp_load || (C::groups == 2 && warp < kWarpMma)) {
      // ================================ loaders ================================
      // A warp has NS of the four 32-key groups of every entry (with two groups
      // of loader warps: of every other entry).
      constexpr int NS = 4 / C::n_load;
      const int lw = warp >= C::warp_load ? warp - C::warp_load : warp & 3, lgrp = warp < kWarpMma ? 1 : 0;
      constexpr int CPK = G::ED / 8;        // 16-byte chunks of an entry's bf16 row
      constexpr int RPP = 32 / CPK;         // rows of a warp's pass
      constexpr int NP = 32 / RPP;          // passes over 32 rows
      const int cc = lane % CPK, rr = lane / CPK;
      int nt;  // key tiles of the item
      // (a wait that gives up ends the item with this tile; looking at the abort
      // flag every tile cost the gathers of a long shared prefix 1.5 %.  e4m3 rows
      // come by plain loads, which may run on: nothing of them is under way later)
      auto slot_wait = [&](uint32_t e) {
        const bool go = wait_all(bar(kBEmpty + e % NE), ((e / NE) & 1) ^ 1, abort_flag, p.err);
        if (MODE != kSharedE4m3 && !go) nt = 0;
      };
      auto dst_off = [&](int key, int c) -> uint32_t {
        return static_cast<uint32_t>((c >> 3) * (KT * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4));
      };
      uint32_t e = 0;   // ring entry
      uint32_t gm = 0;  // key tiles so far
#pragma unroll 1
      for (int it = 0;; ++it) {
        const Work* wk;
        if (!take(it, wk)) break;
        nt = max(wk->n_tiles[0], wk->n_tiles[1]);
        const int head = wk->head, n = wk->n, j_first = wk->j_first, j_edge = wk->j_edge;
        const long long row0 = wk->row0;
        if (p.qtma && lgrp == 0 && lw < NQ) {
          // query tile lw (rows past the sequence may come along: they are never stored)
          const bool go = wait_all(bar(kBQEmpty + lw), static_cast<uint32_t>((it & 1) ^ 1), abort_flag, p.err);
          if (lane == 0 && wk->n_tiles[lw] == 0) {
            mbar_arrive(bar(kBQFull + lw));  // no MMA reads it
          } else if (go && lane == 0) {
            const uint32_t fb = bar(kBQFull + lw);
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(fb),
                         "r"(p.tpb * p.gq * D * 2)
                         : "memory");
#pragma unroll 1
            for (int cb = 0; cb < D / 64; ++cb)
              tma_load_box(q_s + lw * G::QT + cb * (128 * 128), &qmap, fb, cb * 64, head * p.gq,
                           static_cast<int>(row0) + wk->tok0 + lw * p.tpb);
          }
          __syncwarp();
        }
        auto key_at = [&](int j, int kg) { return static_cast<long long>(j_first + j) * KT + 32 * kg + lane; };
        auto load_idx = [&](int j, int kg) -> long long {  // -1 where there is no key
          const long long at = key_at(j, kg);
          if (j >= nt || at >= p.n_keys) return -1;
          return p.idx64 ? __ldg(static_cast<const long long*>(p.idx) + at)
                         : static_cast<long long>(__ldg(static_cast<const int*>(p.idx) + at));
        };
        // the entries of K (kv = 0) or V tile j, of rows loc (a lane's key of each group)
        auto load = [&](int kv, int j, const long long (&loc)[NS], const unsigned (&ok_mask)[NS]) {
          const unsigned char* base = kv ? p.v + head * p.v_s1 : p.k + head * p.k_s1;
          const long long s0 = kv ? p.v_s0 : p.k_s0;
#pragma unroll 1
          for (int h = 0; h < NH; ++h, ++e) {
            if (C::groups == 2 && (e & 1u) != static_cast<uint32_t>(lgrp)) continue;
            unsigned char* ent = smem + G::ring_off + (e % NE) * ENT;
            const uint32_t fb = bar(kBFull + e % NE);
            auto publish_mask = [&](int u) {  // which keys of the group count, with a tile's first entry
              if (!PROMPT && kv == 0 && h == 0 && lane == 0) {
                maskw[4 * (gm % kMaskRing) + lw * NS + u] = ok_mask[u];
                mbar_arrive(bar(kBMask + gm % kMaskRing));
              }
            };
            if constexpr (MODE == kSharedE4m3) {
              // 16 e4m3 values a lane, two 16-byte chunks of bf16 (K) or f16 (V);
              // the rows are under way before the slot is free
              constexpr int LPR = CPK / 2, RP8 = 32 / LPR, NP8 = 32 / RP8;
              const int c8 = lane % LPR, r8 = lane / LPR;
              uint4 x[NP8];
#pragma unroll
              for (int i = 0; i < NP8; ++i) {
                const int kl = i * RP8 + r8;
                const long long lc = __shfl_sync(0xffffffffu, loc[0], kl);
                x[i] = ((ok_mask[0] >> kl) & 1u)
                           ? __ldg(reinterpret_cast<const uint4*>(base + lc * s0 + h * G::ED + c8 * 16))
                           : make_uint4(0u, 0u, 0u, 0u);
              }
              slot_wait(e);
              publish_mask(0);
#pragma unroll
              for (int i = 0; i < NP8; ++i) {
                const int key = 32 * lw + i * RP8 + r8;
                const uint32_t wv[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t y[8];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const auto lo = static_cast<unsigned short>(wv[u] & 0xFFFFu), hi = static_cast<unsigned short>(wv[u] >> 16);
                  y[2 * u] = kv ? e4m3x2_to_f16x2(lo) : e4m3x2_to_bf16x2(lo);
                  y[2 * u + 1] = kv ? e4m3x2_to_f16x2(hi) : e4m3x2_to_bf16x2(hi);
                }
                *reinterpret_cast<uint4*>(ent + dst_off(key, 2 * c8)) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(ent + dst_off(key, 2 * c8 + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
              }
              fence_proxy_async();
              mbar_arrive(fb);
            } else {
              slot_wait(e);
#pragma unroll 1
              for (int u = 0; u < NS; ++u) {
                const int key0 = 32 * (lw * NS + u);  // first key of the group in the tile
                const long long my_loc = loc[u];
                const unsigned my_ok = ok_mask[u];
                publish_mask(u);
                if (PROMPT && p.tma && (kv == 0 || j < j_edge)) {
                  // keys past the sequence may come along, or what was there before
                  // stays: their scores are masked, and V tiles that hold any take
                  // the next branch
                  if (lane == 0) {
                    const uint32_t d0 = smem_u32(ent) + key0 * 128;
                    const bool any = j * KT + key0 < n;
                    mbar_arrive_warp_tx(fb, any ? 32 * G::ED * 2 : 0);
                    for (int cb = 0; any && cb < G::ED / 64; ++cb)
                      tma_load_box(d0 + cb * (KT * 128), kv ? &vmap : &kmap, fb, h * G::ED + cb * 64, head,
                                   static_cast<int>(row0) + j * KT + key0);
                  }
                  __syncwarp();
                } else if (PROMPT && kv == 1 && j >= j_edge) {
                  // V on the diagonal: values that are not finite become 0 here
                  // and are added by the epilogue to the rows that see them
                  bool bad = false;
#pragma unroll 1
                  for (int i0 = 0; i0 < NP; i0 += 8) {
                    uint4 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                      const int kl = (i0 + i) * RPP + rr;
                      const long long lc = __shfl_sync(0xffffffffu, my_loc, kl);
                      x[i] = ((my_ok >> kl) & 1u)
                                 ? __ldg(reinterpret_cast<const uint4*>(base + lc * s0 + h * G::ED * 2 + cc * 16))
                                 : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                      const int key = key0 + (i0 + i) * RPP + rr;
                      x[i].x = finite_bf16x2(x[i].x, bad);
                      x[i].y = finite_bf16x2(x[i].y, bad);
                      x[i].z = finite_bf16x2(x[i].z, bad);
                      x[i].w = finite_bf16x2(x[i].w, bad);
                      *reinterpret_cast<uint4*>(ent + dst_off(key, cc)) = x[i];
                    }
                  }
                  if (bad) *const_cast<volatile int*>(&work[it & 1].bad_v) = 1;
                  fence_proxy_async();
                  mbar_arrive(fb);
                } else if (MODE == kSharedBf16 && p.tma && my_ok == 0xFFFFFFFFu) {
                  // 8 groups of 4 rows x ED / 64 column blocks, one gather a lane
                  constexpr int NB = G::ED / 64;
                  int r[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    r[i] = __shfl_sync(0xffffffffu, static_cast<int>(my_loc), (4 * (lane / NB) + i) & 31);
                  if (lane == 0) mbar_arrive_warp_tx(fb, 32 * G::ED * 2);
                  __syncwarp();
                  if (lane < 8 * NB) {
                    const int grp = lane / NB, cb = lane % NB;
                    tma_gather4(smem_u32(ent) + cb * (KT * 128) + (key0 + 4 * grp) * 128, kv ? &vmap : &kmap, fb,
                                head * static_cast<int>((kv ? p.v_s1 : p.k_s1) / 2) + h * G::ED + cb * 64, r[0], r[1],
                                r[2], r[3]);
                  }
                  __syncwarp();
                } else {
                  const uint32_t d0 = smem_u32(ent);
#pragma unroll 4
                  for (int i = 0; i < NP; ++i) {
                    const int kl = i * RPP + rr;
                    const long long lc = __shfl_sync(0xffffffffu, my_loc, kl);
                    const bool ok = (my_ok >> kl) & 1u;
                    const unsigned char* src = ok ? base + lc * s0 + h * G::ED * 2 + cc * 16 : base;
                    cp_async_16z(d0 + dst_off(key0 + kl, cc), src, ok);
                  }
                  cp_async_arrive_noinc(fb);
                }
              }
            }
          }
        };
        // pool rows of tile j, those of tile j + 1 asked for ahead
        long long loc_next[NS];
        auto rows_of = [&](int j, long long (&loc)[NS], unsigned (&ok_mask)[NS]) {
#pragma unroll
          for (int u = 0; u < NS; ++u) {
            const int kg = lw * NS + u;
            if constexpr (PROMPT) {
              loc[u] = row0 + static_cast<long long>(j) * KT + 32 * kg + lane;
              ok_mask[u] = __ballot_sync(0xffffffffu, j * KT + 32 * kg + lane < n);
            } else {
              loc[u] = loc_next[u];
              loc_next[u] = load_idx(j + 1, kg);
              const bool ok = loc[u] >= 0 && loc[u] < p.pool;
              if (!ok && key_at(j, kg) < p.n_keys) atomicOr(p.err, kErrBadIndex);
              ok_mask[u] = __ballot_sync(0xffffffffu, ok);
            }
          }
        };
        if constexpr (!PROMPT) {
#pragma unroll
          for (int u = 0; u < NS; ++u) loc_next[u] = load_idx(0, lw * NS + u);
        }
        // in the order in which the MMAs take the tiles: K and V in turn, or, where
        // the next scores are issued before a tile's product, K one tile ahead
        // (with V before K there the K tile waited for its entries until the
        // product was done: three documents, 16/2 heads of 256, 39.6 us against 33.4)
        if constexpr (NQ == 2) {
#pragma unroll 1
          for (int j = 0; j < nt; ++j, ++gm) {
            long long loc[NS];
            unsigned ok_mask[NS];
            rows_of(j, loc, ok_mask);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) load(kv, j, loc, ok_mask);
          }
        } else {
          long long loc_k[NS], loc_v[NS];  // of the newest K tile and of the V tile that comes next
          unsigned ok_k[NS], ok_v[NS];
#pragma unroll 1
          for (int st = 0; st < 2 * nt; ++st) {  // K0 K1 V0 K2 V1 ... V(nt - 2) V(nt - 1)
            const int tail = 2 * nt - 1;
            const int kv = st == 0 ? 0 : st == tail ? 1 : ~st & 1;
            const int j = st == 0 ? 0 : st == tail ? nt - 1 : (st + 1) / 2 - kv;
            if (st == 0) rows_of(0, loc_k, ok_k);
            long long loc[NS];
            unsigned ok_mask[NS];
#pragma unroll
            for (int u = 0; u < NS; ++u)
              if (kv == 0 || st == tail) {
                loc_v[u] = loc_k[u];
                ok_v[u] = ok_k[u];
              }
            if (kv == 0 && st > 0) rows_of(j, loc_k, ok_k);
#pragma unroll
            for (int u = 0; u < NS; ++u) {
              loc[u] = kv ? loc_v[u] : loc_k[u];
              ok_mask[u] = kv ? ok_v[u] : ok_k[u];
            }
            load(kv, j, loc, ok_mask);
            if (kv == 0) ++gm;
          }
        }
        if constexpr (PROMPT) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBEdge + (it & 1)));  // bad_v is final
        }
        give_back(it);
      }
      cp_async_wait<0>();
      // TMA copies that no product waits for any more: two milliseconds, far beyond the latency of any
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {
        const unsigned long long t0 = tc::global_ns();
        while (tc::global_ns() - t0 < 2000000ull) __nanosleep(1000);
      }
    }
    __syncwarp();
  }
  // the kernel that joins the partials may start its CTAs where SMs are free
  if (!PROMPT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  // the own prefixes' stream, of which this launch may be a programmatic
  // dependent (it reads nothing of it), is complete before this grid is
  if (!PROMPT && tid == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  // the last CTA leaves the counters at zero for the next call
  if (PROMPT && tid == 0) {
    __threadfence();
    if (atomicAdd(p.sched + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      p.sched[0] = 0;
      p.sched[1] = 0;
      __threadfence();
    }
  }
}

// flash_tc instances by head_dim and mode (fa::Mode)
fa::FaFn kernel_fa(int D, int mode);
fa::FaFn kernel_fa_64(int mode);
fa::FaFn kernel_fa_128(int mode);
fa::FaFn kernel_fa_256(int mode);

}  // namespace vsk
