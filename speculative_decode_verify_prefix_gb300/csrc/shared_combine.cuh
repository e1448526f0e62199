// The last launch of verify_splitkv_shared_fwd: joins, for every draft row,
// the partial softmaxes over the shared prefix (fa_kernel, one per piece),
// those over the sequence's own prefix (the stream-only kernel, one per piece)
// and the causal draft block.
//
// With (lse, o) of each partial in base 2 and m their largest lse, the joined
// row is sum 2^(lse - m) o / sum 2^(lse - m); a draft key counts as a partial
// of one key (lse = its score, o = its value).  All sums are 32-bit.
//
// One CTA per (sequence, KV head, 16-row tile, 32 output columns): thread t
// owns row t / 8 of the tile and four columns.  The eight threads of a row
// share its draft scores (an eighth of the head dimension each).  The drafts
// come first: this kernel is a programmatic dependent of the launch before it,
// and they need nothing of it.  The partials then come from L2.  Measured alone:
// 30 us of latency-bound loads at 64 sequences of 4 drafts, 32/8 heads of 128,
// most of it under the launch before (the call 204 us with the drafts last, 189 so).
#pragma once
#include "flash_tc.cuh"

namespace vsk {

struct ScParams {
  Params v;             // the flat call; its piece cut when has_own
  int has_own;          // the stream-only kernel ran
  long long tiles, share;  // key tiles of the shared prefix (0: none), of one CTA of fa_kernel
  int h_kv, tpb, nq;       // row blocks of fa_kernel: tokens per query tile, tiles per block
  const float* splse;
  const float* spo;
};

template <int D>
__global__ void __launch_bounds__(128) shared_combine_kernel(const __grid_constant__ ScParams s) {
  constexpr int kSlices = D / 32;
  __shared__ long long scan[8];
  const Params& p = s.v;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ch = static_cast<int>(blockIdx.x % kSlices);
  const int tile = static_cast<int>((blockIdx.x / kSlices) % p.MT);
  const int kvh = static_cast<int>((blockIdx.x / (kSlices * p.MT)) % s.h_kv);
  const int b = static_cast<int>(blockIdx.x / (static_cast<long long>(kSlices) * p.MT * s.h_kv));
  const float NEG_INF = -INFINITY;

  const int fr = tid >> 3, fch = tid & 7;
  const int row = 16 * tile + fr;
  const bool live = row < p.R;
  const int rr = live ? row : p.R - 1;
  const int i = rr / p.gq, head = kvh * p.gq + rr % p.gq;
  const int qa = __ldg(p.qo + b), qe = __ldg(p.qo + b + 1);
  const bool ok = qa >= 0 && qe - qa == p.L && static_cast<long long>(qa) + p.L <= p.n_rows;
  if (!ok && tid == 0 && ch == 0 && tile == 0 && kvh == 0) atomicOr(p.err, kErrBadQoIndptr);
  const long long s_b = ok ? qa : static_cast<long long>(b) * p.L;

  float m = NEG_INF, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto fold = [&](float x, const float4& v) {
    if (x == NEG_INF) return;
    if (x > m) {
      const float a = exp2f(m - x);  // 0 while m is -inf
      l *= a;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] *= a;
      m = x;
    }
    const float w = exp2f(x - m);
    l += w;
    acc[0] = fmaf(w, v.x, acc[0]);
    acc[1] = fmaf(w, v.y, acc[1]);
    acc[2] = fmaf(w, v.z, acc[2]);
    acc[3] = fmaf(w, v.w, acc[3]);
  };
  // n partials, `step` rows apart, eight at a time under way
  auto fold_all = [&](int n, const float* lse, const float* o, long long step) {
    for (int k0 = 0; k0 < n; k0 += 8) {
      float x[8];
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = NEG_INF;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < n) {
          x[k] = __ldcg(lse + (k0 + k) * step);
          v[k] = __ldcg(reinterpret_cast<const float4*>(o + (k0 + k) * step * D));
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) fold(x[k], v[k]);
    }
  };
  const int col = 32 * ch + 4 * fch;

  // ---- where the pieces of the sequence's own prefix lie, cut as the stream cut them ----
  long long own_at = 0;
  int own_n = 0;
  if (s.has_own) {
    long long tot = 0, bef = 0;
    for (int bb = tid; bb < p.B; bb += 128) {
      int P_;
      long long k_;
      seq_info(p, bb, P_, k_);
      tot += max(P_, 1);
      if (bb < b) bef += max(P_, 1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      tot += __shfl_xor_sync(0xffffffffu, tot, o);
      bef += __shfl_xor_sync(0xffffffffu, bef, o);
    }
    if (lane == 0) {
      scan[warp] = tot;
      scan[4 + warp] = bef;
    }
    __syncthreads();
    tot = (scan[0] + scan[1] + scan[2] + scan[3]) * p.n_hg;
    bef = scan[4] + scan[5] + scan[6] + scan[7];
    int P;
    long long kv0;
    seq_info(p, b, P, kv0);
    const int hg = kvh / p.HC, hc = kvh % p.HC, len = max(P, 1);
    long long W = (tot + p.n_stream - 1) / p.n_stream;
    if (W < p.w_min) W = p.w_min;
    const long long off = bef * p.n_hg + static_cast<long long>(hg) * len;
    const long long c0 = off / W, c1 = (off + len - 1) / W;
    const long long slot0 = c0 + static_cast<long long>(b) * p.n_hg + hg;
    const int RM = 16 * p.MT;
    own_at = (slot0 * p.HC + hc) * RM + rr;
    own_n = static_cast<int>(c1 - c0 + 1);
  }

  // ---- the drafts up to this row's own, four at a time ----
  {
    constexpr int DE = D / 8;  // head dimensions of one thread's part of a score
    const __nv_bfloat16* qr = p.q + (s_b + i) * p.q_s0 + static_cast<long long>(head) * p.q_s1 + fch * DE;
    const __nv_bfloat16* kr0 = p.ke + s_b * p.ke_s0 + static_cast<long long>(kvh) * p.ke_s1 + fch * DE;
    const __nv_bfloat16* vr0 = p.ve + s_b * p.ve_s0 + static_cast<long long>(kvh) * p.ve_s1 + col;
    uint32_t qv[DE / 2];
#pragma unroll
    for (int u = 0; u < DE / 2; ++u) qv[u] = ld_u32(qr + 2 * u);
    const int last = __reduce_max_sync(0xffffffffu, i);
    for (int t0 = 0; t0 <= last; t0 += 4) {
      float x[4];
      uint32_t vv[4][2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = 0.f;
        vv[k][0] = vv[k][1] = 0u;
        const int t = min(t0 + k, last);
        const __nv_bfloat16* kr = kr0 + t * p.ke_s0;
#pragma unroll
        for (int u = 0; u < DE / 2; ++u) {
          const float2 qf = unpack_bf16(qv[u]), kf = unpack_bf16(ld_u32(kr + 2 * u));
          x[k] = fmaf(qf.x, kf.x, fmaf(qf.y, kf.y, x[k]));
        }
        if (t0 + k <= i) {
          vv[k][0] = ld_u32(vr0 + t * p.ve_s0);
          vv[k][1] = ld_u32(vr0 + t * p.ve_s0 + 2);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] += __shfl_xor_sync(0xffffffffu, x[k], 1);
        x[k] += __shfl_xor_sync(0xffffffffu, x[k], 2);
        x[k] += __shfl_xor_sync(0xffffffffu, x[k], 4);
        if (t0 + k <= i) {
          const float2 v0 = unpack_bf16(vv[k][0]), v1 = unpack_bf16(vv[k][1]);
          fold(x[k] * p.dscale2, make_float4(v0.x, v0.y, v1.x, v1.y));
        }
      }
    }
  }

  // Everything above reads the call's inputs only; the partials are complete
  // once the launches before this one are (fa_kernel completes after the stream).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- the shared prefix: the pieces that fa_kernel's CTAs left of this row's block ----
  if (s.tiles > 0) {
    const long long tok = s_b + i;
    const int bt = s.nq * s.tpb;
    const long long blk = tok / bt;
    const int rem = static_cast<int>(tok - blk * bt);
    const int in_block = (rem / s.tpb) * 128 + (rem % s.tpb) * p.gq + rr % p.gq;
    const long long u = blk * s.h_kv + kvh;
    const long long c0 = u * s.tiles / s.share, c1 = ((u + 1) * s.tiles - 1) / s.share;
    const long long r0 = (c0 + u) * (128LL * s.nq) + in_block;
    fold_all(static_cast<int>(c1 - c0 + 1), s.splse + r0, s.spo + r0 * D + col, 128 * s.nq);
  }

  if (s.has_own) fold_all(own_n, p.plse + own_at, p.po + own_at * D + col, static_cast<long long>(p.HC) * 16 * p.MT);
  if (live) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16* op = p.o + (s_b + i) * p.o_s0 + static_cast<long long>(head) * p.o_s1 + col;
    *reinterpret_cast<uint32_t*>(op) = pack_bf16(acc[0] * inv, acc[1] * inv);
    *reinterpret_cast<uint32_t*>(op + 2) = pack_bf16(acc[2] * inv, acc[3] * inv);
  }
}

}  // namespace vsk
