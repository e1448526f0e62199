// Host side of the calls around the verify call: attention over whole prompts
// (prompt_attn_fwd) and the verify call for a batch that shares a long prefix
// (verify_splitkv_shared_fwd).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "flash_tc.cuh"
#include "shared_combine.cuh"
#include "verify_host.cuh"

namespace vsk {

fa::FaFn kernel_fa(int D, int mode) {
  return D == 64 ? kernel_fa_64(mode) : D == 128 ? kernel_fa_128(mode) : D == 256 ? kernel_fa_256(mode) : nullptr;
}

static int fa_smem(int D) { return D == 64 ? fa::Geo<64>::smem : D == 128 ? fa::Geo<128>::smem : fa::Geo<256>::smem; }
static int fa_nq(int D) { return D == 256 ? 1 : 2; }

static int launch_fa(const fa::FaParams& p, int D, int mode, long long grid, cudaStream_t st) {
  fa::FaFn fn = kernel_fa(D, mode);
  if (grid > INT_MAX) return fail("grid of %lld CTAs too large", grid);
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       fa_smem(D));
  if (e != cudaSuccess) return fail("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  fa::FaParams a = p;
  void* args[] = {&a};
  e = cudaLaunchKernel(reinterpret_cast<const void*>(fn), dim3(static_cast<unsigned>(grid)), dim3(fa::kThreads), args,
                       fa_smem(D), st);
  if (e != cudaSuccess) return fail("kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

// The caller's workspace, or the library's own for the current device.
static unsigned char* take_workspace(void* workspace, size_t bytes, size_t need, cudaStream_t st, size_t* got) {
  if (workspace) {
    if (bytes < need) {
      fail("workspace of %zu bytes is smaller than the %zu bytes needed", bytes, need);
      return nullptr;
    }
    if (!aligned(workspace, 256)) {
      fail("workspace must be 256-byte aligned");
      return nullptr;
    }
    *got = bytes;
    return static_cast<unsigned char*>(workspace);
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    fail("no CUDA device");
    return nullptr;
  }
  void* w = internal_workspace(dev, need, st, got);
  if (!w) fail("cannot allocate a %zu-byte workspace", need);
  return static_cast<unsigned char*>(w);
}

static bool rows16(const vsk_tensor* t, int e) {
  return aligned(t->data, 16) && (t->stride[0] * e) % 16 == 0 && (t->stride[1] * e) % 16 == 0;
}
static bool rows4(const vsk_tensor* t) { return aligned(t->data, 4) && t->stride[0] % 2 == 0 && t->stride[1] % 2 == 0; }

static double softmax_scale(float sm_scale, long long D) {
  return (sm_scale > 0.f && std::isfinite(sm_scale)) ? static_cast<double>(sm_scale)
                                                     : 1.0 / std::sqrt(static_cast<double>(D));
}
constexpr double kLog2e = 1.4426950408889634;

// ---- shared prefix: how its keys are cut ----
// Row blocks x KV heads of work, each cut into key ranges of whole tiles.  An
// item costs its tiles plus about kItemTiles tiles' time to start and drain,
// and the items run in waves of one per SM: the cut with the least waves x
// cost is taken.
constexpr long long kItemTiles = 4;
struct SharedCut {
  int tpb, nq;
  long long blocks, units, tiles, n_split, split_tiles;
};
static SharedCut shared_cut(long long n_rows, long long gq, long long h_kv, long long D, long long n_keys, int sms) {
  SharedCut c;
  c.tpb = static_cast<int>(128 / gq);
  c.nq = fa_nq(static_cast<int>(D));
  c.blocks = (n_rows + c.nq * c.tpb - 1) / (c.nq * c.tpb);
  c.units = c.blocks * h_kv;
  c.tiles = (n_keys + fa::KT - 1) / fa::KT;
  c.n_split = 1;
  long long best = LLONG_MAX;
  for (long long ns = 1; ns <= std::max(1LL, std::min(c.tiles, 2LL * sms / std::max(1LL, c.units))); ++ns) {
    const long long per = (c.tiles + ns - 1) / ns;
    const long long cost = (c.units * ns + sms - 1) / sms * (per + kItemTiles);
    if (cost < best) {
      best = cost;
      c.n_split = ns;
    }
  }
  c.split_tiles = (c.tiles + c.n_split - 1) / c.n_split;
  return c;
}
static size_t shared_partial_bytes(long long items, int nq, long long D) {
  return align256(4 * static_cast<size_t>(items) * 128 * nq) + align256(4 * static_cast<size_t>(items) * 128 * nq * D);
}

static size_t shared_workspace_for_sms(int sms, long long max_bs, long long h_q, long long h_kv, long long D,
                                       long long L) {
  const size_t own = vsk_workspace_size_for_sms(sms, max_bs, h_q, h_kv, D, D, L);
  if (own == 0 || h_q / h_kv > 128) return 0;
  const SharedCut c = shared_cut(max_bs * L, h_q / h_kv, h_kv, D, 1, sms);
  return own + shared_partial_bytes(std::max(c.units, 2LL * sms), c.nq, D);
}

}  // namespace vsk

using namespace vsk;

extern "C" {

int prompt_attn_fwd(const vsk_tensor* q, const vsk_tensor* k, const vsk_tensor* v, const vsk_tensor* o,
                    const vsk_tensor* qo_indptr, float sm_scale, void* workspace, size_t workspace_bytes,
                    void* stream) {
  clear_error();
  if (!check_3d(q, "q") || !check_3d(k, "k") || !check_3d(v, "v") || !check_3d(o, "o") ||
      !check_1d(qo_indptr, "qo_indptr"))
    return 0;
  for (const vsk_tensor* t : {q, k, v, o})
    if (t->dtype != VSK_DTYPE_BF16) return fail("q, k, v and o must be bf16");
  if (qo_indptr->dtype != VSK_DTYPE_I32) return fail("qo_indptr must be int32");
  const long long N = q->shape[0], h_q = q->shape[1], D = q->shape[2], h_kv = k->shape[1];
  const long long B = qo_indptr->shape[0] - 1;
  if (B < 1) return fail("batch size must be >= 1");
  if (h_kv < 1 || h_q < 1 || h_q % h_kv != 0) return fail("h_q (%lld) is not a multiple of h_kv (%lld)", h_q, h_kv);
  if (D != 64 && D != 128 && D != 256) return fail("head_dim %lld not in {64, 128, 256}", D);
  if (k->shape[0] != N || v->shape[0] != N || v->shape[1] != h_kv || k->shape[2] != D || v->shape[2] != D)
    return fail("k and v must be [%lld, h_kv, %lld]", N, D);
  if (o->shape[0] != N || o->shape[1] != h_q || o->shape[2] != D) return fail("o must have the shape of q");
  if (h_q / h_kv > 128) return fail("h_q / h_kv = %lld exceeds 128", h_q / h_kv);
  if (N > INT_MAX) return fail("%lld rows exceed 2^31 - 1", N);
  if (!rows16(k, 2) || !rows16(v, 2)) return fail("k and v rows must be 16-byte aligned");
  if (!rows4(q) || !rows4(o)) return fail("q and o must be 4-byte aligned with even strides");
  if (!aligned(qo_indptr->data, 4)) return fail("qo_indptr must be 4-byte aligned");
  if (workspace && workspace_bytes < 256) return fail("workspace of %zu bytes is smaller than 256", workspace_bytes);
  if (N == 0) return 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  unsigned char* ws = take_workspace(workspace, workspace_bytes, 256, st, &ws_bytes);
  if (!ws) return 0;
  fa::FaParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  p.q_s0 = q->stride[0];
  p.q_s1 = q->stride[1];
  p.k = static_cast<const unsigned char*>(k->data);
  p.k_s0 = 2 * k->stride[0];
  p.k_s1 = 2 * k->stride[1];
  p.v = static_cast<const unsigned char*>(v->data);
  p.v_s0 = 2 * v->stride[0];
  p.v_s1 = 2 * v->stride[1];
  p.o = static_cast<__nv_bfloat16*>(const_cast<void*>(o->data));
  p.o_s0 = o->stride[0];
  p.o_s1 = o->stride[1];
  p.qo = static_cast<const int*>(qo_indptr->data);
  p.B = static_cast<int>(B);
  p.n_rows = N;
  p.h_kv = static_cast<int>(h_kv);
  p.gq = static_cast<int>(h_q / h_kv);
  p.tpb = 128 / p.gq;
  p.scale2 = static_cast<float>(softmax_scale(sm_scale, D) * kLog2e);
  p.q16 = rows16(q, 2);
  p.o16 = rows16(o, 2);
  p.v_scale = 1.f;
  p.err = reinterpret_cast<unsigned*>(ws);
  // every sequence adds at most one row block to its share of N / block
  const long long blocks = N / (fa_nq(static_cast<int>(D)) * p.tpb) + B;
  return launch_fa(p, static_cast<int>(D), fa::kPrompt, blocks * h_kv, st);
}

size_t vsk_shared_workspace_size(int64_t max_bs, int64_t h_q, int64_t h_kv, int64_t head_dim, int64_t max_len_extend) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int sms = device_sms(dev);
  if (sms <= 0 || h_kv <= 0) return 0;
  const size_t own = vsk_workspace_size(max_bs, h_q, h_kv, head_dim, head_dim, max_len_extend);
  const size_t need = shared_workspace_for_sms(sms, max_bs, h_q, h_kv, head_dim, max_len_extend);
  if (own == 0 || need == 0) return 0;
  return need + own - vsk_workspace_size_for_sms(sms, max_bs, h_q, h_kv, head_dim, head_dim, max_len_extend);
}

int verify_splitkv_shared_fwd(const vsk_tensor* q, const vsk_tensor* ke, const vsk_tensor* ve, const vsk_tensor* o,
                              const vsk_tensor* kb, const vsk_tensor* vb, const vsk_tensor* qo, const vsk_tensor* kvp,
                              const vsk_tensor* kvi, const vsk_tensor* shi, int64_t max_len_extend, float k_scale,
                              float v_scale, float sm_scale, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  Params p;
  CallShape cs;
  if (!prepare_verify(q, ke, ve, o, kb, vb, qo, kvp, kvi, 1, max_len_extend, k_scale, v_scale, sm_scale, nullptr,
                      nullptr, nullptr, p, cs))
    return 0;
  if (cs.D != cs.DV) return fail("head_dim %lld and v_head_dim %lld must be equal", cs.D, cs.DV);
  if (!check_1d(shi, "shared_indices")) return 0;
  if (shi->dtype != VSK_DTYPE_I32 && shi->dtype != VSK_DTYPE_I64) return fail("shared_indices must be int32 or int64");
  if (!aligned(shi->data, shi->dtype == VSK_DTYPE_I64 ? 8 : 4)) return fail("shared_indices must be aligned to its type");
  if (cs.B * cs.L > INT_MAX) return fail("%lld rows exceed 2^31 - 1", cs.B * cs.L);
  const int D = static_cast<int>(cs.D);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail("cudaGetDevice: %s", cudaGetErrorString(e));
  const int sms = device_sms(dev);
  if (sms <= 0) return fail("cannot query the SM count of device %d", dev);
  const bool has_own = kvi->shape[0] > 0, has_shared = shi->shape[0] > 0;
  StreamOnly so;
  if (!plan_stream_only(cs, so)) return 0;
  const long long gq = cs.h_q / cs.h_kv;
  const SharedCut c = shared_cut(cs.B * cs.L, gq, cs.h_kv, cs.D, shi->shape[0], sms);
  // the own pieces as the stream lays them out, the shared partials behind
  // them, the tickets of other calls at the end of the buffer
  const long long items = c.units * c.n_split;
  const size_t base = so.wl.total - so.wl.cnt_bytes;
  const size_t sh_o = base + align256(4 * static_cast<size_t>(items) * 128 * c.nq);
  const size_t need = base + shared_partial_bytes(items, c.nq, cs.D) + so.wl.cnt_bytes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  unsigned char* ws = take_workspace(workspace, workspace_bytes, need, st, &ws_bytes);
  if (!ws) return 0;

  const float scale2 = p.scale2;
  ScParams s;
  s.has_own = has_own;
  if (has_own && !launch_stream_only(p, cs, so, ws, ws_bytes, st)) return 0;
  if (has_shared) {
    fa::FaParams f;
    memset(&f, 0, sizeof f);
    f.q = p.q;
    f.q_s0 = p.q_s0;
    f.q_s1 = p.q_s1;
    f.k = p.kb;
    f.k_s0 = p.kb_s0;
    f.k_s1 = p.kb_s1;
    f.v = p.vb;
    f.v_s0 = p.vb_s0;
    f.v_s1 = p.vb_s1;
    f.B = static_cast<int>(cs.B);
    f.n_rows = p.n_rows;
    f.idx = shi->data;
    f.idx64 = shi->dtype == VSK_DTYPE_I64;
    f.n_keys = shi->shape[0];
    f.pool = p.pool;
    f.h_kv = static_cast<int>(cs.h_kv);
    f.gq = static_cast<int>(gq);
    f.tpb = c.tpb;
    f.n_split = static_cast<int>(c.n_split);
    f.split_tiles = static_cast<int>(c.split_tiles);
    // the kernel takes the maximum of the unscaled scores: a negative scale
    // goes into the queries' signs, a zero one makes them zero
    f.qmode = scale2 > 0.f ? 0 : scale2 < 0.f ? 1 : 2;
    f.scale2 = scale2 == 0.f ? 1.f : std::fabs(scale2);
    f.q16 = rows16(q, 2);
    f.v_scale = v_scale;
    f.err = reinterpret_cast<unsigned*>(ws);
    f.plse = reinterpret_cast<float*>(ws + base);
    f.po = reinterpret_cast<float*>(ws + sh_o);
    if (!launch_fa(f, D, cs.fp8 ? fa::kSharedE4m3 : fa::kSharedBf16, items, st)) return 0;
  }
  p.B = static_cast<int>(cs.B);
  p.L = static_cast<int>(cs.L);
  p.gq = so.pl.gq;
  p.R = so.pl.R;
  p.HC = so.pl.HC;
  p.MT = so.pl.MT;
  p.n_hg = so.pl.n_hg;
  p.err = reinterpret_cast<unsigned*>(ws);
  s.v = p;
  s.n_split = static_cast<int>(c.n_split);
  s.n_live = has_shared ? static_cast<int>((c.tiles + c.split_tiles - 1) / c.split_tiles) : 0;
  s.h_kv = static_cast<int>(cs.h_kv);
  s.tpb = c.tpb;
  s.nq = c.nq;
  s.splse = reinterpret_cast<const float*>(ws + base);
  s.spo = reinterpret_cast<const float*>(ws + sh_o);
  const long long grid = cs.B * cs.h_kv * so.pl.MT * (D / 32);
  if (grid > INT_MAX) return fail("grid of %lld CTAs too large", grid);
  const void* fn = D == 64 ? reinterpret_cast<const void*>(shared_combine_kernel<64>)
                 : D == 128 ? reinterpret_cast<const void*>(shared_combine_kernel<128>)
                            : reinterpret_cast<const void*>(shared_combine_kernel<256>);
  void* args[] = {&s};
  e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(128), args, 0, st);
  if (e != cudaSuccess) return fail("combine kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

}  // extern "C"
