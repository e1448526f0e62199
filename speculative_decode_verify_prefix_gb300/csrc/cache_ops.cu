// Host side of the calls around the verify call: attention over whole prompts
// (prompt_attn_fwd), the verify call for a batch that shares a long prefix
// (verify_splitkv_shared_fwd), the attention weight of the cached keys
// (verify_splitkv_mass) and the eviction that goes by it (kv_evict).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <set>
#include <tuple>

#include "flash_tc.cuh"
#include "key_mass.cuh"
#include "kv_evict.cuh"
#include "shared_combine.cuh"
#include "verify_host.cuh"

namespace vsk {

fa::FaFn kernel_fa(int D, int mode) {
  return D == 64 ? kernel_fa_64(mode) : D == 128 ? kernel_fa_128(mode) : D == 256 ? kernel_fa_256(mode) : nullptr;
}

static int fa_smem(int D) { return D == 64 ? fa::Geo<64>::smem : D == 128 ? fa::Geo<128>::smem : fa::Geo<256>::smem; }
constexpr size_t kSchedOff = 64;  // fa_kernel's counters, between the error word and the partials
static int fa_nq(int D) { return D == 256 ? 1 : 2; }

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    cudaGetLastError();
  });
  return encode;
}

// Tensor map of bf16 rows [rows][heads][D] for boxes of [n_rows][n_heads][64
// columns] in the 128-byte swizzle.  False where base or strides are none that
// a map takes (the rows are then copied without one).
static bool rows_map(const vsk_tensor* t, int n_rows, int n_heads, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  // a dimension of one element has any stride
  const long long n = t->shape[0], h = t->shape[1], d = t->shape[2];
  const long long s1 = h > 1 ? t->stride[1] : d, s0 = n > 1 ? t->stride[0] : h * s1;
  if (!encode || !rows16(t, 2) || s1 < d || s0 < d || s0 >= (1LL << 38) || s1 >= (1LL << 38)) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(h), static_cast<cuuint64_t>(n)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * s1), static_cast<cuuint64_t>(2 * s0)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(n_heads), static_cast<cuuint32_t>(n_rows)}, unit[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(t->data), dims, strides, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for gathers of four pool rows of 64 columns at a time: a pool row
// (all its heads) is a row of the map.
static bool pool_map(const vsk_tensor* t, CUtensorMap* map) {
  const long long n = t->shape[0], h = t->shape[1], d = t->shape[2];
  const long long row = (h > 1 ? (h - 1) * t->stride[1] : 0) + d, s0 = n > 1 ? t->stride[0] : row;
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (!encode || n > INT_MAX || row > INT_MAX || s0 < row || s0 >= (1LL << 38)) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(n)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * s0)};
  const cuuint32_t box[2] = {64, 1}, unit[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(t->data), dims, strides, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One CTA per SM at most; maps: queries, K, V.  beside: the grid may start while
// the kernel before it on the stream runs (it needs nothing of that kernel, and
// completes after it).
static int launch_fa(const fa::FaParams& p, const CUtensorMap* maps, int D, int mode, long long n_items, void* ws,
                     bool beside, cudaStream_t st) {
  fa::FaFn fn = kernel_fa(D, mode);
  if (n_items > INT_MAX / 2) return fail("%lld row blocks are too many", n_items);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail("cudaGetDevice: %s", cudaGetErrorString(e));
  const int sms = device_sms(dev);
  if (sms <= 0) return fail("cannot query the SM count of device %d", dev);
  {
    static std::mutex mu;
    static std::set<std::pair<int, const void*>> done;  // (device, kernel) whose attribute is set
    std::lock_guard<std::mutex> lk(mu);
    const std::pair<int, const void*> key{dev, reinterpret_cast<const void*>(fn)};
    if (!done.count(key)) {
      e = cudaFuncSetAttribute(key.second, cudaFuncAttributeMaxDynamicSharedMemorySize, fa_smem(D));
      if (e != cudaSuccess) return fail("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      done.insert(key);
    }
  }
  fa::FaParams a = p;
  a.n_items = static_cast<int>(n_items);
  a.err = static_cast<unsigned*>(ws);
  a.sched = reinterpret_cast<int*>(static_cast<unsigned char*>(ws) + kSchedOff);
  CUtensorMap m[3];
  memcpy(m, maps, sizeof m);
  void* args[] = {&a, &m[0], &m[1], &m[2]};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(n_items, sms)));
  cfg.blockDim = dim3(D == 256 || mode != fa::kPrompt ? fa::Cfg<256, 0>::threads : fa::Cfg<128, 0>::threads);
  cfg.dynamicSmemBytes = fa_smem(D);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = beside ? 1 : 0;
  e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(fn), args);
  if (e != cudaSuccess) return fail("kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

// The caller's workspace, or the library's own for the current device.
unsigned char* take_workspace(void* workspace, size_t bytes, size_t need, cudaStream_t st, size_t* got) {
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

bool rows16(const vsk_tensor* t, int e) {
  return aligned(t->data, 16) && (t->stride[0] * e) % 16 == 0 && (t->stride[1] * e) % 16 == 0;
}
bool rows4(const vsk_tensor* t) { return aligned(t->data, 4) && t->stride[0] % 2 == 0 && t->stride[1] % 2 == 0; }

double softmax_scale(float sm_scale, long long D) {
  return (sm_scale > 0.f && std::isfinite(sm_scale)) ? static_cast<double>(sm_scale)
                                                     : 1.0 / std::sqrt(static_cast<double>(D));
}
// An infinite scale makes every score infinite or NaN.
static bool check_scales(const Params& p) {
  if (!std::isfinite(p.dscale2)) return fail("sm_scale is too large");
  if (!std::isfinite(p.scale2)) return fail("sm_scale * k_scale is too large");
  return true;
}

// ---- shared prefix: how the work is cut ----
// The key tiles of the units (row blocks x KV heads) are laid end to end and
// every CTA (one per SM) takes the same number of them, at least kMinShare: a
// shorter piece costs more to start, write and join than its tiles.  Piece of
// CTA c and unit u: partial c + u.
constexpr long long kMinShare = 2;
struct SharedCut {
  int tpb, nq;
  long long units, tiles, share, n_cta, pieces;
};
static SharedCut shared_cut(long long n_rows, long long gq, long long h_kv, long long D, long long n_keys, int sms) {
  SharedCut c;
  c.tpb = static_cast<int>(128 / gq);
  c.nq = fa_nq(static_cast<int>(D));
  c.units = (n_rows + c.nq * c.tpb - 1) / (c.nq * c.tpb) * h_kv;
  c.tiles = (n_keys + fa::KT - 1) / fa::KT;
  const long long total = c.units * c.tiles;
  c.share = std::max(kMinShare, (total + sms - 1) / sms);
  c.n_cta = (total + c.share - 1) / c.share;
  c.pieces = c.n_cta + c.units;
  return c;
}
static size_t shared_partial_bytes(long long pieces, int nq, long long D) {
  return align256(4 * static_cast<size_t>(pieces) * 128 * nq) + align256(4 * static_cast<size_t>(pieces) * 128 * nq * D);
}

static size_t shared_workspace_for_sms(int sms, long long max_bs, long long h_q, long long h_kv, long long D,
                                       long long L) {
  const size_t own = vsk_workspace_size_for_sms(sms, max_bs, h_q, h_kv, D, D, L);
  if (own == 0 || h_q < 1 || h_q / h_kv > 128) return 0;
  const SharedCut c = shared_cut(max_bs * L, h_q / h_kv, h_kv, D, 1, sms);
  return own + shared_partial_bytes(c.units + sms, c.nq, D);
}

// ---- one thread-block cluster per segment ----
// The largest cluster of at most c CTAs (c, then 8 or fewer by halves) of which
// one fits on the current device; asked from the runtime once per shape (the
// query costs several microseconds).  0: none fits.
static int cluster_fit(const void* fn, int c, int threads, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail("no CUDA device");
  static std::mutex mu;
  static std::map<std::tuple<int, const void*, int, int, size_t>, int> known;
  std::lock_guard<std::mutex> lk(mu);
  int& fit = known[{dev, fn, c, threads, smem}];
  if (fit > 0) return fit;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerCTAMax - 4096);
  if (e != cudaSuccess) return fail("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  if (c > 8 && cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    cudaGetLastError();
    c = 8;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  for (; c >= 1; c = c > 8 ? 8 : c / 2) {
    at[0].val.clusterDim.x = static_cast<unsigned>(c);
    cfg.gridDim = dim3(static_cast<unsigned>(c));
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess && n >= 1) return fit = c;
    cudaGetLastError();  // clear the error the query left
  }
  return fail("a cluster of one CTA does not fit");
}

static int launch_clusters(const void* fn, int c, long long n_seg, int threads, size_t smem, void** args,
                           cudaStream_t st) {
  c = cluster_fit(fn, c, threads, smem);
  if (c == 0) return 0;
  if (n_seg * c > INT_MAX) return fail("grid of %lld CTAs too large", n_seg * c);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(c);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(n_seg * c));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  if (e != cudaSuccess) return fail("kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

// Eviction: a CTA's slice of a sequence of the mean length holds at most 8192
// keys (64 sequences of mean 21,400: 46 us, with 2048 89), unless the cluster
// would pass 16 CTAs; but less, down to 512, while two CTAs an SM have not been
// given out: 8 sequences of 40,000 keys 29 us instead of 35, one of 131,072 among
// 63 of 1000 281 instead of 1188 (lengths are not known here).
static int evict_cluster(long long mean_len, long long n_seq, int sms) {
  int c = 1;
  while (c < 16 && (mean_len > c * 8192LL || (n_seq * c <= sms && mean_len > c * 512LL))) c *= 2;
  return c;
}
// Key weights: the smallest cluster whose CTAs keep the scores of a mean
// segment (or nearly: what does not fit is computed again), since a CTA costs
// some 9 us beside its keys and larger clusters leave more SMs without a place
// (128 sequences of 8,000 keys: 8 CTAs 760 us, 12 915, 16 1203; the serving
// batch, mean 21,400: 8 1120, 12 1072, 14 1373, 16 1213); but more, down to 256
// keys each, while the GPU is not full.
static int mass_cluster(long long mean_len, long long cap, long long n_seg, int sms) {
  constexpr int kSizes[] = {1, 2, 4, 6, 8, 12, 16};
  size_t i = 0;
  while (kSizes[i] < 16 && 10 * mean_len > 12 * kSizes[i] * cap) ++i;
  while (kSizes[i] < 16 && n_seg * kSizes[i] < 2LL * sms && mean_len > 256LL * kSizes[i]) ++i;
  return kSizes[i];
}

// The cluster kernels hold positions in kv_indices in 32 bits and step past the
// last one by a cluster's or a chunk's worth.
constexpr long long kMaxEntries = INT_MAX - 65535LL;

static bool check_rows(const vsk_tensor* t, const char* name, long long rows) {
  if (!check_2d(t, name)) return false;
  if (t->dtype != VSK_DTYPE_F32) return fail("%s must be float32", name);
  if (t->shape[0] != rows) return fail("%s must have one row per KV head (%lld)", name, rows);
  if (!aligned(t->data, 4)) return fail("%s must be 4-byte aligned", name);
  return true;
}

// The memory of a 1-d or 2-d view: n rows of `bytes` bytes, `pitch` bytes apart.
struct RowSpan {
  uintptr_t at;
  long long n, bytes, pitch;
};
static RowSpan row_span(const vsk_tensor* t, long long e) {
  RowSpan r{reinterpret_cast<uintptr_t>(t->data), 1, e * t->shape[t->ndim - 1], 0};
  if (t->ndim == 2 && t->shape[0] != 1) {
    r.n = t->shape[0];
    r.pitch = e * t->stride[0];
    if (r.pitch < 0) {  // the same rows from the lowest one on
      r.at += static_cast<uintptr_t>((r.n - 1) * r.pitch);
      r.pitch = -r.pitch;
    }
  }
  if (r.bytes == 0) r.n = 0;
  return r;
}
static bool rows_overlap(const RowSpan& x) { return x.n > 1 && x.pitch < x.bytes; }
// whether a row of x and one of y share a byte
static bool rows_meet(const RowSpan& x, const RowSpan& y) {
  if (x.n == 0 || y.n == 0) return false;
  const long long base = static_cast<long long>(x.at - y.at);
  for (long long i = 0; i < x.n; ++i) {
    const long long a = base + i * x.pitch;  // this row against the rows at 0, y.pitch, ...
    if (a + x.bytes <= 0 || a >= (y.n - 1) * y.pitch + y.bytes) continue;
    // of the rows that begin before this one ends the last one ends last
    const long long j = y.pitch > 0 ? std::min(y.n - 1, (a + x.bytes - 1) / y.pitch) : 0;
    if (a < j * y.pitch + y.bytes) return true;
  }
  return false;
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
  if (N > INT_MAX - 1024) return fail("%lld rows are too many (2^31 - 1025 at most)", N);
  if (!rows16(k, 2) || !rows16(v, 2)) return fail("k and v rows must be 16-byte aligned");
  if (!rows4(q) || !rows4(o)) return fail("q and o must be 4-byte aligned with even strides");
  if (!aligned(qo_indptr->data, 4)) return fail("qo_indptr must be 4-byte aligned");
  if (!std::isfinite(static_cast<float>(softmax_scale(sm_scale, D) * kLog2e))) return fail("sm_scale is too large");
  if (workspace && workspace_bytes < 256) return fail("workspace of %zu bytes is smaller than 256", workspace_bytes);
  if (N == 0) return 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  WorkspaceHold hold(workspace);
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
  if (p.scale2 == 0.f) {  // below the smallest float: all scores alike
    p.qmode = 2;
    p.scale2 = 1.f;
  }
  p.q16 = rows16(q, 2);
  p.o16 = rows16(o, 2);
  p.v_scale = 1.f;
  // every sequence adds at most one row block to its share of N / block
  const long long blocks = N / (fa_nq(static_cast<int>(D)) * p.tpb) + B;
  CUtensorMap maps[3];
  memset(maps, 0, sizeof maps);
  p.qtma = p.qmode == 0 && rows_map(q, p.tpb, p.gq, &maps[0]);
  p.tma = rows_map(k, 32, 1, &maps[1]) && rows_map(v, 32, 1, &maps[2]);
  return launch_fa(p, maps, static_cast<int>(D), fa::kPrompt, blocks * h_kv, ws, false, st);
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
  if (cs.h_q < 1) return fail("h_q must be >= 1");
  if (cs.D != cs.DV) return fail("head_dim %lld and v_head_dim %lld must be equal", cs.D, cs.DV);
  if (!check_1d(shi, "shared_indices")) return 0;
  if (shi->dtype != VSK_DTYPE_I32 && shi->dtype != VSK_DTYPE_I64) return fail("shared_indices must be int32 or int64");
  if (!aligned(shi->data, shi->dtype == VSK_DTYPE_I64 ? 8 : 4)) return fail("shared_indices must be aligned to its type");
  if (cs.B * cs.L > INT_MAX - 1024) return fail("%lld rows are too many (2^31 - 1025 at most)", cs.B * cs.L);
  if (!check_scales(p)) return 0;
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
  const size_t base = so.wl.total - so.wl.cnt_bytes;
  const size_t sh_o = base + align256(4 * static_cast<size_t>(c.pieces) * 128 * c.nq);
  const size_t need = base + shared_partial_bytes(c.pieces, c.nq, cs.D) + so.wl.cnt_bytes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  WorkspaceHold hold(workspace);
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
    f.n_units = c.units;
    f.share = c.share;
    // the kernel takes the maximum of the unscaled scores: a negative scale
    // goes into the queries' signs, a zero one makes them zero
    f.qmode = scale2 > 0.f ? 0 : scale2 < 0.f ? 1 : 2;
    f.scale2 = scale2 == 0.f ? 1.f : std::fabs(scale2);
    f.q16 = rows16(q, 2);
    f.v_scale = v_scale;
    f.plse = reinterpret_cast<float*>(ws + base);
    f.po = reinterpret_cast<float*>(ws + sh_o);
    CUtensorMap maps[3];
    memset(maps, 0, sizeof maps);
    f.qtma = f.qmode == 0 && rows_map(q, f.tpb, f.gq, &maps[0]);
    f.tma = !cs.fp8 && pool_map(kb, &maps[1]) && pool_map(vb, &maps[2]);
    if (!launch_fa(f, maps, D, cs.fp8 ? fa::kSharedE4m3 : fa::kSharedBf16, c.n_cta, ws, has_own, st)) return 0;
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
  s.tiles = has_shared ? c.tiles : 0;
  s.share = c.share;
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
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = at;
  // starting under fa_kernel's end saves 1.5 us (four short sequences 17.0 ->
  // 15.6) to 8 (32 own prefixes of 100 to 200 keys behind 16,384 e4m3 rows, 16/2
  // heads of 256: 110 -> 101)
  cfg.numAttrs = has_shared ? 1 : 0;
  e = cudaLaunchKernelExC(&cfg, fn, args);
  if (e != cudaSuccess) return fail("combine kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

int verify_splitkv_mass(const vsk_tensor* q, const vsk_tensor* ke, const vsk_tensor* kb, const vsk_tensor* qo,
                        const vsk_tensor* kvp, const vsk_tensor* kvi, const vsk_tensor* mass_in,
                        const vsk_tensor* mass, int64_t max_len_extend, float k_scale, float sm_scale, void* workspace,
                        size_t workspace_bytes, void* stream) {
  clear_error();
  Params p;
  CallShape cs;
  if (!prepare_verify(q, ke, ke, q, kb, kb, qo, kvp, kvi, 1, max_len_extend, k_scale, 1.f, sm_scale, nullptr, nullptr,
                      nullptr, p, cs, true))
    return 0;
  const long long T = kvi->shape[0];
  if (T > kMaxEntries) return fail("%lld kv_indices entries are too many (%lld at most)", T, kMaxEntries);
  if (!check_scales(p)) return 0;
  if (!check_rows(mass, "mass", cs.h_kv)) return 0;
  if (mass->shape[1] != T) return fail("mass must have one column per kv_indices entry (%lld)", T);
  if (mass_in) {
    if (!check_rows(mass_in, "mass_in", cs.h_kv)) return 0;
    if (mass_in->shape[1] != T) return fail("mass_in must have one column per kv_indices entry (%lld)", T);
    const bool same = mass_in->data == mass->data && (cs.h_kv == 1 || mass_in->stride[0] == mass->stride[0]);
    if (!same && rows_meet(row_span(mass, 4), row_span(mass_in, 4))) return fail("mass overlaps mass_in");
  }
  if (rows_overlap(row_span(mass, 4))) return fail("rows of mass overlap");
  if (kb->shape[0] >= 0xFFFFFFFFLL) return fail("a pool of %lld rows is too large", static_cast<long long>(kb->shape[0]));
  if (T == 0) return 1;
  if (kb->shape[0] == 0) return fail("k_buffer has no rows");
  km::MassParams m;
  memset(&m, 0, sizeof m);
  m.h_kv = static_cast<int>(cs.h_kv);
  m.MT = static_cast<int>(((cs.h_q / cs.h_kv) * cs.L + 15) / 16);
  const int rows = static_cast<int>((cs.h_q / cs.h_kv) * cs.L);
  m.x_off = 16 * m.MT * static_cast<int>(cs.D) * 2;
  m.i_off = m.x_off + (16 * rows * 8 + 127) / 128 * 128;
  m.cap = (km::kSmem - m.i_off) / (4 * rows + 4) - 8;
  m.cap = m.cap / 32 * 32;
  m.s_off = m.i_off + 4 * m.cap;
  m.pitch = m.cap + 8;  // 8 mod 32 floats: the four row groups of a fragment store meet different banks
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  WorkspaceHold hold(workspace);
  unsigned char* ws = take_workspace(workspace, workspace_bytes, 256, st, &ws_bytes);
  if (!ws) return 0;
  p.B = static_cast<int>(cs.B);
  p.L = static_cast<int>(cs.L);
  p.gq = static_cast<int>(cs.h_q / cs.h_kv);
  p.R = rows;
  p.err = reinterpret_cast<unsigned*>(ws);
  m.v = p;
  m.in = mass_in ? static_cast<const float*>(mass_in->data) : nullptr;
  m.in_s0 = mass_in ? mass_in->stride[0] : 0;
  m.out = static_cast<float*>(const_cast<void*>(mass->data));
  m.out_s0 = mass->stride[0];
  void* args[] = {&m};
  const size_t smem = m.s_off + static_cast<size_t>(m.pitch) * 4 * rows;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail("no CUDA device");
  const int sms = device_sms(dev);
  if (sms <= 0) return fail("cannot query the SM count of device %d", dev);
  const km::MassFn fn = kernel_mass(static_cast<int>(cs.D), cs.fp8, m.MT == 1 && cs.D <= 128);
  return launch_clusters(reinterpret_cast<const void*>(fn), mass_cluster(cs.mean_len, m.cap, cs.B * cs.h_kv, sms),
                         cs.B * cs.h_kv, km::kThreads, smem, args, st);
}

int kv_evict(const vsk_tensor* mass, const vsk_tensor* kvp, const vsk_tensor* kvi, int64_t budget, int64_t recent,
             const vsk_tensor* out_kvp, const vsk_tensor* out_kvi, const vsk_tensor* out_mass,
             const vsk_tensor* freed, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  if (!check_1d(kvp, "kv_indptr") || !check_1d(kvi, "kv_indices") || !check_1d(out_kvp, "out_kv_indptr") ||
      !check_1d(out_kvi, "out_kv_indices") || !check_1d(freed, "freed") || !check_2d(mass, "mass"))
    return 0;
  const long long B = kvp->shape[0] - 1, T = kvi->shape[0], h_kv = mass->shape[0];
  if (B < 1) return fail("batch size must be >= 1");
  if (T > kMaxEntries) return fail("%lld kv_indices entries are too many (%lld at most)", T, kMaxEntries);
  if (kvp->dtype != VSK_DTYPE_I32 || out_kvp->dtype != VSK_DTYPE_I32) return fail("indptr arrays must be int32");
  if (out_kvp->shape[0] != B + 1) return fail("out_kv_indptr must have B+1 entries");
  if (kvi->dtype != VSK_DTYPE_I32 && kvi->dtype != VSK_DTYPE_I64) return fail("kv_indices must be int32 or int64");
  if (out_kvi->dtype != kvi->dtype || freed->dtype != kvi->dtype)
    return fail("out_kv_indices and freed must have the type of kv_indices");
  const size_t ei = kvi->dtype == VSK_DTYPE_I64 ? 8 : 4;
  if (!aligned(kvi->data, ei) || !aligned(out_kvi->data, ei) || !aligned(freed->data, ei) || !aligned(kvp->data, 4) ||
      !aligned(out_kvp->data, 4))
    return fail("index arrays must be aligned to their type");
  if (h_kv < 1) return fail("mass must have one row per KV head");
  if (!check_rows(mass, "mass", h_kv) || !check_rows(out_mass, "out_mass", h_kv)) return 0;
  if (mass->shape[1] != T) return fail("mass must have one column per kv_indices entry (%lld)", T);
  if (out_mass->shape[1] != out_kvi->shape[0]) return fail("out_mass must have one column per out_kv_indices entry");
  if (budget < 1) return fail("budget must be >= 1");
  if (recent < 0 || recent > budget) return fail("recent must be in [0, budget]");
  // the kernel packs while it reads
  if (rows_overlap(row_span(out_mass, 4))) return fail("rows of out_mass overlap");
  struct Named { const char* name; RowSpan span; };
  const Named ins[] = {{"kv_indptr", row_span(kvp, 4)}, {"kv_indices", row_span(kvi, static_cast<long long>(ei))},
                       {"mass", row_span(mass, 4)}};
  const Named outs[] = {{"out_kv_indptr", row_span(out_kvp, 4)}, {"out_kv_indices", row_span(out_kvi, static_cast<long long>(ei))},
                        {"out_mass", row_span(out_mass, 4)}, {"freed", row_span(freed, static_cast<long long>(ei))}};
  for (const Named& o : outs) {
    for (const Named& i : ins)
      if (rows_meet(o.span, i.span)) return fail("%s overlaps %s", o.name, i.name);
    for (const Named* x = outs; x != &o; ++x)
      if (rows_meet(o.span, x->span)) return fail("%s overlaps %s", o.name, x->name);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  WorkspaceHold hold(workspace);
  unsigned char* ws = take_workspace(workspace, workspace_bytes, 256, st, &ws_bytes);
  if (!ws) return 0;
  ev::EvictParams p;
  memset(&p, 0, sizeof p);
  p.mass = static_cast<const float*>(mass->data);
  p.mass_s0 = mass->stride[0];
  p.kvp = static_cast<const int*>(kvp->data);
  p.kvi = kvi->data;
  p.idx64 = kvi->dtype == VSK_DTYPE_I64;
  p.h_kv = static_cast<int>(h_kv);
  p.B = static_cast<int>(B);
  p.n_idx = T;
  p.budget = budget;
  p.recent = recent;
  p.out_ptr = static_cast<int*>(const_cast<void*>(out_kvp->data));
  p.out_idx = const_cast<void*>(out_kvi->data);
  p.out_mass = static_cast<float*>(const_cast<void*>(out_mass->data));
  p.out_s0 = out_mass->stride[0];
  p.freed = const_cast<void*>(freed->data);
  p.out_cap = out_kvi->shape[0];
  p.freed_cap = freed->shape[0];
  p.err = reinterpret_cast<unsigned*>(ws);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail("no CUDA device");
  const int sms = device_sms(dev);
  if (sms <= 0) return fail("cannot query the SM count of device %d", dev);
  const int c = evict_cluster(T / B, B, sms);
  // slices of up to twice the mean stay in shared memory (more costs L1 its
  // room: 64 sequences of mean 21,400 with 13,312 keys a slice 57 us, so 53)
  p.cap = static_cast<int>(std::min(24576LL, std::max(8192LL, 2 * (T / B / c + 1))));
  void* args[] = {&p};
  return launch_clusters(reinterpret_cast<const void*>(evict_kernel), c, B, ev::kThreads,
                         8 * static_cast<size_t>(p.cap), args, st);
}

}  // extern "C"
