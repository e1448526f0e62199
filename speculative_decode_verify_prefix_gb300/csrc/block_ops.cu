// Host side of the calls between the projections and the verify call: rotary
// positions (rope_fwd), the same with K and V stored into a pool of rows
// (rope_append_fwd) or a block-scaled e4m3 cache (rope_append_block_fwd), and the
// verify call over that cache (verify_splitkv_block_fwd).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>
#include <set>

#include "block_combine.cuh"
#include "rope_append.cuh"
#include "verify_host.cuh"

namespace vsk {

// ---- views that share memory ----
// n x h runs of d bytes, s0 and s1 bytes apart.
struct Runs {
  const char* name;
  uintptr_t at;
  long long n, h, d, s0, s1;
};
static Runs runs_of(const char* name, const vsk_tensor* t, long long e) {
  Runs r{name, 0, 0, 0, 0, 0, 0};
  if (!t) return r;
  r.at = reinterpret_cast<uintptr_t>(t->data);
  if (t->ndim == 3)
    r = Runs{name, r.at, t->shape[0], t->shape[1], e * t->shape[2], e * t->stride[0], e * t->stride[1]};
  else if (t->ndim == 2)
    r = Runs{name, r.at, t->shape[0], 1, e * t->shape[1], e * t->stride[0], 0};
  else
    r = Runs{name, r.at, 1, 1, e * t->shape[0], 0, 0};
  if (r.d == 0 || r.h == 0) r.n = 0;
  return r;
}
// whether two runs of one view share a byte
static bool folds(const Runs& r) {
  if (r.n == 0) return false;
  const bool rows = r.n > 1, heads = r.h > 1;
  if (rows && r.s0 < r.d) return true;
  if (heads && r.s1 < r.d) return true;
  if (!rows || !heads) return false;
  return r.s0 >= r.s1 ? r.s0 < (r.h - 1) * r.s1 + r.d : r.s1 < (r.n - 1) * r.s0 + r.d;
}
// Whether a row of an runs and a row of bn runs, each s bytes after the one before, share a
// byte; the runs are ad and bd bytes long, the first of a lies `delta` behind that of b.
static bool lines_meet(long long delta, long long an, long long bn, long long s, long long ad, long long bd) {
  if (s <= 0) return true;
  auto below = [&](long long x) { return x / s - (x % s < 0 ? 1 : 0); };  // floor(x / s)
  // run j of b against run i of a, y = j - i: -ad < delta - y s < bd
  const long long lo = std::max(below(delta - bd) + 1, 1 - an), hi = std::min(-below(-delta - ad) - 1, bn - 1);
  return lo <= hi;
}
// Whether two views share a byte.  Views of one buffer (equal strides) are told
// apart exactly; of other strides, by the ranges they lie in.  A dimension of one element
// has no stride of its own, whatever its view says.
static bool meet(Runs a, Runs b) {
  if (a.n == 0 || b.n == 0) return false;
  if (a.n == 1) a.s0 = b.n == 1 ? 0 : b.s0;
  if (b.n == 1) b.s0 = a.s0;
  if (a.h == 1) a.s1 = b.h == 1 ? 0 : b.s1;
  if (b.h == 1) b.s1 = a.s1;
  auto last = [](const Runs& r) { return r.at + static_cast<uintptr_t>((r.n - 1) * r.s0 + (r.h - 1) * r.s1 + r.d); };
  if (last(a) <= b.at || last(b) <= a.at) return false;
  if (a.s0 != b.s0 || a.s1 != b.s1) return true;
  const bool rows = a.n > 1 || b.n > 1, heads = a.h > 1 || b.h > 1;
  if (!rows && !heads) return true;
  const long long delta = static_cast<long long>(a.at - b.at);
  if (!rows) return lines_meet(delta, a.h, b.h, a.s1, a.d, b.d);
  if (!heads) return lines_meet(delta, a.n, b.n, a.s0, a.d, b.d);
  const bool rows_wide = a.s0 >= a.s1;
  const long long S = rows_wide ? a.s0 : a.s1, s = rows_wide ? a.s1 : a.s0;
  const long long aw = rows_wide ? a.n : a.h, bw = rows_wide ? b.n : b.h, an = rows_wide ? a.h : a.n, bn = rows_wide ? b.h : b.n;
  if (s <= 0 || (std::max(an, bn) - 1) * s + std::max(a.d, b.d) > S) return true;
  const long long x0 = delta / S;
  for (long long x = x0 - 1; x <= x0 + 1; ++x)  // a's runs against those of b that lie x wide strides on
    if (x > -aw && x < bw && lines_meet(delta - x * S, an, bn, s, a.d, b.d)) return true;
  return false;
}
static bool same_view(const Runs& a, const Runs& b) {
  return a.at == b.at && a.n == b.n && a.h == b.h && a.d == b.d && (a.n == 1 || a.s0 == b.s0) && (a.h == 1 || a.s1 == b.s1);
}

// ---- rotary positions and appends ----
static rp::View view_of(const vsk_tensor* t, long long e) {
  return rp::View{static_cast<unsigned char*>(const_cast<void*>(t->data)), e * t->stride[0], e * t->stride[1]};
}
static bool check_bf16_rows(const vsk_tensor* t, const char* name, long long n, long long h, long long D) {
  if (!check_3d(t, name)) return false;
  if (t->dtype != VSK_DTYPE_BF16) return fail("%s must be bf16", name);
  if (t->shape[0] != n || t->shape[1] != h || t->shape[2] != D)
    return fail("%s must be [%lld, %lld, %lld]", name, n, h, D);
  if (!rows16(t, 2)) return fail("%s rows must be 16-byte aligned", name);
  return true;
}
static bool check_index(const vsk_tensor* t, const char* name, long long n) {
  if (!check_1d(t, name)) return false;
  if (t->dtype != VSK_DTYPE_I32 && t->dtype != VSK_DTYPE_I64) return fail("%s must be int32 or int64", name);
  if (t->shape[0] != n) return fail("%s must have one entry per row (%lld)", name, n);
  if (!aligned(t->data, t->dtype == VSK_DTYPE_I64 ? 8 : 4)) return fail("%s must be aligned to its type", name);
  return true;
}

// What the three calls have in common; v: also values (null: none).
static bool prepare_rope(const vsk_tensor* q, const vsk_tensor* k, const vsk_tensor* v, const vsk_tensor* qo,
                         const vsk_tensor* ko, const vsk_tensor* pos, const vsk_tensor* freq, int interleaved, float size,
                         rp::RopeParams& p, long long& D) {
  if (!check_3d(k, "k")) return false;
  const long long N = k->shape[0], h_kv = k->shape[1];
  D = k->shape[2];
  if (D != 64 && D != 128 && D != 256) return fail("head_dim %lld not in {64, 128, 256}", D);
  if (h_kv < 1) return fail("k must have at least one head");
  if (!check_bf16_rows(k, "k", N, h_kv, D)) return false;
  if ((q == nullptr) != (qo == nullptr)) return fail("q and q_out go together");
  if (q) {
    if (!check_3d(q, "q")) return false;
    if (q->shape[1] < 1) return fail("q must have at least one head");
    if (!check_bf16_rows(q, "q", N, q->shape[1], D) || !check_bf16_rows(qo, "q_out", N, q->shape[1], D)) return false;
  }
  if (ko && !check_bf16_rows(ko, "k_out", N, h_kv, D)) return false;
  if (v && !check_bf16_rows(v, "v", N, h_kv, D)) return false;
  if (!check_index(pos, "positions", N)) return false;
  if (!check_1d(freq, "inv_freq")) return false;
  if (freq->dtype != VSK_DTYPE_F32) return fail("inv_freq must be float32");
  if (!aligned(freq->data, 4)) return fail("inv_freq must be 4-byte aligned");
  const long long rot = 2 * freq->shape[0];
  if (rot < 16 || rot % 16 != 0 || rot > D)
    return fail("%lld rotated elements (twice inv_freq's) are no multiple of 16 up to head_dim %lld", rot, D);
  if (!std::isfinite(size)) return fail("attention_factor must be finite");
  if (N > INT_MAX - 1024) return fail("%lld rows are too many (2^31 - 1025 at most)", N);
  memset(&p, 0, sizeof p);
  if (q) {
    p.q = view_of(q, 2);
    p.qo = view_of(qo, 2);
    p.h_q = static_cast<int>(q->shape[1]);
  }
  p.k = view_of(k, 2);
  if (ko) p.ko = view_of(ko, 2);
  if (v) p.v = view_of(v, 2);
  p.pos = pos->data;
  p.pos64 = pos->dtype == VSK_DTYPE_I64;
  p.freq = static_cast<const float*>(freq->data);
  p.size = size;
  p.n = N;
  p.h_kv = static_cast<int>(h_kv);
  p.rot = static_cast<int>(rot);
  p.inter = interleaved != 0;
  return true;
}
static Runs index_runs(const char* name, const vsk_tensor* t) {
  return runs_of(name, t, t->dtype == VSK_DTYPE_I64 ? 8 : t->dtype == VSK_DTYPE_U8 ? 1 : 4);
}
// Rows are rewritten while others are read: an output may be its own input, and
// shares no byte with anything else (more: the caches; read: what the call reads beside
// q, k and v).
static bool check_apart(const vsk_tensor* q, const vsk_tensor* k, const vsk_tensor* v, const vsk_tensor* qo,
                        const vsk_tensor* ko, std::initializer_list<Runs> more, std::initializer_list<Runs> read) {
  const Runs ins[] = {runs_of("q", q, 2), runs_of("k", k, 2), runs_of("v", v, 2)};
  Runs outs[8];
  int n = 0;
  outs[n++] = runs_of("q_out", qo, 2);
  outs[n++] = runs_of("k_out", ko, 2);
  for (const Runs& r : more) outs[n++] = r;
  for (int i = 0; i < n; ++i) {
    if (folds(outs[i])) return fail("rows of %s overlap", outs[i].name);
    for (int j = 0; j < 3; ++j)
      if (!(i == j && i < 2 && same_view(outs[i], ins[j])) && meet(outs[i], ins[j]))
        return fail("%s overlaps %s", outs[i].name, ins[j].name);
    for (const Runs& r : read)
      if (meet(outs[i], r)) return fail("%s overlaps %s", outs[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return fail("%s overlaps %s", outs[i].name, outs[j].name);
  }
  return true;
}

static int current_sms(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail("cudaGetDevice: %s", cudaGetErrorString(e));
  *sms = device_sms(dev);
  if (*sms <= 0) return fail("cannot query the SM count of device %d", dev);
  return 1;
}
// A kernel's shared-memory limit, once per device.
static int allow_smem(const void* fn, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail("no CUDA device");
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  std::lock_guard<std::mutex> lk(mu);
  if (done.count({dev, fn})) return 1;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return fail("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  done.insert({dev, fn});
  return 1;
}

// Tokens and heads of a CTA that takes rows; the CTAs.  Few tokens: a row's heads
// over several CTAs, a pass of the threads each at least.  More: one wave of CTAs (four an
// SM), rounded up so that it is no more than one (us, with a few CTAs left over in
// brackets: 2,296 rows, 16/2 heads of 256, rotated 9.2 (10.2), appended to an e4m3 pool 10.3
// (11.5), 4,082 rows 16.4 (16.0-16.4), 18.4 (22.4); 4,000 rows of 32/8 heads of 128, bf16
// pool, 22.0 (25.7), but rotated 18.4 (17.7)).  Where that takes more than kMaxTokens,
// `many` a CTA (7,000 rows, 16/2 heads of 256: with 8 27.7 us, with 4 25.0; the queries
// beside 21,716 rows into blocks: with 8 103 us in all, with 4 107).
static long long cut_rows(rp::RopeParams& p, long long heads, long long D, int sms, int threads, int many) {
  if (heads == 0) return 0;
  const long long slots = threads / (D / 16);
  const long long wave = (p.n + 4LL * sms - 1) / (4LL * sms);
  p.tokens = wave <= rp::kMaxTokens ? static_cast<int>(wave) : many;
  const long long tiles = (p.n + p.tokens - 1) / p.tokens;
  const long long parts = std::max<long long>(1, std::min((heads + slots - 1) / slots, 4LL * sms / tiles));
  p.heads = static_cast<int>((heads + parts - 1) / parts);
  return tiles * ((heads + p.heads - 1) / p.heads);
}
static int launch_rope(rp::RopeParams& p, long long D, int pool, cudaStream_t st) {
  if (p.n == 0) return 1;
  int sms = 0;
  if (!current_sms(&sms)) return 0;
  const long long heads = p.h_q + (pool ? 2LL : 1LL) * p.h_kv, ctas = cut_rows(p, heads, D, sms, rp::kThreads, 4);
  const long long per_tile = (heads + p.heads - 1) / p.heads;
  const dim3 grid(static_cast<unsigned>(ctas / per_tile), static_cast<unsigned>(per_tile));
  if (grid.y > 65535) return fail("%lld heads are too many", heads);
  void* args[] = {&p};
  const cudaError_t e =
      cudaLaunchKernel(reinterpret_cast<const void*>(kernel_rope(static_cast<int>(D), pool)), grid, dim3(rp::kThreads), args, 0, st);
  if (e != cudaSuccess) return fail("kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

// ---- the block-scaled cache ----
struct BlockCache {
  long long n_blocks, h_kv, D;
};
static bool check_block_cache(const vsk_tensor* kc, const vsk_tensor* vc, const vsk_tensor* ks, const vsk_tensor* vs,
                              const vsk_tensor* bt, const vsk_tensor* lens, const char* lens_name, int64_t block,
                              long long B, long long h_kv, long long D, BlockCache& c) {
  if (!check_3d(kc, "k_cache") || !check_3d(vc, "v_cache") || !check_2d(ks, "k_scales") || !check_2d(vs, "v_scales") ||
      !check_2d(bt, "block_table") || !check_1d(lens, lens_name))
    return false;
  if (block < 16 || block % 16 != 0 || block > rp::kMaxBlock)
    return fail("block_size %lld is no multiple of 16 up to %d", static_cast<long long>(block), rp::kMaxBlock);
  if (kc->dtype != VSK_DTYPE_FP8E4M3 || vc->dtype != VSK_DTYPE_FP8E4M3) return fail("k_cache and v_cache must be fp8 e4m3");
  if (kc->shape[1] != h_kv || vc->shape[1] != h_kv || kc->shape[2] != D || vc->shape[2] != D || kc->shape[0] != vc->shape[0])
    return fail("k_cache and v_cache must be [blocks * block_size, %lld, %lld]", h_kv, D);
  if (kc->shape[0] % block != 0) return fail("cache rows (%lld) are not a whole number of blocks", static_cast<long long>(kc->shape[0]));
  if (kc->shape[0] > INT_MAX) return fail("a cache of %lld rows is too large", static_cast<long long>(kc->shape[0]));
  if (!rows16(kc, 1) || !rows16(vc, 1)) return fail("k_cache and v_cache rows must be 16-byte aligned");
  c.n_blocks = kc->shape[0] / block;
  c.h_kv = h_kv;
  c.D = D;
  for (const vsk_tensor* t : {ks, vs}) {
    const char* name = t == ks ? "k_scales" : "v_scales";
    if (t->dtype != VSK_DTYPE_F32) return fail("%s must be float32", name);
    if (t->shape[0] != c.n_blocks || t->shape[1] != h_kv) return fail("%s must be [%lld, %lld]", name, c.n_blocks, h_kv);
    if (!aligned(t->data, 4)) return fail("%s must be 4-byte aligned", name);
  }
  if (bt->dtype != VSK_DTYPE_I32 || lens->dtype != VSK_DTYPE_I32) return fail("block_table and %s must be int32", lens_name);
  if (!aligned(bt->data, 4) || !aligned(lens->data, 4)) return fail("block_table and %s must be 4-byte aligned", lens_name);
  if (bt->shape[0] != B) return fail("block_table must have one row per sequence (B = %lld)", B);
  if (lens->shape[0] != B) return fail("%s must have one entry per sequence (B = %lld)", lens_name, B);
  if (bt->shape[1] < 1) return fail("block_table has no columns");
  if (bt->shape[1] * block > INT_MAX) return fail("block_table columns x block_size exceeds 2^31 - 1");
  return true;
}

// Tensor map of e4m3 rows [n][heads][D] for boxes of `rows` rows of one head and
// `cols` columns, swizzled over their width.
static bool block_map(const vsk_tensor* t, int cols, int rows, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (!encode) return fail("cuTensorMapEncodeTiled is not available");
  const long long n = t->shape[0], h = t->shape[1], d = t->shape[2];
  const long long s1 = h > 1 ? t->stride[1] : d, s0 = n > 1 ? t->stride[0] : h * s1;  // one element: any stride
  if (s1 < d || s0 < d || s0 >= (1LL << 38) || s1 >= (1LL << 38)) return fail("the cache's strides fit no tensor map");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(h), static_cast<cuuint64_t>(n)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1), static_cast<cuuint64_t>(s0)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), 1, static_cast<cuuint32_t>(rows)}, unit[3] = {1, 1, 1};
  if (encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(t->data), dims, strides, box, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail("the cache's strides fit no tensor map");
  return true;
}

struct BlockForm {
  bk::BkFn stream;
  bk::BkJoinFn join[2];  // a row a warp, a row a CTA
  int smem, per_sm;
};
template <int D>
static BlockForm form_of(int nr, bk::BkFn s, bk::BkJoinFn j, bk::BkJoinFn j4) {
  const int smem = nr == 8 ? bk::Geo<D, 8>::smem : nr == 16 ? bk::Geo<D, 16>::smem : bk::Geo<D, 32>::smem;
  return BlockForm{s, {j, j4}, smem, bk::Geo<D, 32>::per_sm};
}
static BlockForm block_form(long long D, long long R) {
  const int nr = bk::row_tile(static_cast<int>(R));
  return D == 64    ? form_of<64>(nr, kernel_block_stream_64(nr), kernel_block_combine_64(false), kernel_block_combine_64(true))
         : D == 128 ? form_of<128>(nr, kernel_block_stream_128(nr), kernel_block_combine_128(false), kernel_block_combine_128(true))
                    : form_of<256>(nr, kernel_block_stream_256(nr), kernel_block_combine_256(false), kernel_block_combine_256(true));
}

// Partials: a slot per piece (CTA c, segment s: slot c + s), whole row tiles.
struct BlockWs {
  long long rows;
  size_t o_off, need;
};
static BlockWs block_ws(long long n_cta, long long B, long long h_kv, long long R, long long D) {
  BlockWs w;
  const long long nr = bk::row_tile(static_cast<int>(R));
  w.rows = (R + nr - 1) / nr * nr;
  const size_t rows = static_cast<size_t>(n_cta + B * h_kv) * static_cast<size_t>(w.rows);
  w.o_off = 256 + align256(4 * rows);
  // the buffer's last 64 KiB hold the counters of other calls
  w.need = w.o_off + align256(4 * rows * static_cast<size_t>(D)) + kTicketBytes;
  return w;
}
constexpr long long kBlockCtas = 10;  // appends: CTAs of keys and values per SM, about
constexpr long long kMaxRows = 128;  // packed rows of a KV head
constexpr long long kSplitJoin = 4;  // pieces of a segment from which the joining CTA's warps share a row

}  // namespace vsk

using namespace vsk;

extern "C" {

float vsk_rope_frequencies(float* out, int64_t rot_dim, double base, int scaling, double factor, double original_len,
                           double low, double high) {
  clear_error();
  if (!out) return static_cast<float>(fail("out is NULL"));
  if (rot_dim < 2 || rot_dim % 2 != 0) return static_cast<float>(fail("rot_dim %lld is not an even number", static_cast<long long>(rot_dim)));
  if (!(base > 1.0) || !std::isfinite(base)) return static_cast<float>(fail("base must be greater than 1"));
  if (scaling < VSK_ROPE_PLAIN || scaling > VSK_ROPE_BANDS) return static_cast<float>(fail("scaling %d is none of the five", scaling));
  if (scaling != VSK_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return static_cast<float>(fail("factor must be at least 1"));
  const bool by_turns = scaling == VSK_ROPE_RAMP || scaling == VSK_ROPE_BANDS;
  if (by_turns && (!(original_len >= 1.0) || !std::isfinite(original_len))) return static_cast<float>(fail("original_len must be at least 1"));
  if (by_turns && (!(low > 0.0) || !(high > low) || !std::isfinite(high))) return static_cast<float>(fail("low and high must be 0 < low < high"));
  if (scaling == VSK_ROPE_BASE && rot_dim < 4) return static_cast<float>(fail("a scaled base needs a rot_dim of at least 4"));
  const double kTwoPi = 6.283185307179586, R = static_cast<double>(rot_dim);
  if (scaling == VSK_ROPE_BASE) base *= std::pow(factor, R / (R - 2.0));
  double first = 0.0, last = 0.0;
  if (scaling == VSK_ROPE_RAMP) {
    // the pairs that turn `high` and `low` times over the original length
    auto pair = [&](double turns) { return R * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
    first = std::max(0.0, std::floor(pair(high)));
    last = std::min(R - 1.0, std::ceil(pair(low)));
    if (last - first < 1e-3) last = first + 1e-3;
  }
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * static_cast<double>(i) / R);
    double slow = 0.0;  // how much of the frequency is divided by the factor
    if (scaling == VSK_ROPE_LINEAR) slow = 1.0;
    if (scaling == VSK_ROPE_RAMP) slow = std::min(1.0, std::max(0.0, (static_cast<double>(i) - first) / (last - first)));
    if (scaling == VSK_ROPE_BANDS) slow = 1.0 - std::min(1.0, std::max(0.0, (original_len * f / kTwoPi - low) / (high - low)));
    out[i] = static_cast<float>(f * (1.0 - slow) + f / factor * slow);
  }
  return scaling == VSK_ROPE_RAMP ? static_cast<float>(1.0 + 0.1 * std::log(factor)) : 1.f;
}

int rope_fwd(const vsk_tensor* q, const vsk_tensor* k, const vsk_tensor* q_out, const vsk_tensor* k_out,
             const vsk_tensor* positions, const vsk_tensor* inv_freq, int interleaved, float attention_factor,
             void* stream) {
  clear_error();
  rp::RopeParams p;
  long long D = 0;
  if (!k_out) return fail("k_out is NULL");
  if (!prepare_rope(q, k, nullptr, q_out, k_out, positions, inv_freq, interleaved, attention_factor, p, D)) return 0;
  if (!check_apart(q, k, nullptr, q_out, k_out, {}, {index_runs("positions", positions), index_runs("inv_freq", inv_freq)}))
    return 0;
  return launch_rope(p, D, 0, static_cast<cudaStream_t>(stream));
}

int rope_append_fwd(const vsk_tensor* q, const vsk_tensor* k, const vsk_tensor* v, const vsk_tensor* q_out,
                    const vsk_tensor* k_out, const vsk_tensor* k_buffer, const vsk_tensor* v_buffer,
                    const vsk_tensor* out_cache_loc, const vsk_tensor* positions, const vsk_tensor* inv_freq,
                    int interleaved, float attention_factor, float k_scale, float v_scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
  clear_error();
  rp::RopeParams p;
  long long D = 0;
  if (!v) return fail("v is NULL");
  if (!prepare_rope(q, k, v, q_out, k_out, positions, inv_freq, interleaved, attention_factor, p, D)) return 0;
  if (!check_3d(k_buffer, "k_buffer") || !check_3d(v_buffer, "v_buffer")) return 0;
  if (k_buffer->dtype != v_buffer->dtype || (k_buffer->dtype != VSK_DTYPE_BF16 && k_buffer->dtype != VSK_DTYPE_FP8E4M3))
    return fail("k_buffer and v_buffer must both be bf16 or both fp8 e4m3");
  const int e = k_buffer->dtype == VSK_DTYPE_FP8E4M3 ? 1 : 2;
  for (const vsk_tensor* t : {k_buffer, v_buffer}) {
    if (t->shape[1] != k->shape[1] || t->shape[2] != D || t->shape[0] != k_buffer->shape[0])
      return fail("k_buffer and v_buffer must be [pool, %lld, %lld]", static_cast<long long>(k->shape[1]), D);
    if (!rows16(t, e)) return fail("k_buffer and v_buffer rows must be 16-byte aligned");
  }
  if (!check_index(out_cache_loc, "out_cache_loc", k->shape[0])) return 0;
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return fail("storing into the cache needs finite k_scale > 0 and v_scale > 0");
  if (!check_apart(q, k, v, q_out, k_out, {runs_of("k_buffer", k_buffer, e), runs_of("v_buffer", v_buffer, e)},
                   {index_runs("positions", positions), index_runs("inv_freq", inv_freq), index_runs("out_cache_loc", out_cache_loc)}))
    return 0;
  if (workspace && workspace_bytes < 256) return fail("workspace of %zu bytes is smaller than 256", workspace_bytes);
  if (p.n == 0) return 1;
  p.kc = view_of(k_buffer, e);
  p.vc = view_of(v_buffer, e);
  p.pool = k_buffer->shape[0];
  p.loc = out_cache_loc->data;
  p.loc64 = out_cache_loc->dtype == VSK_DTYPE_I64;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  WorkspaceHold hold(workspace);
  unsigned char* ws = take_workspace(workspace, workspace_bytes, 256, st, &ws_bytes);
  if (!ws) return 0;
  p.err = reinterpret_cast<unsigned*>(ws);
  return launch_rope(p, D, e == 1 ? 2 : 1, st);
}

int rope_append_block_fwd(const vsk_tensor* q, const vsk_tensor* k, const vsk_tensor* v, const vsk_tensor* q_out,
                          const vsk_tensor* k_out, const vsk_tensor* k_cache, const vsk_tensor* v_cache,
                          const vsk_tensor* k_scales, const vsk_tensor* v_scales, const vsk_tensor* qo_indptr,
                          const vsk_tensor* block_table, const vsk_tensor* cache_lens, const vsk_tensor* positions,
                          const vsk_tensor* inv_freq, int64_t block_size, int interleaved, float attention_factor,
                          void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  rp::RopeParams p;
  long long D = 0;
  if (!v) return fail("v is NULL");
  if (!prepare_rope(q, k, v, q_out, k_out, positions, inv_freq, interleaved, attention_factor, p, D)) return 0;
  if (!check_1d(qo_indptr, "qo_indptr")) return 0;
  if (qo_indptr->dtype != VSK_DTYPE_I32) return fail("qo_indptr must be int32");
  if (!aligned(qo_indptr->data, 4)) return fail("qo_indptr must be 4-byte aligned");
  const long long B = qo_indptr->shape[0] - 1;
  if (B < 1) return fail("batch size must be >= 1");
  BlockCache c;
  if (!check_block_cache(k_cache, v_cache, k_scales, v_scales, block_table, cache_lens, "cache_lens", block_size, B,
                         k->shape[1], D, c))
    return 0;
  if (!check_apart(q, k, v, q_out, k_out,
                   {runs_of("k_cache", k_cache, 1), runs_of("v_cache", v_cache, 1), runs_of("k_scales", k_scales, 4),
                    runs_of("v_scales", v_scales, 4)},
                   {index_runs("positions", positions), index_runs("inv_freq", inv_freq), index_runs("qo_indptr", qo_indptr),
                    index_runs("block_table", block_table), index_runs("cache_lens", cache_lens)}))
    return 0;
  if (workspace && workspace_bytes < 256) return fail("workspace of %zu bytes is smaller than 256", workspace_bytes);
  if (p.n == 0) return 1;
  p.kc = view_of(k_cache, 1);
  p.vc = view_of(v_cache, 1);
  p.ks = static_cast<float*>(const_cast<void*>(k_scales->data));
  p.vs = static_cast<float*>(const_cast<void*>(v_scales->data));
  p.ks_s0 = k_scales->stride[0];
  p.vs_s0 = v_scales->stride[0];
  p.qo_ptr = static_cast<const int*>(qo_indptr->data);
  p.lens = static_cast<const int*>(cache_lens->data);
  p.bt = static_cast<const int*>(block_table->data);
  p.bt_s0 = block_table->stride[0];
  p.bt_cols = static_cast<int>(block_table->shape[1]);
  p.block = static_cast<int>(block_size);
  p.B = static_cast<int>(B);
  p.n_blocks = c.n_blocks;
  int sms = 0;
  if (!current_sms(&sms)) return 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  WorkspaceHold hold(workspace);
  unsigned char* ws = take_workspace(workspace, workspace_bytes, 256, st, &ws_bytes);
  if (!ws) return 0;
  p.err = reinterpret_cast<unsigned*>(ws);
  // a sequence adds to at most one block more than its rows fill, twice over, and to none without a row
  const long long units = std::min(p.n, p.n / block_size + 2 * B);
  // warps that hold the K or V rows of a block and head, 16 elements a thread
  // (of the rows a block gets on the average: a prompt beside many single rows gets few
  // warps and reads most of its rows twice, 4,000 rows and 500 single ones in blocks of 64
  // 44 us together, 28 and 14 apart; in blocks of 128 71, 37 and 16)
  const long long held = 32 * 16 / D, mean = std::min<long long>(block_size, (p.n + B - 1) / B);
  for (p.warps = 1; p.warps * held < mean && p.warps < rp::kBlockThreads / 32;) p.warps *= 2;
  const long long groups = rp::kBlockThreads / 32 / p.warps;
  p.units = static_cast<int>(units);
  // CTAs that share a block's heads: some ten an SM (21,716 rows, 32/8 heads of 128, us: blocks of 64
  // with 7, 10, 14 an SM 105.7, 102.7, 106.5; in blocks of 32 as many as four a block 107, so 99, of 16
  // 118, so 104), keys apart from values, which need no table of angles (8/1 heads together 37.9, apart
  // 35.3); two heads a CTA at least (16/2 of 256: one 102, two 94) and 16 at most (32/32, blocks of 32:
  // 32 heads 214, 16 207).  Where that leaves SMs without work, all that there are (4 x 300 rows: 21.5, so
  // 15.4).
  const long long most = (2LL * p.h_kv + groups - 1) / groups, want = (kBlockCtas * sms + units / 2) / units;
  long long parts = std::min(std::max(2LL, most / 2), std::max(std::max(2LL, most / 16), want));
  parts = std::min(most, std::max(parts, 4LL * sms / units));
  const long long each = (most + parts - 1) / parts;
  p.parts = static_cast<int>((most + each - 1) / each);
  const long long kv = units * p.parts, rows = cut_rows(p, p.h_q, D, sms, rp::kBlockThreads, rp::kMaxTokens), grid = kv + rows;
  p.turn = static_cast<int>(1 + rows / kv);
  if (grid > INT_MAX) return fail("grid of %lld CTAs too large", grid);
  const void* fn = reinterpret_cast<const void*>(kernel_rope_block(static_cast<int>(D)));
  const size_t smem = sizeof(float2) * static_cast<size_t>(block_size) * static_cast<size_t>(p.rot / 2);
  if (!allow_smem(fn, sizeof(float2) * rp::kMaxBlock * 128)) return 0;
  void* args[] = {&p};
  const cudaError_t e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(rp::kBlockThreads), args, smem, st);
  if (e != cudaSuccess) return fail("kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

size_t vsk_block_workspace_size(int64_t max_bs, int64_t h_q, int64_t h_kv, int64_t head_dim, int64_t max_len_extend) {
  int sms = 0;
  if (max_bs < 1 || h_kv < 1 || h_q < 1 || h_q % h_kv != 0 || max_len_extend < 1) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  const long long R = h_q / h_kv * max_len_extend;
  if (R > kMaxRows || !current_sms(&sms)) return 0;
  return block_ws(static_cast<long long>(sms) * block_form(head_dim, R).per_sm, max_bs, h_kv, R, head_dim).need;
}

int verify_splitkv_block_fwd(const vsk_tensor* q, const vsk_tensor* ke, const vsk_tensor* ve, const vsk_tensor* o,
                             const vsk_tensor* kc, const vsk_tensor* vc, const vsk_tensor* ks, const vsk_tensor* vs,
                             const vsk_tensor* qo, const vsk_tensor* bt, const vsk_tensor* lens, const vsk_tensor* cm,
                             const vsk_tensor* mi, int64_t block_size, int64_t max_len_extend, float sm_scale,
                             void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  if (!check_3d(q, "q_extend") || !check_3d(ke, "k_extend") || !check_3d(ve, "v_extend") || !check_3d(o, "o_extend") ||
      !check_1d(qo, "qo_indptr"))
    return 0;
  if (max_len_extend < 1) return fail("max_len_extend must be >= 1");
  const long long B = qo->shape[0] - 1, L = max_len_extend;
  if (B < 1) return fail("batch size must be >= 1");
  if (qo->dtype != VSK_DTYPE_I32) return fail("qo_indptr must be int32");
  if (!aligned(qo->data, 4)) return fail("qo_indptr must be 4-byte aligned");
  const long long N = q->shape[0], h_q = q->shape[1], D = q->shape[2], h_kv = ke->shape[1];
  if (L > INT_MAX || N != B * L) return fail("ragged extend: q has %lld rows, expected B*max_len_extend = %lld", N, B * L);
  if (h_kv < 1 || h_q < 1 || h_q % h_kv != 0) return fail("h_q (%lld) is not a multiple of h_kv (%lld)", h_q, h_kv);
  if (D != 64 && D != 128 && D != 256) return fail("head_dim %lld not in {64, 128, 256}", D);
  for (const vsk_tensor* t : {q, ke, ve, o})
    if (t->dtype != VSK_DTYPE_BF16) return fail("q_extend, k_extend, v_extend and o_extend must be bf16");
  if (ke->shape[0] != N || ve->shape[0] != N || ve->shape[1] != h_kv || ke->shape[2] != D || ve->shape[2] != D)
    return fail("k_extend and v_extend must be [%lld, %lld, %lld]", N, h_kv, D);
  if (o->shape[0] != N || o->shape[1] != h_q || o->shape[2] != D) return fail("o_extend must have the shape of q_extend");
  for (const vsk_tensor* t : {q, ke, ve, o})
    if (!rows4(t)) return fail("q_extend, k_extend, v_extend and o_extend must be 4-byte aligned with even strides");
  const long long R = h_q / h_kv * L;
  if (R > kMaxRows) return fail("(h_q/h_kv)*max_len_extend = %lld exceeds %lld", R, kMaxRows);
  BlockCache c;
  if (!check_block_cache(kc, vc, ks, vs, bt, lens, "seq_lens", block_size, B, h_kv, D, c)) return 0;
  if ((cm == nullptr) != (mi == nullptr)) return fail("custom_mask and mask_indptr go together");
  if (cm) {
    if (!check_1d(cm, "custom_mask") || !check_1d(mi, "mask_indptr")) return 0;
    if (cm->dtype != VSK_DTYPE_U8) return fail("custom_mask must be uint8");
    if (mi->dtype != VSK_DTYPE_I32 && mi->dtype != VSK_DTYPE_I64) return fail("mask_indptr must be int32 or int64");
    if (mi->shape[0] != B + 1) return fail("mask_indptr must have B+1 entries");
    if (!aligned(mi->data, mi->dtype == VSK_DTYPE_I64 ? 8 : 4)) return fail("mask_indptr must be aligned to its type");
  }
  bk::BkParams p;
  memset(&p, 0, sizeof p);
  p.scale2 = static_cast<float>(softmax_scale(sm_scale, D) * kLog2e);
  if (!std::isfinite(p.scale2)) return fail("sm_scale is too large");
  {
    const Runs ro = runs_of("o_extend", o, 2);
    if (folds(ro)) return fail("rows of o_extend overlap");
    const Runs none = runs_of("", nullptr, 1);
    for (const Runs& r : {runs_of("q_extend", q, 2), runs_of("k_extend", ke, 2), runs_of("v_extend", ve, 2),
                          runs_of("k_cache", kc, 1), runs_of("v_cache", vc, 1), runs_of("k_scales", ks, 4),
                          runs_of("v_scales", vs, 4), index_runs("qo_indptr", qo), index_runs("block_table", bt),
                          index_runs("seq_lens", lens), cm ? index_runs("custom_mask", cm) : none,
                          mi ? index_runs("mask_indptr", mi) : none})
      if (meet(ro, r)) return fail("o_extend overlaps %s", r.name);
  }
  const BlockForm f = block_form(D, R);
  int sms = 0;
  if (!current_sms(&sms)) return 0;
  const long long n_cta = static_cast<long long>(sms) * f.per_sm;
  const BlockWs w = block_ws(n_cta, B, h_kv, R, D);
  // teams over segments: a segment's pieces, about
  int team = 8;
  while (h_kv % team != 0) --team;
  const long long tiles = w.rows / bk::row_tile(static_cast<int>(R)), n_team = std::max(1LL, n_cta / (team * tiles));
  const bool split = n_team > kSplitJoin * B * (h_kv / team);
  if (B * (h_kv / team) * ((bt->shape[1] * block_size - 1) / bk::KT + 1) > INT_MAX / 2)
    return fail("%lld sequences of up to %lld blocks are too many", B, static_cast<long long>(bt->shape[1]));
  const long long joins = B * h_kv * (split ? R : (R + 3) / 4);
  if (joins > INT_MAX) return fail("grid of %lld CTAs too large", joins);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t ws_bytes = 0;
  WorkspaceHold hold(workspace);
  unsigned char* ws = take_workspace(workspace, workspace_bytes, w.need, st, &ws_bytes);
  if (!ws) return 0;
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  p.q_s0 = q->stride[0];
  p.q_s1 = q->stride[1];
  p.ke = static_cast<const __nv_bfloat16*>(ke->data);
  p.ke_s0 = ke->stride[0];
  p.ke_s1 = ke->stride[1];
  p.ve = static_cast<const __nv_bfloat16*>(ve->data);
  p.ve_s0 = ve->stride[0];
  p.ve_s1 = ve->stride[1];
  p.o = static_cast<__nv_bfloat16*>(const_cast<void*>(o->data));
  p.o_s0 = o->stride[0];
  p.o_s1 = o->stride[1];
  p.qo = static_cast<const int*>(qo->data);
  p.bt = static_cast<const int*>(bt->data);
  p.bt_s0 = bt->stride[0];
  p.bt_cols = static_cast<int>(bt->shape[1]);
  p.lens = static_cast<const int*>(lens->data);
  p.ks = static_cast<const float*>(ks->data);
  p.vs = static_cast<const float*>(vs->data);
  p.ks_s0 = ks->stride[0];
  p.vs_s0 = vs->stride[0];
  p.n_blocks = c.n_blocks;
  p.n_rows = N;
  p.block = static_cast<int>(block_size);
  p.bgroups = p.block / bk::GK;
  p.box = std::min(bk::GT, p.bgroups & -p.bgroups);
  p.B = static_cast<int>(B);
  p.L = static_cast<int>(L);
  p.gq = static_cast<int>(h_q / h_kv);
  p.R = static_cast<int>(R);
  p.h_kv = static_cast<int>(h_kv);
  p.rows = static_cast<int>(w.rows);
  p.team = team;
  p.n_hg = p.h_kv / p.team;
  p.n_team = static_cast<int>(n_team);
  p.tiles = static_cast<int>(tiles);
  if (cm) {
    p.cmask = static_cast<const unsigned char*>(cm->data);
    p.n_mask = cm->shape[0];
    p.mindptr = mi->data;
    p.mindptr64 = mi->dtype == VSK_DTYPE_I64;
  }
  p.err = reinterpret_cast<unsigned*>(ws);
  p.plse = reinterpret_cast<float*>(ws + 256);
  p.po = reinterpret_cast<float*>(ws + w.o_off);
  // a cache without rows: no prefix has a key that is there, and a map needs memory to describe
  CUtensorMap maps[2];
  memset(maps, 0, sizeof maps);
  if (kc->shape[0] > 0) {
    const int cols = D < 128 ? 64 : 128, rows = p.box * bk::GK;
    if (!block_map(kc, cols, rows, &maps[0]) || !block_map(vc, cols, rows, &maps[1])) return 0;
  }
  if (!allow_smem(reinterpret_cast<const void*>(f.stream), f.smem)) return 0;
  void* args[] = {&p, &maps[0], &maps[1]};
  cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(f.stream),
                                   dim3(static_cast<unsigned>(n_team * team * tiles)), dim3(bk::kThreads), args, f.smem, st);
  if (e != cudaSuccess) return fail("kernel launch failed: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(joins));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(f.join[split]), args);
  if (e != cudaSuccess) return fail("combine kernel launch failed: %s", cudaGetErrorString(e));
  return 1;
}

}  // extern "C"
