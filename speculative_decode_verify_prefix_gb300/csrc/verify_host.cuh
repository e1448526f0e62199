// What the host files of the library share: the error text, the argument
// checks, the CTA plan and the workspace layout of the prefix stream
// (verify_splitkv.cu) for the calls built around it (cache_ops.cu).
#pragma once
#include <cuda_runtime.h>

#include "../../include/verify_splitkv.h"
#include "verify_kernel.cuh"

namespace vsk {

struct Plan {
  int gq, R, MT, MTW, HC, n_hg, nwc, threads, ek;
  int stage_bytes, nst, ring_off, head_bytes, misc_off, misc_bytes;
  size_t smem;
  int ctas_per_sm;
};

struct WsLayout {
  size_t lse_off, o_off, cnt_bytes, total;
};

// The static shapes of a flat call.
struct CallShape {
  long long B, h_q, h_kv, D, DV, L, mean_len;
  bool fp8;
};

int fail(const char* fmt, ...);  // sets vsk_last_error, returns 0
void clear_error();
bool check_3d(const vsk_tensor* t, const char* name);
bool check_2d(const vsk_tensor* t, const char* name);
bool check_1d(const vsk_tensor* t, const char* name);
bool aligned(const void* p, size_t a);
size_t align256(size_t x);
int device_sms(int dev);
int prepare_kernel(KernelFn fn);
void* internal_workspace(int dev, size_t need, cudaStream_t stream, size_t* bytes);
// Holds a workspace (NULL: the library-owned one) while a call enqueues its
// launches.  Several launches hand partials on in it, so calls of two host
// threads on one stream must not enqueue theirs in between; and the
// library-owned one must not be replaced between its choice and the launch.
class WorkspaceHold {
 public:
  explicit WorkspaceHold(const void* ws);
  ~WorkspaceHold();
  WorkspaceHold(const WorkspaceHold&) = delete;
  WorkspaceHold& operator=(const WorkspaceHold&) = delete;

 private:
  const void* ws_;
};
bool make_plan(long long h_q, long long h_kv, long long D, long long L, bool fp8, Plan& pl, long long total_tokens,
               int tiles, long long DV = 0, int hc_cap = 0);
WsLayout ws_layout(long long n_cta, long long B, const Plan& pl, long long DV);
// checks and parameter block of a flat call (no launch, no workspace);
// keys_only: the call has no values, ke, kb and q stand in for ve, vb and o
int prepare_verify(const vsk_tensor* q, const vsk_tensor* ke, const vsk_tensor* ve, const vsk_tensor* o,
                   const vsk_tensor* kb, const vsk_tensor* vb, const vsk_tensor* qo, const vsk_tensor* kvp,
                   const vsk_tensor* kvi, int is_causal, int64_t max_len_extend, float k_scale, float v_scale,
                   float sm_scale, const vsk_tensor* cm, const vsk_tensor* mi, const vsk_tensor* ocl, Params& p,
                   CallShape& cs, bool keys_only = false);
// A prefix stream alone (no draft block, partials left in the workspace): its
// plan, and the launch.
struct StreamOnly {
  Plan pl;
  KernelFn fn;
  int threads;
  size_t smem;
  bool rows_m;  // the rows-on-M tensor-memory stream
  long long n_cta, w_min;
  WsLayout wl;
};
int plan_stream_only(const CallShape& cs, StreamOnly& so);
int launch_stream_only(Params& p, const CallShape& cs, const StreamOnly& so, unsigned char* ws, size_t ws_bytes,
                       cudaStream_t st);

}  // namespace vsk
