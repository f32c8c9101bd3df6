// The paged key cache shared by the paged operators (plan, append, select, attention): layout,
// argument block and the internal entry points. A page holds P = 2^pshift tokens; the key of
// sequence b at position t lies in physical page block_table[b][t / P] at offset t % P.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cfloat>
#include <cmath>

#include "mtp.h"
#include "mtp_launch.h"

namespace mtp {
namespace pg {

constexpr int kMaxSms = 160;  // grids and workspaces are sized for at most this many SMs
constexpr int kPlanMaxB = 8192;  // sequences of a page plan
constexpr long long kSpin = 4000000000LL;  // bound of a device wait, about 2 s of clock64 cycles

// A validated mtp_paged_kv, in the form the kernels take.
struct Cache {
  void* k;
  void* v;                  // null: V = K
  const int* table;         // [B][table_stride]
  const int* ctx_len;       // [B]
  signed char* codes;       // page summaries, or null
  float* scales;
  long long sp, st, sh;     // elements between pages, tokens, KV heads
  long long table_stride;
  int n_pages, pshift, max_pages, nkv, d, f32;
};

// Attended range of one sequence: keys [lo, hi) of its positions.
__device__ __forceinline__ void key_range(const Cache& c, int b, int window, int& lo, int& hi) {
  const int cap = c.max_pages << c.pshift;
  hi = min(max(c.ctx_len[b], 0), cap);
  lo = window > 0 ? max(0, hi - window) : 0;
}
// Physical page of logical page lp of sequence b, or -1 when the table's entry is no page. An
// ordinary load: this kernel may have been launched, as a programmatic dependent, while a plan
// still writes the table, and the read-only path would ask that nothing write it meanwhile.
__device__ __forceinline__ int phys_page(const Cache& c, int b, int lp) {
  const int page = c.table[static_cast<size_t>(b) * c.table_stride + lp];
  return static_cast<unsigned>(page) < static_cast<unsigned>(c.n_pages) ? page : -1;
}

// An attended key of score -inf enters as the lowest finite score: beside other keys it has no
// weight, and a row of such keys alone (0 / 0: NaN) is told from one with nothing to attend.
__device__ __forceinline__ float attended(float score) { return score == -INFINITY ? -FLT_MAX : score; }
// The exp-sum `den` of a row whose largest score is M, as its outputs are divided by it.
__device__ __forceinline__ float row_sum(float M, float den) { return M == -FLT_MAX ? NAN : den; }

// Lets a kernel use BYTES of dynamic shared memory, asked of the driver once per device.
template <auto kernel, int BYTES>
inline cudaError_t allow_smem() {
  static std::atomic<unsigned long long> done{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const unsigned long long bit = 1ull << (dev & 63);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) & bit))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

// Launches a kernel that begins with pdl_enter() so that it may be set up while the kernel before
// it on the stream still runs.
template <typename... A>
int launch_pdl(const char* what, void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("%s launch: %s", what, cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  return MTP_OK;
}

struct AttArgs {
  Cache c;
  const float* q;           // [B][nh][d]
  const int* list;          // [B][nkv][n_list] logical pages, or null (every page)
  float* out;               // [B][nh][d]
  float* lse;               // [B][nh] or null
  float* ws_acc;            // partial sums of the splits
  float* ws_ml;             // their (max, exp-sum)
  float scale_log2;         // softmax scale * log2(e)
  int* status;              // gets MTP_ERR_TIMEOUT when a device wait gives up, or null
  long long spin;           // bound of the device waits, in clock64 cycles
  int skip;                 // testing: the tensor-core kernel looks up no page of this sequence (-1: none)
  int B, nh, n_list, window, nsplit;
};

// Attention of a chunk of new tokens per sequence.
struct ChunkArgs {
  Cache c;
  const void* q;            // token t, head h at t * q_stride + h * d, model dtype
  const int* cu;            // [B + 1]: sequence b's tokens are [cu[b], cu[b + 1])
  void* out;                // [T][nh][d], model dtype
  float* lse;               // [T][nh] or null
  float* ws_acc;            // partial sums of the splits
  float* ws_ml;             // their (max, exp-sum)
  long long q_stride;
  long long spin;           // bound of the device waits, in clock64 cycles
  float scale_log2;         // softmax scale * log2(e)
  int skip;                 // testing: the tensor-core kernel looks up no page of this sequence (-1: none)
  int B, T, nh, window, nsplit;
};

// The new tokens of sequence b: rows [s0, s0 + n) of the call, at positions first, first + 1, ...
// of L keys (first < 0 where the sequence holds fewer than its new ones: those attend nothing).
__device__ __forceinline__ void chunk_range(const ChunkArgs& a, int b, int& s0, int& n, int& first, int& L) {
  s0 = min(max(a.cu[b], 0), a.T);
  n = min(max(a.cu[b + 1], s0), a.T) - s0;
  L = min(max(a.c.ctx_len[b], 0), a.c.max_pages << a.c.pshift);
  first = L - n;
}

}  // namespace pg

// Workspace bytes and launch of the attention of a chunk.
long long chunk_att_workspace(const pg::ChunkArgs& a);
int run_chunk_att(pg::ChunkArgs a, void* ws, int num_sms, cudaStream_t st);
// Its tensor-core form (mtp_chunk_tc.cu), which run_chunk_att takes where paged_tc_supported.
long long chunk_tc_workspace(const pg::ChunkArgs& a);
int run_chunk_tc(const pg::ChunkArgs& a, void* ws, int num_sms, cudaStream_t st);

// Workspace bytes and launch of the one-token attention.
long long paged_att_workspace(const pg::Cache& c, int B, int nh, int n_list);
long long page_select_workspace(const pg::Cache& c, int B);
int run_paged_att(pg::AttArgs a, void* ws, int num_sms, cudaStream_t st);

// Its tensor-core form (mtp_paged_tc.cu), which run_paged_att takes where it serves the shape.
bool paged_tc_supported(const pg::Cache& c);
long long paged_tc_workspace(const pg::Cache& c);
int run_paged_tc(const pg::AttArgs& a, void* ws, int num_sms, cudaStream_t st);

int run_page_plan(const int* old_len, const int* new_len, int B, int* table, long long table_stride, int max_pages,
                  int* ring, int n_pages, const int* state, int pshift, int max_tokens, int* len_out, int* slots,
                  int* cu_new, int* state_out, int* status, int num_sms, cudaStream_t st);
int run_page_append(const pg::Cache& c, const void* k_new, const void* v_new, long long row_k, long long row_v,
                    const int* slots, int T, int num_sms, cudaStream_t st);
int run_page_select(const pg::Cache& c, const float* q, int B, int nh, int n_select, int keep_first, int keep_last,
                    int* sel, void* ws, int num_sms, cudaStream_t st);

// Forks of sequences over shared pages; the pages that no sequence holds, and their compaction.
int run_page_fork(const pg::Cache& c, int B, const int* src, const int* dst, const int* len, int n, const int* ring,
                  const int* state, int* len_out, int* state_out, int* status, int num_sms, cudaStream_t st);
long long page_collect_workspace(const pg::Cache& c, bool compact);
int run_page_collect(const pg::Cache& c, int B, int* ring, int* table_out, long long out_stride, int* state_out,
                     int* status, void* ws, int num_sms, cudaStream_t st);

struct Params;
// What a paged draft block adds to its Params: the caches by attention type, the selection of the
// full layers (n_select 0: every page) and the caller's workspace, carved.
struct PagedCall {
  pg::Cache c[2];
  float* qn;
  int* sel;
  void *sel_ws, *att_ws;
  int n_select, keep_first, keep_last, num_sms;
};
// Workspace bytes; with a base the pointers of pc are set.
long long paged_draft_workspace(PagedCall& pc, int B, int nh, int dmax, int has_sliding, int has_full, char* base);
// The attention of layer l: into p.w.o and, for the tensor-core phases, the O projection's operand
// xs [3][bp][n_head * head_dim].
int run_paged_layer(const Params& p, const PagedCall& pc, int l, __nv_bfloat16* xs, int bp, cudaStream_t st);

namespace pg {
// mtp_paged_kv -> Cache, every check made before the device is touched (mtp_paged_api.cu).
int make_cache(const mtp_paged_kv* kv, bool tables, Cache* c);
int check_workspace(const void* ws, int64_t have, long long need);
}  // namespace pg

}  // namespace mtp
