// Attention of a draft block's layer over a paged cache: q_norm and RoPE of the layer's queries
// ("Gemma 4 Multi-Token Prediction (MTP) drafter", "Tensor schema": attn_q_norm; constant
// position), optionally the selection of pages for full-attention layers, the paged attention,
// and for the tensor-core phases the O projection's staged operand. It takes the place of the
// attention and combine phases; every other phase is the one of mtp_phases.cuh.
#include <cstring>

#include "mtp_launch.h"
#include "mtp_paged.cuh"
#include "mtp_phases.cuh"

namespace mtp {

// qn[b][h][i] = RoPE(q_norm(q)): one warp per head, the head's values in registers (head_dim <= 512).
__global__ void __launch_bounds__(kThreads) k_paged_q(const __grid_constant__ Params p, int l, float* qn) {
  pdl_enter();
  const int t = p.L[l].type, d = p.s.d[t], half = d / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float2* cs0 = p.w.cs + static_cast<size_t>(t) * (p.w.dmax / 2);
  const float* gq = p.L[l].q_norm;
  for (int it = blockIdx.x * kWarps + warp; it < p.s.B * p.s.nh; it += gridDim.x * kWarps) {
    const int b = it / p.s.nh, h = it % p.s.nh;
    const float* q = p.w.qraw + static_cast<size_t>(b) * p.s.nh * p.w.dmax + static_cast<size_t>(h) * d;
    const float2* cs = cs0 + static_cast<size_t>(b) * 2 * (p.w.dmax / 2);
    float* out = qn + static_cast<size_t>(it) * d;
    float s = 0.f;
    for (int i = lane; i < d; i += 32) s = fmaf(q[i], q[i], s);
    const float rf = rsqrtf(warp_sum(s) / static_cast<float>(d) + p.s.eps);
    for (int i = lane; i < half; i += 32) {
      const float x = q[i] * rf * gq[i], y = q[i + half] * rf * gq[i + half];
      const float2 r = cs[i];
      out[i] = x * r.x - y * r.y;
      out[i + half] = y * r.x + x * r.y;
    }
  }
}

// The O projection's operand of the tensor-core phases from the attention outputs.
__global__ void __launch_bounds__(kThreads) k_paged_stage(const __grid_constant__ Params p, int l, __nv_bfloat16* xs, int bp) {
  pdl_enter();
  const int K = p.s.nh * p.s.d[p.L[l].type];
  for (int b = blockIdx.x; b < p.s.B; b += gridDim.x)
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < K; i += gridDim.y * kThreads)
      stage_terms(xs, bp, K, b, i, p.w.o[static_cast<size_t>(b) * K + i]);
}

namespace {
long long round16(long long n) { return (n + 15) & ~15ll; }
}  // namespace

long long paged_draft_workspace(PagedCall& pc, int B, int nh, int dmax, int has_sliding, int has_full, char* base) {
  long long at = 0, att = 0;
  auto take = [&](long long bytes) {
    char* p = base ? base + at : nullptr;
    at += round16(bytes);
    return p;
  };
  pc.qn = reinterpret_cast<float*>(take(4ll * B * nh * dmax));
  const bool pick = has_full && pc.n_select > 0;
  pc.sel = pick ? reinterpret_cast<int*>(take(4ll * B * pc.c[1].nkv * pc.n_select)) : nullptr;
  pc.sel_ws = pick ? take(page_select_workspace(pc.c[1], B)) : nullptr;
  if (has_sliding) att = paged_att_workspace(pc.c[0], B, nh, 0);
  if (has_full) {
    const long long n = paged_att_workspace(pc.c[1], B, nh, pick ? pc.n_select : 0);
    att = n > att ? n : att;
  }
  pc.att_ws = take(att);
  return at;
}

int run_paged_layer(const Params& p, const PagedCall& pc, int l, __nv_bfloat16* xs, int bp, cudaStream_t st) {
  const int t = p.L[l].type, B = p.s.B;
  int rc = pg::launch_pdl("paged query", k_paged_q, dim3(ceil_div(B * p.s.nh, kWarps)), kThreads, 0, st, p, l, pc.qn);
  if (rc) return rc;
  pg::AttArgs a;
  memset(&a, 0, sizeof(a));
  a.c = pc.c[t];
  a.q = pc.qn;
  a.out = p.w.o;
  a.scale_log2 = static_cast<float>(static_cast<double>(p.s.scale[t]) * 1.4426950408889634);
  a.B = B;
  a.nh = p.s.nh;
  a.window = t == 0 ? p.s.W : 0;
  a.status = p.w.status;
  a.spin = p.spin_limit;
  a.skip = l == 0 ? p.dbg_skip - 1 : -1;
  if (t == 1 && pc.n_select > 0) {
    if ((rc = run_page_select(a.c, pc.qn, B, p.s.nh, pc.n_select, pc.keep_first, pc.keep_last, pc.sel, pc.sel_ws,
                              pc.num_sms, st)))
      return rc;
    a.list = pc.sel;
    a.n_list = pc.n_select;
  }
  if ((rc = run_paged_att(a, pc.att_ws, pc.num_sms, st))) return rc;
  if (!xs) return MTP_OK;
  return pg::launch_pdl("paged attention staging", k_paged_stage, dim3(B, ceil_div(p.s.nh * p.s.d[t], kThreads)), kThreads, 0,
                    st, p, l, xs, bp);
}

}  // namespace mtp
