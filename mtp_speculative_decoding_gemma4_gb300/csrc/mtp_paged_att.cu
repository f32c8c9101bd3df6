// Attention of one new token over a paged key cache, split over the cache's length and joined:
// out_h = sum_j p_j v_j with p = softmax(scale q_h . k_j) over the attended positions j of the
// sequence, read through the block table (all pages, the last `window` keys, or a list of
// selected pages per KV head).
//
// This file: the CUDA-core kernel for every dtype and head dim, and the join of the splits.
// One CTA of 4 warps per (sequence, KV head, group of heads, split). LPK lanes hold one key row
// (16-byte vectors), 32 / LPK rows side by side in a warp, U row blocks in flight; every lane
// keeps its vectors of GP queries and GP running sums in registers, so a key row is read once
// for all heads of the group. Scores, maxima, sums and outputs are fp32.
// What bounds it: 16 fp32 contexts to 8000 (66 MB of K and V) take 20 us with the join, 3.3 TB/s
// or half of the copy rate; issue slots are 39 % busy and warps wait for their loads, with 5 CTAs
// per SM (registers) and the two launches' starts in the time. Most instructions are around the
// products, so the U * GP scores of a block are reduced by one reduce-scatter, each lane takes the
// softmax of one score, and probabilities are broadcast (27 us without). 5 to 16 CTAs per SM from
// the split and 6 resident CTAs are within 5 % of this.
#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"
#include "mtp_phases.cuh"

namespace mtp {
namespace pg {

constexpr int kAttWarps = 4;

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float* out);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& u, float* out) {
  const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[2 * i] = __uint_as_float(w[i] << 16);
    out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void unpack<float>(const uint4& u, float* out) {
  out[0] = __uint_as_float(u.x);
  out[1] = __uint_as_float(u.y);
  out[2] = __uint_as_float(u.z);
  out[3] = __uint_as_float(u.w);
}

// exp2 of x - m; with no key yet (m = -inf, x = -inf) 0
__device__ __forceinline__ float pexp(float x, float m) { return exp2f(x - (m == -INFINITY ? 0.f : m)); }

template <typename T, int LPK, int NV, int GP>
__global__ void __launch_bounds__(kAttWarps * 32) k_paged_att(const __grid_constant__ AttArgs a) {
  pdl_enter();
  constexpr int VE = Elem<T>::kVec, KPW = 32 / LPK;
  constexpr int U0 = NV >= 4 ? 1 : 4 / NV, U = U0 * GP <= LPK ? U0 : LPK / GP;  // at most a score per lane
  constexpr int N = U * GP, DUP = LPK / N;  // scores of a block, lanes that hold the same one
  static_assert(U >= 1 && DUP >= 1, "lanes for the scores");
  extern __shared__ __align__(16) float sm_att[];  // [warps][GP][d] sums, then [warps][GP] m, l
  const Cache& c = a.c;
  const int d = c.d, nvec = d / VE, G = a.nh / c.nkv, ngrp = (G + GP - 1) / GP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % LPK, sub = lane / LPK;
  int it = blockIdx.x;
  const int sp = it % a.nsplit;
  it /= a.nsplit;
  const int hg = it % ngrp;
  it /= ngrp;
  const int g = it % c.nkv, b = it / c.nkv;
  const int h0 = g * G + hg * GP, nh = min(GP, G - hg * GP);
  int lo, hi;
  key_range(c, b, a.window, lo, hi);
  // keys are numbered by position (dense), or by (list entry, offset)
  const int P = 1 << c.pshift;
  constexpr int R = KPW * U, step = R * kAttWarps;  // rows of a warp's block, of the CTA's
  // blocks begin at multiples of R, so that a block lies in one page when R <= P
  const int i0 = a.list ? 0 : lo / R * R, i1 = a.list ? a.n_list << c.pshift : hi;
  const int chunk = ((max(i1 - i0, 0) + a.nsplit - 1) / a.nsplit + step - 1) / step * step;
  const int j0 = i0 + sp * chunk, j1 = min(i1, j0 + chunk);
  const int* list = a.list ? a.list + (static_cast<size_t>(b) * c.nkv + g) * a.n_list : nullptr;

  // this lane's score of a block: row block su, head sh; its head's reference and its rows' sum
  const int sid = li / DUP, su = sid / GP;
  float q[GP][NV * VE], acc[GP][NV * VE], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int h = 0; h < GP; ++h) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = li + LPK * j;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        acc[h][j * VE + e] = 0.f;
        q[h][j * VE + e] = (h < nh && v < nvec) ? a.q[(static_cast<size_t>(b) * a.nh + h0 + h) * d + v * VE + e] : 0.f;
      }
    }
  }
  const bool one_page = R <= P, whole = nvec == LPK * NV;
  const long long row_step = KPW * c.st;
  for (int base = j0 + warp * R; base < j1; base += step) {
    uint4 kv[U][NV], vv[U][NV];
    bool on[U];
    long long at[U];
    auto find = [&](int i, int& pos) -> int {  // physical page of row i of the range (or -1), its position
      int lp = i >> c.pshift;
      pos = i;
      if (list) {
        lp = list[lp];
        pos = (lp << c.pshift) + (i & (P - 1));
        if (lp < 0 || lp >= c.max_pages) return -1;
      }
      return phys_page(c, b, lp);
    };
    bool all = whole;
    if (one_page) {
      int pos;
      const int page = find(base, pos);
      const long long first = page * c.sp + ((pos & (P - 1)) + sub) * c.st + g * c.sh;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = pos + u * KPW + sub;
        on[u] = page >= 0 && p >= lo && p < hi;
        at[u] = first + u * row_step;
        all = all && on[u];
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = base + u * KPW + sub;
        int pos = 0;
        const int page = i < i1 ? find(i, pos) : -1;
        on[u] = page >= 0 && pos >= lo && pos < hi;
        at[u] = page * c.sp + (pos & (P - 1)) * c.st + g * c.sh;
        all = all && on[u];
      }
    }
    auto load = [&](const void* from, uint4 (&x)[U][NV], bool every) {
      const uint4* base_v = static_cast<const uint4*>(from) + li;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          x[u][j] = every || (on[u] && li + LPK * j < nvec) ? __ldcs(base_v + at[u] / VE + LPK * j) : make_uint4(0, 0, 0, 0);
    };
    if (__all_sync(0xffffffffu, all)) {
      load(c.k, kv, true);
      if (c.v) load(c.v, vv, true);
    } else {
      load(c.k, kv, false);
      if (c.v) load(c.v, vv, false);
    }
    float s[N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[NV * VE];
#pragma unroll
      for (int j = 0; j < NV; ++j) unpack<T>(kv[u][j], x + j * VE);
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < NV * VE; ++e) t = fmaf(q[h][e], x[e], t);
        s[u * GP + h] = t;
      }
    }
    reduce_scatter<N, LPK / 2>(s, lane);
    bool mine = false;
#pragma unroll
    for (int u = 0; u < U; ++u) mine = mine || (su == u && on[u]);
    const float x0 = mine ? attended(s[0] * a.scale_log2) : -INFINITY;
    float mn = x0;
#pragma unroll
    for (int o = GP * DUP; o < LPK; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mn = fmaxf(m, mn);
    const float corr = pexp(m, mn), p = pexp(x0, mn);
    m = mn;
    l = fmaf(l, corr, p);
    if (__any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const float f = __shfl_sync(0xffffffffu, corr, h * DUP, LPK);
#pragma unroll
        for (int e = 0; e < NV * VE; ++e) acc[h][e] *= f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[NV * VE];
#pragma unroll
      for (int j = 0; j < NV; ++j) unpack<T>(c.v ? vv[u][j] : kv[u][j], x + j * VE);
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const float f = __shfl_sync(0xffffffffu, p, (u * GP + h) * DUP, LPK);
#pragma unroll
        for (int e = 0; e < NV * VE; ++e) acc[h][e] = fmaf(f, x[e], acc[h][e]);
      }
    }
  }
  // the row blocks' parts of a head's sum
#pragma unroll
  for (int o = GP * DUP; o < LPK; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  // join the rows held side by side in the warp, then the warps
  float* ml = sm_att + kAttWarps * GP * d;
#pragma unroll
  for (int h = 0; h < GP; ++h) {
    const float mh = __shfl_sync(0xffffffffu, m, h * DUP, LPK);
    float mn = mh, lh = __shfl_sync(0xffffffffu, l, h * DUP, LPK);
#pragma unroll
    for (int o = LPK; o < 32; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    const float corr = pexp(mh, mn);
    lh *= corr;
#pragma unroll
    for (int o = LPK; o < 32; o <<= 1) lh += __shfl_xor_sync(0xffffffffu, lh, o);
#pragma unroll
    for (int e = 0; e < NV * VE; ++e) {
      float t = acc[h][e] * corr;
#pragma unroll
      for (int o = LPK; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      const int v = li + LPK * (e / VE);
      if (sub == 0 && v < nvec) sm_att[(warp * GP + h) * d + v * VE + e % VE] = t;
    }
    if (lane == 0) {
      ml[warp * GP + h] = mn;
      ml[(kAttWarps + warp) * GP + h] = lh;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nh * d; i += kAttWarps * 32) {
    const int h = i / d, e = i % d;
    float M = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, ml[w * GP + h]);
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      const float f = pexp(ml[w * GP + h], M);
      num = fmaf(f, sm_att[(w * GP + h) * d + e], num);
      den = fmaf(f, ml[(kAttWarps + w) * GP + h], den);
    }
    const size_t row = static_cast<size_t>(b) * a.nh + h0 + h;
    if (a.nsplit == 1) {
      den = row_sum(M, den);
      a.out[row * d + e] = den == 0.f ? 0.f : num / den;  // 0: nothing attended
      if (a.lse && e == 0) a.lse[row] = den == 0.f ? -INFINITY : (M + log2f(den)) * 0.6931471805599453f;
    } else {
      a.ws_acc[(row * a.nsplit + sp) * d + e] = num;
      if (e == 0) {
        a.ws_ml[(row * a.nsplit + sp) * 2] = M;
        a.ws_ml[(row * a.nsplit + sp) * 2 + 1] = den;
      }
    }
  }
}

// Joins the splits of one (sequence, head) per CTA: the weights by one warp, the sums by all, a
// group of threads per split and 4 dims each (head dims are multiples of 4).
constexpr int kMaxSplits = 256;

__global__ void __launch_bounds__(256) k_paged_join(const __grid_constant__ AttArgs a) {
  pdl_enter();
  __shared__ float wgt[kMaxSplits], s_m, s_den;
  __shared__ float4 sum[256];
  const size_t row = blockIdx.x;
  const int d = a.c.d, n = a.nsplit, tid = threadIdx.x, vt = d / 4, gr = tid / vt, v = tid - gr * vt, ng = 256 / vt;
  if (tid < 32) {
    const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row * n;
    float M = -INFINITY, den = 0.f;
    for (int s = tid; s < n; s += 32) M = fmaxf(M, ml[s].x);
    M = warp_max(M);
    for (int s = tid; s < n; s += 32) {
      const float f = pexp(ml[s].x, M);
      wgt[s] = f;
      den = fmaf(f, ml[s].y, den);
    }
    den = warp_sum(den);
    if (tid == 0) {
      s_m = M;
      s_den = row_sum(M, den);
    }
  }
  __syncthreads();
  const float den = s_den;
  float4 x = make_float4(0, 0, 0, 0);
  if (gr < ng) {
#pragma unroll 4
    for (int s = gr; s < n; s += ng) {
      const float f = wgt[s];
      const float4 y = *reinterpret_cast<const float4*>(a.ws_acc + (row * n + s) * d + 4 * v);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
  }
  sum[tid] = x;
  __syncthreads();
  if (tid < vt) {
    for (int g = 1; g < ng; ++g) {
      const float4 y = sum[g * vt + tid];
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;  // 0: nothing attended
    *reinterpret_cast<float4*>(a.out + row * d + 4 * tid) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  }
  if (a.lse && tid == 0) a.lse[row] = den == 0.f ? -INFINITY : (s_m + log2f(den)) * 0.6931471805599453f;
}

template <typename T, int LPK, int NV, int GP>
int launch_att(const AttArgs& a, cudaStream_t st) {
  const int G = a.nh / a.c.nkv, ngrp = (G + GP - 1) / GP;
  const long long grid = static_cast<long long>(a.B) * a.c.nkv * ngrp * a.nsplit;
  const int smem = kAttWarps * GP * (a.c.d + 2) * 4;
  return launch_pdl("paged attention", k_paged_att<T, LPK, NV, GP>, dim3(static_cast<unsigned>(grid)), kAttWarps * 32,
                    smem, st, a);
}

// Heads per CTA: the queries and sums of GP heads have to stay in registers (GP * NV * VE <= 64).
template <typename T, int LPK, int NV>
int launch_group(const AttArgs& a, cudaStream_t st) {
  const int G = a.nh / a.c.nkv;
  constexpr int kMost = NV * Elem<T>::kVec >= 16 ? 4 : 8;
  if (G == 1) return launch_att<T, LPK, NV, 1>(a, st);
  if (G == 2) return launch_att<T, LPK, NV, 2>(a, st);
  if (G <= 4 || kMost == 4) return launch_att<T, LPK, NV, 4>(a, st);
  return launch_att<T, LPK, NV, kMost>(a, st);
}

template <typename T>
int launch_type(const AttArgs& a, cudaStream_t st) {
  const int nvec = a.c.d / Elem<T>::kVec;
  if (nvec <= 8) return launch_group<T, 8, 1>(a, st);
  if (nvec <= 16) return launch_group<T, 16, 1>(a, st);
  if (nvec <= 32) return launch_group<T, 32, 1>(a, st);
  if (nvec <= 64) return launch_group<T, 32, 2>(a, st);
  return launch_group<T, 32, 4>(a, st);
}

// Splits of a sequence's keys: about 8 CTAs per SM over the batch, at least 64 keys each.
int choose_splits(const Cache& c, int B, int nh, int n_list, int window, int num_sms) {
  const long long units = static_cast<long long>(B) * nh;
  long long keys = static_cast<long long>(n_list > 0 ? n_list : c.max_pages) << c.pshift;
  if (window > 0 && window < keys) keys = window;
  long long n = 8LL * num_sms * (nh / c.nkv) / units;
  if (n > keys / 64) n = keys / 64;
  if (n > kMaxSplits) n = kMaxSplits;
  return n < 1 ? 1 : static_cast<int>(n);
}

}  // namespace pg

long long paged_att_workspace(const pg::Cache& c, int B, int nh, int n_list) {
  if (paged_tc_supported(c)) return paged_tc_workspace(c);
  // a window only shortens the key range and fewer SMs take fewer splits, so this is a bound
  const long long n = pg::choose_splits(c, B, nh, n_list, 0, pg::kMaxSms);
  return n > 1 ? static_cast<long long>(B) * nh * n * (c.d + 2) * 4 : 0;
}

int run_paged_att(pg::AttArgs a, void* ws, int num_sms, cudaStream_t st) {
  if (paged_tc_supported(a.c)) return run_paged_tc(a, ws, num_sms, st);
  a.nsplit = pg::choose_splits(a.c, a.B, a.nh, a.list ? a.n_list : 0, a.window, num_sms);
  a.ws_acc = static_cast<float*>(ws);
  a.ws_ml = a.ws_acc + static_cast<size_t>(a.B) * a.nh * a.nsplit * a.c.d;
  int rc = a.c.f32 ? pg::launch_type<float>(a, st) : pg::launch_type<__nv_bfloat16>(a, st);
  if (rc || a.nsplit == 1) return rc;
  return pg::launch_pdl("paged attention join", pg::k_paged_join, dim3(a.B * a.nh), 256, 0, st, a);
}

}  // namespace mtp
