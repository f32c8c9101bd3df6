// The page plan (block tables and slot maps from request lengths) and the append into a paged
// key cache with its page summaries.
#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

// ---------------------------------------------------------------- plan
//
// Sequence b goes from old_len to new_len tokens: ceil(new / P) - ceil(old / P) pages are taken
// from the head of the ring of free pages, in batch order, or returned to its tail. A grower is
// granted while the running sums of pages and of tokens over the growers fit, so the granted
// growers are a prefix and every page and slot follows from three prefix sums. Every CTA makes
// the sums itself (B is at most 8192) and takes its share of the pages and slots: one launch
// and no exchange. Pages are taken from [head, head + count) and returned behind it, so no ring
// entry is both read and written.

constexpr int kPlanThreads = 512;

struct PlanArgs {
  const int *old_len, *new_len, *state;
  int *table, *ring, *len_out, *slots, *cu_new, *state_out, *status;
  long long table_stride;
  int B, max_pages, n_pages, pshift, max_tokens;
};

// Exclusive prefix over the CTA of one value per thread; `total` gets the sum. `red` holds 32.
__device__ __forceinline__ long long scan_excl(long long v, long long& total, long long* red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) red[w] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < w) before += red[i];
    all += red[i];
  }
  total = all;
  return before + x - v;
}

// First index i in [0, n) with a[i + 1] > x, for a non-decreasing a[0..n] with a[n] > x.
__device__ __forceinline__ int find_seq(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid + 1] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) k_page_plan(const __grid_constant__ PlanArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) int sm_plan[];
  __shared__ long long red[kPlanThreads / 32];
  __shared__ int s_taken, s_total, s_denied;
  const int B = a.B, P = 1 << a.pshift, tid = threadIdx.x;
  int* cu = sm_plan;               // [B + 1] slots before sequence b (granted growers)
  int* cp = cu + B + 1;            // [B + 1] pages taken before sequence b
  int* cf = cp + B + 1;            // [B + 1] pages returned before sequence b
  const long long cap = static_cast<long long>(a.max_pages) << a.pshift;
  const int count = min(max(a.state[1], 0), a.n_pages);
  const int head = static_cast<unsigned>(a.state[0]) % static_cast<unsigned>(a.n_pages);
  if (tid == 0) s_taken = s_total = s_denied = 0;
  // this thread's run of sequences
  const int per = (B + kPlanThreads - 1) / kPlanThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto lens = [&](int b, int& o, int& n, bool& fits) {
    o = static_cast<int>(min(static_cast<long long>(max(a.old_len[b], 0)), cap));
    n = a.new_len[b];
    fits = n >= 0 && n <= cap;
  };
  auto pages = [&](int n) { return (n + P - 1) >> a.pshift; };
  // ring index below 3 n_pages (a head, at most n_pages pages and at most n_pages returned)
  auto wrap = [&](long long i) {
    if (i >= a.n_pages) i -= a.n_pages;
    return i >= a.n_pages ? i % a.n_pages : i;
  };
  long long need = 0, tok = 0, fre = 0;
  for (int b = b0; b < b1; ++b) {
    int o, n;
    bool fits;
    lens(b, o, n, fits);
    if (fits && n > o) {
      need += pages(n) - pages(o);
      tok += n - o;
    } else if (fits) {
      fre += pages(o) - pages(n);
    }
  }
  long long t0, t1, t2;
  long long pn = scan_excl(need, t0, red), pt = scan_excl(tok, t1, red), pf = scan_excl(fre, t2, red);
  int denied = 0, taken = 0, total = 0;
  for (int b = b0; b < b1; ++b) {
    int o, n;
    bool fits;
    lens(b, o, n, fits);
    bool granted = false;
    cf[b] = static_cast<int>(pf);
    if (fits && n > o) {
      const long long bp = pn, bt = pt;
      pn += pages(n) - pages(o);
      pt += n - o;
      granted = pn <= count && pt <= a.max_tokens;
      cp[b] = granted ? static_cast<int>(bp) : -1;
      cu[b] = granted ? static_cast<int>(bt) : -1;
      if (granted) {
        taken = static_cast<int>(pn);
        total = static_cast<int>(pt);
      } else {
        ++denied;
      }
    } else {
      // between growers: the sums so far, or -1 behind the first that was denied
      const bool ok = pn <= count && pt <= a.max_tokens;
      cp[b] = ok ? static_cast<int>(pn) : -1;
      cu[b] = ok ? static_cast<int>(pt) : -1;
      if (fits) pf += pages(o) - pages(n); else ++denied;
    }
    if (blockIdx.x == 0) a.len_out[b] = (granted || (fits && n <= o)) ? n : o;
  }
  if (taken) atomicMax(&s_taken, taken);
  if (total) atomicMax(&s_total, total);
  if (denied) atomicAdd(&s_denied, denied);
  __syncthreads();
  taken = s_taken;
  total = s_total;
  const int freed = static_cast<int>(t2);
  for (int b = b0; b < b1; ++b) {
    if (cp[b] < 0) {
      cp[b] = taken;
      cu[b] = total;
    }
    if (blockIdx.x == 0) a.cu_new[b] = cu[b];
  }
  if (tid == 0) {
    cu[B] = total;
    cp[B] = taken;
    cf[B] = freed;
    if (blockIdx.x == 0) {
      a.cu_new[B] = total;
      a.state_out[0] = static_cast<int>((static_cast<long long>(head) + taken) % a.n_pages);
      a.state_out[1] = count - taken + freed;
      a.status[0] = total;
      a.status[1] = taken;
      a.status[2] = freed;
      a.status[3] = s_denied;
    }
  }
  __syncthreads();
  const int gt = blockIdx.x * kPlanThreads + tid, gs = gridDim.x * kPlanThreads;
  for (int j = gt; j < taken; j += gs) {
    const int b = find_seq(cp, B, j);
    const int lp = pages(min(static_cast<long long>(max(a.old_len[b], 0)), cap)) + j - cp[b];
    a.table[b * a.table_stride + lp] = a.ring[wrap(static_cast<long long>(head) + j)];
  }
  for (int j = gt; j < freed; j += gs) {
    const int b = find_seq(cf, B, j);
    const int lp = pages(a.new_len[b]) + j - cf[b];
    a.ring[wrap(static_cast<long long>(head) + count + j)] = a.table[b * a.table_stride + lp];
  }
  // slots, 4 per lane: a warp takes a run of consecutive tokens, so it searches its first
  // sequence once and then only moves on
  const int words = (a.max_tokens + 3) / 4, warps = gs >> 5, run = ((words + warps - 1) / warps + 31) & ~31;
  int b = -1;
  for (int j = (gt >> 5) * run + (tid & 31), j1 = min(words, (gt >> 5) * run + run); j < j1; j += 32) {
    int s[4] = {-1, -1, -1, -1};
    const int t0 = 4 * j;
    if (t0 < total) {
      if (b < 0) b = find_seq(cu, B, t0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + u;
        if (t >= total) break;
        while (cu[b + 1] <= t) ++b;
        const int o = static_cast<int>(min(static_cast<long long>(max(a.old_len[b], 0)), cap)), n0 = pages(o);
        const int pos = o + t - cu[b], lp = pos >> a.pshift;
        const int page = lp < n0 ? a.table[b * a.table_stride + lp]
                                 : a.ring[wrap(static_cast<long long>(head) + cp[b] + lp - n0)];
        s[u] = static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages) ? (page << a.pshift) + (pos & (P - 1)) : -1;
      }
    }
    if (t0 + 3 < a.max_tokens) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
      for (int u = 0; t0 + u < a.max_tokens; ++u) a.slots[t0 + u] = s[u];
    }
  }
}

// ---------------------------------------------------------------- append

// A CTA copies `rows` rows (16 bytes per thread and step) into their slots and then makes the
// summaries of the pages that these rows complete:
//   m = fl32(mean of the page's P rows), scale = fl32(max |m| * fl32(1 / 127)),
//   code = rint(fl32(m / scale)); a page whose mean is not finite gets scale NaN and codes 0.
// The sum is kept as an unevaluated pair of fp32 (two-sum), so m is the rounded exact mean for any
// order of the rows. A page's rows are read where this call does not write: the rows of this call
// from k_new (usually just copied, so from the L1), the older ones from the cache; so the copy and
// the summaries need no second launch. What bounds it is the copy: each row read and written once.
__device__ __forceinline__ void two_sum(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), bb = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, bb)), __fsub_rn(x, bb)));
  hi = s;
}

constexpr int kAppThreads = 256, kAppRows = 64;  // threads, most rows of a CTA

template <typename T>
__global__ void __launch_bounds__(kAppThreads)
    k_page_append(const __grid_constant__ Cache c, const uint4* kn, const uint4* vn, long long row_k, long long row_v,
                  const int* slots, int n, int rows) {
  pdl_enter();
  __shared__ int slot_s[kAppRows], done[kAppRows], ndone;
  const int tid = threadIdx.x, P = 1 << c.pshift, t0 = blockIdx.x * rows, nr = min(rows, n - t0);
  constexpr int VE = Elem<T>::kVec;
  const int vph = c.d / VE, vpr = c.nkv * vph;  // 16-byte vectors of a head and of a row
  if (tid == 0) ndone = 0;
  __syncthreads();
  if (tid < nr) {
    const int slot = slots[t0 + tid];
    const bool ok = slot >= 0 && (slot >> c.pshift) < c.n_pages;
    slot_s[tid] = ok ? slot : -1;
    if (ok && c.codes && (slot & (P - 1)) == P - 1) done[atomicAdd(&ndone, 1)] = t0 + tid;
  }
  __syncthreads();
  {
    constexpr int U = 4;
    const int total = nr * vpr;
    for (int i0 = tid; i0 < total; i0 += U * kAppThreads) {
      uint4 x[U], y[U];
      size_t at[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kAppThreads, r = i / vpr, v = i - r * vpr;
        on[u] = i < total && slot_s[r] >= 0;
        if (!on[u]) continue;
        const int h = c.nkv == 1 ? 0 : v / vph, slot = slot_s[r];
        at[u] = (static_cast<size_t>(slot >> c.pshift) * c.sp + static_cast<size_t>(slot & (P - 1)) * c.st +
                 static_cast<size_t>(h) * c.sh) / VE + (v - h * vph);
        x[u] = __ldg(kn + (t0 + r) * row_k + v);
        if (c.v) y[u] = __ldcs(vn + (t0 + r) * row_v + v);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!on[u]) continue;
        static_cast<uint4*>(c.k)[at[u]] = x[u];
        if (c.v) static_cast<uint4*>(c.v)[at[u]] = y[u];
      }
    }
  }
  if (!c.codes) return;
  __shared__ int src[256], missing;           // row of this call for each row of the page, or -1
  __shared__ float part[2][kAppThreads * 8];
  __shared__ float red[kAppThreads / 32];
  int lanes = 1;
  while (lanes < vph) lanes <<= 1;
  const int par = kAppThreads / lanes, v = tid & (lanes - 1), r0 = tid / lanes;
  const int pages = ndone;
  for (int it = 0; it < pages; ++it) {
    const int t = done[it], page = slot_s[t - t0] >> c.pshift;
    if (tid == 0) missing = 0;
    __syncthreads();
    if (tid < P) {  // the rows that usually come right before the last one
      const int ti = t - (P - 1 - tid);
      const bool here = ti >= 0 && slots[ti] == (page << c.pshift) + tid;
      src[tid] = here ? ti : -1;
      if (!here) missing = 1;
    }
    __syncthreads();
    if (missing) {  // else older rows, or rows of this call in another order
      for (int i = tid; i < n; i += kAppThreads) {
        const int slot = slots[i];
        if (slot >= 0 && slot >> c.pshift == page) src[slot & (P - 1)] = i;
      }
      __syncthreads();
    }
    for (int g = 0; g < c.nkv; ++g) {
      const T* base = static_cast<const T*>(c.k) + static_cast<size_t>(page) * c.sp + static_cast<size_t>(g) * c.sh;
      float hi[VE], lo[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) hi[e] = lo[e] = 0.f;
      if (v < vph) {
#pragma unroll 4
        for (int r = r0; r < P; r += par) {
          const int ti = src[r];
          const T* row = ti >= 0 ? reinterpret_cast<const T*>(kn + ti * row_k + g * vph) : base + r * c.st;
          float x[VE];
          load_vec(row + v * VE, x);
#pragma unroll
          for (int e = 0; e < VE; ++e) two_sum(hi[e], lo[e], x[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        part[0][e * kAppThreads + tid] = hi[e];
        part[1][e * kAppThreads + tid] = lo[e];
      }
      __syncthreads();
      float m[VE], mx = 0.f;
      bool fin = true;
      if (tid < lanes && v < vph) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          float h = part[0][e * kAppThreads + tid], l = part[1][e * kAppThreads + tid];
          for (int r = 1; r < par; ++r) {
            two_sum(h, l, part[0][e * kAppThreads + tid + r * lanes]);
            l += part[1][e * kAppThreads + tid + r * lanes];
          }
          m[e] = __fmul_rn(__fadd_rn(h, l), 1.0f / P);
          fin = fin && isfinite(m[e]);
          mx = fmaxf(mx, fabsf(m[e]));
        }
      }
      mx = warp_max(fin ? mx : INFINITY);
      if ((tid & 31) == 0) red[tid >> 5] = mx;
      __syncthreads();
      mx = 0.f;
#pragma unroll
      for (int w = 0; w < kAppThreads / 32; ++w) mx = fmaxf(mx, red[w]);
      const float scale = __fmul_rn(mx, 1.0f / 127.0f);
      if (tid < lanes && v < vph) {
        __align__(8) signed char q[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float f = scale > 0.f && isfinite(scale) ? rintf(__fdiv_rn(m[e], scale)) : 0.f;
          q[e] = static_cast<signed char>(fminf(fmaxf(f, -127.f), 127.f));
        }
        signed char* out = c.codes + (static_cast<size_t>(page) * c.nkv + g) * c.d + v * VE;
        if (VE == 8)
          *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(q);
        else
          *reinterpret_cast<unsigned*>(out) = *reinterpret_cast<const unsigned*>(q);
      }
      if (tid == 0) c.scales[static_cast<size_t>(page) * c.nkv + g] = isfinite(scale) ? scale : NAN;
      __syncthreads();
    }
  }
}

}  // namespace pg

#define MTP_PG_CHECK(what)                                              \
  do {                                                                  \
    const cudaError_t e_ = cudaGetLastError();                          \
    if (e_ != cudaSuccess) {                                            \
      set_error("%s launch: %s", what, cudaGetErrorString(e_));         \
      return MTP_ERR_CUDA;                                              \
    }                                                                   \
  } while (0)

int run_page_plan(const int* old_len, const int* new_len, int B, int* table, long long table_stride, int max_pages,
                  int* ring, int n_pages, const int* state, int pshift, int max_tokens, int* len_out, int* slots,
                  int* cu_new, int* state_out, int* status, int num_sms, cudaStream_t st) {
  const pg::PlanArgs a{old_len, new_len, state, table, ring, len_out, slots, cu_new, state_out, status,
                       table_stride, B, max_pages, n_pages, pshift, max_tokens};
  const int smem = 3 * (B + 1) * 4;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(pg::k_page_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
      set_error("page plan: %s", cudaGetErrorString(e));
      return MTP_ERR_CUDA;
    }
  }
  long long grid = (static_cast<long long>(max_tokens) / 4 + B) / pg::kPlanThreads + 1;
  if (grid > num_sms) grid = num_sms;
  pg::k_page_plan<<<static_cast<int>(grid), pg::kPlanThreads, smem, st>>>(a);
  MTP_PG_CHECK("page plan");
  return MTP_OK;
}

int run_page_append(const pg::Cache& c, const void* k_new, const void* v_new, long long row_k, long long row_v,
                    const int* slots, int T, int num_sms, cudaStream_t st) {
  if (T == 0) return MTP_OK;
  const int es = c.f32 ? 4 : 2;
  // rows of a CTA: about 6 CTAs per SM, so that all of them run at once
  int rows = pg::kAppRows;
  while (rows > 1 && (T + rows - 1) / rows < 6 * num_sms) rows >>= 1;
  const int grid = (T + rows - 1) / rows;
  const uint4 *k = static_cast<const uint4*>(k_new), *v = static_cast<const uint4*>(v_new);
  const long long rk = row_k * es / 16, rv = row_v * es / 16;
  if (c.f32)
    pg::k_page_append<float><<<grid, pg::kAppThreads, 0, st>>>(c, k, v, rk, rv, slots, T, rows);
  else
    pg::k_page_append<__nv_bfloat16><<<grid, pg::kAppThreads, 0, st>>>(c, k, v, rk, rv, slots, T, rows);
  MTP_PG_CHECK("page append");
  return MTP_OK;
}

}  // namespace mtp
