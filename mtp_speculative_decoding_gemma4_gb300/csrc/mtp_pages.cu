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
// entry is both read and written. What bounds it is the chain length, sums, search, table: 5.4 us
// for 8 sequences; 1000 sequences with 2 M slots (8 MB) take 16 us, most of it the slots' lookups.

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
  int b = -1, end = 0, shift = 0, n0 = 0, last = -1, page = -1;  // sequence, its end, position - token; the page at hand
  for (int j = (gt >> 5) * run + (tid & 31), j1 = min(words, (gt >> 5) * run + run); j < j1; j += 32) {
    int s[4] = {-1, -1, -1, -1};
    const int t0 = 4 * j;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u;
      if (t >= total) break;
      if (t >= end) {
        b = b < 0 ? find_seq(cu, B, t) : b + 1;
        while (cu[b + 1] <= t) ++b;
        end = cu[b + 1];
        const int o = static_cast<int>(min(static_cast<long long>(max(a.old_len[b], 0)), cap));
        shift = o - cu[b];
        n0 = pages(o);
        last = -1;
      }
      const int pos = t + shift, lp = pos >> a.pshift;
      if (lp != last) {
        last = lp;
        page = lp < n0 ? a.table[b * a.table_stride + lp] : a.ring[wrap(static_cast<long long>(head) + cp[b] + lp - n0)];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) page = -1;
      }
      s[u] = page >= 0 ? (page << a.pshift) + (pos & (P - 1)) : -1;
    }
    if (t0 + 3 < a.max_tokens) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
      for (int u = 0; t0 + u < a.max_tokens; ++u) a.slots[t0 + u] = s[u];
    }
  }
}

// ---------------------------------------------------------------- append

// Rows of a call into their slots, 16 bytes per thread and step. With summaries a page's sum is
// taken as its rows pass through: a run is a stretch of rows in consecutive slots of one page, and
// the CTA in whose share a run begins copies all of it and, where it completes the page, makes
//   m = fl32(mean of the page's P rows), scale = fl32(max |m| * fl32(1 / 127)),
//   code = rint(fl32(m / scale)); a page whose mean is not finite gets scale NaN and codes 0.
// Every row enters as x / P (a power of two: exact), so that no sum leaves the range that the mean
// lies in. The sum is an unevaluated pair of fp32: hi, and in lo the running sum of what each
// addition to hi rounded away (two-sum, 7 operations a value with the scaling, two values in each).
// lo loses nothing while the values' spread is below 2^24 (bf16, any P): m is then the exact mean,
// rounded once, in any order of the rows. Beyond that, and in fp32, lo's own roundings add at most
// P^2 2^-48 of the largest value. The page's other rows are read where the launch does not write:
// rows of this call in another order from k_new, older ones from the cache; so up to kAppScan rows
// one launch does. What bounds it is the copy: each row read and written once, 134 MB for two
// prompts of 32768 rows at d = 512 in 26 us (5.2 TB/s); with two-sums of one value each 26.5. (Four
// bf16 rows added in fp32 before they enter the pair would take 25, but lose the mean where large
// values cancel.)

// hi + lo += x
__device__ __forceinline__ void two_sum(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), bb = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, bb)), __fsub_rn(x, bb)));
  hi = s;
}
// Packed instructions: two values an issue slot.
__device__ __forceinline__ unsigned long long& u64(float2& a) { return reinterpret_cast<unsigned long long&>(a); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(u64(a)) : "l"(u64(b)));
  return a;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  asm("sub.rn.f32x2 %0, %0, %1;" : "+l"(u64(a)) : "l"(u64(b)));
  return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(u64(c)) : "l"(u64(a)), "l"(u64(b)));
  return c;
}
// hi + lo += x * f for two sums at once, f a power of two.
__device__ __forceinline__ void two_sum2(float2& hi, float2& lo, float2 x, float2 f) {
  const float2 s = fma2(x, f, hi), b = sub2(hi, s);
  lo = add2(lo, add2(sub2(hi, add2(s, b)), fma2(x, f, b)));
  hi = s;
}
constexpr int kAppThreads = 256, kAppRows = 64;  // threads, most rows of a CTA's share
// Most rows of a call whose pages are all summed in one launch. There a run that completes a page
// without covering it looks through all slots of the call, so that the work grows with the square
// of the rows where they come in any order: 12 ms for 2^19 rows at P = 16, d = 8, against 2.3 ms
// where a second launch sums such pages, finding every row in the cache. 131072 rows in order at
// P = 64, d = 512 take 54 us in one launch and 59 in two when they begin with a page, 89 and 64 when
// they begin inside one.
constexpr int kAppScan = 1 << 16;

struct AppArgs {
  Cache c;
  const uint4 *kn, *vn;   // new rows
  long long row_k, row_v; // 16-byte vectors between them
  const int* slots;
  int n, rows;            // rows of the call, of a CTA's share
  int vph, vshift;        // vectors of a head; log2 of a row's (-1: no power of two)
};

// The copy alone.
template <typename T>
__global__ void __launch_bounds__(kAppThreads) k_page_append(const __grid_constant__ AppArgs a) {
  pdl_enter();
  __shared__ long long dst_s[kAppRows];  // first 16-byte vector of a row's place in the cache, or -1
  const Cache& c = a.c;
  constexpr int VE = Elem<T>::kVec, U = 4;
  const int tid = threadIdx.x, P = 1 << c.pshift, t0 = blockIdx.x * a.rows, nr = min(a.rows, a.n - t0);
  const int vpr = c.nkv * a.vph, total = nr * vpr;
  if (tid < nr) {
    const int slot = a.slots[t0 + tid];
    const bool ok = slot >= 0 && (slot >> c.pshift) < c.n_pages;
    dst_s[tid] = ok ? ((slot >> c.pshift) * c.sp + (slot & (P - 1)) * c.st) / VE : -1;
  }
  __syncthreads();
  for (int i0 = tid; i0 < total; i0 += U * kAppThreads) {
    uint4 x[U], y[U];
    long long at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kAppThreads, r = a.vshift >= 0 ? i >> a.vshift : i / vpr, v = i - r * vpr;
      at[u] = i < total ? dst_s[r] : -1;
      if (at[u] < 0) continue;
      at[u] += v;
      if (c.nkv > 1) at[u] += v / a.vph * (c.sh / VE - a.vph);  // a head begins c.sh elements after the one before
      x[u] = __ldcs(a.kn + (t0 + r) * a.row_k + v);
      if (c.v) y[u] = __ldcs(a.vn + (t0 + r) * a.row_v + v);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] < 0) continue;
      static_cast<uint4*>(c.k)[at[u]] = x[u];
      if (c.v) static_cast<uint4*>(c.v)[at[u]] = y[u];
    }
  }
}

// The copy with the summaries of the pages that it completes: all of them (kOne), or those that a
// run covers (kFirst), the others from the cache in a launch behind it that copies nothing (kRest).
enum AppPart { kOne, kFirst, kRest };
template <typename T, AppPart PART>
__global__ void __launch_bounds__(kAppThreads, 4) k_page_append_sum(const __grid_constant__ AppArgs a) {
  pdl_enter();
  constexpr int VE = Elem<T>::kVec;
  const Cache& c = a.c;
  const int tid = threadIdx.x, P = 1 << c.pshift, t0 = blockIdx.x * a.rows, nr = min(a.rows, a.n - t0);
  __shared__ int win[kAppRows + 257];    // slots of rows t0 - 1 .. t0 + nr + P - 1 (-2: no slot)
  __shared__ int begin[kAppRows], nbegin, run_len;
  __shared__ int src[256];               // row of this call for each row of the page, or -1
  __shared__ float part[2][kAppThreads * 8];
  __shared__ int hmax[kAppThreads];      // max |m| of each head of a block of columns, as an integer
  if (tid == 0) nbegin = 0;
  const int slot_end = c.n_pages << c.pshift;
  for (int i = tid; i < nr + P; i += kAppThreads) {
    const int t = t0 - 1 + i, slot = t >= 0 && t < a.n ? a.slots[t] : -1;
    win[i] = slot >= 0 && slot < slot_end ? slot : -2;
  }
  __syncthreads();
  // row t0 + r has slot win[r + 1]; it goes on a run if it follows the row before in the same page
  auto goes_on = [&](int r) { return win[r + 1] == win[r] + 1 && (win[r + 1] & (P - 1)) != 0; };
  if (tid < nr && win[tid + 1] >= 0 && !goes_on(tid)) begin[atomicAdd(&nbegin, 1)] = tid;
  __syncthreads();
  // blocks of whole heads, at most a vector per thread; the threads left over take other rows
  const int hpb = min(c.nkv, max(1, kAppThreads / a.vph)), cols = hpb * a.vph, par = kAppThreads / cols;
  const int r0 = tid / cols, v = tid - r0 * cols, hv = v / a.vph;
  const bool act = r0 < par;
  const int runs = nbegin;
  const float part_of = 1.0f / P;
  for (int it = 0; it < runs; ++it) {
    const int first = begin[it], slot = win[first + 1], page = slot >> c.pshift, off = slot & (P - 1);
    if (tid == 0) run_len = P - off;
    __syncthreads();
    if (tid + 1 < P - off && !goes_on(first + 1 + tid)) atomicMin(&run_len, tid + 1);
    __syncthreads();
    const int len = run_len;
    const bool whole = len == P, done = off + len == P && (PART == kOne || (PART == kFirst) == whole);
    if (PART == kRest && !done) {
      __syncthreads();  // run_len is read
      continue;
    }
    if (PART == kOne && done && !whole) {  // the page's other rows: of this call, or older
      if (tid < P) src[tid] = -1;
      __syncthreads();
      for (int i = tid; i < a.n; i += kAppThreads) {
        const int s = a.slots[i];
        if (s >= 0 && s >> c.pshift == page) src[s & (P - 1)] = i;
      }
    }
    for (int h0 = 0; h0 < c.nkv; h0 += hpb) {
      const int h = h0 + hv;
      const bool on = act && h < c.nkv;
      if (tid < hpb) hmax[tid] = 0;
      __syncthreads();  // src and hmax are set, part of the block before is read
      float2 hi[VE / 2], lo[VE / 2];
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) hi[e] = lo[e] = make_float2(0.f, 0.f);
      auto add = [&](const uint4& u) {
        float x[VE];
        load_vec(reinterpret_cast<const T*>(&u), x);
#pragma unroll
        for (int e = 0; e < VE / 2; ++e)
          two_sum2(hi[e], lo[e], make_float2(x[2 * e], x[2 * e + 1]), make_float2(part_of, part_of));
      };
      if (on) {
        const long long at = (page * c.sp + (off + r0) * c.st + h * c.sh) / VE + (v - hv * a.vph);
        const long long st = c.st / VE * par, row = t0 + first + r0, col = h0 * a.vph + v;
        // loads of 4 rows, then their stores
        auto pass = [&](const uint4* from, long long step, uint4* to, bool sum) {
          for (int r = r0; r < len; r += 4 * par) {
            uint4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = r + u * par < len ? __ldcs(from + u * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (r + u * par < len) to[u * st] = x[u];
            if (sum) {
#pragma unroll
              for (int u = 0; u < 4; ++u) add(x[u]);  // rows that are not there are zero
            }
            from += 4 * step;
            to += 4 * st;
          }
        };
        if (PART != kRest) {
          pass(a.kn + row * a.row_k + col, par * a.row_k, static_cast<uint4*>(c.k) + at, done);
          if (c.v) pass(a.vn + row * a.row_v + col, par * a.row_v, static_cast<uint4*>(c.v) + at, false);
        }
        if (PART != kFirst && done && !whole) {
          const uint4* old = static_cast<const uint4*>(c.k) + (page * c.sp + h * c.sh) / VE + (v - hv * a.vph);
#pragma unroll 4
          for (int r = r0; r < (PART == kRest ? P : off); r += par) {
            const int ti = PART == kRest ? -1 : src[r];
            add(ti >= 0 ? a.kn[ti * a.row_k + col] : old[r * (c.st / VE)]);
          }
        }
      }
      if (!done) continue;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        part[0][e * kAppThreads + tid] = e & 1 ? hi[e / 2].y : hi[e / 2].x;
        part[1][e * kAppThreads + tid] = e & 1 ? lo[e / 2].y : lo[e / 2].x;
      }
      __syncthreads();
      float m[VE];
      if (on && r0 == 0) {
        float mx = 0.f;
        bool fin = true;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          float x = part[0][e * kAppThreads + tid], l = part[1][e * kAppThreads + tid];
          for (int r = 1; r < par; ++r) {
            two_sum(x, l, part[0][e * kAppThreads + tid + r * cols]);
            l += part[1][e * kAppThreads + tid + r * cols];
          }
          m[e] = __fadd_rn(x, l);
          fin = fin && isfinite(m[e]);
          mx = fmaxf(mx, fabsf(m[e]));
        }
        atomicMax(&hmax[hv], __float_as_int(fin ? mx : INFINITY));
      }
      __syncthreads();
      if (on && r0 == 0) {
        const float scale = __fmul_rn(__int_as_float(hmax[hv]), 1.0f / 127.0f);
        __align__(8) signed char q[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float f = scale > 0.f && isfinite(scale) ? rintf(__fdiv_rn(m[e], scale)) : 0.f;
          q[e] = static_cast<signed char>(fminf(fmaxf(f, -127.f), 127.f));
        }
        const int i = v - hv * a.vph;
        signed char* out = c.codes + (static_cast<size_t>(page) * c.nkv + h) * c.d + i * VE;
        if (VE == 8)
          *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(q);
        else
          *reinterpret_cast<unsigned*>(out) = *reinterpret_cast<const unsigned*>(q);
        if (i == 0) c.scales[static_cast<size_t>(page) * c.nkv + h] = isfinite(scale) ? scale : NAN;
      }
      __syncthreads();
    }
  }
}

}  // namespace pg

int run_page_plan(const int* old_len, const int* new_len, int B, int* table, long long table_stride, int max_pages,
                  int* ring, int n_pages, const int* state, int pshift, int max_tokens, int* len_out, int* slots,
                  int* cu_new, int* state_out, int* status, int num_sms, cudaStream_t st) {
  const pg::PlanArgs a{old_len, new_len, state, table, ring, len_out, slots, cu_new, state_out, status,
                       table_stride, B, max_pages, n_pages, pshift, max_tokens};
  const int smem = 3 * (B + 1) * 4;
  // always the most that a call can need: another thread's call may be between this and its launch
  const cudaError_t e = pg::allow_smem<pg::k_page_plan, 3 * (pg::kPlanMaxB + 1) * 4>();
  if (e != cudaSuccess) {
    set_error("page plan: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  long long grid = (static_cast<long long>(max_tokens) / 4 + B) / pg::kPlanThreads + 1;
  if (grid > num_sms) grid = num_sms;
  return pg::launch_pdl("page plan", pg::k_page_plan, dim3(static_cast<unsigned>(grid)), pg::kPlanThreads, smem, st, a);
}

int run_page_append(const pg::Cache& c, const void* k_new, const void* v_new, long long row_k, long long row_v,
                    const int* slots, int T, int num_sms, cudaStream_t st) {
  if (T == 0) return MTP_OK;
  const int es = c.f32 ? 4 : 2;
  pg::AppArgs a{c, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), row_k * es / 16, row_v * es / 16,
                slots, T, pg::kAppRows, c.d * es / 16, 0};
  // about 6 CTAs per SM, so that all of them run at once
  while (a.rows > 1 && (T + a.rows - 1) / a.rows < 6 * num_sms) a.rows >>= 1;
  const int vpr = c.nkv * a.vph;
  while ((1 << a.vshift) < vpr) ++a.vshift;
  if ((1 << a.vshift) != vpr) a.vshift = -1;
  const auto launch = [&](void (*f32)(pg::AppArgs), void (*bf16)(pg::AppArgs)) {
    return pg::launch_pdl("page append", c.f32 ? f32 : bf16, dim3((T + a.rows - 1) / a.rows), pg::kAppThreads, 0, st, a);
  };
  using bf = __nv_bfloat16;
  if (!c.codes) return launch(pg::k_page_append<float>, pg::k_page_append<bf>);
  if (T <= pg::kAppScan) return launch(pg::k_page_append_sum<float, pg::kOne>, pg::k_page_append_sum<bf, pg::kOne>);
  const int rc = launch(pg::k_page_append_sum<float, pg::kFirst>, pg::k_page_append_sum<bf, pg::kFirst>);
  return rc ? rc : launch(pg::k_page_append_sum<float, pg::kRest>, pg::k_page_append_sum<bf, pg::kRest>);
}

}  // namespace mtp
