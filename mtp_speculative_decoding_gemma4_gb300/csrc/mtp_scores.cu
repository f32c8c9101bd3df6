// Log probabilities of given tokens under rows of logits at a temperature, with the rows' entropies
// and their k most probable tokens, in one pass over the logits. With d_i = (x_i - m) log2(e) / T,
// e_i = 2^d_i, S = sum e_i and W = sum e_i d_i for any m near the maximum:
//   log p_t = (x_t - m) / T - ln S,   H = -sum p_i ln p_i = ln 2 (log2 S - W / S).
// Every thread keeps (m, S, W) of its elements under a maximum of its own; the parts are joined
// exactly: from m to m', S' = 2^a S and W' = 2^a (W + a S) with a = (m - m') log2(e) / T.
//
// The k largest: a key is (value, index) as one 64-bit number, so that all are different and ties go
// to the lowest index. A CTA keeps a list of candidates and a bar, the k-th best value so far; an
// element of a later chunk has to exceed it. Where many do (the first chunk, or logits that rise), the
// bar is raised first: the k-th largest of the chunk's 128 group maxima is a lower bound of its k-th
// largest element. By value few more than k elements reach it; where many are equal the same is done by
// key, and then at most k groups have elements at or above it, so the list is bounded whatever the
// logits are. After the first chunk hardly any element passes, and the warps meet only at chunks 0, 4, 16,
// 64, .. to raise the bar (about three times as many elements as asked for pass in between; with a
// meeting at 0, 1, 2, 4, 8, .. 5000 rows of 30000 take 134 us instead of 131 with 20 alternatives, 115
// instead of 108 with 5). Logits that rise with their index, or whose first ones are masked, can
// overfill the list so. Their sums go on, and the list is made in a second pass with a meeting at every
// chunk: 576 rows of 262144 bf16 logits with 20 alternatives take 160 us with the first 8192 masked and
// 281 when rising, 83 otherwise (as called).
//
// A CTA takes a row, or a slice of it where rows are few (k_scores_join then joins the slices). What
// bounds it is reading the logits once: 576 rows of 262144 bf16 logits take 59 us without alternatives
// (5.1 TB/s), 70 with 5 and 78 with 20 of them; issue slots are 70 % busy (an element costs about six
// instructions), and a meeting costs 1 to 2 us of a CTA's time, which other CTAs only partly cover. Five
// rows take 6.7 us without and 10.8 with 5 alternatives, in two launches.
#include <cfloat>
#include <cmath>

#include "mtp_common.cuh"
#include "mtp_f32x2.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace sc {

constexpr int kT = 256;             // threads
constexpr int kU = 4;               // 16-byte vectors of a thread and chunk; the next chunk's are in flight meanwhile
constexpr int kMaxK = 32;
constexpr int kGroups = 128;        // of a chunk's elements
constexpr int kMaxSplits = 64;
constexpr int kCap = kMaxK * (kT * kU * 8 / kGroups) + 2 * kMaxK;  // candidates: kMaxK groups of elements, and what was there

using key_t = unsigned long long;

struct Args {
  const void* x;
  long long stride;                 // elements between rows
  const int* token;
  float* logprob;
  float* entropy;
  int* ids;
  float* best;
  float* ws_sum;                    // [rows][splits][4]: m, S, W
  key_t* ws_key;                    // [rows][splits][k]
  float c, inv_t;                   // log2(e) / T, 1 / T
  int rows, V, k, splits, slice;    // slice: elements of a split, a multiple of a vector's
};

struct Sum {
  float m, s, w;
};

// NaN stays NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// fp32 values as unsigned numbers of the same order (-0 as 0).
__device__ __forceinline__ unsigned order(float v) {
  const unsigned u = __float_as_uint(v + 0.f);
  return u ^ (static_cast<int>(u) < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ key_t make_key(float v, int i) {
  return static_cast<key_t>(order(v)) << 32 | (0xffffffffu - static_cast<unsigned>(i));
}
__device__ __forceinline__ float key_value(key_t k) {
  const unsigned o = static_cast<unsigned>(k >> 32);
  return __uint_as_float(o ^ (o & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int key_index(key_t k) { return static_cast<int>(0xffffffffu - static_cast<unsigned>(k)); }

// Below this exponent a term is 0; kept from -inf, so that 0 * d is 0.
constexpr float kLow = -200.f;

__device__ __forceinline__ void join(Sum& a, const Sum& b, float c) {
  const float m = max_nan(a.m, b.m);
  const float fa = a.m == -INFINITY ? kLow : max_nan((a.m - m) * c, kLow), fb = b.m == -INFINITY ? kLow : max_nan((b.m - m) * c, kLow);
  const float ea = ex2(fa), eb = ex2(fb);
  a.w = ea * fmaf(fa, a.s, a.w) + eb * fmaf(fb, b.s, b.w);
  a.s = fmaf(ea, a.s, eb * b.s);
  a.m = m;
}

template <typename T>
struct Elem2;
template <>
struct Elem2<float> {
  static constexpr int n = 4;
  __device__ static void unpack(const uint4& u, float* v) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  __device__ static float top(const uint4& u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  __device__ static uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
  __device__ static uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Elem2<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static void unpack(const uint4& u, float* v) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static float top(const uint4& u) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ static uint4 none() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  __device__ static uint4 pack(const float* v) {  // (bf16 values: the lower halves are 0)
    auto p = [&](int i) { return __float_as_uint(v[i]) >> 16 | (__float_as_uint(v[i + 1]) & 0xffff0000u); };
    return make_uint4(p(0), p(2), p(4), p(6));
  }
};

struct Shared {
  key_t list[kCap];
  key_t group[kGroups];
  key_t best[kMaxK];
  key_t bar;        // the k-th largest of the group maxima
  alignas(16) float top[kGroups];  // the same by value
  float level;
  int n, n2;        // candidates
  float sum[kT / 32][3];
};

// The k-th largest of the group maxima sh.group (0: fewer are not 0) into sh.bar. All threads.
__device__ void find_bar(Shared& sh, int k) {
  const int tid = threadIdx.x;
  if (tid == 0) sh.bar = 0;
  __syncthreads();
  static_assert(kT == 2 * kGroups, "two threads per group");
  const key_t mine = sh.group[tid / 2];
  int above = 0;
#pragma unroll 8
  for (int i = tid & 1; i < kGroups; i += 2) above += sh.group[i] > mine ? 1 : 0;
  above += __shfl_xor_sync(0xffffffffu, above, 1);
  if (above == k - 1 && mine) sh.bar = mine;  // (keys are different but for those of empty groups)
  __syncthreads();
}

// The list's k largest in descending order into sh.best (0 behind the last), and as its new content.
// All threads; sh.n <= kCap.
__device__ void select(Shared& sh, int k) {
  const int tid = threadIdx.x;
  __syncthreads();
  const int n = sh.n;
  if (n > kGroups) {  // keep what reaches the k-th largest of 128 groups' maxima
    if (tid < kGroups) {
      key_t m = 0;
      for (int i = tid; i < n; i += kGroups) m = sh.list[i] > m ? sh.list[i] : m;
      sh.group[tid] = m;
    }
    if (tid == 0) sh.n2 = 0;
    find_bar(sh, k);
    const key_t bar = sh.bar;
    // (in place: a round's keys are read before any is written, and at most as many are written as read)
    for (int i0 = 0; i0 < n; i0 += kT) {
      const key_t x = i0 + tid < n ? sh.list[i0 + tid] : 0;
      __syncthreads();
      if (x && x >= bar) sh.list[atomicAdd(&sh.n2, 1)] = x;
      __syncthreads();
    }
    if (tid == 0) sh.n = sh.n2;
    __syncthreads();
  }
  const int n2 = sh.n;
  if (tid < kMaxK) sh.best[tid] = 0;
  __syncthreads();
  // four threads count what is above a key
  for (int i0 = 0; i0 + (tid & ~31) / 4 < n2; i0 += kT / 4) {  // (whole warps)
    const int i = i0 + tid / 4;
    const key_t x = i < n2 ? sh.list[i] : 0;
    int above = 0;
#pragma unroll 4
    for (int j = tid & 3; j < n2; j += 4) above += sh.list[j] > x ? 1 : 0;
    above += __shfl_xor_sync(0xffffffffu, above, 1);
    above += __shfl_xor_sync(0xffffffffu, above, 2);
    if (x && above < k) sh.best[above] = x;
  }
  __syncthreads();
  if (tid < kMaxK) sh.list[tid] = sh.best[tid];
  if (tid == 0) sh.n = n2 < k ? n2 : k;
  __syncthreads();
}

__device__ __forceinline__ Sum block_join(Shared& sh, Sum a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sum b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.w, o)};
    // (both lanes join in the same order, so that they agree to the last bit)
    Sum lo = threadIdx.x & o ? b : a;
    join(lo, threadIdx.x & o ? a : b, c);
    a = lo;
  }
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    sh.sum[warp][0] = a.m;
    sh.sum[warp][1] = a.s;
    sh.sum[warp][2] = a.w;
  }
  __syncthreads();
  a = {sh.sum[0][0], sh.sum[0][1], sh.sum[0][2]};
#pragma unroll
  for (int i = 1; i < kT / 32; ++i) join(a, {sh.sum[i][0], sh.sum[i][1], sh.sum[i][2]}, c);
  return a;
}

// A row's outputs from its sums and its k best keys (sh.best). A row without a softmax (a NaN, a +inf,
// nothing above -inf) has S not positive and finite.
template <typename T>
__device__ __forceinline__ void answer(const Args& a, const Shared& sh, int row, const Sum& z) {
  constexpr float kLn2 = 0.6931471805599453f;
  const int tid = threadIdx.x;
  const bool good = z.s > 0.f && z.s < INFINITY && z.m < INFINITY;
  const float ls = log2f(z.s);
  // (not by way of log2, where the type's lowest logits would become -inf; and a difference that leaves the
  // range at a temperature at which it does not is one of quotients)
  auto lp = [&](float x) {
    const float d = x - z.m, y = d < -FLT_MAX ? x * a.inv_t - z.m * a.inv_t : d * a.inv_t;
    return good ? y - kLn2 * ls : NAN;
  };
  if (tid == 0) {
    if (a.logprob) {
      const int t = a.token[row];
      float y = NAN;
      if (static_cast<unsigned>(t) < static_cast<unsigned>(a.V)) {
        const T x = static_cast<const T*>(a.x)[row * a.stride + t];
        y = lp(static_cast<float>(x));
      }
      a.logprob[row] = y;
    }
    if (a.entropy) a.entropy[row] = good ? kLn2 * (ls - z.w / z.s) : NAN;
  }
  if (tid < a.k) {
    const key_t key = sh.best[tid];
    a.ids[static_cast<long long>(row) * a.k + tid] = good ? key_index(key) : -1;
    a.best[static_cast<long long>(row) * a.k + tid] = lp(key_value(key));
  }
}

template <typename T>
__global__ void __launch_bounds__(kT, 4) k_scores(const __grid_constant__ Args a) {
  pdl_enter();
  constexpr int VE = Elem2<T>::n, kChunk = kT * kU * VE;
  __shared__ Shared sh;
  const int tid = threadIdx.x, row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits, k = a.k;
  const T* x = static_cast<const T*>(a.x) + row * a.stride;
  // element i of the row sits i + skew elements behind a 16-byte boundary
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const uint4* base = reinterpret_cast<const uint4*>(x - skew);
  // virtual elements [lo, hi) of a row that begins at `skew`
  const int lo = max(split * a.slice, skew), hi = static_cast<int>(min(static_cast<long long>(a.V) + skew,
                                                                       (split + 1LL) * a.slice));
  if (tid == 0) sh.n = 0;
  __syncthreads();
  Sum z = {-INFINITY, 0.f, 0.f};
  float bar = -INFINITY;  // what an element of a later chunk has to exceed
  bool first = true;
  auto load = [&](uint4* u, int c0) {
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int i = c0 + (j * kT + tid) * VE;
      u[j] = i >= lo && i + VE <= hi ? __ldcs(base + i / VE) : Elem2<T>::none();
    }
    if (c0 < lo || hi - c0 < kChunk) {  // vectors that the row begins or ends in
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        const int i = c0 + (j * kT + tid) * VE;
        if (i < hi && i + VE > lo && !(i >= lo && i + VE <= hi)) {
          float v[VE];
#pragma unroll
          for (int e = 0; e < VE; ++e) v[e] = i + e >= lo && i + e < hi ? static_cast<float>(x[i + e - skew]) : -INFINITY;
          u[j] = Elem2<T>::pack(v);
        }
      }
    }
  };
  // this thread's elements of a chunk that reach `lim` and exceed the bar, into the list while it has room
  auto push = [&](const uint4* u, int c0, float lim) {
    unsigned vecs = 0;
#pragma unroll
    for (int j = 0; j < kU; ++j) vecs |= (Elem2<T>::top(u[j]) >= lim ? 1u : 0u) << j;
#pragma unroll 1
    for (; vecs; vecs &= vecs - 1) {
      const int j = __ffs(vecs) - 1;
      uint4 y = u[0];
#pragma unroll
      for (int q = 1; q < kU; ++q)
        if (q == j) y = u[q];
      float v[VE];
      Elem2<T>::unpack(y, v);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int i = c0 + (j * kT + tid) * VE + e;
        if (i >= lo && i < hi && v[e] >= lim && (first || v[e] > bar)) {
          const int at = atomicAdd(&sh.n, 1);
          if (at < kCap) sh.list[at] = make_key(v[e], i - skew);
        }
      }
    }
  };
  uint4 next[kU];
  bool careful = false;  // the second time over
again:
  if (split * a.slice < hi) load(next, split * a.slice);
#pragma unroll 1
  for (int c0 = split * a.slice, ci = 0; c0 < hi; c0 += kChunk, ++ci) {
    uint4 u[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) u[j] = next[j];
    if (c0 + kChunk < hi) load(next, c0 + kChunk);
    float cm = -INFINITY;
#pragma unroll
    for (int j = 0; j < kU; ++j) cm = fmaxf(cm, Elem2<T>::top(u[j]));
    if (!careful && cm > z.m) {
      if (z.m > -INFINITY) {
        const float f = max_nan((z.m - cm) * a.c, kLow), e = ex2(f);
        z.w = e * fmaf(f, z.s, z.w);
        z.s *= e;
      }
      z.m = cm;
    }
    if (!careful) {
      // (a difference first: scores of the type's lowest value have one, but no product with c)
      const float m = z.m == -INFINITY ? 0.f : -z.m;
      const f2 m2 = two(m, m), c2 = two(a.c, a.c);
      f2 s = two(0.f, 0.f), w = s;
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        float v[VE];
        Elem2<T>::unpack(u[j], v);
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
          float d0, d1;
          split2(mul2(add2(two(v[e], v[e + 1]), m2), c2), d0, d1);
          d0 = max_nan(d0, kLow);
          d1 = max_nan(d1, kLow);
          const f2 p = two(ex2(d0), ex2(d1));
          s = add2(s, p);
          w = fma2(p, two(d0, d1), w);
        }
      }
      float s0, s1, w0, w1;
      split2(s, s0, s1);
      split2(w, w0, w1);
      z.s += s0 + s1;
      z.w += w0 + w1;
    }
    if (k && !careful && ((ci & (ci - 1)) || (ci & 0xaaaaaaab))) {  // (not 0 nor a power of 4 above 1)
      if (cm > bar) push(u, c0, bar);
    } else if (k) {
      __syncthreads();
      const int had = sh.n, over = __syncthreads_count(first || cm > bar);  // (pushes begin behind the barrier)
      if (had > kCap) {
        bar = INFINITY;  // overfull: this list takes no more, and the row is gone over again for another; the sums go on
      } else if (over) {
        // at least `most` candidates may come: the bar is raised first, to the k-th largest of 128 pairs'
        // maxima, which at least k elements reach, and few more unless many are equal
        const int most = over * kU * VE;
        float level = -INFINITY;
        if (first || had + most > kCap) {
          if (had > k) select(sh, k);
          const float other = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 1));
          if (!(tid & 1)) sh.top[tid / 2] = other;
          __syncthreads();
          if (tid < 32) {
            // the 16 leading bits of the k-th largest, one by one: a value that it reaches (comparing each
            // group with all others took most of a meeting)
            unsigned o[kGroups / 32], r = 0;
#pragma unroll
            for (int i = 0; i < kGroups / 32; ++i) o[i] = order(sh.top[32 * i + tid]);
#pragma unroll 1
            for (unsigned bit = 0x80000000u; bit > 0x8000u; bit >>= 1) {
              int n = 0;
#pragma unroll
              for (int i = 0; i < kGroups / 32; ++i) n += __popc(__ballot_sync(0xffffffffu, o[i] >= (r | bit)));
              if (n >= k) r |= bit;
            }
            // (below the lowest finite value there are -inf and, as prefixes, none)
            if (tid == 0) sh.level = r < order(-FLT_MAX) ? -INFINITY : key_value(static_cast<key_t>(r) << 32);
          }
          __syncthreads();
          level = sh.level;
        }
        const int n0 = had > k && (first || had + most > kCap) ? k : had;
        const float lim = fmaxf(level, bar);  // (elements equal to the bar itself are left out below)
        if (level > -INFINITY || !first) push(u, c0, lim);
        // what the list holds decides on branches with barriers: every thread takes the same count, and none
        // pushes elements of the next chunk before all have it
        __syncthreads();
        int now = sh.n;
        __syncthreads();
        if (now > kCap || (first && !(level > -INFINITY))) {
          // Too many are equal (or nothing is above -inf): once more by keys, of which no two are equal, so
          // that at most k groups have elements that reach the k-th largest of the groups' maxima
          key_t mine = 0;
#pragma unroll
          for (int j = 0; j < kU; ++j) {
            float v[VE];
            Elem2<T>::unpack(u[j], v);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              const int i = c0 + (j * kT + tid) * VE + e;
              const key_t x1 = i >= lo && i < hi && (first || v[e] > bar) ? make_key(v[e], i - skew) : 0;
              mine = x1 > mine ? x1 : mine;
            }
          }
          const key_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
          if (!(tid & 1)) sh.group[tid / 2] = mine > other ? mine : other;
          __syncthreads();
          if (tid == 0) sh.n = n0;
          find_bar(sh, k);
          const key_t least = sh.bar;
          if (mine && mine >= least) {
#pragma unroll 1
            for (int j = 0; j < kU; ++j) {
              uint4 y = u[0];
#pragma unroll
              for (int q = 1; q < kU; ++q)
                if (q == j) y = u[q];
              float v[VE];
              Elem2<T>::unpack(y, v);
#pragma unroll
              for (int e = 0; e < VE; ++e) {
                const int i = c0 + (j * kT + tid) * VE + e;
                const key_t x1 = i >= lo && i < hi && (first || v[e] > bar) ? make_key(v[e], i - skew) : 0;
                if (x1 && x1 >= least) sh.list[atomicAdd(&sh.n, 1)] = x1;
              }
            }
          }
          __syncthreads();
          now = sh.n;
          __syncthreads();
        }
        if (first || now > k + kMaxK / 2) {
          select(sh, k);  // (best[] stays as it is until a select behind further barriers)
          bar = now < k ? -INFINITY : key_value(sh.best[k - 1]);
        }
      }
      first = false;
    }
  }
  if (k) {
    __syncthreads();
    const bool full = sh.n > kCap;
    __syncthreads();
    if (full) {
      if (tid == 0) sh.n = 0;
      careful = first = true;
      bar = -INFINITY;
      __syncthreads();
      goto again;
    }
    select(sh, k);
  }
  z = block_join(sh, z, a.c);
  if (a.splits == 1) {
    answer<T>(a, sh, row, z);
    return;
  }
  const long long part = static_cast<long long>(row) * a.splits + split;
  if (tid == 0) *reinterpret_cast<float4*>(a.ws_sum + 4 * part) = make_float4(z.m, z.s, z.w, 0.f);
  if (tid < k) a.ws_key[part * k + tid] = sh.best[tid];
}

// Joins the slices of a row.
template <typename T>
__global__ void __launch_bounds__(kT) k_scores_join(const __grid_constant__ Args a) {
  pdl_enter();
  __shared__ Shared sh;
  const int tid = threadIdx.x, row = blockIdx.x;
  const long long part = static_cast<long long>(row) * a.splits;
  Sum z = {-INFINITY, 0.f, 0.f};
  if (tid < a.splits) {
    const float4 p = *reinterpret_cast<const float4*>(a.ws_sum + 4 * (part + tid));
    z = {p.x, p.y, p.z};
  }
  if (tid == 0) sh.n = 0;
  __syncthreads();
  const int n = a.splits * a.k;
  for (int i = tid; i < n; i += kT) {
    const key_t x = a.ws_key[part * a.k + i];
    if (x) sh.list[atomicAdd(&sh.n, 1)] = x;
  }
  if (a.k) select(sh, a.k);
  z = block_join(sh, z, a.c);
  answer<T>(a, sh, row, z);
}

// Slices of a row: as many CTAs as the GPU holds at once, at least 16384 elements each (5 rows of 262144:
// 11.3 us, 14.6 with slices of 4096, whose lists cost more to join).
int splits_of(int rows, int V, int num_sms) {
  long long n = 4LL * num_sms / rows;
  if (n > V / 16384) n = V / 16384;
  if (n > kMaxSplits) n = kMaxSplits;
  return n < 1 ? 1 : static_cast<int>(n);
}

template <typename T>
int launch(const Args& a, cudaStream_t st) {
  const int rc = pg::launch_pdl("token log probabilities", k_scores<T>, dim3(static_cast<unsigned>(a.rows) * a.splits), kT, 0, st, a);
  if (rc || a.splits == 1) return rc;
  return pg::launch_pdl("token log probabilities' join", k_scores_join<T>, dim3(a.rows), kT, 0, st, a);
}

}  // namespace sc

long long scores_workspace(int rows, int V, int k) {
  // fewer SMs take fewer slices, so this is a bound
  const long long n = sc::splits_of(rows, V, pg::kMaxSms);
  return n > 1 ? n * rows * (16 + 8LL * k) : 0;
}

int run_scores(const void* logits, int f32, long long stride, const int* token, int rows, int V, float temperature,
               int k, float* logprob, float* entropy, int* ids, float* best, void* ws, int num_sms, cudaStream_t st) {
  sc::Args a;
  a.x = logits;
  a.stride = stride;
  a.token = token;
  a.logprob = logprob;
  a.entropy = entropy;
  a.ids = ids;
  a.best = best;
  a.c = static_cast<float>(1.4426950408889634 / temperature);
  a.inv_t = static_cast<float>(1.0 / temperature);
  a.rows = rows;
  a.V = V;
  a.k = k;
  a.splits = sc::splits_of(rows, V, num_sms);
  const int ve = f32 ? 4 : 8;
  a.slice = static_cast<int>((static_cast<long long>(V) + ve + a.splits - 1) / a.splits + ve - 1) / ve * ve;  // (a row begins inside a vector)
  a.ws_sum = static_cast<float*>(ws);
  a.ws_key = reinterpret_cast<sc::key_t*>(a.ws_sum + 4LL * rows * a.splits);
  return f32 ? sc::launch<float>(a, st) : sc::launch<__nv_bfloat16>(a, st);
}

}  // namespace mtp
