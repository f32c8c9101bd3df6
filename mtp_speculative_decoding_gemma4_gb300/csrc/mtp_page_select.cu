// Selection of the pages a query attends: every page of a sequence is scored by the integer dot
// product of the quantised query with the page's summary (the quantised mean of its keys), and
// the n_select best pages of each KV head are listed in increasing order. The dot product is at
// most 512 * 127 * 127 < 2^24, so it converts to fp32 exactly and a score does not depend on the
// order of its sums: the selected sets are reproducible, ties going to the lower page.
//
// One thread-block cluster per (sequence, KV head): its CTAs score their shares of the pages (one
// read of d + 4 bytes per page, the only large one), and after a cluster barrier the first CTA
// picks. The pick is a chain of small steps on one SM: the range of the scores, the threshold key
// by 8-bit digits from the highest bit in which they differ (so that the first digit already
// spreads over its counters), then one ordered compaction.
//
// What bounds it is that chain: length, table, codes, the cluster barrier, up to 4 digits, the
// compaction, and the code's own first fetches. One sequence of 1024 pages (a cluster of 16) takes
// 8.5 us, 16 sequences of 2048 pages (clusters of 8; 17 MB of codes, 2.5 us at the copy rate) 17.5.
#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelCache = 8192;  // scores that the picking CTA keeps in shared memory

constexpr unsigned kInf = 0xff800000u, kKept = 0xffffffffu;  // ord_f32(+inf); above it: a page that is kept

struct SelArgs {
  Cache c;
  const float* q;
  unsigned* score;  // [B][nkv][max_pages] ordered keys
  int* sel;
  int B, nh, n_select, keep_first, keep_last, cl;
};

// The query heads' codes, packed [G][d / 4], and steps: a warp per head, its values in registers.
__device__ __forceinline__ void quantise(const SelArgs& a, const float* q, int G, int* codes, float* qs) {
  const int d = a.c.d, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nv = d >> 2;  // 4 values each, nv <= 128
  for (int h = warp; h < G; h += kSelWarps) {
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[j] = lane + 32 * j < nv ? reinterpret_cast<const float4*>(q + static_cast<size_t>(h) * d)[lane + 32 * j]
                                : make_float4(0, 0, 0, 0);
    float mx = 0.f;
    bool fin = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x[j].x), fabsf(x[j].y)), fmaxf(fabsf(x[j].z), fabsf(x[j].w))));
      // a sum of |x| * 0 is NaN as soon as one value is not finite
      fin = fin && fabsf(x[j].x) * 0.f + fabsf(x[j].y) * 0.f + fabsf(x[j].z) * 0.f + fabsf(x[j].w) * 0.f == 0.f;
    }
    mx = warp_max(mx);
    fin = __all_sync(0xffffffffu, fin);
    const float step = fin ? __fmul_rn(mx, 1.0f / 127.0f) : 0.f;
    if (lane == 0) qs[h] = step;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      if (lane + 32 * j >= nv) break;
      const float v[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
      unsigned w = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = step > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(v[e], step)), -127.f), 127.f) : 0.f;
        w |= (static_cast<unsigned>(static_cast<int>(f)) & 255u) << (8 * e);
      }
      codes[h * nv + lane + 32 * j] = static_cast<int>(w);
      x[0] = x[1];
      x[1] = x[2];
      x[2] = x[3];
    }
  }
}

// Scores of this CTA's share of n pages: 8 lanes hold a page's codes (VL 16-byte vectors each),
// 4 pages side by side. A warp takes `per` pages at a time, one per lane, and requests its first
// codes before the query is quantised. The warps' loads are enough in flight: with two or four
// groups of pages per warp the longer code costs more than they bring (55 and 53 us against 50
// with the attention after it, 16 sequences of 2048 pages; 21.3 against 20.4 for one of 1024).
template <int VL>
__device__ __forceinline__ void score_pages(const SelArgs& a, int b, int g, int G, int n, int rank, const float* q,
                                            int* codes, float* qs, unsigned* score) {
  const Cache& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane & 7, nv = c.d >> 4;
  // with few pages every warp of the cluster gets some
  const int warps = a.cl * kSelWarps, per = min(32, (n + warps - 1) / warps);
  int4 x[VL];
  int page = -1;
  auto fetch = [&](int i) {
    const int at = i + (lane >> 3), p = __shfl_sync(0xffffffffu, page, at & 31);
    const int4* row = reinterpret_cast<const int4*>(c.codes + (static_cast<size_t>(max(p, 0)) * c.nkv + g) * c.d);
#pragma unroll
    for (int v = 0; v < VL; ++v)
      x[v] = at < per && p >= 0 && li + 8 * v < nv ? __ldcs(row + li + 8 * v) : make_int4(0, 0, 0, 0);
  };
  bool first = true;
  for (int i0 = (rank * kSelWarps + warp) * per; i0 < n || first; i0 += warps * per) {
    const int lp = lane < per ? i0 + lane : n;
    page = lp < n ? phys_page(c, b, lp) : -1;
    fetch(0);
    const float ks = page >= 0 ? c.scales[static_cast<size_t>(page) * c.nkv + g] : 0.f;
    if (first) {
      quantise(a, q, G, codes, qs);
      __syncthreads();
      first = false;
    }
    float keep = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < per; i += 4) {
      if (i > 0) fetch(i);
      float s = -INFINITY;
      const float k = __shfl_sync(0xffffffffu, ks, (i + (lane >> 3)) & 31);
#pragma unroll 1
      for (int h = 0; h < G; ++h) {
        int dot = 0;
#pragma unroll
        for (int v = 0; v < VL; ++v) {
          const int4 w = li + 8 * v < nv ? reinterpret_cast<const int4*>(codes)[h * nv + li + 8 * v] : make_int4(0, 0, 0, 0);
          dot = __dp4a(x[v].x, w.x, __dp4a(x[v].y, w.y, __dp4a(x[v].z, w.z, __dp4a(x[v].w, w.w, dot))));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        s = fmaxf(s, __fmul_rn(__fmul_rn(static_cast<float>(dot), qs[h]), k));
      }
      const float v = __shfl_sync(0xffffffffu, s, (lane & 3) * 8);
      if (lane >> 2 == i >> 2) keep = v;
    }
    if (page < 0) keep = -INFINITY;
    if (isnan(ks)) keep = INFINITY;  // a page whose keys are not finite is always read
    if (lp < n) score[lp] = lp < a.keep_first || lp >= n - a.keep_last ? kKept : ord_f32(keep);
  }
}

// The same for a head dim that is no multiple of 16: 4-byte loads, a page at a time.
__device__ __noinline__ void score_pages_any(const SelArgs& a, int b, int g, int G, int n, int rank, const float* q,
                                             int* codes, float* qs, unsigned* score) {
  const Cache& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = c.d >> 2;
  quantise(a, q, G, codes, qs);
  __syncthreads();
  for (int lp = rank * kSelWarps + warp; lp < n; lp += a.cl * kSelWarps) {
    const int page = phys_page(c, b, lp);
    float s = -INFINITY;
    if (page >= 0) {
      const int* row = reinterpret_cast<const int*>(c.codes + (static_cast<size_t>(page) * c.nkv + g) * c.d);
      const float k = c.scales[static_cast<size_t>(page) * c.nkv + g];
      for (int h = 0; h < G; ++h) {
        int dot = 0;
        for (int i = lane; i < nw; i += 32) dot = __dp4a(row[i], codes[h * nw + i], dot);
        dot = __reduce_add_sync(0xffffffffu, dot);
        s = fmaxf(s, __fmul_rn(__fmul_rn(static_cast<float>(dot), qs[h]), k));
      }
      if (isnan(k)) s = INFINITY;
    }
    if (lane == 0) score[lp] = lp < a.keep_first || lp >= n - a.keep_last ? kKept : ord_f32(s);
  }
}

__global__ void __launch_bounds__(kSelThreads) k_page_select(const __grid_constant__ SelArgs a) {
  pdl_enter();
  const Cache& c = a.c;
  const int unit = blockIdx.x / a.cl, rank = blockIdx.x % a.cl, g = unit % c.nkv, b = unit / c.nkv;
  const int d = c.d, G = a.nh / c.nkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = a.n_select;
  extern __shared__ __align__(16) int sm_sel[];  // packed query codes [G][d / 4], steps [G], scores
  float* qs = reinterpret_cast<float*>(sm_sel + G * (d / 4));
  unsigned* cache = reinterpret_cast<unsigned*>(qs + G);
  int lo, L;
  key_range(c, b, 0, lo, L);
  const int P = 1 << c.pshift, n = (L + P - 1) >> c.pshift;
  int* sel = a.sel + static_cast<size_t>(unit) * k;
  if (n <= k) {  // all of them (the whole cluster leaves here)
    for (int i = rank * kSelThreads + tid; i < k; i += a.cl * kSelThreads) sel[i] = i < n ? i : -1;
    return;
  }
  unsigned* score = a.score + static_cast<size_t>(unit) * c.max_pages;
  const float* q = a.q + (static_cast<size_t>(b) * a.nh + g * G) * d;
  if (d % 16 != 0) score_pages_any(a, b, g, G, n, rank, q, sm_sel, qs, score);
  else if (d > 256) score_pages<4>(a, b, g, G, n, rank, q, sm_sel, qs, score);
  else if (d > 128) score_pages<2>(a, b, g, G, n, rank, q, sm_sel, qs, score);
  else score_pages<1>(a, b, g, G, n, rank, q, sm_sel, qs, score);
  // the scores of the whole cluster are in place; only the first CTA goes on
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank != 0) return;

  __shared__ unsigned hist[256], s_key;
  __shared__ int s_left, s_all;
  __shared__ long long wsum[kSelWarps];
  __shared__ unsigned wmin[kSelWarps], wmax[kSelWarps];
  __shared__ int winf[kSelWarps];
  static_assert(kSelWarps <= 32, "the reductions over warps take one lane per warp");
  const bool cached = n <= kSelCache;
  if (cached)
    for (int i = tid; i < n; i += kSelThreads) cache[i] = __ldcg(score + i);
  auto get = [&](int i) { return cached ? cache[i] : __ldcg(score + i); };
  // range of the scores below +inf, and how many are at least that
  unsigned least = 0xffffffffu, most = 0;
  int infs = 0;
  for (int i = tid; i < n; i += kSelThreads) {
    const unsigned x = get(i);
    if (x >= kInf) {
      ++infs;
    } else {
      least = min(least, x);
      most = max(most, x);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  infs = __reduce_add_sync(0xffffffffu, infs);
  if (lane == 0) {
    wmin[warp] = least;
    wmax[warp] = most;
    winf[warp] = infs;
  }
  __syncthreads();
  least = __reduce_min_sync(0xffffffffu, wmin[lane % kSelWarps]);
  most = __reduce_max_sync(0xffffffffu, wmax[lane % kSelWarps]);
  infs = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? winf[lane] : 0);
  // the scores' common leading bits; of those that have them, `left` are selected
  unsigned key = kInf, mask = 0xffffffffu;
  int left = k - a.keep_first - a.keep_last, top = -1;  // top: highest bit in which the scores still differ
  if (infs < k) {
    left = k - infs;
    top = 31 - __clz(least ^ most);  // -1: all equal
    mask = top < 31 ? ~0u << (top + 1) : 0u;
    key = most & mask;
  }
  while (top >= 0) {
    const int shift = max(top - 7, 0);
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const unsigned x = get(i);
      if ((x & mask) == key && x < kInf) atomicAdd(&hist[(x >> shift) & (0xffu >> (7 - (top - shift)))], 1u);
    }
    __syncthreads();
    if (tid < 32) {
      // digits from the top: lane l holds digits 255 - 8 l .. 248 - 8 l
      int h[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += h[j] = static_cast<int>(hist[255 - 8 * tid - j]);
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (tid >= o) before += y;
      }
      before -= sum;
      if (before < left && before + sum >= left) {
        int at = 0, cnt = 0;
        bool found = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!found && before + h[j] >= left) {
            found = true;
            at = j;
            cnt = h[j];
          }
          if (!found) before += h[j];
        }
        s_key = key | (static_cast<unsigned>(255 - 8 * tid - at) << shift);
        s_left = left - before;
        s_all = cnt == left - before;  // every score with these digits is selected
      }
    }
    __syncthreads();
    key = s_key;
    left = s_left;
    mask = ~0u << shift;
    top = shift - 1;
    if (s_all) break;
  }
  // scores above the key are all taken, of those equal to it the first `left`: a run of pages per
  // thread, one prefix sum over (above, equal)
  const bool in_infs = infs >= k;
  auto rank_of = [&](unsigned x) {  // 2: above, 1: equal
    if (x >= kInf) return in_infs && x == kInf ? 1 : 2;
    return in_infs ? 0 : (x & mask) > key ? 2 : (x & mask) == key ? 1 : 0;
  };
  const int run = (n + kSelThreads - 1) / kSelThreads, i0 = min(n, tid * run), i1 = min(n, i0 + run);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) {
    const int r = rank_of(get(i));
    mine += r == 2 ? 1ll << 32 : r;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
  for (int w = 0; w < warp; ++w) before += wsum[w];
  int above = static_cast<int>(before >> 32), equal = static_cast<int>(before & 0xffffffffll);
  for (int i = i0; i < i1; ++i) {
    const int r = rank_of(get(i));
    if (r == 2) {
      sel[above + min(equal, left)] = i;
      ++above;
    } else if (r == 1) {
      if (equal < left) sel[above + equal] = i;
      ++equal;
    }
  }
}

}  // namespace pg

long long page_select_workspace(const pg::Cache& c, int B) {
  return 4LL * B * c.nkv * c.max_pages;
}

int run_page_select(const pg::Cache& c, const float* q, int B, int nh, int n_select, int keep_first, int keep_last,
                    int* sel, void* ws, int num_sms, cudaStream_t st) {
  pg::SelArgs a{c, q, static_cast<unsigned*>(ws), sel, B, nh, n_select, keep_first, keep_last, 1};
  const int G = nh / c.nkv, units = B * c.nkv;
  // CTAs of a cluster: one wave over the batch (the last doubling, beyond the portable size, only
  // where clusters of 16 still fit side by side), at least 64 pages each
  while (a.cl < 16 && 2 * a.cl * units <= num_sms - (a.cl == 8 ? num_sms / 8 : 0) && 64 * 2 * a.cl <= c.max_pages)
    a.cl *= 2;
  const int kept = c.max_pages < pg::kSelCache ? c.max_pages : pg::kSelCache;
  const int smem = G * (c.d + 4) + 4 * kept;
  static_assert(32 * (512 + 4) + 4 * pg::kSelCache <= 64 * 1024, "shared memory of the selection");
  cudaError_t e = pg::allow_smem<pg::k_page_select, 64 * 1024>();
  if (e == cudaSuccess && a.cl > 8)
    e = cudaFuncSetAttribute(pg::k_page_select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(units * a.cl);
    cfg.blockDim = dim3(pg::kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    e = cudaLaunchKernelEx(&cfg, pg::k_page_select, a);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("page selection launch: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  return MTP_OK;
}

}  // namespace mtp
