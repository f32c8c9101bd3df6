// Selection of the pages a query attends: every page of a sequence is scored by the integer dot
// product of the quantised query with the page's summary (the quantised mean of its keys), and
// the n_select best pages of each KV head are listed in increasing order. The dot product is at
// most 512 * 127 * 127 < 2^24, so it converts to fp32 exactly and a score does not depend on the
// order of its sums: the selected sets are reproducible, ties going to the lower page.
//
// One thread-block cluster per (sequence, KV head): its CTAs score their shares of the pages (one
// read of d + 4 bytes per page, the only large one), and after a cluster barrier the first CTA
// picks. The pick is a chain of small steps on one SM: the threshold key by 8-bit digits from the
// top (one count per distinct digit of a warp, not one atomic per score: most scores share their
// leading bits), then one ordered compaction.
#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelCache = 8192;  // scores that the picking CTA keeps in shared memory

struct SelArgs {
  Cache c;
  const float* q;
  unsigned* score;  // [B][nkv][max_pages] ordered keys
  int* sel;
  int B, nh, n_select, keep_first, keep_last, cl;
};

// Scores of 32 pages, one per lane, with 16-byte loads: LP lanes hold a page's codes (d / 16
// vectors), 32 / LP pages side by side, four such groups in flight.
template <int LP>
__device__ __forceinline__ float score32(const SelArgs& a, int g, int G, int page, float ks, const int4* qc, const float* qs) {
  const Cache& c = a.c;
  constexpr int PW = 32 / LP, U = LP < 4 ? LP : 4;
  const int lane = threadIdx.x & 31, li = lane & (LP - 1), nv = c.d >> 4;
  float keep = -INFINITY;
#pragma unroll 1
  for (int it = 0; it < LP; it += U) {
    int4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = __shfl_sync(0xffffffffu, page, (it + u) * PW + lane / LP);
      x[u] = p >= 0 && li < nv ? __ldcs(reinterpret_cast<const int4*>(c.codes + (static_cast<size_t>(p) * c.nkv + g) * c.d) + li)
                               : make_int4(0, 0, 0, 0);
    }
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = -INFINITY;
    float k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) k[u] = __shfl_sync(0xffffffffu, ks, (it + u) * PW + lane / LP);
#pragma unroll 2
    for (int h = 0; h < G; ++h) {
      const int4 q = li < nv ? qc[h * nv + li] : make_int4(0, 0, 0, 0);
      const float step = qs[h];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int dot = __dp4a(x[u].x, q.x, __dp4a(x[u].y, q.y, __dp4a(x[u].z, q.z, __dp4a(x[u].w, q.w, 0))));
        if (LP == 32) {
          dot = __reduce_add_sync(0xffffffffu, dot);
        } else {
#pragma unroll
          for (int o = LP / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        s[u] = fmaxf(s[u], __fmul_rn(__fmul_rn(static_cast<float>(dot), step), k[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float v = __shfl_sync(0xffffffffu, s[u], (lane & (PW - 1)) * LP);
      if (lane / PW == it + u) keep = v;
    }
  }
  return keep;
}

// The same for a head dim that is no multiple of 16: 4-byte loads, a page at a time.
__device__ __noinline__ float score32_any(const SelArgs& a, int g, int G, int page, float ks, const int* qc, const float* qs) {
  const Cache& c = a.c;
  const int lane = threadIdx.x & 31, nw = c.d >> 2;
  float keep = -INFINITY;
  for (int p = 0; p < 32; ++p) {
    const int pg = __shfl_sync(0xffffffffu, page, p);
    if (pg < 0) continue;
    const int* row = reinterpret_cast<const int*>(c.codes + (static_cast<size_t>(pg) * c.nkv + g) * c.d);
    const float k = __shfl_sync(0xffffffffu, ks, p);
    float s = -INFINITY;
    for (int h = 0; h < G; ++h) {
      int dot = 0;
      for (int i = lane; i < nw; i += 32) dot = __dp4a(row[i], qc[h * nw + i], dot);
      dot = __reduce_add_sync(0xffffffffu, dot);
      s = fmaxf(s, __fmul_rn(__fmul_rn(static_cast<float>(dot), qs[h]), k));
    }
    if (lane == p) keep = s;
  }
  return keep;
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
  for (int h = warp; h < G; h += kSelWarps) {
    const float* q = a.q + (static_cast<size_t>(b) * a.nh + g * G + h) * d;
    float mx = 0.f;
    bool fin = true;
    for (int i = lane; i < d; i += 32) {
      mx = fmaxf(mx, fabsf(q[i]));
      fin = fin && isfinite(q[i]);
    }
    mx = warp_max(mx);
    fin = __all_sync(0xffffffffu, fin);
    const float step = fin ? __fmul_rn(mx, 1.0f / 127.0f) : 0.f;
    if (lane == 0) qs[h] = step;
    signed char* out = reinterpret_cast<signed char*>(sm_sel + h * (d / 4));
    for (int i = lane; i < d; i += 32)
      out[i] = step > 0.f ? static_cast<signed char>(fminf(fmaxf(rintf(__fdiv_rn(q[i], step)), -127.f), 127.f)) : 0;
  }
  __syncthreads();
  const int4* qc = reinterpret_cast<const int4*>(sm_sel);
  for (int i0 = (rank * kSelWarps + warp) * 32; i0 < n; i0 += a.cl * kSelWarps * 32) {
    const int lp = i0 + lane;
    const int page = lp < n ? phys_page(c, b, lp) : -1;
    const float ks = page >= 0 ? c.scales[static_cast<size_t>(page) * c.nkv + g] : 0.f;
    float s;
    if (d % 16 != 0) s = score32_any(a, g, G, page, ks, sm_sel, qs);
    else if (d > 256) s = score32<32>(a, g, G, page, ks, qc, qs);
    else if (d > 128) s = score32<16>(a, g, G, page, ks, qc, qs);
    else if (d > 64) s = score32<8>(a, g, G, page, ks, qc, qs);
    else s = score32<4>(a, g, G, page, ks, qc, qs);
    if (page < 0) s = -INFINITY;
    if (isnan(ks)) s = INFINITY;  // a page whose keys are not finite is always read
    if (lp < a.keep_first || lp >= n - a.keep_last) s = INFINITY;
    if (lp < n) score[lp] = ord_f32(s);
  }
  // the scores of the whole cluster are in place; only the first CTA goes on
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank != 0) return;

  __shared__ unsigned hist[256], s_key;
  __shared__ int s_left, s_all;
  __shared__ long long wsum[kSelWarps];
  const bool cached = n <= kSelCache;
  if (cached)
    for (int i = tid; i < n; i += kSelThreads) cache[i] = __ldcg(score + i);
  auto get = [&](int i) { return cached ? cache[i] : __ldcg(score + i); };
  unsigned key = 0, mask = 0;
  int left = k;  // of the scores that share the key's digits so far, how many are selected
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i0 = warp * 32; i0 < n; i0 += kSelThreads) {
      const int i = i0 + lane;
      const unsigned x = i < n ? get(i) : 0;
      const bool in = i < n && (x & mask) == key;
      const unsigned digit = in ? (x >> shift) & 255 : 256;
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], static_cast<unsigned>(__popc(same)));
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
    mask |= 255u << shift;
    if (s_all) break;
  }
  // scores above the key are all taken, of those equal to it the first `left`: a run of pages per
  // thread, one prefix sum over (above, equal)
  const int run = (n + kSelThreads - 1) / kSelThreads, i0 = min(n, tid * run), i1 = min(n, i0 + run);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) {
    const unsigned x = get(i) & mask;
    mine += x > key ? 1ll << 32 : (x == key ? 1 : 0);
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
    const unsigned x = get(i) & mask;
    if (x > key) {
      sel[above + min(equal, left)] = i;
      ++above;
    } else if (x == key) {
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
  // CTAs of a cluster: about two waves over the batch, at least 64 pages each
  while (a.cl < 8 && 2 * a.cl * units <= 2 * num_sms && 64 * 2 * a.cl <= c.max_pages) a.cl *= 2;
  const int kept = c.max_pages < pg::kSelCache ? c.max_pages : pg::kSelCache;
  const int smem = G * (c.d + 4) + 4 * kept;
  static_assert(32 * (512 + 4) + 4 * pg::kSelCache <= 64 * 1024, "shared memory of the selection");
  cudaError_t e = pg::allow_smem<pg::k_page_select, 64 * 1024>();
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
