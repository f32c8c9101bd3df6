// Selection of the pages a query attends: every page of a sequence is scored by the integer dot
// product of the quantised query with the page's summary (the quantised mean of its keys), and
// the n_select best pages of each KV head are listed in increasing order. The dot product is at
// most 512 * 127 * 127 < 2^24, so it converts to fp32 exactly and a score does not depend on the
// order of its sums: the selected sets are reproducible, ties going to the lower page.
#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;

struct SelArgs {
  Cache c;
  const float* q;
  unsigned* score;  // [B][nkv][max_pages] ordered keys
  int* sel;
  int B, nh, n_select, keep_first, keep_last;
};

// Scores of the pages of one (sequence, KV head): warps over pages, a lane's 16 codes per load.
__global__ void __launch_bounds__(kSelThreads) k_page_score(const __grid_constant__ SelArgs a) {
  pdl_enter();
  const Cache& c = a.c;
  const int d = c.d, G = a.nh / c.nkv, g = blockIdx.x % c.nkv, b = blockIdx.x / c.nkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ __align__(16) int qc[];     // [G][d / 4] packed codes, then [G] steps
  float* qs = reinterpret_cast<float*>(qc + G * (d / 4));
  int lo, L;
  key_range(c, b, 0, lo, L);
  const int P = 1 << c.pshift, n = (L + P - 1) >> c.pshift;
  if (static_cast<int>(blockIdx.y) * kSelWarps >= n || n <= a.n_select) return;
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
    signed char* out = reinterpret_cast<signed char*>(qc + h * (d / 4));
    for (int i = lane; i < d; i += 32)
      out[i] = step > 0.f ? static_cast<signed char>(fminf(fmaxf(rintf(__fdiv_rn(q[i], step)), -127.f), 127.f)) : 0;
  }
  __syncthreads();
  unsigned* score = a.score + (static_cast<size_t>(b) * c.nkv + g) * c.max_pages;
  for (int lp = blockIdx.y * kSelWarps + warp; lp < n; lp += gridDim.y * kSelWarps) {
    const int page = phys_page(c, b, lp);
    float s = -INFINITY;
    if (page >= 0) {
      const int* row = reinterpret_cast<const int*>(c.codes + (static_cast<size_t>(page) * c.nkv + g) * d);
      const float ks = c.scales[static_cast<size_t>(page) * c.nkv + g];
      for (int h = 0; h < G; ++h) {
        int dot = 0;
        for (int i = lane; i < d / 4; i += 32) dot = __dp4a(row[i], qc[h * (d / 4) + i], dot);
        dot = __reduce_add_sync(0xffffffffu, dot);
        s = fmaxf(s, __fmul_rn(__fmul_rn(static_cast<float>(dot), qs[h]), ks));
      }
      if (isnan(ks)) s = INFINITY;  // a page whose keys are not finite is always read
    }
    if (lp < a.keep_first || lp >= n - a.keep_last) s = INFINITY;
    if (lane == 0) score[lp] = ord_f32(s);
  }
}

// The n_select largest of n scores, listed in increasing page order: the threshold key by four
// 8-bit digit passes, then one ordered compaction (equal keys: the lower pages first).
__global__ void __launch_bounds__(kSelThreads) k_page_pick(const __grid_constant__ SelArgs a) {
  pdl_enter();
  const Cache& c = a.c;
  const int g = blockIdx.x % c.nkv, b = blockIdx.x / c.nkv, tid = threadIdx.x, k = a.n_select;
  int lo, L;
  key_range(c, b, 0, lo, L);
  const int P = 1 << c.pshift, n = (L + P - 1) >> c.pshift;
  int* sel = a.sel + static_cast<size_t>(blockIdx.x) * k;
  if (n <= k) {
    for (int i = tid; i < k; i += kSelThreads) sel[i] = i < n ? i : -1;
    return;
  }
  const unsigned* score = a.score + static_cast<size_t>(blockIdx.x) * c.max_pages;
  __shared__ unsigned hist[256], s_key;
  __shared__ int s_left, wsum[2][kSelWarps], s_base[2];
  unsigned key = 0, mask = 0;
  int left = k;  // of the scores that share the key's digits so far, how many are selected
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const unsigned x = score[i];
      if ((x & mask) == key) atomicAdd(&hist[(x >> shift) & 255], 1u);
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
        int j = 0;
        while (before + h[j] < left) before += h[j++];
        s_key = key | (static_cast<unsigned>(255 - 8 * tid - j) << shift);
        s_left = left - before;
      }
    }
    __syncthreads();
    key = s_key;
    left = s_left;
    mask |= 255u << shift;
  }
  // scores above the key are all taken, of those equal to it the first `left`
  if (tid == 0) s_base[0] = s_base[1] = 0;
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const unsigned x = i < n ? score[i] : 0;
    const bool gt = i < n && x > key, eq = i < n && x == key;
    const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      wsum[0][warp] = __popc(mg);
      wsum[1][warp] = __popc(me);
    }
    __syncthreads();
    int bg = s_base[0], be = s_base[1];
    for (int w = 0; w < warp; ++w) {
      bg += wsum[0][w];
      be += wsum[1][w];
    }
    const unsigned below = (1u << lane) - 1;
    bg += __popc(mg & below);
    be += __popc(me & below);
    if (gt) sel[bg + min(be, left)] = i;
    if (eq && be < left) sel[bg + be] = i;
    __syncthreads();
    if (tid == 0)
      for (int w = 0; w < kSelWarps; ++w) {
        s_base[0] += wsum[0][w];
        s_base[1] += wsum[1][w];
      }
    __syncthreads();
  }
}

}  // namespace pg

long long page_select_workspace(const pg::Cache& c, int B) {
  return 4LL * B * c.nkv * c.max_pages;
}

int run_page_select(const pg::Cache& c, const float* q, int B, int nh, int n_select, int keep_first, int keep_last,
                    int* sel, void* ws, int num_sms, cudaStream_t st) {
  const pg::SelArgs a{c, q, static_cast<unsigned*>(ws), sel, B, nh, n_select, keep_first, keep_last};
  const int G = nh / c.nkv;
  int gx = (c.max_pages + pg::kSelWarps - 1) / pg::kSelWarps;
  const int cap = (8 * num_sms + B * c.nkv - 1) / (B * c.nkv);
  if (gx > cap) gx = cap;
  if (c.max_pages > n_select) {
    pg::k_page_score<<<dim3(B * c.nkv, gx), pg::kSelThreads, G * (c.d + 4), st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
      set_error("page score launch: %s", cudaGetErrorString(e));
      return MTP_ERR_CUDA;
    }
  }
  pg::k_page_pick<<<B * c.nkv, pg::kSelThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("page pick launch: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  return MTP_OK;
}

}  // namespace mtp
