// Sharing and collecting the pages of a cache: forks of sequences, whose complete pages are shared and
// whose partial page is copied, and the pages that no sequence holds, as the ring of free pages, with
// the held ones moved into the front of the pool where that is asked for. No page carries a count of
// its holders: the block tables say who holds it.
// What bounds them is the chain of dependent reads and launches: 64 samples of a prompt take 6.2 us, 256
// beams 6.7, the collection of a pool of 131072 pages 11.8 (three launches). A compaction is bound by
// its copy: 33 us for 135 MB read and written in pages of 16 KB, 20 at the copy rate.
#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

namespace {

// Rows [0, rows) of page `from` into page `to`, this block's part of `parts`.
__device__ __forceinline__ void copy_rows(const Cache& c, void* x, int from, int to, int rows, int part, int parts) {
  const int size = c.f32 ? 4 : 2, vec = c.d * size / 16;  // 16-byte vectors of a head's row
  char* const src = static_cast<char*>(x) + from * c.sp * size;
  char* const dst = static_cast<char*>(x) + to * c.sp * size;
  const int at = part * blockDim.x + threadIdx.x, step = parts * blockDim.x;
  if (c.st == static_cast<long long>(c.nkv) * c.d && (c.sh == c.d || c.nkv == 1)) {  // token-major: one run
    const int n = rows * c.nkv * vec;
#pragma unroll 4
    for (int i = at; i < n; i += step) reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(src)[i];
    return;
  }
  const int n = rows * c.nkv * vec;
#pragma unroll 2
  for (int i = at; i < n; i += step) {
    const int v = i % vec, r = i / vec, t = r % rows, h = r / rows;
    const long long off = (t * c.st + h * c.sh) * size + 16LL * v;
    *reinterpret_cast<uint4*>(dst + off) = *reinterpret_cast<const uint4*>(src + off);
  }
}

// ---------------------------------------------------------------- forks

constexpr int kForkThreads = 512;
constexpr int kForkMax = 8192;  // forks, and sequences
constexpr int kForkEach = kForkMax / kForkThreads;

struct ForkArgs {
  Cache c;
  int* table;
  const int *src, *dst, *len;
  const int *ring, *state;
  int *len_out, *state_out, *status;
  int B, n, parts;  // parts: blocks of a fork
};

// Every block decides all forks by itself (who is granted is a scan over them) and then carries out
// its own: block b part b % parts of fork b / parts. What bounds it is the chain of reads (forks,
// lengths, the ring's head, a table row, the page), a few microseconds whatever the sizes.
__global__ void __launch_bounds__(kForkThreads) k_page_fork(const __grid_constant__ ForkArgs a) {
  pdl_enter();
  extern __shared__ int sm_fork[];
  int* const owner = sm_fork;       // [B]: the fork that a sequence is the destination of
  int* const grant = owner + a.B;   // [n]: pages taken up to and with this fork, -1: denied
  __shared__ int warp_sum_s[kForkThreads / 32], totals[3];
  const Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = 1 << c.pshift, cap = c.max_pages << c.pshift;
  auto clamped = [&](int b) { return min(max(c.ctx_len[b], 0), cap); };
  for (int i = tid; i < a.B; i += kForkThreads) owner[i] = INT_MAX;
  if (tid < 3) totals[tid] = 0;
  __syncthreads();
  auto range = [&](int x) { return static_cast<unsigned>(x) < static_cast<unsigned>(a.B); };
  for (int i = tid; i < a.n; i += kForkThreads)
    if (range(a.src[i]) && range(a.dst[i])) atomicMin(owner + a.dst[i], i);
  const int head0 = a.state[0], count = min(max(a.state[1], 0), c.n_pages);
  const int head = (head0 % c.n_pages + c.n_pages) % c.n_pages;
  __syncthreads();
  // fork i is good when no earlier one has its destination and no other one its source as destination
  int need[kForkEach], sum = 0;
  const int each = (a.n + kForkThreads - 1) / kForkThreads, i0 = tid * each;
#pragma unroll
  for (int j = 0; j < kForkEach; ++j) {
    need[j] = -1;
    if (j >= each || i0 + j >= a.n) continue;
    const int i = i0 + j, s = a.src[i], d = a.dst[i], len = a.len[i];
    if (range(s) && range(d) && owner[d] == i && (s == d || owner[s] == INT_MAX) && len >= 0 && len <= clamped(s)) {
      need[j] = (len & (P - 1)) != 0;
      sum += need[j];
    }
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum_s[warp] = incl;
  __syncthreads();
  int before = incl - sum;
  for (int w = 0; w < warp; ++w) before += warp_sum_s[w];
  int granted = 0, taken = 0, shared = 0;
#pragma unroll
  for (int j = 0; j < kForkEach; ++j) {
    if (j >= each || i0 + j >= a.n) continue;
    int g = -1;
    if (need[j] >= 0) {
      before += need[j];
      if (before <= count) {
        g = before;
        ++granted;
        taken += need[j];
        shared += a.len[i0 + j] >> c.pshift;
      }
    }
    grant[i0 + j] = g;
  }
  if (blockIdx.x == 0) {
    if (granted) {
      atomicAdd(totals, granted);
      atomicAdd(totals + 1, taken);
      atomicAdd(totals + 2, shared);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = tid; b < a.B; b += kForkThreads) {
      const int i = owner[b];
      a.len_out[b] = i < a.n && grant[i] >= 0 ? a.len[i] : clamped(b);
    }
    if (tid == 0) {
      a.state_out[0] = (head + totals[1]) % c.n_pages;
      a.state_out[1] = count - totals[1];
      a.status[0] = totals[0];
      a.status[1] = totals[1];
      a.status[2] = totals[2];
      a.status[3] = a.n - totals[0];
    }
  }
  for (int w = blockIdx.x; w < a.n * a.parts; w += gridDim.x) {
    const int i = w / a.parts, part = w - i * a.parts;
    if (grant[i] < 0) continue;
    const int s = a.src[i], d = a.dst[i], len = a.len[i], whole = len >> c.pshift, rest = len & (P - 1);
    // a sequence forked onto itself: its partial page's entry is read and then replaced, by one block
    if (s == d && part) continue;
    const int parts = s == d ? 1 : a.parts;
    const long long from = s * c.table_stride, to = d * c.table_stride;
    int fresh = -1, old = -1;
    if (rest) {
      fresh = a.ring[(head + grant[i] - 1) % c.n_pages];
      old = phys_page(c, s, whole);
    }
    if (s != d)
      for (int t = part * kForkThreads + tid; t < whole; t += parts * kForkThreads) a.table[to + t] = a.table[from + t];
    if (rest) {
      __syncthreads();  // (old is read)
      if (part == 0 && tid == 0) a.table[to + whole] = fresh;
      if (old >= 0 && static_cast<unsigned>(fresh) < static_cast<unsigned>(c.n_pages) && old != fresh) {
        copy_rows(c, c.k, old, fresh, rest, part, parts);
        if (c.v) copy_rows(c, c.v, old, fresh, rest, part, parts);
      }
    }
  }
}

// ---------------------------------------------------------------- collection

struct CollectArgs {
  Cache c;
  int* ring;
  int* table_out;           // null: pages stay where they are
  long long out_stride;
  int *state_out, *status;
  unsigned* mark;           // a bit per page: held
  int* before;              // [words]: held pages before a word's
  int* low;                 // free pages in front of `used`, in order
  int* high;                // held pages from there on, in order
  int* none;                // table entries of held positions that are no page
  int B, words;
};

constexpr int kCollectThreads = 256;
constexpr int kMarkEntries = 4 * kCollectThreads;  // table entries of a block

__global__ void __launch_bounds__(kCollectThreads) k_page_clear(const __grid_constant__ CollectArgs a) {
  pdl_enter();
  for (int i = blockIdx.x * kCollectThreads + threadIdx.x; i < a.words; i += gridDim.x * kCollectThreads) a.mark[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.none = 0;
}

__device__ __forceinline__ int held_pages(const Cache& c, int b) {
  const int L = min(max(c.ctx_len[b], 0), c.max_pages << c.pshift);
  return (L + (1 << c.pshift) - 1) >> c.pshift;
}

__global__ void __launch_bounds__(kCollectThreads) k_page_mark(const __grid_constant__ CollectArgs a) {
  pdl_enter();
  const Cache& c = a.c;
  const int per = (c.max_pages + kMarkEntries - 1) / kMarkEntries;
  for (long long w = blockIdx.x; w < static_cast<long long>(a.B) * per; w += gridDim.x) {
    const int b = static_cast<int>(w / per), t0 = static_cast<int>(w - static_cast<long long>(b) * per) * kMarkEntries;
    const int n = held_pages(c, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j * kCollectThreads + threadIdx.x;
      if (t >= n) continue;
      const int page = phys_page(c, b, t);
      if (page < 0) atomicAdd(a.none, 1); else atomicOr(a.mark + (page >> 5), 1u << (page & 31));
    }
  }
}

// The ring (or, for a compaction, the pages that change places and the ring behind them). Every block
// counts the marks before its words for itself: the marks are a bit per page, so reading them all
// costs less than a launch more.
__global__ void __launch_bounds__(1024) k_page_ring(const __grid_constant__ CollectArgs a) {
  pdl_enter();
  __shared__ int part[2][32], s_before, s_used;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.c.n_pages;
  const int per = (a.words + gridDim.x - 1) / gridDim.x, w0 = min(a.words, static_cast<int>(blockIdx.x) * per), w1 = min(a.words, w0 + per);
  int front = 0, all = 0;
#pragma unroll 4
  for (int i = tid; i < a.words; i += 1024) {
    const int x = __popc(a.mark[i]);
    all += x;
    front += i < w0 ? x : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    front += __shfl_xor_sync(0xffffffffu, front, o);
  }
  if (lane == 0) {
    part[0][warp] = front;
    part[1][warp] = all;
  }
  __syncthreads();
  if (tid == 0) {
    int x = 0, y = 0;
    for (int i = 0; i < 32; ++i) {
      x += part[0][i];
      y += part[1][i];
    }
    s_before = x;
    s_used = y;
  }
  __syncthreads();
  const int used = s_used;
  if (blockIdx.x == 0 && tid == 0) {
    a.state_out[0] = 0;
    a.state_out[1] = n - used;
    a.status[0] = used;
    a.status[1] = n - used;
    a.status[3] = *a.none;
    // held pages behind the first `used` ones, counted below where a compaction is asked for
    if (!a.table_out) a.status[2] = 0;
  }
  int before = s_before;
  for (int base = w0; base < w1; base += 1024) {  // 1024 words at a time, a scan over the block
    const int i = base + tid;
    const unsigned m = i < w1 ? a.mark[i] : 0;
    int incl = __popc(m);
    const int own = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) part[0][warp] = incl;
    __syncthreads();
    int at = before + incl - own, total = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at += part[0][w];
      total += part[0][w];
    }
    before += total;
    if (i < w1 && a.table_out) a.before[i] = at;
    // a warp writes its 32 words' pages together, a word at a time
    for (int l = 0; l < 32; ++l) {
      const unsigned word = __shfl_sync(0xffffffffu, m, l);
      const int first = __shfl_sync(0xffffffffu, at, l), wi = base + warp * 32 + l, p = 32 * wi + lane;
      if (wi >= w1 || p >= n) continue;
      const bool held = word >> lane & 1;
      const int held_before = first + __popc(word & ((1u << lane) - 1)), free_before = p - held_before;
      if (!a.table_out) {
        if (!held) a.ring[free_before] = p;
        continue;
      }
      if (p >= used) a.ring[p - used] = p;
      // as many held pages lie behind `used` as free ones in front of it
      if (!held && p < used) a.low[free_before] = p;
      // the h-th held page from the last: its place among those behind `used`, which are counted from the end
      if (held && p >= used) a.high[used - 1 - held_before] = p;
    }
  }
}

// The table under the pages' new numbers, and the pages' contents. Held pages behind the first `used`
// take the free places in front in order; high[] lists the former from the last one back, m of them.
__global__ void __launch_bounds__(kCollectThreads) k_page_move(const __grid_constant__ CollectArgs a) {
  pdl_enter();
  const Cache& c = a.c;
  const int used = a.status[0], uw = used >> 5;
  // held pages in front of `used`; behind it there are m
  const int front = uw < a.words ? a.before[uw] + __popc(a.mark[uw] & ((1u << (used & 31)) - 1)) : used;
  const int m = used - front;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.status[2] = m;
  const int per = (c.max_pages + kMarkEntries - 1) / kMarkEntries;
  for (long long w = blockIdx.x; w < static_cast<long long>(a.B) * per; w += gridDim.x) {
    const int b = static_cast<int>(w / per), t0 = static_cast<int>(w - static_cast<long long>(b) * per) * kMarkEntries;
    const int n = held_pages(c, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j * kCollectThreads + threadIdx.x;
      if (t >= c.max_pages) continue;
      int page = t < n ? phys_page(c, b, t) : -1;
      if (page >= used)
        page = a.low[a.before[page >> 5] + __popc(a.mark[page >> 5] & ((1u << (page & 31)) - 1)) - front];
      a.table_out[b * a.out_stride + t] = page;
    }
  }
  const int quads = c.nkv * c.d / 4;  // of a page's codes
  for (int h = blockIdx.x; h < m; h += gridDim.x) {
    const int from = a.high[m - 1 - h], to = a.low[h];
    copy_rows(c, c.k, from, to, 1 << c.pshift, 0, 1);
    if (c.v) copy_rows(c, c.v, from, to, 1 << c.pshift, 0, 1);
    if (c.codes) {
      for (int i = threadIdx.x; i < quads; i += kCollectThreads)
        reinterpret_cast<int*>(c.codes)[static_cast<long long>(to) * quads + i] = reinterpret_cast<const int*>(c.codes)[static_cast<long long>(from) * quads + i];
      for (int i = threadIdx.x; i < c.nkv; i += kCollectThreads)
        c.scales[static_cast<long long>(to) * c.nkv + i] = c.scales[static_cast<long long>(from) * c.nkv + i];
    }
  }
}

}  // namespace

}  // namespace pg

int run_page_fork(const pg::Cache& c, int B, const int* src, const int* dst, const int* len, int n, const int* ring,
                  const int* state, int* len_out, int* state_out, int* status, int num_sms, cudaStream_t st) {
  using namespace pg;
  ForkArgs a;
  a.c = c;
  a.table = const_cast<int*>(c.table);
  a.src = src;
  a.dst = dst;
  a.len = len;
  a.ring = ring;
  a.state = state;
  a.len_out = len_out;
  a.state_out = state_out;
  a.status = status;
  a.B = B;
  a.n = n;
  // a block for every 16 KB of a page, as long as the blocks are few
  const long long bytes = (static_cast<long long>(c.nkv) * c.d * (c.f32 ? 4 : 2) * (c.v ? 2 : 1)) << c.pshift;
  long long parts = bytes / 16384, most = n > 0 ? 4LL * num_sms / n : 1;
  if (parts > most) parts = most;
  a.parts = parts < 1 ? 1 : static_cast<int>(parts);
  const long long grid = static_cast<long long>(n) * a.parts;
  const cudaError_t e = allow_smem<k_page_fork, 2 * kForkMax * 4>();
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("page fork: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  return launch_pdl("page fork", k_page_fork, dim3(static_cast<unsigned>(grid < 1 ? 1 : grid < 8LL * num_sms ? grid : 8LL * num_sms)),
                    kForkThreads, (B + n) * 4, st, a);
}

long long page_collect_workspace(const pg::Cache& c, bool compact) {
  const long long words = (c.n_pages + 31LL) / 32;
  // marks, counts before them, a page less than half of the pool twice
  return 16 + 4 * words + (compact ? 4 * words + 8 * (c.n_pages / 2 + 1LL) : 0);
}

int run_page_collect(const pg::Cache& c, int B, int* ring, int* table_out, long long out_stride, int* state_out,
                     int* status, void* ws, int num_sms, cudaStream_t st) {
  using namespace pg;
  CollectArgs a;
  a.c = c;
  a.ring = ring;
  a.table_out = table_out;
  a.out_stride = out_stride;
  a.state_out = state_out;
  a.status = status;
  a.B = B;
  a.words = static_cast<int>((c.n_pages + 31LL) / 32);
  a.none = static_cast<int*>(ws);
  a.mark = reinterpret_cast<unsigned*>(a.none + 4);
  a.before = reinterpret_cast<int*>(a.mark + a.words);
  a.low = a.before + a.words;
  a.high = a.low + c.n_pages / 2 + 1;
  auto blocks = [&](long long want, long long most) { return dim3(static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most)); };
  const long long rows = static_cast<long long>(B) * ((c.max_pages + kMarkEntries - 1) / kMarkEntries);
  int rc = launch_pdl("page collection", k_page_clear, blocks((a.words + 1023) / 1024, num_sms), kCollectThreads, 0, st, a);
  if (!rc) rc = launch_pdl("page collection", k_page_mark, blocks(rows, 8LL * num_sms), kCollectThreads, 0, st, a);
  if (!rc) rc = launch_pdl("page collection", k_page_ring, blocks((a.words + 31) / 32, num_sms), 1024, 0, st, a);
  if (!rc && table_out) rc = launch_pdl("page collection", k_page_move, dim3(8 * num_sms), kCollectThreads, 0, st, a);
  return rc;
}

}  // namespace mtp
