// Attention of a chunk of new tokens over a paged key cache on tensor cores (bf16, head_dim 128, 256
// or 512, pages of at least 8 tokens): the formula of mtp_chunk_att.cu.
//
// Both products run as tcgen05.mma with the keys as the 128-row operand, straight from the TMA tile
// (64 rows at d = 512, whose tile of 128 keys would fill the ring), and N query rows as the N side:
//   scores  S^T [KT keys][N] = K_tile [KT][d] Q^T,          A = K_tile, K-major, B = Q, K-major
//   sums    O^T [d][N]      += V_tile^T [d][KT] P^T,        A = V_tile, MN-major (the same bytes when
//                                                            V = K), B = P, MN-major
// so that a head of 512 dims has its sums of 64 rows in 256 columns of tensor memory, where the rows
// as the 128-row operand would need all 512 and leave none for scores; and few rows (a draft block's
// tokens) cost few columns. A row is a (token, query head of the KV head); a tile takes a power of
// two of tokens.
//
// The sums stay in tensor memory over a unit's key tiles. A row's softmax reference is a maximum that
// moves only when a score exceeds it by 2^8, so they are rarely rescaled (a published variant of the
// softmax in one pass). (The tensor-memory adder
// truncates: over 32768 keys, 2048 additions, that is some 10^-4 of a sum, beside the 2^-9 of the
// output's own rounding and that of the probabilities, which enter as bf16; their sum is fp32.)
//
// One CTA per SM. Four warpgroups (two at N = 32) take the softmax of a quarter of the columns each, a
// thread per key: with two, of twice the columns, a tile of 128 x 128 scores took 5000 cycles, since
// two warps per scheduler do not cover for the latencies of tensor memory, barriers and exponentials.
// Of four more warps one finds the units of this CTA's share (a ring of their descriptions) and the
// tiles' pages, one loads the tiles (slots of [KT keys][128 dims]), one loads queries, and one thread
// of the last issues the products (whichever of the next scores and the next sums is ready; scores are
// double-buffered). The key tiles of all units are numbered through and dealt evenly over the CTAs
// (mtp_chunk.cuh); a unit that crosses CTAs leaves unnormalised sums and (max, exp-sum) per part,
// which k_chunk_tc_join adds in CTA order.
//
// Values that are not finite in keys that only some rows of a unit attend, or none, are zeroed before
// the sums (0 * NaN would not vanish), and the attending rows get NaN.
//
// Waits are bounded; a CTA that gives up writes NaN. The softmax warps meet at hardware barriers, which
// have no bound, so they all take the same units and agree on when references move, whatever waits
// have run out: then every one reaches each of the barriers.
//
// What bounds it, and what it measured (with the join):
//   d = 512, two slices of 2048 tokens of 8 heads over 21800 keys on average: 1.96 ms, 710 Tflop/s, the
//   tensor pipe 46 % active. A tile of 64 KB stays in the ring from its load to its sums, 5000 cycles (load 1700,
//   scores 900, softmax 1650, sums 600), and the ring holds 2.25 of them beside 64 rows' queries: 2800
//   cycles a tile. The products themselves (N = 64) would take 1500.
//   d = 128 with a V, 8 ragged prompts to 4096 of 8 heads on 2: 181 us; d = 256, four slices in a window
//   of 512: 77 us. 128 rows' softmax takes 3000 to 3600 cycles a tile, the products 1000 to 1500. It is a
//   chain without a single bound: of 190 and 81 us (before columns without a row were kept out of the
//   agreement) the two kept 185 and 79 without the exponentials, 171 and 73 without the scores' load, 174
//   and 71 without the agreement, 175 and 66 with an eighth of the products; half of the warps starting a
//   unit half a tile later changed nothing.
//   Few rows (8 x 7 tokens of 4 heads over ragged long contexts, d = 512): 46.8 us for 135 MB, 20 at the
//   copy rate, of which 38 before the join; 7 us pass before the first scores. (With the tiles prefetched
//   into the L2 as their pages are found 54, when it was 51.5 without.)
#include <cstring>

#include "mtp_chunk.cuh"
#include "mtp_common.cuh"
#include "mtp_f32x2.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"
#include "mtp_paged_mma.cuh"
#include "mtp_phases.cuh"

namespace mtp {
namespace pgc {

using namespace pgt;
using pg::Cache;
using pg::ChunkArgs;
using pg::kSpin;
using pg::Tiles;

constexpr int kAhead = 4;       // tiles that the find warp runs ahead of the load warp
constexpr int kInfo = 12;       // tiles whose pages are kept: kAhead and those between load and softmax
constexpr int kSegs = 4;        // units whose descriptions are kept
// What beginning a unit costs, in key tiles: 8 ragged prompts of d = 128 take 223 us with 2, 181 with 4, 182
// with 6; four slices in a window of 512 73, 77 and 77 us; long contexts are indifferent.
constexpr int kExtra = 4;

struct Args {
  ChunkArgs a;
  int rshift;   // log2 of the keys per TMA box (min(P, keys per tile))
  int grid;
  int ts;       // log2 of the tokens of a tile
  int hgs;      // groups of N query heads per KV head (1 unless it has more than N)
  int qbytes;   // of a box of queries: 64 dims x min(N, heads per KV head) x 2^ts tokens
  int* meta;    // [grid][8]: last CTA (-1: none), first token, tokens, first head, heads of the unit a CTA starts and does not end
};

template <int D, int N_>
struct Lay {
  static constexpr int N = N_;                           // rows
  static constexpr int WG = N == 32 ? 2 : 4, NC = N / WG;  // softmax warpgroups, columns of each
  static constexpr int threads = 128 * (WG + 1);
  static constexpr int NP = D / 128;                     // 128-dim slots per tile and operand
  static constexpr int KT = D == 512 ? 64 : 128;         // keys per tile
  static constexpr int KS = KT == 64 ? 6 : 7;
  static constexpr int box = KT * 128;                   // KT keys x 64 dims
  static constexpr int slot = 2 * box;
  static constexpr int QBY = D * N * 2;                  // 64-dim blocks of [N][128 bytes]
  static constexpr int PBY = KT * 128 * ((N + 63) / 64); // 64-row blocks of [KT][128 bytes]
  static constexpr int PB = D == 256 && N == 128 ? 1 : 2;  // probability buffers
  static constexpr int misc_bytes = 3 * 1024;
  static constexpr int room = 232448 - misc_bytes - QBY - PB * PBY;
  static constexpr int ring = room / slot > 12 ? 12 : room / slot;  // (a tile's slots may wrap)
  static constexpr int q = ring * slot;
  static constexpr int p = q + QBY;
  static constexpr int mref = p + PB * PBY;              // [N] minus the rows' references
  static constexpr int top = mref + N * 4;               // [N] a tile's maxima, as ordered integers
  static constexpr int fac = top + N * 4;                // [N] factors of the sums under a new reference
  static constexpr int segs = fac + N * 4;               // [kSegs][12] units (Seg below)
  static constexpr int info = segs + kSegs * 48;         // [kInfo][16] physical pages of a tile's boxes
  static constexpr int holes = info + kInfo * 64;        // [kInfo] whether a tile lacks a page
  static constexpr int bad = holes + kInfo * 4;          // per warpgroup [4]: rows that attend values that are not finite
  static constexpr int over = bad + WG * 16;             // per warpgroup [2]: a score of a tile of this parity exceeds its reference by 2^8
  static constexpr int bars = over + WG * 8;
  static constexpr int nbars = 2 * ring + 2 * 4 + 3 + 2 * kSegs + kInfo + WG;
  static constexpr int misc = bars + nbars * 8;          // tensor-memory address, dead word, tiles begun, units
  static constexpr int total = misc + 16;
  static constexpr int want = (NP + 2) * N;              // tensor-memory columns: sums, two of scores
  static constexpr int cols = want <= 128 ? 128 : want <= 256 ? 256 : 512;
};

// A part of a unit (a tile of rows of one KV head, and group of its heads, of one sequence) as the
// warps of a CTA take it.
struct Seg {
  int tiles;           // key tiles
  int k0;              // the first one
  int kvh;
  int tok0, nt, pos0;  // first token of the rows in q and out, tokens, position of the first
  int h0, heads;       // first query head, heads
  int lo, hi;          // keys that a row of the unit attends
  int whole;           // the whole unit is here
  int part;            // else: its place among the parts
};

__device__ __forceinline__ unsigned pack2(float lo, float hi) {
  unsigned r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void ld16(unsigned t, float* v) {
  unsigned* r = reinterpret_cast<unsigned*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}
__device__ __forceinline__ void ld32(unsigned t, float* v) {
  unsigned* r = reinterpret_cast<unsigned*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(t));
}
__device__ __forceinline__ void st16(unsigned t, const float* v) {
  const unsigned* r = reinterpret_cast<const unsigned*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// fp32 values as integers of the same order (NaN as the lowest value), and back.
__device__ __forceinline__ int ordered(float v) {
  const int i = __float_as_int(fmaxf(v, -INFINITY));
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
constexpr int kLowest = static_cast<int>(0xff800000u ^ 0x7fffffffu);  // ordered(-inf)

// The maxima of N <= 32 values over the warp: lane i ends with that of value i * N / 32 in v[0] (O: 16).
template <int N, int O>
__device__ __forceinline__ void max_scatter(float* v, int lane) {
  if constexpr (O > 0) {
    if constexpr (N > 1) {
      constexpr int h = N / 2;
      const bool up = (lane & O) != 0;
#pragma unroll
      for (int i = 0; i < h; ++i) v[i] = fmaxf(up ? v[i + h] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + h], O));
      max_scatter<h, O / 2>(v, lane);
    } else {
      v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], O));
      max_scatter<1, O / 2>(v, lane);
    }
  }
}

// Bounded wait; false when this CTA has given up (the word `dead`) or gives up here. (Inlined: a call
// would keep the softmax from its registers.)
__device__ __forceinline__ bool wait_in(unsigned bar, unsigned parity, volatile int* dead, long long limit) {
  if (test_wait(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!try_wait(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > limit) {
      *dead = 1;
      return false;
    }
  }
  return true;
}

// A wait for warps that arrive in any case, since all that they wait for is bounded: the word `dead`
// does not cut it short, so that whoever waits returns behind the same arrivals.
__device__ __forceinline__ void wait_sure(unsigned bar, unsigned parity) {
  if (test_wait(bar, parity)) return;
  const long long t0 = clock64();
#pragma unroll 1
  while (!try_wait(bar, parity) && clock64() - t0 < 4 * kSpin) {
  }
}

__device__ __forceinline__ Tiles tiles_of(const Args& g, int ks, int b, int& s0) {
  Tiles t;
  pg::chunk_range(g.a, b, s0, t.n, t.first, t.L);
  t.window = g.a.window;
  t.ts = g.ts;
  t.ks = ks;
  t.extra = kExtra;
  return t;
}

// Walks the parts of units of a CTA's share: costs [r, r1).
template <int KS>
struct Walk {
  long long r, r1, per;
  int b, sub, tile, off;  // the unit at r, and how far into it r is
  Tiles t;
  int s0;

  __device__ __forceinline__ void locate(const Args& g, int subs) {
    const int lane = threadIdx.x & 31, each = (g.a.B + 31) >> 5, b0 = min(g.a.B, lane * each), b1 = min(g.a.B, b0 + each);
    long long mine = 0;
    Tiles x;  // of the lane's last sequence: its only one in small batches
    int x0 = 0;
#pragma unroll 1
    for (int i = b0; i < b1; ++i) {
      x = tiles_of(g, KS, i, x0);
      mine += x.cost(x.count());
    }
    mine *= subs;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    per = total < (1 << 30) ? static_cast<unsigned>(total + g.grid - 1) / static_cast<unsigned>(g.grid) : (total + g.grid - 1) / g.grid;
    r = min(total, blockIdx.x * per);
    r1 = min(total, r + per);
    b = sub = tile = off = 0;
    if (r >= r1) return;
    const int f = __ffs(__ballot_sync(0xffffffffu, incl > r)) - 1;
    if (lane == f) {
      long long at = r - (incl - mine), c;
#pragma unroll 1
      for (b = b0;; ++b) {
        t = x;
        if (each > 1) t = tiles_of(g, KS, b, x0);
        c = each > 1 ? t.cost(t.count()) : subs > 1 ? mine / subs : mine;
        if (at < c * subs) break;
        at -= c * subs;
      }
      sub = subs > 1 ? static_cast<int>(at / c) : 0;
      at -= sub * c;
      int lo = 0, hi = t.count() - 1;  // the last tile that begins at or before `at`
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.cost(mid) <= at) lo = mid; else hi = mid - 1;
      }
      tile = lo;
      off = static_cast<int>(at - t.cost(lo));
    }
    b = __shfl_sync(0xffffffffu, b, f);
    sub = __shfl_sync(0xffffffffu, sub, f);
    tile = __shfl_sync(0xffffffffu, tile, f);
    off = __shfl_sync(0xffffffffu, off, f);
    t.window = g.a.window;  // (x of a lane without a sequence holds nothing)
    t.ts = g.ts;
    t.ks = KS;
    t.extra = kExtra;
    t.n = __shfl_sync(0xffffffffu, t.n, f);
    t.first = __shfl_sync(0xffffffffu, t.first, f);
    t.L = __shfl_sync(0xffffffffu, t.L, f);
    s0 = __shfl_sync(0xffffffffu, x0, f);
    if (each > 1) t = tiles_of(g, KS, b, s0);
  }
  struct Part {
    int b, sub, tile;  // sub: KV head * groups + group
    int k, a, e;       // the unit's key tiles, those of this part [a, e)
    bool begins;       // the unit's first key tile is here (or it has none)
    long long last;    // the unit's last cost
  };
  // The next part of a unit. Units without a key tile come with k = 0.
  __device__ __forceinline__ bool next(const Args& g, int subs, Part& s) {
#pragma unroll 1
    while (r < r1) {
      const int nt = t.count();
      if (tile >= nt) {
        tile = 0;
        if (nt == 0 || ++sub >= subs) {
          sub = 0;
          ++b;
          t = tiles_of(g, KS, b, s0);
        }
        continue;
      }
      const int k = t.tiles(tile), c = k + kExtra;
      const int to = static_cast<int>(min(static_cast<long long>(c), off + (r1 - r)));
      s.b = b;
      s.sub = sub;
      s.tile = tile;
      s.k = k;
      s.a = max(off - kExtra, 0);
      s.e = max(to - kExtra, 0);
      s.begins = k > 0 ? s.a == 0 : off == 0;
      s.last = r - off + c - 1;
      r += to - off;
      off = to;
      if (off >= c) {
        off = 0;
        ++tile;
      }
      if (s.e > s.a || (k == 0 && s.begins)) return true;
    }
    return false;
  }
};

template <int D, int N>
__global__ void __launch_bounds__(Lay<D, N>::threads, 1)
    k_chunk_tc(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
               const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ Args g) {
  using LY = Lay<D, N>;
  constexpr int NP = LY::NP, KT = LY::KT, kRing = LY::ring, NC = LY::NC, PB = LY::PB, WG = LY::WG;
  extern __shared__ __align__(1024) char sm[];  // (swizzled tiles begin at multiples of 1024)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const unsigned base = sa(sm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // barriers: loaded slots, free slots; per score buffer: scores done, scores read; per parity of a
  // tile: probabilities written, sums done; queries loaded, queries used, drained; per place of a
  // unit: its sums are read, it is found; pages of a tile found; per warpgroup: a tile's maxima compared
  const unsigned full0 = base + LY::bars, empty0 = full0 + 8 * kRing, sfull0 = empty0 + 8 * kRing, sfree0 = sfull0 + 16,
                 pfull0 = sfree0 + 16, odone0 = pfull0 + 16, qfull = odone0 + 16, qused = qfull + 8, drain = qused + 8,
                 ofree0 = drain + 8, seg0 = ofree0 + 8 * kSegs, ifull0 = seg0 + 8 * kSegs, agree0 = ifull0 + 8 * kInfo;
  int* info = reinterpret_cast<int*>(sm + LY::info);
  int* holes = reinterpret_cast<int*>(sm + LY::holes);
  Seg* segs = reinterpret_cast<Seg*>(sm + LY::segs);
  int* misc = reinterpret_cast<int*>(sm + LY::misc);  // 0: tensor memory, 1: dead, 2: begun
  // begun: tiles that the load warp has begun; units: how many units this CTA has, once all are found
  volatile int *dead = misc + 1, *begun = misc + 2, *units = misc + 3;
  const ChunkArgs& a = g.a;
  const Cache& c = a.c;
  const bool own_v = c.v != nullptr;
  const int PT = own_v ? 2 * NP : NP;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull0 + 8 * i, 1);
      mbar_init(sfree0 + 8 * i, 4 * WG);
      mbar_init(pfull0 + 8 * i, 4 * WG);
      mbar_init(odone0 + 8 * i, 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qused, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(ofree0 + 8 * i, 4 * WG);
      mbar_init(seg0 + 8 * i, 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(ifull0 + 8 * i, 1);
    for (int i = 0; i < WG; ++i) mbar_init(agree0 + 8 * i, 4);
    for (int i = 0; i < 2 * WG; ++i) reinterpret_cast<int*>(sm + LY::over)[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    misc[1] = (base & 1023u) != 0;  // (every wait then gives up)
    misc[2] = 0;
    misc[3] = INT_MAX;
  }
  for (int i = tid; i < N; i += LY::threads) reinterpret_cast<int*>(sm + LY::top)[i] = kLowest;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(misc)), "r"(LY::cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = *reinterpret_cast<volatile unsigned*>(misc);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // unit i of this CTA, once it is found; false behind the last
  auto get_seg = [&](int i, Seg& s) {
    if (!wait_in(seg0 + 8 * (i % kSegs), (i / kSegs) & 1, dead, a.spin)) return false;
    s = segs[i % kSegs];
    return i < *units;
  };

  if (warp == 4 * WG + 2) {
    // ---------------- finds the units, and their tiles' pages up to kAhead tiles before they are loaded
    // (a lane per box, several tiles at once)
    const int G = a.nh / c.nkv, subs = c.nkv * g.hgs;
    const int rs = g.rshift, ngs = LY::KS - rs, ng = 1 << ngs, nb = min(32 >> ngs, kAhead);
    Walk<LY::KS> w;
    w.locate(g, subs);
    int* meta = g.meta + 8 * blockIdx.x;
    if (lane == 0) meta[0] = -1;
    int tt = 0, ns = 0, slot = 0;
    bool ok = true;
    typename Walk<LY::KS>::Part u;
    auto put_seg = [&](const Seg& s) {  // its place is free once the unit kSegs before is answered
      if (ns >= kSegs) ok = __all_sync(0xffffffffu, wait_in(ofree0 + 8 * (ns % kSegs), (ns / kSegs - 1) & 1, dead, a.spin));
      if (!ok) return;
      if (lane == 0) {
        segs[ns % kSegs] = s;
        mbar_arrive(seg0 + 8 * (ns % kSegs));
      }
      __syncwarp();
      ++ns;
    };
    Seg s;
    while (ok && w.next(g, subs, u)) {
      const int hg = u.sub % g.hgs;
      s.kvh = u.sub / g.hgs;
      s.heads = min(N, G - hg * N);
      s.h0 = s.kvh * G + hg * N;
      s.tok0 = w.s0 + (u.tile << g.ts);
      s.nt = min(1 << g.ts, w.t.n - (u.tile << g.ts));
      s.pos0 = static_cast<int>(w.t.pos(u.tile));
      s.lo = w.t.begin(u.tile);
      s.hi = w.t.end(u.tile);
      s.k0 = (s.lo >> LY::KS) + u.a;
      s.tiles = u.e - u.a;
      s.whole = u.a == 0 && u.e == u.k;
      s.part = 2 * blockIdx.x + (u.begins ? 1 : 0);
      if (!u.k) {  // nothing to attend
#pragma unroll 1
        for (int i = lane; i < s.nt * s.heads * (D / 8); i += 32) {
          const int r = i / (D / 8);
          const long long row = static_cast<long long>(s.tok0 + r / s.heads) * a.nh + s.h0 + r % s.heads;
          reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
          if (a.lse && i % (D / 8) == 0) a.lse[row] = -INFINITY;
        }
        continue;
      }
      if (!s.whole && u.begins && lane == 0) {
        meta[0] = static_cast<int>(u.last / w.per);
        meta[1] = s.tok0;
        meta[2] = s.nt;
        meta[3] = s.h0;
        meta[4] = s.heads;
      }
      put_seg(s);
      if (u.b == a.skip) ok = false;  // testing: the other warps wait for these tiles until they give up
#pragma unroll 1
      for (int k = 0; k < s.tiles && ok; k += nb) {
        int page = -1;
        const int pos = ((s.k0 + k) << LY::KS) + (lane << rs);  // the tiles' boxes follow one another
        if (lane < nb * ng && pos < s.hi) page = pg::phys_page(c, u.b, pos >> c.pshift);
#pragma unroll 1
        for (int j = 0; j < nb && k + j < s.tiles; ++j, ++tt) {
          // the load warp has begun tile tt - kAhead, so tile tt - kInfo is done with
          if (tt >= kAhead) {
            const long long t0 = clock64();
            while (*begun < tt - kAhead + 1 && ok) {
              if (*dead || clock64() - t0 > a.spin) {
                *dead = 1;
                ok = false;
              }
              __nanosleep(200);  // (issue slots are the softmax's)
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          const unsigned none = __ballot_sync(0xffffffffu, lane >> ngs == j && page < 0);
          if (lane >> ngs == j) info[slot * 16 + (lane & (ng - 1))] = page;
          if (lane == 0) holes[slot] = none != 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(ifull0 + 8 * slot);
          if (++slot == kInfo) slot = 0;
        }
      }
    }
    if (lane == 0) {  // (in any case: the softmax waits for it)
      *units = ns;
      mbar_arrive(seg0 + 8 * (ns % kSegs));
    }
    __syncwarp();
  } else if (warp == 4 * WG) {
    // ---------------- loads. The whole warp walks, with everything that a copy takes in uniform
    // registers; one elected thread issues (a tile of 64 KB took 1800 cycles to issue from one thread's
    // own registers, as long as its keys take from memory).
    const int rs = g.rshift, R = 1 << rs, ng = KT >> rs, P = 1 << c.pshift;
    int pc = 0, slot = 0, tt = 0, is = 0;  // slots so far, the next slot and the ring's phase there; tiles, place of their pages
    unsigned phase = 0, iphase = 0;
    bool ok = true;
    Seg s;
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
#pragma unroll 1
    for (int i = 0; ok && all(get_seg(i, s)); ++i) {
      const int tiles = __shfl_sync(0xffffffffu, s.tiles, 0), kvh = __shfl_sync(0xffffffffu, s.kvh, 0), k0 = __shfl_sync(0xffffffffu, s.k0, 0);
#pragma unroll 1
      for (int k = 0; k < tiles; ++k, ++tt) {
        ok = all(wait_in(ifull0 + 8 * is, iphase, dead, a.spin));
        if (!ok) break;
        const int mine = info[is * 16 + (lane & 15)];  // -1: zeros
        const int off0 = ((k0 + k) << LY::KS) & (P - 1);  // 0 unless a page is longer than a tile
#pragma unroll
        for (int j = 0; j < 2 * NP; ++j) {
          if (j >= PT) break;
          const unsigned bar = full0 + 8 * slot;
          if (pc >= kRing) ok = all(wait_in(empty0 + 8 * slot, phase ^ 1, dead, a.spin));
          if (!ok) break;
          if (j == 0 && lane == 0) *begun = tt + 1;
          const unsigned dst = base + slot * LY::slot;
          if (elect()) mbar_expect_tx(bar, LY::slot);
          __syncwarp();
#pragma unroll 1
          for (int r = 0; r < ng; ++r) {
            const int page = __shfl_sync(0xffffffffu, mine, r);
            if (elect()) {
              tma_4d(dst + r * R * 128, j < NP ? &mapK : &mapV, (j < NP ? j : j - NP) * 128, off0, kvh, page, bar);
              tma_4d(dst + r * R * 128 + LY::box, j < NP ? &mapK : &mapV, (j < NP ? j : j - NP) * 128 + 64, off0, kvh, page, bar);
            }
          }
          ++pc;
          if (++slot == kRing) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (++is == kInfo) {
          is = 0;
          iphase ^= 1;
        }
      }
    }
    // no copy may be in flight when the CTA ends
#pragma unroll 1
    for (int i = max(0, pc - kRing); i < pc; ++i) {
      const long long t0 = clock64();
      while (!all(try_wait(full0 + 8 * (i % kRing), (i / kRing) & 1)) && all(clock64() - t0 < kSpin)) {
      }
    }
    __syncwarp();
  } else if (warp == 4 * WG + 3) {
    // ---------------- queries: boxes of 64 dims x the heads x the tokens (rows behind a unit's hold
    // those of other tokens or zeros, for columns that nothing reads)
    if (elect()) {
      Seg s;
      int n = 0;
#pragma unroll 1
      for (; get_seg(n, s); ++n) {
        if (n && !wait_in(qused, (n - 1) & 1, dead, a.spin)) break;
        mbar_expect_tx(qfull, g.qbytes * (D / 64));
#pragma unroll 1
        for (int j = 0; j < D / 64; ++j) tma_4d(base + LY::q + j * (N * 128), &mapQ, 64 * j, s.h0, s.tok0, 0, qfull);
      }
      const long long t0 = clock64();
      while (n && !try_wait(qfull, (n - 1) & 1) && clock64() - t0 < kSpin) {
      }
    }
    __syncwarp();
  } else if (warp == 4 * WG + 1) {
    // ---------------- MMA issue: the next sums or the next scores, whichever are ready. The whole warp
    // walks, on conditions that are votes, so that addresses and descriptors are uniform registers; one
    // elected thread (always the same) issues.
    // fp32 += bf16 x bf16, N columns; scores: M = KT; sums: M = 128, A and B MN-major
    constexpr unsigned id = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<unsigned>(N >> 3) << 17);
    constexpr unsigned idS = id | (static_cast<unsigned>(KT >> 4) << 24), idO = id | (1u << 15) | (1u << 16) | (8u << 24);
    const unsigned tO = tmem, tS = tmem + NP * N;
    const unsigned kd = desc_lo(base, 16), vd = desc_lo(base, LY::box), qd = desc_lo(base + LY::q, 16),
                   pd = desc_lo(base + LY::p, KT * 128);
    auto wrap = [](int slot) { return slot >= kRing ? slot - kRing : slot; };
    auto done = [](unsigned bar, unsigned parity) { return __all_sync(0xffffffffu, test_wait(bar, parity)) != 0; };
    // tiles whose scores / sums are issued; tiles left of the scores' unit; units begun by either; ring
    // places
    int tq = 0, tp = 0, left = 0, nseg = 0, pseg = 0, sq = 0, sp = own_v ? NP : 0;
    unsigned fq = 0, fp = 0, starts = 0;  // starts bit i: tile tp + i is its unit's first
    int got = 0;  // of the next scores' conditions (queries, buffer, slots), how many hold: each is polled until it does
    bool more = true, fresh = false;
    long long t0 = clock64();
#pragma unroll 1
    while (more || tp < tq) {
      bool did = false;
      if (more && left == 0 && done(seg0 + 8 * (nseg % kSegs), (nseg / kSegs) & 1)) {
        more = __shfl_sync(0xffffffffu, nseg < *units ? 1 : 0, 0) != 0;
        left = more ? __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&segs[nseg % kSegs].tiles), 0) : 0;
        ++nseg;
        fresh = true;
        did = true;
      }
      if (tp < tq) {
        const bool first = starts & 1;
        bool ready = done(pfull0 + 8 * (tp & 1), (tp >> 1) & 1) &&
                     (!first || pseg == 0 || done(ofree0 + 8 * ((pseg - 1) % kSegs), ((pseg - 1) / kSegs) & 1));
        if (own_v)
          for (int i = 0; i < NP; ++i) ready = ready && done(full0 + 8 * wrap(sp + i), fp ^ (sp + i >= kRing));
        if (ready) {
          if (elect()) {
            fence_after();
            const unsigned p0 = pd + (PB == 1 ? 0 : (tp & 1) * (LY::PBY >> 4));
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const unsigned v0 = vd + wrap(sp + i) * (LY::slot >> 4);
#pragma unroll
              for (int x = 0; x < KT / 16; ++x) mma(tO + i * N, v0 + (x * 2048 >> 4), p0 + (x * 2048 >> 4), idO, x > 0 || !first);
              commit(empty0 + 8 * wrap(sp + i));
            }
            commit(odone0 + 8 * (tp & 1));
          }
          __syncwarp();
          if (first) ++pseg;
          starts >>= 1;
          ++tp;
          if ((sp += PT) >= kRing) {
            sp -= kRing;
            fp ^= 1;
          }
          did = true;
        }
      }
      if (left > 0 && tq < tp + 2) {
        if (got == 0 && (!fresh || done(qfull, (nseg - 1) & 1))) got = 1;
        if (got == 1 && (tq < 2 || done(sfree0 + 8 * (tq & 1), ((tq >> 1) - 1) & 1))) got = 2;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (got == 2 + i && done(full0 + 8 * wrap(sq + i), fq ^ (sq + i >= kRing))) got = 3 + i;
        if (got == 2 + NP) {
          got = 0;
          if (elect()) {
            fence_after();
            const unsigned d = tS + (tq & 1) * N;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const unsigned k0 = kd + wrap(sq + i) * (LY::slot >> 4);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mma(d, k0 + (((x >> 2) * LY::box + (x & 3) * 32) >> 4),
                    qd + (((2 * i + (x >> 2)) * (N * 128) + (x & 3) * 32) >> 4), idS, i > 0 || x > 0);
              if (own_v) commit(empty0 + 8 * wrap(sq + i));
            }
            commit(sfull0 + 8 * (tq & 1));
            if (left == 1) commit(qused);
          }
          __syncwarp();
          starts = (starts & ~(1u << (tq - tp))) | (static_cast<unsigned>(fresh) << (tq - tp));
          fresh = false;
          ++tq;
          --left;
          if ((sq += PT) >= kRing) {
            sq -= kRing;
            fq ^= 1;
          }
          did = true;
        }
      }
      if (did) {
        t0 = clock64();
      } else if (__any_sync(0xffffffffu, *dead || clock64() - t0 > a.spin)) {
        *dead = 1;
        break;
      } else if (tq == tp + 2) {
        // scores are ahead as far as they may be: nothing but probabilities can come next, and a wait
        // leaves the softmax its issue slots
        try_wait(pfull0 + 8 * (tp & 1), (tp >> 1) & 1);
      }
    }
    __syncwarp();
    if (elect()) {  // no product may run when the CTA ends, however the others' waits end
      commit(drain);
      t0 = clock64();
      while (!try_wait(drain, 0) && clock64() - t0 < kSpin) {
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax and outputs: a warpgroup per NC columns, a thread per key of a tile, and
    // per dim of each 128-dim block of the sums
    const int wg = warp >> 2, wt = tid & 127, ww = warp & 3, col0 = wg * NC;
    const unsigned tw = tmem + (static_cast<unsigned>(32 * ww) << 16);
    const unsigned tO = tw + col0, tS = tw + NP * N + col0;
    const f2 scale2 = two(a.scale_log2, a.scale_log2);
    float* const negm = reinterpret_cast<float*>(sm + LY::mref) + col0;
    int* const top = reinterpret_cast<int*>(sm + LY::top) + col0;
    float* const fac = reinterpret_cast<float*>(sm + LY::fac) + col0;
    unsigned* const bad = reinterpret_cast<unsigned*>(sm + LY::bad);
    volatile int* const over = reinterpret_cast<int*>(sm + LY::over) + 2 * wg;
    unsigned agreed = 0;  // the phase of the warpgroup's agreement
    // this thread's key of a tile: the accumulator row of its tensor-memory lane (M = 64 fills the
    // lower half of each warp's lanes)
    const int key = KT == 128 ? wt : 16 * ww + lane;
    const bool has = KT == 128 || lane < 16;
    const int rs = g.rshift;
    auto bar_wg = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
    // (under the fixed bound, as the other warps' waits end it sooner: with a.spin prompt slices take 1 % longer)
    auto wait = [&](unsigned bar, unsigned parity) { wait_in(bar, parity, dead, kSpin); };
    auto wait_sums = [&](int t) { wait(odone0 + 8 * (t & 1), (t >> 1) & 1); };
    // unit i, whatever waits have run out; false behind the last (asked by way of its tiles: with the
    // comparison itself the compiler spills twice as much, and prompts with a V take 216 us instead of 190)
    auto take = [&](int i, Seg& s) {
      wait_sure(seg0 + 8 * (i % kSegs), (i / kSegs) & 1);
      s = segs[i % kSegs];
      s.tiles = i < *units ? s.tiles : 0;
      return s.tiles > 0;
    };
    // the bits i of 0..31 with lo <= i < hi
    auto bits = [](int lo, int hi) {
      lo = max(lo, 0);
      hi = min(hi, 32);
      return lo < hi ? 0xffffffffu >> (32 - hi + lo) << lo : 0u;
    };
    int at = 0, is = 0;  // tiles so far; the place of their pages
    Seg s;
#pragma unroll 1
    for (int ns = 0; take(ns, s); ++ns) {
      const int nr = s.nt * s.heads, nrw = __shfl_sync(0xffffffffu, min(max(nr - col0, 0), NC), 0);  // rows; of this warpgroup
      // (columns behind the rows hold scores of anything, which no reference of a row may move for: under a
      // reference of +inf none exceeds it)
      if (wt < NC) negm[wt] = wt < nrw ? INFINITY : -INFINITY;
      if (wt < 4) bad[4 * wg + wt] = 0;
      bar_wg();
      f2 l[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l[i] = two(0.f, 0.f);
      // keys that every row attends: [in_lo, in_hi)
      const int in_lo = max(s.lo, a.window > 0 ? s.pos0 + s.nt - a.window : 0), in_hi = s.pos0 + 1;
#pragma unroll 1
      for (int t = 0; t < s.tiles; ++t, ++at) {
        const int buf = at & 1;
        char* const pbuf = sm + LY::p + (PB == 1 ? 0 : buf * LY::PBY);
        wait(sfull0 + 8 * buf, (at >> 1) & 1);
        __syncwarp();
        fence_after();
        // x: the exponents under the references; a second time where these have moved
        float x[NC], first = 0.f;  // (first: the score with the warpgroup's first row)
        // the rows [cmin, cmax) of this warpgroup attend this thread's key (its pages were found before
        // they were loaded)
        const int pos = ((s.k0 + t) << LY::KS) + key, rel = pos - s.pos0;
        bool valid = true, edge = pos - key < in_lo || pos - key + KT > in_hi || holes[is] != 0;
        int page = 0, cmin = -col0, cmax = nr - col0;
        if (edge) {
          page = has ? info[is * 16 + (key >> rs)] : -1;
          valid = page >= 0 && pos >= s.lo && pos < s.hi;
          if (!valid) cmin = NC;
          else if (rel > 0) cmin += rel * s.heads;
          if (a.window > 0 && a.window < s.nt - rel) cmax = (rel + a.window) * s.heads - col0;
        }
        if (++is == kInfo) is = 0;
        if (nrw) {
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            if constexpr (NC == 32) ld32(tS + buf * N, x);
            else ld16(tS + buf * N, x);
            ld_wait();
            first = x[0];
#pragma unroll
            for (int i = 0; i < NC; i += 4) {
              const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(negm + i);
              split2(fma2(two(x[i], x[i + 1]), scale2, m.x), x[i], x[i + 1]);
              split2(fma2(two(x[i + 2], x[i + 3]), scale2, m.y), x[i + 2], x[i + 3]);
            }
            if (edge) {
              const unsigned on = bits(cmin, cmax);
#pragma unroll
              for (int i = 0; i < NC; ++i) x[i] = on >> i & 1 ? x[i] : -INFINITY;
            }
            if (!pass && t) {
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int i = 0; i < NC; i += 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], fmaxf(x[i + 2 * e], x[i + 2 * e + 1]));
              }
              const bool up = has && fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) > 8.f;
              const bool any = __any_sync(0xffffffffu, up);
              if (lane == 0) {
                if (any) over[buf] = 1;
                mbar_arrive(agree0 + 8 * wg);
              }
            }
            // (while the warps agree that no reference has to move)
#pragma unroll
            for (int i = 0; i < NC; ++i) x[i] = ex2(x[i]);
            if (pass) break;
            if (t) {
              wait_sure(agree0 + 8 * wg, agreed);
              agreed ^= 1;
              if (!over[buf]) break;
            }
            // new references: the maxima so far, 16 rows at a time from the scores once more (a short
            // loop: a unit's first tile meets a cold instruction cache)
            if (t > 0) wait_sums(at - 1);
            __syncwarp();
            fence_after();
#pragma unroll 1
            for (int i0 = 0; i0 < nrw; i0 += 16) {
              float v[16];
              ld16(tS + buf * N + i0, v);
              ld_wait();
              const unsigned on = has ? bits(cmin - i0, cmax - i0) : 0u;
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = on >> i & 1 ? pg::attended(v[i] * a.scale_log2) : -INFINITY;
              max_scatter<16, 16>(v, lane);
              if (!(lane & 1)) atomicMax(top + i0 + lane / 2, ordered(v[0]));
            }
            bar_wg();
            if (wt == 0) over[buf] = 0;
            if (wt < NC) {
              // (each reference by its own row's scores, so that a row's bits do not depend on other rows)
              const float mo = -negm[wt], tm = unordered(top[wt]), mn = tm > mo + 8.f ? tm : mo;
              top[wt] = kLowest;
              if (wt < nrw) {
                fac[wt] = mo == -INFINITY ? 0.f : ex2(mo - mn);
                negm[wt] = -mn;
              } else {
                fac[wt] = 0.f;
              }
            }
            bar_wg();
            if (t > 0) {
#pragma unroll
              for (int i = 0; i < NC; i += 4) {
                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(fac + i);
                l[i / 2] = mul2(l[i / 2], f.x);
                l[i / 2 + 1] = mul2(l[i / 2 + 1], f.y);
              }
#pragma unroll 1
              for (int b = 0; b < NP; ++b)
#pragma unroll 1
                for (int i = 0; i < nrw; i += 16) {
                  float v[16];
                  ld16(tO + b * N + i, v);
                  ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) v[e] *= fac[i + e];
                  st16(tO + b * N + i, v);
                }
              asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree0 + 8 * buf);
        // the buffer's last probabilities are used: with two buffers the scores of this tile were issued
        // behind the sums of the tile before the last
        if (PB == 1 && at > 0) wait_sums(at - 1);
        if (nrw) {
          char* const prow = pbuf + (col0 >> 6) * (KT * 128) + key * 128;
#pragma unroll
          for (int i = 0; i < NC; i += 8) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) l[(i + e) / 2] = add2(l[(i + e) / 2], two(x[i + e], x[i + e + 1]));
            if (has)
              *reinterpret_cast<uint4*>(prow + (((((col0 & 63) + i) >> 3) ^ (key & 7)) << 4)) =
                  make_uint4(pack2(x[i], x[i + 1]), pack2(x[i + 2], x[i + 3]), pack2(x[i + 4], x[i + 5]), pack2(x[i + 6], x[i + 7]));
          }
        }
        // Keys of the tile that no row of the unit attends, and keys that only some do: what is not finite in
        // their values becomes 0, and the rows that attend it get NaN. With V = K a key whose score with
        // the first row is finite is finite itself, and is not looked at.
        if (edge) {
          const int amin = cmin + col0, amax = min(cmax + col0, nr);
          bool look = has && page >= 0 && (!valid || amin > 0 || amax < nr);
          if (!own_v) look = look && wg == 0 && !isfinite(first);
          const unsigned todo = __ballot_sync(0xffffffffu, look);
          if (todo) {
            // the warp's keys, V vectors of 8 dims of each: all dims, or with a V this warpgroup's part
            constexpr int kPart = D / 8 / WG;
            const int V = own_v ? kPart : D / 8, v0 = own_v ? wg * kPart : 0;
            if (own_v)
              for (int i = 0; i < NP; ++i) wait(full0 + 8 * ((at * PT + NP + i) % kRing), ((at * PT + NP + i) / kRing) & 1);
#pragma unroll 2
            for (int it = 0; it < V; ++it) {
              const int src = (it * 32 + lane) / V, e = (it * 32 + lane) % V + v0;
              const int lo = __shfl_sync(0xffffffffu, valid ? amin : -1, src), hi = __shfl_sync(0xffffffffu, amax, src);
              if (!(todo >> src & 1)) continue;
              const int slot = (at * PT + (own_v ? NP : 0) + (e >> 4)) % kRing, row = KT == 128 ? 32 * ww + src : 16 * ww + src;
              uint4* const at16 = reinterpret_cast<uint4*>(sm + slot * LY::slot + ((e >> 3) & 1) * LY::box + row * 128) + (e & 7);
              uint4 v = *at16;
              unsigned* u = reinterpret_cast<unsigned*>(&v);
              bool off = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((u[i] & 0x7f800000u) == 0x7f800000u) off = true, u[i] &= 0xffffu;
                if ((u[i] & 0x7f80u) == 0x7f80u) off = true, u[i] &= 0xffff0000u;
              }
              if (off) {
                *at16 = v;
                if (lo >= 0)
#pragma unroll 1
                  for (int i = lo; i < hi; ++i) atomicOr(bad + 4 * wg + (i >> 5), 1u << (i & 31));
              }
            }
          }
        }
        fence_async();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull0 + 8 * buf);
      }
      // ---- the unit's sums. Every product is done: the probabilities' buffer serves as scratch
      wait_sums(at - 1);
      __syncwarp();
      fence_after();
      float* const red = reinterpret_cast<float*>(sm + LY::p) + wg * 4 * NC;  // [4][NC] parts of the exp-sums
      {
        float v[NC];
#pragma unroll
        for (int e = 0; e < NC; e += 2) split2(has ? l[e / 2] : two(0.f, 0.f), v[e], v[e + 1]);
        reduce_scatter<NC, 16>(v, lane);
        if (lane % (32 / NC) == 0) red[ww * NC + lane / (32 / NC)] = v[0];
      }
      bar_wg();
      const long long part = static_cast<long long>(s.part) * N;
      if (wt < nrw) {
        const int col = col0 + wt;
        float den = (red[wt] + red[NC + wt]) + (red[2 * NC + wt] + red[3 * NC + wt]);
        const float m = -negm[wt];
        unsigned off = 0;
#pragma unroll
        for (int i = 0; i < WG; ++i) off |= bad[4 * i + (col >> 5)];
        if (*dead || (off >> (col & 31) & 1)) den = NAN;
        if (s.whole) {
          den = pg::row_sum(m, den);
          fac[wt] = den == 0.f ? 0.f : 1.f / den;  // 0: nothing attended
          if (a.lse)
            a.lse[static_cast<long long>(s.tok0 + col / s.heads) * a.nh + s.h0 + col % s.heads] =
                den == 0.f ? -INFINITY : (m + log2f(den)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float2*>(a.ws_ml + (part + col) * 2) = make_float2(m, den);
        }
      }
      bar_wg();
      if (s.whole) {
        // by way of shared memory, 128 dims at a time: 16-byte stores of whole rows
        __nv_bfloat16* const rows = reinterpret_cast<__nv_bfloat16*>(sm + LY::p) + col0 * 128;
        const unsigned inv = (65536 + s.heads - 1) / s.heads;  // r / heads = r * inv >> 16 for r, heads <= 128
        __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.out) + (static_cast<long long>(s.tok0) * a.nh + s.h0) * D;
        asm volatile("bar.sync 5, %0;" ::"n"(128 * WG) : "memory");  // (every warpgroup's parts are read)
#pragma unroll 1
        for (int b = 0; b < NP; ++b) {
#pragma unroll
          for (int i = 0; i < NC; i += 16) {
            float v[16], f[16];
            ld16(tO + b * N + i, v);
#pragma unroll
            for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(f + e) = *reinterpret_cast<const float4*>(fac + i + e);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) rows[(i + e) * 128 + wt] = __float2bfloat16_rn(f[e] == 0.f ? 0.f : v[e] * f[e]);
          }
          bar_wg();
#pragma unroll 1
          for (int i = wt; i < nrw * 16; i += 128) {
            const int r = col0 + (i >> 4), tok = static_cast<int>(r * inv >> 16);
            *reinterpret_cast<uint4*>(out + (static_cast<long long>(tok) * a.nh + r - tok * s.heads) * D + b * 128 + (i & 15) * 8) =
                *reinterpret_cast<const uint4*>(rows + (i >> 4) * 128 + (i & 15) * 8);
          }
          bar_wg();
        }
      } else {
        float* acc = a.ws_acc + (part + col0) * D + wt;
#pragma unroll 1
        for (int b = 0; b < NP; ++b, acc += 128) {
#pragma unroll
          for (int i = 0; i < NC; i += 16) {
            float v[16];
            ld16(tO + b * N + i, v);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (i + e < nrw) acc[(i + e) * D] = v[e];
          }
        }
      }
      fence_before();
      // every warpgroup has read the scratch, the marks and the references
      asm volatile("bar.sync 5, %0;" ::"n"(128 * WG) : "memory");
      if (lane == 0) mbar_arrive(ofree0 + 8 * (ns % kSegs));
    }
    fence_before();
  }
  __syncthreads();
  if (*dead) {  // the rows of every unit of this CTA get NaN
    const int G = a.nh / c.nkv;
    Walk<LY::KS> w;
    w.locate(g, c.nkv * g.hgs);
    typename Walk<LY::KS>::Part u;
    while (w.next(g, c.nkv * g.hgs, u)) {
      const int kvh = u.sub / g.hgs, hg = u.sub % g.hgs, heads = min(N, G - hg * N), tok0 = w.s0 + (u.tile << g.ts);
      const bool whole = u.a == 0 && u.e == u.k;
      const int nt = min(1 << g.ts, w.t.n - (u.tile << g.ts));
      for (int r = tid; r < nt * heads; r += LY::threads) {
        const long long row = static_cast<long long>(tok0 + r / heads) * a.nh + kvh * G + hg * N + r % heads;
        if (!whole) {
          float* ml = a.ws_ml + ((2LL * blockIdx.x + (u.begins ? 1 : 0)) * N + r) * 2;
          ml[0] = 0.f;
          ml[1] = NAN;
          continue;
        }
        for (int i = 0; i < D; ++i) static_cast<__nv_bfloat16*>(a.out)[row * D + i] = __float2bfloat16_rn(NAN);
        if (a.lse) a.lse[row] = NAN;
      }
      if (!whole && u.begins && tid == 0) {
        int* meta = g.meta + 8 * blockIdx.x;
        meta[0] = static_cast<int>(u.last / w.per);
        meta[1] = tok0;
        meta[2] = nt;
        meta[3] = kvh * G + hg * N;
        meta[4] = heads;
      }
    }
  }
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(LY::cols) : "memory");
  }
}

// Adds the parts of the unit that CTA blockIdx.x of k_chunk_tc starts and does not end, a row per warp,
// in CTA order: a lane takes every 32nd part's weight and 4 dims of each block of 128.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_chunk_tc_join(const __grid_constant__ Args g, int N) {
  pdl_enter();
  const int4 meta = *reinterpret_cast<const int4*>(g.meta + 8 * blockIdx.x);  // last CTA, first token, tokens, first head
  const int heads = g.meta[8 * blockIdx.x + 4];
  if (meta.x < 0) return;
  const ChunkArgs& a = g.a;
  const int lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), c0 = blockIdx.x, np = meta.x - c0 + 1;
  if (r >= meta.z * heads) return;
  const long long row = (static_cast<long long>(meta.y) + r / heads) * a.nh + meta.w + r % heads;
  // part i: slot 1 of the first CTA, slot 0 of the next ones
  auto part = [&](int i) { return static_cast<size_t>((c0 + i) * 2 + (i == 0 ? 1 : 0)) * N + r; };
  constexpr int PW = (pg::kMaxSms + 31) / 32, V = D / 128;
  float2 ml[PW];
  float M = -INFINITY, den = 0.f, wgt[PW];
#pragma unroll
  for (int j = 0; j < PW; ++j) {
    ml[j] = lane + 32 * j < np ? *reinterpret_cast<const float2*>(a.ws_ml + 2 * part(lane + 32 * j)) : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, ml[j].x);
  }
  M = warp_max(M);
#pragma unroll
  for (int j = 0; j < PW; ++j) {
    wgt[j] = ml[j].x == -INFINITY ? 0.f : exp2f(ml[j].x - M);  // (a part in which the row attends nothing)
    den += ml[j].x == -INFINITY ? ml[j].y : wgt[j] * ml[j].y;
  }
  den = pg::row_sum(M, warp_sum(den));
  float4 x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = make_float4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < PW; ++j) {
    const int most = min(32, np - 32 * j);
#pragma unroll 4
    for (int i = 0; i < most; ++i) {
      const float f = __shfl_sync(0xffffffffu, wgt[j], i);
      const float4* from = reinterpret_cast<const float4*>(a.ws_acc + part(32 * j + i) * D) + lane;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float4 y = from[32 * v];
        x[v].x = fmaf(f, y.x, x[v].x);
        x[v].y = fmaf(f, y.y, x[v].y);
        x[v].z = fmaf(f, y.z, x[v].z);
        x[v].w = fmaf(f, y.w, x[v].w);
      }
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * D;
#pragma unroll
  for (int v = 0; v < V; ++v)
    *reinterpret_cast<uint2*>(out + 128 * v + 4 * lane) = make_uint2(pack2(x[v].x * inv, x[v].y * inv), pack2(x[v].z * inv, x[v].w * inv));
  if (a.lse && lane == 0) a.lse[row] = den == 0.f ? -INFINITY : (M + log2f(den)) * 0.6931471805599453f;
}

template <int D, int N>
int launch(const Args& g, cudaStream_t st) {
  using LY = Lay<D, N>;
  static_assert(LY::total <= 232448, "shared memory of one CTA");
  static_assert(LY::ring >= 2 * LY::NP, "a tile of K and one of V, or two tiles");
  static_assert(LY::want <= 512, "tensor memory columns");
  static_assert(N * 256 <= LY::PB * LY::PBY && sizeof(Seg) == 48, "128 dims of the rows; the places of the units");
  CUtensorMap mk, mv, mq;
  int rc = make_map(&mk, g.a.c, g.a.c.k, 1 << g.rshift);
  if (rc) return rc;
  mv = mk;
  if (g.a.c.v && (rc = make_map(&mv, g.a.c, g.a.c.v, 1 << g.rshift))) return rc;
  const ChunkArgs& a = g.a;
  const unsigned long long dim[4] = {D, static_cast<unsigned long long>(a.nh), static_cast<unsigned long long>(a.T), 1};
  const unsigned long long stride[3] = {2 * D, 2ull * a.q_stride, 2ull * a.q_stride};
  const unsigned box[4] = {64, static_cast<unsigned>(min(N, a.nh / a.c.nkv)), 1u << g.ts, 1};
  if ((rc = encode_map(&mq, a.q, dim, stride, box, "the queries"))) return rc;
  const cudaError_t e = pg::allow_smem<k_chunk_tc<D, N>, LY::total>();
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("chunk attention: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  rc = pg::launch_pdl("chunk attention", k_chunk_tc<D, N>, dim3(g.grid), LY::threads, LY::total, st, mk, mv, mq, g);
  return rc ? rc : pg::launch_pdl("chunk attention join", k_chunk_tc_join<D>, dim3(g.grid, N / kJoinWarps), kJoinWarps * 32, 0, st, g, N);
}

}  // namespace pgc

// Rows of a tile: 64 at d = 512, 128 below, and 32 where the sequences have at most 32 rows each on
// average (8 x 7 tokens of 4 heads at d = 512: 46.8 us, 52.4 with 64 rows; one window of 512 keys at d = 256:
// 12.4 us, 14.8 with 128).
static int chunk_tc_rows(const pg::ChunkArgs& a) {
  if (static_cast<long long>(a.T) * (a.nh / a.c.nkv) <= 32LL * a.B) return 32;
  return a.c.d == 512 ? 64 : 128;
}

long long chunk_tc_workspace(const pg::ChunkArgs& a) {
  return pg::kMaxSms * (32LL + 2LL * chunk_tc_rows(a) * (a.c.d + 2) * 4);
}

int run_chunk_tc(const pg::ChunkArgs& a, void* ws, int num_sms, cudaStream_t st) {
  using namespace pgc;
  Args g;
  memset(&g, 0, sizeof(g));
  g.a = a;
  const int P = 1 << a.c.pshift, G = a.nh / a.c.nkv, N = chunk_tc_rows(a), KT = a.c.d == 512 ? 64 : 128;
  const int rows = P < KT ? P : KT;
  while ((1 << g.rshift) < rows) ++g.rshift;
  while ((2 << g.ts) * G <= N) ++g.ts;
  g.hgs = (G + N - 1) / N;
  g.qbytes = 128 * (G < N ? G : N) << g.ts;
  g.grid = num_sms;
  g.meta = static_cast<int*>(ws);
  g.a.ws_ml = reinterpret_cast<float*>(g.meta + 8 * pg::kMaxSms);
  g.a.ws_acc = g.a.ws_ml + pg::kMaxSms * 2 * N * 2;
  if (a.c.d == 512) return N == 32 ? launch<512, 32>(g, st) : launch<512, 64>(g, st);
  if (a.c.d == 256) return N == 32 ? launch<256, 32>(g, st) : launch<256, 128>(g, st);
  return N == 32 ? launch<128, 32>(g, st) : launch<128, 128>(g, st);
}

}  // namespace mtp
