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
// moves only when a score exceeds it by 2^8, so they are rarely rescaled. (The tensor-memory adder
// truncates: over 32768 keys, 2048 additions, that is some 10^-4 of a sum, beside the 2^-9 of the
// output's own rounding and that of the probabilities, which enter as bf16; their sum is fp32.)
//
// One CTA per SM: warp 10 finds the tiles' pages through the block table, warp 8 loads them (slots of
// [KT keys][128 dims]), one thread of warp 9 issues the products (whichever of the next scores and the
// next sums is ready; scores are double-buffered), and two warpgroups take the softmax of one half of
// the columns each, a thread per key. The key tiles of all units are numbered through and dealt evenly
// over the CTAs (mtp_chunk.cuh); a unit that crosses CTAs leaves unnormalised sums and (max, exp-sum)
// per part, which k_chunk_tc_join adds in CTA order.
//
// Keys that no row of the unit attends are zero before the sums (0 * NaN would not vanish). Of a key
// that only some rows attend, values that are not finite are zeroed and the attending rows get NaN.
// Waits are bounded; a CTA that gives up writes NaN.
#include <cstring>

#include "mtp_chunk.cuh"
#include "mtp_common.cuh"
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

constexpr int kThreads = 384;   // two warpgroups for the softmax; load, MMA, find and no-work warps
constexpr int kAhead = 4;       // tiles that the find warp runs ahead of the load warp
constexpr int kInfo = 12;       // tiles whose pages are kept: kAhead and those between load and softmax
constexpr int kExtra = 2;       // what beginning a unit costs, in key tiles

struct Args {
  ChunkArgs a;
  int rshift;   // log2 of the keys per TMA box (min(P, keys per tile))
  int grid;
  int tpt;      // tokens of a tile
  int hgs;      // groups of N query heads per KV head (1 unless it has more than N)
  int* meta;    // [grid][4]: sequence, KV head and group, tile, last CTA of the unit a CTA starts and does not end
};

template <int D, int N_>
struct Lay {
  static constexpr int N = N_, NC = N / 2;               // rows; of a warpgroup
  static constexpr int NP = D / 128;                     // 128-dim slots per tile and operand
  static constexpr int KT = D == 512 ? 64 : 128;         // keys per tile
  static constexpr int KS = KT == 64 ? 6 : 7;
  static constexpr int box = KT * 128;                   // KT keys x 64 dims
  static constexpr int slot = 2 * box;
  static constexpr int QBY = D * N * 2;                  // 64-dim blocks of [N][128 bytes]
  static constexpr int PBY = KT * 128 * ((N + 63) / 64); // 64-row blocks of [KT][128 bytes]
  static constexpr int PB = D == 256 && N == 128 ? 1 : 2;  // probability buffers
  // the softmax's scratch, [5][NC] floats per warpgroup: with 128 rows a 64-row block of the
  // probabilities is one warpgroup's alone and serves; fewer rows share a block, but leave room
  static constexpr int scratch_bytes = N == 128 ? 0 : 5 * N * 4;
  static constexpr int misc_bytes = 2048 - 64 + scratch_bytes;
  static constexpr int room = 232448 - 1024 - misc_bytes - QBY - PB * PBY;
  static constexpr int ring0 = room / slot > 16 ? 16 : room / slot;
  static constexpr int ring = ring0 / NP * NP;           // a tile's slots of one operand are neighbours
  static constexpr int q = ring * slot;
  static constexpr int p = q + QBY;
  static constexpr int mref = p + PB * PBY;              // [N] minus the rows' references
  static constexpr int info = mref + N * 4;              // [kInfo][16] physical pages of a tile's boxes
  static constexpr int bad = info + kInfo * 64;          // per warpgroup [4]: rows that attend values that are not finite
  static constexpr int scratch = bad + 32;
  static constexpr int bars = scratch + scratch_bytes;
  static constexpr int nbars = 2 * ring + 2 * 4 + 3 + kInfo;
  static constexpr int misc = bars + nbars * 8;          // tensor-memory address, dead word, tiles begun
  static constexpr int total = misc + 16 + 1024;         // + alignment
  static constexpr int want = (NP + 2) * N;              // tensor-memory columns: sums, two of scores
  static constexpr int cols = want <= 128 ? 128 : want <= 256 ? 256 : 512;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
__device__ __forceinline__ void st16(unsigned t, const float* v) {
  const unsigned* r = reinterpret_cast<const unsigned*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// The largest of the warp's values (NaN left out).
__device__ __forceinline__ float warp_max_redux(float v) {
  int i = __float_as_int(fmaxf(v, -INFINITY));
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(0xffffffffu, i);
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// A unit: a tile of rows of one KV head (and group of its heads) of one sequence.
struct Unit {
  int b, sub, tile;      // sub: KV head * hgs + group
  int s0, nt, pos0;      // first token of the sequence in q; tokens of the tile; position of its first
  int lo, hi;            // its keys
  int k0, n;             // first key tile, number of key tiles
};

__device__ __forceinline__ Tiles tiles_of(const Args& g, int ks, int b, int& s0) {
  Tiles t;
  pg::chunk_range(g.a, b, s0, t.n, t.first, t.L);
  t.window = g.a.window;
  t.tpt = g.tpt;
  t.ks = ks;
  t.extra = kExtra;
  return t;
}

// Walks the segments (parts of units) of a CTA's share: costs [r, r1).
template <int KS>
struct Walk {
  long long r, r1, per;
  int b, sub, tile, off;  // the unit at r, and how far into it r is
  Tiles t;
  int s0;

  __device__ __forceinline__ void locate(const Args& g, int subs) {
    const int lane = threadIdx.x & 31, each = (g.a.B + 31) >> 5, b0 = min(g.a.B, lane * each), b1 = min(g.a.B, b0 + each);
    long long mine = 0;
#pragma unroll 1
    for (int i = b0; i < b1; ++i) {
      const Tiles x = tiles_of(g, KS, i, s0);
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
    per = (total + g.grid - 1) / g.grid;
    r = min(total, blockIdx.x * per);
    r1 = min(total, r + per);
    b = sub = tile = off = 0;
    if (r >= r1) return;
    const int f = __ffs(__ballot_sync(0xffffffffu, incl > r)) - 1;
    if (lane == f) {
      long long at = r - (incl - mine), c;
#pragma unroll 1
      for (b = b0;; ++b) {
        t = tiles_of(g, KS, b, s0);
        c = t.cost(t.count());
        if (at < c * subs) break;
        at -= c * subs;
      }
      sub = static_cast<int>(at / c);
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
    t = tiles_of(g, KS, b, s0);
  }
  struct Seg : Unit {
    int a, e;        // key tiles [a, e) of n
    bool begins;     // the unit's first key tile is here (or it has none)
    long long last;  // the unit's last cost
  };
  // The next segment. Units without a key tile come with n = 0.
  __device__ __forceinline__ bool next(const Args& g, int subs, Seg& s) {
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
      s.a = max(off - kExtra, 0);
      s.e = max(to - kExtra, 0);
      s.begins = k > 0 ? s.a == 0 : off == 0;
      s.last = r - off + c - 1;
      r += to - off;
      const bool none = s.e == s.a && !(k == 0 && s.begins);
      s.b = b;
      s.sub = sub;
      s.tile = tile;
      s.s0 = s0;
      s.nt = min(g.tpt, t.n - tile * g.tpt);
      s.pos0 = static_cast<int>(t.pos(tile));
      s.lo = t.begin(tile);
      s.hi = t.end(tile);
      s.k0 = s.lo >> KS;
      s.n = k;
      off = to;
      if (off >= c) {
        off = 0;
        ++tile;
      }
      if (none) continue;
      return true;
    }
    return false;
  }
};

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_tc(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
               const __grid_constant__ Args g) {
  using LY = Lay<D, N>;
  constexpr int NP = LY::NP, KT = LY::KT, kRing = LY::ring, NC = LY::NC, PB = LY::PB;
  extern __shared__ __align__(1024) char sm_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  char* sm = sm_raw + ((1024u - (sa(sm_raw) & 1023u)) & 1023u);
  const unsigned base = sa(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // barriers: loaded slots, free slots; per score buffer: scores done, scores read; per parity of a
  // tile: probabilities written, sums done; queries written, sums read, drained; pages of a tile found
  const unsigned full0 = base + LY::bars, empty0 = full0 + 8 * kRing, sfull0 = empty0 + 8 * kRing, sfree0 = sfull0 + 16,
                 pfull0 = sfree0 + 16, odone0 = pfull0 + 16, qfull = odone0 + 16, ofree = qfull + 8, drain = ofree + 8,
                 ifull0 = drain + 8;
  int* info = reinterpret_cast<int*>(sm + LY::info);
  int* misc = reinterpret_cast<int*>(sm + LY::misc);  // 0: tensor memory, 1: dead, 2: begun
  volatile int *dead = misc + 1, *begun = misc + 2;  // begun: tiles that the load warp has begun
  const ChunkArgs& a = g.a;
  const Cache& c = a.c;
  const bool own_v = c.v != nullptr;
  const int G = a.nh / c.nkv, subs = c.nkv * g.hgs, PT = own_v ? 2 * NP : NP;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull0 + 8 * i, 1);
      mbar_init(sfree0 + 8 * i, 8);
      mbar_init(pfull0 + 8 * i, 8);
      mbar_init(odone0 + 8 * i, 1);
    }
    mbar_init(qfull, 8);
    mbar_init(ofree, 8);
    mbar_init(drain, 1);
    for (int i = 0; i < kInfo; ++i) mbar_init(ifull0 + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    misc[1] = misc[2] = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(misc)), "r"(LY::cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = *reinterpret_cast<volatile unsigned*>(misc);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's share (every warp for itself: no exchange)
  using W = Walk<LY::KS>;
  W w;
  w.locate(g, subs);
  typename W::Seg s;
  int* meta = g.meta + 4 * blockIdx.x;
  if (tid == 0) meta[3] = -1;

  if (warp == 10) {
    // ---------------- pages: looks up the tiles' pages up to kAhead tiles before they are loaded
    // (a lane per box, several tiles at once)
    const int rs = g.rshift, ngs = LY::KS - rs, ng = 1 << ngs, nb = min(32 >> ngs, kAhead);
    int tt = 0;
    bool ok = true;
    while (ok && w.next(g, subs, s)) {
#pragma unroll 1
      for (int k = s.a; k < s.e && ok; k += nb) {
        int page = -1;
        const int pos = ((s.k0 + k) << LY::KS) + (lane << rs);  // the tiles' boxes follow one another
        if (lane < nb * ng && pos < s.hi) page = pg::phys_page(c, s.b, pos >> c.pshift);
#pragma unroll 1
        for (int j = 0; j < nb && k + j < s.e; ++j, ++tt) {
          // the load warp has begun tile tt - kAhead, so tile tt - kInfo is done with
          if (tt >= kAhead) {
            const long long t0 = clock64();
            while (*begun < tt - kAhead + 1 && ok) {
              if (*dead || clock64() - t0 > kSpin) {
                *dead = 1;
                ok = false;
              }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          int* in = info + (tt % kInfo) * 16;
          if (lane >> ngs == j) in[lane & (ng - 1)] = page;
          __syncwarp();
          if (lane == 0) mbar_arrive(ifull0 + 8 * (tt % kInfo));
        }
      }
    }
  } else if (warp == 8) {
    // ---------------- loads
    if (elect()) {
      const int rs = g.rshift, R = 1 << rs, ng = KT >> rs, P = 1 << c.pshift;
      int pc = 0, slot = 0, tt = 0;  // slots so far, the next slot and the ring's phase there, tiles
      unsigned phase = 0;
      bool ok = true;
      while (ok && w.next(g, subs, s)) {
        const int kvh = s.sub / g.hgs;
#pragma unroll 1
        for (int k = s.a; k < s.e && ok; ++k, ++tt) {
          if (!wait_bar(ifull0 + 8 * (tt % kInfo), (tt / kInfo) & 1, dead, kSpin)) {
            ok = false;
            break;
          }
          const int* in = info + (tt % kInfo) * 16;
          const int off0 = ((s.k0 + k) << LY::KS) & (P - 1);  // 0 unless a page is longer than a tile
#pragma unroll 1
          for (int j = 0; j < PT; ++j) {
            const unsigned bar = full0 + 8 * slot;
            if (pc >= kRing && !wait_bar(empty0 + 8 * slot, phase ^ 1, dead, kSpin)) {
              ok = false;
              break;
            }
            if (j == 0) *begun = tt + 1;
            mbar_expect_tx(bar, LY::slot);
            const int x = (j < NP ? j : j - NP) * 128;
            const CUtensorMap* map = j < NP ? &mapK : &mapV;
            unsigned dst = base + slot * LY::slot;
#pragma unroll 1
            for (int r = 0; r < ng; ++r, dst += R * 128) {
              const int page = in[r];  // -1: zeros
              tma_4d(dst, map, x, off0, kvh, page, bar);
              tma_4d(dst + LY::box, map, x + 64, off0, kvh, page, bar);
            }
            ++pc;
            if (++slot == kRing) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
      }
      // no copy may be in flight when the CTA ends
#pragma unroll 1
      for (int i = max(0, pc - kRing); i < pc; ++i) {
        const long long t0 = clock64();
        while (!try_wait(full0 + 8 * (i % kRing), (i / kRing) & 1) && clock64() - t0 < kSpin) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    if (elect()) {
      // ---------------- MMA issue: the next sums or the next scores, whichever are ready.
      // fp32 += bf16 x bf16, N columns; scores: M = KT; sums: M = 128, A and B MN-major
      const unsigned id = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<unsigned>(N >> 3) << 17);
      const unsigned idS = id | (static_cast<unsigned>(KT >> 4) << 24), idO = id | (1u << 15) | (1u << 16) | (8u << 24);
      const unsigned tO = tmem, tS = tmem + NP * N;
      const unsigned kd = desc_lo(base, 16), vd = desc_lo(base, LY::box), qd = desc_lo(base + LY::q, 16),
                     pd = desc_lo(base + LY::p, KT * 128);
      // tiles whose scores / sums are issued; tiles left of the scores' segment; segments begun by
      // either; ring places
      int tq = 0, tp = 0, left = 0, nseg = 0, pseg = 0, sq = 0, sp = own_v ? NP : 0;
      unsigned fq = 0, fp = 0, starts = 0;  // starts bit i: tile tp + i is its segment's first
      bool more = true, fresh = false;
      long long t0 = clock64();
      while (more || tp < tq) {
        bool did = false;
        if (more && left == 0) {
          more = w.next(g, subs, s);
          if (more) {
            left = s.e - s.a;
            if (left) ++nseg;
            fresh = true;
          }
          continue;
        }
        if (tp < tq) {
          const bool first = starts & 1;
          if (test_wait(pfull0 + 8 * (tp & 1), (tp >> 1) & 1) && (!first || pseg == 0 || test_wait(ofree, (pseg - 1) & 1))) {
            if (own_v)
              for (int i = 0; i < NP; ++i) wait_bar(full0 + 8 * (sp + i), fp, dead, kSpin);
            fence_after();
            const unsigned v0 = vd + sp * (LY::slot >> 4), p0 = pd + (PB == 1 ? 0 : (tp & 1) * (LY::PBY >> 4));
#pragma unroll
            for (int i = 0; i < NP; ++i) {
#pragma unroll
              for (int x = 0; x < KT / 16; ++x)
                mma(tO + i * N, v0 + ((i * LY::slot + x * 2048) >> 4), p0 + (x * 2048 >> 4), idO, x > 0 || !first);
              commit(empty0 + 8 * (sp + i));
            }
            commit(odone0 + 8 * (tp & 1));
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
        if (!did && more && tq < tp + 2) {
          bool ready = (!fresh || test_wait(qfull, (nseg - 1) & 1)) &&
                       (tq < 2 || test_wait(sfree0 + 8 * (tq & 1), ((tq >> 1) - 1) & 1));
#pragma unroll
          for (int i = 0; i < NP; ++i) ready = ready && test_wait(full0 + 8 * (sq + i), fq);
          if (ready) {
            fence_after();
            const unsigned k0 = kd + sq * (LY::slot >> 4), d = tS + (tq & 1) * N;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mma(d, k0 + ((i * LY::slot + (x >> 2) * LY::box + (x & 3) * 32) >> 4),
                    qd + (((2 * i + (x >> 2)) * (N * 128) + (x & 3) * 32) >> 4), idS, i > 0 || x > 0);
              if (own_v) commit(empty0 + 8 * (sq + i));
            }
            commit(sfull0 + 8 * (tq & 1));
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
        } else if (*dead) {
          break;
        } else if (clock64() - t0 > kSpin) {
          *dead = 1;
          break;
        }
      }
      if (*dead) {  // the products that were issued still run: wait for them
        commit(drain);
        t0 = clock64();
        while (!try_wait(drain, 0) && clock64() - t0 < kSpin) {
        }
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---------------- softmax and outputs: a warpgroup per half of the columns, a thread per key of a
    // tile, and per dim of each 128-dim block of the sums
    const int wg = warp >> 2, wt = tid & 127, ww = warp & 3, col0 = wg * NC;
    const unsigned tw = tmem + (static_cast<unsigned>(32 * ww) << 16);
    const unsigned tO = tw + col0, tS = tw + NP * N + col0;
    float* const negm = reinterpret_cast<float*>(sm + LY::mref) + col0;
    unsigned* const bad = reinterpret_cast<unsigned*>(sm + LY::bad);
    // this thread's key of a tile: the accumulator row of its tensor-memory lane (M = 64 fills the
    // lower half of each warp's lanes)
    const int key = KT == 128 ? wt : 16 * ww + lane;
    const bool has = KT == 128 || lane < 16;
    auto bar_wg = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
    auto heads = [&](const Unit& u) { return min(N, G - (u.sub % g.hgs) * N); };
    auto head0 = [&](const Unit& u) { return (u.sub / g.hgs) * G + (u.sub % g.hgs) * N; };
    auto put_q = [&](const Unit& u) {
      const int Gc = heads(u), nr = u.nt * Gc, h0 = head0(u);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) +
                               static_cast<long long>(u.s0 + u.tile * g.tpt) * a.q_stride + static_cast<long long>(h0) * D;
#pragma unroll 4
      for (int i = tid; i < N * (D / 8); i += 256) {
        const int r = i / (D / 8), ch = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < nr) {
          const int tok = r / Gc, h = r - tok * Gc;
          v = *reinterpret_cast<const uint4*>(q + tok * a.q_stride + h * D + ch * 8);
        }
        *reinterpret_cast<uint4*>(sm + LY::q + (ch >> 3) * (N * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
    };
    auto scratch = [&](char* p) {
      return reinterpret_cast<float*>(N == 128 ? p + wg * (KT * 128) : sm + LY::scratch + wg * (LY::scratch_bytes / 2));
    };
    auto wait_sums = [&](int t) { wait_bar(odone0 + 8 * (t & 1), (t >> 1) & 1, dead, kSpin); };
    typename W::Seg sn;
    // units without a key are answered here: they have no tile
    auto next_unit = [&](typename W::Seg& u) {
      while (w.next(g, subs, u)) {
        if (u.n) return true;
        const int Gc = heads(u), h0 = head0(u);
        for (int i = tid; i < u.nt * Gc * (D / 8); i += 256) {
          const int r = i / (D / 8), tok = u.s0 + u.tile * g.tpt + r / Gc;
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                    (static_cast<long long>(tok) * a.nh + h0 + r % Gc) * D + i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        }
        if (a.lse)
          for (int r = tid; r < u.nt * Gc; r += 256)
            a.lse[static_cast<long long>(u.s0 + u.tile * g.tpt + r / Gc) * a.nh + h0 + r % Gc] = -INFINITY;
      }
      return false;
    };
    const int rs = g.rshift;
    bool have = next_unit(s);
    if (have) put_q(s);
    int tt = 0;  // tiles of the CTA before this segment
    while (have) {
      const int Gc = heads(s), nr = s.nt * Gc, nrw = min(max(nr - col0, 0), NC);  // rows; of this warpgroup
      const int ntl = s.e - s.a;
      // (columns behind the rows: scores of zero queries under a reference of 0)
      if (wt < NC) negm[wt] = wt < nrw ? INFINITY : 0.f;
      if (wt < 4) bad[4 * wg + wt] = 0;
      bar_wg();
      float l[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) l[i] = 0.f;
#pragma unroll 1
      for (int t = 0; t < ntl; ++t) {
        const int at = tt + t, buf = at & 1;
        char* const pbuf = sm + LY::p + (PB == 1 ? 0 : buf * LY::PBY);
        wait_bar(ifull0 + 8 * (at % kInfo), (at / kInfo) & 1, dead, kSpin);
        // the rows [cmin, cmax) of this warpgroup attend this thread's key
        const int pos = ((s.k0 + s.a + t) << LY::KS) + key, rel = pos - s.pos0;
        const int page = has ? info[(at % kInfo) * 16 + (key >> rs)] : -1;
        const bool valid = page >= 0 && pos >= s.lo && pos < s.hi;
        const int cmin = (valid ? max(rel, 0) * Gc : N) - col0;
        const int cmax = (a.window > 0 && a.window < s.nt - rel ? (rel + a.window) * Gc : nr) - col0;
        const bool masked = !__all_sync(0xffffffffu, !has || (cmin <= 0 && cmax >= nrw));
        wait_bar(sfull0 + 8 * buf, (at >> 1) & 1, dead, kSpin);
        __syncwarp();
        fence_after();
        float x[NC];
#pragma unroll
        for (int i = 0; i < NC; i += 16)
          if (i < nrw) ld16(tS + buf * N + i, x + i);
        ld_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree0 + 8 * buf);
        bool up = t == 0;
        if (!masked) {
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < NC; i += 4)
            if (i < nrw) {
              const float4 m4 = *reinterpret_cast<const float4*>(negm + i);
              mx = fmaxf(fmaxf(mx, fmaf(x[i], a.scale_log2, m4.x)), fmaf(x[i + 1], a.scale_log2, m4.y));
              mx = fmaxf(fmaxf(mx, fmaf(x[i + 2], a.scale_log2, m4.z)), fmaf(x[i + 3], a.scale_log2, m4.w));
            }
          up = up || (has && mx > 8.f);
        } else {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (i < nrw && i >= cmin && i < cmax) up = up || (has && !(fmaf(x[i], a.scale_log2, negm[i]) <= 8.f));
        }
        int any;
        asm volatile("{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.s32 %0, 1, 0, q;\n}"
                     : "=r"(any)
                     : "r"(up ? 1 : 0), "r"(1 + wg)
                     : "memory");
        if (any) {  // new references: the maxima so far
          if (t > 0) wait_sums(at - 1);
          __syncwarp();
          fence_after();
          float* const red = scratch(pbuf);
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (i < nrw) {
              const float v = has && i >= cmin && i < cmax ? pg::attended(x[i] * a.scale_log2) : -INFINITY;
              const float m = warp_max_redux(v);
              if (lane == (i & 31)) red[ww * NC + i] = m;
            }
          bar_wg();
          if (wt < nrw) {
            const float mo = -negm[wt], mn = fmaxf(fmaxf(fmaxf(red[wt], red[NC + wt]), fmaxf(red[2 * NC + wt], red[3 * NC + wt])), mo);
            red[4 * NC + wt] = mo == -INFINITY ? 0.f : ex2(mo - mn);
            negm[wt] = -mn;
          }
          bar_wg();
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (i < nrw) l[i] *= red[4 * NC + i];
          if (t > 0) {
#pragma unroll 1
            for (int b = 0; b < NP; ++b)
#pragma unroll
              for (int i = 0; i < NC; i += 16)
                if (i < nrw) {
                  float v[16];
                  ld16(tO + b * N + i, v);
                  ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) v[e] *= i + e < nrw ? red[4 * NC + i + e] : 0.f;
                  st16(tO + b * N + i, v);
                }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            fence_before();
          }
          bar_wg();  // the scratch is read
        }
        if (at >= PB) wait_sums(at - PB);  // the buffer's last probabilities are used
        char* const prow = pbuf + key * 128;
#pragma unroll
        for (int i = 0; i < NC; i += 8)
          if (i < nrw) {
            float p[8];
            const float4 m0 = *reinterpret_cast<const float4*>(negm + i), m1 = *reinterpret_cast<const float4*>(negm + i + 4);
            const float mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = ex2(fmaf(x[i + e], a.scale_log2, mm[e]));
            if (masked) {
#pragma unroll
              for (int e = 0; e < 8; ++e) p[e] = i + e >= cmin && i + e < cmax ? p[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) l[i + e] += p[e];
            const int col = col0 + i;
            if (has)
              *reinterpret_cast<uint4*>(prow + (col >> 6) * (KT * 128) + ((((col & 63) >> 3) ^ (key & 7)) << 4)) =
                  make_uint4(pack2(p[0], p[1]), pack2(p[2], p[3]), pack2(p[4], p[5]), pack2(p[6], p[7]));
          }
        // keys of the tile that no row of the unit attends, and values that are not finite in keys that
        // only some do: this warpgroup's half of the dims
        const int amin = cmin + col0, amax = min(cmax + col0, nr);
        if (has && page >= 0 && (!valid || amin > 0 || amax < nr)) {
#pragma unroll 1
          for (int j = wg * NP; j < (wg + 1) * NP; ++j) {  // blocks of 64 dims
            const int pc = at * PT + (own_v ? NP : 0) + (j >> 1), slot = pc % kRing;
            if (own_v && !wait_bar(full0 + 8 * slot, (pc / kRing) & 1, dead, kSpin)) break;
            uint4* row = reinterpret_cast<uint4*>(sm + slot * LY::slot + (j & 1) * LY::box + key * 128);
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
              if (!valid) {
                row[e] = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint4 v = row[e];
              unsigned* u = reinterpret_cast<unsigned*>(&v);
              bool off = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((u[i] & 0x7f800000u) == 0x7f800000u) off = true, u[i] &= 0xffffu;
                if ((u[i] & 0x7f80u) == 0x7f80u) off = true, u[i] &= 0xffff0000u;
              }
              if (off) {
                row[e] = v;
#pragma unroll 1
                for (int i = amin; i < amax; ++i) atomicOr(bad + 4 * wg + (i >> 5), 1u << (i & 31));
              }
            }
          }
        }
        fence_async();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull0 + 8 * buf);
      }
      const bool more = next_unit(sn);
      if (more) put_q(sn);  // every product with this unit's queries is done
      // ---- the unit's sums
      wait_sums(tt + ntl - 1);
      __syncwarp();
      fence_after();
      float* const red = scratch(sm + LY::p);
#pragma unroll
      for (int i = 0; i < NC; ++i) l[i] = has ? l[i] : 0.f;
      if constexpr (NC >= 32) {
#pragma unroll
        for (int i = 0; i < NC; i += 32) {
          reduce_scatter<32, 16>(l + i, lane);
          red[ww * NC + i + lane] = l[i];
        }
      } else {
        reduce_scatter<NC, 16>(l, lane);
        if (lane % (32 / NC) == 0) red[ww * NC + lane / (32 / NC)] = l[0];
      }
      bar_wg();
      const bool whole = s.a == 0 && s.e == s.n;
      const int h0 = head0(s);
      const long long tok0 = s.s0 + static_cast<long long>(s.tile) * g.tpt;
      const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + (s.begins ? 1 : 0)) * N;
      if (wt < nrw) {
        const int col = col0 + wt;
        float den = (red[wt] + red[NC + wt]) + (red[2 * NC + wt] + red[3 * NC + wt]);
        const float m = -negm[wt];
        if (*dead || ((bad[col >> 5] | bad[4 + (col >> 5)]) >> (col & 31) & 1)) den = NAN;
        if (whole) {
          den = pg::row_sum(m, den);
          red[4 * NC + wt] = den == 0.f ? 0.f : 1.f / den;  // 0: nothing attended
          if (a.lse)
            a.lse[(tok0 + col / Gc) * a.nh + h0 + col % Gc] = den == 0.f ? -INFINITY : (m + log2f(den)) * 0.6931471805599453f;
        } else {
          a.ws_ml[(part + col) * 2] = m;
          a.ws_ml[(part + col) * 2 + 1] = den;
        }
      }
      bar_wg();
#pragma unroll 1
      for (int b = 0; b < NP; ++b) {
#pragma unroll 1
        for (int i = 0; i < nrw; i += 16) {
          float v[16];
          ld16(tO + b * N + i, v);
          ld_wait();
          const int dim = b * 128 + wt;
          int tok = (col0 + i) / Gc, h = (col0 + i) - tok * Gc;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (i + e < nrw) {
              if (whole)
                static_cast<__nv_bfloat16*>(a.out)[((tok0 + tok) * a.nh + h0 + h) * D + dim] =
                    __float2bfloat16_rn(red[4 * NC + i + e] == 0.f ? 0.f : v[e] * red[4 * NC + i + e]);
              else
                a.ws_acc[(part + col0 + i + e) * D + dim] = v[e];
              if (++h == Gc) {
                h = 0;
                ++tok;
              }
            }
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);
      if (!whole && s.begins && tid == 0) {
        meta[0] = s.b;
        meta[1] = s.sub;
        meta[2] = s.tile;
        meta[3] = static_cast<int>(s.last / w.per);
      }
      asm volatile("bar.sync 3, 256;" ::: "memory");  // both warpgroups have read the scratch, the marks and the references
      tt += ntl;
      s = sn;
      have = more;
    }
    fence_before();
  }
  __syncthreads();
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
  const int4 meta = *reinterpret_cast<const int4*>(g.meta + 4 * blockIdx.x);  // sequence, KV head and group, tile, last CTA
  if (meta.w < 0) return;
  const ChunkArgs& a = g.a;
  int s0, n, first, L;
  pg::chunk_range(a, meta.x, s0, n, first, L);
  const int G = a.nh / a.c.nkv, hg = meta.y % g.hgs, Gc = min(N, G - hg * N), nt = min(g.tpt, n - meta.z * g.tpt);
  const int lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), c0 = blockIdx.x, np = meta.w - c0 + 1;
  if (r >= nt * Gc) return;
  const long long row = (static_cast<long long>(s0) + meta.z * g.tpt + r / Gc) * a.nh + (meta.y / g.hgs) * G + hg * N + r % Gc;
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
  static_assert(N != 128 || 5 * LY::NC * 4 <= LY::KT * 128, "the softmax's scratch");
  CUtensorMap mk, mv;
  int rc = make_map(&mk, g.a.c, g.a.c.k, 1 << g.rshift);
  if (rc) return rc;
  mv = mk;
  if (g.a.c.v && (rc = make_map(&mv, g.a.c, g.a.c.v, 1 << g.rshift))) return rc;
  const cudaError_t e = pg::allow_smem<k_chunk_tc<D, N>, LY::total>();
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("chunk attention: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  rc = pg::launch_pdl("chunk attention", k_chunk_tc<D, N>, dim3(g.grid), kThreads, LY::total, st, mk, mv, g);
  return rc ? rc : pg::launch_pdl("chunk attention join", k_chunk_tc_join<D>, dim3(g.grid, N / kJoinWarps), kJoinWarps * 32, 0, st, g, N);
}

}  // namespace pgc

// Rows of a tile: 64 at d = 512, 128 below, and 32 where the sequences have at most 32 rows each on
// average.
static int chunk_tc_rows(const pg::ChunkArgs& a) {
  if (static_cast<long long>(a.T) * (a.nh / a.c.nkv) <= 32LL * a.B) return 32;
  return a.c.d == 512 ? 64 : 128;
}

long long chunk_tc_workspace(const pg::ChunkArgs& a) {
  return pg::kMaxSms * (16LL + 2LL * chunk_tc_rows(a) * (a.c.d + 2) * 4);
}

int run_chunk_tc(const pg::ChunkArgs& a, void* ws, int num_sms, cudaStream_t st) {
  using namespace pgc;
  Args g;
  memset(&g, 0, sizeof(g));
  g.a = a;
  const int P = 1 << a.c.pshift, G = a.nh / a.c.nkv, N = chunk_tc_rows(a), KT = a.c.d == 512 ? 64 : 128;
  const int rows = P < KT ? P : KT;
  while ((1 << g.rshift) < rows) ++g.rshift;
  g.tpt = 1;
  while (g.tpt * 2 * G <= N) g.tpt *= 2;
  g.hgs = (G + N - 1) / N;
  g.grid = num_sms;
  g.meta = static_cast<int*>(ws);
  g.a.ws_ml = reinterpret_cast<float*>(g.meta + 4 * pg::kMaxSms);
  g.a.ws_acc = g.a.ws_ml + pg::kMaxSms * 2 * N * 2;
  if (a.c.d == 512) return N == 32 ? launch<512, 32>(g, st) : launch<512, 64>(g, st);
  if (a.c.d == 256) return N == 32 ? launch<256, 32>(g, st) : launch<256, 128>(g, st);
  return N == 32 ? launch<128, 32>(g, st) : launch<128, 128>(g, st);
}

}  // namespace mtp
