// Attention of one new token over a paged key cache on tensor cores (bf16 cache, head_dim 128,
// 256 or 512, pages of at least 8 tokens): the formula of mtp_paged_att.cu.
//
// What bounds it is reading the cache once: with the join 151 MB take 35.3 us at d = 512 (8 long
// ragged contexts, 4.3 TB/s), 134 MB 30.7 us at d = 128 (32 x 8192, 4.4 TB/s), 128 MB of K and V
// 32.9 us at d = 128 (61 short contexts, 3.9 TB/s). From one length to the double the time grows by
// the keys at 6.6 to 7.1 TB/s (8 x 8192 to 8 x 32768 keys at d = 512, 32 x 4096 to 32 x 16384 at
// d = 128); the rest, 10 to 11 us, is the start (3 us: length, table, keys), the tail and the join
// (3 to 4 us). On CUDA cores it is the arithmetic instead: with G
// query heads per KV head and V = K a 2-byte key element costs 4 G flops, 16 flop per byte at
// G = 8, which at the cache's bandwidth is more than the fp32 pipes give. So both products run as
// tcgen05.mma with the *keys* as the 128-row operand, straight from the TMA-loaded tile:
//   scores  S^T [128 keys][N] = K_tile [128][d] Q^T,        A = K_tile, K-major
//   sums    O^T [d][N]        = V_tile^T [d][128] P^T,      A = V_tile, MN-major (the same bytes
//                                                            when V = K: each is read once)
// and the few query heads as the N side: every fp32 query value and probability is split into
// three bf16 terms (hi + mid + lo, exact), N = 3 columns per head, so every product is exact and
// the sums are fp32. The tensor-memory adder truncates, so no chain is long: scores accumulate
// 128 dims (8 instructions), sums 128 keys, and the parts are added in registers, rounded to
// nearest; a score's parts term by term, so that a part of the first term does not round away what
// the last term adds in another.
//
// Work split: the granules (32 to 128 keys) of all (sequence, KV head, head group) units are
// numbered through and dealt evenly over one CTA per SM, whatever the lengths; a unit's beginning
// counts as `extra` granules, since a CTA that goes from one unit to the next drains and refills
// its pipeline (3 us at d = 512, where such CTAs were the last to finish). A unit that crosses
// CTAs leaves unnormalised sums, (max, exp-sum) per part; k_paged_tc_join adds them in CTA order.
// (Joined by the last CTA to arrive instead, the 8 long contexts took 48 us against 41: its chain
// of round trips runs while the memory is busy with the others' keys.)
//
// With few, short units (kCluster CTAs for each fit, a CTA's share is a few tiles) a thread-block
// cluster takes a unit instead: the parts stay in shared memory, and after a cluster barrier every
// CTA joins a slice of the outputs through distributed shared memory; no second launch.
//
// One CTA: warp 10 finds the tiles' pages through the block table, warp 8 loads them (slots of
// [KT keys][128 dims] in two 128-byte-swizzled boxes, a ring of 192 KB), one thread of warp 9
// issues the MMAs (whichever of the next score slot and the next sum is ready), and two warpgroups
// take the tiles in turn, each with a softmax reference and sums of its own (one thread per key,
// then one per dim of each 128-dim block); they are joined at the end of a segment. The reference is a maximum that moves
// only when a score exceeds it by 2^8 (one barrier per tile agrees on that), so running sums are
// rarely rescaled.
// Rows that hold no attended key but lie in an attended page are set to zero before the sums
// (0 * NaN would not vanish). Waits are bounded; a CTA that gives up writes NaN and reports it in
// the caller's status word, if there is one.
#include <cudaTypedefs.h>

#include <atomic>
#include <cstring>

#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"
#include "mtp_paged_mma.cuh"

namespace mtp {
namespace pgt {

using pg::AttArgs;
using pg::Cache;
using pg::kSpin;

constexpr int kRingBytes = 192 * 1024;     // loaded keys
constexpr int kThreadsTc = 352;            // two warpgroups for the softmax; load, MMA and find warps
constexpr int kCluster = 8;                // CTAs of a unit in the clustered form
constexpr int kClusterBytes = 256 * 1024;  // most keys of one of them
constexpr int kAhead = 8;                  // tiles that the find warp runs ahead of the load warp
constexpr int kInfo = 2 * kAhead;          // tiles whose pages and positions are kept

struct Args {
  AttArgs a;
  int gshift;    // log2 of the keys of a granule, which are dealt as a whole
  int extra;     // what beginning a unit costs, in granules
  int rshift;    // log2 of the keys per TMA box (min(P, keys per tile))
  int grid;      // CTAs that share the granules
  int clustered; // a cluster per unit
  int ngrp;      // head groups per KV head
  int* meta;     // [grid][4]: first output row, heads, last CTA of the unit a CTA starts and does not end
};

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of a peer of the cluster, at this CTA's address of the same variable.
__device__ __forceinline__ unsigned peer(unsigned addr, int rank) {
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_f32(unsigned addr, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer(addr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f32x4(unsigned addr, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer(addr, rank))
               : "memory");
  return v;
}

// The three term columns of NH heads at tensor-memory address t: v[3 * NH].
template <int NH>
__device__ __forceinline__ void ld_terms(unsigned t, float* v) {
  if (NH == 4) {
    ld8(t, v);
    ld4(t + 8, v + 8);
  } else {
    ld8(t, v);
    ld8(t + 8, v + 8);
    ld8(t + 16, v + 16);
  }
}

__device__ __forceinline__ void split3(float v, __nv_bfloat16& hi, __nv_bfloat16& mid, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float r = v - __bfloat162float(hi);
  mid = __float2bfloat16_rn(r);
  lo = __float2bfloat16_rn(r - __bfloat162float(mid));
}

template <int D, int NH>
struct Lay {
  static constexpr int N = NH == 4 ? 16 : 32;           // MMA columns (3 NH used, the rest ignored)
  static constexpr int NP = D / 128;                    // 128-dim slots per tile and operand
  // keys per tile: 64 where a tile of 128 keys would leave too little of the ring for loads in
  // flight (d = 512) or the query buffers no room
  static constexpr int KT = D == 512 || (D == 256 && NH == 8) ? 64 : 128;
  static constexpr int KS = KT == 64 ? 6 : 7;           // log2 KT
  static constexpr int box = KT * 128;                  // KT keys x 64 dims
  static constexpr int slot = 2 * box;
  static constexpr int ring = kRingBytes / slot;        // 6 or 12 slots
  static constexpr int RB = (NH == 4 ? 16 : 24) * 128;  // bytes of one 64-element block of the N side (3 NH rows, whole swizzle blocks)
  static constexpr int QB = D == 512 ? 1 : 2;           // query buffers
  static constexpr int PBY = KT / 64 * RB;              // bytes of one probability buffer
  static constexpr int q = kRingBytes;
  static constexpr int p = q + QB * (D / 64) * RB;
  static constexpr int bars = p + 2 * PBY;
  static constexpr int nbars = 2 * ring + 2 * 6 + 1 + kInfo;
  // per tile: first position of each row group (-1: none), its physical page, the KV head
  static constexpr int info = bars + nbars * 8;
  static constexpr int red = info + kInfo * 33 * 4;      // per warpgroup [4][8] maxima, [4][8] sums, [8] references
  static constexpr int misc = red + 2 * 72 * 4;          // tensor-memory address, dead word, tiles begun
  static constexpr int total = misc + 16 + 1024;     // + alignment
  static constexpr int cols = 4 * NP * N;                // 2 score and 2 sum regions of NP * N columns
};

// Walks the segments (parts of units) of a CTA's share: costs [r, r1), where a unit of n granules
// is `extra` costs without a granule and then one cost per granule.
struct Walk {
  int r, r1, b, sub, off, n, lo, hi, base;
  // granules of a unit of sequence b
  __device__ __forceinline__ static int count(const Args& g, int b, int& lo, int& hi, int& base) {
    pg::key_range(g.a.c, b, g.a.window, lo, hi);
    base = 0;
    int keys;
    if (g.a.list) {
      keys = hi > 0 ? g.a.n_list << g.a.c.pshift : 0;
    } else {
      base = lo >> g.rshift << g.rshift;
      keys = hi - base;
    }
    return (keys + (1 << g.gshift) - 1) >> g.gshift;
  }
  __device__ __forceinline__ static int cost(const Args& g, int n) { return n > 0 ? n + g.extra : 0; }
  // This CTA's share and the unit it begins in: the whole warp, a lane for 1/32 of the sequences.
  // Returns the costs per CTA.
  __device__ __forceinline__ int locate(const Args& g, int subs) {
    const int lane = threadIdx.x & 31, per_b = (g.a.B + 31) >> 5, b0 = min(g.a.B, lane * per_b), b1 = min(g.a.B, b0 + per_b);
    int mine = 0;
#pragma unroll 1
    for (int i = b0; i < b1; ++i) mine += cost(g, count(g, i, lo, hi, base));
    mine *= subs;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31), per = (total + g.grid - 1) / g.grid;
    r = min(total, static_cast<int>(blockIdx.x) * per);
    r1 = min(total, r + per);
    b = sub = off = n = 0;
    if (r >= r1) return per;
    const int f = __ffs(__ballot_sync(0xffffffffu, incl > r)) - 1;
    if (lane == f) {
      int at = r - (incl - mine), c;
#pragma unroll 1
      for (b = b0;; ++b) {
        n = count(g, b, lo, hi, base);
        c = cost(g, n);
        if (at < c * subs) break;
        at -= c * subs;
      }
      if (subs > 1) {
        sub = at / c;
        at -= sub * c;
      }
      off = at;
    }
    b = __shfl_sync(0xffffffffu, b, f);
    sub = __shfl_sync(0xffffffffu, sub, f);
    off = __shfl_sync(0xffffffffu, off, f);
    n = __shfl_sync(0xffffffffu, n, f);
    lo = __shfl_sync(0xffffffffu, lo, f);
    hi = __shfl_sync(0xffffffffu, hi, f);
    base = __shfl_sync(0xffffffffu, base, f);
    return per;
  }
  // The clustered form: this CTA's part of its cluster's unit (extra is 0).
  __device__ __forceinline__ void place(const Args& g, int subs) {
    const int unit = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
    b = unit / subs;
    sub = unit - b * subs;
    n = count(g, b, lo, hi, base);
    off = static_cast<int>(static_cast<long long>(n) * rank / kCluster);
    r = 0;
    r1 = static_cast<int>(static_cast<long long>(n) * (rank + 1) / kCluster) - off;
  }
  struct Seg {
    int b, kvh, hg, a, e, n, lo, hi, base;  // KV head and group of its heads; granules [a, e) of n
    int end;                                // one past the unit's last cost
  };
  __device__ __forceinline__ bool next(const Args& g, int subs, Seg& s) {
#pragma unroll 1
    while (r < r1) {
      const int c = cost(g, n);
      if (off >= c) {  // the next unit
        off = 0;
        if (n == 0 || ++sub == subs) {
          sub = 0;
          ++b;
          n = count(g, b, lo, hi, base);
        }
        continue;
      }
      const int to = min(c, off + (r1 - r));
      s.a = max(off - g.extra, 0);
      s.e = max(to - g.extra, 0);
      s.end = r - off + c;
      r += to - off;
      off = to;
      if (s.e == s.a) continue;
      s.b = b;
      s.kvh = sub;
      s.hg = 0;
      if (g.ngrp > 1) {
        s.kvh = sub / g.ngrp;
        s.hg = sub - s.kvh * g.ngrp;
      }
      s.n = n;
      s.lo = lo;
      s.hi = hi;
      s.base = base;
      return true;
    }
    return false;
  }
  // one past the last key number of a segment (its first is s.a << g.gshift)
  __device__ __forceinline__ int end(const Args& g, const Seg& s) const {
    return min(g.a.list ? g.a.n_list << g.a.c.pshift : s.hi - s.base, s.e << g.gshift);
  }
};

template <int D, int NH>
__global__ void __launch_bounds__(kThreadsTc, 1)
    k_paged_tc(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
               const __grid_constant__ Args g) {
  using LY = Lay<D, NH>;
  constexpr int N = LY::N, NP = LY::NP, RB = LY::RB, KT = LY::KT, kRing = LY::ring, QB = LY::QB;
  extern __shared__ __align__(1024) char sm_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  char* sm = sm_raw + ((1024u - (sa(sm_raw) & 1023u)) & 1023u);
  const unsigned base = sa(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned full0 = base + LY::bars, empty0 = full0 + 8 * kRing, sfull0 = empty0 + 8 * kRing, sfree0 = sfull0 + 16,
                 pfull0 = sfree0 + 16, ofull0 = pfull0 + 16, ofree0 = ofull0 + 16, qfull0 = ofree0 + 16,
                 drain = qfull0 + 16, ifull0 = drain + 8;
  int* info = reinterpret_cast<int*>(sm + LY::info);
  int* misc = reinterpret_cast<int*>(sm + LY::misc);  // 0: tensor memory, 1: dead, 2: begun
  volatile int *dead = misc + 1, *begun = misc + 2;  // begun: tiles that the load warp has begun
  const AttArgs& a = g.a;
  const Cache& c = a.c;
  const bool own_v = c.v != nullptr;
  const int subs = c.nkv * g.ngrp, G = a.nh / c.nkv, PT = own_v ? 2 * NP : NP;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull0 + 8 * i, 1);
      mbar_init(sfree0 + 8 * i, 4);
      mbar_init(pfull0 + 8 * i, 4);
      mbar_init(ofull0 + 8 * i, 1);
      mbar_init(ofree0 + 8 * i, 4);
      mbar_init(qfull0 + 8 * i, 4);
    }
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

  // ---- this CTA's share: granules [r, r1) of all units (every warp for itself: no exchange)
  Walk w;
  int per = 0;
  if (g.clustered)
    w.place(g, subs);
  else
    per = w.locate(g, subs);
  const bool work = w.r < w.r1;
  // a unit that starts here and goes on in the next CTAs
  int* meta = g.meta + 4 * blockIdx.x;
  if (tid == 0 && !g.clustered) meta[1] = 0;

  if (warp == 10) {
    // ---------------- pages: looks up the tiles' pages up to kAhead tiles before they are loaded
    // (a lane per row group, several tiles at once)
    const int rs = g.rshift, ngs = LY::KS - rs, ng = 1 << ngs, P = 1 << c.pshift, nb = min(32 >> ngs, kAhead);
    int tt = 0;
    bool ok = true;
    Walk::Seg s;
    while (ok && w.next(g, subs, s)) {
      if (s.b == a.skip) {  // testing: the other warps wait for these tiles until they give up
        ok = false;
        break;
      }
      const int kvh = s.kvh, i1 = w.end(g, s);
      const int* list = a.list ? a.list + (static_cast<size_t>(s.b) * c.nkv + kvh) * a.n_list : nullptr;
#pragma unroll 1
      for (int i0 = (s.a << g.gshift); i0 < i1 && ok; i0 += nb * KT) {
        int page = -1, pos = -1;
        const int i = i0 + (lane << rs);  // the tiles' row groups follow one another
        if (lane < nb * ng && i < i1) {
          int lp, off;
          if (list) {
            lp = list[i >> c.pshift];
            off = i & (P - 1);
          } else {
            lp = (s.base + i) >> c.pshift;
            off = (s.base + i) & (P - 1);
          }
          if (lp >= 0 && lp < c.max_pages && (lp << c.pshift) < s.hi) {
            page = pg::phys_page(c, s.b, lp);
            if (page >= 0) pos = (lp << c.pshift) + off;
          }
        }
#pragma unroll 1
        for (int j = 0; j < nb && i0 + j * KT < i1; ++j, ++tt) {
          // the load warp has begun tile tt - kAhead, so tile tt - kInfo is done with
          if (tt >= kAhead) {
            const long long t0 = clock64();
            while (*begun < tt - kAhead + 1 && ok) {
              if (*dead || clock64() - t0 > a.spin) {
                *dead = 1;
                ok = false;
              }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          int* in = info + (tt % kInfo) * 33;
          if (lane >> ngs == j) {
            in[lane & (ng - 1)] = pos;
            in[16 + (lane & (ng - 1))] = page;
          }
          if (lane == 0) in[32] = kvh;
          __syncwarp();
          if (lane == 0) mbar_arrive(ifull0 + 8 * (tt % kInfo));
        }
      }
    }
    if (ok) {  // the end
      if (tt >= kAhead) {
        const long long t0 = clock64();
        while (*begun < tt - kAhead + 1 && !*dead && clock64() - t0 < a.spin) {
        }
      }
      __syncwarp();
      if (lane == 0) {
        info[(tt % kInfo) * 33 + 32] = -1;
        mbar_arrive(ifull0 + 8 * (tt % kInfo));
      }
    }
  } else if (warp == 8) {
    // ---------------- loads
    if (elect()) {
      const int R = 1 << g.rshift, ng = KT >> g.rshift, P = 1 << c.pshift;
      // keys pass through once: they leave the L2 before the tables, the code and the parts do
      unsigned long long policy;
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      int pc = 0, slot = 0;  // slots so far, the next slot and the ring's phase there
      unsigned phase = 0;
      bool ok = true;
      for (int tt = 0; ok; ++tt) {
        if (!wait_bar(ifull0 + 8 * (tt % kInfo), (tt / kInfo) & 1, dead, a.spin)) break;
        const int* in = info + (tt % kInfo) * 33;
        const int kvh = in[32];
        if (kvh < 0) break;
#pragma unroll 1
        for (int j = 0; j < PT; ++j) {
          const unsigned bar = full0 + 8 * slot;
          if (pc >= kRing && !wait_bar(empty0 + 8 * slot, phase ^ 1, dead, a.spin)) {
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
            const int pos = in[r], off = pos < 0 ? 0 : pos & (P - 1), page = in[16 + r];  // page -1: zeros
            tma_4d(dst, map, x, off, kvh, page, bar, policy);
            tma_4d(dst + LY::box, map, x + 64, off, kvh, page, bar, policy);
          }
          ++pc;
          if (++slot == kRing) {
            slot = 0;
            phase ^= 1;
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
      // ---------------- MMA issue: the next score tile or the next sum tile, whichever is ready.
      // A tile's slots of one operand are NP neighbours (the ring is a multiple of NP).
      // fp32 += bf16 x bf16, N columns, M = KT (scores) or 128 with A MN-major (sums)
      const unsigned id = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<unsigned>(N >> 3) << 17);
      const unsigned idS = id | (static_cast<unsigned>(KT >> 4) << 24), idO = id | (1u << 15) | (8u << 24);
      const unsigned tS = tmem, tO = tmem + 2 * NP * N;
      const unsigned kd = desc_lo(base, 16), vd = desc_lo(base, LY::box), qd = desc_lo(base + LY::q, 16),
                     pd = desc_lo(base + LY::p, 16);
      // tiles whose scores / sums are issued, their first slots and the ring's phases there
      int tq = 0, tp = 0, left = 0, nseg = 0, wq = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;
      int sq = 0, sp = own_v ? NP : 0;
      unsigned fq = 0, fp = 0, owner = 0;  // owner bit i: the warpgroup of tile tp + i
      bool more = work;
      long long t0 = clock64();
      while (more || tp < tq) {
        bool did = false;
        if (more && left == 0) {
          Walk::Seg s;
          more = w.next(g, subs, s);
          if (more) {
            left = (w.end(g, s) - (s.a << g.gshift) + KT - 1) / KT;
            wq = 0;
            ++nseg;
          }
          continue;
        }
        if (tp < tq) {
          const int wp = owner & 1, use = wp ? np1 : np0;
          if (test_wait(pfull0 + 8 * wp, use & 1) && (use == 0 || test_wait(ofree0 + 8 * wp, (use - 1) & 1))) {
            if (own_v)
              for (int i = 0; i < NP; ++i) wait_bar(full0 + 8 * (sp + i), fp, dead, a.spin);
            fence_after();
            const unsigned v0 = vd + sp * (LY::slot >> 4), p0 = pd + wp * (LY::PBY >> 4), d = tO + wp * NP * N;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
#pragma unroll
              for (int x = 0; x < KT / 16; ++x)
                mma(d + i * N, v0 + ((i * LY::slot + x * 2048) >> 4), p0 + (((x >> 2) * RB + (x & 3) * 32) >> 4), idO, x > 0);
              commit(empty0 + 8 * (sp + i));
            }
            commit(ofull0 + 8 * wp);
            owner >>= 1;
            ++tp;
            if (wp) ++np1; else ++np0;
            if ((sp += PT) >= kRing) {
              sp -= kRing;
              fp ^= 1;
            }
            did = true;
          }
        }
        if (!did && more && tq < tp + 3) {
          const int use = wq ? nq1 : nq0, qb = (nseg - 1) % QB;
          bool ready = test_wait(qfull0 + 8 * qb, ((nseg - 1) / QB) & 1) &&
                       (use == 0 || test_wait(sfree0 + 8 * wq, (use - 1) & 1));
#pragma unroll
          for (int i = 0; i < NP; ++i) ready = ready && test_wait(full0 + 8 * (sq + i), fq);
          if (ready) {
            fence_after();
            const unsigned k0 = kd + sq * (LY::slot >> 4), q0 = qd + qb * ((D / 64) * RB >> 4), d = tS + wq * NP * N;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mma(d + i * N, k0 + ((i * LY::slot + (x >> 2) * LY::box + (x & 3) * 32) >> 4),
                    q0 + (((2 * i + (x >> 2)) * RB + (x & 3) * 32) >> 4), idS, x > 0);
            }
            if (own_v) {
#pragma unroll
              for (int i = 0; i < NP; ++i) commit(empty0 + 8 * (sq + i));
            }
            commit(sfull0 + 8 * wq);
            owner = (owner & ~(1u << (tq - tp))) | (static_cast<unsigned>(wq) << (tq - tp));
            ++tq;
            --left;
            if (wq) ++nq1; else ++nq0;
            wq ^= 1;
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
        } else if (clock64() - t0 > a.spin) {
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
  } else {
    // ---------------- softmax, sums, outputs. A warpgroup takes every other tile of a segment
    // with a reference, sums and outputs of its own: thread = key of a tile, and dim of each
    // 128-dim block of the sums. The two are joined at the segment's end.
    const int wg = warp >> 2, wt = tid & 127, ww = warp & 3;
    float* red = reinterpret_cast<float*>(sm + LY::red) + 72 * wg;
    const float* red0 = reinterpret_cast<const float*>(sm + LY::red);
    const unsigned tw = tmem + (static_cast<unsigned>(32 * ww) << 16);
    const unsigned tS = tw + wg * NP * N, tO = tw + (2 + wg) * NP * N;
    char* const pbuf = sm + LY::p + wg * LY::PBY;
    // this thread's key of a tile: the accumulator row of its tensor-memory lane (M = 64 fills
    // the lower half of each warp's lanes)
    const int key = KT == 128 ? wt : 16 * ww + lane;
    const bool has = KT == 128 || lane < 16;
    auto bar_wg = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
    // the queries of a unit as three bf16 terms per value: row term * NH + head
    auto put_q = [&](const Walk::Seg& u, int buf) {
      const int h0 = u.kvh * G + u.hg * NH, nh = min(NH, G - u.hg * NH);
#pragma unroll 1
      for (int i = wt; i < NH * (D / 8); i += 128) {
        const int h = i / (D / 8), ch = i % (D / 8);
        float v[8];
        if (h < nh) {
          const float4* q4 = reinterpret_cast<const float4*>(a.q + (static_cast<size_t>(u.b) * a.nh + h0 + h) * D) + 2 * ch;
          *reinterpret_cast<float4*>(v) = q4[0];
          *reinterpret_cast<float4*>(v + 4) = q4[1];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 0.f;
        }
        __align__(16) __nv_bfloat16 t[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split3(v[e], t[0][e], t[1][e], t[2][e]);
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          const int r = term * NH + h;
          *reinterpret_cast<uint4*>(sm + LY::q + (buf * (D / 64) + (ch >> 3)) * RB + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
              *reinterpret_cast<const uint4*>(t[term]);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull0 + 8 * buf);
    };
    const int rs = g.rshift;
    Walk::Seg s, sn;
    bool have = work && w.next(g, subs, s);
    if (have && wg == 0) put_q(s, 0);
    int tt = 0, own = 0, seg = 0;  // tiles of the CTA before this segment, tiles of this warpgroup, segments
    while (have) {
      const bool more = w.next(g, subs, sn);
      // with two query buffers the next unit's queries are ready before its first tile; the
      // buffer's last products ended with the segment before this one
      if (QB == 2 && more && wg == 1) put_q(sn, (seg + 1) & 1);
      float acc[NP][NH], m[NH], l[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int b = 0; b < NP; ++b) acc[b][h] = 0.f;
      }
      auto take_o = [&](int use) {  // the sums of this warpgroup's tile `use`
        wait_bar(ofull0 + 8 * wg, use & 1, dead, a.spin);
        __syncwarp();
        fence_after();
#pragma unroll
        for (int b = 0; b < NP; ++b) {
          float v[3 * NH];
          ld_terms<NH>(tO + b * N, v);
          ld_wait();
#pragma unroll
          for (int h = 0; h < NH; ++h) acc[b][h] += (v[2 * NH + h] + v[NH + h]) + v[h];
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree0 + 8 * wg);
      };
      const int nt = (w.end(g, s) - (s.a << g.gshift) + KT - 1) / KT;
#pragma unroll 1
      for (int t = wg; t < nt; t += 2, ++own) {
        const int at = tt + t;
        wait_bar(ifull0 + 8 * (at % kInfo), (at / kInfo) & 1, dead, a.spin);
        const int pb = has ? info[(at % kInfo) * 33 + (key >> rs)] : -1, pos = pb + (key & ((1 << rs) - 1));
        const bool on = pb >= 0 && pos >= s.lo && pos < s.hi;
        wait_bar(sfull0 + 8 * wg, own & 1, dead, a.spin);
        __syncwarp();
        fence_after();
        // the terms' parts of 128 dims, term by term
        float sc[3 * NH];
        ld_terms<NH>(tS, sc);
        ld_wait();
#pragma unroll
        for (int b = 1; b < NP; ++b) {
          float v[3 * NH];
          ld_terms<NH>(tS + b * N, v);
          ld_wait();
#pragma unroll
          for (int i = 0; i < 3 * NH; ++i) sc[i] += v[i];
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) sc[h] += sc[2 * NH + h] + sc[NH + h];
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree0 + 8 * wg);
        bool up = false;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          sc[h] = on ? pg::attended(sc[h] * a.scale_log2) : -INFINITY;
          up = up || (on && !(sc[h] <= m[h] + 8.f));  // NaN counts
        }
        int any;
        asm volatile("{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.s32 %0, 1, 0, q;\n}"
                     : "=r"(any)
                     : "r"(up ? 1 : 0), "r"(1 + wg)
                     : "memory");
        // the sums of this warpgroup's last tile: its probability buffer is free after them
        if (t > wg) take_o(own - 1);
        if (any) {  // a new reference: the maximum so far of every head
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float x = warp_max(sc[h]);
            if (lane == 0) red[ww * 8 + h] = x;
          }
          bar_wg();
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float mn = fmaxf(fmaxf(fmaxf(red[h], red[8 + h]), fmaxf(red[16 + h], red[24 + h])), m[h]);
            const float corr = mn == -INFINITY ? 0.f : exp2f(m[h] - mn);
            m[h] = mn;
            l[h] *= corr;
#pragma unroll
            for (int b = 0; b < NP; ++b) acc[b][h] *= corr;
          }
          bar_wg();
        }
        if (has) {
          char* pt = pbuf + (key >> 6) * RB + (key & 7) * 2;
          const int ch = (key & 63) >> 3;
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float p = exp2f(sc[h] - (m[h] == -INFINITY ? 0.f : m[h]));
            l[h] += p;
            __nv_bfloat16 x[3];
            split3(p, x[0], x[1], x[2]);
#pragma unroll
            for (int term = 0; term < 3; ++term) {
              const int r = term * NH + h;
              *reinterpret_cast<__nv_bfloat16*>(pt + r * 128 + ((ch ^ (r & 7)) << 4)) = x[term];
            }
          }
          if (pb >= 0 && !on) {  // a stale row of an attended page
#pragma unroll 1
            for (int j = 0; j < NP; ++j) {
              const int pc = at * PT + (own_v ? NP : 0) + j, slot = pc % kRing;
              if (own_v && !wait_bar(full0 + 8 * slot, (pc / kRing) & 1, dead, a.spin)) break;
#pragma unroll
              for (int x = 0; x < 16; ++x)
                *reinterpret_cast<uint4*>(sm + slot * LY::slot + (x >> 3) * LY::box + key * 128 + (x & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
          }
          fence_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull0 + 8 * wg);
      }
      // one query buffer: it is free once the last tile's scores are done
      if (QB == 1 && more && wg == ((nt - 1) & 1)) put_q(sn, 0);
      if (nt > wg) take_o(own - 1);
      // ---- warpgroup 0 joins the two (the other's sums come through tensor memory, where both
      // have the same lanes) and normalises, or leaves the part for k_paged_tc_join
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float x = warp_sum(l[h]);
        if (lane == 0) red[32 + ww * 8 + h] = x;
        if (wt == 0) red[64 + h] = m[h];
      }
      if (wg == 1) {
        if (nt > 1) {
#pragma unroll
          for (int b = 0; b < NP; ++b)
#pragma unroll
            for (int h = 0; h < NH; h += 4) st4(tO + b * NH + h, acc[b] + h);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        fence_before();
        asm volatile("bar.arrive 3, 256;" ::: "memory");
        asm volatile("bar.sync 4, 256;" ::: "memory");  // warpgroup 0 has read them
        tt += nt;
        ++seg;
        s = sn;
        have = more;
        continue;
      }
      asm volatile("bar.sync 3, 256;" ::: "memory");
      fence_after();
      float den[NH], f1[NH];
      const float bad = *dead ? NAN : 0.f;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float m1 = red0[72 + 64 + h], M = fmaxf(m[h], m1), ref = M == -INFINITY ? 0.f : M;
        const float f0 = exp2f(m[h] - ref);
        f1[h] = exp2f(m1 - ref);
        const float* r0 = red0 + 32 + h;
        const float* r1 = red0 + 72 + 32 + h;
        den[h] = f0 * ((r0[0] + r0[8]) + (r0[16] + r0[24])) + f1[h] * ((r1[0] + r1[8]) + (r1[16] + r1[24])) + bad;
        m[h] = M;
#pragma unroll
        for (int b = 0; b < NP; ++b) acc[b][h] *= f0;
      }
      if (nt > 1) {
#pragma unroll
        for (int b = 0; b < NP; ++b) {
          float v[NH];
#pragma unroll
          for (int h = 0; h < NH; h += 4) ld4(tO + NP * N + b * NH + h, v + h);
          ld_wait();
#pragma unroll
          for (int h = 0; h < NH; ++h) acc[b][h] = fmaf(f1[h], v[h], acc[b][h]);
        }
        fence_before();
      }
      asm volatile("bar.arrive 4, 256;" ::: "memory");
      const int h0 = s.kvh * G + s.hg * NH, nh = min(NH, G - s.hg * NH);
      const size_t row0 = static_cast<size_t>(s.b) * a.nh + h0;
      if (g.clustered) {
        // the ring is idle: every copy has landed and every product of this CTA's one segment is
        // done. (Unless a wait gave up: then the exp-sums are NaN, and no copy comes to where they are.)
        float *part = reinterpret_cast<float*>(sm), *ml = reinterpret_cast<float*>(sm + LY::p);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
          for (int b = 0; b < NP; ++b) part[h * D + b * 128 + wt] = acc[b][h];
          if (wt == 0) {
            ml[2 * h] = m[h];
            ml[2 * h + 1] = den[h];
          }
        }
        break;
      }
      const bool whole = s.a == 0 && s.e == s.n;
      {
        const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + (s.a == 0 ? 1 : 0)) * NH;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if (h >= nh) break;
          if (whole) {
            den[h] = pg::row_sum(m[h], den[h]);
            const float inv = den[h] == 0.f ? 0.f : 1.f / den[h];  // 0: nothing attended
#pragma unroll
            for (int b = 0; b < NP; ++b) a.out[(row0 + h) * D + b * 128 + wt] = acc[b][h] * inv;
            if (a.lse && wt == 0)
              a.lse[row0 + h] = den[h] == 0.f ? -INFINITY : (m[h] + log2f(den[h])) * 0.6931471805599453f;
          } else {
#pragma unroll
            for (int b = 0; b < NP; ++b) a.ws_acc[(part + h) * D + b * 128 + wt] = acc[b][h];
            if (wt == 0) {
              a.ws_ml[(part + h) * 2] = m[h];
              a.ws_ml[(part + h) * 2 + 1] = den[h];
            }
          }
        }
        if (!whole && s.a == 0 && wt == 0) {
          meta[0] = static_cast<int>(row0);
          meta[1] = nh;
          meta[2] = (s.end - 1) / per;
        }
      }
      tt += nt;
      ++seg;
      s = sn;
      have = more;
    }
    // sequences with nothing to attend have no granule: out 0, lse -inf
#pragma unroll 1
    for (int b = g.clustered ? a.B : blockIdx.x; b < a.B; b += gridDim.x) {
      int lo, hi, bs;
      if (Walk::count(g, b, lo, hi, bs) == 0) {
#pragma unroll 1
        for (int i = tid; i < a.nh * D; i += 256) a.out[static_cast<size_t>(b) * a.nh * D + i] = 0.f;
        if (a.lse)
#pragma unroll 1
          for (int i = tid; i < a.nh; i += 256) a.lse[static_cast<size_t>(b) * a.nh + i] = -INFINITY;
      }
    }
    fence_before();
  }
  __syncthreads();
  if (tid == 0 && *dead && a.status) atomicCAS(a.status, 0, static_cast<int>(MTP_ERR_TIMEOUT));
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(LY::cols) : "memory");
  }
  if (!g.clustered) return;

  // ---- the clustered form's join
  const int rank = blockIdx.x % kCluster;
  if (!work && tid < NH) {
    reinterpret_cast<float*>(sm + LY::p)[2 * tid] = -INFINITY;
    reinterpret_cast<float*>(sm + LY::p)[2 * tid + 1] = 0.f;
  }
  cluster_barrier();
  // every rank's (max, exp-sum) of every head
  float2* ml = reinterpret_cast<float2*>(sm + LY::q);
  if (tid < kCluster * NH)
    ml[tid] = make_float2(peer_f32(base + LY::p + 8 * (tid % NH), tid / NH),
                          peer_f32(base + LY::p + 8 * (tid % NH) + 4, tid / NH));
  __syncthreads();
  const int kvh = w.sub / g.ngrp, hg = w.sub - kvh * g.ngrp, nh = min(NH, G - hg * NH);
  const size_t row0 = static_cast<size_t>(w.b) * a.nh + kvh * G + hg * NH;
  const int total = nh * (D / 4), i1 = total * (rank + 1) / kCluster;
  for (int i = total * rank / kCluster + tid; i < i1; i += kThreadsTc) {
    const int h = i / (D / 4);
    float M = -INFINITY, den = 0.f;
#pragma unroll
    for (int j = 0; j < kCluster; ++j) M = fmaxf(M, ml[j * NH + h].x);
    float4 y[kCluster], x = make_float4(0, 0, 0, 0);
    float f[kCluster];
#pragma unroll
    for (int j = 0; j < kCluster; ++j) {
      f[j] = exp2f(ml[j * NH + h].x - (M == -INFINITY ? 0.f : M));
      den = fmaf(f[j], ml[j * NH + h].y, den);
      // a rank without keys has written no sums
      y[j] = ml[j * NH + h].y != 0.f ? peer_f32x4(base + 16 * i, j) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kCluster; ++j) {
      x.x = fmaf(f[j], y[j].x, x.x);
      x.y = fmaf(f[j], y[j].y, x.y);
      x.z = fmaf(f[j], y[j].z, x.z);
      x.w = fmaf(f[j], y[j].w, x.w);
    }
    den = pg::row_sum(M, den);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    reinterpret_cast<float4*>(a.out + row0 * D)[i] = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (a.lse && i % (D / 4) == 0) a.lse[row0 + h] = den == 0.f ? -INFINITY : (M + log2f(den)) * 0.6931471805599453f;
  }
  cluster_barrier();  // peers may still read this CTA's part
}

// Adds the parts of the unit that CTA blockIdx.x of k_paged_tc starts and does not end, HB heads per
// blockIdx.y, the threads over the parts and the dims; a fixed order of sums. What bounds it is its
// chain of reads (the unit, the weights, the sums: the first sums are requested with the weights)
// and the number of blocks, most of which find nothing: with a head per block at d = 128 the 61
// short sequences took 34.6 us in all, with four 32.5.
constexpr int kJoinThreads = 512;

template <int D, int HB>
__global__ void __launch_bounds__(kJoinThreads) k_paged_tc_join(const __grid_constant__ Args g, int NH) {
  pdl_enter();
  constexpr int VT = D / 4, PT = HB * VT, GR = kJoinThreads / PT, PRE = 4;  // threads of a head and a part, parts side by side
  const int4 meta = *reinterpret_cast<const int4*>(g.meta + 4 * blockIdx.x);  // first row, heads, last CTA
  const int h0 = blockIdx.y * HB, c0 = blockIdx.x;
  if (h0 >= meta.y) return;
  const int n = meta.z - c0 + 1, nh = min(HB, meta.y - h0);
  const AttArgs& a = g.a;
  __shared__ float wgt[HB][pg::kMaxSms], sden[HB], sm[HB];
  __shared__ float4 sum[GR][PT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, at = tid % PT, gr = tid / PT, h = at / VT, v = at % VT;
  // part i: slot 1 of the first CTA, slot 0 of the next ones
  auto part = [&](int i, int hh) { return static_cast<size_t>((c0 + i) * 2 + (i == 0 ? 1 : 0)) * NH + h0 + hh; };
  auto from = [&](int i) { return reinterpret_cast<const float4*>(a.ws_acc + part(i, h) * D) + v; };
  const bool on = h < nh && gr < GR;
  float4 y[PRE];
#pragma unroll
  for (int j = 0; j < PRE; ++j)
    if (on && gr + j * GR < n) y[j] = *from(gr + j * GR);
  if (warp < nh) {  // a warp per head: the weights of the parts
    float M = -INFINITY, den = 0.f;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, a.ws_ml[part(i, warp) * 2]);
    M = warp_max(M);
    for (int i = lane; i < n; i += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(a.ws_ml + part(i, warp) * 2);
      const float f = M == -INFINITY ? 0.f : exp2f(ml.x - M);
      wgt[warp][i] = f;
      den = fmaf(f, ml.y, den);
    }
    den = warp_sum(den);
    if (lane == 0) {
      sm[warp] = M;
      sden[warp] = pg::row_sum(M, den);
    }
  }
  __syncthreads();
  float4 x = make_float4(0, 0, 0, 0);
  auto add = [&](float f, const float4& z) {
    x.x = fmaf(f, z.x, x.x);
    x.y = fmaf(f, z.y, x.y);
    x.z = fmaf(f, z.z, x.z);
    x.w = fmaf(f, z.w, x.w);
  };
  if (on) {
#pragma unroll
    for (int j = 0; j < PRE; ++j)
      if (gr + j * GR < n) add(wgt[h][gr + j * GR], y[j]);
#pragma unroll 4
    for (int i = gr + PRE * GR; i < n; i += GR) add(wgt[h][i], *from(i));
  }
  if (GR > 1) {
    if (gr < GR) sum[gr][at] = x;
    __syncthreads();
    if (gr == 0) {
#pragma unroll
      for (int i = 1; i < GR; ++i) add(1.f, sum[i][at]);
    }
  }
  if (gr == 0 && on) {
    const size_t row = static_cast<size_t>(meta.x) + h0 + h;
    const float den = sden[h], inv = den == 0.f ? 0.f : 1.f / den;
    *reinterpret_cast<float4*>(a.out + row * D + 4 * v) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (a.lse && v == 0) a.lse[row] = den == 0.f ? -INFINITY : (sm[h] + log2f(den)) * 0.6931471805599453f;
  }
}

static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

int encode_map(CUtensorMap* map, const void* p, const unsigned long long* dims, const unsigned long long* strides,
               const unsigned* box_dims, const char* what) {
  cuuint64_t dim[4], str[3];
  cuuint32_t box[4];
  for (int i = 0; i < 4; ++i) {
    dim[i] = dims[i];
    box[i] = box_dims[i];
    if (i < 3) str[i] = strides[i];
  }
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  const auto encode = [&] {
    return enc ? enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dim, str, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE)
               : CUDA_ERROR_NOT_FOUND;
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    // a host thread whose first CUDA call this is: bind the device's primary context to it
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  }
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for %s", static_cast<int>(r), what);
    return MTP_ERR_CUDA;
  }
  return MTP_OK;
}

int make_map(CUtensorMap* map, const Cache& c, const void* p, int rows) {
  const unsigned long long dim[4] = {static_cast<unsigned long long>(c.d), 1ull << c.pshift,
                                     static_cast<unsigned long long>(c.nkv), static_cast<unsigned long long>(c.n_pages)};
  const unsigned long long str[3] = {2ull * c.st, 2ull * c.sh, 2ull * c.sp};
  const unsigned box[4] = {64, static_cast<unsigned>(rows), 1, 1};
  return encode_map(map, p, dim, str, box, "a paged cache");
}

// Clusters of the clustered form that the current device runs side by side (each CTA takes an SM, and
// a cluster's SMs share a GPC), asked once per device.
template <int D, int NH>
int clusters_at_once() {
  static std::atomic<int> known[64];  // 1 + the number
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreadsTc);
  cfg.dynamicSmemBytes = Lay<D, NH>::total;
  n = 0;
  if (pg::allow_smem<k_paged_tc<D, NH>, Lay<D, NH>::total>() != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k_paged_tc<D, NH>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (dev < 64) known[dev].store(n + 1);
  return n;
}

template <int D, int NH>
int launch(const Args& g, cudaStream_t st) {
  using LY = Lay<D, NH>;
  static_assert(LY::total <= 232448, "shared memory of one CTA");
  static_assert(LY::KT == 64 || LY::KT == 128, "keys per tile");
  static_assert(LY::cols <= 512 && (LY::cols & (LY::cols - 1)) == 0, "tensor memory columns");
  CUtensorMap mk, mv;
  int rc = make_map(&mk, g.a.c, g.a.c.k, 1 << g.rshift);
  if (rc) return rc;
  mv = mk;
  if (g.a.c.v && (rc = make_map(&mv, g.a.c, g.a.c.v, 1 << g.rshift))) return rc;
  cudaError_t e = pg::allow_smem<k_paged_tc<D, NH>, LY::total>();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kCluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = g.clustered ? 2 : 1;
    cfg.gridDim = dim3(g.grid);
    cfg.blockDim = dim3(kThreadsTc);
    cfg.dynamicSmemBytes = LY::total;
    cfg.stream = st;
    e = cudaLaunchKernelEx(&cfg, k_paged_tc<D, NH>, mk, mv, g);
    if (e == cudaSuccess && !g.clustered) {
      constexpr int HB = 512 / D;  // 128 threads per part
      cfg.gridDim = dim3(g.grid, NH / HB);
      cfg.blockDim = dim3(kJoinThreads);
      cfg.dynamicSmemBytes = 0;
      e = cudaLaunchKernelEx(&cfg, k_paged_tc_join<D, HB>, g, NH);
    }
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("paged attention launch: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  return MTP_OK;
}

}  // namespace pgt

static int clusters_fit(int d, int NH) {
  if (NH == 4) return d == 128 ? pgt::clusters_at_once<128, 4>() : d == 256 ? pgt::clusters_at_once<256, 4>() : pgt::clusters_at_once<512, 4>();
  return d == 128 ? pgt::clusters_at_once<128, 8>() : d == 256 ? pgt::clusters_at_once<256, 8>() : pgt::clusters_at_once<512, 8>();
}

// The tensor-core kernel serves bf16 caches of head_dim 128, 256 or 512 (128-dim MMA rows) with
// pages of at least 8 tokens (one swizzle block) whose strides fit a tensor map.
bool paged_tc_supported(const pg::Cache& c) {
  const long long most = (1LL << 40) / 2 - 8;
  return !c.f32 && (c.d == 128 || c.d == 256 || c.d == 512) && c.pshift >= 3 && c.sp <= most && c.st <= most && c.sh <= most;
}

long long paged_tc_workspace(const pg::Cache& c) {
  return pg::kMaxSms * (16LL + 2 * 8 * (static_cast<long long>(c.d) + 2) * 4);
}

int run_paged_tc(const pg::AttArgs& a, void* ws, int num_sms, cudaStream_t st) {
  using namespace pgt;
  Args g;
  memset(&g, 0, sizeof(g));
  g.a = a;
  const int P = 1 << a.c.pshift, G = a.nh / a.c.nkv, NH = G <= 4 ? 4 : 8;
  const int tile = a.c.d == 512 || (a.c.d == 256 && NH == 8) ? 64 : 128;  // Lay::KT
  const int rows = P < tile ? P : tile;
  while ((1 << g.rshift) < rows) ++g.rshift;
  g.ngrp = (G + NH - 1) / NH;
  // the most keys a unit can have; with few of them, smaller granules spread them over the SMs
  long long keys = static_cast<long long>(a.list ? a.n_list : a.c.max_pages) * P;
  if (!a.list && a.window > 0 && static_cast<long long>(a.window) + rows < keys) keys = a.window + rows;
  const long long units = static_cast<long long>(a.B) * a.c.nkv * g.ngrp;
  // a cluster per unit where they fit side by side and a CTA's share of the longest unit is at most
  // kClusterBytes: with one launch less 7 us against 9 for 512 keys at d = 256, level at 2048 keys
  // at d = 512 (256 KB); in two waves of clusters 14 us against 10
  const long long unit_bytes = keys * a.c.d * (a.c.v ? 4 : 2);
  g.clustered = units * kCluster <= num_sms && unit_bytes <= static_cast<long long>(kCluster) * kClusterBytes &&
                units <= clusters_fit(a.c.d, NH);
  g.gshift = a.c.d == 512 ? 6 : 7;
  const auto granules = [&] { return units * ((keys + (1 << g.gshift) - 1) >> g.gshift); };
  while (g.gshift > 5 && (1 << g.gshift) > rows && (granules() < num_sms || g.clustered)) --g.gshift;
  const long long most = granules();
  // beginning a unit, in the time of so many bytes loaded (longer with one query buffer)
  const int begin = a.c.d == 512 ? 128 * 1024 : 64 * 1024, bytes = (a.c.d * (a.c.v ? 4 : 2)) << g.gshift;
  g.extra = most > num_sms && !g.clustered ? (begin + bytes - 1) / bytes : 0;
  if (most + units * g.extra > INT32_MAX - pg::kMaxSms) {
    set_error("too many keys: B * heads * max_pages * page_size = %lld", units * keys);
    return MTP_ERR_UNSUPPORTED_SHAPE;
  }
  g.grid = g.clustered ? static_cast<int>(units) * kCluster : static_cast<int>(most < num_sms ? most : num_sms);
  g.meta = static_cast<int*>(ws);
  g.a.ws_ml = reinterpret_cast<float*>(g.meta + 4 * pg::kMaxSms);
  g.a.ws_acc = g.a.ws_ml + pg::kMaxSms * 2 * 8 * 2;
  if (NH == 4) {
    if (a.c.d == 128) return launch<128, 4>(g, st);
    return a.c.d == 256 ? launch<256, 4>(g, st) : launch<512, 4>(g, st);
  }
  if (a.c.d == 128) return launch<128, 8>(g, st);
  return a.c.d == 256 ? launch<256, 8>(g, st) : launch<512, 8>(g, st);
}

}  // namespace mtp
