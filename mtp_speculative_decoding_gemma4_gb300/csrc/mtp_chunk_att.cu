// Attention of a chunk of new tokens over a paged key cache: the last n_b tokens of sequence b are
// new, token i of them (position t = ctx_len[b] - n_b + i) attends the keys j <= t, j > t - window:
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j),  lse = log sum_j exp(scale q . k_j),
// in one pass over the keys with a running maximum and sum per query row.
//
// This file: the CUDA-core kernel for every dtype and head dim, and the join of the splits. A tile
// is R = 16 RI rows (the query heads of one KV head for R / G tokens), a CTA of 256 threads takes 64
// keys at a time: scores by 4 RI values per thread from shared memory (dims in blocks of 64, the
// next block's global loads in flight), then the sums, RI rows x 4 dims per block of 64 and thread; with
// few rows (RI = 1) a warp takes two of them, so that a vector of shared memory serves more products.
// What bounds it is the fp32 pipes where rows are many (RI = 4: 16 products per two shared-memory
// vectors), shared memory and latency where they are few (16 fp32 contexts to 4000 keys, up to 17 tokens
// of 4 heads on 2, d = 64: 46 us, of which the join 4; 66 with one row and one key vector at a time); a
// unit's keys are split over CTAs while the GPU has room.
#include "mtp_common.cuh"
#include "mtp_launch.h"
#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

namespace {

constexpr int kTokThreads = 256;
constexpr int kKeys = 64;          // keys of a step
constexpr int kPad = 68;           // floats between rows of 64 in shared memory
constexpr int kMaxChunkSplits = 64;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  __device__ static void get(const float* p, float* v) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
  }
  __device__ static void put(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static void get(const __nv_bfloat16* p, float* v) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void put(__nv_bfloat16* p, float a, float b, float c, float d) {
    __nv_bfloat162 x[2] = {__floats2bfloat162_rn(a, b), __floats2bfloat162_rn(c, d)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(x);
  }
};

__device__ __forceinline__ float pexp(float x, float m) { return exp2f(x - (m == -INFINITY ? 0.f : m)); }

// The tile that slot i of the grid stands for. Sequence b's tiles of `tpt` tokens begin at slot
// cu[b] / tpt + b, which leaves room for each of them whatever the lengths (floor((c + n) / t) + 1 -
// floor(c / t) >= ceil(n / t)); slots between are empty.
__device__ __forceinline__ bool find_tile(const ChunkArgs& a, int slot, int tpt, int& b, int& tile) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (min(max(a.cu[mid], 0), a.T) / tpt + mid <= slot) lo = mid; else hi = mid - 1;
  }
  b = lo;
  const int s0 = min(max(a.cu[b], 0), a.T);
  tile = slot - (s0 / tpt + b);
  return tile >= 0;
}

// (d <= 128: two CTAs per SM; without the bound 2048 fp32 rows of d = 128 take 110 us instead of 92, and with
// it for all d the registers of the others grow until one CTA fits)
template <typename T, int DC, int RI>
__global__ void __launch_bounds__(kTokThreads, DC <= 2 ? 2 : 0) k_chunk(const __grid_constant__ ChunkArgs a) {
  pdl_enter();
  constexpr int R = 16 * RI, D = 64 * DC, QP = D + 4, VE = Vec<T>::n, LV = kKeys * 64 / VE / kTokThreads;
  constexpr int KP = RI == 1 ? 80 : kPad;  // floats between keys
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                 // [R][QP]
  float* sk = sq + R * QP;        // [64 keys][KP]: 64 dims of keys or values
  float* sp = sk + kKeys * KP;    // [R][kPad] scores, probabilities
  __shared__ long long s_at[kKeys];  // a key's row in the cache, -1: no row that any query may read
  __shared__ int s_bad[kKeys], s_any;
  const Cache& c = a.c;
  const int d = c.d, G = a.nh / c.nkv, hgs = (G + R - 1) / R;
  const int tpt = G <= R ? R / G : 1;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  int b, tile;
  if (!find_tile(a, blockIdx.x, tpt, b, tile)) return;
  const int g = blockIdx.y / hgs, hg = blockIdx.y - g * hgs, Gc = min(R, G - hg * R);
  int s0, n, first, L;
  chunk_range(a, b, s0, n, first, L);
  const int t0 = tile * tpt, nt = min(tpt, n - t0);  // tokens [t0, t0 + nt) of the sequence's new ones
  if (nt <= 0) return;
  const int nr = nt * Gc;  // rows: token-major, head within
  const int pos0 = first + t0;
  const int hi = min(max(pos0 + nt, 0), L), lo = a.window > 0 ? max(0, pos0 - a.window + 1) : 0;
  const int steps = hi > lo ? (hi - lo + kKeys - 1) / kKeys : 0;
  const int per = (steps + a.nsplit - 1) / a.nsplit, z0 = min(steps, static_cast<int>(blockIdx.z) * per),
            z1 = min(steps, z0 + per);

  auto q_row = [&](int r) { return static_cast<size_t>(s0 + t0 + r / Gc); };
  auto head = [&](int r) { return g * G + hg * R + r % Gc; };
  for (int i = tid; i < R * (D / VE); i += kTokThreads) {
    const int r = i / (D / VE), v = i % (D / VE) * VE;
    float x[VE];
    if (r < nr && v < d) {
      Vec<T>::get(static_cast<const T*>(a.q) + q_row(r) * a.q_stride + static_cast<size_t>(head(r)) * d + v, x);
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) sq[r * QP + v + e] = x[e];
  }
  // RI = 4: rows ty + 16 i, scores with keys tx + 16 j, sums of dims 4 tx ..
  // RI = 1: a warp for two rows. Scores: both rows, keys kq + 8 j, every fourth vector of the dims, then
  // added up so that a thread has 4 scores of row `mine`; sums: both rows, dims 4 tx .., every other key
  constexpr int RA = RI == 1 ? 2 : RI;  // rows of a thread's sums
  const int warp = tid >> 5, lane = tid & 31, dg = lane & 3, kq = lane >> 2, kh = lane >> 4;
  const int mine = 2 * warp + (dg >> 1);
  auto row_of = [&](int i) { return RI == 1 ? mine : ty + 16 * i; };                                  // of m, l and scores
  auto key_of = [&](int j) { return RI == 1 ? kq + 8 * (4 * (dg & 1) + j) : tx + 16 * j; };
  float acc[RA][4 * DC], m[RI], l[RI];
  int qpos[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    const int r = row_of(i);
    qpos[i] = r < nr ? pos0 + r / Gc : -1;  // -1: a row of no token attends nothing
  }
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int e = 0; e < 4 * DC; ++e) acc[i][e] = 0.f;
  // one block of 64 dims of 64 rows: into registers, then into shared memory
  float buf[LV][VE];
  auto fetch = [&](const void* from, int dim0) {
#pragma unroll
    for (int j = 0; j < LV; ++j) {
      const int i = tid + j * kTokThreads, key = i / (64 / VE), v = dim0 + i % (64 / VE) * VE;
      const long long at = s_at[key];
      if (at >= 0 && v < d) {
        Vec<T>::get(static_cast<const T*>(from) + at + v, buf[j]);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) buf[j][e] = 0.f;
      }
    }
  };
  // clean: values that are not finite become 0 and mark their key (a query that does not attend
  // the key would get 0 * NaN)
  auto stage = [&](bool clean) {
#pragma unroll
    for (int j = 0; j < LV; ++j) {
      const int i = tid + j * kTokThreads, key = i / (64 / VE), v = i % (64 / VE) * VE;
      if (clean) {
        bool bad = false;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (!isfinite(buf[j][e])) {
            buf[j][e] = 0.f;
            bad = true;
          }
        if (bad) s_bad[key] = s_any = 1;
      }
#pragma unroll
      for (int e = 0; e < VE; e += 4)
        *reinterpret_cast<float4*>(sk + key * KP + v + e) = make_float4(buf[j][e], buf[j][e + 1], buf[j][e + 2], buf[j][e + 3]);
    }
  };
  const void* vals = c.v ? c.v : c.k;
  for (int z = z0; z < z1; ++z) {
    const int k0 = lo + z * kKeys;
    __syncthreads();  // the last step's reads of s_at, sk and sp are done
    if (tid < kKeys) {
      const int pos = k0 + tid;
      long long at = -1;
      if (pos < hi) {
        const int page = phys_page(c, b, pos >> c.pshift);
        if (page >= 0) at = page * c.sp + (pos & ((1 << c.pshift) - 1)) * c.st + g * c.sh;
      }
      s_at[tid] = at;
      s_bad[tid] = 0;
      if (tid == 0) s_any = 0;
    }
    __syncthreads();
    fetch(c.k, 0);
    float s[RI == 1 ? 4 : RI][4];  // RI = 1: s[2 row + half of the keys][..]
#pragma unroll
    for (int i = 0; i < (RI == 1 ? 4 : RI); ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 1
    for (int x = 0; x < DC; ++x) {
      stage(false);
      __syncthreads();
      if (x + 1 < DC) fetch(c.k, 64 * (x + 1));
      if constexpr (RI == 1) {
#pragma unroll
        for (int e = 4 * dg, n = 0; n < 4; ++n, e += 16) {
          const float4 q0 = *reinterpret_cast<const float4*>(sq + 2 * warp * QP + 64 * x + e),
                       q1 = *reinterpret_cast<const float4*>(sq + (2 * warp + 1) * QP + 64 * x + e);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 kv = *reinterpret_cast<const float4*>(sk + (kq + 8 * j) * KP + e);
            float &a0 = s[j >> 2][j & 3], &a1 = s[2 + (j >> 2)][j & 3];
            a0 = fmaf(q0.x, kv.x, fmaf(q0.y, kv.y, fmaf(q0.z, kv.z, fmaf(q0.w, kv.w, a0))));
            a1 = fmaf(q1.x, kv.x, fmaf(q1.y, kv.y, fmaf(q1.z, kv.z, fmaf(q1.w, kv.w, a1))));
          }
        }
      } else {
#pragma unroll 4
        for (int e = 0; e < 64; e += 4) {
          float4 kv[4], qv;
#pragma unroll
          for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * KP + e);
#pragma unroll
          for (int i = 0; i < RI; ++i) {
            qv = *reinterpret_cast<const float4*>(sq + (ty + 16 * i) * QP + 64 * x + e);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              s[i][j] = fmaf(qv.x, kv[j].x, fmaf(qv.y, kv[j].y, fmaf(qv.z, kv[j].z, fmaf(qv.w, kv[j].w, s[i][j]))));
          }
        }
      }
      if (x + 1 < DC) __syncthreads();
    }
    fetch(vals, 0);
    if constexpr (RI == 1) {  // over the four groups of dims: the row, then the half of the keys
      const bool r1 = dg & 2, k1 = dg & 1;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = (r1 ? s[2 + i][j] : s[i][j]) + __shfl_xor_sync(0xffffffffu, r1 ? s[i][j] : s[2 + i][j], 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[0][j] = (k1 ? s[1][j] : s[0][j]) + __shfl_xor_sync(0xffffffffu, k1 ? s[0][j] : s[1][j], 1);
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key_of(j), pos = k0 + key;
        const bool on = pos <= qpos[i] && s_at[key] >= 0 && (a.window <= 0 || pos > qpos[i] - a.window);
        s[i][j] = on ? attended(s[i][j] * a.scale_log2) : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int o = 1; o < (RI == 1 ? 32 : 16); o <<= 1)
        if (RI != 1 || o != 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(m[i], mx);
      const float corr = pexp(m[i], mx);
      m[i] = mx;
      l[i] *= corr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = pexp(s[i][j], mx);
        l[i] += p;
        sp[row_of(i) * kPad + key_of(j)] = p;
      }
      if constexpr (RI == 1) {
        const float c0 = __shfl_sync(0xffffffffu, corr, 0), c1 = __shfl_sync(0xffffffffu, corr, 2);
        if (c0 != 1.f || c1 != 1.f) {
#pragma unroll
          for (int e = 0; e < 4 * DC; ++e) {
            acc[0][e] *= c0;
            acc[RA - 1][e] *= c1;
          }
        }
      } else if (corr != 1.f) {
#pragma unroll
        for (int e = 0; e < 4 * DC; ++e) acc[i][e] *= corr;
      }
    }
    __syncthreads();  // scores are done with sk
#pragma unroll
    for (int x = 0; x < DC; ++x) {
      stage(true);
      __syncthreads();
      if (x + 1 < DC) fetch(vals, 64 * (x + 1));
#pragma unroll 2
      for (int key = RI == 1 ? 4 * kh : 0; key < kKeys; key += RI == 1 ? 8 : 4) {
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float4*>(sk + (key + j) * KP + 4 * tx);
#pragma unroll
        for (int i = 0; i < RA; ++i) {
          const float4 p = *reinterpret_cast<const float4*>(sp + (RI == 1 ? 2 * warp + i : ty + 16 * i) * kPad + key);
          float* o = acc[i] + 4 * x;
          o[0] = fmaf(p.x, v[0].x, fmaf(p.y, v[1].x, fmaf(p.z, v[2].x, fmaf(p.w, v[3].x, o[0]))));
          o[1] = fmaf(p.x, v[0].y, fmaf(p.y, v[1].y, fmaf(p.z, v[2].y, fmaf(p.w, v[3].y, o[1]))));
          o[2] = fmaf(p.x, v[0].z, fmaf(p.y, v[1].z, fmaf(p.z, v[2].z, fmaf(p.w, v[3].z, o[2]))));
          o[3] = fmaf(p.x, v[0].w, fmaf(p.y, v[1].w, fmaf(p.z, v[2].w, fmaf(p.w, v[3].w, o[3]))));
        }
      }
      if (x + 1 < DC) __syncthreads();
    }
    if (s_any) {  // rows that attend a value that is not finite, whatever its weight (V = K: but for scores of -inf)
#pragma unroll 1
      for (int key = 0; key < kKeys; ++key)
        if (s_bad[key]) {
          const int pos = k0 + key;
#pragma unroll
          for (int i = 0; i < RI; ++i)
            if (c.v ? pos <= qpos[i] && (a.window <= 0 || pos > qpos[i] - a.window) : sp[row_of(i) * kPad + key] != 0.f)
              l[i] = NAN;
        }
    }
  }
  if constexpr (RI == 1) {  // the halves of the keys; then a half of the warp keeps one row
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (o != 2) l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
    l[0] = __shfl_sync(0xffffffffu, l[0], 2 * kh);
    m[0] = __shfl_sync(0xffffffffu, m[0], 2 * kh);
#pragma unroll
    for (int e = 0; e < 4 * DC; ++e)
      acc[0][e] = (kh ? acc[RA - 1][e] : acc[0][e]) + __shfl_xor_sync(0xffffffffu, kh ? acc[0][e] : acc[RA - 1][e], 16);
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    if constexpr (RI != 1) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    }
    const int r = RI == 1 ? 2 * warp + kh : ty + 16 * i;
    if (r >= nr) continue;
    const size_t row = q_row(r) * a.nh + head(r);
    if (a.nsplit == 1) {
      const float den = row_sum(m[i], l[i]), inv = den == 0.f ? 0.f : 1.f / den;  // 0: nothing attended
#pragma unroll
      for (int x = 0; x < DC; ++x) {
        const float* o = acc[i] + 4 * x;
        if (64 * x + 4 * tx < d)
          Vec<T>::put(static_cast<T*>(a.out) + row * d + 64 * x + 4 * tx, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
      }
      if (a.lse && tx == 0) a.lse[row] = den == 0.f ? -INFINITY : (m[i] + log2f(den)) * 0.6931471805599453f;
    } else {
      const size_t part = row * a.nsplit + blockIdx.z;
#pragma unroll
      for (int x = 0; x < DC; ++x) {
        const float* o = acc[i] + 4 * x;
        if (64 * x + 4 * tx < d)
          *reinterpret_cast<float4*>(a.ws_acc + part * d + 64 * x + 4 * tx) = make_float4(o[0], o[1], o[2], o[3]);
      }
      if (tx == 0) {
        a.ws_ml[2 * part] = m[i];
        a.ws_ml[2 * part + 1] = l[i];
      }
    }
  }
}

// Joins the splits of a (token, head) per warp, in split order: a lane keeps up to two of the
// weights and 4 dims per step.
template <typename T>
__global__ void __launch_bounds__(256) k_chunk_join(const __grid_constant__ ChunkArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31, n = a.nsplit, d = a.c.d;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t0 = min(max(a.cu[0], 0), a.T), t1 = min(max(a.cu[a.B], 0), a.T);
  if (row < static_cast<long long>(t0) * a.nh || row >= static_cast<long long>(t1) * a.nh) return;
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row * n;
  float2 x[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) x[j] = lane + 32 * j < n ? ml[lane + 32 * j] : make_float2(-INFINITY, 0.f);
  const float M = warp_max(fmaxf(x[0].x, x[1].x));
  float w[2], den = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] = pexp(x[j].x, M);
    den = fmaf(w[j], x[j].y, den);
  }
  den = row_sum(M, warp_sum(den));
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const float* acc = a.ws_acc + row * n * d;
  for (int v0 = 0; v0 < d; v0 += 128) {
    const int v = v0 + 4 * lane;
    float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float f = __shfl_sync(0xffffffffu, i < 32 ? w[0] : w[1], i & 31);
      if (v < d) {
        const float4 y = *reinterpret_cast<const float4*>(acc + static_cast<long long>(i) * d + v);
        s.x = fmaf(f, y.x, s.x);
        s.y = fmaf(f, y.y, s.y);
        s.z = fmaf(f, y.z, s.z);
        s.w = fmaf(f, y.w, s.w);
      }
    }
    if (v < d) Vec<T>::put(static_cast<T*>(a.out) + row * d + v, s.x * inv, s.y * inv, s.z * inv, s.w * inv);
  }
  if (a.lse && lane == 0) a.lse[row] = den == 0.f ? -INFINITY : (M + log2f(den)) * 0.6931471805599453f;
}

// Rows of a tile: 16 where the sequences have at most 32 rows on average, else 64. 16 fp32 contexts of 2000
// keys, with 16 and with 64 rows, us: 16 rows each, d = 64 26 and 34, d = 512 111 and 192; 32 rows each, d =
// 64 33 and 36, 128 47 and 52, 256 80 and 107, 512 183 and 202; 48 rows each, 41 and 38, 62 and 53, 107 and
// 112, 251 and 212. 64 as well where a grid has fewer rows than there would be groups of 16 heads.
int rows_of(const ChunkArgs& a) {
  const int G = a.nh / a.c.nkv;
  if (a.c.nkv * ((G + 15) / 16) > 65535) return 64;
  return static_cast<long long>(a.T) * G <= 32LL * a.B ? 16 : 64;
}

long long slots_of(const ChunkArgs& a, int R) {
  const int G = a.nh / a.c.nkv, tpt = G <= R ? R / G : 1;
  return a.T / tpt + a.B;
}

// Splits of a tile's keys: about 8 CTAs per SM over the call (sequences are not equally long), at least
// 64 keys each.
int choose_chunk_splits(const ChunkArgs& a, int R, int window, int num_sms) {
  const int G = a.nh / a.c.nkv;
  const long long units = slots_of(a, R) * a.c.nkv * ((G + R - 1) / R);
  long long keys = static_cast<long long>(a.c.max_pages) << a.c.pshift;
  if (window > 0 && static_cast<long long>(window) + R < keys) keys = window + R;
  long long n = 8LL * num_sms / units;
  if (n > keys / 64) n = keys / 64;
  if (n > kMaxChunkSplits) n = kMaxChunkSplits;
  return n < 1 ? 1 : static_cast<int>(n);
}

template <typename T, int DC, int RI>
int launch_chunk(const ChunkArgs& a, cudaStream_t st) {
  constexpr int R = 16 * RI, smem = (R * (64 * DC + 4) + kKeys * (RI == 1 ? 80 : kPad) + R * kPad) * 4;
  static_assert(smem <= 232448 - 1024, "shared memory of one CTA");
  const cudaError_t e = allow_smem<k_chunk<T, DC, RI>, smem>();
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("chunk attention: %s", cudaGetErrorString(e));
    return MTP_ERR_CUDA;
  }
  const int G = a.nh / a.c.nkv;
  return launch_pdl("chunk attention", k_chunk<T, DC, RI>,
                    dim3(static_cast<unsigned>(slots_of(a, R)), a.c.nkv * ((G + R - 1) / R), a.nsplit), kTokThreads, smem, st, a);
}

template <typename T>
int launch_dims(const ChunkArgs& a, int R, cudaStream_t st) {
  const int dc = (a.c.d + 63) / 64;
  if (R == 16) {
    if (dc <= 1) return launch_chunk<T, 1, 1>(a, st);
    if (dc <= 2) return launch_chunk<T, 2, 1>(a, st);
    return dc <= 4 ? launch_chunk<T, 4, 1>(a, st) : launch_chunk<T, 8, 1>(a, st);
  }
  if (dc <= 1) return launch_chunk<T, 1, 4>(a, st);
  if (dc <= 2) return launch_chunk<T, 2, 4>(a, st);
  return dc <= 4 ? launch_chunk<T, 4, 4>(a, st) : launch_chunk<T, 8, 4>(a, st);
}

}  // namespace

}  // namespace pg

long long chunk_att_workspace(const pg::ChunkArgs& a) {
  if (paged_tc_supported(a.c)) return chunk_tc_workspace(a);
  // a window only shortens the key range and fewer SMs take fewer splits, so this is a bound
  const long long n = pg::choose_chunk_splits(a, pg::rows_of(a), 0, pg::kMaxSms);
  return n > 1 ? static_cast<long long>(a.T) * a.nh * n * (a.c.d + 2) * 4 : 0;
}

int run_chunk_att(pg::ChunkArgs a, void* ws, int num_sms, cudaStream_t st) {
  if (paged_tc_supported(a.c)) return run_chunk_tc(a, ws, num_sms, st);
  const int R = pg::rows_of(a);
  a.nsplit = pg::choose_chunk_splits(a, R, a.window, num_sms);
  a.ws_acc = static_cast<float*>(ws);
  a.ws_ml = a.ws_acc + static_cast<size_t>(a.T) * a.nh * a.nsplit * a.c.d;
  const int rc = a.c.f32 ? pg::launch_dims<float>(a, R, st) : pg::launch_dims<__nv_bfloat16>(a, R, st);
  if (rc || a.nsplit == 1) return rc;
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.T) * a.nh + 7) / 8));
  return a.c.f32 ? pg::launch_pdl("chunk attention join", pg::k_chunk_join<float>, grid, 256, 0, st, a)
                 : pg::launch_pdl("chunk attention join", pg::k_chunk_join<__nv_bfloat16>, grid, 256, 0, st, a);
}

}  // namespace mtp
