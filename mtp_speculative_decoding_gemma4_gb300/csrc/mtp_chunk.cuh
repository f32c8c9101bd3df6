// How the tensor-core attention of a chunk deals its work: units (a tile of query rows of one KV
// head), each a run of key tiles, numbered through and dealt evenly over the CTAs.
#pragma once

#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

// The new tokens of one sequence as tiles of `tpt` tokens (a power of two): tile i's last token
// attends the keys below end(i), its first one those from begin(i) on. Key tiles are 2^ks keys, at
// multiples of 2^ks. The cost of a unit is its key tiles and `extra` for its beginning; the sums of
// costs have closed forms, so that any CTA finds its place without a pass over the tiles.
struct Tiles {
  int n, first, L, window, tpt, ks, extra;

  __host__ __device__ int count() const { return (n + tpt - 1) / tpt; }
  __host__ __device__ long long pos(int i) const { return static_cast<long long>(first) + static_cast<long long>(i) * tpt; }
  __host__ __device__ int end(int i) const {
    const long long e = i + 1 < count() ? pos(i + 1) : L;
    return e > 0 ? static_cast<int>(e) : 0;
  }
  __host__ __device__ int begin(int i) const {
    const long long b = window > 0 ? pos(i) - window + 1 : 0;
    return b > 0 ? static_cast<int>(b) : 0;
  }
  __host__ __device__ int tiles(int i) const {
    const int k = ((end(i) + (1 << ks) - 1) >> ks) - (begin(i) >> ks);
    return k > 0 ? k : 0;
  }
  // sum over j < y of floor(j / c)
  __host__ __device__ static long long steps(long long y, long long c) {
    const long long u = y / c, v = y % c;
    return c * (u * (u - 1) / 2) + u * v;
  }
  // sum over i < k of floor((a + i tpt) / 2^ks), a >= 0
  __host__ __device__ long long floors(long long a, long long k) const {
    const int K = 1 << ks;
    if (tpt >= K) return k * (a >> ks) + static_cast<long long>(tpt >> ks) * (k * (k - 1) / 2);
    const long long q = a / tpt, c = K / tpt;  // tpt divides K: floor((a + i tpt) / K) = floor((q + i) / c)
    return steps(q + k, c) - steps(q, c);
  }
  // cost of the first `i` tiles
  __host__ __device__ long long cost(int i) const {
    const int K = 1 << ks, nt = count();
    long long sum = static_cast<long long>(extra) * i;
    const int inner = i < nt ? i : nt - 1;  // tiles that end at the next one's first token
    const int skip = first < 0 ? static_cast<int>(-static_cast<long long>(first) / tpt) : 0;  // those end at or before 0
    if (inner > skip) sum += floors(pos(skip + 1) + K - 1, inner - skip);
    if (i >= nt && nt > 0) sum += (end(nt - 1) + K - 1) >> ks;
    if (window > 0) {
      const long long c = static_cast<long long>(first) - window + 1;
      const long long j = c < 0 ? (-c + tpt - 1) / tpt : 0;  // tiles that begin at key 0
      if (i > j) sum -= floors(c + j * tpt, i - j);
    }
    return sum;
  }
};

}  // namespace pg
}  // namespace mtp
