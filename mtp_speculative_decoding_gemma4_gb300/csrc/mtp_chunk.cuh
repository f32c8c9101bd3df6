// How the tensor-core attention of a chunk deals its work: units (a tile of query rows of one KV
// head), each a run of key tiles, numbered through and dealt evenly over the CTAs.
#pragma once

#include "mtp_paged.cuh"

namespace mtp {
namespace pg {

// The new tokens of one sequence as tiles of 2^ts tokens: tile i's last token
// attends the keys below end(i), its first one those from begin(i) on. Key tiles are 2^ks keys, at
// multiples of 2^ks. The cost of a unit is its key tiles and `extra` for its beginning; the sums of
// costs have closed forms, so that any CTA finds its place without a pass over the tiles.
struct Tiles {
  int n, first, L, window, ts, ks, extra;

  __host__ __device__ int count() const { return (n + (1 << ts) - 1) >> ts; }
  __host__ __device__ long long pos(int i) const { return first + (static_cast<long long>(i) << ts); }
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
  // sum over j < y of floor(j / 2^s)
  __host__ __device__ static long long steps(long long y, int s) {
    const long long u = y >> s, v = y & ((1 << s) - 1);
    return ((u * (u - 1) >> 1) << s) + u * v;
  }
  // sum over i < k of floor((a + i 2^ts) / 2^ks), a >= 0
  __host__ __device__ long long floors(long long a, long long k) const {
    if (ts >= ks) return k * (a >> ks) + ((k * (k - 1) >> 1) << (ts - ks));
    const long long q = a >> ts;  // floor((a + i 2^ts) / 2^ks) = floor((q + i) / 2^(ks - ts))
    return steps(q + k, ks - ts) - steps(q, ks - ts);
  }
  // cost of the first `i` tiles
  __host__ __device__ long long cost(int i) const {
    const int K = 1 << ks, nt = count();
    long long sum = static_cast<long long>(extra) * i;
    const int inner = i < nt ? i : nt - 1;  // tiles that end at the next one's first token
    const int skip = first < 0 ? static_cast<int>(-static_cast<long long>(first) >> ts) : 0;  // those end at or before 0
    if (inner > skip) sum += floors(pos(skip + 1) + K - 1, inner - skip);
    if (i >= nt && nt > 0) sum += (end(nt - 1) + K - 1) >> ks;
    if (window > 0) {
      const long long c = static_cast<long long>(first) - window + 1;
      const long long j = c < 0 ? (-c + (1 << ts) - 1) >> ts : 0;  // tiles that begin at key 0
      if (i > j) sum -= floors(c + (j << ts), i - j);
    }
    return sum;
  }
};

}  // namespace pg
}  // namespace mtp
