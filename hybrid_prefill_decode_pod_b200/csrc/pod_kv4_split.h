// pod_kv4_split.h -- how a decode call's work is cut, shared by the kernel and
// the host tests.
//
// The W = Hk * sum(blocks) blocks of 16 tokens, in the order (request, KV head,
// block), are one line; a (request, KV head) is a segment of it. N workers cut
// the line into parts of equal cost: a segment of n blocks costs what its tiles
// of four blocks cost and kv4_start blocks more for its queries and its end. The
// cuts are therefore made on a second line, of costs, on which worker c takes
// [c V / N, (c + 1) V / N), and carried over to the blocks.
//
// A segment may lie in several workers. Where all segments are short the cuts
// move to the next boundary between two, so that none does; a worker may then
// have no block.
#pragma once

namespace pod {

#ifdef __CUDACC__
#define POD_HD __host__ __device__ __forceinline__
#else
#define POD_HD inline
#endif

// a / b, both not negative: a 32-bit division takes a third of the time
POD_HD long long kv4_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// What a segment of n blocks costs: its tiles, and `start` before them.
constexpr int kKv4Start = 4;
POD_HD int kv4_cost(int n) { return n ? ((n + 3) & ~3) + kKv4Start : 0; }

POD_HD long long kv4_begin(long long V, int N, int c) { return kv4_div(c * V, N); }

// Where x of a line lies: first[r] is the length of one head of the requests in
// front of r (first[R] of all), 0 <= x < Hk * first[R].
struct Kv4Place {
  int r, h, blk, nblk;
};
POD_HD Kv4Place kv4_place(const int* first, int R, int Hk, long long x) {
  const int v = (int)kv4_div(x, Hk);
  int lo = 0, hi = R;  // first[lo] <= v < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  Kv4Place p;
  p.r = lo;
  p.nblk = first[lo + 1] - first[lo];
  const long long rem = x - (long long)Hk * first[lo];
  p.h = (int)kv4_div(rem, p.nblk);
  p.blk = (int)(rem - (long long)p.h * p.nblk);
  return p;
}

// The segment boundary next to v on the line of costs, 0 <= v <= Hk * cost[R].
POD_HD long long kv4_snap(const int* cost, int R, int Hk, long long v) {
  if (v >= (long long)Hk * cost[R]) return (long long)Hk * cost[R];
  const Kv4Place p = kv4_place(cost, R, Hk, v);
  return 2 * p.blk <= p.nblk ? v - p.blk : v + (p.nblk - p.blk);
}

// The first block behind the cut at v of the line of costs. first and cost: blocks
// and costs of one head in front of each request.
POD_HD long long kv4_cut(const int* first, const int* cost, int R, int Hk, long long v) {
  if (v >= (long long)Hk * cost[R]) return (long long)Hk * first[R];
  const Kv4Place p = kv4_place(cost, R, Hk, v);
  const int n = first[p.r + 1] - first[p.r], blk = p.blk - kKv4Start;
  return (long long)Hk * first[p.r] + (long long)p.h * n + (blk < 0 ? 0 : blk > n ? n : blk);
}

// The worker that holds block blk of (r, h), where cuts are not moved.
POD_HD int kv4_worker(const int* cost, int R, int Hk, int N, int r, int h, int blk) {
  const long long V = (long long)Hk * cost[R];
  const long long v = (long long)Hk * cost[r] + (long long)h * (cost[r + 1] - cost[r]) + kKv4Start + blk;
  return (int)kv4_div((v + 1) * N - 1, V);
}

// Workers of a call: no more than there are CTAs, each with at least
// `least` blocks (one worker where there are fewer).
POD_HD int kv4_workers(long long W, int ctas, int least) {
  const long long n = W / least;
  return n < 1 ? 1 : n < ctas ? (int)n : ctas;
}

}  // namespace pod
