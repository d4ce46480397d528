// pod_kv4_split.h -- how a decode call's work is cut, shared by the kernel and
// the host tests.
//
// The W = Hk * sum(blocks) blocks of 16 tokens, in the order (request, KV head,
// block), are one line that N workers cut into equal lengths: worker c takes
// [c W / N, (c + 1) W / N). A (request, KV head) is a segment of that line and
// may lie in several workers. With N <= W every worker has a block. Where all
// segments are short the cuts move to the next boundary between two, so that no
// segment lies in several workers; a worker may then have none.
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
POD_HD long long kv4_begin(long long W, int N, int c) { return kv4_div(c * W, N); }

// The worker that holds block x: the largest c with c W / N <= x.
POD_HD int kv4_worker(long long W, int N, long long x) {
  return (int)kv4_div((x + 1) * N - 1, W);
}

// Where block x of the line lies: first[r] is the number of blocks of one head
// in front of request r (first[R] their sum), 0 <= x < Hk * first[R].
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

// The segment boundary next to x, 0 <= x <= W.
POD_HD long long kv4_snap(const int* first, int R, int Hk, long long W, long long x) {
  if (x >= W) return W;
  const Kv4Place p = kv4_place(first, R, Hk, x);
  return 2 * p.blk <= p.nblk ? x - p.blk : x + (p.nblk - p.blk);
}

// Workers of a call: no more than there are CTAs, each with at least
// `least` blocks (one worker where there are fewer).
POD_HD int kv4_workers(long long W, int ctas, int least) {
  const long long n = W / least;
  return n < 1 ? 1 : n < ctas ? (int)n : ctas;
}

}  // namespace pod
