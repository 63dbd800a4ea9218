// tree.cuh -- what the draft-tree kernels (attention and key mass) share: their
// parameters, the argument checks, and the rules on which token a row sees.
#pragma once

#include <math.h>

#include "common.cuh"

namespace skv {

constexpr int kMaxTree = 64;  // drafted tokens per sequence: one mask word per row

struct TreeParams {
  const uint16_t* q;
  const uint16_t* k_pool;
  const uint16_t* v_pool;
  const int* block_table;
  const int* seq_lens;
  const int* tree_lens;
  const unsigned long long* tree_mask;
  const float* slopes;
  int B, T, Hq, Hkv, G, max_blocks, num_pages, max_seq_len;
  int sink, recent, window;  // window: the sink + recent rule applies
  float scale, softcap;
  float* out;
  float* lse;
  uint32_t* status;
};

// Host-side checks of the fields both entry points read; fills *p.
skv_status tree_params(const skv_tree_args* a, TreeParams* p);

// Token counts of sequence b.  A bad length leaves an empty sequence.
struct TreeSeq {
  int L, n, ctx;
  bool bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  s.L = p.seq_lens[b];
  s.n = p.tree_lens ? p.tree_lens[b] : p.T;
  s.bad = s.L < 0 || s.L > p.max_seq_len || s.n < 0 || s.n > p.T || s.n > s.L;
  if (s.bad) s.L = s.n = 0;
  s.ctx = s.L - s.n;
  return s;
}

// Drafted tokens that row t sees, as a bit mask over [0, n).
__device__ __forceinline__ unsigned long long tree_word(const TreeParams& p, int b, int t, int n) {
  const unsigned long long in = n >= 64 ? ~0ull : (1ull << n) - 1;
  const unsigned long long w = p.tree_mask ? p.tree_mask[(size_t)b * p.T + t] : (2ull << t) - 1;
  return w & in;
}

__device__ __forceinline__ int tree_depth(unsigned long long word, int t) {
  return __popcll(word & ~(1ull << t));
}

// Which 128-token tiles of a sequence its rows can attend: `head` tiles from
// token 0, then the rest from token `lo` on, a page border (no window: all from
// 0).  Without a row to serve there is none.
struct TreeTiles {
  int count, head, lo;
};

__host__ __device__ inline TreeTiles tree_tiles(int window, int sink, int recent, int L, int n) {
  TreeTiles t{0, 0, 0};
  if (n == 0) return t;
  if (window) {
    const int a = sink < L ? sink : L, ctx = L - n;
    t.head = (a + 127) / 128;
    const int lo = recent > ctx ? 0 : recent > 0 ? ctx + 1 - recent : ctx;
    t.lo = lo / kBlock * kBlock;
    if (t.lo <= t.head * 128) t.head = t.lo = 0;
  }
  t.count = t.head + (L - t.lo + 127) / 128;
  return t;
}

__host__ __device__ inline int tree_tile_start(const TreeTiles& t, int j) {
  return j < t.head ? j * 128 : t.lo + (j - t.head) * 128;
}

}  // namespace skv
