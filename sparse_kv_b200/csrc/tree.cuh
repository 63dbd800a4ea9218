// tree.cuh -- what the draft-tree kernels (attention and key mass) share: their
// parameters, the argument checks, and the rules on which token a row sees.
#pragma once

#include <math.h>

#include "common.cuh"
#include "tcgen.cuh"

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

// ---- the tile list.  The tiles of all (sequence, KV head) groups in order, cut into
// shares that differ by one tile at most: worker w of W has tiles
// [w q + min(w, r), ...) with q, r = divmod(total, W).

// Workers that share `total` tiles: one tile each at least.
__host__ __device__ inline int tree_workers(int slots, int total) {
  return total < slots ? (total > 0 ? total : 1) : slots;
}
__device__ __forceinline__ int share_begin(int w, int total, int workers) {
  const int q = total / workers, r = total - q * workers;
  return w * q + min(w, r);
}
__device__ __forceinline__ int share_of(int tile, int total, int workers) {  // the worker of a tile
  const int q = total / workers, r = total - q * workers, cut = r * (q + 1);
  return tile < cut ? tile / (q + 1) : r + (tile - cut) / q;
}

// A run of tiles [a, e) of one group.
struct Segment {
  int b, kvh, a, e;
  TreeSeq s;
  TreeTiles t;
};

// The tiles of a sequence's groups: those its rows can attend (attention), or all of
// them (ALL: the mass of every token is written).
template <bool ALL>
__device__ __forceinline__ TreeTiles list_tiles(const TreeParams& p, const TreeSeq& s) {
  if (ALL) return TreeTiles{(s.L + 127) / 128, 0, 0};
  return tree_tiles(p.window, p.sink, p.recent, s.L, s.n);
}

// Walks the segments of a share.  Every role of a CTA walks the same list.
template <bool ALL>
struct Walk {
  int left, b, kvh, a;
  __device__ __forceinline__ bool next(const TreeParams& p, Segment& g) {
    if (left <= 0) return false;
    for (;; ++b, kvh = 0, a = 0) {
      if (b >= p.B) return false;
      g.s = tree_seq(p, b);
      g.t = list_tiles<ALL>(p, g.s);
      if (g.t.count > 0) break;
    }
    g.b = b;
    g.kvh = kvh;
    g.a = a;
    g.e = min(g.t.count, a + left);
    left -= g.e - a;
    if (g.e == g.t.count) {
      a = 0;
      if (++kvh == p.Hkv) {
        kvh = 0;
        ++b;
      }
    }
    return true;
  }
};

// Tiles before sequence b0 + lane, over the KV heads, given those before b0 (`base`,
// moved on by 32 sequences).  All lanes of a warp.
template <bool ALL>
__device__ __forceinline__ int scan_tiles(const TreeParams& p, int b0, int lane, int& base, int& mine) {
  mine = 0;
  if (b0 + lane < p.B) mine = list_tiles<ALL>(p, tree_seq(p, b0 + lane)).count * p.Hkv;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const int before = base + x - mine;
  base += __shfl_sync(0xffffffffu, x, 31);
  return before;
}

// Worker w's share; every warp finds it for itself (all lanes).  Up to 32 sequences
// their lengths are read once.
template <bool ALL>
__device__ __forceinline__ Walk<ALL> find_share(const TreeParams& p, int slots, int w, int lane, int& total) {
  int base = 0, mine;
  int before = scan_tiles<ALL>(p, 0, lane, base, mine);
  int sum = mine;
  for (int b = lane + 32; b < p.B; b += 32) sum += list_tiles<ALL>(p, tree_seq(p, b)).count * p.Hkv;
  total = p.B <= 32 ? base : __reduce_add_sync(0xffffffffu, sum);
  const int workers = tree_workers(slots, total);
  Walk<ALL> walk{0, 0, 0, 0};
  if (w >= workers || total == 0) return walk;
  const int q = total / workers, r = total - q * workers;
  const int t0 = w * q + min(w, r);
  walk.left = q + (w < r ? 1 : 0);
  int b0 = 0;
  while (base <= t0 && b0 < p.B) {  // the share begins in a later chunk of 32 sequences
    b0 += 32;
    before = scan_tiles<ALL>(p, b0, lane, base, mine);
  }
  const uint32_t hit = __ballot_sync(0xffffffffu, before <= t0 && t0 < before + mine);
  if (hit == 0) {  // the lengths changed under the call
    walk.left = 0;
    return walk;
  }
  const int at = __ffs(hit) - 1;
  const int off = t0 - __shfl_sync(0xffffffffu, before, at);
  const int per_head = __shfl_sync(0xffffffffu, mine, at) / p.Hkv;
  walk.b = b0 + at;
  walk.kvh = off / per_head;
  walk.a = off - walk.kvh * per_head;
  return walk;
}

// Programmatic dependent launch: a kernel's set-up (barriers, tensor memory, tensor
// maps) runs while the kernel before it in the stream drains; nothing that kernel may
// have written is read before this.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// First context token that the recent part of a window still shows to some row: the
// lowest row's position + 1 - recent (0 without a window).  All lanes of a warp.
__device__ __forceinline__ int window_low(const TreeParams& p, const Segment& g, int lane) {
  if (!p.window) return 0;
  int d = kMaxTree;
  for (int t = lane; t < g.s.n; t += 32) d = min(d, tree_depth(tree_word(p, g.b, t, g.s.n), t));
  return g.s.ctx + __reduce_min_sync(0xffffffffu, d) + 1 - p.recent;
}

// A producer's table entries: lane i holds page i & 1 of tile i / 2 of sixteen, read a
// batch ahead.  One by one they took 970 of the 1,400 clocks that HBM leaves a tile of the
// mass, now 450.
constexpr int kPageTiles = 16;
struct PageBatch {
  int page;
  bool wanted;
  // the page of the 64 tokens from `first` (negative: none)
  __device__ __forceinline__ void fetch(const TreeParams& p, const Segment& g, int low, int first) {
    wanted = first >= 0 && first < g.s.L &&
             !(p.window && first >= p.sink && first + kBlock <= low && first + kBlock <= g.s.ctx);
    page = wanted ? p.block_table[(size_t)g.b * p.max_blocks + first / kBlock] : 0;
  }
  // its first row in the pool; -1 where no row attends a token of it, or for a bad page
  __device__ __forceinline__ int row(const TreeParams& p, const Segment& g, bool report) const {
    if (!wanted) return -1;
    if (page < 0 || page >= p.num_pages) {
      if (report) dev_error(p.status, SKV_DEV_BAD_PAGE);
      return -1;
    }
    return (page * p.Hkv + g.kvh) * kBlock;
  }
};

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

constexpr int kKeys = 128;                    // keys per tile
constexpr int kHalfTile = kKeys * 64 * 2;     // [128 keys][64 dims] bf16: 16 KiB
constexpr int kTileKV = 2 * kHalfTile;        // 32 KiB
constexpr float kLog2e = 1.4426950408889634f;

// Score transforms.  PLAIN: z = qscale * s with qscale > 0, folded into the exponent;
// BIAS: any scale, with the distance bias; CAP: that under the tanh cap.
enum { PLAIN = 0, BIAS = 1, CAP = 2 };

struct ScoreFactors {
  float qscale;  // scale * log2 e
  float cap2;    // softcap * log2 e
  float cap_k;   // 2 * scale / softcap * log2 e
  float cap_u;   // scale / softcap
  int bias;      // there are slopes
};

inline ScoreFactors score_factors(const TreeParams& p) {
  ScoreFactors f{p.scale * kLog2e, 0.f, 0.f, 0.f, p.slopes != nullptr};
  if (p.softcap > 0.f) {
    f.cap2 = p.softcap * kLog2e;
    f.cap_u = p.scale / p.softcap;
    f.cap_k = 2.f * f.cap_u * kLog2e;
  }
  return f;
}

inline int score_mode(const TreeParams& p) {
  return p.softcap > 0.f ? CAP : p.slopes || !(p.scale > 0.f) ? BIAS : PLAIN;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The capped score in base 2, cap2 tanh(u) with u = scale s / softcap.  Up to |u| = 1/2, well
// inside the cap and the usual case, it is the score times P(u^2), P a least-maximum fit of
// tanh(u) / u (relative error 1.3e-8), so that a small score keeps its bits however large the
// cap.  Beyond, cap2 (1 - 2 / (1 + e^2|u|)) on the MUFU unit, which would cancel for small u.
// (The second form for half of the columns at any u would save 1 us of 58.5, 7 ragged x 24k
// with cap and bias, and leaves small scores an error of 2^-23 of the cap.)
constexpr float kTanhLimit = 0.25f;  // of u^2
__device__ constexpr float kTanh[5] = {1.000000000e+00f, -3.333306939e-01f, 1.332477932e-01f,
                                      -5.298607527e-02f, 1.713500658e-02f};

__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// 2^x of two numbers on the FMA and integer pipes: x = n + f with n whole and |f| <= 1/2, a
// least-maximum fit of 2^f (relative error 2e-7 with its roundings) and n added to the
// exponent.  0 at and below -127, infinite from 128 on; a NaN, which the integer sum loses,
// is put back by the last product.  For part of a tile's exponentials, beside the MUFU unit:
// 8 clocks a warp there, about 8 FMA-pipe clocks here.
__device__ __forceinline__ void exp2_fma(float& x0, float& x1) {
  float a, b;
  asm("max.NaN.f32 %0, %1, 0fC2FE0000;" : "=f"(a) : "f"(x0));  // -127
  asm("max.NaN.f32 %0, %1, 0fC2FE0000;" : "=f"(b) : "f"(x1));
  asm("min.NaN.f32 %0, %0, 0f43000000;" : "+f"(a));  // 128
  asm("min.NaN.f32 %0, %0, 0f43000000;" : "+f"(b));
  const f2 x = pack2(a, b), magic = pack2(12582912.f, 12582912.f);  // 1.5 * 2^23
  const f2 r = fadd2(x, magic), n = fadd2(r, pack2(-12582912.f, -12582912.f));
  const f2 f = fma2(n, pack2(-1.f, -1.f), x);
  f2 y = fma2(pack2(1.327647245e-03f, 1.327647245e-03f), f, pack2(9.675540961e-03f, 9.675540961e-03f));
  y = fma2(y, f, pack2(5.550713092e-02f, 5.550713092e-02f));
  y = fma2(y, f, pack2(2.402212024e-01f, 2.402212024e-01f));
  y = fma2(y, f, pack2(6.931469440e-01f, 6.931469440e-01f));
  y = fma2(y, f, pack2(1.f, 1.f));
  float y0, y1, r0, r1;
  unpack2(y, y0, y1);
  unpack2(r, r0, r1);
  y0 = __int_as_float(__float_as_int(y0) + (__float_as_int(r0) << 23));
  y1 = __int_as_float(__float_as_int(y1) + (__float_as_int(r1) << 23));
  unpack2(fma2(x, pack2(0.f, 0.f), pack2(y0, y1)), x0, x1);
}

// Scores in base 2 of raw scores s[0 .. N) of one key (in place): cap, then the bias
// slope * place + offset of each column (arrays of N floats, 16-byte aligned).
template <int MODE, int N>
__device__ __forceinline__ void transform(float* s, const ScoreFactors& f, const float* slope, const float* offset,
                                          float place) {
  if (MODE == CAP) {
    const f2 k = pack2(f.cap_u, f.cap_u), q = pack2(f.qscale, f.qscale);
    auto by_fit = [&](f2 x, f2 u) {
      const f2 t = fmul2(u, u);
      f2 r = fma2(pack2(kTanh[4], kTanh[4]), t, pack2(kTanh[3], kTanh[3]));
#pragma unroll
      for (int d = 2; d >= 0; --d) r = fma2(r, t, pack2(kTanh[d], kTanh[d]));
      return fmul2(fmul2(x, q), r);
    };
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) top = fmaxf(top, fabsf(s[c]));
    top *= fabsf(f.cap_u);
    if (__any_sync(0xffffffffu, top * top > kTanhLimit)) {
      auto by_mufu = [&](float x, float u, float y) {  // y: the other form's value
        const float r = f.cap2 * fmaf(-2.f, rcp(1.f + ex2(fabsf(x * f.cap_k))), 1.f);
        return u * u > kTanhLimit ? copysignf(r, u) : y;
      };
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const f2 x = pack2(s[c], s[c + 1]), u = fmul2(x, k);
        float u0, u1, y0, y1;
        unpack2(u, u0, u1);
        unpack2(by_fit(x, u), y0, y1);
        s[c] = by_mufu(s[c], u0, y0);
        s[c + 1] = by_mufu(s[c + 1], u1, y1);
      }
    } else {
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const f2 x = pack2(s[c], s[c + 1]);
        unpack2(by_fit(x, fmul2(x, k)), s[c], s[c + 1]);
      }
    }
  }
  if (MODE == CAP && !f.bias) return;
  const f2 p2 = pack2(place, place), q2 = pack2(f.qscale, f.qscale);
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    const float4 a = *reinterpret_cast<const float4*>(slope + c), o = *reinterpret_cast<const float4*>(offset + c);
    f2 s0 = pack2(s[c], s[c + 1]), s1 = pack2(s[c + 2], s[c + 3]);
    const f2 b0 = fma2(pack2(a.x, a.y), p2, pack2(o.x, o.y)), b1 = fma2(pack2(a.z, a.w), p2, pack2(o.z, o.w));
    s0 = MODE == CAP ? fadd2(s0, b0) : fma2(s0, q2, b0);
    s1 = MODE == CAP ? fadd2(s1, b1) : fma2(s1, q2, b1);
    unpack2(s0, s[c], s[c + 1]);
    unpack2(s1, s[c + 2], s[c + 3]);
  }
}

// Rows t of [t0, t1) that attend the key at position `pos` (drafted token jd, or a
// context token where jd < 0), as bits; `words` are the sequence's masks.
__device__ __forceinline__ unsigned long long rows_of_key(const TreeParams& p, const TreeSeq& s,
                                                          const unsigned long long* words, int jd, int pos, int t0,
                                                          int t1) {
  if (jd < 0 && !p.window) return ~0ull;
  unsigned long long rows = 0;
#pragma unroll 4
  for (int t = t0; t < t1; ++t) {
    const unsigned long long w = words[t];
    bool in = jd < 0 || ((w >> jd) & 1);
    if (p.window) in = in && (pos < p.sink || pos > s.ctx + tree_depth(w, t) - p.recent);
    rows |= (unsigned long long)in << t;
  }
  return rows;
}

}  // namespace skv
