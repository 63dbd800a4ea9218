// evict.cu -- which tokens a cache of a given budget keeps: the first `sink`, the
// newest `recent`, and the heaviest of the tokens in between by accumulated attention
// weight.
//
// A cluster of CTAs per (sequence, KV head), each with a run of the tokens.  Weights
// map to 32-bit keys of the same order.
//   sample  4096 weights of the whole cache (the same in every CTA) bracket the weight
//           of the last kept token: four standard deviations of its sampled rank
//   pass    the cache is read once: above the bracket a token is surely kept, inside
//           it stays open (a bit each in shared memory); open keys are also listed.
//           If the bracket missed, once more with every token open
//   select  radix select of the last kept key among the open ones, 12 bits at a time from
//           the top of the bracket's span.  Every CTA reads the lists of its cluster
//           through distributed shared memory once and finds the key for itself; where
//           the open tokens are too many to list (a run of equal weights) their bits are
//           walked, the weights read again and the histograms added over the cluster
//   last    open tokens above that key are kept, the first few equal to it too;
//           positions are written from the bits, a run of words per thread
// (A histogram of all weights in place of the sample took 100,000 clocks a CTA for 32k
// tokens: shared-memory atomics on neighbouring weights collide.)  Bound by the
// instructions of the pass and the cluster's barriers; the floor is one read.  64 groups
// of 131,072 tokens take 34 us (3.2 us of reads at the copy rate): the pass about 16,000
// clocks, the sample 8,000, the rest the open list and the positions; 2 to 8 groups of 4,096
// take 11.6 to 11.8, a chain of barriers and of single trips to memory.  (Lognormal weights
// over 3 octaves, one token in eight kept.  Weights closer together, or half of them kept,
// leave more tokens open than the lists hold and are read again per digit: 85 to 187 us.)
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "decode.cuh"

namespace skv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kTopBins = 4096;                 // bins of a 12-bit digit
constexpr int kMaxCluster = 8;
constexpr int kListed = 4096;                  // open tokens a CTA lists
constexpr int kSample = 4096;
constexpr int kFew = 256;                      // keys ranked against one another
constexpr int kGathered = 10240;               // open weights of a cluster that a CTA copies, two to an SM
constexpr int kSmemMax = 220 * 1024;
constexpr int kMaxTokens = 1 << 22;            // two bits per token fit in a cluster's shared memory

struct EvictParams {
  const float* mass;
  const int* seq_lens;
  int Hkv, max_seq_len, stride, keep, sink, recent;
  int words;  // mask words of shared memory per CTA
  int gathered;  // open weights of a cluster that a CTA copies
  int* ids;
  int* keep_lens;
  uint32_t* status;
};

// Order-preserving key: a < b as floats gives key(a) < key(b); -0 equals +0 and NaN is
// below every number.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the threads before this one; `total` over all.  Two barriers.
__device__ __forceinline__ int block_before(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int s = lane < kSelWarps ? warp_sums[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, s);
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
  __syncthreads();
  return before + x - v;
}

// the float of a key (NaN for keys that no number has)
__device__ __forceinline__ float key_mass(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const EvictParams p) {
  extern __shared__ int dyn[];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
  int* hist = dyn;                                                     // [kTopBins]
  float* list = reinterpret_cast<float*>(hist + kTopBins);             // [kListed]: weights of open tokens
  int* where = reinterpret_cast<int*>(list + kListed);                 // [kListed]: their tokens in the run
  float* all = reinterpret_cast<float*>(where + kListed);              // [gathered] in a cluster: its open weights
  uint32_t* kept = reinterpret_cast<uint32_t*>(all + (cs > 1 ? p.gathered : 0));  // [words]
  uint32_t* open = kept + p.words;                                     // [words]
  __shared__ int warp_sums[kSelWarps];
  __shared__ int s_digit[2], s_count, s_rank, s_kept, s_open, s_above, s_equal, s_few, s_off[kMaxCluster + 1];
  __shared__ uint32_t s_last;
  const int g = blockIdx.x / cs, b = g / p.Hkv, kvh = g % p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int L = p.seq_lens[b];
  if (L < 0 || L > p.max_seq_len) {
    if (tid == 0 && kvh == 0 && cr == 0) dev_error(p.status, SKV_DEV_BAD_SEQLEN);
    L = 0;
  }
  const int n = min(L, p.keep);
  if (tid == 0 && kvh == 0 && cr == 0) p.keep_lens[b] = n;
  int* ids = p.ids + (size_t)g * p.keep;
  for (int i = n + cr * kSelThreads + tid; i < p.keep; i += cs * kSelThreads) ids[i] = -1;
  if (L <= p.keep) {  // the whole cluster leaves here
    for (int i = cr * kSelThreads + tid; i < n; i += cs * kSelThreads) ids[i] = i;
    return;
  }
  const float* mass = p.mass + (size_t)g * p.stride;
  const int lo = p.sink, hi = L - p.recent;            // the tokens to choose from
  const int want = p.keep - p.sink - p.recent;
  const int all_words = (L + 31) / 32;
  const int w0 = (int)((long long)all_words * cr / cs), nw = (int)((long long)all_words * (cr + 1) / cs) - w0;
  const int per = (nw + kSelThreads - 1) / kSelThreads, a = min(tid * per, nw), e = min(a + per, nw);  // thread t's words
  constexpr int kPer = kTopBins / kSelThreads;         // bins of a thread

  auto clear_hist = [&] {
    for (int i = tid; i < kTopBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
  };
  // The digit that holds the rank-th largest key of the histogram (s_digit[slot]), its
  // count (s_count) and the rank within it (s_rank): thread t owns bins from the top.
  // The results stay until the next pick, whose own barriers part them from it; the
  // histogram itself may be cleared by a faster warp at once.
  auto pick = [&](int rank, int slot, const int (&c)[kPer]) {
    const int top = kTopBins - 1 - tid * kPer;
    int sum = 0, total;
#pragma unroll
    for (int u = 0; u < kPer; ++u) sum += c[u];
    const int before = block_before(sum, warp_sums, total);
    int left = rank - before;
    if (left > 0 && left <= sum) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        if (left > 0 && left <= c[u]) {
          s_digit[slot] = top - u;
          s_count = c[u];
          s_rank = left;
        }
        left -= c[u];
      }
    }
    __syncthreads();
  };
  auto my_bins = [&](int (&c)[kPer]) {  // of this CTA's histogram
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u) c[u] = hist[kTopBins - 1 - tid * kPer - u];
  };

  // ---- sample
  float above = INFINITY, below = 0.f;  // kept: > above; open: not kept, and >= below unless `bottom`
  bool bottom = true;
  const int from = hi - lo;
  if (want > 0 && from > kListed) {
    clear_hist();
    float x[kSample / kSelThreads];
#pragma unroll
    for (int u = 0; u < kSample / kSelThreads; ++u)
      x[u] = mass[lo + (int)((long long)(tid + u * kSelThreads) * from / kSample)];
#pragma unroll
    for (int u = 0; u < kSample / kSelThreads; ++u) atomicAdd(&hist[mass_key(x[u]) >> 20], 1);
    const float f = (float)want / (float)from, mid = f * kSample, d = 4.f * sqrtf(kSample * f * (1.f - f)) + 2.f;
    const int r1 = (int)(mid - d), r2 = (int)(mid + d) + 1;
    int c[kPer];
    my_bins(c);
    if (r1 >= 1) {
      pick(r1, 0, c);
      above = key_mass(((uint32_t)s_digit[0] << 20) | 0xFFFFFu);
    }
    if (r2 <= kSample) {
      pick(r2, 1, c);
      bottom = s_digit[1] < 8;  // -inf and NaN lie there
      if (!bottom) below = key_mass((uint32_t)s_digit[1] << 20);
    }
  }
  // ---- the pass
  int before_kept = 0, rank = 0, open_all = 0, open_max = 0;
  for (int round = 0; round < 2; ++round) {
    if (tid == 0) s_kept = s_open = s_above = s_equal = s_few = 0;
    __syncthreads();
    for (int w = warp; w < nw; w += kSelWarps * 8) {
      float x[8];
      uint32_t my_kept = 0, my_open = 0;  // lane u keeps the bits of word u
      const int i0 = (w0 + w) * 32;
      const bool inner = want > 0 && i0 >= lo && (w0 + w + 7 * kSelWarps) * 32 + 31 < hi && w + 7 * kSelWarps < nw;
      if (inner) {  // no edge among these words
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = mass[i0 + u * (kSelWarps * 32) + lane];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const bool up = x[u] > above;
          const uint32_t k = __ballot_sync(0xffffffffu, up);
          const uint32_t o = __ballot_sync(0xffffffffu, !up && (bottom || x[u] >= below));
          my_kept = lane == u ? k : my_kept;
          my_open = lane == u ? o : my_open;
        }
      } else {
#pragma unroll 2
        for (int u = 0; u < 8; ++u) {
          const int ww = w + u * kSelWarps, i = (w0 + ww) * 32 + lane;
          const bool here = ww < nw && i < L, in = here && want > 0 && i >= lo && i < hi;
          const float y = in ? mass[i] : 0.f;
          const bool up = in && y > above;
          const uint32_t k = __ballot_sync(0xffffffffu, up || (here && (i < lo || i >= hi)));
          const uint32_t o = __ballot_sync(0xffffffffu, in && !up && (bottom || y >= below));
          my_kept = lane == u ? k : my_kept;
          my_open = lane == u ? o : my_open;
        }
      }
      if (lane < 8 && w + lane * kSelWarps < nw) {
        kept[w + lane * kSelWarps] = my_kept;
        open[w + lane * kSelWarps] = my_open;
      }
    }
    __syncthreads();
    // the open tokens' list: thread t has a run of words; with every token open it is a
    // copy of the run (if it is short enough to be listed)
    int n_kept = 0, n_open = 0, all_open;
    for (int w = a; w < e; ++w) {
      n_kept += __popc(kept[w]);
      n_open += __popc(open[w]);
    }
    int slot = block_before(n_open, warp_sums, all_open);
    n_kept = __reduce_add_sync(0xffffffffu, n_kept);
    if (lane == 0) atomicAdd(&s_kept, n_kept);
    if (tid == 0) s_open = all_open;
    if (bottom && above == INFINITY) {
      const int i0 = max(w0 * 32, lo);
      if (all_open <= kListed)
        for (int i = tid; i < all_open; i += kSelThreads) list[i] = mass[i0 + i];
    } else if (all_open <= kListed) {
      for (int w = a; w < e; ++w)
        for (uint32_t o = open[w]; o != 0u; o &= o - 1, ++slot) {
          where[slot] = w * 32 + __ffs(o) - 1;
          list[slot] = mass[w0 * 32 + where[slot]];
        }
    }
    cluster.sync();
    int sure = 0;
    before_kept = open_all = open_max = 0;
    for (int r = 0; r < cs; ++r) {
      const int k = *cluster.map_shared_rank(&s_kept, r), o = *cluster.map_shared_rank(&s_open, r);
      sure += k;
      if (r < cr) before_kept += k;
      if (tid == 0) s_off[r] = open_all;
      open_all += o;
      open_max = max(open_max, o);
    }
    if (tid == 0) s_off[cs] = open_all;
    rank = p.keep - sure;  // the fixed tokens are among the kept
    if (rank >= 0 && rank <= open_all) break;
    above = INFINITY;  // the bracket missed: every token is open
    bottom = true;
    cluster.sync();  // the counts are read
  }
  // ---- select: the key of the last kept token
  uint32_t last = 0;
  int equal_before = 0;  // tokens equal to it in the CTAs before
  if (rank > 0) {
    // the open keys less the lowest possible one: digits of 12 bits from the top of their span
    const uint32_t base = bottom ? 0u : mass_key(below);
    const uint32_t span = (above < INFINITY ? mass_key(above) : 0xFFFFFFFFu) - base;
    int shift = 32 - __clz(span | 1u);
    if (open_max <= kListed && open_all <= p.gathered) {
      // Every CTA copies the open weights of the whole cluster and finds the key for itself.
      // (Short loops: code that runs once waits for its instructions; twenty unrolled keys a
      // thread took twice as long.)
      const float* from_all = list;
      if (cs > 1) {
        from_all = all;
        __syncthreads();
        for (int r = 0; r < cs; ++r) {
          const float* from_r = r == cr ? list : cluster.map_shared_rank(list, r);
          const int off = s_off[r], m = s_off[r + 1] - off;
#pragma unroll 4
          for (int i = tid; i < m; i += kSelThreads) all[off + i] = from_r[i];
        }
        __syncthreads();
      }
      for (int was = 32; shift > 0; was = shift) {
        shift = max(0, shift - 12);
        clear_hist();
#pragma unroll 4
        for (int i = tid; i < open_all; i += kSelThreads) {
          const uint32_t k = mass_key(from_all[i]) - base;
          if (was == 32 || k >> was == last >> was) atomicAdd(&hist[(k >> shift) & (kTopBins - 1)], 1);
        }
        int c[kPer];
        my_bins(c);
        pick(rank, 0, c);
        last |= (uint32_t)s_digit[0] << shift;
        rank = s_rank;
        const int left = s_count;           // keys with this prefix
        if (shift > 0 && left <= kFew) {    // few enough to be ranked against one another
          __syncthreads();
#pragma unroll 4
          for (int i = tid; i < open_all; i += kSelThreads) {
            const uint32_t k = mass_key(from_all[i]) - base;
            if (k >> shift == last >> shift) hist[atomicAdd(&s_few, 1)] = (int)k;
          }
          __syncthreads();
          if (tid < left) {
            const uint32_t mine = (uint32_t)hist[tid];
            int more = 0, same = 0;
            for (int i = 0; i < left; ++i) {
              more += (uint32_t)hist[i] > mine;
              same += (uint32_t)hist[i] == mine;
            }
            if (more < rank && rank <= more + same) {  // equal keys write the same
              s_last = mine;
              s_rank = rank - more;
            }
          }
          __syncthreads();
          last = s_last;
          rank = s_rank;
          break;
        }
      }
      last += base;
      int up = 0, eq = 0;  // in the CTAs before this one
#pragma unroll 4
      for (int i = tid; i < s_off[cr]; i += kSelThreads) {
        const uint32_t k = mass_key(from_all[i]);
        up += k > last;
        eq += k == last;
      }
      up = __reduce_add_sync(0xffffffffu, up);
      eq = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) {
        atomicAdd(&s_above, up);
        atomicAdd(&s_equal, eq);
      }
      // open tokens above the last key are kept, only those equal to it stay open
      if (bottom && above == INFINITY) {  // the list is a copy of the run: a warp per word
        const int i0 = max(w0 * 32, lo) - w0 * 32;
        for (int w = warp; w < nw; w += kSelWarps) {
          const bool in = (open[w] >> lane) & 1;
          const uint32_t k = in ? mass_key(list[w * 32 + lane - i0]) : 0u;
          const uint32_t more = __ballot_sync(0xffffffffu, in && k > last), same = __ballot_sync(0xffffffffu, in && k == last);
          if (lane == 0) {
            kept[w] |= more;
            open[w] = same;
          }
        }
      } else {
        const int m = s_open;
        for (int i = tid; i < m; i += kSelThreads) {
          const uint32_t k = mass_key(list[i]), w = (uint32_t)where[i] >> 5, bit = 1u << (where[i] & 31);
          if (k > last) atomicOr(&kept[w], bit);
          if (k != last) atomicAnd(&open[w], ~bit);
        }
      }
      __syncthreads();
      before_kept += s_above;
      equal_before = s_equal;
    } else {
      // the open keys of this CTA by their bits, eight words at a time
      auto walk = [&](auto use) {
        for (int w = warp; w < nw; w += kSelWarps * 8) {
          float x[8];
          uint32_t o[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int ww = w + u * kSelWarps;
            o[u] = ww < nw ? open[ww] : 0u;
            x[u] = (o[u] >> lane) & 1 ? mass[(w0 + ww) * 32 + lane] : 0.f;
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) use(w + u * kSelWarps, (o[u] >> lane) & 1, mass_key(x[u]));
        }
      };
      for (int was = 32; shift > 0; was = shift) {
        shift = max(0, shift - 12);
        clear_hist();
        walk([&](int, bool in, uint32_t key) {
          const uint32_t k = key - base;
          if (in && (was == 32 || k >> was == last >> was)) atomicAdd(&hist[(k >> shift) & (kTopBins - 1)], 1);
        });
        cluster.sync();
        int c[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) c[u] = 0;
        for (int r = 0; r < cs; ++r) {
          const int* h = cluster.map_shared_rank(hist, r);
#pragma unroll
          for (int u = 0; u < kPer; ++u) c[u] += h[kTopBins - 1 - tid * kPer - u];
        }
        pick(rank, 0, c);
        last |= (uint32_t)s_digit[0] << shift;
        rank = s_rank;
        cluster.sync();  // every histogram has been read
      }
      last += base;
      int up = 0, eq = 0;
      walk([&](int w, bool in, uint32_t k) {
        const uint32_t u = __ballot_sync(0xffffffffu, in && k > last), q = __ballot_sync(0xffffffffu, in && k == last);
        if (lane == 0 && w < nw) {
          kept[w] |= u;
          open[w] = q;
          up += __popc(u);
          eq += __popc(q);
        }
      });
      if (lane == 0) {
        atomicAdd(&s_above, up);
        atomicAdd(&s_equal, eq);
      }
      cluster.sync();
      for (int r = 0; r < cr; ++r) {
        before_kept += *cluster.map_shared_rank(&s_above, r);
        equal_before += *cluster.map_shared_rank(&s_equal, r);
      }
    }
    before_kept += min(equal_before, rank);
  }
  __syncthreads();
  // ---- positions, by thread runs; the first `rank` tokens equal to the
  // last key are kept, in token order
  int total;
  if (rank > 0) {
    int mine = 0;
    for (int w = a; w < e; ++w) mine += __popc(open[w]);
    int no = equal_before + block_before(mine, warp_sums, total);
    for (int w = a; w < e; ++w) {
      uint32_t o = open[w];
      const int c = __popc(o);
      if (no + c <= rank) {
        kept[w] |= o;
      } else {
        for (int left = rank - no; left > 0; --left) {
          kept[w] |= o & (0u - o);
          o &= o - 1;
        }
      }
      no += c;
    }
  }
  int mine = 0;
  for (int w = a; w < e; ++w) mine += __popc(kept[w]);
  int at = block_before(mine, warp_sums, total);
  int* stage = reinterpret_cast<int*>(list);  // [2 * kListed]
  if (total <= 2 * kListed) {  // written through shared memory: neighbours to neighbours
    cluster.sync();            // the lists are read
    for (int w = a; w < e; ++w)
      for (uint32_t k = kept[w]; k != 0u; k &= k - 1) stage[at++] = (w0 + w) * 32 + __ffs(k) - 1;
    __syncthreads();
    for (int i = tid; i < total; i += kSelThreads) ids[before_kept + i] = stage[i];
  } else {
    cluster.sync();
    for (int w = a; w < e; ++w)
      for (uint32_t k = kept[w]; k != 0u; k &= k - 1) ids[before_kept + at++] = (w0 + w) * 32 + __ffs(k) - 1;
  }
}

}  // namespace
}  // namespace skv

extern "C" {

SKV_API skv_status attn_evict_select(const float* mass, const int32_t* seq_lens, int batch, int kv_heads,
                                     int max_seq_len, int mass_stride, int keep, int sink, int recent,
                                     int32_t* keep_ids, int32_t* keep_lens, uint32_t* status_word,
                                     skv_stream_t stream) {
  using namespace skv;
  if (!mass || !seq_lens || !keep_ids || !keep_lens) return SKV_EINVAL;
  if (batch < 1 || kv_heads < 1 || max_seq_len < 0 || mass_stride < max_seq_len) return SKV_EINVAL;
  if (keep < 1 || sink < 0 || recent < 0 || (long long)sink + recent > keep) return SKV_EINVAL;
  const long long groups = (long long)batch * kv_heads;
  if (groups > (1 << 24) || max_seq_len > kMaxTokens || keep > (1 << 30)) return SKV_EUNSUPPORTED;
  if (shared_words(keep_lens, seq_lens, batch)) return SKV_EINVAL;  // one CTA writes while others read
  // CTAs per cluster: as many as a run of 4096 tokens each asks for, while the GPU holds
  // them all at once (two per SM).  Twice as many took 59 us against 37 for 64 groups of
  // 131,072 tokens and 35 against 21 for 128 of 32,768; half as many 40 and 20.
  int cs = 1;
  while (cs < kMaxCluster && max_seq_len > 4096 * cs && groups * cs * 2 <= 2ll * num_sms()) cs *= 2;
  while (cs < kMaxCluster && max_seq_len > (kMaxTokens / kMaxCluster) * cs) cs *= 2;  // the masks must fit
  const int words = (max_seq_len + 31) / 32 / cs + 1;
  // With an SM to each CTA there is room for all lists of a cluster (8 groups of 262,144
  // tokens: 33 us, 157 where they did not fit).
  const size_t fixed = (kTopBins + 2 * (size_t)words + 2 * kListed) * sizeof(int);
  int gathered = kGathered;
  if (groups * cs <= num_sms() && max_seq_len > (1 << 17))
    gathered = std::min(kMaxCluster * kListed, (int)((kSmemMax - fixed) / sizeof(int)));
  const size_t smem = fixed + (cs > 1 ? gathered * sizeof(int) : 0);
  static std::atomic<bool> attr_set[64];  // per device; racing first calls only repeat the set-up
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SKV_ECUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return SKV_ECUDA;
    attr_set[dev] = true;
  }
  const EvictParams p{mass, seq_lens, kv_heads, max_seq_len, mass_stride, keep, sink, recent, words, gathered,
                      keep_ids, keep_lens, status_word};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(groups * cs));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)cs;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, p) == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
