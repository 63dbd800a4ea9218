// evict.cu -- which tokens a cache of a given budget keeps: the first `sink`, the
// newest `recent`, and the heaviest of the tokens in between by accumulated attention
// weight.
//
// A cluster of CTAs per (sequence, KV head), each with a run of the tokens.  Weights
// map to 32-bit keys of the same order.
//   sample  2048 weights of the whole cache (the same in every CTA) bracket the weight
//           of the last kept token: four standard deviations of its sampled rank
//   pass    the cache is read once: above the bracket a token is surely kept, inside
//           it stays open (a bit each in shared memory); open keys are also listed.
//           If the bracket missed, once more with every token open
//   select  radix select of the last kept key among the open ones, 12, 10 and 10 bits;
//           every CTA reads the lists of its cluster through distributed shared memory
//           and finds it for itself.  Where the open tokens are too many to list (a run
//           of equal weights) their bits are walked, the weights read again and the
//           histograms added over the cluster
//   last    open tokens above that key are kept, the first few equal to it too;
//           positions are written from the bits, 32 tokens a word, in order
// (A histogram of all weights in place of the sample took 100,000 clocks a CTA for 32k
// tokens: shared-memory atomics on neighbouring weights collide.)  Bound by the
// instructions of the pass and the cluster's barriers; the floor is one read.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "decode.cuh"

namespace skv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kTopBins = 4096;                 // first digit: 12 bits, then 10 and 10
constexpr int kMaxCluster = 8;
constexpr int kListed = 4096;                  // open tokens a CTA lists
constexpr int kSample = 2048;
constexpr int kMaxTokens = 1 << 22;            // two bits per token fit in a cluster's shared memory

struct EvictParams {
  const float* mass;
  const int* seq_lens;
  int Hkv, max_seq_len, stride, keep, sink, recent;
  int words;  // mask words of shared memory per CTA
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

__global__ void __launch_bounds__(kSelThreads, 3) evict_select_kernel(const EvictParams p) {
  extern __shared__ int dyn[];
  int* hist = dyn;                                                     // [kTopBins]
  uint2* list = reinterpret_cast<uint2*>(hist + kTopBins);             // [kListed]: token of the run, key
  uint32_t* kept = reinterpret_cast<uint32_t*>(list + kListed);        // [words]
  uint32_t* open = kept + p.words;                                     // [words], at the end word offsets
  __shared__ int warp_sums[kSelWarps];
  __shared__ int s_digit[2], s_rank, s_kept, s_sure, s_open, s_count;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
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
  constexpr int kPer = kTopBins / kSelThreads;         // bins of a thread, at most

  auto clear_hist = [&](int bins) {
    for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
  };
  // The digit that holds the rank-th largest key of the histogram (s_digit[slot]) and
  // the rank within it (s_rank): thread t owns bins from the top.
  auto pick = [&](int bins, int rank, int slot, const int (&c)[kPer]) {
    const int top = bins - 1 - tid * (bins / kSelThreads);
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
          s_rank = left;
        }
        left -= c[u];
      }
    }
    __syncthreads();
  };
  auto my_bins = [&](int bins, int (&c)[kPer]) {  // of this CTA's histogram
    __syncthreads();
    const int per = bins / kSelThreads, top = bins - 1 - tid * per;
#pragma unroll
    for (int u = 0; u < kPer; ++u) c[u] = u < per ? hist[top - u] : 0;
  };

  // ---- sample
  float above = INFINITY, below = 0.f;  // kept: > above; open: not kept, and >= below unless `bottom`
  bool bottom = true;
  const int from = hi - lo;
  if (want > 0 && from > kListed) {
    clear_hist(kTopBins);
    float x[kSample / kSelThreads];
#pragma unroll
    for (int u = 0; u < kSample / kSelThreads; ++u)
      x[u] = mass[lo + (int)((long long)(tid + u * kSelThreads) * from / kSample)];
#pragma unroll
    for (int u = 0; u < kSample / kSelThreads; ++u) atomicAdd(&hist[mass_key(x[u]) >> 20], 1);
    const float f = (float)want / (float)from, mid = f * kSample, d = 4.f * sqrtf(kSample * f * (1.f - f)) + 2.f;
    const int r1 = (int)(mid - d), r2 = (int)(mid + d) + 1;
    int c[kPer];
    my_bins(kTopBins, c);
    if (r1 >= 1) {
      pick(kTopBins, r1, 0, c);
      above = key_mass(((uint32_t)s_digit[0] << 20) | 0xFFFFFu);
    }
    if (r2 <= kSample) {
      pick(kTopBins, r2, 1, c);
      bottom = s_digit[1] < 8;  // -inf and NaN lie there
      if (!bottom) below = key_mass((uint32_t)s_digit[1] << 20);
    }
  }
  // ---- the pass
  int before_kept = 0, open_max = 0, rank = 0, open_all = 0;
  for (int round = 0; round < 2; ++round) {
    if (tid == 0) s_kept = s_sure = s_open = s_count = 0;
    __syncthreads();
    int n_kept = 0, n_sure = 0;
    for (int w = warp; w < nw; w += kSelWarps * 8) {
      float x[8];
      uint32_t o[8], k[8];
      int n_open = 0;
      const int i0 = (w0 + w) * 32;
      const bool inner = want > 0 && i0 >= lo && (w0 + w + 7 * kSelWarps) * 32 + 31 < hi && w + 7 * kSelWarps < nw;
      if (inner) {  // no edge among these words
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = mass[i0 + u * (kSelWarps * 32) + lane];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const bool up = x[u] > above;
          k[u] = __ballot_sync(0xffffffffu, up);
          o[u] = __ballot_sync(0xffffffffu, !up && (bottom || x[u] >= below));
          n_sure += __popc(k[u]);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int ww = w + u * kSelWarps, i = (w0 + ww) * 32 + lane;
          const bool here = ww < nw && i < L, in = here && want > 0 && i >= lo && i < hi;
          x[u] = in ? mass[i] : 0.f;
          const bool up = in && x[u] > above;
          k[u] = __ballot_sync(0xffffffffu, up);
          o[u] = __ballot_sync(0xffffffffu, in && !up && (bottom || x[u] >= below));
          n_sure += __popc(k[u]);
          k[u] |= __ballot_sync(0xffffffffu, here && (i < lo || i >= hi));
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        n_kept += __popc(k[u]);
        n_open += __popc(o[u]);
      }
      if (n_open > 0) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&s_open, n_open);
        at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int slot = at + __popc(o[u] & ((1u << lane) - 1));
          if (((o[u] >> lane) & 1) && slot < kListed)
            list[slot] = make_uint2((uint32_t)((w + u * kSelWarps) * 32 + lane), mass_key(x[u]));
          at += __popc(o[u]);
        }
      }
      if (lane < 8 && w + lane * kSelWarps < nw) {
        uint32_t kk = k[0], oo = o[0];
#pragma unroll
        for (int u = 1; u < 8; ++u) {
          kk = lane == u ? k[u] : kk;
          oo = lane == u ? o[u] : oo;
        }
        kept[w + lane * kSelWarps] = kk;
        open[w + lane * kSelWarps] = oo;
      }
    }
    if (lane == 0) {
      atomicAdd(&s_kept, n_kept);
      atomicAdd(&s_sure, n_sure);
    }
    cluster.sync();
    int sure = 0;
    before_kept = open_max = open_all = 0;
    for (int r = 0; r < cs; ++r) {
      sure += *cluster.map_shared_rank(&s_sure, r);
      const int o = *cluster.map_shared_rank(&s_open, r);
      open_all += o;
      open_max = max(open_max, o);
      if (r < cr) before_kept += *cluster.map_shared_rank(&s_kept, r);
    }
    rank = want - sure;
    if (rank >= 0 && rank <= open_all) break;
    above = INFINITY;  // the bracket missed: every token is open
    bottom = true;
    cluster.sync();  // the counts are read
  }
  // ---- select: the key of the last kept token
  uint32_t last = 0xFFFFFFFFu;
  int equal_before = 0;  // tokens equal to it in the CTAs before
  const bool listed = open_max <= kListed;
  if (rank > 0) {
    last = 0;
    if (listed) {
      // every CTA counts the open tokens of the whole cluster
      for (int shift = 20; shift >= 0; shift -= 10) {
        const int bins = shift == 20 ? kTopBins : 1024;
        clear_hist(bins);
        for (int r = 0; r < cs; ++r) {
          const uint2* from_r = cluster.map_shared_rank(list, r);
          const int m = *cluster.map_shared_rank(&s_open, r);
#pragma unroll 4
          for (int i = tid; i < m; i += kSelThreads) {
            const uint32_t k = from_r[i].y;
            if (shift == 20 || k >> (shift + 10) == last >> (shift + 10)) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
          }
        }
        int c[kPer];
        my_bins(bins, c);
        pick(bins, rank, 0, c);
        last |= (uint32_t)s_digit[0] << shift;
        rank = s_rank;
      }
      int up = 0, eq = 0;  // in the CTAs before this one
      for (int r = 0; r < cr; ++r) {
        const uint2* from_r = cluster.map_shared_rank(list, r);
        const int m = *cluster.map_shared_rank(&s_open, r);
#pragma unroll 4
        for (int i = tid; i < m; i += kSelThreads) {
          const uint32_t k = from_r[i].y;
          up += k > last;
          eq += k == last;
        }
      }
      int t_up, t_eq;
      block_before(up, warp_sums, t_up);
      block_before(eq, warp_sums, t_eq);
      equal_before = t_eq;
      before_kept += t_up + min(t_eq, rank);
      const int m = s_open;
      for (int i = tid; i < m; i += kSelThreads) {
        const uint32_t k = list[i].y, w = list[i].x >> 5, bit = 1u << (list[i].x & 31u);
        if (k > last) atomicOr(&kept[w], bit);
        if (k != last) atomicAnd(&open[w], ~bit);
      }
    } else {
      // this CTA's open tokens by their bits, eight words at a time
      auto each_open = [&](auto use) {
        for (int w = warp; w < nw; w += kSelWarps * 8) {
          float x[8];
          uint32_t o[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int ww = w + u * kSelWarps;
            o[u] = ww < nw ? open[ww] : 0u;
            if ((o[u] >> lane) & 1) x[u] = mass[(w0 + ww) * 32 + lane];
          }
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if ((o[u] >> lane) & 1) use(w + u * kSelWarps, mass_key(x[u]));
        }
      };
      for (int shift = 20; shift >= 0; shift -= 10) {
        const int bins = shift == 20 ? kTopBins : 1024;
        clear_hist(bins);
        each_open([&](int, uint32_t k) {
          if (shift == 20 || k >> (shift + 10) == last >> (shift + 10)) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
        });
        cluster.sync();
        int c[kPer];
        const int per = bins / kSelThreads, top = bins - 1 - tid * per;
#pragma unroll
        for (int u = 0; u < kPer; ++u) c[u] = 0;
        for (int r = 0; r < cs; ++r) {
          const int* h = cluster.map_shared_rank(hist, r);
#pragma unroll
          for (int u = 0; u < kPer; ++u)
            if (u < per) c[u] += h[top - u];
        }
        pick(bins, rank, 0, c);
        last |= (uint32_t)s_digit[0] << shift;
        rank = s_rank;
        cluster.sync();  // every histogram has been read
      }
      int up = 0, eq = 0;
      each_open([&](int w, uint32_t k) {
        up += k > last;
        eq += k == last;
        if (k > last) atomicOr(&kept[w], 1u << lane);
        if (k != last) atomicAnd(&open[w], ~(1u << lane));
      });
      int t_up, t_eq;
      block_before(up, warp_sums, t_up);
      block_before(eq, warp_sums, t_eq);
      if (tid == 0) {
        s_sure = t_up;
        s_count = t_eq;
      }
      cluster.sync();
      int up_before = 0;
      for (int r = 0; r < cr; ++r) {
        up_before += *cluster.map_shared_rank(&s_sure, r);
        equal_before += *cluster.map_shared_rank(&s_count, r);
      }
      before_kept += up_before + min(equal_before, rank);
    }
  }
  __syncthreads();
  // ---- positions.  Thread t has a run of words; the first `rank` tokens equal to the
  // last key are kept, in token order
  const int per = (nw + kSelThreads - 1) / kSelThreads, a = min(tid * per, nw), e = min(a + per, nw);
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
  int at = before_kept + block_before(mine, warp_sums, total);
  for (int w = a; w < e; ++w) {
    open[w] = (uint32_t)at;
    at += __popc(kept[w]);
  }
  __syncthreads();
#pragma unroll 4
  for (int w = warp; w < nw; w += kSelWarps) {
    const uint32_t k = kept[w];
    if ((k >> lane) & 1) ids[open[w] + __popc(k & ((1u << lane) - 1))] = (w0 + w) * 32 + lane;
  }
  cluster.sync();  // lists and counts are read before any CTA ends
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
  if (groups > (1 << 24) || max_seq_len > kMaxTokens) return SKV_EUNSUPPORTED;
  // CTAs per cluster: as many as a run of 4096 tokens each asks for, while the GPU holds
  // them all at once (three per SM)
  int cs = 1;
  while (cs < kMaxCluster && max_seq_len > 4096 * cs && groups * cs * 2 <= 3ll * num_sms()) cs *= 2;
  while (cs < kMaxCluster && max_seq_len > (kMaxTokens / kMaxCluster) * cs) cs *= 2;  // the masks must fit
  const int words = (max_seq_len + 31) / 32 / cs + 1;
  const size_t smem = (kTopBins + 2 * (size_t)words + 2 * kListed) * sizeof(int);
  static std::atomic<bool> attr_set[64];  // per device; racing first calls only repeat the set-up
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SKV_ECUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) != cudaSuccess)
      return SKV_ECUDA;
    attr_set[dev] = true;
  }
  const EvictParams p{mass, seq_lens, kv_heads, max_seq_len, mass_stride, keep, sink, recent, words,
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
