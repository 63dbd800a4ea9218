// evict.cu -- which tokens a cache of a given budget keeps: the first `sink`, the
// newest `recent`, and the heaviest of the tokens in between by accumulated attention
// weight.
//
// A cluster of CTAs per (sequence, KV head), each with a run of the tokens.  Weights
// map to 32-bit keys of the same order, and a radix select finds the key of the last
// kept token from the top: 12, 10 and 10 bits.
//   pass 1  histogram of the top 12 bits (the whole cache is read)
//   pass 2  one bit per token in shared memory: surely kept (a higher digit, or one of
//           the fixed tokens), or still open (the same digit); the cache is read again,
//           from L2
//   then    only open tokens are looked at: histograms of the next digits, the bits of
//           those above the last kept key, and of the first few equal to it.  Pass 2
//           lists them in shared memory; where they are too many (a run of equal
//           weights) their bits are walked and the weights read again
//   last    positions written from the bits, 32 tokens a word, in order
// The histograms of a cluster are added through distributed shared memory.  Bound by
// the shared-memory atomics of pass 1 and the cluster's barriers: the floor is one read.
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

__global__ void __launch_bounds__(kSelThreads, 3) evict_select_kernel(const EvictParams p) {
  extern __shared__ int dyn[];
  int* hist = dyn;                                                     // [kTopBins]
  uint32_t* kept = reinterpret_cast<uint32_t*>(dyn + kTopBins);        // [words]
  uint32_t* open = kept + p.words;                                     // [words], at the end word offsets
  uint2* list = reinterpret_cast<uint2*>(hist + ((kTopBins + 2 * p.words + 1) & ~1));  // [kListed]: token of the run, key
  __shared__ int warp_sums[kSelWarps];
  __shared__ int s_digit, s_rank, s_count, s_listed;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
  const int g = blockIdx.x / cs, b = g / p.Hkv, kvh = g % p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

  // The digit that holds the rank-th largest key, and the rank within it: the bins are
  // added over the cluster, thread t owns bins from the top.
  auto pick = [&](int bins, int rank) {
    cluster.sync();
    const int per = bins / kSelThreads, top = bins - 1 - tid * per;
    int c[kTopBins / kSelThreads], sum = 0;
#pragma unroll
    for (int u = 0; u < kTopBins / kSelThreads; ++u) c[u] = 0;
    for (int r = 0; r < cs; ++r) {
      const int* h = cluster.map_shared_rank(hist, r);
#pragma unroll
      for (int u = 0; u < kTopBins / kSelThreads; ++u)
        if (u < per) c[u] += h[top - u];
    }
#pragma unroll
    for (int u = 0; u < kTopBins / kSelThreads; ++u) sum += c[u];
    int total;
    const int before = block_before(sum, warp_sums, total);
    if (before < rank && rank <= before + sum) {
      int left = rank - before;
#pragma unroll
      for (int u = 0; u < kTopBins / kSelThreads; ++u) {
        if (left > 0 && left <= c[u]) {
          s_digit = top - u;
          s_rank = left;
        }
        left -= c[u];
      }
    }
    cluster.sync();  // every histogram has been read; s_digit and s_rank are written
  };

  uint32_t last = 0;  // key of the last kept token, digit by digit
  int rank = want;
  if (want > 0) {
    // ---- pass 1
    for (int i = tid; i < kTopBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const int i0 = max(w0 * 32, lo), i1 = min((w0 + nw) * 32, hi);
    const uint32_t zero = mass_key(0.f) >> 20;
    for (int i = i0 + tid; i - tid < i1; i += kSelThreads * 8) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u * kSelThreads < i1) x[u] = mass[i + u * kSelThreads];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool in = i + u * kSelThreads < i1;
        const uint32_t d = in ? mass_key(x[u]) >> 20 : 0u;
        // tokens that nothing attended share one bin: counted once per warp
        const uint32_t z = __ballot_sync(0xffffffffu, in && d == zero);
        if (in && d != zero) atomicAdd(&hist[d], 1);
        if (lane == 0 && z != 0u) atomicAdd(&hist[zero], __popc(z));
      }
    }
    pick(kTopBins, rank);
    last = (uint32_t)s_digit << 20;
    rank = s_rank;
  }
  // ---- pass 2: bits of the surely kept and of the open tokens
  if (tid == 0) s_listed = s_count = 0;
  __syncthreads();
  for (int w = warp; w < nw; w += kSelWarps * 8) {
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = (w0 + w + u * kSelWarps) * 32 + lane;
      x[u] = 0.f;
      if (w + u * kSelWarps < nw && i < hi && i >= lo && want > 0) x[u] = mass[i];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int ww = w + u * kSelWarps, i = (w0 + ww) * 32 + lane;
      const bool fixed = i < L && (i < lo || i >= hi), in = ww < nw && i < L && !fixed && want > 0;
      const uint32_t key = mass_key(x[u]), d = key >> 20;
      const uint32_t k = __ballot_sync(0xffffffffu, fixed || (in && d > last >> 20));
      const uint32_t o = __ballot_sync(0xffffffffu, in && d == last >> 20);
      if (o != 0u) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&s_listed, __popc(o));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(o & ((1u << lane) - 1));
        if (((o >> lane) & 1) && at < kListed) list[at] = make_uint2((uint32_t)(ww * 32 + lane), key);
      }
      if (lane == 0 && ww < nw) {
        kept[ww] = k;
        open[ww] = o;
      }
    }
  }
  __syncthreads();
  const int listed = s_listed;
  // ---- the other digits, among the open tokens
  if (want > 0) {
    // the open tokens' keys, from the list or, eight words at a time, from the cache
    auto each_open = [&](auto use) {
      if (listed <= kListed) {
        for (int i = tid; i < listed; i += kSelThreads) use((int)(list[i].x >> 5), list[i].x & 31u, list[i].y);
        return;
      }
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
          if ((o[u] >> lane) & 1) use(w + u * kSelWarps, (uint32_t)lane, mass_key(x[u]));
      }
    };
    for (int shift = 10; shift >= 0; shift -= 10) {
      for (int i = tid; i < 1024; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      each_open([&](int, uint32_t, uint32_t k) {
        if (k >> (shift + 10) == last >> (shift + 10)) atomicAdd(&hist[(k >> shift) & 1023], 1);
      });
      pick(1024, rank);
      last |= (uint32_t)s_digit << shift;
      rank = s_rank;
    }
    // open tokens above the last kept key are kept; those equal to it stay open
    int ties = 0;
    each_open([&](int w, uint32_t bit, uint32_t k) {
      if (k > last) atomicOr(&kept[w], 1u << bit);
      if (k == last) ++ties;
      else atomicAnd(&open[w], ~(1u << bit));
    });
    __syncthreads();
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) atomicAdd(&s_count, ties);
    cluster.sync();
    int before = 0;
    for (int r = 0; r < cr; ++r) before += *cluster.map_shared_rank(&s_count, r);
    // the first `rank` of the equal ones, in token order: thread t has a run of words
    const int per = (nw + kSelThreads - 1) / kSelThreads, a = min(tid * per, nw), e = min(a + per, nw);
    int mine = 0, total;
    for (int w = a; w < e; ++w) mine += __popc(open[w]);
    int no = before + block_before(mine, warp_sums, total);
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
    cluster.sync();  // the counts are read
  }
  __syncthreads();
  // ---- positions: words before, over the cluster and within it
  const int per = (nw + kSelThreads - 1) / kSelThreads, a = min(tid * per, nw), e = min(a + per, nw);
  int mine = 0, total;
  for (int w = a; w < e; ++w) mine += __popc(kept[w]);
  const int before = block_before(mine, warp_sums, total);
  if (tid == 0) s_count = total;
  cluster.sync();
  int at = before;
  for (int r = 0; r < cr; ++r) at += *cluster.map_shared_rank(&s_count, r);
  for (int w = a; w < e; ++w) {
    open[w] = (uint32_t)at;
    at += __popc(kept[w]);
  }
  __syncthreads();
  for (int w = warp; w < nw; w += kSelWarps) {
    const uint32_t k = kept[w];
    if ((k >> lane) & 1) ids[open[w] + __popc(k & ((1u << lane) - 1))] = (w0 + w) * 32 + lane;
  }
  cluster.sync();  // the counts are read before any CTA ends
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
  const size_t smem = (kTopBins + 2 * (size_t)words + 2 + 2 * kListed) * sizeof(int);
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
