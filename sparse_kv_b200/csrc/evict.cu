// evict.cu -- which tokens a cache of a given budget keeps: the first `sink`,
// the newest `recent`, and the heaviest of the tokens in between by accumulated
// attention weight.
//
// One CTA per (sequence, KV head).  Weights map to 32-bit keys of the same
// order; four radix passes of 8 bits find the key of the last kept token, and a
// walk in token order writes the kept positions (ties to the lower index).
#include "common.cuh"

namespace skv {
namespace {

constexpr int kSelThreads = 1024;

struct EvictParams {
  const float* mass;
  const int* seq_lens;
  int Hkv, max_seq_len, stride, keep, sink, recent;
  int* ids;
  int* keep_lens;
  uint32_t* status;
};

// Order-preserving key: a < b as floats gives key(a) < key(b); -0 equals +0 and
// NaN is below every number.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int block_sum_before(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_rank;
  const int g = blockIdx.x, b = g / p.Hkv, kvh = g % p.Hkv, tid = threadIdx.x;
  int L = p.seq_lens[b];
  if (L < 0 || L > p.max_seq_len) {
    if (tid == 0 && kvh == 0) dev_error(p.status, SKV_DEV_BAD_SEQLEN);
    L = 0;
  }
  const int n = min(L, p.keep);
  if (tid == 0 && kvh == 0) p.keep_lens[b] = n;
  int* ids = p.ids + (size_t)g * p.keep;
  for (int i = n + tid; i < p.keep; i += kSelThreads) ids[i] = -1;
  if (L <= p.keep) {
    for (int i = tid; i < n; i += kSelThreads) ids[i] = i;
    return;
  }
  const float* mass = p.mass + (size_t)g * p.stride;
  const int lo = p.sink, hi = L - p.recent;  // the tokens to choose from
  const int want = p.keep - p.sink - p.recent;
  uint32_t prefix = 0;
  int rank = want;  // rank of the last kept key among those with this prefix
  for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      const uint32_t k = mass_key(mass[i]);
      if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, left = rank;
      while (hist[d] < left) left -= hist[d--];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_rank = left;
    }
    __syncthreads();
    prefix = s_prefix;
    rank = s_rank;
  }
  // kept: key > prefix, and the first `rank` tokens with key == prefix
  int written = 0, ties = 0;
  for (int i0 = 0; i0 < L; i0 += kSelThreads) {
    const int i = i0 + tid;
    const bool fixed = i < L && (i < lo || i >= hi);
    uint32_t k = 0;
    bool tie = false, keep = fixed;
    if (i < L && !fixed && want > 0) {
      k = mass_key(mass[i]);
      tie = k == prefix;
      keep = k > prefix;
    }
    int total;
    const int tie_no = ties + block_sum_before(tie, warp_sums, total);
    ties += total;
    keep = keep || (tie && tie_no < rank);
    const int at = written + block_sum_before(keep, warp_sums, total);
    written += total;
    if (keep) ids[at] = i;
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
  if ((long long)batch * kv_heads > (1 << 24) || max_seq_len > (1 << 30)) return SKV_EUNSUPPORTED;
  const EvictParams p{mass, seq_lens, kv_heads, max_seq_len, mass_stride, keep, sink, recent,
                      keep_ids, keep_lens, status_word};
  evict_select_kernel<<<batch * kv_heads, kSelThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
