// compact.cu -- moves the kept tokens of a paged cache together: K and V rows,
// and the tokens' accumulated weight.
//
// In place, chunk by chunk in list order: a CTA reads a chunk's rows, waits, and
// writes them.  Row i goes to first + i and comes from ids[i] >= first + i, so a
// chunk writes only positions below every row that a later chunk reads, and needs to
// wait for nobody else.  The columns of a row are independent: a CTA takes 1/NS of
// every row (16 .. 256 bytes), so that a few groups fill the GPU too.  HBM-bound: 512
// bytes read and written per moved token and KV head; the next chunk's list entries and
// page numbers are fetched while this one's rows are on their way.
#include <algorithm>

#include "common.cuh"
#include "decode.cuh"

namespace skv {
namespace {

constexpr int kMoveThreads = 512;
constexpr int kRowVecs = kRowBytes / 16;       // 16-byte vectors of a row
constexpr int kPasses = 4;                     // 16-byte loads in flight per thread

struct CompactParams {
  const uint4* k;
  const uint4* v;
  const int* table;
  const int* seq_lens;
  const int* ids;
  const int* keep_lens;
  const int* first;
  uint4* dst_k;
  uint4* dst_v;
  const int* dst_table;
  float* mass;
  int* new_lens;
  int Hkv, max_blocks, num_pages, max_seq_len, ids_heads, max_keep, dst_max_blocks, dst_num_pages, stride;
  bool in_place;
  bool ordered;  // ids must not precede their destinations
  uint32_t* status;
};

// grid (batch * kv_heads, 2 NS or 2 NS + 1): slices of the K rows, of the V rows, weights
template <int NS>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  constexpr int kLanes = kRowVecs / NS;             // threads per row
  constexpr int kRows = kMoveThreads / kLanes;      // rows per pass
  const int g = blockIdx.x, b = g / p.Hkv, kvh = g % p.Hkv, what = blockIdx.y, tid = threadIdx.x;
  const int L = p.seq_lens[b], n = p.keep_lens[b], f = p.first ? p.first[b] : 0;
  if (L < 0 || L > p.max_seq_len || n < 0 || n > p.max_keep || f < 0 || f > L) {
    if (what == 0 && kvh == 0 && tid == 0) {
      dev_error(p.status, SKV_DEV_BAD_SEQLEN);
      p.new_lens[b] = max(0, min(L, p.max_seq_len));
    }
    return;
  }
  if (what == 0 && kvh == 0 && tid == 0) p.new_lens[b] = f + n;
  const int* ids = p.ids + ((size_t)b * p.ids_heads + (p.ids_heads > 1 ? kvh : 0)) * p.max_keep;
  const int* src_table = p.table + (size_t)b * p.max_blocks;
  const int* dst_table = p.dst_table + (size_t)b * p.dst_max_blocks;
  // row numbers in the pools of list entry i, which is token `id`; src < 0 if it does not move
  auto locate = [&](int i, int id, bool report, int& src, int& dst) {
    const int to = f + i;
    src = -1;
    if (id < 0 || id >= L || (p.ordered && id < to)) {
      if (report) dev_error(p.status, SKV_DEV_BAD_ORDER);
      return;
    }
    const int sp = src_table[id / kBlock];
    const int dp = to / kBlock < p.dst_max_blocks ? dst_table[to / kBlock] : -1;
    if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.dst_num_pages) {
      if (report) dev_error(p.status, SKV_DEV_BAD_PAGE);
      return;
    }
    src = (sp * p.Hkv + kvh) * kBlock + id % kBlock;
    dst = (dp * p.Hkv + kvh) * kBlock + to % kBlock;
  };
  if (what == 2 * NS) {
    float* mass = p.mass + (size_t)g * p.stride;
    for (int i0 = 0; i0 < n; i0 += kMoveThreads * 4) {
      float x[4];
      bool moves[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kMoveThreads + tid, id = i < n ? ids[i] : -1;
        int src = -1, dst;
        if (i < n) locate(i, id, false, src, dst);
        moves[u] = src >= 0;
        if (moves[u]) x[u] = mass[id];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (moves[u]) mass[f + i0 + u * kMoveThreads + tid] = x[u];
    }
    return;
  }
  const uint4* from = (what < NS ? p.k : p.v) + (what % NS) * kLanes + tid % kLanes;
  uint4* into = (what < NS ? p.dst_k : p.dst_v) + (what % NS) * kLanes + tid % kLanes;
  const int row = tid / kLanes;
  int src[kPasses], dst[kPasses];
  auto fetch = [&](int i0) {
    int id[kPasses];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int i = i0 + u * kRows + row;
      id[u] = i < n ? ids[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int i = i0 + u * kRows + row;
      src[u] = -1;
      // one thread per row flags its faults; a row that is in its place stays
      if (i < n && !(p.in_place && id[u] == f + i && id[u] < L)) locate(i, id[u], what == 0 && tid % kLanes == 0, src[u], dst[u]);
    }
  };
  fetch(0);
  for (int i0 = 0; i0 < n; i0 += kRows * kPasses) {
    uint4 x[kPasses];
    int to[kPasses];
    uint32_t moves = 0;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      if (src[u] >= 0) {
        x[u] = from[(size_t)src[u] * kRowVecs];
        moves |= 1u << u;
      }
      to[u] = dst[u];
    }
    if (i0 + kRows * kPasses < n) fetch(i0 + kRows * kPasses);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPasses; ++u)
      if ((moves >> u) & 1) into[(size_t)to[u] * kRowVecs] = x[u];
  }
}

template <int NS>
cudaError_t launch_compact(const CompactParams& p, int groups, bool mass, cudaStream_t s) {
  compact_kernel<NS><<<dim3(groups, 2 * NS + (mass ? 1 : 0)), kMoveThreads, 0, s>>>(p);
  return cudaGetLastError();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace skv

extern "C" {

SKV_API skv_status attn_compact_cache(const skv_compact_args* a, skv_stream_t stream) {
  using namespace skv;
  if (!a) return SKV_EINVAL;
  if (!a->k_pool || !a->v_pool || !a->block_table || !a->seq_lens || !a->keep_ids || !a->keep_lens ||
      !a->new_lens)
    return SKV_EINVAL;
  if (a->batch < 1 || a->kv_heads < 1 || a->max_seq_len < 0 || a->num_pages < 1 || a->max_blocks < 0 ||
      a->max_keep < 1)
    return SKV_EINVAL;
  if (shared_words(a->new_lens, a->seq_lens, a->batch) || shared_words(a->new_lens, a->keep_lens, a->batch) ||
      (a->first && shared_words(a->new_lens, a->first, a->batch)))
    return SKV_EINVAL;  // one CTA of a sequence writes while others read
  if (a->head_dim != kHeadDim || a->block_size != kBlock) return SKV_EUNSUPPORTED;
  if ((long long)a->max_blocks * kBlock < (long long)a->max_seq_len) return SKV_EINVAL;
  if (a->ids_heads != 1 && a->ids_heads != a->kv_heads) return SKV_EINVAL;
  const bool copy = a->dst_block_table != nullptr;
  if (!copy && (a->dst_k_pool || a->dst_v_pool)) return SKV_EINVAL;
  if (copy && (!a->dst_k_pool != !a->dst_v_pool || a->dst_max_blocks < 0 || a->dst_num_pages < 1)) return SKV_EINVAL;
  if (a->mass && a->mass_stride < a->max_seq_len) return SKV_EINVAL;
  if (!aligned16(a->k_pool) || !aligned16(a->v_pool) || !aligned16(a->dst_k_pool) || !aligned16(a->dst_v_pool))
    return SKV_EINVAL;
  if ((long long)a->batch * a->kv_heads > (1 << 24) || a->max_seq_len > (1 << 30) || a->max_keep > (1 << 30))
    return SKV_EUNSUPPORTED;
  if (std::max((long long)a->num_pages, copy ? (long long)a->dst_num_pages : 0ll) * a->kv_heads * kBlock >= (1ll << 31))
    return SKV_EUNSUPPORTED;  // row numbers are 32-bit
  CompactParams p{};
  p.k = static_cast<const uint4*>(a->k_pool);
  p.v = static_cast<const uint4*>(a->v_pool);
  p.table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.ids = a->keep_ids;
  p.keep_lens = a->keep_lens;
  p.first = a->first;
  p.dst_k = static_cast<uint4*>(copy && a->dst_k_pool ? a->dst_k_pool : a->k_pool);
  p.dst_v = static_cast<uint4*>(copy && a->dst_v_pool ? a->dst_v_pool : a->v_pool);
  p.dst_table = copy ? a->dst_block_table : a->block_table;
  p.dst_max_blocks = copy ? a->dst_max_blocks : a->max_blocks;
  p.dst_num_pages = copy ? a->dst_num_pages : a->num_pages;
  p.mass = a->mass;
  p.new_lens = a->new_lens;
  p.Hkv = a->kv_heads;
  p.max_blocks = a->max_blocks;
  p.num_pages = a->num_pages;
  p.max_seq_len = a->max_seq_len;
  p.ids_heads = a->ids_heads;
  p.max_keep = a->max_keep;
  p.stride = a->mass_stride;
  p.in_place = p.dst_table == p.table && p.dst_k == p.k && p.dst_v == p.v;
  p.ordered = p.in_place || a->mass != nullptr;
  p.status = a->status_word;
  // Whole rows unless that leaves SMs without a CTA: 4k of 32k tokens for 128 KV heads
  // took 104 us with whole rows (256 CTAs), 140 with halves, 147 with quarters; for 8 KV
  // heads whole rows would run on 16 SMs.
  const int groups = a->batch * a->kv_heads, sms = num_sms();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool mass = a->mass != nullptr;
  const cudaError_t e = groups * 2ll >= sms   ? launch_compact<1>(p, groups, mass, s)
                        : groups * 4ll >= sms ? launch_compact<2>(p, groups, mass, s)
                        : groups * 8ll >= sms ? launch_compact<4>(p, groups, mass, s)
                                                : launch_compact<8>(p, groups, mass, s);
  return e == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
