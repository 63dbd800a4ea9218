// compact.cu -- moves the kept tokens of a paged cache together: K and V rows,
// and the tokens' accumulated weight.
//
// In place, chunk by chunk in list order: a CTA reads a chunk's rows, waits, and
// writes them.  Row i goes to first + i and comes from ids[i] >= first + i, so a
// chunk writes only positions below every row that a later chunk reads.
#include "common.cuh"

namespace skv {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kRowLanes = kRowBytes / 16;                // threads per row
constexpr int kRowsPer = kMoveThreads / kRowLanes;       // rows per pass
constexpr int kPasses = 8;                               // 16-byte loads in flight per thread

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
  bool ordered;  // ids must not precede their destinations
  uint32_t* status;
};

// grid (batch * kv_heads, 2 or 3): K rows, V rows, weights
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  const int g = blockIdx.x, b = g / p.Hkv, kvh = g % p.Hkv, what = blockIdx.y, tid = threadIdx.x;
  int L = p.seq_lens[b], n = p.keep_lens[b];
  int f = p.first ? p.first[b] : 0;
  const bool report = what == 0 && tid % kRowLanes == 0;  // one thread per row flags its faults
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
  // source and destination rows of list entry i; false if it does not move
  auto locate = [&](int i, size_t& src, size_t& dst) {
    const int id = ids[i], to = f + i;
    if (id < 0 || id >= L || (p.ordered && id < to)) {
      if (report) dev_error(p.status, SKV_DEV_BAD_ORDER);
      return false;
    }
    const int sp = src_table[id / kBlock];
    const int dp = to / kBlock < p.dst_max_blocks ? dst_table[to / kBlock] : -1;
    if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.dst_num_pages) {
      if (report) dev_error(p.status, SKV_DEV_BAD_PAGE);
      return false;
    }
    src = ((size_t)sp * p.Hkv + kvh) * kBlock + id % kBlock;
    dst = ((size_t)dp * p.Hkv + kvh) * kBlock + to % kBlock;
    return true;
  };
  if (what == 2) {
    float* mass = p.mass + (size_t)g * p.stride;
    for (int i0 = 0; i0 < n; i0 += kMoveThreads) {
      const int i = i0 + tid;
      size_t src, dst;
      const bool moves = i < n && locate(i, src, dst);
      const float x = moves ? mass[ids[i]] : 0.f;
      __syncthreads();
      if (moves) mass[f + i] = x;
    }
    return;
  }
  const uint4* from = what == 0 ? p.k : p.v;
  uint4* into = what == 0 ? p.dst_k : p.dst_v;
  const int lane = tid % kRowLanes;
  for (int i0 = 0; i0 < n; i0 += kRowsPer * kPasses) {
    uint4 x[kPasses];
    size_t dst[kPasses];
    bool moves[kPasses];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int i = i0 + u * kRowsPer + tid / kRowLanes;
      size_t src;
      moves[u] = i < n && locate(i, src, dst[u]);
      if (moves[u]) x[u] = from[src * kRowLanes + lane];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPasses; ++u)
      if (moves[u]) into[dst[u] * kRowLanes + lane] = x[u];
  }
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
  if (a->new_lens == a->seq_lens || a->new_lens == a->keep_lens || a->new_lens == a->first) return SKV_EINVAL;
  if (a->batch < 1 || a->kv_heads < 1 || a->max_seq_len < 0 || a->num_pages < 1 || a->max_blocks < 0 ||
      a->max_keep < 1)
    return SKV_EINVAL;
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
  p.ordered = !copy || a->mass != nullptr;
  p.status = a->status_word;
  compact_kernel<<<dim3(a->batch * a->kv_heads, a->mass ? 3 : 2), kMoveThreads, 0,
                   reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
