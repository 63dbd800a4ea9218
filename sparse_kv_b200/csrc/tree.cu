// tree.cu -- attention of a tree of drafted tokens over the paged cache.
//
// One warp per row (drafted token, query head): a lane owns four dims of every
// key, the warp walks the row's tokens with an online softmax (running max m,
// sum l, output O).
#include "tree.cuh"

namespace skv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

skv_status tree_params(const skv_tree_args* a, TreeParams* p) {
  if (!a) return SKV_EINVAL;
  if (!a->q || !a->k_pool || !a->block_table || !a->seq_lens || !a->lse) return SKV_EINVAL;
  if (a->batch < 1 || a->q_tokens < 1 || a->q_heads < 1 || a->kv_heads < 1) return SKV_EINVAL;
  if (a->q_heads % a->kv_heads != 0) return SKV_EINVAL;
  if (a->max_seq_len < 0 || a->num_pages < 1 || a->max_blocks < 0) return SKV_EINVAL;
  if (a->head_dim != kHeadDim || a->block_size != kBlock) return SKV_EUNSUPPORTED;
  if ((long long)a->max_blocks * kBlock < (long long)a->max_seq_len) return SKV_EINVAL;
  if (!aligned16(a->q) || !aligned16(a->k_pool)) return SKV_EINVAL;
  if (!isfinite(a->scale) || !isfinite(a->softcap) || a->softcap < 0.f) return SKV_EINVAL;
  if (a->window.sink_tokens < 0 || a->window.recent_tokens < 0) return SKV_EINVAL;
  const int G = a->q_heads / a->kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return SKV_EUNSUPPORTED;
  if (a->q_tokens > kMaxTree) return SKV_EUNSUPPORTED;
  // tile counts and row numbers are 32-bit
  if ((long long)a->batch * a->kv_heads * ((a->max_seq_len + 127ll) / 128) >= (1ll << 30) ||
      (long long)a->batch * a->q_tokens * a->q_heads >= (1ll << 30))
    return SKV_EUNSUPPORTED;
  *p = TreeParams{};
  p->q = static_cast<const uint16_t*>(a->q);
  p->k_pool = static_cast<const uint16_t*>(a->k_pool);
  p->v_pool = static_cast<const uint16_t*>(a->v_pool);
  p->block_table = a->block_table;
  p->seq_lens = a->seq_lens;
  p->tree_lens = a->tree_lens;
  p->tree_mask = reinterpret_cast<const unsigned long long*>(a->tree_mask);
  p->slopes = a->slopes;
  p->B = a->batch;
  p->T = a->q_tokens;
  p->Hq = a->q_heads;
  p->Hkv = a->kv_heads;
  p->G = G;
  p->max_blocks = a->max_blocks;
  p->num_pages = a->num_pages;
  p->max_seq_len = a->max_seq_len;
  p->sink = a->window.sink_tokens;
  p->recent = a->window.recent_tokens;
  p->window = p->sink != 0 || p->recent != 0;
  p->scale = a->scale;
  p->softcap = a->softcap;
  p->out = a->out;
  p->lse = a->lse;
  p->status = a->status_word;
  return SKV_OK;
}

namespace {

constexpr int kRowWarps = 4;

__device__ __forceinline__ float4 bf16x4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

__global__ void __launch_bounds__(kRowWarps * 32) tree_row_kernel(const TreeParams p) {
  const int row = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= p.B * p.T * p.Hq) return;
  const int h = row % p.Hq, t = row / p.Hq % p.T, b = row / p.Hq / p.T, kvh = h / p.G;
  const TreeSeq s = tree_seq(p, b);
  if (s.bad && t == 0 && h == 0 && lane == 0) dev_error(p.status, SKV_DEV_BAD_SEQLEN);
  if (t >= s.n && !s.bad) return;
  const unsigned long long word = tree_word(p, b, t, s.n);
  const int pos = s.ctx + tree_depth(word, t);
  const float4 q = bf16x4(p.q + (size_t)row * kHeadDim + lane * 4);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < s.L; ++i) {
    int at = i;
    if (i >= s.ctx) {
      const int j = i - s.ctx;
      if (!((word >> j) & 1)) continue;
      at = s.ctx + tree_depth(tree_word(p, b, j, s.n), j);
    }
    if (p.window && at >= p.sink && at <= pos - p.recent) continue;
    const int page = p.block_table[(size_t)b * p.max_blocks + i / kBlock];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) dev_error(p.status, SKV_DEV_BAD_PAGE);
      continue;
    }
    const size_t at_kv = (((size_t)page * p.Hkv + kvh) * kBlock + i % kBlock) * kHeadDim + lane * 4;
    const float4 k = bf16x4(p.k_pool + at_kv);
    float z = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int o2 = 16; o2 >= 1; o2 >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o2);
    z *= p.scale;
    if (p.softcap > 0.f) z = p.softcap * tanhf(z / p.softcap);
    if (p.slopes) z += p.slopes[h] * (float)(at - pos);
    const float m2 = fmaxf(m, z);
    const float a = expf(m - m2), w = expf(z - m2);
    const float4 v = bf16x4(p.v_pool + at_kv);
    l = l * a + w;
    o.x = o.x * a + w * v.x;
    o.y = o.y * a + w * v.y;
    o.z = o.z * a + w * v.z;
    o.w = o.w * a + w * v.w;
    m = m2;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<float4*>(p.out + (size_t)row * kHeadDim + lane * 4) =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (lane == 0) p.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace skv

extern "C" {

SKV_API size_t skv_tree_workspace_size(const skv_tree_args* args) {
  skv::TreeParams p;
  if (skv::tree_params(args, &p) != SKV_OK) return 0;
  return 0;
}

SKV_API skv_status attn_tree_decode(const skv_tree_args* a, skv_stream_t stream) {
  using namespace skv;
  TreeParams p;
  const skv_status st = tree_params(a, &p);
  if (st != SKV_OK) return st;
  if (!p.v_pool || !p.out || !aligned16(p.v_pool) || !aligned16(p.out)) return SKV_EINVAL;
  const int rows = p.B * p.T * p.Hq;
  tree_row_kernel<<<(rows + kRowWarps - 1) / kRowWarps, kRowWarps * 32, 0,
                    reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
