// mass.cu -- attention weight received by every cached token (the rows' scores
// again, normalised by the log-sum-exp the attention call returned).
//
// One warp per (sequence, KV head, token): a lane owns four dims of the key and
// the warp walks the rows in order, so each entry is one sum in a fixed order.
#include "tree.cuh"

namespace skv {
namespace {

constexpr int kKeyWarps = 8;

struct MassParams {
  const float* row_weight;
  const float* prev;
  float* mass;
  float decay;
  int stride;
};

__device__ __forceinline__ float4 bf16x4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

__global__ void __launch_bounds__(kKeyWarps * 32) key_mass_kernel(const TreeParams p, const MassParams mp) {
  const int lane = threadIdx.x & 31, kvh = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv;
  const int i = blockIdx.x * kKeyWarps + (threadIdx.x >> 5);
  const TreeSeq s = tree_seq(p, b);
  if (s.bad && kvh == 0 && blockIdx.x == 0 && threadIdx.x == 0) dev_error(p.status, SKV_DEV_BAD_SEQLEN);
  if (i >= s.L) return;
  const size_t at_mass = ((size_t)b * p.Hkv + kvh) * mp.stride + i;
  const int page = p.block_table[(size_t)b * p.max_blocks + i / kBlock];
  const bool ok = page >= 0 && page < p.num_pages;
  const int j = i - s.ctx;
  const int at = j < 0 ? i : s.ctx + tree_depth(tree_word(p, b, j, s.n), j);
  float4 k = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ok) k = bf16x4(p.k_pool + (((size_t)page * p.Hkv + kvh) * kBlock + i % kBlock) * kHeadDim + lane * 4);
  float sum = 0.f;
  bool seen = false;
  for (int t = 0; t < s.n; ++t) {
    const unsigned long long word = tree_word(p, b, t, s.n);
    const int pos = s.ctx + tree_depth(word, t);
    if (j >= 0 && !((word >> j) & 1)) continue;
    if (p.window && at >= p.sink && at <= pos - p.recent) continue;
    seen = true;
    const float w = mp.row_weight ? mp.row_weight[(size_t)b * p.T + t] : 1.f;
    if (!ok || w == 0.f) continue;
    for (int g = 0; g < p.G; ++g) {
      const size_t row = ((size_t)b * p.T + t) * p.Hq + (size_t)kvh * p.G + g;
      const float4 q = bf16x4(p.q + row * kHeadDim + lane * 4);
      float z = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      z *= p.scale;
      if (p.softcap > 0.f) z = p.softcap * tanhf(z / p.softcap);
      if (p.slopes) z += p.slopes[kvh * p.G + g] * (float)(at - pos);
      const float lse = p.lse[row];
      if (lse != -INFINITY) sum += w * expf(z - lse);
    }
  }
  if (lane != 0) return;
  if (!ok && seen) dev_error(p.status, SKV_DEV_BAD_PAGE);
  mp.mass[at_mass] = (mp.prev ? mp.decay * mp.prev[at_mass] : 0.f) + sum;
}

}  // namespace
}  // namespace skv

extern "C" {

SKV_API skv_status attn_key_mass(const skv_tree_args* a, const float* row_weight, const float* prev,
                                 float decay, int mass_stride, float* mass, skv_stream_t stream) {
  using namespace skv;
  TreeParams p;
  const skv_status st = tree_params(a, &p);
  if (st != SKV_OK) return st;
  if (!mass || !isfinite(decay) || mass_stride < p.max_seq_len) return SKV_EINVAL;
  if ((long long)p.B * p.Hkv > 65535) return SKV_EUNSUPPORTED;
  if (p.max_seq_len == 0) return SKV_OK;
  const MassParams mp{row_weight, prev, mass, decay, mass_stride};
  key_mass_kernel<<<dim3((p.max_seq_len + kKeyWarps - 1) / kKeyWarps, p.B * p.Hkv), kKeyWarps * 32, 0,
                    reinterpret_cast<cudaStream_t>(stream)>>>(p, mp);
  return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
