// mass.cu -- attention weight received by every cached token, on the tcgen05 tensor
// cores: the rows' scores again, normalised by the log-sum-exp that the attention
// call returned, summed over the rows of each key.
//
//   S^T[128 keys][NR rows] = K . Q^T   (A = K tile, B = Q rows, both K-major)
//   mass[key] += sum over rows of w_r 2^(z_r - lse_r)
// A thread owns a key (a TMEM lane), so the sum over the rows stays in a register:
// no value crosses a thread and each entry is one sum in a fixed order.
//
// All rows of a group (512 at most) stay in shared memory and are taken 128 at a time;
// the tiles of all groups are one list, cut evenly over the CTAs.
//
// Warp roles (20 warps): warp 0 K producer (TMA tensor loads into a ring), warp 1 MMA
// issuer, warps 4-19 four warpgroups that take the tiles in turn, each with a score
// buffer of 128 TMEM columns.  Tiles that a window hides from every row are only decayed.
//
// Bounds (256 bytes of K per token and KV head are read once):
//   few rows   HBM: 16 x 32k tokens x 8 KV heads, 4 rows a group, 181-192 us for 1.1 GB,
//              89-94% of the copy rate (170 where part of K is still in L2)
//   128 rows   HBM and exponentials: 8 x 16k tokens 57 us, 76% of the copy rate
//   256 rows   instruction issue, the MUFU unit and the broadcast reads of the column data
//              from shared memory, none of them full: 4 x 128k tokens 326 us,
//              half the copy rate
// One pass width serves all: 32 or 64 columns for fewer rows were as fast or slower (5% for
// those 4 rows, 3% for 64), and 256, two warpgroups to a tile, 3% slower for 256 rows.
#include <algorithm>

#include "decode.cuh"
#include "tree.cuh"

namespace skv {
namespace {

constexpr int kGroups = 4;                       // warpgroups, and score buffers
constexpr int NR = 128;                          // rows of a pass: columns of a score buffer
constexpr int kMassThreads = 128 + kGroups * 128;
constexpr int kMaxRows = kMaxTree * 8;
constexpr int kMaxStages = 6;
constexpr int kMassFlags = 16;                   // ring of per-tile page flags

struct MassParams {
  const float* row_weight;
  const float* prev;
  float* mass;
  float decay;
  int stride;
  int slots, passes, stages;  // CTAs, row passes of NR, K ring stages
  ScoreFactors f;
};

// shared memory: Q passes, K ring, then the column data and barriers
constexpr size_t kOffCol = 0;                                   // float4 [256], two columns: -lse log2 e of both, weight of both
constexpr size_t kOffSlope = kOffCol + kMaxRows * 8;            // float [512]: slope log2 e
constexpr size_t kOffOffset = kOffSlope + kMaxRows * 4;         // float [512]: -slope * depth
constexpr size_t kOffWords = kOffOffset + kMaxRows * 4;         // u64 [64]
constexpr size_t kOffMassBar = kOffWords + kMaxTree * 8;        // k_full[6], k_empty[6], s_full[4], s_empty[4], q_full, fin
constexpr size_t kOffMassMisc = kOffMassBar + (2 * kMaxStages + 2 * kGroups + 2) * 8;
constexpr size_t kMassFixed = ((kOffMassMisc + 8 + kMassFlags) + 1023) / 1024 * 1024;

// Whether some row may attend a token of the tile at k0.
__device__ __forceinline__ bool tile_needed(const TreeParams& p, const Segment& g, int k0) {
  return g.s.n > 0 && (!p.window || k0 < p.sink || k0 + kKeys > min(g.s.ctx, g.s.ctx + 1 - p.recent));
}

// Whether some tile of a segment has scores.  The needed tiles are the first of a sequence
// (the sink) and the last, so a segment's ends tell.  The sum warps and the issuing thread
// pass over other segments alike: the rows' barrier has one phase per segment with scores,
// and the wait for those scores keeps the sum warps from arriving a second phase ahead of
// the issuing thread.
__device__ __forceinline__ bool scored(const TreeParams& p, const Segment& g) {
  return tile_needed(p, g, g.a * kKeys) || tile_needed(p, g, (g.e - 1) * kKeys);
}

template <int MODE>
__global__ void __launch_bounds__(kMassThreads, 1)
    mass_kernel(const TreeParams p, const MassParams mp, const __grid_constant__ CUtensorMap tmK) {
  extern __shared__ __align__(1024) unsigned char smem[];
  float* col = reinterpret_cast<float*>(smem + kOffCol);
  float* slope = reinterpret_cast<float*>(smem + kOffSlope);
  float* offset = reinterpret_cast<float*>(smem + kOffOffset);
  unsigned long long* words = reinterpret_cast<unsigned long long*>(smem + kOffWords);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + kOffMassBar);
  uint64_t* k_empty = k_full + kMaxStages;
  uint64_t* s_full = k_empty + kMaxStages;
  uint64_t* s_empty = s_full + kGroups;
  uint64_t* q_full = s_empty + kGroups;
  uint64_t* fin = q_full + 1;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffMassMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile unsigned char* page_ok = smem + kOffMassMisc + 8;
  unsigned char* sq = smem + kMassFixed;                               // [passes][2 halves][NR][128 B]
  unsigned char* sk = sq + (size_t)mp.passes * NR * kRowBytes;         // [stages][32 KiB]

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 128);
    }
    mbar_init(q_full, kGroups * 128);
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32((const void*)tmem_slot)),
                 "r"((uint32_t)(kGroups * NR))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
  wait_for_stream();
  int total;
  Walk<true> walk = find_share<true>(p, mp.slots, blockIdx.x, lane, total);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Segment g{};
  int it = 0;    // tiles of the segments before
  int kc = 0;    // tiles with scores so far
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ K producer
    while (__any_sync(0xffffffffu, ok && walk.next(p, g))) {
      const int low = window_low(p, g, lane);
      auto first = [&](int j) {  // of this lane's page, where the batch begins with tile j
        const int tile = j + lane / 2;
        return tile < g.e && tile_needed(p, g, tile * kKeys) ? tile * kKeys + (lane & 1) * kBlock : -1;
      };
      PageBatch batch;
      batch.fetch(p, g, low, first(g.a));
      for (int j0 = g.a; j0 < g.e; j0 += kPageTiles) {
        const int y = batch.row(p, g, true);
        batch.fetch(p, g, low, first(j0 + kPageTiles));
        for (int u = 0; u < min(kPageTiles, g.e - j0); ++u) {
          const int y0 = __shfl_sync(0xffffffffu, y, 2 * u), y1 = __shfl_sync(0xffffffffu, y, 2 * u + 1);
          if (lane != 0 || !ok || !tile_needed(p, g, (j0 + u) * kKeys)) continue;
          const int st = kc % mp.stages, round = kc / mp.stages;
          if (round > 0 && !mbar_wait_bounded(&k_empty[st], (round - 1) & 1, abort_flag)) {
            ok = false;
            continue;
          }
          const int nh = (y0 >= 0) + (y1 >= 0);
          page_ok[kc % kMassFlags] = (unsigned char)((y0 >= 0) | (y1 >= 0) << 1);
          unsigned char* dst = sk + (size_t)st * kTileKV;
          if (nh == 0) {
            mbar_arrive(&k_full[st]);
          } else {
            mbar_arrive_expect_tx(&k_full[st], (uint32_t)nh * 2 * (kBlock * 64 * 2));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if ((h ? y1 : y0) < 0) continue;
#pragma unroll
              for (int d = 0; d < 2; ++d)
                tma_load_2d(dst + d * kHalfTile + h * (kHalfTile / 2), &tmK, d * 64, h ? y1 : y0, &k_full[st]);
            }
          }
          ++kc;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0) {
      if (!ok) {
        dev_error(p.status, SKV_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      // every copy has landed before the CTA may end (at once unless a wait ran out)
      for (int i = max(0, kc - mp.stages); i < kc; ++i)
        mbar_wait_bounded(&k_full[i % mp.stages], (i / mp.stages) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // One thread issues; its arithmetic is a tile's pace where few rows are scored, so
    // ring positions are counted, not divided, and descriptors only moved on (16 x 32k
    // tokens, 4 rows a group: 197 -> 175 us).  With several passes the tiles go in bunches,
    // pass by pass over a bunch, so that the warpgroups' score buffers alternate.
    constexpr uint32_t idesc = instr_desc_bf16(128, NR, false, false);
    const int bunch = mp.passes == 1 ? 1 : min(kGroups, mp.stages);
    uint32_t used = 0;            // bit w: parity of the score tiles given to buffer w
    int ks = 0, kpar = 0, kw = 0; // ring stage, its parity and score buffer of the next tile
    int seg = 0;                  // segments with scores so far
    while (lane == 0 && ok && walk.next(p, g)) {
      if (!scored(p, g)) continue;
      if (!mbar_wait_bounded(q_full, seg++ & 1, abort_flag)) { ok = false; break; }
      const int n = g.e - g.a;
      const int passes = (g.s.n * p.G + NR - 1) / NR;
      for (int j = 0; ok && j < n; j += bunch) {
        int st = ks, par = kpar, w = kw;
        for (int q = 0; ok && q < passes; ++q) {
          st = ks;
          par = kpar;
          w = kw;
          const uint64_t q_desc = smem_desc(smem_u32(sq + (size_t)q * NR * kRowBytes), 16, 1024);
          for (int u = j; u < min(j + bunch, n); ++u) {
            if (p.window && !tile_needed(p, g, (g.a + u) * kKeys)) continue;
            if ((q == 0 && !mbar_wait_bounded(&k_full[st], par, abort_flag)) ||
                !mbar_wait_bounded(&s_empty[w], ((used >> w) & 1) ^ 1, abort_flag)) {
              ok = false;
              break;
            }
            fence_after_sync();
            const uint64_t k_desc = smem_desc(smem_u32(sk + (size_t)st * kTileKV), 16, 1024);
#pragma unroll
            for (int k = 0; k < kHeadDim / 16; ++k)
              mma_bf16(tmem + w * NR, desc_at(k_desc, (k >> 2) * kHalfTile + (k & 3) * 32),
                       desc_at(q_desc, (k >> 2) * (NR * 128) + (k & 3) * 32), idesc, k > 0);
            mma_commit(&s_full[w]);
            if (q == passes - 1) mma_commit(&k_empty[st]);
            used ^= 1u << w;
            if (++w == kGroups) w = 0;
            if (++st == mp.stages) {
              st = 0;
              par ^= 1;
            }
          }
        }
        ks = st;
        kpar = par;
        kw = w;
      }
    }
    if (lane == 0) {
      if (!ok) {
        dev_error(p.status, SKV_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      mma_commit(fin);
      mbar_wait_bounded(fin, 0, nullptr);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    const int wg = (warp - 4) >> 2, st = tid - 128, key = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int lg = __ffs(p.G) - 1;
    uint32_t seen = 0;  // score tiles of this buffer so far
    while (__any_sync(0xffffffffu, walk.next(p, g))) {  // no early exit: the barrier needs every thread
      g.a = uniform(g.a);
      g.e = uniform(g.e);
      g.s.n = uniform(g.s.n);
      g.s.L = uniform(g.s.L);
      g.s.ctx = g.s.L - g.s.n;
      const int rows = g.s.n * p.G, passes = (rows + NR - 1) / NR;
      // ---- Q rows and column data; every score of the segment before has been read
      if (scored(p, g)) {
        asm volatile("bar.sync 1, %0;" ::"n"(kGroups * 128) : "memory");
        // A row that does not count is zero, whatever it holds: its weight 0 would not stop a NaN.
        // One that counts with a NaN lse is NaN itself and its column's lse 0, so that the NaN
        // goes through the mask like any score: to the tokens that the row attends.  Four loads
        // of each kind at a time: with eight, or row by row's state before its query, 1 to 2 us
        // slower for 256 rows (1 x 128k x 64: 91.9 us, 93.6 and 98.3), by more code.
        for (int i0 = st; i0 < passes * NR * 16; i0 += kGroups * 128 * 4) {
          uint4 x[4];
          float lse[4], w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = (i0 + u * kGroups * 128) >> 4, t = r >> lg, h = r & (p.G - 1);
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            lse[u] = -INFINITY;
            w[u] = 1.f;
            if (r < rows) {
              const size_t row = ((size_t)g.b * p.T + t) * p.Hq + (size_t)g.kvh * p.G + h;
              x[u] = reinterpret_cast<const uint4*>(p.q + row * kHeadDim)[i0 & 15];
              lse[u] = p.lse[row];
              if (mp.row_weight) w[u] = mp.row_weight[(size_t)g.b * p.T + t];
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = (i0 + u * kGroups * 128) >> 4, c = i0 & 15;
            if (w[u] == 0.f || lse[u] == -INFINITY) x[u] = make_uint4(0u, 0u, 0u, 0u);
            else if (lse[u] != lse[u]) x[u] = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (r < passes * NR)
              *reinterpret_cast<uint4*>(sq + (size_t)(r / NR) * (NR * kRowBytes) + (c >> 3) * (NR * 128) +
                                        swz(r % NR, c & 7)) = x[u];
          }
        }
        fence_async_smem();
        mbar_arrive(q_full);
        if (st < kMaxTree) words[st] = st < g.s.n ? tree_word(p, g.b, st, g.s.n) : 0ull;
        if (st < passes * NR) {
          const int t = st >> lg, h = st & (p.G - 1);
          float2 x = make_float2(-INFINITY, 0.f);  // 2^-inf: no contribution
          if (st < rows) {
            const float w = mp.row_weight ? mp.row_weight[(size_t)g.b * p.T + t] : 1.f;
            const float lse = p.lse[((size_t)g.b * p.T + t) * p.Hq + (size_t)g.kvh * p.G + h];
            if (w != 0.f && lse != -INFINITY) x = make_float2(lse == lse ? -lse * kLog2e : 0.f, w);
            if (MODE != PLAIN) {
              const float a = p.slopes ? p.slopes[g.kvh * p.G + h] * kLog2e : 0.f;
              slope[st] = a;
              offset[st] = -a * (float)tree_depth(tree_word(p, g.b, t, g.s.n), t);
            }
          } else if (MODE != PLAIN) {
            slope[st] = offset[st] = 0.f;
          }
          col[2 * (st & ~1) + (st & 1)] = x.x;
          col[2 * (st & ~1) + 2 + (st & 1)] = x.y;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kGroups * 128) : "memory");
      }
      const size_t row_mass = ((size_t)g.b * p.Hkv + g.kvh) * mp.stride;
      const int n = g.e - g.a;
      // without a window all tiles have scores, or none: straight to this buffer's
      const bool whole_list = !p.window;
      const int step = whole_list ? kGroups : 1;
      for (int j = whole_list ? (wg - (g.s.n > 0 ? kc : it)) & (kGroups - 1) : 0; j < n; j += step) {
        const int k0 = (g.a + j) * kKeys, kp = k0 + key;
        bool need = g.s.n > 0;
        int slot = (kc + j) % kMassFlags;
        if (!whole_list) {
          need = tile_needed(p, g, k0);
          slot = kc % kMassFlags;
          const int owner = (need ? kc : it + j) % kGroups;
          kc += need;
          if (owner != wg) continue;
        }
        float old = 0.f;
        if (mp.prev && kp < g.s.L) old = mp.prev[row_mass + kp];
        f2 acc[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
        if (need) {
          const int jd = kp - g.s.ctx;  // drafted token, if >= 0
          int place = jd;               // position of the key less ctx
          if (jd >= 0 && jd < g.s.n) place = tree_depth(words[jd], jd);
          bool whole = k0 + kKeys <= g.s.ctx &&
                       (!p.window || k0 + kKeys <= p.sink || k0 > g.s.ctx + g.s.n - 1 - p.recent);
          uint32_t s_lo = 0, s_hi = 0;  // rows that attend the key, where not all do
          for (int q = 0; q < passes; ++q, ++seen) {
            ok &= mbar_wait_bounded(&s_full[wg], seen & 1, abort_flag);
            __syncwarp();
            fence_after_sync();
            if (q == 0) {
              const uint32_t pages = (uint32_t)uniform(page_ok[slot]);
              whole = whole && pages == 3u;
              if (!whole) {
                unsigned long long sees = 0;
                if (kp < g.s.L && ((pages >> (key >> 6)) & 1)) sees = rows_of_key(p, g.s, words, jd, g.s.ctx + place, 0, g.s.n);
                __syncwarp();
                s_lo = (uint32_t)sees;
                s_hi = (uint32_t)(sees >> 32);
              }
            }
            const int cols = min(NR, rows - q * NR);
#pragma unroll 1
            for (int cc = 0; cc < cols; cc += 32) {
              float v[32];
              tmem_ld32(tmem + lanes + wg * NR + cc, v);
              tmem_wait_ld();
              if (cc + 32 >= cols) {  // the buffer may be written again
                fence_before_sync();
                mbar_arrive(&s_empty[wg]);
              }
              const int r0 = q * NR + cc;
              if (MODE != PLAIN) transform<MODE, 32>(v, mp.f, slope + r0, offset + r0, (float)place);
              if (!whole) {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const int t = (r0 + c) >> lg;
                  if (!(((t < 32 ? s_lo : s_hi) >> (t & 31)) & 1)) v[c] = -INFINITY;
                }
              }
              const float qs = MODE == PLAIN ? mp.f.qscale : 1.f;
              const f2 qs2 = pack2(qs, qs);
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const float4 a = *reinterpret_cast<const float4*>(col + 2 * (r0 + c));
                float x0, x1;
                unpack2(fma2(pack2(v[c], v[c + 1]), qs2, pack2(a.x, a.y)), x0, x1);
                if (c == 12) {  // one pair of sixteen beside the MUFU unit: none or two 2% slower, three 6%
                  exp2_fma(x0, x1);
                } else {
                  x0 = ex2(x0);
                  x1 = ex2(x1);
                }
                acc[(c >> 1) & 1] = fma2(pack2(x0, x1), pack2(a.z, a.w), acc[(c >> 1) & 1]);
              }
            }
          }
        }
        float s0, s1, s2, s3;
        unpack2(acc[0], s0, s1);
        unpack2(acc[1], s2, s3);
        float sum = (s0 + s1) + (s2 + s3);
        if (kp < g.s.L) mp.mass[row_mass + kp] = mp.prev ? fmaf(mp.decay, old, sum) : sum;
      }
      it += n;
      if (whole_list && g.s.n > 0) kc += n;
    }
    if (!ok) {
      dev_error(p.status, SKV_DEV_TIMEOUT);
      *abort_flag = 1;
    }
  } else if (warp == 3 && blockIdx.x == 0) {
    for (int b = lane; b < p.B; b += 32)
      if (tree_seq(p, b).bad) dev_error(p.status, SKV_DEV_BAD_SEQLEN);
  }
  // ---- teardown: free TMEM once every role is through
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)(kGroups * NR))
                 : "memory");
}

template <int MODE>
cudaError_t launch_mass(const TreeParams& p, const MassParams& mp, size_t smem, const CUtensorMap& tk, cudaStream_t s) {
  static std::atomic<bool> attr_set[64];  // per device; racing first calls only repeat the set-up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(mass_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  return launch_early(mass_kernel<MODE>, mp.slots, kMassThreads, smem, s, p, mp, tk);
}

cudaError_t launch_mass(const TreeParams& p, MassParams& mp, const CUtensorMap& tk, cudaStream_t s) {
  mp.passes = (p.T * p.G + NR - 1) / NR;
  const size_t q_bytes = (size_t)mp.passes * NR * kRowBytes;
  mp.stages = (int)std::min<size_t>(kMaxStages, (227 * 1024 - kMassFixed - q_bytes) / kTileKV);
  const size_t smem = kMassFixed + q_bytes + (size_t)mp.stages * kTileKV;
  const int mode = score_mode(p);
  if (mode == CAP) return launch_mass<CAP>(p, mp, smem, tk, s);
  if (mode == BIAS) return launch_mass<BIAS>(p, mp, smem, tk, s);
  return launch_mass<PLAIN>(p, mp, smem, tk, s);
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
  MassParams mp{};
  mp.row_weight = row_weight;
  mp.prev = prev;
  mp.mass = mass;
  mp.decay = decay;
  mp.stride = mass_stride;
  mp.f = score_factors(p);
  mp.slots = (int)std::min<long long>(num_sms(), std::max(1ll, (long long)p.B * p.Hkv * ((p.max_seq_len + 127) / 128)));
  CUtensorMap tk;
  if (!make_pool_map(&tk, p.k_pool, (long long)p.num_pages * p.Hkv * kBlock)) return SKV_ECUDA;
  return launch_mass(p, mp, tk, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
