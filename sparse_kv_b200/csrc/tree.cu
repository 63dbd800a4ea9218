// tree.cu -- attention of a tree of drafted tokens over the paged cache, on the
// tcgen05 tensor cores.
//
// A KV group's G query heads and the T drafted tokens form R = T*G rows (row r =
// token r / G, head r % G).  A CTA serves NR of them (32, 64 or 128) against a
// run of 128-key tiles, with the keys along the M side of both products:
//   S^T[128 keys][NR]      = K . Q^T            A = K tile (K-major), B = Q rows
//   O^T[128 dims][2 NR]   += V^T . [P_hi | P_lo]  A = V tile (MN-major), B = P
// so the tensor work shrinks with the number of rows, an output dim is a TMEM
// lane (coalesced stores) and V is read once for both bf16 terms of the weights
// (P = hi + lo keeps 16 significant bits; the halves of O^T are added at the end).
//
// Warp roles:
//   warp 0      K producer: TMA tensor loads (128B swizzle) of 64-key pages into a ring
//   warp 1      MMA: allocates 4 NR TMEM columns (two S buffers, O hi, O lo) and issues
//   warp 2      V producer
//   warp 3      rows: Q (one TMA load per dim half), masks and slopes of the next segment
//               into a second buffer (one buffer for 128 rows), so that its first S runs
//               under the last segment's epilogue
//   warps 4-    softmax: two warpgroups (four for 128 rows), each for its share of the
//               columns, 32 at most (scores and partial sums stay in registers); a
//               thread owns one key.  The running maximum m of a column is kept until
//               some score of the tile passes it by 2^8 (a vote of the warpgroup); only
//               then the maxima are reduced over the keys and O and l rescaled, so in the
//               usual tile no value crosses a thread.  P goes to shared memory as the
//               MN-major B operand.
// A CTA walks its run from the newest tile to the oldest, so that under a distance bias
// the maxima come first.  The tiles of all KV groups are one list, cut evenly over the
// CTAs; a group that is cut leaves partial records (O unnormalised, m, l) in the
// workspace, and a second kernel merges them.  Row tiles beyond 128 rows go to
// neighbouring CTAs that walk the same tiles at the same time, so K and V come from DRAM
// once.
//
// Bounds (512 bytes of K and V per token and KV head; 32 heads, 8 KV heads):
//   16 x 32k tokens, 64 rows a group   HBM: 344-360 us in bursts, 92-97% of the copy rate;
//              396-428 when repeated for seconds, at the power limit
//   4 x 128k tokens, 256 rows a group  866-908 us, 38% of the copy rate: the chain scores ->
//              weights -> P.V, 3,300 clocks a tile of 128 rows, of which the products with
//              both bf16 terms of P need 1,960
//   1 x 4k tokens, 8 drafted           10.7 us: launch, barrier set-up, one tile's chain
//              and the merge launch; the bytes alone are 0.7 us
#include <cuda_bf16.h>

#include <algorithm>

#include "decode.cuh"
#include "tcgen.cuh"
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
  // in base 2 too, as the scores are taken
  if (!isfinite(a->scale * kLog2e) || !isfinite(a->softcap * kLog2e) || a->softcap < 0.f) return SKV_EINVAL;
  if (a->softcap > 0.f && !isfinite(2.f * kLog2e * a->scale / a->softcap)) return SKV_EINVAL;
  if (a->window.sink_tokens < 0 || a->window.recent_tokens < 0) return SKV_EINVAL;
  const int G = a->q_heads / a->kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return SKV_EUNSUPPORTED;
  if (a->q_tokens > kMaxTree) return SKV_EUNSUPPORTED;
  // positions, tile counts and row numbers are 32-bit
  if (a->max_seq_len > (1 << 30) ||
      (long long)a->batch * a->kv_heads * ((a->max_seq_len + 127ll) / 128) >= (1ll << 30) ||
      (long long)a->batch * a->q_tokens * a->q_heads >= (1ll << 30) ||
      (long long)a->num_pages * a->kv_heads * kBlock >= (1ll << 31))
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

constexpr float kUnseen = -1e30f;             // maximum of no record
constexpr int kPageFlags = 8;                 // ring of per-tile page flags
// Tiles whose P.V accumulate in tensor memory.  The tensor core cuts its fp32 sums instead
// of rounding them, an error that grows with the length of the chain (relative 6e-5 after
// 443 tiles); every 32 tiles the sums move to the record of the segment, with rounded
// additions (4e-6).
constexpr int kFlush = 32;

template <int NR>
struct TreeCfg {
  static constexpr int NWG = NR == 128 ? 4 : 2;         // softmax warpgroups
  static constexpr int NC = NR / NWG;                   // columns of a warpgroup
  static constexpr int SOFT = NWG * 128;                // softmax threads
  static constexpr int THREADS = 128 + SOFT;
  static constexpr int KS = NR == 128 ? 2 : 3;          // K ring stages
  static constexpr int VS = 2;                          // V ring stages
  static constexpr int PB = NR == 32 ? 2 : 1;           // P buffers
  static constexpr int QB = NR == 128 ? 1 : 2;          // buffers of a segment's rows
  static constexpr int P_ATOMS = 2 * NR / 64;           // 64-column atoms of [P_hi | P_lo]
  static constexpr size_t Q_BYTES = (size_t)NR * 256;
  static constexpr size_t P_BYTES = (size_t)P_ATOMS * kHalfTile;
  static constexpr size_t OFF_Q = 0;
  static constexpr size_t OFF_P = OFF_Q + QB * Q_BYTES;
  static constexpr size_t OFF_K = OFF_P + PB * P_BYTES;
  static constexpr size_t OFF_V = OFF_K + (size_t)KS * kTileKV;
  static constexpr size_t OFF_NM = OFF_V + (size_t)VS * kTileKV;  // float [NR]: -m
  static constexpr size_t OFF_CA = OFF_NM + NR * 4;               // float [NR]: growth of m; at the end 1 / l
  static constexpr size_t OFF_SLOPE = OFF_CA + NR * 4;            // float [NR]: slope * log2 e
  static constexpr size_t OFF_OFFSET = OFF_SLOPE + NR * 4;        // float [NR]: -slope * depth
  static constexpr size_t OFF_ROWS = OFF_OFFSET + NR * 4;         // [QB]: u64 [64] mask words, float [8] slopes
  static constexpr size_t ROWS_BYTES = 64 * 8 + 8 * 4;
  static constexpr size_t OFF_BAR = OFF_ROWS + QB * ROWS_BYTES;
  // k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], s_full[2], p_full[2][2], o_half[2], o_done[2], q_full[QB],
  // q_free[QB], fin
  static constexpr int NBAR = 2 * KS + 2 * VS + 2 * QB + 11;
  static constexpr size_t OFF_MISC = OFF_BAR + NBAR * 8;  // tmem slot, abort flag; page flags; unseen columns
  static constexpr size_t BYTES = OFF_MISC + 8 + kPageFlags + 4 * NWG;
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
  static_assert(NR >= 32 && OFF_BAR % 8 == 0 && OFF_P % 1024 == 0, "layout");
};

struct TreeLaunch {
  int m_tiles;     // row tiles; CTA c serves row tile c % m_tiles
  int slots;       // CTAs per row tile
  ScoreFactors f;
  int4* starts;    // [slots + 1]: where each share begins: sequence, KV head, tile, the group's
                   // tiles; then the total
  int4* groups;    // NULL (more groups than shares) or [groups]: first tile, tiles, slot of the first record
  float* rec;      // [2 * slots][m_tiles][NR * 130]: O [NR][128], m [NR], l [NR]
};

__device__ __forceinline__ bool bar_any(int id, bool pred) {  // vote over a warpgroup
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id)
      : "memory");
  return __any_sync(0xffffffffu, r != 0);
}
__device__ __forceinline__ void bar_wg(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}

// Q of a segment's rows: tensor [B * T][Hq][128], box [NR / G][G][64], rows in (token,
// head) order
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, int x, int head, int token,
                                              uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token), "r"(smem_u32(bar))
      : "memory");
}

template <int NR, int MODE>
__global__ void __launch_bounds__(TreeCfg<NR>::THREADS, 1)
    tree_kernel(const TreeParams p, const TreeLaunch L, const __grid_constant__ CUtensorMap tmQ,
                const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = TreeCfg<NR>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_empty = k_full + C::KS;
  uint64_t* v_full = k_empty + C::KS;
  uint64_t* v_empty = v_full + C::VS;
  uint64_t* s_full = v_empty + C::VS;  // [2]: S of tiles with it & 1 == i is in TMEM
  uint64_t* p_full = s_full + 2;       // [2][2]: P of keys 0-63, 64-127 of those tiles is written
  uint64_t* o_half = p_full + 4;       // [2]: P.V over keys 0-63 of those tiles has run
  uint64_t* o_done = o_half + 2;       // [2]: P.V of those tiles has run
  uint64_t* q_full = o_done + 2;       // [QB]: a segment's rows are in shared memory
  uint64_t* q_free = q_full + C::QB;   // [QB]: the softmax warps are through with them
  uint64_t* fin = q_free + C::QB;      // every MMA issued has run
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile unsigned char* page_ok = smem + C::OFF_MISC + 8;  // [kPageFlags]: bit h: page h of tile it & 7

  // Values that a whole warp shares go through a lane-0 shuffle or a vote, so that the
  // compiler knows the branches on them as uniform, and the warps converge after every
  // wait: warp-wide instructions of a warp that had drifted apart took ten times longer.
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int m_tile = blockIdx.x % L.m_tiles, worker = blockIdx.x / L.m_tiles;

  if (tid == 0) {
    for (int i = 0; i < C::KS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::VS; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], C::SOFT / 2);
      mbar_init(&p_full[2 * i + 1], C::SOFT / 2);
      mbar_init(&o_half[i], 1);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < C::QB; ++i) {
      mbar_init(&q_full[i], 2);  // with the TMA loads, and once the masks are written
      mbar_init(&q_free[i], C::SOFT / 32);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32((const void*)misc)),
                 "r"((uint32_t)(4 * NR))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &tmK : lane == 1 ? &tmV : &tmQ))
                 : "memory");
  wait_for_stream();
  int total;
  Walk<false> walk = find_share<false>(p, L.slots, worker, lane, total);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = misc[0];
  Segment g{};
  int it = 0;   // tiles of this CTA so far
  int seg = 0;  // segments so far
  // 640 threads start with 96 registers each: 128 x 64 + 512 x 104 of those 61,440
  if constexpr (NR == 128) {
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  auto skipped = [&] { return m_tile * NR >= g.s.n * p.G; };  // no row of this row tile

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers
    const bool is_k = warp == 0;
    const int stages = is_k ? C::KS : C::VS;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    unsigned char* ring = smem + (is_k ? C::OFF_K : C::OFF_V);
    const CUtensorMap* map = is_k ? &tmK : &tmV;
    int st = 0, round = 0;
    bool ok = true;
    while (__any_sync(0xffffffffu, ok && walk.next(p, g))) {
      if (skipped()) continue;
      const int low = window_low(p, g, lane);
      auto first = [&](int j) {  // of this lane's page, where the batch begins with tile j
        const int tile = j - lane / 2;
        return tile >= g.a ? tree_tile_start(g.t, tile) + (lane & 1) * kBlock : -1;
      };
      PageBatch batch;
      batch.fetch(p, g, low, first(g.e - 1));
      for (int j0 = g.e - 1; j0 >= g.a; j0 -= kPageTiles) {
        const int y = batch.row(p, g, is_k);
        batch.fetch(p, g, low, first(j0 - kPageTiles));
        for (int u = 0; u < min(kPageTiles, j0 - g.a + 1); ++u) {
          const int y0 = __shfl_sync(0xffffffffu, y, 2 * u), y1 = __shfl_sync(0xffffffffu, y, 2 * u + 1);
          if (lane != 0 || !ok) continue;
          if (round > 0 && !mbar_wait_bounded(&empty[st], (round - 1) & 1, abort_flag)) {
            ok = false;
            continue;
          }
          const int nh = (y0 >= 0) + (y1 >= 0);
          if (is_k) page_ok[it % kPageFlags] = (unsigned char)((y0 >= 0) | (y1 >= 0) << 1);
          unsigned char* dst = ring + (size_t)st * kTileKV;
          if (nh == 0) {
            mbar_arrive(&full[st]);
          } else {
            mbar_arrive_expect_tx(&full[st], (uint32_t)nh * 2 * (kBlock * 64 * 2));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if ((h ? y1 : y0) < 0) continue;
#pragma unroll
              for (int d = 0; d < 2; ++d)
                tma_load_2d(dst + d * kHalfTile + h * (kHalfTile / 2), map, d * 64, h ? y1 : y0, &full[st]);
            }
          }
          ++it;
          if (++st == stages) {
            st = 0;
            ++round;
          }
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
      for (int i = max(0, it - stages); i < it; ++i)
        mbar_wait_bounded(&full[i % stages], (i / stages) & 1, nullptr);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ rows
    bool ok = true;
    int at = 0;  // tiles of the segments before
    if (m_tile == 0 && lane == 0) {  // for the merge
      if (walk.left > 0)
        L.starts[worker] = make_int4(walk.b, walk.kvh, walk.a, list_tiles<false>(p, tree_seq(p, walk.b)).count);
      if (worker == 0) L.starts[L.slots] = make_int4(total, 0, 0, 0);
    }
    while (__any_sync(0xffffffffu, ok && walk.next(p, g))) {
      if (skipped()) continue;
      const int buf = seg % C::QB, round = seg / C::QB;
      ++seg;
      if (round > 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&q_free[buf], (round - 1) & 1, abort_flag));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[buf], (uint32_t)C::Q_BYTES);
        unsigned char* dst = smem + C::OFF_Q + buf * C::Q_BYTES;
        const int token = g.b * p.T + m_tile * (NR / p.G);
        tma_load_rows(dst, &tmQ, 0, g.kvh * p.G, token, &q_full[buf]);
        tma_load_rows(dst + C::Q_BYTES / 2, &tmQ, 64, g.kvh * p.G, token, &q_full[buf]);
        if (L.groups && m_tile == 0 && g.a == 0)  // for the merge: the group's first tile and slot
          L.groups[g.b * p.Hkv + g.kvh] = make_int4(share_begin(worker, total, tree_workers(L.slots, total)) + at,
                                                    g.t.count, seg > 1 ? 1 : 0, 0);
      }
      at += g.e - g.a;
      __syncwarp();
      unsigned char* rows = smem + C::OFF_ROWS + buf * C::ROWS_BYTES;
      unsigned long long* words = reinterpret_cast<unsigned long long*>(rows);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = lane + u * 32;
        words[t] = t < g.s.n ? tree_word(p, g.b, t, g.s.n) : 0ull;
      }
      if (lane < p.G)
        reinterpret_cast<float*>(rows + 64 * 8)[lane] = p.slopes ? p.slopes[g.kvh * p.G + lane] * kLog2e : 0.f;
      __syncwarp();
      mbar_arrive_if(&q_full[buf], lane == 0);
    }
    if (lane == 0) {
      if (!ok) {
        dev_error(p.status, SKV_DEV_TIMEOUT);
        *abort_flag = 1;
        --seg;  // that one was not issued
      }
      for (int i = max(0, seg - C::QB); i < seg; ++i)
        mbar_wait_bounded(&q_full[i % C::QB], (i / C::QB) & 1, nullptr);
    }
    // rows of sequences with bad lengths attend nothing
    __syncwarp();
    if (m_tile == 0)
      for (int b = worker; b < p.B; b += L.slots)
        if (tree_seq(p, b).bad) {
          if (lane == 0) dev_error(p.status, SKV_DEV_BAD_SEQLEN);
          const size_t r0 = (size_t)b * p.T * p.Hq;
          for (int i = lane; i < p.T * p.Hq; i += 32) p.lse[r0 + i] = -INFINITY;
          for (int i = lane; i < p.T * p.Hq * (kHeadDim / 4); i += 32)
            reinterpret_cast<float4*>(p.out + r0 * kHeadDim)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = instr_desc_bf16(128, NR, false, false);
    constexpr uint32_t idesc_o = instr_desc_bf16(128, 2 * NR, true, true);
    int ks = 0, kround = 0, vs = 0, vround = 0;
    bool ok = true;
    // S of one tile
    auto issue_s = [&](int i, int buf) {
      if (!mbar_wait_bounded(&k_full[ks], kround & 1, abort_flag)) return false;
      fence_after_sync();
      const uint64_t k_desc = smem_desc(smem_u32(smem + C::OFF_K + (size_t)ks * kTileKV), 16, 1024);
      const uint64_t q_desc = smem_desc(smem_u32(smem + C::OFF_Q + buf * C::Q_BYTES), 16, 1024);
#pragma unroll
      for (int k = 0; k < kHeadDim / 16; ++k)
        mma_bf16(tmem + (i & 1) * NR, desc_at(k_desc, (k >> 2) * kHalfTile + (k & 3) * 32),
                 desc_at(q_desc, (k >> 2) * (NR * 128) + (k & 3) * 32), idesc_s, k > 0);
      mma_commit(&s_full[i & 1]);
      mma_commit(&k_empty[ks]);
      if (++ks == C::KS) {
        ks = 0;
        ++kround;
      }
      return true;
    };
    // The first S of a segment is issued behind the last P.V of the one before: it runs
    // under the epilogue.
    auto begin = [&]() {  // the next segment with rows of this row tile, its first S issued
      while (walk.next(p, g)) {
        if (skipped()) continue;
        const int buf = seg % C::QB, round = seg / C::QB;
        ++seg;
        ok = mbar_wait_bounded(&q_full[buf], round & 1, abort_flag) && issue_s(it, buf);
        return ok;
      }
      return false;
    };
    bool more = lane == 0 && begin();
    while (more) {
      const int n = g.e - g.a, buf = (seg - 1) % C::QB;
      more = false;
      for (int j = 0; ok && j < n; ++j, ++it) {
        if (j + 1 < n) {
          if (!issue_s(it + 1, buf)) { ok = false; break; }
        }
        // P.V in two halves of the keys, each as soon as its P is there
        if (!mbar_wait_bounded(&v_full[vs], vround & 1, abort_flag)) { ok = false; break; }
        const uint64_t v_desc = smem_desc(smem_u32(smem + C::OFF_V + (size_t)vs * kTileKV), kHalfTile, 1024);
        const uint64_t p_desc = smem_desc(smem_u32(smem + C::OFF_P + (size_t)(it % C::PB) * C::P_BYTES), kHalfTile, 1024);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait_bounded(&p_full[2 * (it & 1) + half], (it >> 1) & 1, abort_flag)) { ok = false; break; }
          fence_after_sync();
#pragma unroll
          for (int k = half * (kKeys / 32); k < (half + 1) * (kKeys / 32); ++k)
            mma_bf16(tmem + 2 * NR, desc_at(v_desc, k * 2048), desc_at(p_desc, k * 2048), idesc_o,
                     j % kFlush > 0 || k > 0);
          if (half == 0) mma_commit(&o_half[it & 1]);
        }
        if (!ok) break;
        mma_commit(&o_done[it & 1]);
        mma_commit(&v_empty[vs]);
        if (++vs == C::VS) {
          vs = 0;
          ++vround;
        }
      }
      if (ok) more = begin();
    }
    if (lane == 0) {
      if (!ok) {
        dev_error(p.status, SKV_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      mma_commit(fin);
      mbar_wait_bounded(fin, 0, nullptr);
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (NR == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    constexpr int NC = C::NC;
    const int wg = (warp - 4) >> 2;
    const int key = tid & 127;                          // key of the tile = TMEM lane
    const int c0 = wg * NC;                             // first column
    const int bar_id = 1 + wg;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    float* nm = reinterpret_cast<float*>(smem + C::OFF_NM) + c0;
    float* ca = reinterpret_cast<float*>(smem + C::OFF_CA) + c0;
    float* slope = reinterpret_cast<float*>(smem + C::OFF_SLOPE) + c0;
    float* offset = reinterpret_cast<float*>(smem + C::OFF_OFFSET) + c0;
    volatile uint32_t* unseen_of = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 8 + kPageFlags) + wg;
    const int lg = __ffs(p.G) - 1;                      // G is a power of two
    const int row0 = m_tile * NR;
    bool ok = true;  // no early exit: the barriers below need every thread
    // Scratch inside tile i's P buffer: float (k, c) of this warpgroup, in the 16-byte
    // chunks of key row k that the warpgroup fills itself.
    auto scratch = [&](int i, int k, int c) {
      const int q = c >> 2, n = c0 + 8 * (q % (NC / 8)) + (q >= NC / 8 ? NR : 0);
      return reinterpret_cast<float*>(smem + C::OFF_P + (size_t)(i % C::PB) * C::P_BYTES + (n >> 6) * kHalfTile +
                                      swz(k, (n & 63) >> 3)) + (c & 3);
    };
    // x[c] combined over the keys of the tile, for column `key` in thread key < NC: through
    // the scratch, NC keys a thread and then 128 / NC partial results.  (Under the vote's
    // branch a shuffle took 235 clocks, a column's reduction over the warp 3,800.)
    auto over_keys = [&](int i, const float* x, bool largest) {
#pragma unroll
      for (int c = 0; c < NC; c += 4)
        *reinterpret_cast<float4*>(scratch(i, key, c)) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
      bar_wg(bar_id);
      const int part = key / NC, c = key % NC;
      float r = *scratch(i, part * NC, c);
#pragma unroll
      for (int k = 1; k < NC; ++k) {
        const float y = *scratch(i, part * NC + k, c);
        r = largest ? fmaxf(r, y) : r + y;
      }
      bar_wg(bar_id);
      *scratch(i, part, c) = r;
      bar_wg(bar_id);
#pragma unroll
      for (int k = 1; k < 128 / NC; ++k) {
        const float y = *scratch(i, k, c);
        r = largest ? fmaxf(r, y) : r + y;
      }
      return r;
    };
    for (bool first = true; __any_sync(0xffffffffu, walk.next(p, g)); first = false) {
      g.a = uniform(g.a);
      g.e = uniform(g.e);
      g.s.n = uniform(g.s.n);
      g.s.L = uniform(g.s.L);
      g.s.ctx = g.s.L - g.s.n;
      const int rows = g.s.n * p.G - row0;  // valid rows of this row tile
      if (rows <= 0) continue;
      // ---- column data of the segment
      const int buf = seg % C::QB;
      ok &= mbar_wait_bounded(&q_full[buf], (seg / C::QB) & 1, abort_flag);
      ++seg;
      __syncwarp();
      const unsigned long long* words = reinterpret_cast<const unsigned long long*>(smem + C::OFF_ROWS + buf * C::ROWS_BYTES);
      if (key < NC) {
        nm[key] = 0.f;
        if (MODE != PLAIN) {
          const int r = row0 + c0 + key, t = r >> lg;
          const float a = reinterpret_cast<const float*>(words + 64)[r & (p.G - 1)];
          slope[key] = a;
          offset[key] = t < g.s.n ? -a * (float)tree_depth(words[t], t) : 0.f;
        }
      }
      __syncwarp();
      bar_wg(bar_id);
      // columns that have seen no key yet: their m is unset
      uint32_t unseen = rows - c0 >= NC ? (NC == 32 ? ~0u : (1u << (NC & 31)) - 1u) : (1u << max(rows - c0, 0)) - 1u;
      f2 l2[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) l2[c] = pack2(0.f, 0.f);
      const int n = g.e - g.a;
      // this thread's place in the segment's record: column c of dim `key` is at [c * 128].
      // (Worked out where it is needed: kept in registers it costs spills at 128 rows.)
      auto record = [&] {
        int slot = 2 * worker + (first ? 0 : 1);
        asm volatile("" : "+r"(slot));
        return L.rec + ((size_t)slot * L.m_tiles + m_tile) * (NR * 130) + (size_t)c0 * kHeadDim + key;
      };
      for (int j = 0; j < n; ++j) {
        const int i = it + j;
        const int k0 = tree_tile_start(g.t, g.e - 1 - j), kp = k0 + key;
        if (j > 0 && j % kFlush == 0) {  // the sums so far to the record; the next P.V starts afresh
          ok &= mbar_wait_bounded(&o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          fence_after_sync();
          float* rec_o = record();
#pragma unroll 1
          for (int c = 0; c < NC; c += 16) {
            float o[16], o2[16];
            tmem_ld16(tmem + lanes + 2 * NR + c0 + c, o);
            tmem_ld16(tmem + lanes + 3 * NR + c0 + c, o2);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] += o2[x];
            if (j > kFlush) {
#pragma unroll
              for (int x = 0; x < 16; ++x) o2[x] = rec_o[(c + x) * kHeadDim];
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] += o2[x];
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) rec_o[(c + x) * kHeadDim] = o[x];
          }
          // The product over keys 0-63 writes all 128 lanes of O and waits only for the threads of
          // those keys: they know through a barrier between two fences that the other lanes are
          // read (here) or rescaled (below).
          fence_before_sync();
          bar_wg(bar_id);
          fence_after_sync();
        }
        ok &= mbar_wait_bounded(&s_full[i & 1], (i >> 1) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        fence_after_sync();
        float v[NC];
#pragma unroll
        for (int c = 0; c < NC; c += 16) tmem_ld16(tmem + lanes + (i & 1) * NR + c0 + c, v + c);
        const uint32_t pages = (uint32_t)uniform(page_ok[i % kPageFlags]);
        tmem_wait_ld();
        // ---- scores in base 2 (PLAIN: times qscale below)
        const int jd = kp - g.s.ctx;  // drafted token, if >= 0
        int place = jd;               // position of the key less ctx
        if (jd >= 0 && jd < g.s.n) place = tree_depth(words[jd], jd);
        if (MODE != PLAIN) transform<MODE, NC>(v, L.f, slope, offset, (float)place);
        // ---- which rows attend this key: all of them, unless the tile touches the
        // drafted tokens, the sequence's end, a window's edge or a missing page
        const bool whole = k0 + kKeys <= g.s.ctx && pages == 3u &&
                           (!p.window || k0 + kKeys <= p.sink || k0 > g.s.ctx + g.s.n - 1 - p.recent);
        if (!whole) {
          const int t0 = row0 >> lg, t1 = min(g.s.n, (row0 + NR - 1 >> lg) + 1);
          unsigned long long sees = 0;
          if (kp < g.s.L && ((pages >> (key >> 6)) & 1)) sees = rows_of_key(p, g.s, words, jd, g.s.ctx + place, t0, t1);
          __syncwarp();
          const uint32_t s_lo = (uint32_t)sees, s_hi = (uint32_t)(sees >> 32);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int t = (row0 + c0 + c) >> lg;
            if (!(((t < 32 ? s_lo : s_hi) >> (t & 31)) & 1)) v[c] = -INFINITY;
          }
          // a V row that no row attends may hold anything: 0 * it must stay 0
          ok &= mbar_wait_bounded(&v_full[i % C::VS], (i / C::VS) & 1, abort_flag);
          if (sees == 0) {
            unsigned char* sv = smem + C::OFF_V + (size_t)(i % C::VS) * kTileKV;
#pragma unroll
            for (int c = wg * (16 / C::NWG); c < (wg + 1) * (16 / C::NWG); ++c)
              *reinterpret_cast<uint4*>(sv + (c >> 3) * kHalfTile + swz(key, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
        // ---- v = z - m; does some score pass its column's maximum by 2^8?
        {
          const float qs = MODE == PLAIN ? L.f.qscale : 1.f;
          const f2 q2 = pack2(qs, qs);
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(nm + c);
            f2 a = pack2(m4.x, m4.y), b = pack2(m4.z, m4.w);
            if (MODE == PLAIN) {
              ffma2(a, pack2(v[c], v[c + 1]), q2);
              ffma2(b, pack2(v[c + 2], v[c + 3]), q2);
            } else {
              a = fadd2(a, pack2(v[c], v[c + 1]));
              b = fadd2(b, pack2(v[c + 2], v[c + 3]));
            }
            unpack2(a, v[c], v[c + 1]);
            unpack2(b, v[c + 2], v[c + 3]);
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; c += 4) top = fmaxf(top, fmaxf(fmaxf(v[c], v[c + 1]), fmaxf(v[c + 2], v[c + 3])));
        if (bar_any(bar_id, top > 8.f || unseen != 0u)) {
          // every P.V issued so far has run: O may be rescaled, and this tile's P buffer
          // serves as scratch (only the 16-byte chunks that this warpgroup fills itself)
          if (i > 0) {
            ok &= mbar_wait_bounded(&o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            fence_after_sync();
          }
          const float top_c = over_keys(i, v, true);
          if (warp == 4 * wg + 4) {  // one warp holds every column
            const bool new_c = key < NC && ((unseen >> (key & 31)) & 1);
            // a column's first maximum may lie anywhere; later ones only grow
            const float d = new_c ? (top_c == -INFINITY ? 0.f : top_c) : fmaxf(top_c, 0.f);
            const uint32_t still = __ballot_sync(0xffffffffu, new_c && top_c == -INFINITY);
            if (key < NC) {
              ca[key] = d;
              nm[key] -= d;
            }
            if (lane == 0) *unseen_of = still;
          }
          bar_wg(bar_id);
          unseen = (uint32_t)uniform((int)*unseen_of);
#pragma unroll
          for (int c = 0; c < NC; c += 2) {  // l = O = 0 in a column just seen: any finite factor will do
            const float2 d2 = *reinterpret_cast<const float2*>(ca + c);
            l2[c / 2] = fmul2(l2[c / 2], pack2(exp2f(fminf(-d2.x, 0.f)), exp2f(fminf(-d2.y, 0.f))));
            v[c] -= d2.x;
            v[c + 1] -= d2.y;
          }
          if (j > 0) {  // O, and the record, hold the segment's tiles so far
#pragma unroll 1
            for (int c = 0; c < 2 * NC; c += 16) {
              float o[16];
              const uint32_t at = tmem + lanes + (c < NC ? 2 * NR + c0 + c : 3 * NR + c0 + c - NC);
              const float* f = ca + (c < NC ? c : c - NC);
              tmem_ld16(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] *= exp2f(fminf(-f[x], 0.f));
              tmem_st16(at, o);
            }
            tmem_wait_st();
            fence_before_sync();
            if (j >= kFlush) {
              float* rec_o = record();
#pragma unroll 4
              for (int c = 0; c < NC; ++c) rec_o[c * kHeadDim] *= exp2f(fminf(-ca[c], 0.f));
            }
          }
          bar_wg(bar_id);  // the growths are read before the next tile replaces them
          fence_after_sync();
        }
        // ---- P = 2^(z - m) as bf16 hi + lo (each rounded: |p - hi - lo| <= 2^-18 p), into the
        // B operand
        if (i >= C::PB) {
          const int w = i - C::PB;  // the P.V that read this buffer last, or its half over these keys
          ok &= mbar_wait_bounded((key < 64 ? o_half : o_done) + (w & 1), (w >> 1) & 1, abort_flag);
          __syncwarp();
        }
        unsigned char* sp = smem + C::OFF_P + (size_t)(i % C::PB) * C::P_BYTES;
        const f2 minus = pack2(-1.f, -1.f);
#pragma unroll
        for (int c8 = 0; c8 < NC; c8 += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int c = c8 + 2 * u;
            const float p0 = ex2(v[c]), p1 = ex2(v[c + 1]);
            f2 r = pack2(p0, p1);
            l2[c / 2] = fadd2(l2[c / 2], r);
            const __nv_bfloat162 hw = __floats2bfloat162_rn(p0, p1);
            hi[u] = *reinterpret_cast<const uint32_t*>(&hw);
            ffma2(r, bf2_to_f2(hi[u]), minus);  // exact
            float r0, r1;
            unpack2(r, r0, r1);
            const __nv_bfloat162 lw = __floats2bfloat162_rn(r0, r1);
            lo[u] = *reinterpret_cast<const uint32_t*>(&lw);
          }
          const int nh = c0 + c8, nl = NR + c0 + c8;
          *reinterpret_cast<uint4*>(sp + (nh >> 6) * kHalfTile + swz(key, (nh & 63) >> 3)) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(sp + (nl >> 6) * kHalfTile + swz(key, (nl & 63) >> 3)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_async_smem();
        fence_before_sync();
        mbar_arrive(&p_full[2 * (i & 1) + (key >> 6)]);
      }
      it += n;
      __syncwarp();
      mbar_arrive_if(&q_free[buf], lane == 0);  // the words are read, and every S has run
      // ---- the segment's result: l over the keys, then O^T out of TMEM
      {
        const int i = it - 1;
        ok &= mbar_wait_bounded(&o_done[i & 1], (i >> 1) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        fence_after_sync();
      }
      // the P buffers are free now (the last P.V has run)
      float sum;
      {
        float l[NC];
#pragma unroll
        for (int c = 0; c < NC; c += 2) unpack2(l2[c / 2], l[c], l[c + 1]);
        sum = over_keys(0, l, false);
      }
      const bool alone = g.a == 0 && g.e == g.t.count;
      if (key < NC) {
        const float m = -nm[key];
        ca[key] = sum == 0.f ? 0.f : 1.f / sum;  // a NaN stays one
        const int r = row0 + c0 + key;
        if (c0 + key < rows) {
          if (alone) {
            p.lse[((size_t)g.b * p.T + (r >> lg)) * p.Hq + (size_t)g.kvh * p.G + (r & (p.G - 1))] =
                sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
          } else {
            float* ml = record() - key - (size_t)c0 * kHeadDim + NR * 128 + c0 + key;
            ml[0] = m;
            ml[NR] = sum;
          }
        }
      }
      __syncwarp();
      bar_wg(bar_id);
      float* rec_o = record();
      float* out = p.out + (((size_t)g.b * p.T) * p.Hq + (size_t)g.kvh * p.G) * kHeadDim + key;
#pragma unroll
      for (int c = 0; c < NC; c += 16) {
        if (c0 + c >= rows) break;
        float o[16], o2[16];
        tmem_ld16(tmem + lanes + 2 * NR + c0 + c, o);
        tmem_ld16(tmem + lanes + 3 * NR + c0 + c, o2);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] += o2[x];
        if (n > kFlush) {
#pragma unroll
          for (int x = 0; x < 16; ++x) o2[x] = rec_o[(c + x) * kHeadDim];
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] += o2[x];
        }
        if (alone) {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int r = c0 + c + x, rr = row0 + r;
            if (r < rows) out[((size_t)(rr >> lg) * p.Hq + (rr & (p.G - 1))) * kHeadDim] = o[x] * ca[c + x];
          }
        } else {  // rows past the tree are written too: nobody reads them
#pragma unroll
          for (int x = 0; x < 16; ++x) rec_o[(c + x) * kHeadDim] = o[x];
        }
      }
      fence_before_sync();
      bar_wg(bar_id);  // the factors are read before the next segment writes them
    }
    if (!ok) {
      dev_error(p.status, SKV_DEV_TIMEOUT);
      *abort_flag = 1;
    }
  }
  // ---- teardown: free TMEM once every role is through
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)(4 * NR)) : "memory");
}

// ---------------------------------------------------------------------------
// Merge of the partial records, a row's dims over the lanes of a warp.
//  - Fewer groups than shares (most groups are cut, often into many records): CTA (g, y)
//    looks at group g.
//  - Else: a group is cut where a share begins inside it, so CTA (w - 1, y) looks at share
//    w and serves the group if that is its first cut.
// SHARED: a row per CTA, its records shared out over the warps, which meet in shared
// memory; else a row per warp.  Eight records are in flight in a warp.
// A record without weight (l = 0) is passed over; one whose l is NaN makes the row NaN.
constexpr int kMergeWarps = 4;

template <bool SHARED>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeParams p, const TreeLaunch L, int NR) {
  __shared__ float4 part[kMergeWarps][32];
  __shared__ float2 part_ml[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = SHARED ? blockIdx.y : blockIdx.y * kMergeWarps + warp, t = r / p.G;
  wait_for_stream();
  const int total = L.starts[L.slots].x, workers = tree_workers(L.slots, total);
  int b, kvh, first, tiles, odd;  // the group: its first tile, its tiles, slot of its first record
  if (L.groups) {
    b = blockIdx.x / p.Hkv;
    kvh = blockIdx.x % p.Hkv;
    const int4 x = L.groups[blockIdx.x];  // written if the sequence has rows
    if (t >= tree_seq(p, b).n) return;
    first = x.x;
    tiles = x.y;
    odd = x.z;
  } else {
    const int w = blockIdx.x + 1;
    const int4 here = L.starts[w], prev = L.starts[w - 1];
    if (w >= workers || here.z == 0) return;
    const bool same = prev.x == here.x && prev.y == here.y;
    if (same && prev.z > 0) return;  // not the group's first cut
    b = here.x;
    kvh = here.y;
    if (t >= tree_seq(p, b).n) return;
    first = share_begin(w, total, workers) - here.z;
    tiles = here.w;
    odd = same ? 0 : 1;  // the share before began with another group
  }
  const int c_first = share_of(first, total, workers), c_last = share_of(first + tiles - 1, total, workers);
  if (c_first == c_last) return;
  const int m_tile = r / NR, rr = r % NR;
  const size_t step = (size_t)2 * L.m_tiles * (NR * 130);
  const float* rec0 = L.rec + (size_t)m_tile * (NR * 130);
  const size_t row = ((size_t)b * p.T + t) * p.Hq + (size_t)kvh * p.G + r % p.G;
  float4* out = reinterpret_cast<float4*>(p.out + row * kHeadDim) + lane;
  constexpr int kStride = SHARED ? kMergeWarps : 1;
  float M = kUnseen, W = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = c_first + (SHARED ? warp : 0); c0 <= c_last; c0 += kStride * 8) {
    float4 o[8];
    float m[8], l[8];
    float top = M;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = c0 + u * kStride;
      o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      l[u] = 0.f;
      m[u] = kUnseen;
      if (c <= c_last) {
        const float* y = rec0 + c * step + (c == c_first && odd ? step / 2 : 0);
        o[u] = *reinterpret_cast<const float4*>(y + rr * kHeadDim + lane * 4);
        l[u] = y[NR * 129 + rr];
        m[u] = y[NR * 128 + rr];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (l[u] != 0.f) top = fmaxf(top, m[u]);
    const float old = exp2f(M - top);
    M = top;
    W *= old;
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (l[u] == 0.f) continue;  // attends nothing; a NaN is not left out
      const float f = exp2f(m[u] - top);
      W += f * l[u];
      acc.x += f * o[u].x;
      acc.y += f * o[u].y;
      acc.z += f * o[u].z;
      acc.w += f * o[u].w;
    }
  }
  if (SHARED) {
    part[warp][lane] = acc;
    if (lane == 0) part_ml[warp] = make_float2(M, W);
    __syncthreads();
    if (warp != 0) return;
    M = kUnseen;
#pragma unroll
    for (int v = 0; v < kMergeWarps; ++v) M = fmaxf(M, part_ml[v].x);
    W = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int v = 0; v < kMergeWarps; ++v) {
      const float f = exp2f(part_ml[v].x - M);
      W += f * part_ml[v].y;
      acc.x += f * part[v][lane].x;
      acc.y += f * part[v][lane].y;
      acc.z += f * part[v][lane].z;
      acc.w += f * part[v][lane].w;
    }
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;
  *out = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (lane == 0) p.lse[row] = W == 0.f ? -INFINITY : (M + log2f(W)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// Host side
struct TreePlan {
  int nr, m_tiles, slots;
  bool by_group;  // merge CTAs by group, not by cut
  size_t hdr_bytes, ws_bytes;
};

TreePlan tree_plan(const TreeParams& p) {
  TreePlan pl{};
  // The narrowest CTA that holds all rows, 128 at most: at 64 x 2k tokens 32 rows took 103
  // us with 32 columns, 128 with 64 and 186 with 128; at 16 x 8k tokens 64 rows took 105 us
  // with 64 and 146 with 128; at 4 x 32k tokens 128 rows took 140 us with 128 and 168 as
  // two CTAs of 64.
  const int rows = p.T * p.G;
  pl.nr = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  pl.m_tiles = (rows + pl.nr - 1) / pl.nr;
  const TreeTiles t = tree_tiles(p.window, p.sink, p.recent, p.max_seq_len, std::min(p.T, p.max_seq_len));
  const long long tiles = std::max(1ll, (long long)p.B * p.Hkv * t.count);
  pl.slots = (int)std::min<long long>(std::max(1, num_sms() / pl.m_tiles), tiles);
  const long long groups = (long long)p.B * p.Hkv;
  // A merge CTA per group if there are fewer groups than cuts (1 x 4k tokens, 64 rows: 17.1
  // us against 20.4 by cut), else per cut (64 x 2k tokens: 103 us against 106 by group).
  pl.by_group = groups < pl.slots;
  pl.hdr_bytes = ((size_t)(pl.slots + 1 + (pl.by_group ? groups : 0)) * sizeof(int4) + 255) / 256 * 256;
  pl.ws_bytes = pl.hdr_bytes + (size_t)2 * pl.slots * pl.m_tiles * pl.nr * 130 * sizeof(float);
  return pl;
}

// Q [B * T][Hq][128] as a 3-D tensor, boxes of `tokens` tokens x G heads x 64 dims landing
// 128B-swizzled; tokens past the tensor read as zero.
bool make_rows_map(CUtensorMap* m, const TreeParams& p, int tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)p.Hq, (cuuint64_t)p.B * p.T};
  const cuuint64_t strides[2] = {(cuuint64_t)kRowBytes, (cuuint64_t)p.Hq * kRowBytes};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)tokens};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NR, int MODE>
cudaError_t launch_tree(const TreeParams& p, const TreeLaunch& L, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  static std::atomic<bool> attr_set[64];  // per device; racing first calls only repeat the set-up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(tree_kernel<NR, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)TreeCfg<NR>::BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  return launch_early(tree_kernel<NR, MODE>, L.slots * L.m_tiles, TreeCfg<NR>::THREADS, TreeCfg<NR>::BYTES, s, p, L, tq, tk, tv);
}

template <int NR>
cudaError_t launch_tree(const TreeParams& p, const TreeLaunch& L, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  const int mode = score_mode(p);
  if (mode == CAP) return launch_tree<NR, CAP>(p, L, tq, tk, tv, s);
  if (mode == BIAS) return launch_tree<NR, BIAS>(p, L, tq, tk, tv, s);
  return launch_tree<NR, PLAIN>(p, L, tq, tk, tv, s);
}

}  // namespace
}  // namespace skv

extern "C" {

SKV_API size_t skv_tree_workspace_size(const skv_tree_args* args) {
  skv::TreeParams p;
  if (skv::tree_params(args, &p) != SKV_OK) return 0;
  return skv::tree_plan(p).ws_bytes;
}

SKV_API skv_status attn_tree_decode(const skv_tree_args* a, skv_stream_t stream) {
  using namespace skv;
  TreeParams p;
  const skv_status st = tree_params(a, &p);
  if (st != SKV_OK) return st;
  if (!p.v_pool || !p.out || !aligned16(p.v_pool) || !aligned16(p.out)) return SKV_EINVAL;
  const TreePlan pl = tree_plan(p);
  if (!a->workspace || a->workspace_bytes < pl.ws_bytes || !aligned16(a->workspace)) return SKV_EWORKSPACE;
  TreeLaunch L{};
  L.m_tiles = pl.m_tiles;
  L.slots = pl.slots;
  L.f = score_factors(p);
  L.starts = static_cast<int4*>(a->workspace);
  L.groups = pl.by_group ? L.starts + pl.slots + 1 : nullptr;
  L.rec = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + pl.hdr_bytes);
  CUtensorMap tq, tk, tv;
  const long long pool_rows = (long long)p.num_pages * p.Hkv * kBlock;
  if (!make_pool_map(&tk, p.k_pool, pool_rows) || !make_pool_map(&tv, p.v_pool, pool_rows) ||
      !make_rows_map(&tq, p, pl.nr / p.G))
    return SKV_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = pl.nr == 32   ? launch_tree<32>(p, L, tq, tk, tv, s)
                        : pl.nr == 64 ? launch_tree<64>(p, L, tq, tk, tv, s)
                                      : launch_tree<128>(p, L, tq, tk, tv, s);
  if (e != cudaSuccess) return SKV_ECUDA;
  if (pl.slots == 1) return SKV_OK;  // nothing is cut
  // a row per CTA where a group's records are many (one KV head, 64k tokens: 25 us against
  // 44 with a row per warp), per warp where they are few
  const int rows = p.T * p.G, x = pl.by_group ? p.B * p.Hkv : pl.slots - 1;
  const bool shared = pl.by_group && pl.slots / (p.B * p.Hkv) >= 8;
  const cudaError_t m =
      shared ? launch_early(tree_merge_kernel<true>, dim3(x, rows), kMergeWarps * 32, 0, s, p, L, pl.nr)
             : launch_early(tree_merge_kernel<false>, dim3(x, (rows + kMergeWarps - 1) / kMergeWarps), kMergeWarps * 32, 0,
                            s, p, L, pl.nr);
  return m == cudaSuccess ? SKV_OK : SKV_ECUDA;
}

}  // extern "C"
