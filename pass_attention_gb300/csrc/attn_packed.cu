// Attention forward over packed sequences with grouped key heads, on the
// tcgen05 tensor cores.
//
// The recurrence, the tensor-memory layout and the roles of the warps are those
// of the dense attention forward (attn_fwd.cu): 8 softmax warps, a TMA producer,
// one thread that issues S = Q K^T and one that issues O += P V, three score
// buffers in tensor memory, the O rescale past a threshold of 2^8. What bounds
// it is the same chain; what is different here:
//
// Rows. A tile's 128 rows are 128 / P' consecutive queries times P' query heads of
// one key head, P' the largest power of two that divides G = Hq / Hkv (up to
// 128): row r is query r / P', head r % P'. The tile arrives by one 4-D TMA box.
// A group's heads share each K and V tile, and sequences shorter than 128 tokens fill more of a
// tile (32 queries x 4 heads instead of 128 x 1).
//
// Division. Lengths are known on the device only. The items (query tile x KV
// tiles) stand in a row, each as long as its KV tiles and a constant, and every
// CTA takes equal shares of the length (packed_plan.h): no tile list, no sorting, no
// idle CTA behind the longest sequence, and one query tile behind a long prefix
// spreads over the GPU. A share that begins or ends inside an item leaves an
// unnormalised (m, l, O) in the workspace; a second kernel joins the parts in
// share order. No atomics: every run gives the same bits. The shares of a
// round are neighbours, so the K and V that the CTAs read at one time stay in L2
// (rounds in launch_attn_packed).
//
// Foreign rows. The last KV tile of a sequence reaches into the next sequence's
// rows, or into rows that nobody wrote. Their scores are replaced by -inf; their V rows
// are set to zero in shared memory, since a weight of 0 times NaN or infinity
// would still reach O.

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "device_common.cuh"
#include "oss_internal.h"
#include "packed_plan.h"
#include "tcgen05.cuh"

namespace oss {
namespace {

constexpr int kBM = 128;          // rows per query tile (= tensor-memory lanes)
constexpr int kBN = 128;          // keys per KV tile
constexpr int kStages = 3;        // K ring, V ring, score buffers
constexpr int kKLead = 2;         // K loads run this many steps ahead of V loads
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kProducerWarp = 8;
constexpr int kQkWarp = 9;
constexpr int kPvWarp = 10;
constexpr int kThreads = (kPvWarp + 1) * 32;
constexpr int kHalf = 128 * 128;  // 128 rows x 64 dims x 2 bytes
constexpr int kMaxRounds = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 384;
constexpr float kRescaleSlack = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;
static_assert(kBN == kKeysPerTile, "the plan counts KV tiles of this size");
__device__ __forceinline__ uint32_t col_s(int b) { return 128u * b; }

template <int D>
struct Smem {
  static constexpr int kTile = (D / 64) * kHalf;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kBytes = kOffV + kStages * kTile + 1024;  // + alignment slack
};

struct PackedParams {
  uint16_t* o;
  float* lse;
  const int32_t *cu_q, *cu_k;
  int32_t batch, tokens_q, tokens_k, Hq, packs, packs_per_key_head, pos_shift, rounds;
  float C;  // scale * log2(e)
  int causal;
  unsigned int* err;
  uint64_t timeout_ns;
  unsigned int tag;
  int skip_v_step;  // test hook: the producer skips the V load of this step (-1: none)
  // workspace: a part's rows in the softmax threads' layout
  float4* part_o;   // [2 shares][D / 8][kSoftThreads]: unnormalised O
  float4* part_ml;  // [2 shares][kSoftThreads]: base-2 m, l of rows a, b
  int4* meta;       // [shares]: {parts, first query row, queries, pack} of the item cut at its end
};

#define wait_bar(bar, parity, abort_flag, err, site) \
  (mbar_test_wait((bar), (parity)) ||                 \
   wait_bar_slow<kKernelAttnPacked>((bar), (parity), (abort_flag), (err), (site), p.timeout_ns, p.tag))

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

struct Barriers {
  uint64_t q_full;   // Q tile landed
  uint64_t q_free;   // every QK^T of the item in the Q buffer is done
  uint64_t k_full[kStages], v_full[kStages];
  uint64_t s_full[kStages];
  uint64_t p_ready[2][kStages];  // P of keys 0..63 / 64..127 written
  uint64_t o_done[kStages];      // P V done, for the steps of each buffer
  uint64_t o_free;               // the epilogue has read O out of tensor memory
  uint64_t drain[2];
};

// Where a share begins and ends: the item at place w of the row of items, and
// the KV step inside it.
struct ShareStart {
  int64_t w;
  int32_t seq, pack, tile, step;
};
struct ShareEnd {
  int64_t w;
  int32_t step;
};
struct Shares {
  ShareStart start[kMaxRounds];
  ShareEnd end[kMaxRounds];
  int64_t total;
  int32_t count;
};

__device__ __forceinline__ PackedSeq load_seq(const PackedParams& p, int b) {
  return packed_seq(row_range(p.cu_q[b], p.cu_q[b + 1], p.tokens_q),
                    row_range(p.cu_k[b], p.cu_k[b + 1], p.tokens_k), p.pos_shift);
}

// Finds this CTA's shares: every thread measures a run of sequences, a block
// scan places the runs, and the thread whose run holds a boundary locates it.
__device__ void find_shares(const PackedParams& p, Shares* sh) {
  __shared__ int64_t warp_len[kThreads / 32], warp_items[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool causal = p.causal != 0;
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  int64_t mine = 0, items = 0;
  for (int b = b0; b < b1; ++b) {
    const PackedSeq s = load_seq(p, b);
    mine += length_before(s, s.tiles, p.pos_shift, causal);
    items += s.tiles;
    if (blockIdx.x == 0 && (row_range(p.cu_q[b], p.cu_q[b + 1], p.tokens_q).clamped ||
                            row_range(p.cu_k[b], p.cu_k[b + 1], p.tokens_k).clamped))
      report_error(p.err, kKernelPaged | (kSiteBadOffsets << 8));
  }
  mine *= p.packs;
  items *= p.packs;
  int64_t upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
    items += __shfl_xor_sync(0xffffffffu, items, off);
  }
  if (lane == 31) {
    warp_len[warp] = upto;
    warp_items[warp] = items;
  }
  if (tid < kMaxRounds) {
    sh->start[tid] = ShareStart{0, 0, 0, 0, 0};
    sh->end[tid] = ShareEnd{0, 0};
  }
  __syncthreads();
  int64_t before = upto - mine, total = 0, n_items = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += warp_len[i];
    total += warp_len[i];
    n_items += warp_items[i];
  }
  const int ctas = gridDim.x;
  const int n = total > 0 ? share_count(total, n_items, ctas, p.rounds) : 0;
  if (tid == 0) {
    sh->total = total;
    sh->count = n;
  }
  if (mine > 0) {
    for (int r = 0; r < p.rounds; ++r) {
      const int64_t share = static_cast<int64_t>(r) * ctas + blockIdx.x;
      if (share >= n) break;
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
        const int64_t at = share_begin(share + e, total, n);
        if (at < before || at >= before + mine) {
          if (at == total && at == before + mine) sh->end[r] = ShareEnd{total, 0};
          continue;
        }
        int64_t w = before;
        for (int b = b0; b < b1; ++b) {
          const PackedSeq s = load_seq(p, b);
          const int64_t len = length_before(s, s.tiles, p.pos_shift, causal);
          if (at >= w + len * p.packs) {
            w += len * p.packs;
            continue;
          }
          const int pack = static_cast<int>((at - w) / len);
          w += pack * len;
          const int tile = tile_at(s, at - w, p.pos_shift, causal);
          w += length_before(s, tile, p.pos_shift, causal);
          const int steps = kv_tiles(s, tile, p.pos_shift, causal);
          const int step = cut_step(at - w, steps);
          if (e == 0)
            sh->start[r] = ShareStart{w, b, pack, tile, step};
          else
            sh->end[r] = step == steps ? ShareEnd{w + kTileWeight + steps, 0} : ShareEnd{w, step};
          break;
        }
      }
    }
  }
  __syncthreads();
}

// A piece of an item: KV steps [s0, s1) of its n_kv.
struct Unit {
  int q_row, n_pos;       // first query row, queries of the tile
  int k_row, k_len, vis;  // first key row, keys, keys that the tile's first query sees
  int n_kv, n_diag, s0, s1, pack, share;
  int64_t w;              // the item's place
};

// The walk of a CTA over its shares; every role makes the same one.
struct Walk {
  PackedSeq s;
  int64_t w, end_w;
  int seq, pack, tile, s0, end_step, round;
  bool fetch;  // the next item belongs to a later sequence

  __device__ __forceinline__ void begin_round(const PackedParams& p, const Shares& sh) {
    const ShareStart a = sh.start[round];
    w = a.w;
    seq = a.seq;
    pack = a.pack;
    tile = a.tile;
    s0 = a.step;
    end_w = sh.end[round].w;
    end_step = sh.end[round].step;
    fetch = false;
    if (w < end_w || (w == end_w && end_step > 0)) s = load_seq(p, seq);
  }
  __device__ __forceinline__ void begin(const PackedParams& p, const Shares& sh) {
    round = 0;
    begin_round(p, sh);
  }
  __device__ __forceinline__ bool next(const PackedParams& p, const Shares& sh, Unit& u) {
    const bool causal = p.causal != 0;
    for (;;) {
      if (!(w < end_w || (w == end_w && end_step > 0))) {
        if (++round >= p.rounds) return false;
        begin_round(p, sh);
        continue;
      }
      if (fetch) {
        fetch = false;
        do {
          s = load_seq(p, ++seq);
        } while (s.tiles == 0 && seq + 1 < p.batch);
      }
      const int steps = kv_tiles(s, tile, p.pos_shift, causal);
      const int s1 = w == end_w ? end_step : steps;
      const int from = s0;
      if (from < s1) {
        const int pos0 = tile << p.pos_shift;
        u.q_row = s.q_start + pos0;
        u.n_pos = min(1 << p.pos_shift, s.q_len - pos0);
        u.k_row = s.k_start;
        u.k_len = s.k_len;
        u.vis = visible_keys(s, pos0, causal);
        u.n_kv = steps;
        // KV tiles that the first query does not see whole are visited first
        u.n_diag = causal ? max(0, steps - max(0, u.vis) / kBN) : 0;
        u.s0 = from;
        u.s1 = s1;
        u.pack = pack;
        u.share = round * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
        u.w = w;
      }
      w += kTileWeight + steps;
      s0 = 0;
      if (++tile == s.tiles) {
        tile = 0;
        if (++pack == p.packs) {
          pack = 0;
          fetch = true;
        }
      }
      if (from < s1) return true;
    }
  }
};

// KV tile visited at step j of an item.
__device__ __forceinline__ int kv_tile(const Unit& u, int j) {
  return j < u.n_diag ? u.n_kv - 1 - j : j - u.n_diag;
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t w;
  if constexpr (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Stores 32 dims (from chunk 4 mb of half h) of rows a and b. v[4 i + e]: the
// thread's values of 8-dim chunk i, a's two dims then b's two; a 4 x 4 transpose
// among a row's four threads hands each a whole chunk. A row without keys (inv
// 0) is written as zeros whatever its accumulator holds.
template <bool kF16>
__device__ __forceinline__ void store_chunks(uint4* oa, uint4* ob, const float (&v)[16], float inv_a, float inv_b,
                                             int chunk0, int jj, bool live_a, bool live_b) {
  uint32_t wa[4], wb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wa[i] = inv_a > 0.f ? pack16<kF16>(v[4 * i] * inv_a, v[4 * i + 1] * inv_a) : 0u;
    wb[i] = inv_b > 0.f ? pack16<kF16>(v[4 * i + 2] * inv_b, v[4 * i + 3] * inv_b) : 0u;
  }
  lane_transpose4(wa, jj);
  lane_transpose4(wb, jj);
  if (live_a) oa[chunk0 + jj] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  if (live_b) ob[chunk0 + jj] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

// Row r of a tile, as a row of o and lse.
__device__ __forceinline__ int64_t out_row(const PackedParams& p, int q_row, int pack, int r) {
  const int head_shift = 7 - p.pos_shift;
  return static_cast<int64_t>(q_row + (r >> head_shift)) * p.Hq + (pack << head_shift) + (r & ((1 << head_shift) - 1));
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads, 1)
attn_packed_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const PackedParams p) {
  using L = Smem<D>;
  constexpr int kHalves = D / 64;
  constexpr uint32_t kIdescQK = make_idesc(kBM, kBN, false, kF16);
  constexpr uint32_t kIdescPV = make_idesc(kBM, D, true, kF16);
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bars;
  __shared__ Shares shares;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag_s;
  volatile int* abort_flag = &abort_flag_s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const uint32_t sbase = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(smem_addr(&bars.q_full), 1);
    mbar_init(smem_addr(&bars.q_free), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&bars.k_full[s]), 1);
      mbar_init(smem_addr(&bars.v_full[s]), 1);
      mbar_init(smem_addr(&bars.s_full[s]), 1);
      mbar_init(smem_addr(&bars.p_ready[0][s]), kSoftThreads);
      mbar_init(smem_addr(&bars.p_ready[1][s]), kSoftThreads);
      mbar_init(smem_addr(&bars.o_done[s]), 1);
    }
    mbar_init(smem_addr(&bars.o_free), kSoftThreads);
    mbar_init(smem_addr(&bars.drain[0]), 1);
    mbar_init(smem_addr(&bars.drain[1]), 1);
    abort_flag_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kQkWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_base_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  if (threadIdx.x < p.rounds) p.meta[threadIdx.x * gridDim.x + blockIdx.x] = make_int4(0, 0, 0, 0);
  find_shares(p, &shares);  // its barriers publish the set-up above
  tc_fence_after();
  const uint32_t tbase = tmem_base_slot;

  // Every role walks the same units and counts KV steps g across them: step g
  // uses ring stage and score buffer g % 3, in round g / 3.
  Walk walk;
  walk.begin(p, shares);
  Unit u;
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_q)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
      const uint32_t qbar = smem_addr(&bars.q_full);
      int k_issued = 0, v_issued = 0, q_loads = 0, skipped_v = -1;
      int key_row[kStages] = {0, 0, 0}, key_head[kStages] = {0, 0, 0};
      int kt = 0, j = 0;
      bool have = walk.next(p, shares, u);
      if (have) j = u.s0;
      for (int g = 0;; ++g) {
        // V of step g - kKLead first: it is the load the P V thread waits on soonest
        const int gv = g - kKLead;
        if (gv >= 0 && gv < k_issued) {
          if (gv == p.skip_v_step) {
            skipped_v = gv;
          } else {
            const int s = gv % kStages;
            const int round = gv / kStages;
            if (round > 0 && !wait_bar(smem_addr(&bars.o_done[s]), (round - 1) & 1, abort_flag, p.err, kSiteVEmpty))
              break;
            const uint32_t vb = smem_addr(&bars.v_full[s]);
            mbar_expect_tx(vb, L::kTile);
            for (int h = 0; h < kHalves; ++h)
              tma_load_3d(sbase + L::kOffV + s * L::kTile + h * kHalf, &tmap_v, vb, h * 64, key_head[s], key_row[s]);
            v_issued = gv + 1;
          }
        }
        if (!have) {
          if (gv + 1 >= k_issued) break;
          continue;
        }
        if (j == u.s0) {
          if (kt > 0 && !wait_bar(smem_addr(&bars.q_free), (kt - 1) & 1, abort_flag, p.err, kSiteQEmpty)) break;
          mbar_expect_tx(qbar, L::kTile);
          for (int h = 0; h < kHalves; ++h)
            tma_load_4d(sbase + L::kOffQ + h * kHalf, &tmap_q, qbar, h * 64, 0, u.pack, u.q_row);
          ++q_loads;
        }
        const int s = g % kStages;
        const int round = g / kStages;
        if (round > 0 && !wait_bar(smem_addr(&bars.s_full[s]), (round - 1) & 1, abort_flag, p.err, kSiteKEmpty))
          break;
        const uint32_t kb = smem_addr(&bars.k_full[s]);
        mbar_expect_tx(kb, L::kTile);
        key_row[s] = u.k_row + kv_tile(u, j) * kBN;
        key_head[s] = u.pack / p.packs_per_key_head;
        for (int h = 0; h < kHalves; ++h)
          tma_load_3d(sbase + L::kOffK + s * L::kTile + h * kHalf, &tmap_k, kb, h * 64, key_head[s], key_row[s]);
        k_issued = g + 1;
        if (++j == u.s1) {
          ++kt;
          have = walk.next(p, shares, u);
          if (have) j = u.s0;
        }
      }
      // drain: every issued copy must land before the CTA may exit
      if (q_loads > 0) drain_bar<kKernelAttnPacked>(qbar, (q_loads - 1) & 1, p.err);
      for (int i = k_issued - 1; i >= 0 && i >= k_issued - kStages; --i)
        drain_bar<kKernelAttnPacked>(smem_addr(&bars.k_full[i % kStages]), (i / kStages) & 1, p.err);
      for (int i = v_issued - 1; i >= 0 && i >= v_issued - kStages; --i)
        if (i != skipped_v)
          drain_bar<kKernelAttnPacked>(smem_addr(&bars.v_full[i % kStages]), (i / kStages) & 1, p.err);
    }
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------ QK issuer
    if (lane == 0) {
      bool ok = true;
      const uint64_t dq = smem_desc(sbase + L::kOffQ, 16, 1024);
      int g = 0;
      for (int kt = 0; ok && walk.next(p, shares, u); ++kt) {
        if (!(ok = wait_bar(smem_addr(&bars.q_full), kt & 1, abort_flag, p.err, kSiteQFull))) break;
        // the previous item's last P V goes through the tensor pipe before this
        // one's first QK^T: its epilogue waits on it
        if (kt > 0 && !(ok = wait_bar(smem_addr(&bars.o_done[(g - 1) % kStages]), ((g - 1) / kStages) & 1, abort_flag,
                                      p.err, kSiteODone)))
          break;
        for (int j = u.s0; j < u.s1; ++j, ++g) {
          const int s = g % kStages;
          if (!(ok = wait_bar(smem_addr(&bars.k_full[s]), (g / kStages) & 1, abort_flag, p.err, kSiteKFull))) break;
          if (g >= kStages && !(ok = wait_bar(smem_addr(&bars.o_done[s]), (g / kStages - 1) & 1, abort_flag, p.err,
                                              kSiteODone)))
            break;
          tc_fence_after();
          const uint64_t dk = smem_desc(sbase + L::kOffK + s * L::kTile, 16, 1024);
          const uint32_t d_s = tbase + col_s(s);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(d_s, dq + kstep_kmajor(kk, kHalf), dk + kstep_kmajor(kk, kHalf), kIdescQK, kk > 0 ? 1u : 0u);
          tc_commit(smem_addr(&bars.s_full[s]));
        }
        if (ok) tc_commit(smem_addr(&bars.q_free));
      }
      tc_commit(smem_addr(&bars.drain[0]));
      drain_bar<kKernelAttnPacked>(smem_addr(&bars.drain[0]), 0, p.err);
    }
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0) {
      bool ok = true;
      const uint32_t d_o = tbase + kColO;
      int g = 0;
      for (int kt = 0; ok && walk.next(p, shares, u); ++kt) {
        for (int j = u.s0; j < u.s1; ++j, ++g) {
          const int s = g % kStages;
          if (!(ok = wait_bar(smem_addr(&bars.v_full[s]), (g / kStages) & 1, abort_flag, p.err, kSiteVFull))) break;
          if (j == u.s0 && kt > 0 &&
              !(ok = wait_bar(smem_addr(&bars.o_free), (kt - 1) & 1, abort_flag, p.err, kSiteOFree)))
            break;
          const uint64_t dv = smem_desc(sbase + L::kOffV + s * L::kTile, kHalf, 1024);
          const uint32_t a_p = tbase + col_s(s);
#pragma unroll
          for (int hp = 0; hp < 2; ++hp) {
            if (!(ok = wait_bar(smem_addr(&bars.p_ready[hp][s]), (g / kStages) & 1, abort_flag, p.err, kSitePReady)))
              break;
            tc_fence_after();
#pragma unroll
            for (int kk = 4 * hp; kk < 4 * hp + 4; ++kk)
              mma_ts(d_o, a_p + kk * 8, dv + static_cast<uint64_t>(kk * (2048 >> 4)), kIdescPV,
                     (j > u.s0 || kk > 0) ? 1u : 0u);
          }
          if (!ok) break;
          tc_commit(smem_addr(&bars.o_done[s]));
        }
      }
      tc_commit(smem_addr(&bars.drain[1]));
      drain_bar<kKernelAttnPacked>(smem_addr(&bars.drain[1]), 0, p.err);
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Warp w owns rows 32 (w % 4) + 16 (w / 4) .. + 15; thread t holds rows
    // ra = t/4 and rb = 8 + t/4 of them, columns 8k + cq + {0, 1}.
    const int lane0 = (warp & 3) * 32 + (warp >> 2) * 16;
    const int ra = lane0 + (lane >> 2);
    const int rb = ra + 8;
    const int cq = 2 * (lane & 3);
    const int head_shift = 7 - p.pos_shift;
    const int pos_a = ra >> head_shift, pos_b = rb >> head_shift;
    const uint32_t tl = tbase + (static_cast<uint32_t>(lane0) << 16);
    const float C = p.C;
    bool ok = true;
    int g = 0;
    while (ok && walk.next(p, shares, u)) {
      float m_a = neg_inf(), m_b = neg_inf();  // reference maxima, base 2
      float l_a = 0.f, l_b = 0.f;              // this thread's share of the row sums
      const int vis_a = p.causal ? min(u.k_len, u.vis + pos_a) : u.k_len;  // keys the rows see
      const int vis_b = p.causal ? min(u.k_len, u.vis + pos_b) : u.k_len;
      for (int j = u.s0; j < u.s1; ++j, ++g) {
        const int b = g % kStages;
        const uint32_t colS = col_s(b);
        ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.s_full[b]), (g / kStages) & 1, abort_flag, p.err,
                                              kSiteSFull));
        if (!ok) break;
        tc_fence_after();
        uint32_t r0[32], r1[32];
        tmem_ld16x256_x8(tl + colS, r0);
        tmem_ld16x256_x8(tl + colS + 64, r1);
        tmem_ld_wait(r0);
        tmem_ld_wait(r1);
        float sa[32], sb[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sa[2 * k + e] = __uint_as_float(r0[4 * k + e]);
            sb[2 * k + e] = __uint_as_float(r0[4 * k + 2 + e]);
            sa[16 + 2 * k + e] = __uint_as_float(r1[4 * k + e]);
            sb[16 + 2 * k + e] = __uint_as_float(r1[4 * k + 2 + e]);
          }
        }
        const int key0 = kv_tile(u, j) * kBN;
        if (key0 + kBN > (p.causal ? u.vis : u.k_len)) {
          const int lim_a = vis_a - key0, lim_b = vis_b - key0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int col = (i >> 4) * 64 + ((i >> 1) & 7) * 8 + cq + (i & 1);
            if (col >= lim_a) sa[i] = neg_inf();
            if (col >= lim_b) sb[i] = neg_inf();
          }
        }
        float xa0 = neg_inf(), xa1 = neg_inf(), xb0 = neg_inf(), xb1 = neg_inf();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          xa0 = fmax3(xa0, sa[i], sa[i + 1]);
          xa1 = fmax3(xa1, sa[i + 2], sa[i + 3]);
          xb0 = fmax3(xb0, sb[i], sb[i + 1]);
          xb1 = fmax3(xb1, sb[i + 2], sb[i + 3]);
        }
        float xa = fmaxf(xa0, xa1), xb = fmaxf(xb0, xb1);
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
        const float mnew_a = fmaxf(m_a, xa * C), mnew_b = fmaxf(m_b, xb * C);
        const bool rescale = __any_sync(0xffffffffu, (mnew_a > m_a + kRescaleSlack) || (mnew_b > m_b + kRescaleSlack));
        float corr_a = 1.f, corr_b = 1.f;
        if (rescale) {
          corr_a = ex2(m_a - ((mnew_a == neg_inf()) ? 0.f : mnew_a));  // 0 while m = -inf
          corr_b = ex2(m_b - ((mnew_b == neg_inf()) ? 0.f : mnew_b));
          m_a = mnew_a;
          m_b = mnew_b;
        }
        if (rescale && j > u.s0) {
          // wait for P_{j-1} V (its completion implies every earlier one), then
          // rescale this warp's rows of O
          ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.o_done[(g - 1) % kStages]), ((g - 1) / kStages) & 1,
                                                abort_flag, p.err, kSiteODone));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < kHalves; ++h) {
            uint32_t ov[32];
            tmem_ld16x256_x8(tl + kColO + 64 * h, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float2 oa = __fmul2_rn(make_float2(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1])),
                                           make_float2(corr_a, corr_a));
              const float2 ob = __fmul2_rn(make_float2(__uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3])),
                                           make_float2(corr_b, corr_b));
              ov[4 * k] = __float_as_uint(oa.x);
              ov[4 * k + 1] = __float_as_uint(oa.y);
              ov[4 * k + 2] = __float_as_uint(ob.x);
              ov[4 * k + 3] = __float_as_uint(ob.y);
            }
            tmem_st16x256_x8(tl + kColO + 64 * h, ov);
          }
        }
        if (key0 + kBN > u.k_len) {
          // rows of V behind the sequence's keys: zeros (a 16-byte chunk's place
          // in its 128-byte row does not matter for them)
          ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.v_full[b]), (g / kStages) & 1, abort_flag, p.err,
                                                kSiteVFull));
          if (!ok) break;
          const int first = max(0, u.k_len - key0);
          uint8_t* vt = smem_raw + (sbase - smem_addr(smem_raw)) + L::kOffV + b * L::kTile;
          for (int i = first * 8 + static_cast<int>(threadIdx.x); i < kBN * 8; i += kSoftThreads)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              *reinterpret_cast<uint4*>(vt + h * kHalf + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        const float2 Cv = make_float2(C, C);
        const float ref_a = (m_a == neg_inf()) ? 0.f : m_a, ref_b = (m_b == neg_inf()) ? 0.f : m_b;
        const float2 mva = make_float2(-ref_a, -ref_a), mvb = make_float2(-ref_b, -ref_b);
        float2 acc_a = make_float2(0.f, 0.f), acc_b = acc_a;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int kk = 8 * h + k;
            const float2 ta = __ffma2_rn(make_float2(sa[2 * kk], sa[2 * kk + 1]), Cv, mva);
            const float2 tb = __ffma2_rn(make_float2(sb[2 * kk], sb[2 * kk + 1]), Cv, mvb);
            const float2 ea = make_float2(ex2(ta.x), ex2(ta.y));
            const float2 eb = make_float2(ex2(tb.x), ex2(tb.y));
            acc_a = __fadd2_rn(acc_a, ea);
            acc_b = __fadd2_rn(acc_b, eb);
            pk[2 * k] = pack16<kF16>(ea.x, ea.y);
            pk[2 * k + 1] = pack16<kF16>(eb.x, eb.y);
          }
          tmem_st16x128_x8(tl + colS + 32 * h, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(smem_addr(&bars.p_ready[h][b]));
        }
        l_a = fmaf(l_a, corr_a, acc_a.x + acc_a.y);
        l_b = fmaf(l_b, corr_b, acc_b.x + acc_b.y);
      }
      l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
      l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
      if (ok)
        ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.o_done[(g - 1) % kStages]), ((g - 1) / kStages) & 1,
                                              abort_flag, p.err, kSiteODone));
      if (ok) {
        tc_fence_after();
        if (u.s0 == 0 && u.s1 == u.n_kv) {
          const bool live_a = pos_a < u.n_pos, live_b = pos_b < u.n_pos;
          const float inv_a = (l_a > 0.f) ? 1.0f / l_a : 0.f;
          const float inv_b = (l_b > 0.f) ? 1.0f / l_b : 0.f;
          const int64_t row_a = out_row(p, u.q_row, u.pack, ra), row_b = out_row(p, u.q_row, u.pack, rb);
          uint4* oa = reinterpret_cast<uint4*>(p.o + row_a * D);
          uint4* ob = reinterpret_cast<uint4*>(p.o + row_b * D);
#pragma unroll 1
          for (int h = 0; h < kHalves; ++h) {
            uint32_t ov[32];
            tmem_ld16x256_x8(tl + kColO + 64 * h, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
              float v[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(ov[16 * mb + i]);
              store_chunks<kF16>(oa, ob, v, inv_a, inv_b, 8 * h + 4 * mb, lane & 3, live_a, live_b);
            }
          }
          if ((lane & 3) == 0 && p.lse) {
            if (live_a) p.lse[row_a] = (l_a > 0.f) ? (m_a + log2f(l_a)) * kLn2 : neg_inf();
            if (live_b) p.lse[row_b] = (l_b > 0.f) ? (m_b + log2f(l_b)) * kLn2 : neg_inf();
          }
        } else {
          // a part of an item: unnormalised, every warp access 512 contiguous bytes
          const int64_t slot = 2 * static_cast<int64_t>(u.share) + (u.s0 == 0 ? 1 : 0);
          float4* wo = p.part_o + slot * (D / 8) * kSoftThreads + threadIdx.x;
#pragma unroll 1
          for (int h = 0; h < kHalves; ++h) {
            uint32_t ov[32];
            tmem_ld16x256_x8(tl + kColO + 64 * h, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              wo[(8 * h + e) * kSoftThreads] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                                           __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
          }
          p.part_ml[slot * kSoftThreads + threadIdx.x] = make_float4(m_a, l_a, m_b, l_b);
          if (u.s0 == 0 && threadIdx.x == 0) {
            const int64_t last = last_boundary(u.w + kTileWeight + u.n_kv - kMinSteps, shares.total, shares.count);
            p.meta[u.share] = make_int4(static_cast<int>(last) - u.share + 1, u.q_row, u.n_pos, u.pack);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(smem_addr(&bars.o_free));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTmemCols) : "memory");
  }
}

// The join: CTA (share, quarter) merges 32 dims of the item that is cut at the
// share's end. Part 0 lies in slot 2 share + 1, part i in slot 2 (share + i).
template <int D, bool kF16>
__global__ void __launch_bounds__(kSoftThreads) attn_packed_join_kernel(const PackedParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int share = blockIdx.x, mb = blockIdx.y;
  const int4 meta = p.meta[share];
  const int parts = meta.x;
  if (parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lane0 = (warp & 3) * 32 + (warp >> 2) * 16;
  const int ra = lane0 + (lane >> 2), rb = ra + 8;
  auto slot = [&](int i) -> int64_t { return 2 * (static_cast<int64_t>(share) + i) + (i == 0 ? 1 : 0); };
  float M_a = neg_inf(), M_b = neg_inf();
  for (int i = 0; i < parts; ++i) {
    const float4 st = p.part_ml[slot(i) * kSoftThreads + threadIdx.x];
    M_a = fmaxf(M_a, st.x);
    M_b = fmaxf(M_b, st.z);
  }
  float L_a = 0.f, L_b = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
#pragma unroll 2
  for (int i = 0; i < parts; ++i) {
    const int64_t s = slot(i);
    const float4 st = p.part_ml[s * kSoftThreads + threadIdx.x];
    const float4* src = p.part_o + (s * (D / 8) + 4 * mb) * kSoftThreads + threadIdx.x;
    float4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = src[e * kSoftThreads];
    // a part whose rows see none of its keys has m = -inf and adds nothing
    const float fa = st.x == neg_inf() ? 0.f : ex2(st.x - M_a);
    const float fb = st.z == neg_inf() ? 0.f : ex2(st.z - M_b);
    L_a = fmaf(st.y, fa, L_a);
    L_b = fmaf(st.w, fb, L_b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[4 * e] = fmaf(v[e].x, fa, acc[4 * e]);
      acc[4 * e + 1] = fmaf(v[e].y, fa, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(v[e].z, fb, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(v[e].w, fb, acc[4 * e + 3]);
    }
  }
  const int head_shift = 7 - p.pos_shift;
  const bool live_a = (ra >> head_shift) < meta.z, live_b = (rb >> head_shift) < meta.z;
  const float inv_a = L_a > 0.f ? 1.f / L_a : 0.f, inv_b = L_b > 0.f ? 1.f / L_b : 0.f;
  const int64_t row_a = out_row(p, meta.y, meta.w, ra), row_b = out_row(p, meta.y, meta.w, rb);
  store_chunks<kF16>(reinterpret_cast<uint4*>(p.o + row_a * D), reinterpret_cast<uint4*>(p.o + row_b * D), acc, inv_a,
                     inv_b, 4 * mb, lane & 3, live_a, live_b);
  if (mb == 0 && (lane & 3) == 0 && p.lse) {
    if (live_a) p.lse[row_a] = L_a > 0.f ? (M_a + log2f(L_a)) * kLn2 : neg_inf();
    if (live_b) p.lse[row_b] = L_b > 0.f ? (M_b + log2f(L_b)) * kLn2 : neg_inf();
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A tensor of `rank` dimensions, boxes of 64 x box[1] x ... elements, 128B
// swizzle. strides in elements, from dimension 1 on; a dimension of size 1 takes
// any stride.
bool make_map(CUtensorMap* map, const uint16_t* base, bool f16, int rank, const int64_t* dims, const int64_t* strides,
              const int* boxes) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t gd[4], gs[3];
  cuuint32_t box[4], es[4];
  for (int i = 0; i < rank; ++i) {
    gd[i] = static_cast<cuuint64_t>(dims[i]);
    box[i] = static_cast<cuuint32_t>(boxes[i]);
    es[i] = 1;
    if (i > 0) gs[i - 1] = static_cast<cuuint64_t>(dims[i] > 1 ? strides[i - 1] * 2 : dims[0] * 2);
  }
  return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank),
             const_cast<uint16_t*>(base), gd, gs, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// Heads of one key head that a tile packs: a power of two, at most 128.
int pack_heads(int group) {
  int n = 1;
  while (n < kBM && group % (2 * n) == 0) n *= 2;
  return n;
}

// Shares a CTA takes one after the other. The CTAs' shares of one round are
// neighbours in the row of items, so that the K and V they read at one time are
// about 1 / rounds of all; that part should stay in L2 (half of its 129 MB), since
// every query tile reads it again.
int round_count(int64_t tokens_k, int Hkv, int D) {
  const int64_t bytes = tokens_k * Hkv * D * 4, part = int64_t(64) << 20;
  const int64_t n = (bytes + part - 1) / part;
  return n < 1 ? 1 : (n > kMaxRounds ? kMaxRounds : static_cast<int>(n));
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

template <int D, bool kF16>
cudaError_t launch_shape(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PackedParams& p,
                         int ctas, cudaStream_t stream) {
  static std::atomic<bool> smem_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_packed_kernel<D, kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) smem_set[dev].store(true, std::memory_order_release);
  }
  attn_packed_kernel<D, kF16><<<ctas, kThreads, Smem<D>::kBytes, stream>>>(mq, mk, mv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * p.rounds, D / 32);
  cfg.blockDim = dim3(kSoftThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_packed_join_kernel<D, kF16>, p);
}

}  // namespace

int device_sms() {
  static std::atomic<int> cached[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if ((sms = cached[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cached[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

int64_t attn_packed_workspace_bytes(int64_t tokens_k, int Hkv, int D) {
  const int sms = device_sms();
  if (sms < 1) return -1;
  const int64_t shares = static_cast<int64_t>(sms) * round_count(tokens_k, Hkv, D);
  return round256(2 * shares * (D / 8) * kSoftThreads * 16) + round256(2 * shares * kSoftThreads * 16) +
         round256(shares * 16);
}

cudaError_t launch_attn_packed(const PackedArgs& a, void* workspace, unsigned int* err, const AttnFault& fault,
                               cudaStream_t stream) {
  const int sms = device_sms();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int group = a.Hq / a.Hkv, heads = pack_heads(group);
  int pos_shift = 7;
  while ((kBM >> pos_shift) < heads) --pos_shift;

  CUtensorMap mq, mk, mv;
  const int64_t q_dims[4] = {a.D, heads, a.Hq / heads, a.tokens_q};
  const int64_t q_strides[3] = {a.ld_q_head, a.ld_q_head * heads, a.ld_q_token};
  const int q_box[4] = {64, heads, 1, kBM / heads};
  // without keys nothing of k and v is read: any mapped row stands in for them
  const bool keys = a.tokens_k > 0;
  const int64_t k_dims[3] = {a.D, keys ? a.Hkv : 1, keys ? a.tokens_k : 1};
  const int64_t k_strides[2] = {a.ld_kv_head, a.ld_kv_token};
  const int k_box[3] = {64, 1, kBN};
  if (!make_map(&mq, a.q, a.f16, 4, q_dims, q_strides, q_box) ||
      !make_map(&mk, keys ? a.k : a.q, a.f16, 3, k_dims, k_strides, k_box) ||
      !make_map(&mv, keys ? a.v : a.q, a.f16, 3, k_dims, k_strides, k_box))
    return cudaErrorInvalidValue;

  PackedParams p;
  p.o = a.o;
  p.lse = a.lse;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.batch = a.batch;
  p.tokens_q = static_cast<int32_t>(a.tokens_q);
  p.tokens_k = static_cast<int32_t>(a.tokens_k);
  p.Hq = a.Hq;
  p.packs = a.Hq / heads;
  p.packs_per_key_head = group / heads;
  p.pos_shift = pos_shift;
  p.rounds = round_count(a.tokens_k, a.Hkv, a.D);
  p.C = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634074);
  p.causal = a.causal ? 1 : 0;
  p.err = err;
  p.timeout_ns = fault.timeout_ns > 0 ? static_cast<uint64_t>(fault.timeout_ns) : kTimeoutNs;
  static std::atomic<unsigned int> launches{0};
  p.tag = launches.fetch_add(1, std::memory_order_relaxed) % 65535u + 1u;
  p.skip_v_step = fault.skip_v_step;
  const int64_t shares = static_cast<int64_t>(sms) * p.rounds;
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float4*>(ws);
  ws += round256(2 * shares * (a.D / 8) * kSoftThreads * 16);
  p.part_ml = reinterpret_cast<float4*>(ws);
  ws += round256(2 * shares * kSoftThreads * 16);
  p.meta = reinterpret_cast<int4*>(ws);
  if (a.D == 128)
    return a.f16 ? launch_shape<128, true>(mq, mk, mv, p, sms, stream) : launch_shape<128, false>(mq, mk, mv, p, sms, stream);
  return a.f16 ? launch_shape<64, true>(mq, mk, mv, p, sms, stream) : launch_shape<64, false>(mq, mk, mv, p, sms, stream);
}

}  // namespace oss
