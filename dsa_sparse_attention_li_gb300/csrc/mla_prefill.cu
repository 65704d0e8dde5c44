// mla_prefill.cu -- dense latent attention, expanded form: causal flash attention over packed
// sequences with 192-column queries and keys (128 of the head's own, 64 of the rope key that all
// heads share) and 128-column values.
//
// A CTA takes 256 consecutive tokens of one sequence and head as two row tiles A and B of 128, and
// walks the keys in tiles of 128.  The tensor pipe works on one row tile while the softmax of the
// other runs:
//   ... P_A(j).V(j) -> O_A,  Q_A.K(j+1)^T -> S_A,  P_B(j).V(j) -> O_B,  Q_B.K(j+1)^T -> S_B ...
// TMEM: S_A, S_B, O_A, O_B, 128 columns each; P (bf16) takes the place of the first half of its S,
// as the A operand of P.V.  A softmax thread owns a row: no exchange, the maximum and the sum stay
// in registers; O is rescaled only when a row's maximum outgrows its reference by 2^8 (per warp).
// P is handed over in two halves, so that P.V starts under the second half's exponentials (in four:
// 1,274 us against 1,201).
//
// Shared memory: Q (96 KB) and a ring of eight 16-KB blocks: a key tile is three (64 columns each), a
// value tile two (64 keys each), in the order K0 V0 K1 V1 ...  V(j) then loads a whole step ahead of
// its use, and K(j+1) from the release of V(j-1) on, which leaves it half a step (with K(j+1) before
// V(j) the tensor pipe waited 1,500 of 4,400 cycles a step for V).
//
// Items (token block, head) are the grid's blocks; a CTA asks for another block that has not started
// (cluster launch control) while it works on one, so that the next item's loads and first products
// run under the last softmax and the epilogue of the one before.
//
// Bound: the tensor pipe, 2 * (12 + 8) MMAs of 64 cycles (67 measured) a key tile and CTA = 2,560 cycles for 21
// MFLOP; the keys and values come from L2, which the CTAs of a head share (heads in groups of 16,
// the longest token blocks of a group first).
#include <algorithm>

#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {
namespace mlap {

constexpr int kThreads = 384;   // warps 0-3 softmax of A, 4-7 of B, 8 MMA, 9 loads, 10-11 edge tiles
constexpr int kRows = 128, kKeys = 128, kTokens = 2 * kRows;
constexpr int kDqk = 192, kDv = 128;
constexpr int kBlock = 16384;   // 128 keys x 64 columns, or 64 keys x 128 columns
constexpr int kBlocks = 8;
constexpr int kParts = 2;       // of P, handed over one by one
constexpr int kHeadGroup = 16;
constexpr float kRescaleLog2 = 8.0f;
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;  // A, then B 128 columns on

struct Params {
  int B, n_q, n_kv, H, max_q, blocks;
  float scale_log2;
  const int* q_start;
  const int* kv_start;
  __nv_bfloat16* out;
  float* lse;
  int* status;
#ifdef DSA_TEST_HOOKS
  int stall;       // test build: the first CTA's MMA warp waits on a barrier nothing arrives on (4), or
                   // its first load of keys (7), of values (8) or of queries (9) is left out
#endif
};

struct Layout {
  static constexpr int q = 0;                       // [A, B][3 blocks of 64 columns][128 rows]
  static constexpr int ring = q + 6 * kBlock;
  static constexpr int ctl = ring + kBlocks * kBlock;
  static constexpr int total = ctl + 2048;
};

// What the warps know of an item.
struct Item {
  int h, tok, key, n_key;   // head; first token and first key row; keys of the sequence
  int seen0;                // keys that the block's first token sees (may be < 1)
  int rows_a, rows_b, na, nb;   // tokens and key tiles of A and B
  int tiles;                // max(na, nb); 0: no further item
  int edge0;                // tiles from here on are edge tiles: some token does not see all of it
};

struct Ctl {
  uint64_t q_full[2], q_empty[2], full[kBlocks], empty[kBlocks];
  uint64_t s_full[2], p_full[2][kParts], pv_done[2];
  uint64_t edge[2][2];       // values of an edge tile (by its count & 1), half, have landed
  uint64_t item_full[2], item_empty[2], answer_full;
  alignas(16) uint8_t answer[16];
  Item item[2];
#ifdef DSA_TEST_HOOKS
  uint64_t never;      // test build: no thread ever arrives here
#endif
  uint32_t tmem_base;
  int abort;
  uint32_t any_bad[2][2];    // t + 1 if a half of edge tile t (of all the CTA's tiles) has value rows
                             // that are not finite
  alignas(4) uint8_t bad[2][kKeys];   // those rows (by t & 1)
};
static_assert(sizeof(Ctl) <= 2048, "control block");

// Position of a key tile's first block, and of a value tile's, in the line of blocks that the ring
// carries (`at`: the item's first); block i lies in slot i % 8, in its (i / 8)th use.
DSA_DEV uint32_t k_block(uint32_t at, int j) { return at + 5u * j; }
DSA_DEV uint32_t v_block(uint32_t at, int j) { return at + 5u * j + 3u; }

// Where the sequences before the lane's end, at most: `ends` for those of earlier chunks.
__device__ __noinline__ int earlier_end(int end, int ends) {
  const int lane = threadIdx.x & 31;
  int upto = max(ends, __shfl_up_sync(0xffffffffu, end, 1));
  if (lane == 0) upto = ends;
  for (int o = 1; o < 32; o <<= 1) upto = max(upto, __shfl_up_sync(0xffffffffu, upto, o));
  return upto;
}

// The line of all sequences' token blocks, one sequence after the other, of which p.blocks is the
// host's bound; the loading warp looks items up in it.  Lane i holds sequence b0 + i.
// The bound holds for sequences that share no token.  Where q_start falls, two could claim the same ones:
// the first has them, and one that starts before the end of an earlier one is skipped.
struct Line {
  int s0, s1, k0, k1, first, count;   // its ranges, and its blocks in the line
  int ends;      // where the sequences so far end, at most
  bool rising;   // no q_start so far was out of order

  // Sequences b0 .. b0 + 31, which the line reaches at `before` (the chunks in their order, the first
  // one at 0); returns where they end.
  DSA_DEV int chunk(const Params& p, int b0, int before, int lane, bool tell) {
    if (b0 == 0) {
      ends = 0;
      rising = true;
    }
    const int b = b0 + lane;
    s0 = s1 = k0 = k1 = 0;
    if (b < p.B) {
      s0 = p.q_start[b];
      s1 = p.q_start[b + 1];
      k0 = p.kv_start[b];
      k1 = p.kv_start[b + 1];
    }
    bool fine = s0 >= 0 && s1 >= s0 && s1 <= p.n_q;
    const int end = fine && s1 > s0 ? s1 : 0;
    rising = rising && __all_sync(0xffffffffu, fine);   // (each starts where the one before it ends)
    if (!rising) {
      const int from = earlier_end(end, ends);   // (of the whole warp)
      fine = fine && s0 >= from;
    }
    ends = max(ends, __reduce_max_sync(0xffffffffu, end));
    fine = fine && k0 >= 0 && k1 >= k0 && k1 <= p.n_kv;
    if (tell && (!fine || s1 - s0 > p.max_q)) report(p.status, kStatusDeviceCheck);
    count = fine ? (s1 - s0 + kTokens - 1) / kTokens : 0;
    int upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    first = before + upto - count;
    return before + __shfl_sync(0xffffffffu, upto, 31);
  }
  // Grid block i: by head group, then token blocks by their place in their sequence, the last first
  // (the longest; with more than 32 sequences: from the line's end), then heads.
  DSA_DEV bool find(const Params& p, int i, int lane, Item& w) {
    const int group = i / (p.blocks * kHeadGroup);
    const int heads = min(kHeadGroup, p.H - group * kHeadGroup);
    i -= group * p.blocks * kHeadGroup;
    w.h = group * kHeadGroup + i % heads;
    int rank = i / heads, l = -1, block = 0;
    if (p.B <= 32) {
      for (int k = __reduce_max_sync(0xffffffffu, count) - 1; k >= 0; --k) {
        const uint32_t have = __ballot_sync(0xffffffffu, count > k);
        if (rank < __popc(have)) {  // its (rank + 1)th sequence
          l = __ffs((int)__ballot_sync(0xffffffffu, count > k && __popc(have & ((1u << lane) - 1u)) == rank)) - 1;
          block = k;
          break;
        }
        rank -= __popc(have);
      }
    } else {
      const int want = p.blocks - 1 - rank;
      uint32_t hit = 0;
      for (int b0 = 0, at = 0; b0 < p.B && hit == 0; b0 += 32) {
        at = chunk(p, b0, at, lane, false);
        hit = __ballot_sync(0xffffffffu, want >= first && want < first + count);
      }
      if (hit != 0) {
        l = __ffs((int)hit) - 1;
        block = want - __shfl_sync(0xffffffffu, first, l);
      }
    }
    if (l < 0) return false;  // the line is shorter than its bound
    const int t0 = block * kTokens;
    const int q0 = __shfl_sync(0xffffffffu, s0, l), n_tok = __shfl_sync(0xffffffffu, s1, l) - q0;
    w.key = __shfl_sync(0xffffffffu, k0, l);
    w.n_key = __shfl_sync(0xffffffffu, k1, l) - w.key;
    w.tok = q0 + t0;
    w.seen0 = w.n_key - n_tok + t0 + 1;
    w.rows_a = min(kRows, n_tok - t0);
    w.rows_b = max(0, min(kRows, n_tok - t0 - kRows));
    w.na = max(1, (w.seen0 + w.rows_a - 1 + kKeys - 1) / kKeys);
    w.nb = w.rows_b > 0 ? max(1, (w.seen0 + kRows + w.rows_b - 1 + kKeys - 1) / kKeys) : 0;
    w.tiles = max(w.na, w.nb);
    w.edge0 = min(max(w.seen0, 0) / kKeys, w.tiles);
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_r,
                       const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + Layout::ctl);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort = &ctl->abort;

  if (tid == 0) {
    mbar_init(&ctl->answer_full, 1);
    for (int i = 0; i < kBlocks; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      for (int c = 0; c < kParts; ++c) mbar_init(&ctl->p_full[i][c], 4);
      mbar_init(&ctl->pv_done[i], 1);
      mbar_init(&ctl->item_full[i], 1);
      mbar_init(&ctl->item_empty[i], 11);  // all warps but this one
      mbar_init(&ctl->edge[i][0], 1);
      mbar_init(&ctl->edge[i][1], 1);
    }
#ifdef DSA_TEST_HOOKS
    mbar_init(&ctl->never, 1);
#endif
    ctl->abort = 0;
    for (int i = 0; i < 4; ++i) ctl->any_bad[i >> 1][i & 1] = 0u;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  griddep_wait();  // nothing above reads global memory
  uint32_t at = 0;   // the item's first ring block; at / 5 is its first tile of the CTA's

  if (warp == 9) {
    // ---------------- items and loads
    uint32_t edges = 0, loads_a = 0, loads_b = 0;   // edge tiles, and loads of A's and B's queries, so far
    // (test build: whether the first CTA leaves a load out, so that its bytes never come)
    auto lost = [&](int which) {
#ifdef DSA_TEST_HOOKS
      return p.stall == which && blockIdx.x == 0;
#else
      return false;
#endif
    };
    // After a wait that gave up nothing is armed any more, and the warps of the edge tiles arrive on nothing
    // that is: an arrival on a barrier whose bytes are still on their way, its only expected one, faulted.
    auto load = [&](const Item& w) {
      // (A's last product with its queries is half a step or more before B's, whose new queries are
      // waited for after the first keys and values)
      auto load_q = [&](int x, uint32_t& loads) {
        if (loads > 0 && !mbar_wait_fast(&ctl->q_empty[x], (loads - 1) & 1u, abort, p.status)) return;
        ++loads;
        mbar_arrive_expect_tx(&ctl->q_full[x], 3 * kBlock);
        for (int c = lost(9) ? 1 : 0; c < 3; ++c)
          tma_load_3d(smem + Layout::q + (x * 3 + c) * kBlock, &tm_q, &ctl->q_full[x], c * 64, w.h, w.tok + x * kRows);
      };
      load_q(0, loads_a);
      // block i may take its slot once block i - 8 is used up
      auto free = [&](uint32_t i) {
        if (i >= kBlocks) mbar_wait_fast(&ctl->empty[i % kBlocks], (i / kBlocks - 1) & 1u, abort, p.status);
        return !*abort;
      };
      auto arm = [&](uint32_t i, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, kBlock);
        return smem + Layout::ring + (i % kBlocks) * kBlock;
      };
      for (int j = 0; j < w.tiles && !*abort; ++j) {
        const int key = w.key + j * kKeys;
        for (int c = 0; c < 3; ++c) {
          const uint32_t i = k_block(at, j) + c;
          uint64_t* bar = &ctl->full[i % kBlocks];
          if (!free(i)) return;
          uint8_t* dst = arm(i, bar);
          if (i == 0 && lost(7)) continue;
          if (c < 2)
            tma_load_3d(dst, &tm_k, bar, c * 64, w.h, key);
          else
            tma_load_2d(dst, &tm_r, bar, 0, key);
        }
        for (int c = 0; c < 2; ++c) {
          const uint32_t i = v_block(at, j) + c;
          uint64_t* bar = j < w.edge0 ? &ctl->full[i % kBlocks] : &ctl->edge[edges & 1u][c];
          if (!free(i)) return;
          uint8_t* dst = arm(i, bar);
          for (int u = i == 3 && lost(8) ? 1 : 0; u < 2; ++u)
            tma_load_3d(dst + u * (kBlock / 2), &tm_v, bar, 128 + u * 64, w.h, key + c * 64);
        }
        if (j >= w.edge0) ++edges;
        if (j == 0 && w.nb > 0) load_q(1, loads_b);
      }
    };
    Line line;
    const bool tell = blockIdx.x == 0;   // this CTA looks at every sequence
    for (int b0 = 0, end = 0; b0 < (tell ? p.B : min(p.B, 32)); b0 += 32) end = line.chunk(p, b0, end, lane, tell);
    uint32_t item = 0;
    // room for item number `item` in its slot, two items back (after a wait that gave up the slot may still be
    // read: it stays as it is, and the others leave by the abort flag)
    auto room = [&] {
      if (item > 1) mbar_wait_fast(&ctl->item_empty[item & 1u], ((item >> 1) - 1) & 1u, abort, p.status);
      __syncwarp();
    };
    int index = (int)blockIdx.x;
    for (uint32_t asked = 0; index >= 0; ++asked) {
      if (lane == 0) {  // the next index is on its way while this item's loads are issued
        mbar_arrive_expect_tx(&ctl->answer_full, 16);
        clc_try_cancel(ctl->answer, &ctl->answer_full);
      }
      Item w;
      if (line.find(p, index, lane, w)) {
        room();
        if (lane == 0 && !*abort) {
          ctl->item[item & 1u] = w;
          mbar_arrive(&ctl->item_full[item & 1u]);
          load(w);
        }
        __syncwarp();
        at += 5u * w.tiles;
        ++item;
      }
      warp_wait(&ctl->answer_full, asked & 1u, abort, p.status);
      index = __shfl_sync(0xffffffffu, *abort ? -1 : clc_block(ctl->answer), 0);
      // (the next answer is written through the async proxy, after these reads)
      fence_proxy_async_smem();
      __syncwarp();
    }
    room();
    if (lane == 0 && !*abort) {
      ctl->item[item & 1u].tiles = 0;
      mbar_arrive(&ctl->item_full[item & 1u]);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------- edge tiles: half c of the values of a tile that some token of the block does not
    // see to its end.  What a token does not see must not reach it, and a weight of 0 times NaN would:
    // value rows past the sequence become zeros, and in the others what is not finite, whose tokens
    // then get their NaN through the score.
    const int c = warp - 10;
    uint32_t edges = 0;
    for (uint32_t item = 0;; ++item) {
      warp_wait(&ctl->item_full[item & 1u], (item >> 1) & 1u, abort, p.status);
      const Item& w = ctl->item[item & 1u];
      const int tiles = w.tiles, edge0 = w.edge0, n_key = w.n_key;
      if (tiles == 0 || __any_sync(0xffffffffu, *abort)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->item_empty[item & 1u]);
      for (int j = edge0; j < tiles; ++j, ++edges) {
        warp_wait(&ctl->edge[edges & 1u][c], (edges >> 1) & 1u, abort, p.status);
        const uint32_t t = at / 5u + j, slot = (v_block(at, j) + c) % kBlocks;
        const int rows = min(max(n_key - j * kKeys - c * 64, 0), 64);   // of the sequence
        uint8_t* half = smem + Layout::ring + slot * kBlock;
        auto piece = [&](int r, int ch) {   // 16 bytes of row r
          return reinterpret_cast<uint4*>(half + (ch >> 3) * (kBlock / 2) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
        };
        // is anything not finite?  (an exponent of all ones is the only one that a 1 carries out of)
        uint32_t odd = 0;
#pragma unroll 8
        for (int r2 = 0; r2 < 64; r2 += 2) {  // two rows at a time, 16 lanes each
          const int r = r2 + (lane >> 4);
          const uint4 v = *piece(r, lane & 15);
          const uint32_t o = ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                             ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
          if (r < rows) odd |= o;
        }
        const bool any = __any_sync(0xffffffffu, (odd & 0x80008000u) != 0u);
        if (lane < 16) reinterpret_cast<uint32_t*>(ctl->bad[t & 1u] + c * 64)[lane] = 0u;
        __syncwarp();
        for (int r2 = any ? 0 : rows & ~1; r2 < 64; r2 += 2) {
          const int r = r2 + (lane >> 4), ch = lane & 15;
          uint4 v = *piece(r, ch);
          const uint4 was = v;
          v = r < rows ? make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w))
                       : make_uint4(0u, 0u, 0u, 0u);
          *piece(r, ch) = v;
          const uint32_t votes = __ballot_sync(
              0xffffffffu, r < rows && (v.x != was.x || v.y != was.y || v.z != was.z || v.w != was.w));
          if (ch == 0 && ((votes >> (lane & 16)) & 0xffffu)) ctl->bad[t & 1u][c * 64 + r] = 1;
        }
        if (any && lane == 0) ctl->any_bad[t & 1u][c] = t + 1u;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !*abort) mbar_arrive(&ctl->full[slot]);   // (see the loads)
      }
      at += 5u * tiles;
    }
  } else if (warp == 8) {
    // ---------------- MMA issue: the whole warp walks, one lane issues
    constexpr uint32_t idesc_qk = idesc_bf16(kRows, kKeys);
    constexpr uint32_t idesc_pv = idesc_bf16(kRows, kDv, /*b_mn_major=*/true);
    const uint64_t qd = sdesc_sw128(smem_u32(smem + Layout::q), 16, 1024);
    const uint64_t kd = sdesc_sw128(smem_u32(smem + Layout::ring), 16, 1024);
    const uint64_t vd = sdesc_sw128(smem_u32(smem + Layout::ring), kBlock / 2, 1024);
    const uint32_t me = elect_one();
    auto issue_wait = [&](uint64_t* bar, uint32_t parity) {
      mbar_wait_issue<false>(bar, parity, abort, p.status);
      __syncwarp();
    };
    auto wait_block = [&](uint32_t i) {
      issue_wait(&ctl->full[i % kBlocks], (i / kBlocks) & 1u);
      tc_fence_after();
    };
    // Q_x . K(j)^T; the first row tile to use a key tile waits for it, the last one releases it
    uint32_t done[2] = {0, 0}, with_b = 0;   // tiles that row tile x had in earlier items; items with a B
    auto qk = [&](int x, int j, bool wait, bool release, bool last) {
      const uint64_t a = desc_at(qd, x * 3 * kBlock);
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const uint32_t i = k_block(at, j) + c;
        if (wait) wait_block(i);
        const uint64_t k = desc_at(kd, (i % kBlocks) * kBlock);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_ss_by(tmem + kColS + x * 128, desc_at(a, c * kBlock + kk * 32), desc_at(k, kk * 32), idesc_qk,
                        (c > 0 || kk > 0) ? 1u : 0u, me);
        if (release) mma_commit_by(&ctl->empty[i % kBlocks], me);
      }
      mma_commit_by(&ctl->s_full[x], me);
      if (last) mma_commit_by(&ctl->q_empty[x], me);
    };
    auto pv = [&](int x, int j, bool wait, bool release) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t i = v_block(at, j) + c;
        if (wait) wait_block(i);
        const uint64_t v = desc_at(vd, (i % kBlocks) * kBlock);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk % (8 / kParts) == 0) {
            issue_wait(&ctl->p_full[x][(c * 4 + kk) * kParts / 8], (done[x] + j) & 1u);
            tc_fence_after();
          }
          mma_f16_ts_by(tmem + kColO + x * 128, tmem + kColS + x * 128 + c * 32 + kk * 8, desc_at(v, kk * 2048),
                        idesc_pv, (c > 0 || kk > 0) ? 1u : j > 0 ? 1u : 0u, me);
        }
        if (release) mma_commit_by(&ctl->empty[i % kBlocks], me);
      }
      mma_commit_by(&ctl->pv_done[x], me);
    };
#ifdef DSA_TEST_HOOKS
    if (p.stall == 4 && blockIdx.x == 0) warp_wait(&ctl->never, 0, abort, p.status);
#endif
    // (a row tile's first products of an item may overwrite S, whose weights the last P.V has read by
    // then, and O, which its softmax warps have read before they hand over new weights)
    for (uint32_t item = 0;; ++item) {
      warp_wait(&ctl->item_full[item & 1u], (item >> 1) & 1u, abort, p.status);
      const Item& w = ctl->item[item & 1u];
      const int na = __shfl_sync(0xffffffffu, w.na, 0), nb = __shfl_sync(0xffffffffu, w.nb, 0),
                tiles = __shfl_sync(0xffffffffu, w.tiles, 0);
      if (tiles == 0 || __any_sync(0xffffffffu, *abort)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->item_empty[item & 1u]);
      issue_wait(&ctl->q_full[0], item & 1u);
      qk(0, 0, true, nb == 0, na == 1);
      if (nb > 0) {
        issue_wait(&ctl->q_full[1], with_b & 1u);
        ++with_b;
        qk(1, 0, false, true, nb == 1);
      }
#pragma unroll 1
      for (int j = 0; j < tiles; ++j) {
        if (__any_sync(0xffffffffu, *abort)) break;
        if (j < na) pv(0, j, true, j >= nb);
        if (j + 1 < na) qk(0, j + 1, true, j + 1 >= nb, j + 2 == na);
        if (j < nb) pv(1, j, j >= na, true);
        if (j + 1 < nb) qk(1, j + 1, j + 1 >= na, true, j + 2 == nb);
      }
      done[0] += na;
      done[1] += nb;
      at += 5u * tiles;
    }
  } else if (warp < 8) {
    // ---------------- softmax of row tile x: a thread is a row
    const int x = warp >> 2;
    const int row = tid & 127;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_addr + kColS + x * 128, o_at = lane_addr + kColO + x * 128;
    uint32_t done = 0;   // tiles of earlier items
    for (uint32_t item = 0;; ++item) {
      warp_wait(&ctl->item_full[item & 1u], (item >> 1) & 1u, abort, p.status);
      const volatile Item& w = ctl->item[item & 1u];
      if (w.tiles == 0 || __any_sync(0xffffffffu, *abort)) break;
      const int n = x == 0 ? w.na : w.nb, rows = x == 0 ? w.rows_a : w.rows_b;
      // rows past the block's tokens count as seeing everything: no masking, nothing of them is kept
      const int seen = row < rows ? w.seen0 + x * kRows + row : 0x7fffffff;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        warp_wait(&ctl->s_full[x], (done + j) & 1u, abort, p.status);
        bool bad_tile = false;
        const uint32_t t = at / 5u + j;
        if (j >= w.edge0) {
          // (after the scores: the slots' previous uses, of K(j-1), are over by then, so that the parity
          // of this wait means this use)
          for (uint32_t i = v_block(at, j); i < v_block(at, j) + 2; ++i)
            warp_wait(&ctl->full[i % kBlocks], (i / kBlocks) & 1u, abort, p.status);
          const volatile uint32_t* any = ctl->any_bad[t & 1u];
          bad_tile = any[0] == t + 1u || any[1] == t + 1u;
        }
        tc_fence_after();
        uint32_t s[128];
        tmem_ld_x32(s_at, s);
        tmem_ld_x32(s_at + 32, s + 32);
        tmem_ld_wait();
        tmem_ld_x32(s_at + 64, s + 64);   // on its way under the first half's maxima
        tmem_ld_x32(s_at + 96, s + 96);
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const int keep = seen - j * kKeys;  // the first keys of the tile that are seen
        const bool all = __all_sync(0xffffffffu, keep >= kKeys) && !bad_tile;
        auto maxima = [&](int from) {   // of half a row, with what is not seen taken out
          if (!all) {
#pragma unroll
            for (int c = from; c < from + 64; ++c)
              if (c >= keep) s[c] = 0xff800000u;
            if (bad_tile) {
#pragma unroll
              for (int c = from; c < from + 64; ++c)
                if (c < keep && ctl->bad[t & 1u][c]) s[c] = 0x7fffffffu;
            }
          }
#pragma unroll
          for (int c = from; c < from + 64; c += 2)
            m4[(c >> 1) & 3] = max3(m4[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        };
        maxima(0);
        tmem_ld_wait();
        maxima(64);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
        if (__any_sync(0xffffffffu, row < rows && mx > m_ref + kRescaleLog2)) {
          const float m_new = fmaxf(m_ref, mx);
          const float alpha = m_new == m_ref ? 1.f : fast_exp2(m_ref - m_new);
          m_ref = m_new;
          l *= alpha;
          if (j > 0) {
            warp_wait(&ctl->pv_done[x], (done + j - 1) & 1u, abort, p.status);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld_x16(o_at + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st_x16(o_at + c * 16, o);
            }
            tmem_st_wait();
          }
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          constexpr int kCols = 128 / kParts;
#pragma unroll
          for (int c = part * kCols; c < part * kCols + kCols; c += 2) {
            float2 e = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), p.scale_log2, -m_use);
            e.x = fast_exp2(e.x);
            e.y = fast_exp2(e.y);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], e);
            s[c >> 1] = pack_bf16(e.x, e.y);  // P.V takes bf16 weights: 2^-8 relative each, unbiased
          }
#pragma unroll
          for (int c = part * (kCols / 2); c < (part + 1) * (kCols / 2); c += 16) tmem_st_x16(s_at + c, s + c);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->p_full[x][part]);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // ---------------- rows out
      done += n;
      if (n > 0) {
        warp_wait(&ctl->pv_done[x], (done - 1) & 1u, abort, p.status);
        tc_fence_after();
        if (l == 0.f && seen > 0) l = __uint_as_float(0x7fffffffu);   // all scores -inf, or +inf by the scale
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t to = (size_t)(w.tok + x * kRows + row) * p.H + w.h;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld_x32(o_at + c * 32, o);
          tmem_ld_wait();
          if (row < rows) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              o[k] = pack_bf16(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
            st_global_v8(p.out + to * kDv + c * 32, o);
            st_global_v8(p.out + to * kDv + c * 32 + 16, o + 8);
          }
        }
        if (row < rows && p.lse) p.lse[to] = l == 0.f ? -INFINITY : m_ref * 0.69314718055994531f + logf(l);
      }
      at += 5u * w.tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->item_empty[item & 1u]);
    }
  }
  if (ctl->abort) {  // copies may still be in flight: give them time to land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000u) {
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace mlap

dsa_status launch_mla_prefill(const dsa_mla_prefill_args& a, cudaStream_t stream, std::string& err) {
  using namespace mlap;
  Params p;
  p.B = a.B;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.H = a.H;
  p.max_q = a.max_q_per_seq;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.q_start = a.q_start;
  p.kv_start = a.kv_start;
  p.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  // every sequence has at most one block that is not full
  const long long blocks = (long long)a.n_q / kTokens + a.B, grid = blocks * a.H;
  if (blocks * std::max(a.H, kHeadGroup) > 0x7fff0000LL) {
    err = "mla_prefill: token blocks * heads (at least 16) must number below 2^31";
    return DSA_ERR_UNSUPPORTED;
  }
  p.blocks = (int)blocks;
#ifdef DSA_TEST_HOOKS
  p.stall = g_test_stall;
#endif
  // without any keys nothing is seen: any valid memory stands in for them
  const bool none = a.n_kv == 0;
  const uint64_t H = (uint64_t)a.H, keys = none ? 1 : (uint64_t)a.n_kv;
  const void* kv = none ? a.q : a.kv;
  const void* rope = none ? a.q : a.k_rope;
  const uint64_t qdims[3] = {kDqk, H, (uint64_t)a.n_q}, qstr[2] = {kDqk * 2, H * kDqk * 2};
  const uint64_t kvdims[3] = {none ? 192u : 256u, none ? 1 : H, keys}, kvstr[2] = {512, H * 512};
  const uint32_t box128[3] = {64, 1, 128}, box64[3] = {64, 1, 64};
  CUtensorMap tm_q, tm_k, tm_v, tm_r;
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_tmap_3d(&tm_q, bf, a.q, qdims, qstr, box128, sw, err) ||
      !encode_tmap_3d(&tm_k, bf, kv, kvdims, kvstr, box128, sw, err) ||
      !encode_tmap_3d(&tm_v, bf, kv, kvdims, kvstr, box64, sw, err) ||
      !encode_tmap_2d(&tm_r, bf, rope, 64, keys, none ? 128 : (uint64_t)a.k_rope_stride * 2, 64, 128, sw, err))
    return DSA_ERR_CUDA;
  const int smem = Layout::total + 1024;
  DeviceInfo dev;
  if (!device_info(dev, err)) return DSA_ERR_CUDA;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(mla_prefill_kernel), smem, dev.device, done);
  if (e != cudaSuccess) return cuda_fail(e, "mla_prefill: set shared memory size", err);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, mla_prefill_kernel, tm_q, tm_k, tm_v, tm_r, p);
  if (e != cudaSuccess) return cuda_fail(e, "mla_prefill: launch", err);
  return DSA_OK;
}

}  // namespace dsa
