// mla_decode.cu -- dense latent attention over the paged cache, absorbed form.
//
//   z_j = scale q.kv_j (576 columns),  out = sum_j softmax(z)_j kv_j[0:512],  j up to the token's own
//   position; flash attention with a running maximum and sum, the 64-token page as unit of the cache.
//
// Rows.  The T tokens of a sequence that share a pass over its cache, T = min(128 / H, tokens), give
// T * H <= 128 query rows: the M = 128 of one two-CTA MMA (cta_group::2), 64 rows a CTA.  O is then
// 64 x 512 fp32 a CTA, which in the two-CTA layout (two lanes a row) is 256 of the 512 TMEM columns,
// so each CTA owns whole rows: no score, maximum or weight ever crosses the pair (dsa_sfa_decode,
// whose O is split by columns, exchanges all three).
//
// Tiles of two pages.  Q.K^T has N = 128: CTA r supplies the 64 rows of page r (all 576 columns).
// P.V has N = 256 twice: CTA r supplies value columns [256 r, 256 r + 256) of both pages, 64-column
// blocks as MN-major operands.  The two uses need different halves of the tile, so a CTA loads its
// page and the other page's value half, and its own page's value half again (the operands of both
// CTAs must lie at the same offsets): 139 KB a tile and CTA against 74 KB that are distinct, from L2.
//
// Shared memory has room for one tile beside Q, so both operands are recycled in blocks: a K block
// (64 columns, 8 KB) is reloaded for the next tile as soon as its four MMAs are done, a V slot (64
// rows x 128 columns) likewise; the pages three tiles ahead are prefetched into L2 meanwhile.
//
// Work split.  Every group of T tokens counts ceil(length / 128) units of work; the units of all
// groups form one line, cut into one equal range per CTA pair (whole wave, any mix of lengths).  A
// group cut by a range border leaves normalised fp32 rows and their log-sum-exp in the workspace (at
// most two such pieces a pair), and a second kernel joins the pieces in order.
//
// An FP8 cache is read with plain loads and converted by eight warps into the same operands (at the MMAs'
// rate a code would need its scale, one a row and 128 columns, which no e4m3 MMA applies).
//
// Bound: HBM for one token a sequence (1152 B and 278,528 FLOP a position at H = 128: 242 FLOP/B),
// the tensor pipe for more.  A tile's 36 + 16 MMAs take 36 * 49 + 16 * 64 = 2,800 cycles.  With an FP8
// cache the conversion: K's slots are free only between two Q.K^T, and its three parts, one after the
// other, are 1,700 cycles each of loads, conversion and stores.
//
// Measured (join included, alone): 32 sequences of 32,768, one token: 128 heads 230 to 238 us by the GPU (5.2 TB/s,
// 78% of a copy's rate; 1,250 TFLOP/s; 250 us in a run of calls, at a lower clock), 16 heads 216 us; one of
// 131,072: 55 us; one of 4,096, 16 heads: 19 us.  FP8: 32 of 32,768, 128 heads 335 us, 16 ragged ones of
// up to 131,072 with two tokens and 64 heads 196 us.
#include <algorithm>

#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {
namespace mlad {

// Warps 0-3 softmax, 4 MMA (even CTA), 5 Q and K loads, 6 V loads; with an FP8 cache 5 loads Q, 8-11
// convert K and 12-15 convert V.
template <bool KV8>
constexpr int kThreads = KV8 ? 512 : 256;
constexpr int kKv8Row = 608;    // 576 e4m3 codes, 5 fp32 scales, 12 unused bytes
constexpr int kTile = 128;      // positions a tile
constexpr int kDqk = 576;
constexpr int kDv = 512;
constexpr int kKBlocks = 9;     // 64-column blocks of K (and of Q)
constexpr int kKGroups = 3;     // a barrier, and a reload, per three blocks
constexpr int kVPages = 2;      // V: a barrier, and a reload, per page of this CTA's 256 value columns
constexpr int kBlockBytes = 64 * 128;   // 64 rows x 64 bf16
constexpr int kKGroupBytes = 3 * kBlockBytes;
constexpr int kVHalfBytes = 2 * kBlockBytes;   // 128 columns of a page
constexpr int kVPageBytes = 2 * kVHalfBytes;
constexpr int kPrefetch = 3;    // tiles
constexpr float kRescaleLog2 = 8.0f;
constexpr float kNoScore = -3.402823466e38f;   // log-sum-exp of a piece with positions, but no score above -inf
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;

struct Params {
  int B, n_q, H, T, max_pages, num_pages;
  int pairs;
  float scale_log2;
  const uint8_t* kv;
  const int* page_table;
  const int* seq_lens;
  const int* q_start;
  __nv_bfloat16* out;
  float* lse;
  int* status;
  float* ws_o;     // [pairs][2][rows][512]
  float* ws_lse;   // [pairs][2][rows], log2
  int4* ws_join;   // [pairs] {first token, rows, first piece's slot, pieces} of the group that a
                   // pair's first unit continues; pieces 0: none, or another pair joins it
  int ws_rows;
#ifdef DSA_TEST_HOOKS
  int stall;       // test build: the first pair's MMA warp waits on a barrier nothing arrives on (3), or
                   // the first CTA's first load of keys (5) or values (6) is left out
#endif
};

struct Layout {
  static constexpr int q = 0;
  static constexpr int k = q + kKBlocks * kBlockBytes;
  static constexpr int v = k + kKBlocks * kBlockBytes;
  static constexpr int p = v + kVPages * kVPageBytes;
  static constexpr int ctl = p + 2 * kBlockBytes;
  static constexpr int total = ctl + 2048;
};

struct Ctl {
  uint64_t q_full, q_empty;
  uint64_t k_full[kKGroups], k_empty[kKGroups];
  uint64_t v_full[kVPages], v_empty[kVPages];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full, pv_done, o_free, edge;
  uint64_t written[kKGroups + kVPages];   // FP8: a part is in shared memory (four warps)
#ifdef DSA_TEST_HOOKS
  uint64_t never;      // test build: no thread ever arrives here
#endif
  uint32_t tmem_base;
  int abort;
  int start_b;
  int bad_pages;
  int piece[2];   // tiles of a piece
  long long start_at, part[16];
  float x[128];
};
static_assert(sizeof(Ctl) <= 2048, "control block");

// The same value, newly made: what is computed from it is not kept in registers over a loop (the MMA
// warp's 104 descriptor words cost the other warps their registers).
DSA_DEV uint32_t fresh(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}

// 16 e4m3 codes times their scale as bf16 (fp32 product, both roundings to nearest even): the operand
// that an element of an FP8 latent row stands for.
DSA_DEV void dequant16(const uint4& c, float s, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t two = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    const float2 f = mul2(__half22float2(*reinterpret_cast<const __half2*>(&h)), s);
    o[i] = pack_bf16(f.x, f.y);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// A lane's chunks of 16 codes of one FP8 row in one part of a tile, three of K or four of V, and the row's
// two scales there; chunks from `split` on have the second.
struct RowPart {
  uint4 code[4];
  float s0, s1;

  DSA_DEV void fetch(const uint8_t* row, int first, int q4, bool four) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u < 3 || four) code[u] = *reinterpret_cast<const uint4*>(row + (first + q4 + 4 * u) * 16);
    const float* s = reinterpret_cast<const float*>(row + kDqk) + (first >> 3);
    s0 = s[0];
    s1 = s[1];
  }
  // Into the row's line of 64-column blocks: chunk q4 + 4 u is pieces 2 q4 and 2 q4 + 1 of block u.
  DSA_DEV void store(uint8_t* line, uint32_t piece0, uint32_t piece1, int split, bool four) const {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (u == 3 && !four) break;
      uint4 lo, hi;
      dequant16(code[u], u >= split ? s1 : s0, lo, hi);
      *reinterpret_cast<uint4*>(line + u * kBlockBytes + piece0) = lo;
      *reinterpret_cast<uint4*>(line + u * kBlockBytes + piece1) = hi;
    }
  }
};

// Test build: whether the first CTA leaves a load out, so that its bytes never come.
DSA_DEV bool lost(const Params& p, int which) {
#ifdef DSA_TEST_HOOKS
  return p.stall == which && blockIdx.x == 0;
#else
  return false;
#endif
}

// How many of the 64 positions from pos0 on, a page of the sequence, a query row may use: those up to `seen`,
// none of a page that does not exist.  A row that is no one's (`owned` false: it counts as seeing everything)
// goes on past the sequence's last page, whose table may end there, so its pages are not looked up.
__host__ __device__ inline int visible_columns(bool owned, int seen, int pos0, bool check_pages, const int* pages,
                                               int num_pages) {
  const int keep = seen - pos0 < 64 ? seen - pos0 : 64;
  if (check_pages && owned && keep > 0) {
    const int pg = pages[pos0 >> 6];
    if (pg < 0 || pg >= num_pages) return 0;
  }
  return keep;
}

// A sequence's tokens and length, checked: n = 0 where q_start is out of order.
struct Seq {
  int s0, n, len;
};
DSA_DEV Seq sequence(const Params& p, int b, bool tell) {
  Seq s = {0, 0, 0};
  if (b < p.B) {
    const int s0 = p.q_start[b], s1 = p.q_start[b + 1], len = p.seq_lens[b];
    const int most = p.max_pages * 64;
    s.s0 = s0;
    s.len = max(0, min(len, most));
    const bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.n_q;
    s.n = ok ? s1 - s0 : 0;
    if (tell && (!ok || (s.n > 0 && (len < 0 || len > most)))) report(p.status, kStatusDeviceCheck);
  }
  return s;
}
DSA_DEV int unit_count(const Seq& s) { return max(1, (s.len + kTile - 1) / kTile); }
DSA_DEV long long units(const Params& p, const Seq& s) {
  return (long long)((s.n + p.T - 1) / p.T) * unit_count(s);
}

// One pair's share of the line of units, group by group.  Every warp walks it on its own.
struct Walk {
  int b, g;             // sequence, token group
  long long at;         // line position of the group's first unit
  long long pos, end;   // the rest of the pair's range
  Seq s;
  // the current piece: tiles [tile0, tile1) of the group's `tiles`
  int tile0, tile1, tiles, t0, rows, seen_first, seen_last;
  bool first;

  DSA_DEV void set(const Params& p) {
    const int i0 = g * p.T, n = min(p.T, s.n - i0);
    t0 = s.s0 + i0;
    rows = n * p.H;
    seen_first = s.len - s.n + i0 + 1;   // positions that the group's first and last token see
    seen_last = seen_first + n - 1;
    tiles = max(1, (seen_last + kTile - 1) / kTile);
    const long long u = unit_count(s);
    const long long stop = at + u < end ? at + u : end;
    tile0 = (int)(pos - at);
    tile1 = min((int)(stop - at), tiles);
  }
  // Next piece with any tile in it; false at the end of the range.
  DSA_DEV bool next(const Params& p, int lane) {
    while (true) {
      const long long u = unit_count(s);
      pos = at + u;
      first = false;
      if (pos >= end) return false;
      at = pos;
      ++g;
      if ((long long)g * p.T >= s.n) {
        g = 0;
        while (true) {  // the next sequence with tokens (there is one: the range goes on)
          const Seq c = sequence(p, b + 1 + lane, false);
          const uint32_t some = __ballot_sync(0xffffffffu, c.n > 0);
          if (some == 0) {
            b += 32;
            if (b >= p.B) return false;
            continue;
          }
          const int l = __ffs((int)some) - 1;
          b += 1 + l;
          s.s0 = __shfl_sync(0xffffffffu, c.s0, l);
          s.n = __shfl_sync(0xffffffffu, c.n, l);
          s.len = __shfl_sync(0xffffffffu, c.len, l);
          break;
        }
      }
      set(p);
      if (tile0 < tile1) return true;
    }
  }
  DSA_DEV bool whole() const { return tile0 == 0 && tile1 == tiles; }
};

// Two rare questions, out of line: inlined, the code that is skipped cost a call on one page 4 us of 19
// (instructions come from memory then).

// Does a query row, which sees the sequence up to `seen`, see any position of the tiles [tile0, tile1)?
__device__ __noinline__ bool sees_any(const int* pages, int num_pages, int tile0, int tile1, int seen) {
  const int to = min(seen, tile1 * kTile);
  for (int i = tile0 * 2; i * 64 < to; ++i)
    if (pages[i] >= 0 && pages[i] < num_pages) return true;
  return false;
}

// First of the positions [first, last), which lie in one page, whose value columns hold something that is not
// finite; a large number if none does.  For a whole warp.
template <bool KV8>
__device__ __noinline__ int first_odd_row(const uint8_t* kv, const int* pages, int num_pages, int first, int last) {
  const int pg = first < last ? pages[first >> 6] : -1, lane = threadIdx.x & 31;
  if (pg < 0 || pg >= num_pages) return 0x7fffffff;
  for (int j = first; j < last; ++j) {
    const size_t row = (size_t)pg * 64 + (j & 63);
    uint4 v, w;
    if constexpr (KV8) {
      const uint8_t* r = kv + row * kKv8Row;
      dequant16(reinterpret_cast<const uint4*>(r)[lane], reinterpret_cast<const float*>(r + kDqk)[lane >> 3], v, w);
    } else {
      const uint4* r = reinterpret_cast<const uint4*>(kv + row * (kDqk * 2));
      v = r[lane];
      w = r[lane + 32];
    }
    auto odd = [](uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; };   // carries out of an exponent of all ones
    const uint32_t o = odd(v.x) | odd(v.y) | odd(v.z) | odd(v.w) | odd(w.x) | odd(w.y) | odd(w.z) | odd(w.w);
    if (__any_sync(0xffffffffu, (o & 0x80008000u) != 0u)) return j;
  }
  return 0x7fffffff;
}

template <bool KV8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<KV8>, 1)
    mla_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                      const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + Layout::ctl);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1;
  volatile int* abort = &ctl->abort;
  constexpr int kThr = kThreads<KV8>;
  constexpr uint32_t kFills = KV8 ? 2 : 1;   // arrivals that fill a K group or V page: one a CTA, or
                                             // one expect_tx
  if (tid == 0) {
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < kKGroups; ++i) {
      mbar_init(&ctl->k_full[i], kFills);
      mbar_init(&ctl->k_empty[i], 1);
    }
    for (int i = 0; i < kVPages; ++i) {
      mbar_init(&ctl->v_full[i], kFills);
      mbar_init(&ctl->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->s_free[i], 8);   // four softmax warps of either CTA
    }
    mbar_init(&ctl->p_full, 8);
    mbar_init(&ctl->pv_done, 1);
    mbar_init(&ctl->o_free, 8);
    mbar_init(&ctl->edge, 1);
    for (int i = 0; i < kKGroups + kVPages; ++i) mbar_init(&ctl->written[i], 4);
#ifdef DSA_TEST_HOOKS
    mbar_init(&ctl->never, 1);
#endif
    ctl->abort = 0;
    ctl->bad_pages = 0;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc2(&ctl->tmem_base, kTmemCols);
    tmem_relinquish2();
  }
  if (warp == 5 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_kv);
  }
  griddep_wait();  // nothing above reads global memory

  // ---------------- this pair's range of the line of units
  long long mine = 0;
  for (int b = tid; b < p.B; b += kThr) mine += units(p, sequence(p, b, blockIdx.x == 0));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) ctl->part[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kThr / 32; ++w) total += ctl->part[w];
  const long long share = max(1LL, (total + p.pairs - 1) / p.pairs);
  Walk w0;
  w0.pos = share * pair;
  w0.end = min(total, w0.pos + share);
  const bool any = w0.pos < total;
  if (any) {
    long long before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThr) {
      const long long u = units(p, sequence(p, b0 + tid, false));
      long long incl = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      __syncthreads();
      if (lane == 31) ctl->part[warp] = incl;
      __syncthreads();
      long long base = before, all = 0;
#pragma unroll
      for (int w = 0; w < kThr / 32; ++w) {
        if (w < warp) base += ctl->part[w];
        all += ctl->part[w];
      }
      const long long lo = base + incl - u;
      if (lo <= w0.pos && w0.pos < lo + u) {
        ctl->start_b = b0 + tid;
        ctl->start_at = lo;
      }
      before += all;
      if (before > w0.pos) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers and tensor memory of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  bool have = false;
  if (any) {
    w0.b = ctl->start_b;
    w0.s = sequence(p, w0.b, false);
    const long long u = unit_count(w0.s);
    w0.g = (int)((w0.pos - ctl->start_at) / u);
    w0.at = ctl->start_at + w0.g * u;
    w0.first = true;
    w0.set(p);
    have = w0.tile0 < w0.tile1 || w0.next(p, lane);
  }
  Walk w = w0;
  if (warp == 5) {
    // ---------------- Q and K loads, and the L2 prefetch
    const uint32_t q_full = map_cluster(&ctl->q_full, 0), k_full = map_cluster(&ctl->k_full[0], 0);
    const int oob = p.num_pages * 64;
    uint32_t it = 0, seg = 0;
    bool ok = true;
    for (; have && ok; have = w.next(p, lane), ++seg) {
      if (lane == 0) {
        ok = seg == 0 || mbar_wait(&ctl->q_empty, (seg - 1) & 1u, abort, p.status);
        if (ok) {
          if (rank == 0) {
            ctl->piece[seg & 1u] = w.tile1 - w.tile0;
            mbar_arrive_expect_tx(&ctl->q_full, 2 * kKBlocks * kBlockBytes);
          }
          for (int c = 0; c < kKBlocks; ++c)
            tma_load_2d_pair(smem + Layout::q + c * kBlockBytes, &tm_q, q_full, c * 64,
                             w.t0 * p.H + (int)rank * 64);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if constexpr (KV8) continue;
      const int* pt = p.page_table + (size_t)w.b * p.max_pages;
      const int pages = (max(w.seen_last, 0) + 63) >> 6;
      auto window = [&](int tile) {  // this CTA's page of tile + lane, -1: none
        const int i = 2 * (tile + lane) + (int)rank;
        if (tile + lane >= w.tile1 || i >= pages) return -1;
        const int pg = pt[i];
        return pg < p.num_pages ? pg : -1;
      };
      auto warm = [&](int pg) {
        if (pg >= 0 && lane == 0) prefetch_l2_bulk(p.kv + (size_t)pg * 64 * (kDqk * 2), 64 * kDqk * 2);
      };
      int cur = window(w.tile0), nxt = window(w.tile0 + 32);
      for (int i = w.tile0; i < w.tile1 && ok; ++i, ++it) {
        const int j = (i - w.tile0) & 31;
        if (j == 0 && i > w.tile0) {
          cur = nxt;
          nxt = window(i + 32);
        }
        const int pg = __shfl_sync(0xffffffffu, cur, j);
        const int ja = j + kPrefetch;
        const int far = ja < 32 ? __shfl_sync(0xffffffffu, cur, ja) : __shfl_sync(0xffffffffu, nxt, ja - 32);
        if (lane == 0) {
          const int y = pg < 0 ? oob : pg * 64;
          for (int c = 0; c < kKGroups && ok; ++c) {
            ok = it == 0 || mbar_wait_fast(&ctl->k_empty[c], (it - 1) & 1u, abort, p.status);
            if (!ok) break;
            if (rank == 0) mbar_arrive_expect_tx(&ctl->k_full[c], 2 * kKGroupBytes);
#pragma unroll
            for (int u = 0; u < 3; ++u)
              if (!(it == 0 && c == 0 && u == 0 && lost(p, 5)))
                tma_load_2d_pair(smem + Layout::k + (3 * c + u) * kBlockBytes, &tm_kv, k_full + c * 8, (3 * c + u) * 64, y);
          }
        }
        if (i == w.tile0)  // (after the first tile's loads, which are waited for)
          for (int d = 1; d < kPrefetch; ++d) warm(__shfl_sync(0xffffffffu, cur, d));
        warm(far);
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    }
    if (lane == 0 && rank == 0 && ok) {
      ok = seg == 0 || mbar_wait(&ctl->q_empty, (seg - 1) & 1u, abort, p.status);
      ctl->piece[seg & 1u] = 0;
      if (ok) mbar_arrive(&ctl->q_full);
    }
    __syncwarp();
  } else if (!KV8 && warp == 6) {
    // ---------------- V loads: this CTA's 256 value columns of both pages
    const uint32_t v_full = map_cluster(&ctl->v_full[0], 0);
    const int oob = p.num_pages * 64;
    uint32_t it = 0;
    bool ok = true;
    for (; have && ok; have = w.next(p, lane)) {
      const int* pt = p.page_table + (size_t)w.b * p.max_pages;
      const int pages = (max(w.seen_last, 0) + 63) >> 6;
      int ids = -1;
      for (int i = w.tile0; i < w.tile1 && ok; ++i, ++it) {
        const int j = (i - w.tile0) & 15;
        if (j == 0) {  // both pages of 16 tiles
          const int page = 2 * i + lane;
          ids = page < pages ? pt[page] : -1;
          if (ids >= p.num_pages) ids = -1;
        }
        const int pg0 = __shfl_sync(0xffffffffu, ids, 2 * j), pg1 = __shfl_sync(0xffffffffu, ids, 2 * j + 1);
        if (lane == 0) {
          // a tile that some row does not see to its end: the softmax warps clean it first
          const bool edge = (i + 1) * kTile > w.seen_first;
          for (int s = 0; s < kVPages && ok; ++s) {
            ok = it == 0 || mbar_wait_fast(&ctl->v_empty[s], (it - 1) & 1u, abort, p.status);
            if (!ok) break;
            const int pg = s == 0 ? pg0 : pg1, y = pg < 0 ? oob : pg * 64;
            uint8_t* dst = smem + Layout::v + s * kVPageBytes;
            if (edge) {
              // (page 0 is free: the previous tile's weights were complete, and with them its
              // phase of this barrier)
              if (s == 0) mbar_arrive_expect_tx(&ctl->edge, kVPages * kVPageBytes);
              if (rank == 0) mbar_arrive(&ctl->v_full[s]);
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (!(it == 0 && u == 0 && lost(p, 6)))
                  tma_load_2d(dst + u * kBlockBytes, &tm_kv, &ctl->edge, (int)rank * 256 + u * 64, y);
            } else {
              if (rank == 0) mbar_arrive_expect_tx(&ctl->v_full[s], 2 * kVPageBytes);
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (!(it == 0 && u == 0 && lost(p, 6)))
                  tma_load_2d_pair(dst + u * kBlockBytes, &tm_kv, v_full + s * 8, (int)rank * 256 + u * 64, y);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    }
  } else if (KV8 && warp >= 8) {
    // ---------------- FP8 cache: warps 8-11 convert this CTA's page into K (all 576 columns, three
    // parts a tile), warps 12-15 both pages' value columns of this CTA into V (two parts).  A warp has
    // 16 rows of a page; four lanes share a row, a lane takes every fourth 16-code chunk of it (two
    // passes of eight rows), so the 16-byte stores into the 128-byte-swizzled blocks meet no bank
    // conflict.  A part's registers are loaded for the next part as soon as they are stored.
    // One body for both kinds, and the rare cleaning in a pass of its own: the warps' instructions
    // share one cache (with a body each 32 sequences of 32k tokens took 400 us instead of 337; all
    // eight warps on each part, eight rows each, 421; row groups in a loop, whose register moves
    // wait for the loads, 430).
    const int r = (warp & 3) * 16 + (lane >> 2), q4 = lane & 3;
    // Warps 6 and 7 pass the news on: they order the part toward the tensor core's (async) proxy
    // and tell the issuing CTA.  That fence waits for the thread's outstanding loads too, which would
    // cost these warps an L2 latency a part.
    const bool is_v = warp >= 12;
    const int parts = is_v ? kVPages : kKGroups, part_bytes = is_v ? kVPageBytes : kKGroupBytes;
    uint64_t* const written = &ctl->written[is_v ? kKGroups : 0];
    uint64_t* const empty = is_v ? ctl->v_empty : ctl->k_empty;
    uint8_t* const slot = smem + (is_v ? Layout::v : Layout::k) + r * 128;
    const int first_v = is_v ? (int)rank * 16 : 0;
    const uint32_t piece0 = (uint32_t)(((q4 * 2) ^ (r & 7)) << 4), piece1 = (uint32_t)(((q4 * 2 + 1) ^ (r & 7)) << 4);
    uint32_t it = 0;
    for (; have; have = w.next(p, lane)) {
      const int* pt = p.page_table + (size_t)w.b * p.max_pages;
      const int pages = min((max(w.seen_last, 0) + 63) >> 6, 2 * w.tile1);
      // page ids, 32 at a time (a load whose value is wanted at once would stall a tile); -1: none
      // (never read: page 0 stands in for it)
      int ids = -1, base = -0x7fffffff;
      auto id = [&](int page) {
        if (page >= base + 32) {
          base = page & ~31;
          ids = base + lane < pages ? pt[base + lane] : -1;
          if (ids >= p.num_pages) ids = -1;
        }
        return __shfl_sync(0xffffffffu, ids, page & 31);
      };
      auto row = [&](int pg) { return p.kv + ((size_t)max(pg, 0) * 64 + r) * kKv8Row; };
      RowPart a, b;
      int pg = id(2 * w.tile0 + (is_v ? 0 : (int)rank)), far = -1;
      a.fetch(row(pg), first_v, q4, is_v);
      b.fetch(row(pg) + 8 * kKv8Row, first_v, q4, is_v);
      for (int i = w.tile0; i < w.tile1; ++i, ++it) {
        if (warp == 8) {  // a later tile's page into L2, its id loaded a tile ahead
          if (far >= 0 && far < p.num_pages && lane == 0)
            prefetch_l2_bulk(p.kv + (size_t)far * 64 * kKv8Row, 64 * kKv8Row);
          const int page = 2 * (i + kPrefetch + 1) + (int)rank;
          far = page < pages ? pt[page] : -1;
        }
#pragma unroll 1
        for (int part = 0; part < parts; ++part) {
          const bool turn = is_v || part == kKGroups - 1;   // the next part is of another page
          const int next = !turn ? pg : id(is_v ? 2 * i + part + 1 : 2 * i + 2 + (int)rank);
          const int first = is_v ? first_v : turn ? 0 : part * 12 + 12, split = !is_v && part == 1 ? 1 : 2;
          if (it > 0) warp_wait(empty + part, (it - 1) & 1u, abort, p.status);
          uint8_t* line = slot + part * part_bytes;
          a.store(line, piece0, piece1, split, is_v);
          a.fetch(row(next), first, q4, is_v);
          b.store(line + 8 * 128, piece0, piece1, split, is_v);
          b.fetch(row(next) + 8 * kKv8Row, first, q4, is_v);
          // value rows that no token sees, or that are not there, become zeros; of those that only some
          // see, what is not finite does (see the softmax warps)
          if (is_v && ((i + 1) * kTile > w.seen_first || pg < 0)) {
#pragma unroll 1
            for (int n = 0; n < 16; ++n) {   // row group, block, piece of what this lane has stored
              const int pos = i * kTile + part * 64 + r + (n >> 3) * 8;
              uint4* at = reinterpret_cast<uint4*>(line + (n >> 3) * 8 * 128 + ((n >> 1) & 3) * kBlockBytes +
                                                   (n & 1 ? piece1 : piece0));
              if (pg < 0 || pos >= w.seen_last) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else if (pos >= w.seen_first) {
                const uint4 v = *at;
                *at = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w));
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(written + part);
          pg = next;
        }
        if (__any_sync(0xffffffffu, *abort)) break;
      }
      if (__any_sync(0xffffffffu, *abort)) break;
    }
  } else if (KV8 && (warp == 6 || warp == 7)) {
    const int parts = warp == 6 ? kKGroups : kVPages;
    uint64_t* written = &ctl->written[warp == 6 ? 0 : kKGroups];
    const uint32_t full = warp == 6 ? map_cluster(&ctl->k_full[0], 0) : map_cluster(&ctl->v_full[0], 0);
    uint32_t it = 0;
    for (; have; have = w.next(p, lane)) {
      for (int i = w.tile0; i < w.tile1; ++i, ++it)
        for (int part = 0; part < parts; ++part) {
          warp_wait(&written[part], it & 1u, abort, p.status);
          fence_proxy_async_smem();
          if (lane == 0) mbar_arrive_pair(full + part * 8);
        }
      if (__any_sync(0xffffffffu, *abort)) break;
    }
  } else if (warp == 4 && rank == 0) {
    // ---------------- MMA issue, for both CTAs
    constexpr uint32_t idesc_qk = idesc_bf16(128, kTile);
    constexpr uint32_t idesc_pv = idesc_bf16(128, 256, /*b_mn_major=*/true);
    const uint32_t q_at = smem_u32(smem + Layout::q), k_at = smem_u32(smem + Layout::k),
                   v_at = smem_u32(smem + Layout::v), p_at = smem_u32(smem + Layout::p);
    // The whole warp walks the tiles and one lane issues, in the order Q.K^T of tile i + 1, P.V of tile
    // i: the softmax of a tile runs under the next tile's Q.K^T.  Fully unrolled, with operand offsets
    // that are constants: an issue loop with integer work around each instruction ran at a third of
    // the tensor pipe's rate.  The K loads say how many tiles each piece has (0: the end) when they
    // arm its Q barrier.
    {
      const uint32_t me = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        mbar_wait_issue<true>(bar, parity, abort, p.status);
        __syncwarp();
      };
      auto qk = [&](uint32_t n) {
        if (n >= 2) wait(&ctl->s_free[n & 1u], ((n >> 1) - 1) & 1u);
        const uint32_t d = tmem + kColS + (n & 1u) * 64u;
        const uint64_t qd = sdesc_sw128(fresh(q_at), 16, 1024), kd = sdesc_sw128(fresh(k_at), 16, 1024);
#pragma unroll
        for (int c = 0; c < kKGroups; ++c) {
          wait(&ctl->k_full[c], n & 1u);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 12; ++kk) {
            const int at = c * kKGroupBytes + (kk >> 2) * kBlockBytes + (kk & 3) * 32;
            mma2_f16_ss(d, desc_at(qd, at), desc_at(kd, at), idesc_qk, (c > 0 || kk > 0) ? 1u : 0u, me);
          }
          mma2_commit_both(&ctl->k_empty[c], me);
        }
        mma2_commit_both(&ctl->s_full[n & 1u], me);
      };
      auto pv = [&](uint32_t n, bool first) {
        wait(&ctl->p_full, n & 1u);
        const uint64_t pd = sdesc_sw128(fresh(p_at), 16, 1024), vd = sdesc_sw128(fresh(v_at), kBlockBytes, 1024);
#pragma unroll
        for (int v = 0; v < kVPages; ++v) {
          wait(&ctl->v_full[v], n & 1u);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma2_f16_ss(tmem + kColO + (uint32_t)(h * 128), desc_at(pd, v * kBlockBytes + kk * 32),
                          desc_at(vd, v * kVPageBytes + h * kVHalfBytes + kk * 2048), idesc_pv,
                          (v > 0 || kk > 0) ? 1u : first ? 0u : 1u, me);
          mma2_commit_both(&ctl->v_empty[v], me);
        }
        mma2_commit_both(&ctl->pv_done, me);
      };
#ifdef DSA_TEST_HOOKS
      if (p.stall == 3 && blockIdx.x == 0) warp_wait(&ctl->never, 0, abort, p.status);
#endif
      // after a wait that gave up, the rest runs on whatever is there: nothing of it is kept
      uint32_t n = 0;       // tiles whose Q.K^T is issued; their P.V runs one behind
      bool behind_first = false;
      for (uint32_t seg = 0;; ++seg) {
        wait(&ctl->q_full, seg & 1u);
        const int tiles = __shfl_sync(0xffffffffu, ctl->piece[seg & 1u], 0);
        if (tiles == 0 || __any_sync(0xffffffffu, *abort)) break;
#pragma unroll 1
        for (int i = 0; i < tiles; ++i, ++n) {
          if (__any_sync(0xffffffffu, *abort)) break;
          qk(n);
          if (i + 1 == tiles) mma2_commit_both(&ctl->q_empty, me);
          if (n > 0) pv(n - 1, behind_first);
          // O is the previous piece's until its rows have been read
          if (i == 0 && seg > 0) wait(&ctl->o_free, (seg - 1) & 1u);
          behind_first = i == 0;
        }
      }
      if (n > 0) pv(n - 1, behind_first);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------- softmax: lane l of the CTA's 128 is row l & 63, page l >> 6 of a tile
    const int row = tid & 63, half = tid >> 6;
    const int mrow = (int)rank * 64 + row;           // row of the group
    const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t s_free = map_cluster(&ctl->s_free[0], 0), p_full = map_cluster(&ctl->p_full, 0),
                   o_free = map_cluster(&ctl->o_free, 0);
    uint8_t* p_row = smem + Layout::p + half * kBlockBytes + row * 128;
    uint32_t it = 0, edges = 0;
    int nseg = 0;
    bool ok = true;
    for (; have && ok; have = w.next(p, lane), ++nseg) {
      const bool active = mrow < w.rows;
      const bool busy = __any_sync(0xffffffffu, active);
      // (rows that are no one's count as seeing everything: no masking, and nothing of them is kept)
      const int seen = active ? w.seen_first + mrow / p.H : 0x7fffffff;
      // pages that do not exist are masked: look for them once
      {
        const int* pt = p.page_table + (size_t)w.b * p.max_pages;
        const int pages = min((max(w.seen_last, 0) + 63) >> 6, 2 * w.tile1);
        int bad = 0;
        for (int i = 2 * w.tile0 + tid; i < pages; i += 128) {
          const int pg = pt[i];
          bad |= pg < 0 || pg >= p.num_pages;
        }
        if (bad) {
          report(p.status, kStatusDeviceCheck);
          ctl->bad_pages = nseg + 1;
        }
      }
      named_barrier(1, 128);
      const bool check_pages = ctl->bad_pages == nseg + 1;
      float m_ref = -INFINITY, l = 0.f;
      for (int i = w.tile0; i < w.tile1; ++i, ++it) {
        const uint32_t buf = it & 1u;
        warp_wait(&ctl->s_full[buf], (it >> 1) & 1u, abort, p.status);
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld_x32(lane_addr + kColS + buf * 64u, sr);
        tmem_ld_x32(lane_addr + kColS + buf * 64u + 32u, sr + 32);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(s_free + buf * 8);
        const int pos0 = i * kTile + half * 64;
        const int keep = visible_columns(active, seen, pos0, check_pages, p.page_table + (size_t)w.b * p.max_pages,
                                         p.num_pages);  // of ours
        if (w.seen_last > w.seen_first && (i + 1) * kTile > w.seen_first) {
          // cache rows that only some of the group's tokens see lose what is not finite in their values
          // (below).  An infinite value makes a score that is not finite: NaN or +inf makes the row NaN as
          // it is; -inf has a weight of 0, and 0 times infinity is NaN where the tile is not cleaned.  So
          // a row that sees an infinite value here becomes NaN by its sum.
          float low = INFINITY;
#pragma unroll
          for (int c = 0; c < 64; c += 2) low = min3(low, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          if (__any_sync(0xffffffffu, low == -INFINITY) &&
              seen > first_odd_row<KV8>(p.kv, p.page_table + (size_t)w.b * p.max_pages, p.num_pages,
                                        max(w.seen_first, pos0), min(w.seen_last, pos0 + 64)))
            l = __uint_as_float(0x7fffffffu);
        }
        if (!__all_sync(0xffffffffu, keep == 64)) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= keep) sr[c] = 0xff800000u;
        }
        float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          m2[(c >> 1) & 1] = max3(m2[(c >> 1) & 1], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
        float mx = fmaxf(m2[0], m2[1]);
        mx *= p.scale_log2;
        // one vote a tile; a warp whose wait gave up brings all to the second one, where they leave
        if (!named_barrier_and(2, 128, !*abort && !(active && mx > m_ref + kRescaleLog2))) {
          // some row's maximum has outgrown its reference: every row takes its true maximum
          ctl->x[tid] = mx;
          ok = named_barrier_and(1, 128, !*abort);
          if (!ok) break;
          const float m_new = fmaxf(m_ref, fmaxf(mx, ctl->x[tid ^ 64]));
          const float alpha = m_new == m_ref ? 1.f : fast_exp2(m_ref - m_new);
          m_ref = m_new;
          l *= alpha;
          if (i > w.tile0) {
            warp_wait(&ctl->pv_done, (it - 1) & 1u, abort, p.status);
            tc_fence_after();
            if (busy) {
#pragma unroll 1
              for (int cc = 0; cc < 16; ++cc) {
                uint32_t o[16];
                tmem_ld_x16(lane_addr + kColO + (uint32_t)(cc * 16), o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st_x16(lane_addr + kColO + (uint32_t)(cc * 16), o);
              }
              tmem_st_wait();
            }
            tc_fence_before();
          }
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        if (busy) {
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float2 e = fma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), p.scale_log2, -m_use);
            e.x = fast_exp2(e.x);
            e.y = fast_exp2(e.y);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], e);
            sr[c >> 1] = pack_bf16(e.x, e.y);  // P.V takes bf16 weights: 2^-8 relative each, unbiased
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        // P is free once the previous tile's P.V has read it
        if (it > 0) warp_wait(&ctl->pv_done, (it - 1) & 1u, abort, p.status);
        if (busy) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(p_row + ((c ^ (row & 7)) << 4)) =
                make_uint4(sr[4 * c], sr[4 * c + 1], sr[4 * c + 2], sr[4 * c + 3]);
        }
        bool come = true;   // the tile's values (else its weights are not handed over, and its slots not released)
        if (!KV8 && (i + 1) * kTile > w.seen_first) {
          // value rows that some row of the group does not see: a weight of 0 times what they hold
          // must be 0.  Past every token's end they become 0; among the tokens' own rows only what
          // is not finite does (the rows that see it get their NaN from the scores, whose keys are
          // the same columns, or, see above, from their sums).
          come = mbar_wait_fast(&ctl->edge, edges & 1u, abort, p.status);
          __syncwarp();
          ++edges;
          const int r0 = max(0, w.seen_first - i * kTile);
          for (int c = r0 * 32 + tid; c < kTile * 32; c += 128) {
            const int r = c >> 5, ch = c & 31;  // tile row; 16-byte chunk of our 256 columns
            uint4* at = reinterpret_cast<uint4*>(smem + Layout::v + (r >> 6) * kVPageBytes + (ch >> 3) * kBlockBytes +
                                                 (r & 63) * 128 +
                                                 (((ch & 7) ^ (r & 7)) << 4));
            if (i * kTile + r >= w.seen_last) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              uint4 v = *at;
              uint32_t* e = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
              for (int k = 0; k < 4; ++k) e[k] = finite_bf16x2(e[k]);
              *at = v;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && come) mbar_arrive_pair(p_full);
      }
      // ---------------- the piece's rows: O is complete once its last P.V is
      if (!ok) break;
      warp_wait(&ctl->pv_done, (it - 1) & 1u, abort, p.status);
      ctl->x[tid] = l;
      ok = named_barrier_and(1, 128, !*abort);
      if (!ok) break;
      tc_fence_after();
      const float l_all = ctl->x[row] + ctl->x[row + 64];
      float inv = l_all == 0.f ? 0.f : 1.f / l_all;
      float lse2 = l_all == 0.f ? -INFINITY : m_ref + log2f(l_all);
      const bool whole = w.whole();
      // a row that sees something and has no weight: its scores are all -inf, or +inf by the scale
      if (active && l_all == 0.f && sees_any(p.page_table + (size_t)w.b * p.max_pages, p.num_pages,
                                                w.tile0, w.tile1, seen)) {
        lse2 = whole || m_ref > 0.f ? __uint_as_float(0x7fffffffu) : kNoScore;
        if (whole) inv = lse2;
      }
      const size_t slot = (size_t)pair * 2 + (w.first ? 0 : 1);
      if (busy) {
        const size_t grow = (size_t)w.t0 * p.H + mrow;
        __nv_bfloat16* o_out = p.out + grow * kDv + half * 256;
        float* o_ws = p.ws_o + (slot * p.ws_rows + mrow) * kDv + half * 256;
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          uint32_t o[32];
          tmem_ld_x32(lane_addr + kColO + (uint32_t)(cc * 32), o);
          tmem_ld_wait();
          if (active) {
            // 32 bytes a store: with 16-byte ones (half a sector each) a piece took 5 us to leave
            if (whole) {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                o[k] = pack_bf16(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
              st_global_v8(o_out + cc * 32, o);
              st_global_v8(o_out + cc * 32 + 16, o + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * inv);
#pragma unroll
              for (int k = 0; k < 4; ++k) st_global_v8(o_ws + cc * 32 + 8 * k, o + 8 * k);
            }
          }
        }
        if (active && half == 0) {
          if (!whole)
            p.ws_lse[slot * p.ws_rows + mrow] = lse2;
          else if (p.lse)
            p.lse[grow] = lse2 * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(o_free);
    }
  }
  // A range that starts inside a group, the first to do so, names the group's pieces for the join.
  if (rank == 0 && tid == 0) {
    int4 j = make_int4(0, 0, 0, 0);
    if (any) {
      const Seq s = sequence(p, ctl->start_b, false);
      const long long u = unit_count(s), pos = share * pair;
      const int g = (int)((pos - ctl->start_at) / u);
      const long long at = ctl->start_at + g * u;
      const int i0 = g * p.T, n = min(p.T, s.n - i0);
      const int seen_last = s.len - s.n + i0 + n;
      const long long tiles = max(1, (seen_last + kTile - 1) / kTile);
      if (pos > at && pos < at + tiles && pos - share <= at) {
        const long long p0 = at / share, p1 = (at + tiles - 1) / share;
        j = make_int4(s.s0 + i0, n * p.H, (int)(p0 * 2 + (p0 * share == at ? 0 : 1)), (int)(p1 - p0 + 1));
      }
    }
    p.ws_join[pair] = j;
  }
  if (ctl->abort) {  // copies may still be in flight: give them time to land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000u) {
    }
  }
  griddep_launch_dependents();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 4) tmem_dealloc2(tmem, kTmemCols);
}

// Joins the pieces of the groups that a range border cuts.  A warp does a row of a group of up to four
// pieces, or 128 columns of one of up to 16; a block does 128 columns of one of more, its warp g adding
// up pieces g, g + 8, ....  The sums are added in a fixed order.  The blocks share all groups' work: a
// block for every row that there might be (9,728) took 5 us to launch, and one for every row there is
// 12 us for a group of 74 pieces.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinRow = 4, kJoinFew = 16;
constexpr int kJoinChunks = kDv / 128, kJoinBlocksPerSm = 4, kMostPairs = 256;
// (offsets into the workspace fit 32 bits: 2 * kMostPairs pieces of at most 128 rows)

DSA_DEV void add_to(float4& o, float e, const float4& x) {
  o.x = fmaf(e, x.x, o.x);
  o.y = fmaf(e, x.y, o.y);
  o.z = fmaf(e, x.z, o.z);
  o.w = fmaf(e, x.w, o.w);
}

// Weights of the pieces whose log-sum-exps (log2) start in slot z, relative to the largest: into wgt,
// by a whole warp; returns the reference (NaN if a piece is, 0 if nothing was seen, kNoScore if no
// score is above -inf) and their sum.
// (Out of line: inlined twice it cost the join half of its registers.)
__device__ __noinline__ float2 join_weights(const float* lse, int z, int parts, int rows, float* wgt, int lane) {
  float top = -INFINITY;
  bool nan = false;
#pragma unroll 1
  for (int k = lane; k < parts; k += 32) {
    const float v = lse[(k == 0 ? z : ((z >> 1) + k) * 2) * rows];
    wgt[k] = v;
    nan |= v != v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float m = __any_sync(0xffffffffu, nan) ? __uint_as_float(0x7fffffffu) : top == -INFINITY ? 0.f : top;
  float sum = 0.f;
#pragma unroll 1
  for (int k = lane; k < parts; k += 32) {
    const float e = exp2f(wgt[k] - m);
    wgt[k] = e;
    sum += e;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  __syncwarp();
  return make_float2(m, sum);
}

// The pieces of one row, C times four columns a lane (col4, col4 + 32, ...); wgt: the warp's weights.
template <int C>
struct Pieces {
  static constexpr int kAtOnce = 8 / C;
  const Params& p;
  int4 j;
  int r, col4, lane;
  float* wgt;
  float m, sum;      // reference of the weights (see join_weights), their sum
  float4 o[C];

  // piece 0 lies in slot j.z, the following ones each at the start of the next pair's range
  DSA_DEV const float4* cols(int k) const {
    const int slot = k == 0 ? j.z : ((j.z >> 1) + k) * 2;
    return reinterpret_cast<const float4*>(p.ws_o) + ((slot * p.ws_rows + r) * (kDv / 4) + col4);
  }
  // o = weighted sum of pieces first, first + step, ...
  DSA_DEV void add_up(int first, int step) {
    // (on their way while the weights are worked out, without the registers that loads would take)
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (first + i * step < j.w)
#pragma unroll
        for (int c = 0; c < C; ++c) asm volatile("prefetch.global.L1 [%0];" ::"l"(cols(first + i * step) + c * 32));
    const float2 w = join_weights(p.ws_lse + r, j.z, j.w, p.ws_rows, wgt, lane);
    m = w.x;
    sum = w.y;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = first; k0 < j.w; k0 += step * kAtOnce) {
      float4 x[kAtOnce][C];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (k0 + i * step < j.w)
#pragma unroll
          for (int c = 0; c < C; ++c) x[i][c] = cols(k0 + i * step)[c * 32];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (k0 + i * step < j.w)
#pragma unroll
          for (int c = 0; c < C; ++c) add_to(o[c], wgt[k0 + i * step], x[i][c]);
    }
  }
  DSA_DEV void finish() const {
    const bool none = m == kNoScore;   // a softmax of -inf only: NaN
    const float inv = none ? __uint_as_float(0x7fffffffu) : sum == 0.f ? 0.f : 1.f / sum;
    const size_t grow = (size_t)j.x * p.H + r;
#pragma unroll
    for (int c = 0; c < C; ++c)
      reinterpret_cast<uint2*>(p.out + grow * kDv)[col4 + c * 32] =
          make_uint2(pack_bf16(o[c].x * inv, o[c].y * inv), pack_bf16(o[c].z * inv, o[c].w * inv));
    if (col4 == 0 && p.lse)
      p.lse[grow] = none ? inv : sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
  }
};

__global__ void __launch_bounds__(kJoinThreads, 2) mla_join_kernel(const __grid_constant__ Params p) {
  __shared__ float4 part[kJoinWarps][32];
  __shared__ float wgt[kJoinWarps][kMostPairs];
  __shared__ int4 groups[kMostPairs];
  __shared__ int ends[kMostPairs];      // items of the groups up to and with each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  if (warp == 0) {
    int before = 0;
#pragma unroll 1
    for (int b = 0; b < p.pairs; b += 32) {
      const int4 j = b + lane < p.pairs ? p.ws_join[b + lane] : make_int4(0, 0, 0, 0);
      int n = j.w == 0 ? 0 : j.w <= kJoinRow ? j.y : j.y * kJoinChunks;
      if (j.w <= kJoinFew) n = (n + kJoinWarps - 1) / kJoinWarps;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += x;
      }
      groups[b + lane] = j;
      ends[b + lane] = before + n;
      before += __shfl_sync(0xffffffffu, n, 31);
    }
  }
  __syncthreads();
  const int total = ends[p.pairs - 1];
#pragma unroll 1
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int lo = 0, hi = p.pairs - 1;
    while (lo < hi) {  // the first group that ends beyond the item
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > item) hi = mid; else lo = mid + 1;
    }
    const int4 j = groups[lo];
    const int i = item - (lo > 0 ? ends[lo - 1] : 0);
    if (j.w <= kJoinRow) {
      Pieces<kJoinChunks> w = {p, j, i * kJoinWarps + warp, lane, lane, wgt[warp]};
      if (w.r < j.y) {
        w.add_up(0, 1);
        w.finish();
      }
    } else {
      const bool few = j.w <= kJoinFew;
      const int u = few ? i * kJoinWarps + warp : i;
      Pieces<1> w = {p, j, u / kJoinChunks, u % kJoinChunks * 32 + lane, lane, wgt[warp]};
      if (w.r < j.y) w.add_up(few ? 0 : warp, few ? 1 : kJoinWarps);
      if (!few) {
        __syncthreads();   // the previous item's sums have been read
        part[warp][lane] = w.o[0];
        __syncthreads();
        if (warp == 0)
#pragma unroll
          for (int g = 1; g < kJoinWarps; ++g) add_to(w.o[0], 1.f, part[g][lane]);
      }
      if (w.r < j.y && (few || warp == 0)) w.finish();
    }
    __syncwarp();
  }
}

// Tokens of a group, and the rows of a piece in the workspace.
static int group_tokens(const dsa_mla_decode_args& a) {
  return std::max(1, std::min({128 / a.H, a.max_q_per_seq, a.n_q}));
}

static int pair_count() {
  DeviceInfo dev;
  std::string err;
  return std::min(kMostPairs, (device_info(dev, err) ? dev.sm_count : 152) / 2);
}

}  // namespace mlad

size_t mla_decode_workspace_bytes(const dsa_mla_decode_args& a) {
  using namespace mlad;
  const size_t pieces = (size_t)pair_count() * 2, rows = (size_t)group_tokens(a) * a.H;
  size_t bytes = pieces * rows * kDv * 4;
  bytes += (pieces * rows * 4 + 255) / 256 * 256;
  return bytes + ((size_t)pair_count() * sizeof(int4) + 255) / 256 * 256;
}

dsa_status launch_mla_decode(const dsa_mla_decode_args& a, cudaStream_t stream, std::string& err) {
  using namespace mlad;
  const bool kv8 = a.kv_dtype == DSA_FP8_E4M3;
  Params p;
  p.B = a.B;
  p.n_q = a.n_q;
  p.H = a.H;
  p.T = group_tokens(a);
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.pairs = pair_count();
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.kv = reinterpret_cast<const uint8_t*>(a.kv_pool);
  p.page_table = a.page_table;
  p.seq_lens = a.seq_lens;
  p.q_start = a.q_start;
  p.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  p.ws_rows = p.T * p.H;
#ifdef DSA_TEST_HOOKS
  p.stall = g_test_stall;
#endif
  const size_t pieces = (size_t)p.pairs * 2;
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.workspace);
  p.ws_o = reinterpret_cast<float*>(ws);
  ws += pieces * p.ws_rows * kDv * 4;
  p.ws_lse = reinterpret_cast<float*>(ws);
  ws += (pieces * p.ws_rows * 4 + 255) / 256 * 256;
  p.ws_join = reinterpret_cast<int4*>(ws);

  CUtensorMap tm_q, tm_kv;
  if (!encode_tmap_2d(&tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kDqk, (uint64_t)a.n_q * a.H, kDqk * 2, 64, 64,
                      CU_TENSOR_MAP_SWIZZLE_128B, err) ||
      // (an FP8 cache is read with plain loads: its map is never used, any valid one will do)
      !encode_tmap_2d(&tm_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv_pool, kDqk, (uint64_t)(kv8 ? 1 : a.num_pages * 64), kDqk * 2,
                      64, 64, CU_TENSOR_MAP_SWIZZLE_128B, err))
    return DSA_ERR_CUDA;
  const int smem = Layout::total + 1024;
  auto kern = kv8 ? mla_decode_kernel<true> : mla_decode_kernel<false>;
  DeviceInfo dev;
  if (!device_info(dev, err)) return DSA_ERR_CUDA;
  static std::atomic<uint64_t> done[2];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, dev.device, done[kv8]);
  if (e != cudaSuccess) return cuda_fail(e, "mla_decode: set shared memory size", err);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * p.pairs));
  cfg.blockDim = dim3(kv8 ? kThreads<true> : kThreads<false>);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm_q, tm_kv, p);
  if (e != cudaSuccess) return cuda_fail(e, "mla_decode: launch", err);
  // at most one group a token, and one a border
  const long long items = (long long)std::min(p.pairs, a.n_q) * p.ws_rows * kJoinChunks;
  cfg.gridDim = dim3((unsigned)std::min<long long>(items, (long long)p.pairs * 2 * kJoinBlocksPerSm));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, mla_join_kernel, p);
  if (e != cudaSuccess) return cuda_fail(e, "mla_decode: launch of the join", err);
  return DSA_OK;
}

}  // namespace dsa

#ifdef DSA_TEST_HOOKS
extern "C" int dsa_test_mla_visible_columns(int owned, int seen, int pos0, int check_pages, const int32_t* pages,
                                            int num_pages) {
  return dsa::mlad::visible_columns(owned != 0, seen, pos0, check_pages != 0, pages, num_pages);
}
#endif
