// matmul_fp8.cu -- product of e4m3 rows with one fp32 scale per 128 columns and e4m3 weights with one per block of
// 128 x 128:
//   out[m][n] = sum_i f_i(m, n) P_i(m, n),   f_i = a_scale[m][i] b_scale[n / 128][i],
//   P_i = the product over the 128 columns of block i, four tcgen05 MMAs of 32 columns
//
// No e4m3 MMA applies an fp32 scale, so every P_i passes through registers: the MMAs write it to one of two buffers in
// tensor memory, and eight warps add f_i P_i to fp32 sums that they hold in registers, a row of the tile a thread (f_i
// is then one number, or two, a thread), while the MMAs fill the other buffer.
//
// Wide tiles (prompts): 256 rows x 256 columns by a CTA pair (cta_group::2; each CTA has 128 rows of a, 128 of b
// and 128 x 256 sums), a ring of four 32-KB stages, one persistent pair per two SMs.  A block's MMAs, 512 cycles at
// the nominal rate, are issued and handed over in halves of 128 columns (one scale of b each), which leaves the sums
// 768 cycles until a buffer is wanted back; a warp's products come from tensor memory a step of 32 columns ahead of its
// multiply-adds, across blocks.  Two warps multiply the scales, eight blocks at a time.  Rows go out by TMA.
// Bound: loads and MMAs alone run 4,096 x 7,168 x 16,384 in 250 us (3,850 TFLOP/s, at the power limit: 1,440 MHz
// after a second of it); the multiply-adds, 256 of a block's cycles on the fp32 pipe, their hand-over and their power
// make it 317 us (3,040 TFLOP/s; 355 to 367 us, at some 1,650 MHz, after a second).  With 512 columns in all a tile's end
// (rounding, boxes, TMA) is a third of the time: 8,192 x 32,768 in 166 to 176 us, 111 without it.
// Measured on the way: waits by suspension or by spinning alike; the scales loaded by the sums themselves, a row a lane,
// 430 (each load takes 32 lines of L1); tiles of 256 x 192 390; sums that spill a few registers 370 to 510.
//
// Narrow tiles (few rows): 128 rows x 32 to 128 columns a CTA.  A cluster of up to eight CTAs shares a tile's blocks, and
// its parts are added in rank order through distributed shared memory: many CTAs stream the weights, the result does not
// depend on their timing, and there is no workspace.  Two CTAs an SM, so that one's start and end run under the
// other's stream.  Bound: HBM with long rows (32 x 7,168 x 16,384 in 25 us, 4.8 TB/s of weights), else launch, a
// tile's chain of blocks (0.25 to 0.38 us each) and the parts' exchange (1 x 2,112 x 7,168 in 9.6 us).
#include <algorithm>
#include <type_traits>

#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {
namespace mm {

constexpr int kRows = 128;        // of a CTA's tile
constexpr int kThreads = 320;     // of a narrow CTA: warps 0-7 add up, 8 MMA, 9 loads
constexpr int kWideThreads = 384; // of a wide one: 10 and 11 multiply the scales
constexpr int kScaleBlocks = 8;   // blocks whose scales are multiplied at a time
constexpr int kScalePitch = kRows + 4;   // floats from one block's to the next
constexpr int kBlock = 128;       // columns of a scale block: a row of a stage
constexpr int kMostStages = 32;
constexpr int kMostSplits = 8;    // CTAs of a portable cluster
constexpr int kRing = 96 * 1024;  // of a narrow CTA that shares its SM, and half of one's that has it alone
constexpr int kGroupRows = 8;     // wide tiles of a column of tiles that run one after the other

struct Params {
  int M, N, blocks;
  int elem;
  int vec, even;           // rows of out start 16-byte aligned; on an even element
  int tiles_m, tiles_n;
  int a_box, stages, ring; // narrow: rows of a that are loaded, stages and bytes of the ring
  long long a_scale_stride, b_scale_stride, out_stride;
  const float* a_scale;
  const float* b_scale;
  uint8_t* out;
  int* status;
#ifdef DSA_TEST_HOOKS
  int stall;               // test build: the first CTA's MMA warp waits on a barrier nothing arrives on (10), or its
                           // first load of a (11) is left out
#endif
};

struct Ctl {
  uint64_t full[kMostStages], empty[kMostStages];
  uint64_t sum_full[2][2], sum_free[2][2];   // by buffer and half of the columns (narrow: the first half's)
  uint64_t scale_full[2], scale_free[2];
#ifdef DSA_TEST_HOOKS
  uint64_t never;          // test build: no thread ever arrives here
#endif
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

template <int E>
DSA_DEV uint32_t pack16(float a, float b) {
  if (E == DSA_ELEM_BF16) return pack_bf16(a, b);
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// `cols` outputs (at most 128) from column n on of rows m, m + step, ..., `some` of them and R at a time, value(r, c) the
// c-th of the r-th and the one after it, by a whole warp: for rows of out that do not start 16-byte aligned.  A lane
// stores a column, or two where rows start on an even element (and n is even).  Bound by instructions: 4 bytes a lane out of
// rows that start anywhere, with the lines' ends apart, took 340 us for 4,096 x 20,001 bf16 of 512 columns against 128
// (aligned rows of 20,000 columns 57, on even elements 110).
template <int R, class Value>
DSA_DEV void store_rows(const Params& p, int m, int step, int some, int n, int cols, Value&& value) {
  const int lane = threadIdx.x & 31;
  const long long apart = (long long)step * p.out_stride;
  auto singles = [&](auto* out, auto&& rounded) {
    auto* o = out + ((long long)m * p.out_stride + n + lane);
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      if (c + lane >= cols) break;
      float x[R];
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = r < some ? value(r, c + lane, false).x : 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < some) o[r * apart + c] = rounded(x[r]);
    }
  };
  auto pairs = [&](auto* out, auto&& rounded) {
    auto* o = out + (((long long)m * p.out_stride + n) / 2 + lane);
#pragma unroll
    for (int c = 0; c < 128; c += 64) {
      if (c + 2 * lane >= cols) break;
      float2 x[R];
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = r < some ? value(r, c + 2 * lane, true) : make_float2(0.f, 0.f);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < some) o[r * (apart / 2) + c / 2] = rounded(x[r]);
    }
  };
  if (p.even && (cols & 1) == 0) {
    if (p.elem == DSA_ELEM_FP32)
      pairs(reinterpret_cast<float2*>(p.out), [](float2 x) { return x; });
    else if (p.elem == DSA_ELEM_BF16)
      pairs(reinterpret_cast<uint32_t*>(p.out), [](float2 x) { return pack16<DSA_ELEM_BF16>(x.x, x.y); });
    else
      pairs(reinterpret_cast<uint32_t*>(p.out), [](float2 x) { return pack16<DSA_ELEM_FP16>(x.x, x.y); });
  } else if (p.elem == DSA_ELEM_FP32) {
    singles(reinterpret_cast<float*>(p.out), [](float x) { return x; });
  } else if (p.elem == DSA_ELEM_BF16) {
    singles(reinterpret_cast<__nv_bfloat16*>(p.out), [](float x) { return __float2bfloat16_rn(x); });
  } else {
    singles(reinterpret_cast<__half*>(p.out), [](float x) { return __float2half_rn(x); });
  }
}

// Eight rows of 128 sums in shared memory, 16-byte piece i of row r at i ^ r, to rows m .. of out, columns n on.
__device__ __noinline__ void store_eight(const Params& p, const uint8_t* rows, int m, int n) {
  store_rows<8>(p, m, 1, p.M - m, n, min(128, p.N - n), [&](int r, int c, bool two) {
    const float* x = reinterpret_cast<const float*>(rows + r * 512 + (((c >> 2) ^ r) << 4) + (c & 3) * 4);
    return two ? *reinterpret_cast<const float2*>(x) : make_float2(*x, 0.f);
  });
}

// The share of CTA `rank` of a narrow tile's rows, from `cols` columns of the parts [128][pitch] of `splits` CTAs.
__device__ __noinline__ void store_parts(const Params& p, const float* part, int pitch, int splits, int rank, int m0, int n0,
                                         int cols) {
  const int rows = min(kRows, p.M - m0), step = kThreads / 32 * splits;
  for (int row = (int)(threadIdx.x >> 5) * splits + rank; row < rows; row += 4 * step)
    store_rows<4>(p, m0 + row, step, (rows - row + step - 1) / step, n0, cols, [&](int r, int c, bool two) {
      const float* from = part + (row + r * step) * pitch + c;
      if (splits == 1) return make_float2(from[0], two ? from[1] : 0.f);
      uint2 u[kMostSplits];
#pragma unroll
      for (int s = 0; s < kMostSplits; ++s)
        if (s < splits) {
          const uint32_t at = map_cluster(from, (uint32_t)s);
          u[s] = two ? ld_cluster_v2(at) : make_uint2(ld_cluster_u32(at), 0u);
        }
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int s = 0; s < kMostSplits; ++s)
        if (s < splits) v = add2(v, make_float2(__uint_as_float(u[s].x), __uint_as_float(u[s].y)));
      return v;
    });
}

// N values to element `at` of out on, `left` columns from the end of its row.
template <int N>
DSA_DEV void store(const Params& p, long long at, int left, const float* v) {
  if (left <= 0) return;
  if (p.elem == DSA_ELEM_FP32) {
    float* o = reinterpret_cast<float*>(p.out) + at;
    if (p.vec && left >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) o[i] = v[i];
    }
    return;
  }
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    w[i] = p.elem == DSA_ELEM_BF16 ? pack16<DSA_ELEM_BF16>(v[2 * i], v[2 * i + 1]) : pack16<DSA_ELEM_FP16>(v[2 * i], v[2 * i + 1]);
  uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at;
  if (p.vec && left >= N) {
    if constexpr (N == 16) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(o + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) o[i] = (uint16_t)(w[i >> 1] >> ((i & 1) * 16));
  }
}

// A thread's sums of one row over kCols columns; a step of kStep columns at a time comes from tensor memory, two steps in
// flight.
template <int kCols, int kStep>
struct Sums {
  static constexpr int kSteps = kCols / kStep;
  static_assert(kCols % kStep == 0 && (kStep == 16 || kStep == 32), "whole steps");
  uint64_t v[kCols / 2];    // two columns each

  DSA_DEV void clear() {
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) v[i] = 0u;
  }
  static DSA_DEV void load(uint32_t tmem, uint32_t* r) {
    if constexpr (kStep == 32)
      tmem_ld_x32(tmem, r);
    else
      tmem_ld_x16(tmem, r);
  }
  DSA_DEV void multiply_add(int step, const uint32_t* r, uint64_t f) {
#pragma unroll
    for (int i = 0; i < kStep; i += 2) {
      uint64_t& x = v[(step * kStep + i) / 2];
      x = fma2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), f, x);
    }
  }
  // N columns from the c-th on.
  template <int N>
  DSA_DEV void values(int c, float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 two = unpack2(v[(c + i) / 2]);
      x[i] = two.x;
      x[i + 1] = two.y;
    }
  }
  // Adds the block's products at `tmem`, times the first of the factors for columns below `split`, a multiple of kStep,
  // and times the second for the others; factors() is asked while the first products are on their way, done() called
  // once all have been read.
  template <class Factors, class Done>
  DSA_DEV void add(uint32_t tmem, int split, Factors&& factors, Done&& done) {
    uint32_t r[2][kStep];
    load(tmem, r[0]);
    if (kSteps > 1) load(tmem + kStep, r[1]);
    const float2 f = factors();
    const uint64_t f0 = pack2(f.x, f.x), f1 = pack2(f.y, f.y);
#pragma unroll
    for (int c = 0; c < kSteps; c += 2) {
      tmem_ld_wait_for<kStep>(r[0]);
      if (c + 1 < kSteps) tmem_ld_wait_for<kStep>(r[1]);
      if (c + 2 >= kSteps) done();
      multiply_add(c, r[0], c * kStep < split ? f0 : f1);
      if (c + 2 < kSteps) load(tmem + (c + 2) * kStep, r[0]);
      if (c + 1 < kSteps) multiply_add(c + 1, r[1], (c + 1) * kStep < split ? f0 : f1);
      if (c + 3 < kSteps) load(tmem + (c + 3) * kStep, r[1]);
    }
  }
};

// The copies of a call that gave up may still be in flight: gives them time to land.
DSA_DEV void drain(const Ctl* ctl) {
  if (!*(volatile const int*)&ctl->abort) return;
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 2000000u) {
  }
}

// ---------------------------------------------------------------- narrow tiles

// CH: 32-column steps of a tile.
template <int CH>
__global__ void __launch_bounds__(kThreads, 2)
    narrow_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ Params p) {
  constexpr int BN = 32 * CH, HC = BN / 2, kBuf = CH == 1 ? 32 : CH == 2 ? 64 : 128, kPitch = BN + 4;
  static_assert(kRows * kPitch * 4 <= kRing, "parts of a tile");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + p.ring);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort = &ctl->abort;
  const int splits = (int)cluster_nrank(), rank = (int)cluster_rank();
  const int m0 = (int)blockIdx.y * kRows, n0 = (int)blockIdx.x / splits * BN;
  const int first = (int)((long long)p.blocks * rank / splits), n = (int)((long long)p.blocks * (rank + 1) / splits) - first;
  const int quarters = min(4, (p.M - m0 + 31) / 32);   // of the tile's rows, a warp each, that have any
  const bool direct = splits == 1 && p.vec;             // sums go out as they lie in registers
  const int a_bytes = p.a_box * kBlock, b_at = p.stages * a_bytes;   // (the MMAs read 128 rows of a: of later slots, and b)

  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->sum_full[i][0], 1);
      mbar_init(&ctl->sum_free[i][0], 2 * quarters);
    }
#ifdef DSA_TEST_HOOKS
    mbar_init(&ctl->never, 1);
#endif
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&ctl->tmem_base, 2 * kBuf);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  griddep_wait();  // nothing above reads global memory

  float* part = reinterpret_cast<float*>(smem);   // [128][kPitch], once the ring is done with
  if (warp == 9) {
    // ---------------- loads
    if (lane == 0) {
      int slot = 0;
      uint32_t turn = 0;
      for (int i = 0; i < n; ++i) {
        if (turn > 0 && !mbar_wait_fast(&ctl->empty[slot], (turn - 1) & 1u, abort, p.status)) break;
        mbar_arrive_expect_tx(&ctl->full[slot], a_bytes + BN * kBlock);
        bool load_a = true;
#ifdef DSA_TEST_HOOKS
        load_a = !(p.stall == 11 && blockIdx.x == 0 && i == 0);
#endif
        if (load_a) tma_load_2d(smem + slot * a_bytes, &tm_a, &ctl->full[slot], (first + i) * kBlock, m0);
        tma_load_2d(smem + b_at + slot * BN * kBlock, &tm_b, &ctl->full[slot], (first + i) * kBlock, n0);
        if (++slot == p.stages) {
          slot = 0;
          ++turn;
        }
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---------------- MMA issue: the whole warp walks, one lane issues
    constexpr uint32_t idesc = idesc_e4m3(kRows, BN);
    const uint64_t ad = sdesc_sw128(smem_u32(smem), 16, 1024), bd = sdesc_sw128(smem_u32(smem + b_at), 16, 1024);
    const uint32_t me = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      mbar_wait_issue<false>(bar, parity, abort, p.status);
      __syncwarp();
    };
#ifdef DSA_TEST_HOOKS
    if (p.stall == 10 && blockIdx.x == 0) warp_wait(&ctl->never, 0, abort, p.status);
#endif
    int slot = 0;
    uint32_t turn = 0;
    for (int i = 0; i < n; ++i) {
      wait(&ctl->full[slot], turn & 1u);
      if (i >= 2) wait(&ctl->sum_free[i & 1][0], ((i >> 1) - 1) & 1u);
      if (__any_sync(0xffffffffu, *abort)) break;
      tc_fence_after();
      const uint64_t a = desc_at(ad, slot * a_bytes), b = desc_at(bd, slot * BN * kBlock);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_f8_ss_by(tmem + (i & 1) * kBuf, desc_at(a, k * 32), desc_at(b, k * 32), idesc, k > 0 ? 1u : 0u, me);
      mma_commit_by(&ctl->empty[slot], me);
      mma_commit_by(&ctl->sum_full[i & 1][0], me);
      if (++slot == p.stages) {
        slot = 0;
        ++turn;
      }
    }
    __syncwarp();
  } else if ((warp & 3) < quarters) {
    // ---------------- sums
    const int local = (warp & 3) * 32 + lane, half = (warp >> 2) * HC;
    Sums<HC, 16> sums;
    sums.clear();
    // the scales of the row, and of the columns' one or two blocks
    const float* a_scale = p.a_scale + (long long)min(m0 + local, p.M - 1) * p.a_scale_stride + first;
    const int block0 = min(n0 + half, p.N - 1) >> 7, block1 = min(n0 + half + HC - 1, p.N - 1) >> 7;
    const float* b_scale0 = p.b_scale + block0 * p.b_scale_stride + first;
    const float* b_scale1 = p.b_scale + block1 * p.b_scale_stride + first;
    const int split = block0 == block1 ? HC : (block0 + 1) * kBlock - n0 - half;
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half;
    // a block ahead, and multiplied when they are used: what needs a load holds up the warp until it is there
    float a = a_scale[0], b0 = b_scale0[0], b1 = b_scale1[0];
    for (int i = 0; i < n; ++i) {
      const int next = min(i + 1, n - 1);
      const float next_a = a_scale[next], next_b0 = b_scale0[next], next_b1 = b_scale1[next];
      warp_wait(&ctl->sum_full[i & 1][0], (i >> 1) & 1u, abort, p.status);
      if (__any_sync(0xffffffffu, *abort)) break;
      auto done = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->sum_free[i & 1][0]);
      };
      tc_fence_after();
      sums.add(at + (i & 1) * kBuf, split, [&] { return make_float2(a * b0, a * b1); }, done);
      a = next_a;
      b0 = next_b0;
      b1 = next_b1;
    }
    if (direct) {
      if (m0 + local < p.M && !*abort) {
        const long long out = (long long)(m0 + local) * p.out_stride + n0 + half;
#pragma unroll
        for (int c = 0; c < HC; c += 16) {
          float x[16];
          sums.values(c, x);
          store<16>(p, out + c, p.N - n0 - half - c, x);
        }
      }
    } else if (!*abort) {
      // (every MMA of this CTA is done: the last block's sums have been read)
      float* to = part + local * kPitch + half;
#pragma unroll
      for (int c = 0; c < HC; c += 16) {
        float x[16];
        sums.values(c, x);
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(to + c + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
    }
  }
  drain(ctl);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // Tensor memory goes before any other CTA is waited for: a CTA that holds some never waits for one that may itself
  // wait for some, on an SM that it shares with another kernel's cluster.
  if (warp == 8) tmem_dealloc(tmem, 2 * kBuf);
  __syncwarp();
  if (!direct) {
    // ---------------- the parts of a tile: each CTA adds up those of its share, in rank order
    if (splits > 1) cluster_sync();
    const int rows = min(kRows, p.M - m0);
    if (p.vec) {   // a share of the columns, four at a time
      const int quads = BN / 4 / splits, items = rows * quads;
      for (int it = tid; it < items; it += kThreads) {
        const int row = it / quads, col = (rank * quads + it - row * quads) * 4;
        const float* from = part + row * kPitch + col;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        uint4 u[kMostSplits];   // (all on their way before the first is used)
#pragma unroll
        for (int s = 0; s < kMostSplits; ++s)
          if (s < splits) u[s] = ld_cluster_v4(map_cluster(from, (uint32_t)s));
#pragma unroll
        for (int s = 0; s < kMostSplits; ++s) {
          if (s >= splits) break;
          v.x += __uint_as_float(u[s].x);
          v.y += __uint_as_float(u[s].y);
          v.z += __uint_as_float(u[s].z);
          v.w += __uint_as_float(u[s].w);
        }
        store<4>(p, (long long)(m0 + row) * p.out_stride + n0 + col, p.N - n0 - col, &v.x);
      }
    } else {       // a share of the rows
      store_parts(p, part, kPitch, splits, rank, m0, n0, min(BN, p.N - n0));
    }
  }
  __syncwarp();
  if (splits > 1) cluster_sync();   // no CTA's parts go before all have read them
}

// ---------------------------------------------------------------- wide tiles

constexpr int kWideCols = 256;
struct Wide {
  static constexpr int kCols = kWideCols / 2;                // of a thread: a block of b
  static constexpr int kA = kRows * kBlock, kB = kCols * kBlock, kStage = kA + kB;
  static constexpr int kStages = 4;
  static constexpr int kBox = 32 * 64, kBoxes = 4;           // of a warp's outputs: 32 rows of 64 bytes
  static constexpr int kScales = kScaleBlocks * kScalePitch; // floats, of a half's columns
  static constexpr int out = kStages * kStage, scales = out + 8 * kBoxes * kBox, ctl = scales + 4 * kScales * 4,
                       total = ctl + 1024;
};
static_assert(Wide::total + 1024 <= 232448, "shared memory of a CTA");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ Params p) {
  using W = Wide;
  constexpr int kCols = W::kCols, kSteps = kCols / 32;
  static_assert(kCols == kBlock && kSteps % 2 == 0, "one block of b, and a block's first step is r0");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + W::ctl);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort = &ctl->abort;
  const int rank = (int)cluster_rank(), pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
  const int tiles = p.tiles_m * p.tiles_n;

  if (tid == 0) {
    for (int i = 0; i < W::kStages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ctl->sum_full[i >> 1][i & 1], 1);
      mbar_init(&ctl->sum_free[i >> 1][i & 1], 8);   // four warps of either CTA
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->scale_full[i], 2);
      mbar_init(&ctl->scale_free[i], 8);
    }
#ifdef DSA_TEST_HOOKS
    mbar_init(&ctl->never, 1);
#endif
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc2(&ctl->tmem_base, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers and tensor memory of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  griddep_wait();  // nothing above reads global memory

  // Tiles in groups of kGroupRows rows of tiles, column by column: what runs at one time shares rows of a and of b.
  auto place = [&](int t, int& m0, int& n0) {
    const int group = kGroupRows * p.tiles_n;
    const int g = t / group, in = t - g * group;
    const int rows = min(kGroupRows, p.tiles_m - g * kGroupRows);
    m0 = (g * kGroupRows + in % rows) * 2 * kRows;
    n0 = in / rows * kWideCols;
  };

  // (2 * 232 + 40: the 3 * 168 registers a lane that the three warpgroups were launched with)
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  if (warp == 9) {
    // ---------------- loads: this CTA's half of a's rows and of b's, counted on the even CTA's barrier
    if (lane == 0) {
      const uint32_t full = map_cluster(&ctl->full[0], 0);
      int slot = 0;
      uint32_t turn = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int m0, n0;
        place(t, m0, n0);
        for (int i = 0; i < p.blocks; ++i) {
          ok = turn == 0 || mbar_wait_fast(&ctl->empty[slot], (turn - 1) & 1u, abort, p.status);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&ctl->full[slot], 2 * W::kStage);
          uint8_t* to = smem + slot * W::kStage;
          bool load_a = true;
#ifdef DSA_TEST_HOOKS
          load_a = !(p.stall == 11 && blockIdx.x == 0 && t == pair && i == 0);
#endif
          if (load_a) tma_load_2d_pair(to, &tm_a, full + slot * 8, i * kBlock, m0 + rank * kRows);
          for (int h = 0; h < 2; ++h)
            tma_load_2d_pair(to + W::kA + h * (W::kB / 2), &tm_b, full + slot * 8, i * kBlock, n0 + h * kCols + rank * (kCols / 2));
          if (++slot == W::kStages) {
            slot = 0;
            ++turn;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 8 && rank == 0) {
    // ---------------- MMA issue, for both CTAs: the whole warp walks, one lane issues
    constexpr uint32_t idesc = idesc_e4m3(2 * kRows, kCols);
    const uint64_t ad = sdesc_sw128(smem_u32(smem), 16, 1024), bd = sdesc_sw128(smem_u32(smem + W::kA), 16, 1024);
    const uint32_t me = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) {   // false: it gave up
      const bool ok = mbar_test(bar, parity) || mbar_try_wait(bar, parity) || mbar_wait_issue<true>(bar, parity, abort, p.status);
      return (bool)__all_sync(0xffffffffu, ok);
    };
#ifdef DSA_TEST_HOOKS
    if (p.stall == 10 && blockIdx.x == 0) warp_wait(&ctl->never, 0, abort, p.status);
#endif
    int slot = 0;
    uint32_t turn = 0, it = 0;
    bool go = true;
    for (int t = pair; t < tiles && go; t += pairs) {
#pragma unroll 1
      for (int i = 0; i < p.blocks; ++i, ++it) {
        go = wait(&ctl->full[slot], turn & 1u);
        const uint64_t a = desc_at(ad, slot * W::kStage), b = desc_at(bd, slot * W::kStage);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (it >= 2) go = go && wait(&ctl->sum_free[it & 1u][h], ((it >> 1) - 1) & 1u);
          if (!go) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma2_f8_ss(tmem + (it & 1u) * 256u + h * kCols, desc_at(a, k * 32), desc_at(b, h * (W::kB / 2) + k * 32), idesc,
                       k > 0 ? 1u : 0u, me);
          if (h == 1) mma2_commit_both(&ctl->empty[slot], me);
          mma2_commit_both(&ctl->sum_full[it & 1u][h], me);
        }
        if (!go) break;
        if (++slot == W::kStages) {
          slot = 0;
          ++turn;
        }
      }
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------- scales: products a_scale b_scale of the tile's rows with a half of the columns, eight blocks at a
    // time, a lane a block and every fourth row.  (Loaded by the sums, a row a lane, they took 32 lines of L1 a load,
    // beside the MMAs' operands.)
    const int h = warp - 10, in = lane & (kScaleBlocks - 1), first = lane / kScaleBlocks;
    uint32_t set = 0;
    bool go = true;
    for (int t = pair; t < tiles && go; t += pairs) {
      int m0, n0;
      place(t, m0, n0);
      m0 += rank * kRows;
      const float* b = p.b_scale + (min(n0 + h * kCols, p.N - 1) >> 7) * p.b_scale_stride;
      for (int i = 0; i < p.blocks; i += kScaleBlocks, ++set) {
        const int block = min(i + in, p.blocks - 1);
        const float* a = p.a_scale + block;
        const float bs = b[block];
        go = set < 2 || mbar_wait_fast(&ctl->scale_free[set & 1u], ((set >> 1) - 1) & 1u, abort, p.status);
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        float* to = reinterpret_cast<float*>(smem + W::scales) + ((set & 1u) * 2 + h) * W::kScales + in * kScalePitch;
#pragma unroll 8
        for (int r = first; r < kRows; r += 32 / kScaleBlocks)
          to[r] = a[(long long)min(m0 + r, p.M - 1) * p.a_scale_stride] * bs;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->scale_full[set & 1u]);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---------------- sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int local = (warp & 3) * 32 + lane, h = warp >> 2, half = h * kCols;
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half;
    const uint32_t sum_free = map_cluster(&ctl->sum_free[0][h], 0);
    const float* scales = reinterpret_cast<const float*>(smem + W::scales) + h * W::kScales + local;
    uint32_t it = 0, set = 0;
    bool go = true;
    for (int t = pair; t < tiles && go; t += pairs) {
      Sums<kCols, 32> sums;
      sums.clear();
      // Two steps of 32 columns in turn: one is on its way while the other's products are added, a block's first while
      // the last one's are.
      uint32_t r0[32], r1[32];
      auto full = [&](uint32_t block) { return &ctl->sum_full[block & 1u][h]; };
      auto products = [&](uint32_t block) { return at + (block & 1u) * 256u; };
      // (waits stand inline: a call would cost registers)
      go = mbar_wait(full(it), (it >> 1) & 1u, abort, p.status);
      go = __all_sync(0xffffffffu, go);
      if (!go) break;
      tc_fence_after();
      tmem_ld_x32(products(it), r0);
#pragma unroll 2
      for (int i = 0;; ++i) {   // (votes only where a wait has to wait: one more a block took 15 of 328 us)
        const int in = i & (kScaleBlocks - 1);
        if (in == 0) {
          go = mbar_wait(&ctl->scale_full[set & 1u], (set >> 1) & 1u, abort, p.status);
          go = __all_sync(0xffffffffu, go);
          if (!go) {
            tmem_ld_wait();
            break;
          }
        }
        const float f = scales[(set & 1u) * (2 * W::kScales) + in * kScalePitch];
        const uint64_t ff = pack2(f, f);
#pragma unroll
        for (int c = 0; c < kSteps - 1; ++c) {
          uint32_t* r = c & 1 ? r1 : r0;
          tmem_ld_wait_for<32>(r);
          tmem_ld_x32(products(it) + (c + 1) * 32, c & 1 ? r0 : r1);
          sums.multiply_add(c, r, ff);
        }
        tmem_ld_wait_for<32>(r1);
        tc_fence_before();
        __syncwarp();   // (lane 0 arrives for all: after their reads of the products and of the scales)
        mbar_arrive_pair_by(sum_free + (it & 1u) * 16, lane == 0);
        if (in == kScaleBlocks - 1 || i + 1 == p.blocks) {
          if (lane == 0) mbar_arrive(&ctl->scale_free[set & 1u]);
          ++set;
        }
        ++it;
        if (i + 1 == p.blocks) {
          sums.multiply_add(kSteps - 1, r1, ff);
          break;
        }
        const bool ready = __all_sync(0xffffffffu, mbar_test(full(it), (it >> 1) & 1u));
        if (ready) {
          tc_fence_after();
          tmem_ld_x32(products(it), r0);
        }
        sums.multiply_add(kSteps - 1, r1, ff);
        if (!ready) {
          go = mbar_wait(full(it), (it >> 1) & 1u, abort, p.status);
          go = __all_sync(0xffffffffu, go);
          if (!go) break;
          tc_fence_after();
          tmem_ld_x32(products(it), r0);
        }
      }
      if (!go) break;
      // The warp's 32 rows go out in boxes of 32 columns, by way of shared memory (a row a lane, stores to memory took a
      // line of it each: 8,192 x 32,768 outputs of 512 columns 213 us).
      int m0, n0;
      place(t, m0, n0);
      m0 += rank * kRows + (warp & 3) * 32;
      n0 += half;
      if (m0 >= p.M) continue;
      uint8_t* boxes = smem + W::out + warp * (W::kBoxes * W::kBox);
      if (!p.vec) {
        if (n0 >= p.N) continue;
#pragma unroll 1
        for (int r = 0; r < 32; r += 8) {   // eight rows at a time
          if ((lane & ~7) == r) {
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
              float x[16];
              sums.values(c, x);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(boxes + (lane & 7) * 512 + ((((c >> 2) + i) ^ (lane & 7)) << 4)) =
                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
          }
          __syncwarp();
          store_eight(p, boxes, m0 + r, n0);
          __syncwarp();
        }
        continue;
      }
      // Four boxes of 64 bytes a row, `cols` columns each, go out together: piece(i, k) gives the k-th 16 bytes of the
      // i-th.  (A store reads its box some time after it is issued.)
      static_assert(W::kBoxes == 4, "boxes that go out together");
      auto put = [&](int col, int cols, auto&& piece) {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(boxes + i * W::kBox + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = piece(i, k);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + i * cols < p.N) tma_store_2d(&tm_out, boxes + i * W::kBox, col + i * cols, m0);
          bulk_commit();
        }
      };
      auto put16 = [&](auto type) {
        put(n0, 32, [&](int i, int k) {
          constexpr int E = decltype(type)::value;
          float x[8];
          sums.values(i * 32 + k * 8, x);
          return make_uint4(pack16<E>(x[0], x[1]), pack16<E>(x[2], x[3]), pack16<E>(x[4], x[5]), pack16<E>(x[6], x[7]));
        });
      };
      if (p.elem == DSA_ELEM_BF16) {
        put16(std::integral_constant<int, DSA_ELEM_BF16>());
      } else if (p.elem == DSA_ELEM_FP16) {
        put16(std::integral_constant<int, DSA_ELEM_FP16>());
      } else {
#pragma unroll
        for (int c = 0; c < kCols; c += 64)
          put(n0 + c, 16, [&](int i, int k) {
            float x[4];
            sums.values(c + i * 16 + k * 4, x);
            return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
          });
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  __syncwarp();
  drain(ctl);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 8) tmem_dealloc2(tmem, 512);
}

using NarrowKernel = void (*)(CUtensorMap, CUtensorMap, Params);

struct Plan {
  bool wide;
  int bn, splits;
};

// The plan with the least estimated time (us).  Measured, launch included:
//   wide     4, and a round of tiles 1 and 0.42 a block of 128 columns
//   narrow   4, or 5 with splits, a round of CTAs, two an SM (a cluster has to find its CTAs in one group of SMs, which
//            leaves 5% and 15% of them out with four and eight), and the longest of
//            - a CTA's blocks, 0.2 + 0.0014 a column each, a sixth more with two CTAs an SM,
//            - the weights at 6.0 TB/s,
//            - all that the CTAs load, 12.5 TB/s from L2;
//            then with splits a CTA's sums, 20 KB a us.
// For instance (rows x columns x K; best narrow against wide): 1 x 2,112 x 7,168 9 against 25, 32 x 7,168 x 16,384 25
// against 53, 200 x 8,192 x 1,536 9.7 against 11.4, 300 x 4,096 x 4,096 14.6 against 18.1, 777 x 24,576 x 1,536 48 against 40.
Plan plan(int M, int N, int blocks, int sms) {
  const double pairs = std::max(1, sms / 2);
  auto up = [](double a, double b) { return std::ceil(a / b); };
  Plan best = {true, kWideCols, 1};
  double least = 4.0 + up(up(M, 256) * up(N, kWideCols), pairs) * (1.0 + 0.42 * blocks);
  const double tiles_m = up(M, kRows), rows = std::min(M, kRows), K = blocks * 128.0;
  if (tiles_m > 65535) return best;
  for (int bn = 32; bn <= 128; bn += 32)
    for (int s = 1; s <= kMostSplits && s <= blocks; s *= 2) {
      const double ctas = tiles_m * up(N, bn) * s, rounds = up(ctas, 2.0 * sms * (s == 8 ? 0.85 : s == 4 ? 0.95 : 1.0));
      const double block = (0.2 + 0.0014 * bn) * (ctas > sms ? 1.15 : 1.0);
      const double t = rounds * (s > 1 ? 5.0 : 4.0) +
                       std::max({rounds * up(blocks, s) * block, N * K / 6.0e6, ctas / s * (bn + rows) * K / 12.5e6}) +
                       (s > 1 ? up(ctas, sms) * rows * bn * 4 / 20e3 : 0.0);
      if (t < least) {
        least = t;
        best = {false, bn, s};
      }
    }
  return best;
}

}  // namespace mm

#ifdef DSA_TEST_HOOKS
extern "C" int dsa_test_matmul_plan(int M, int N, int K, int sms) {
  const mm::Plan w = mm::plan(M, N, (K + mm::kBlock - 1) / mm::kBlock, sms);
  return w.wide ? 0 : w.bn * 16 + w.splits;
}
#endif

dsa_status launch_matmul_fp8(const dsa_matmul_fp8_args& a, cudaStream_t stream, std::string& err) {
  using namespace mm;
  DeviceInfo dev;
  if (!device_info(dev, err)) return DSA_ERR_CUDA;
  Params p;
  p.M = a.M;
  p.N = a.N;
  p.blocks = (a.K + kBlock - 1) / kBlock;
  p.elem = a.elem;
  const int size = a.elem == DSA_ELEM_FP32 ? 4 : 2;
  p.vec = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && (a.M == 1 || a.out_stride * size % 16 == 0);
  p.even = (reinterpret_cast<uintptr_t>(a.out) & (2 * size - 1)) == 0 && (a.M == 1 || a.out_stride % 2 == 0);
  p.a_scale_stride = a.a_scale_stride;
  p.b_scale_stride = a.b_scale_stride;
  p.out_stride = a.out_stride;
  p.a_scale = a.a_scale;
  p.b_scale = a.b_scale;
  p.out = reinterpret_cast<uint8_t*>(a.out);
  p.status = a.status;
#ifdef DSA_TEST_HOOKS
  p.stall = g_test_stall;
#endif
  const Plan w = plan(a.M, a.N, p.blocks, dev.sm_count);
  const int rows = w.wide ? 2 * kRows : kRows;
  p.tiles_m = (int)(((long long)a.M + rows - 1) / rows);
  p.tiles_n = (int)(((long long)a.N + w.bn - 1) / w.bn);
  p.a_box = w.wide ? kRows : std::min(kRows, (a.M + 7) / 8 * 8);
  // All of an SM's shared memory where every CTA has its SM alone, in clusters of up to two: 1,269 x 640 x 9,328 29.3 -> 25.2
  // us, 1,875 x 432 x 5,312 21.1 -> 19.1, 1,666 x 936 x 2,176 17.0 -> 15.0, others alike.  One CTA an SM leaves room for
  // few clusters of more: 1 x 4,632 x 15,056 (four) 27 -> 36 us, 688 x 72 x 13,232 (eight) 17 -> 23.
  p.ring = w.splits <= 2 && (long long)p.tiles_m * p.tiles_n * w.splits <= dev.sm_count ? 2 * kRing : kRing;
  p.stages = w.wide ? 0 : std::min(kMostStages, p.ring / ((p.a_box + w.bn) * kBlock));
  CUtensorMap tm_a, tm_b;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t K = (uint64_t)a.K;
  if (!encode_tmap_2d(&tm_a, u8, a.a, K, (uint64_t)a.M, a.M == 1 ? K : (uint64_t)a.a_stride, kBlock, (uint32_t)p.a_box, sw, err) ||
      !encode_tmap_2d(&tm_b, u8, a.b, K, (uint64_t)a.N, a.N == 1 ? K : (uint64_t)a.b_stride, kBlock,
                      (uint32_t)(w.wide ? w.bn / 4 : w.bn), sw, err))
    return DSA_ERR_CUDA;
  const NarrowKernel narrow = w.bn == 32   ? narrow_kernel<1>
                              : w.bn == 64 ? narrow_kernel<2>
                              : w.bn == 96 ? narrow_kernel<3>
                                           : narrow_kernel<4>;
  const void* k = w.wide ? reinterpret_cast<const void*>(wide_kernel) : reinterpret_cast<const void*>(narrow);
  const int smem = w.wide ? Wide::total + 1024 : p.ring + 1024 + 1024;
  static std::atomic<uint64_t> done[5];
  cudaError_t e = allow_smem(k, w.wide ? smem : 2 * kRing + 1024 + 1024, dev.device, done[w.wide ? 0 : w.bn / 32]);
  if (e != cudaSuccess) return cuda_fail(e, "matmul_fp8: set shared memory size", err);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  CUtensorMap tm_out;
  if (w.wide) {
    // (a TMA store writes 16 bytes where the row ends inside them)
    p.vec = p.vec && (long long)a.N * size % 16 == 0;
    if (p.vec && !encode_tmap_2d(&tm_out, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, a.out,
                                 (uint64_t)a.N, (uint64_t)a.M, a.M == 1 ? ((uint64_t)a.N * size + 15) / 16 * 16 : (uint64_t)a.out_stride * size, 64 / size, 32,
                                 CU_TENSOR_MAP_SWIZZLE_64B, err))
      return DSA_ERR_CUDA;
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    if (tiles > 0x70000000LL) {
      err = "matmul_fp8: too many outputs for one launch";
      return DSA_ERR_UNSUPPORTED;
    }
    cfg.gridDim = dim3((unsigned)std::min<long long>(tiles, std::max(1, dev.sm_count / 2)) * 2);
    cfg.numAttrs = 1;
  } else {
    cfg.gridDim = dim3((unsigned)p.tiles_n * w.splits, (unsigned)p.tiles_m);   // (at most 2^26 * 8)
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)w.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.blockDim = dim3(w.wide ? kWideThreads : kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  e = w.wide ? cudaLaunchKernelEx(&cfg, wide_kernel, tm_a, tm_b, tm_out, p) : cudaLaunchKernelEx(&cfg, narrow, tm_a, tm_b, p);
  if (e != cudaSuccess) return cuda_fail(e, "matmul_fp8: launch", err);
  return DSA_OK;
}

}  // namespace dsa
