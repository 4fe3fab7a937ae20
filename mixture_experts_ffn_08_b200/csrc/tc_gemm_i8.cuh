// Persistent, warp-specialised tcgen05 matrix product of 8-bit integers, dense or grouped by
// expert, with one scale per row of A (a token) and one per row of B (an output channel):
//
//   out[r, n] = a_scale[r] * w_scale[n] * sum_k A[r, k] * B[n, k]  (+ bias[n])
//   h[r, n]   = SiLU(g) * u, g and u two such products              (SWIGLU)
//
// The sums are exact: kind::i8 accumulates s8 products in s32, and the callers keep
// K * 128 * 128 below 2^31.  The scales leave the sum, so they cost one multiplication per
// output in the epilogue and the main loop is a plain int8 product at the e4m3 rate.
//
// CG = 1: a CTA computes 128 x BN tiles on its own.  CG = 2: a cluster of two CTAs computes a
// 256 x BN tile with one stream of cta_group::2 MMAs, each CTA holding 128 rows of A and half
// of the BN rows of B; the operand bytes that cross L2 -> SM per MAC are those of a 256 x 256
// tile while each SM's TMEM still holds two accumulators, so the epilogue of one tile runs
// under the main loop of the next.  (At K = 1536 a tile's MMAs last only 6000 cycles and its
// epilogue nearly as long.)  Narrower one-SM tiles spread few rows over more SMs.
// What bounds it on B200: the power cap for large products (8192 x 14336 x 4096 in 287-321 us, the
// tensor pipe busy 96 % of the cycles at 1.6 GHz), HBM for a decode batch's weights (6.2-6.6 TB/s).
// A group's first row is a multiple of 128, not of 256: the second half of a group's last pair
// tile may lie past the group, and then it is neither loaded nor stored.
//
// Rows: group g's real rows are the first count(g) of those that start at offsets[g] (or at
// g * masked_cap).  The schedule comes from the counts alone: work items are (group, N-tile,
// M-tile) with the counts and a prefix sum over the groups in shared memory, all of the same cost, and
// walked in steps of the grid.
//
// Warp roles (192 threads): warp 0 issues TMA loads into the stage ring, warp 1 allocates TMEM
// and issues MMAs, warps 2-5 run the epilogue.  Every wait is bounded; on a timeout the CTA
// sets MOE_DEV_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#pragma once

#include <type_traits>

#include "i8_choice.h"
#include "tc_gemm_2cta.cuh"

namespace moe {

constexpr int kI8MaxGroups = 1024;
constexpr int kI8OutBox = 32 * 128;  // bytes of an output box: 32 rows x 128 bytes

struct I8Params {
  const int32_t* offsets;  // [G+1] first row of each group (contiguous layout, grouped)
  const int32_t* counts;   // [G] real rows; nullptr: offsets[g+1] - offsets[g], or dense_rows
  int G;
  int dense_rows;          // > 0: one group of that many rows, offsets and counts unused
  int masked_cap;          // > 0: group g's rows start at g * masked_cap
  int K;                   // reduction length, a multiple of 16
  int N;                   // output columns of a group
  const float* a_scale;    // [rows of A]
  const float* w_scale;    // [G * N]
  const float* w_scale_up; // [G * N] (SWIGLU)
  const float* bias;       // [N] or nullptr
  void* out;               // SWIGLU: fp32 [rows, ldo]; else out_type
  int out_type;            // moe_out_type_t
  int tma_store;           // the output's tensor map is usable (16-byte aligned rows)
  int prefetch;            // dot products: ask for the first weights before waiting for the kernel before
  int64_t ldo;
  int32_t* status;
};

// D format s32, A and B signed 8-bit, both K-major.
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <int CG>
MOE_DEVINL void umma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int CG_, int BN_, bool SWIGLU_, int STAGES_, int SUB_ = 1>
struct I8Cfg {
  static constexpr int CG = CG_;
  static constexpr int BN = BN_;
  static constexpr bool SWIGLU = SWIGLU_;
  static constexpr int STAGES = STAGES_;
  static constexpr int SUB = SUB_;               // K-blocks per stage
  static constexpr int BK = 128;                 // codes per K-block: one 128-byte swizzle row
  static constexpr int A_BYTES = 128 * BK;
  static constexpr int B_ROWS = BN / CG;         // B rows held by each CTA
  static constexpr int B_BYTES = B_ROWS * BK;
  static constexpr int BLOCK_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGE_BYTES = SUB * BLOCK_BYTES;
  static constexpr int OUT_BYTES = 4 * kI8OutBox;  // one box per epilogue warp
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + 1024;
  static constexpr int OUT_COLS = SWIGLU ? BN / 2 : BN;
  static constexpr int TMEM_COLS = 2 * BN;       // two accumulators
  static constexpr int TILE_M = 128 * CG;
  static constexpr int THREADS = 192;
  static_assert(BN == 64 || BN == 128 || BN == 256, "two accumulators in a power of two of TMEM columns");
  static_assert(CG == 1 || BN == 256, "pair tiles are 256 x 256");
  static_assert(SMEM_BYTES + 8 * (kI8MaxGroups + 1) + 4 * 512 * 4 + 512 <= 227 * 1024, "shared memory");
};

struct I8Tile {
  int group;
  int n_tile;
  int m0;            // first row of the tile inside its group
  int count;         // real rows of the group
  long long row0;    // first row of the tile in A and out
};

// Real rows of group g: its count, but never more than its rows in the layout.
MOE_DEVINL int real_rows(const int32_t* offsets, const int32_t* counts, int cap, int g) {
  const int room = cap > 0 ? cap : __ldg(offsets + g + 1) - __ldg(offsets + g);
  const int n = counts != nullptr ? __ldg(counts + g) : room;
  return n < 0 ? 0 : (n < room ? n : room);
}
MOE_DEVINL int i8_count(const I8Params& p, int g) {
  return p.dense_rows > 0 ? p.dense_rows : real_rows(p.offsets, p.counts, p.masked_cap, g);
}

// Work item -> tile; pref[g] = NT * sum over e < g of M-tiles(e).  Inside a group the operand
// with fewer rows is the one that the CTAs running side by side read again from L2.
template <class Cfg>
MOE_DEVINL I8Tile i8_decode(int item, int NT, const I8Params& p, const int* pref, const int* cnt) {
  int lo = 0, hi = p.G - 1;  // group with pref[g] <= item < pref[g+1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pref[mid] <= item) lo = mid; else hi = mid - 1;
  }
  I8Tile t;
  t.group = lo;
  t.count = cnt[lo];
  const int tiles = (t.count + Cfg::TILE_M - 1) / Cfg::TILE_M;
  const int local = item - pref[lo];
  const bool m_outer = static_cast<long long>(tiles) * Cfg::TILE_M > static_cast<long long>(NT) * Cfg::BN;
  t.m0 = (m_outer ? local / NT : local % tiles) * Cfg::TILE_M;
  t.n_tile = m_outer ? local % NT : local / tiles;
  const long long first = p.dense_rows > 0 ? 0
                          : p.masked_cap > 0 ? static_cast<long long>(lo) * p.masked_cap : __ldg(p.offsets + lo);
  t.row0 = first + t.m0;
  return t;
}

// Rows of A that a CTA loads for `rows` real rows from its half of the tile on.
MOE_DEVINL int i8_box_rows(int rows) { return rows <= 0 ? 0 : (rows <= kI8SmallRows ? kI8SmallRows : 128); }

// 32 outputs in bf16 or fp16.
MOE_DEVINL void i8_pack32(int out_type, const float (&v)[32], uint32_t (&w)[16]) {
  if (out_type == MOE_OUT_BF16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half2 hv = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&hv);
    }
  }
}

// 32 sums of a row times its scale and the columns' (cols[0..31]), plus their biases where there
// are any: packed pairs, the columns read as vectors (the same ones in every lane).
MOE_DEVINL void i8_scale32(const uint32_t (&r)[32], float sa, const float* cols, const float* bias, float (&v)[32]) {
  const float2 s2 = make_float2(sa, sa);
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(cols + i);
    const float2 a = mul2(make_float2(__int2float_rn(static_cast<int>(r[i])), __int2float_rn(static_cast<int>(r[i + 1]))), s2);
    const float2 b = mul2(make_float2(__int2float_rn(static_cast<int>(r[i + 2])), __int2float_rn(static_cast<int>(r[i + 3]))), s2);
    float2 x, y;
    if (bias != nullptr) {
      const float4 t = *reinterpret_cast<const float4*>(bias + i);
      x = fma2(a, make_float2(c.x, c.y), make_float2(t.x, t.y));
      y = fma2(b, make_float2(c.z, c.w), make_float2(t.z, t.w));
    } else {
      x = mul2(a, make_float2(c.x, c.y));
      y = mul2(b, make_float2(c.z, c.w));
    }
    v[i] = x.x;
    v[i + 1] = x.y;
    v[i + 2] = y.x;
    v[i + 3] = y.y;
  }
}

// 32 fp32 outputs of one row, columns col .. col + 31 of which the first n are stored.
MOE_DEVINL void i8_store32(const I8Params& p, long long row, int col, const float (&v)[32], int n) {
  const long long at = row * p.ldo + col;
  if (p.out_type == MOE_OUT_FP32) {
    float* o = static_cast<float*>(p.out) + at;
    if (n >= 32 && (reinterpret_cast<uintptr_t>(o) & 31) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) st_global_v8(o + 8 * i, reinterpret_cast<const uint32_t*>(v) + 8 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < n) o[i] = v[i];
    }
    return;
  }
  uint32_t w[16];
  i8_pack32(p.out_type, v, w);
  uint16_t* o = static_cast<uint16_t*>(p.out) + at;
  if (n >= 32 && (reinterpret_cast<uintptr_t>(o) & 31) == 0) {
    st_global_v8(o, w);
    st_global_v8(o + 16, w + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) o[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

MOE_DEVINL void i8_store1(const I8Params& p, long long row, int col, float v) {
  const long long at = row * p.ldo + col;
  if (p.out_type == MOE_OUT_FP32) static_cast<float*>(p.out)[at] = v;
  else if (p.out_type == MOE_OUT_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p.out)[at] = __float2half_rn(v);
}

// ---- output boxes: 32 rows x 128 bytes, 128-byte swizzle (16-byte piece j of row r at
// j ^ (r & 7)), one per warp.
// Direct stores of a lane's own row touch 32 lines per instruction; measured on B200 they cost
// the 8192 x 14336 x 4096 product 16 of 345 us and the 128-expert prefill 300 of 2690 us, where
// the TMA unit writes whole segments on its own.  (Two boxes of 64-byte rows: 16384 x 4096 x 1536 to
// bf16 91 us against 87, medians of five runs in turn on a warm box; it takes 73 on a cool one.)
struct I8Boxes {
  uint8_t* base;
  // A box that starts at (row, col): w0 and w1 are the halves of this lane's row.
  MOE_DEVINL void store(const CUtensorMap* m, int lane, int row, int col, const uint32_t* w0, const uint32_t* w1) {
    // (this warp's earlier store has read the box)
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t* w = j < 4 ? w0 + 4 * j : w1 + 4 * (j - 4);
      *reinterpret_cast<uint4*>(base + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                       reinterpret_cast<uint64_t>(m)),
                   "r"(col), "r"(row), "r"(smem_u32(base))
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  // 32 outputs of each of the warp's rows, the first `rows` of which are real, columns col .. col +
  // n - 1: through the boxes as 32 x 32 words (word c of row r at c ^ r), so that a warp stores along
  // a row.  For rows that are not whole sectors and for the last columns: element by element from
  // each lane's own row, 4000 x 3401 x 2048 in bf16 took 155 us, this way 36 (3400 columns: 27).
  MOE_DEVINL void store_rows(const I8Params& p, int lane, long long row, int rows, int col, const float (&v)[32], int n) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    float* words = reinterpret_cast<float*>(base);
#pragma unroll
    for (int i = 0; i < 32; ++i) words[lane * 32 + (i ^ lane)] = v[i];
    __syncwarp();
    const long long at = row * p.ldo + col + lane;
    if (lane < n) {
      if (p.out_type == MOE_OUT_FP32) copy_rows(words, lane, rows, static_cast<float*>(p.out) + at, p.ldo);
      else if (p.out_type == MOE_OUT_BF16) copy_rows(words, lane, rows, static_cast<__nv_bfloat16*>(p.out) + at, p.ldo);
      else copy_rows(words, lane, rows, static_cast<__half*>(p.out) + at, p.ldo);
    }
    __syncwarp();
  }
  template <class T>
  static MOE_DEVINL void copy_rows(const float* words, int lane, int rows, T* out, int64_t ldo) {
    float x[32];  // all reads before the first store, which they would wait for
#pragma unroll
    for (int r = 0; r < 32; ++r) x[r] = words[r * 32 + (lane ^ r)];
    if (rows >= 32) {
#pragma unroll
      for (int r = 0; r < 32; ++r, out += ldo) *out = static_cast<T>(x[r]);
    } else {
#pragma unroll
      for (int r = 0; r < 32; ++r, out += ldo)
        if (r < rows) *out = static_cast<T>(x[r]);
    }
  }
};

// tmA: boxes of 128 rows of A, tmA32: of 32.  tmB0 (and tmB1, the up weights of SWIGLU): boxes
// of B_ROWS rows, or of BN / 2 for SWIGLU.  tmOut (with p.tma_store): boxes of 32 rows x 128 bytes.
template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    tc_gemm_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                      const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                      const __grid_constant__ CUtensorMap tmOut, const I8Params p) {
  constexpr int CG = Cfg::CG, BN = Cfg::BN, BK = Cfg::BK, SUB = Cfg::SUB, STAGES = Cfg::STAGES;
  constexpr bool PAIR = CG == 2;
  constexpr uint32_t IDESC = idesc_i8_s32(Cfg::TILE_M, BN);

  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t full_bar[STAGES], empty_bar[STAGES];
  __shared__ uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ int pref[kI8MaxGroups + 1], cnt[kI8MaxGroups];
  __shared__ __align__(16) float col_sh[4][512];  // per epilogue warp: column scales, then biases
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ int no_abort_sh[2];

  const int warp = warp_id(), lane = lane_id();
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const uint32_t pad = (1024u - (smem_u32(dsmem) & 1023u)) & 1023u;
  uint8_t* smem = dsmem + pad;
  const int NT = (p.N + Cfg::OUT_COLS - 1) / Cfg::OUT_COLS;
  const int KB = (p.K + SUB * BK - 1) / (SUB * BK);  // stages' worth
  const int first_item = blockIdx.x / CG, step = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tempty_bar[a], 4 * CG);  // one lane of each epilogue warp
    }
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    no_abort_sh[0] = no_abort_sh[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmA32);
    prefetch_tmap(&tmB0);
    if (Cfg::SWIGLU) prefetch_tmap(&tmB1);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&tmem_base_sh, Cfg::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&tmem_base_sh, Cfg::TMEM_COLS);
      tmem_relinquish();
    }
  }
  // the counts and A come from the kernels before this one
  pdl_launch_dependents();
  pdl_wait();
  for (int g = threadIdx.x; g < p.G; g += Cfg::THREADS) cnt[g] = i8_count(p, g);
  __syncthreads();
  if (warp == 2) {
    // pref[] over the groups, one warp: each lane sums a contiguous run, then a scan
    const int per = (p.G + 31) / 32;
    const int g0 = lane * per;
    int run = 0;
    for (int g = g0; g < g0 + per && g < p.G; ++g) run += NT * ((cnt[g] + Cfg::TILE_M - 1) / Cfg::TILE_M);
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int acc = incl - run;
    for (int g = g0; g < g0 + per && g < p.G; ++g) {
      pref[g] = acc;
      acc += NT * ((cnt[g] + Cfg::TILE_M - 1) / Cfg::TILE_M);
    }
    if (lane == 31) pref[p.G] = incl;
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (PAIR) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  const int total = pref[p.G];

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    // (the whole warp in the loop and one elected lane issuing, as for the MMAs below)
    int s = 0;
    uint32_t ph = 0;
    long long issued = 0;
    bool ok = true;
    for (int item = first_item; item < total && ok; item += step) {
      const I8Tile t = i8_decode<Cfg>(item, NT, p, pref, cnt);
      const int a_box = i8_box_rows(t.count - t.m0 - 128 * static_cast<int>(rank));
      uint32_t tx = SUB * (static_cast<uint32_t>(a_box) * BK + Cfg::B_BYTES);
      if (PAIR) tx += SUB * (static_cast<uint32_t>(i8_box_rows(t.count - t.m0 - 128)) * BK + Cfg::B_BYTES);  // (the leader's)
      const int a_row = static_cast<int>(t.row0) + 128 * static_cast<int>(rank);
      const int b_row = t.group * p.N + t.n_tile * Cfg::OUT_COLS +
                        (PAIR && !Cfg::SWIGLU ? static_cast<int>(rank) * Cfg::B_ROWS : 0);
      const CUtensorMap* mA = a_box == kI8SmallRows ? &tmA32 : &tmA;
      for (int kb = 0; kb < KB; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty_bar[s], ph ^ 1u, &abort_flag));
        if (!ok) break;
        if (elect_one()) {
          if constexpr (PAIR) {
            if (leader) mbar_arrive_expect_tx(&full_bar[s], tx);
          } else {
            mbar_arrive_expect_tx(&full_bar[s], tx);
          }
#pragma unroll
          for (int j = 0; j < SUB; ++j) {  // (past K: zeros)
            uint8_t* sa = smem + s * Cfg::STAGE_BYTES + j * Cfg::BLOCK_BYTES;
            uint8_t* sb = sa + Cfg::A_BYTES;
            const int k = (kb * SUB + j) * BK;
            if constexpr (PAIR) {
              const uint32_t bar = mapa_shared(smem_u32(&full_bar[s]), 0);
              if (a_box > 0) tma_load_2d_pair(sa, mA, k, a_row, bar);
              tma_load_2d_pair(sb, (Cfg::SWIGLU && rank == 1) ? &tmB1 : &tmB0, k, b_row, bar);
            } else {
              tma_load_2d(sa, mA, k, a_row, &full_bar[s]);
              tma_load_2d(sb, &tmB0, k, b_row, &full_bar[s]);
              if constexpr (Cfg::SWIGLU) tma_load_2d(sb + Cfg::B_BYTES / 2, &tmB1, k, b_row, &full_bar[s]);
            }
          }
        }
        __syncwarp();
        ++issued;
        if (++s == STAGES) { s = 0; ph ^= 1u; }
      }
    }
    if (leader) {
      // (the leader's stage barriers count the peer's bytes too)
      volatile int* no_abort = &no_abort_sh[0];
      const long long back = issued < STAGES ? issued : STAGES;
      for (long long j = 0; j < back; ++j) {
        if (s == 0) { s = STAGES - 1; ph ^= 1u; } else { --s; }
        mbar_wait_bounded(&full_bar[s], ph, no_abort);
      }
      if (*no_abort) abort_flag = 1;
    }
    if (!ok) abort_flag = 1;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA (the leader's)
    // The whole warp runs the loop and one elected lane issues: what an MMA takes stays in
    // uniform registers.  With one lane in the loop every descriptor is moved there first, and
    // issuing four MMAs took longer than their 512 cycles (tensor pipe 83% busy without any
    // load or epilogue to wait for, 98% with uniform descriptors).
    if (leader) {
      int s = 0, acc = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));
      for (int item = first_item; item < total && ok; item += step) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&tempty_bar[acc], acc_ph ^ 1u, &abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < KB; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full_bar[s], ph, &abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = desc0 + static_cast<uint32_t>(s * (Cfg::STAGE_BYTES >> 4));
          const uint64_t db = da + (Cfg::A_BYTES >> 4);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
              for (int k = 0; k < BK / 32; ++k)
                umma_i8<CG>(d_tmem, da + j * (Cfg::BLOCK_BYTES >> 4) + 2 * k, db + j * (Cfg::BLOCK_BYTES >> 4) + 2 * k, IDESC,
                            (kb | j | k) != 0);
            if constexpr (PAIR) umma_commit_pair(&empty_bar[s]); else umma_commit(&empty_bar[s]);
          }
          __syncwarp();
          if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        if (elect_one()) {
          if constexpr (PAIR) umma_commit_pair(&tfull_bar[acc]); else umma_commit(&tfull_bar[acc]);
        }
        __syncwarp();
        if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
      }
      if (elect_one()) {
        if constexpr (PAIR) umma_commit_pair_local(&drain_bar); else umma_commit(&drain_bar);
      }
      __syncwarp();
      volatile int* no_abort = &no_abort_sh[1];
      mbar_wait_bounded(&drain_bar, 0, no_abort);
      if (!ok || *no_abort) abort_flag = 1;
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quadrant
    float* cols = col_sh[q];
    I8Boxes out_boxes{smem + STAGES * Cfg::STAGE_BYTES + q * kI8OutBox};
    // a row's 32 outputs are whole 32-byte sectors
    const bool whole = ((reinterpret_cast<uintptr_t>(p.out) |
                         static_cast<uintptr_t>(p.ldo * (Cfg::SWIGLU || p.out_type == MOE_OUT_FP32 ? 4 : 2))) & 31) == 0;
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&tempty_bar[0]), 0) : 0u;
    const uint32_t tempty1 = PAIR ? mapa_shared(smem_u32(&tempty_bar[1]), 0) : 0u;
    // A tile's scales are on their way while the tile before it is stored (read at its start they cost
    // 142 experts of 384 x 2048 with five rows each 121 us for 88, 81 of 896 x 384 with 477 126 for 111).
    constexpr int PER = Cfg::OUT_COLS / 32;
    I8Tile next;
    float next_sa = 0.f, next_cols[PER], next_more[PER];
    auto fetch = [&](int item) {
      next = i8_decode<Cfg>(item, NT, p, pref, cnt);
      const int col0 = next.n_tile * Cfg::OUT_COLS;
      const long long wrow = static_cast<long long>(next.group) * p.N + col0;
      const int in_tile = 128 * static_cast<int>(rank) + q * 32 + lane;
      next_sa = next.m0 + in_tile < next.count ? __ldg(p.a_scale + next.row0 + in_tile) : 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = 32 * i + lane;
        const bool in = col0 + c < p.N;
        next_cols[i] = in ? __ldg(p.w_scale + wrow + c) : 0.f;
        if constexpr (Cfg::SWIGLU) next_more[i] = in ? __ldg(p.w_scale_up + wrow + c) : 0.f;
        else next_more[i] = in && p.bias != nullptr ? __ldg(p.bias + col0 + c) : 0.f;
      }
    };
    if (first_item < total) fetch(first_item);
    int acc = 0;
    uint32_t acc_ph = 0;
    for (int item = first_item; item < total; item += step) {
      const I8Tile t = next;
      const int col0 = t.n_tile * Cfg::OUT_COLS;
      const int in_tile = 128 * static_cast<int>(rank) + q * 32 + lane;
      const long long row = t.row0 + in_tile;
      const bool row_ok = t.m0 + in_tile < t.count;
      const float sa = next_sa;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        cols[32 * i + lane] = next_cols[i];
        cols[(Cfg::SWIGLU ? 128 : 256) + 32 * i + lane] = next_more[i];
      }
      if (item + step < total) fetch(item + step);
      __syncwarp();
      const bool ready = __all_sync(0xffffffffu, mbar_wait_bounded(&tfull_bar[acc], acc_ph, &abort_flag));
      if (!ready) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
      // a warp's 32 rows go out in boxes where all of them are real, else row by row
      const bool boxes = p.tma_store && t.m0 + 128 * static_cast<int>(rank) + q * 32 + 32 <= t.count;
      const int box_row = static_cast<int>(t.row0) + 128 * static_cast<int>(rank) + q * 32;
      const int rows_here = t.count - t.m0 - 128 * static_cast<int>(rank) - q * 32;  // 32 or more: all
      if constexpr (Cfg::SWIGLU) {
        float* out = static_cast<float*>(p.out) + row * p.ldo + col0;
#pragma unroll 1
        for (int c = 0; c < Cfg::OUT_COLS; c += 32) {
          __syncwarp();
          uint32_t rg[32], ru[32];
          tmem_ld_32x32b_x32(tbase + c, rg);
          tmem_ld_32x32b_x32(tbase + BN / 2 + c, ru);
          tmem_ld_wait(rg);
          reg_fence(ru);
          float g[32], u[32];
          i8_scale32(rg, sa, cols + c, nullptr, g);
          i8_scale32(ru, sa, cols + 128 + c, nullptr, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) rg[i] = __float_as_uint(silu_mul(g[i], u[i]));
          if (boxes) {
            out_boxes.store(&tmOut, lane, box_row, col0 + c, rg, rg + 16);
          } else if (row_ok) {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global_v8(out + c + 8 * i, rg + 8 * i);
          }
        }
      } else {
        // 64 columns at a time: one wait and one fence for a box of 16-bit outputs
#pragma unroll 1
        for (int c = 0; c < BN; c += 64) {
          __syncwarp();
          uint32_t r[2][32];
#pragma unroll
          for (int j = 0; j < 2; ++j) tmem_ld_32x32b_x32(tbase + c + 32 * j, r[j]);
          tmem_ld_wait(r[0]);
          reg_fence(r[1]);
          if (col0 + c >= p.N) continue;
          if (boxes && p.out_type != MOE_OUT_FP32) {
            uint32_t w[2][16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float v[32];
              i8_scale32(r[j], sa, cols + c + 32 * j, p.bias != nullptr ? cols + 256 + c + 32 * j : nullptr, v);
              i8_pack32(p.out_type, v, w[j]);
            }
            out_boxes.store(&tmOut, lane, box_row, col0 + c, w[0], w[1]);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int col = col0 + c + 32 * j;
              if (col >= p.N) continue;
              float v[32];
              i8_scale32(r[j], sa, cols + c + 32 * j, p.bias != nullptr ? cols + 256 + c + 32 * j : nullptr, v);
              if (boxes) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
                out_boxes.store(&tmOut, lane, box_row, col, w, w + 16);
              } else if (whole && p.N - col >= 32) {
                if (row_ok) i8_store32(p, row, col, v, 32);
              } else if (rows_here > 0) {
                out_boxes.store_rows(p, lane, row - lane, rows_here, col, v, p.N - col);
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(acc == 0 ? tempty0 : tempty1);
        else mbar_arrive(&tempty_bar[acc]);
      }
      if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  __syncthreads();
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();  // both CTAs done with TMEM and with each other's barriers
  tc_fence_after();
  if (abort_flag && threadIdx.x == 0) set_status(p.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    else tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------- few rows
// The dense product where its tiles do not fill the SMs: KS CTAs of a cluster share one
// 128 x BN tile, each over its part of K.  A CTA finishes BN / KS of the columns: the others push
// their s32 sums of those columns into its shared memory (posted stores, nothing waits for a
// round trip), and after one cluster barrier it adds the KS parts (any order gives the same
// integer), scales and stores them.  No workspace, no atomics, one launch.
// What bounds it: HBM for long weights, else the K-loop's steps and the exchange.  Measured on B200:
// reading the parts from the peers instead of having them pushed 18.1 us against 15.4 (128 x 7168 x
// 4096); loads issued by one lane in the loop 0.24 us a step, by an elected lane of the whole warp
// 0.18, and with two K-blocks per step 0.14 a block (512 x 4096, 8 rows, one part: 10.5, 8.7, 6.9 us).
// LONE: one part, whose sums may go into the stage ring (others' could arrive while it is in use).
template <int BN_, int ROWS_, int SUB_, int STAGES_, bool LONE_>
struct I8SplitCfg {
  static constexpr int BN = BN_;
  static constexpr int ROWS = ROWS_;             // rows of A loaded (the MMA reads 128: what lies behind)
  static constexpr int SUB = SUB_;               // K-blocks of 128 per stage
  static constexpr int STAGES = STAGES_;
  static constexpr int BK = 128;
  static constexpr int A_BYTES = ROWS * BK;      // per K-block
  static constexpr int B_BYTES = BN * BK;
  static constexpr int RING_BYTES = STAGES * SUB * (A_BYTES + B_BYTES);  // all of A's blocks, then all of B's
  // received parts: [part][column group of 4][row ^ (group & 7)] int4: a warp's push (a lane per
  // row) is 512 contiguous bytes, and lanes that read along a row meet no bank twice
  static constexpr int GROUP_BYTES = ROWS * 16;
  static constexpr int PART_BYTES = ROWS * BN * 4;
  static constexpr bool LONE = LONE_;
  static constexpr int SMEM_BYTES = RING_BYTES + (LONE ? 0 : PART_BYTES) + 1024;
  static_assert(PART_BYTES <= RING_BYTES, "the sums fit the ring");
  static_assert(STAGES * SUB * B_BYTES >= 128 * BK - A_BYTES, "what the MMA reads behind A is in the ring");
  static constexpr int TMEM_COLS = BN;
  static constexpr int THREADS = 192;
  static_assert(SMEM_BYTES + 2 * BN * 4 + 2048 <= 227 * 1024, "shared memory");
};

MOE_DEVINL void st_cluster_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}

// Adds the KS parts of this CTA's 4 * groups columns from `col` on and stores them, `rows` rows from
// m0 on.  128 threads, lanes along a row: thread t keeps column group t % groups and takes every
// (128 / groups)th row.  KS and the output type are fixed at compile time: a CTA has one such warp
// per scheduler, so the stage takes as long as its instructions (with them in registers, and four
// rows at a time, 1 us instead of 3).
template <int KS, int TYPE, int GROUP_BYTES>
MOE_DEVINL void i8_finish_parts(const I8Params& p, const uint8_t* parts, int t, int log_groups, int m0, int rows, int col,
                                const float* scale, const float* bias, const float* row_scale) {
  using Word = typename std::conditional<TYPE == MOE_OUT_FP32, float4, uint2>::type;
  constexpr int ESZ = TYPE == MOE_OUT_FP32 ? 4 : 2;
  const int groups = 1 << log_groups, g = t & (groups - 1);
  col += 4 * g;
  if (col >= p.N) return;
  const float4 sw = *reinterpret_cast<const float4*>(scale + 4 * g);
  const float4 sb = *reinterpret_cast<const float4*>(bias + 4 * g);
  uint8_t* out = static_cast<uint8_t*>(p.out) + (m0 * p.ldo + col) * ESZ;
  const int64_t pitch = p.ldo * ESZ;
  const bool vec = p.N - col >= 4 && ((reinterpret_cast<uintptr_t>(out) | static_cast<uintptr_t>(pitch)) & (sizeof(Word) - 1)) == 0;
  const uint8_t* at = parts + g * GROUP_BYTES;
  const int part_bytes = groups * GROUP_BYTES, swz = g & 7;
#pragma unroll 4
  for (int r = t >> log_groups; r < rows; r += 128 >> log_groups) {
    int4 a[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) a[k] = *reinterpret_cast<const int4*>(at + k * part_bytes + ((r ^ swz) << 4));
#pragma unroll
    for (int k = 1; k < KS; ++k) {
      a[0].x += a[k].x; a[0].y += a[k].y; a[0].z += a[k].z; a[0].w += a[k].w;
    }
    const float2 s2 = make_float2(row_scale[r], row_scale[r]);
    const float2 lo = fma2(mul2(make_float2(__int2float_rn(a[0].x), __int2float_rn(a[0].y)), s2), make_float2(sw.x, sw.y),
                           make_float2(sb.x, sb.y));
    const float2 hi = fma2(mul2(make_float2(__int2float_rn(a[0].z), __int2float_rn(a[0].w)), s2), make_float2(sw.z, sw.w),
                           make_float2(sb.z, sb.w));
    if (vec) {
      Word w;
      if constexpr (TYPE == MOE_OUT_FP32) {
        w = make_float4(lo.x, lo.y, hi.x, hi.y);
      } else if constexpr (TYPE == MOE_OUT_BF16) {
        w = make_uint2(pack_bf16x2(lo.x, lo.y), pack_bf16x2(hi.x, hi.y));
      } else {
        const __half2 l = __floats2half2_rn(lo.x, lo.y), h = __floats2half2_rn(hi.x, hi.y);
        w = make_uint2(*reinterpret_cast<const uint32_t*>(&l), *reinterpret_cast<const uint32_t*>(&h));
      }
      *reinterpret_cast<Word*>(out + r * pitch) = w;
    } else {
      const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < p.N - col) i8_store1(p, m0 + r, col + i, v[i]);
    }
  }
}

// Grid: (KS, N-tiles, M-tiles), clusters of KS.
template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    tc_gemm_i8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                            const I8Params p) {
  constexpr int BN = Cfg::BN, BK = Cfg::BK, SUB = Cfg::SUB, STAGES = Cfg::STAGES;
  constexpr uint32_t IDESC = idesc_i8_s32(128, BN);
  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t full_bar[STAGES], empty_bar[STAGES], done_bar;
  __shared__ __align__(16) float scale_sh[BN], bias_sh[BN], row_sh[128];
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;

  const int warp = warp_id(), lane = lane_id();
  const uint32_t pad = (1024u - (smem_u32(dsmem) & 1023u)) & 1023u;
  uint8_t* smem = dsmem + pad;
  uint8_t* ring_b = smem + STAGES * SUB * Cfg::A_BYTES;
  uint8_t* parts = smem + (Cfg::LONE ? 0 : Cfg::RING_BYTES);
  const int ks = Cfg::LONE ? 1 : gridDim.x, part = blockIdx.x;  // the cluster spans the grid's x
  const int steps = (p.K + SUB * BK - 1) / (SUB * BK);
  int step0, step1;
  k_slice(part, ks, steps, step0, step1);
  const int m0 = blockIdx.z * 128, col0 = blockIdx.y * BN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  // (a CTA's shared memory may be written once it runs: waited for before the first push)
  if (ks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    // (the whole warp in the loop, one lane issues: see tc_gemm_i8_kernel)
    int s = 0;
    uint32_t ph = 0;
    int issued = 0;
    for (int step = step0; step < step1; ++step) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty_bar[s], ph ^ 1u, &abort_flag))) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full_bar[s], SUB * (Cfg::A_BYTES + Cfg::B_BYTES));
#pragma unroll
        for (int j = 0; j < SUB; ++j) {  // (past K: zeros)
          tma_load_2d(smem + (s * SUB + j) * Cfg::A_BYTES, &tmA, (step * SUB + j) * BK, m0, &full_bar[s]);
          tma_load_2d(ring_b + (s * SUB + j) * Cfg::B_BYTES, &tmB, (step * SUB + j) * BK, col0, &full_bar[s]);
        }
      }
      __syncwarp();
      ++issued;
      if (++s == STAGES) { s = 0; ph ^= 1u; }
    }
    volatile int no_abort = 0;
    const int back = issued < STAGES ? issued : STAGES;
    for (int j = 0; j < back; ++j) {
      if (s == 0) { s = STAGES - 1; ph ^= 1u; } else { --s; }
      mbar_wait_bounded(&full_bar[s], ph, &no_abort);
    }
    if (no_abort) abort_flag = 1;
  } else if (warp == 1) {
    int s = 0;
    uint32_t ph = 0;
    const uint64_t desc_a = smem_desc_sw128(smem_u32(smem)), desc_b = smem_desc_sw128(smem_u32(ring_b));
    for (int step = step0; step < step1; ++step) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full_bar[s], ph, &abort_flag))) break;
      tc_fence_after();
      const uint64_t da = desc_a + static_cast<uint32_t>(s * SUB * (Cfg::A_BYTES >> 4));
      const uint64_t db = desc_b + static_cast<uint32_t>(s * SUB * (Cfg::B_BYTES >> 4));
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            umma_i8<1>(tmem_base, da + j * (Cfg::A_BYTES >> 4) + 2 * k, db + j * (Cfg::B_BYTES >> 4) + 2 * k, IDESC,
                       step != step0 || (j | k) != 0);
        umma_commit(&empty_bar[s]);
      }
      __syncwarp();
      if (++s == STAGES) { s = 0; ph ^= 1u; }
    }
    if (elect_one()) umma_commit(&done_bar);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait_bounded(&done_bar, 0, &no_abort);
    if (no_abort) abort_flag = 1;
  }
  if (warp >= 2) {
    for (int c = threadIdx.x - 64; c < BN; c += 128) {
      const bool in = col0 + c < p.N;
      scale_sh[c] = in ? __ldg(p.w_scale + col0 + c) : 0.f;
      bias_sh[c] = in && p.bias != nullptr ? __ldg(p.bias + col0 + c) : 0.f;
    }
    const int r = threadIdx.x - 64;
    row_sh[r] = m0 + r < p.dense_rows ? __ldg(p.a_scale + m0 + r) : 0.f;
  }
  // the products and the copies are done, or were given up
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int q = warp & 3;
  const int row = q * 32 + lane;
  const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
  // groups of four columns that a CTA finishes: BN / ks columns, 8 at least
  const int log_groups = 29 - __clz(BN / ks), groups = 1 << log_groups;
  if (ks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // a lone CTA stores its rows straight from TMEM where they are whole 32-byte sectors (128 x 7168 x
  // 4096 12.0 us against 13.1 by way of shared memory; with unaligned rows 200 x 3000 x 2000 12.9
  // against 9.2)
  const int esz = p.out_type == MOE_OUT_FP32 ? 4 : 2;
  const bool direct = ks == 1 && ((reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(p.ldo * esz)) & 31) == 0;
  if (direct) {
    if (warp >= 2 && m0 + q * 32 < p.dense_rows) {
      const float sa = row_sh[row];
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        __syncwarp();
        uint32_t r[32];
        tmem_ld_32x32b_x32(tbase + c, r);
        tmem_ld_wait(r);
        if (m0 + row >= p.dense_rows || col0 + c >= p.N) continue;
        float v[32];
        i8_scale32(r, sa, scale_sh + c, p.bias != nullptr ? bias_sh + c : nullptr, v);
        i8_store32(p, m0 + row, col0 + c, v, p.N - col0 - c);
      }
    }
  } else if (warp >= 2 && m0 + q * 32 < p.dense_rows) {
    const uint32_t mine = smem_u32(parts) + part * groups * Cfg::GROUP_BYTES;
#pragma unroll 1
    for (int c = 0; c < BN; c += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tbase + c, r);
      tmem_ld_wait(r);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const int g = ((c + i) >> 2) & (groups - 1);
        const uint32_t to = mine + g * Cfg::GROUP_BYTES + ((row ^ (g & 7)) << 4);
        st_cluster_v4(ks > 1 ? mapa_shared(to, (c + i) >> (log_groups + 2)) : to, r + i);
      }
    }
  }
  __syncwarp();
  if (ks > 1) cluster_sync(); else __syncthreads();
  if (warp >= 2 && !direct) {
    const int t = threadIdx.x - 64, first = part * 4 * groups;
    const int rows = p.dense_rows - m0 < 128 ? p.dense_rows - m0 : 128;
    auto finish = [&](auto ks_c) {
      constexpr int KS = decltype(ks_c)::value;
      if (p.out_type == MOE_OUT_BF16)
        i8_finish_parts<KS, MOE_OUT_BF16, Cfg::GROUP_BYTES>(p, parts, t, log_groups, m0, rows, col0 + first, scale_sh + first, bias_sh + first, row_sh);
      else if (p.out_type == MOE_OUT_FP16)
        i8_finish_parts<KS, MOE_OUT_FP16, Cfg::GROUP_BYTES>(p, parts, t, log_groups, m0, rows, col0 + first, scale_sh + first, bias_sh + first, row_sh);
      else
        i8_finish_parts<KS, MOE_OUT_FP32, Cfg::GROUP_BYTES>(p, parts, t, log_groups, m0, rows, col0 + first, scale_sh + first, bias_sh + first, row_sh);
    };
    if constexpr (Cfg::LONE) finish(std::integral_constant<int, 1>());
    else if (ks == 2) finish(std::integral_constant<int, 2>());
    else finish(std::integral_constant<int, 4>());
  }
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) set_status(p.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

// 16 bytes read once (zero where !in); volatile: issued in the order written.
MOE_DEVINL int4 ld_stream(const int4* p, bool in) {
  int4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.cs.v4.s32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p), "r"(static_cast<int>(in)));
  return v;
}

// One to four rows: nothing to share in a tile, the weights are read once whatever is done with
// them.  A warp per R output channels, 16 codes per lane and load, integer dot products; the few
// rows of A come from L1, each load of them used for R channels.  Many warps keep the loads in
// flight, 64 an SM for one row (32 registers), 32 for four (52).  1 x 4096 x 7168 takes 7.1 us (4.1
// TB/s), most of the rest the first bytes' way.
template <int M, int R>
__global__ void __launch_bounds__(256) i8_gemv_kernel(const int8_t* __restrict__ a, int64_t lda,
                                                      const int8_t* __restrict__ w, int64_t ldw, const I8Params p) {
  pdl_launch_dependents();
  constexpr int UNROLL = M == 1 ? 16 : 4;
  const int lane = lane_id();
  const int n0 = (blockIdx.x * 8 + warp_id()) * R;
  // The first 4 KB of the warp's weights on their way into L2 while the kernel before this one still
  // runs: for the blocks that start before it ends.  (One that starts later asks just before it loads.)
  // A prefetch is not a read: whatever that kernel writes there is what is loaded below.
  if (p.prefetch) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (n0 + r < p.N && 128 * lane < p.K) asm volatile("prefetch.global.L2 [%0];" ::"l"(w + (n0 + r) * ldw + 128 * lane));
  }
  pdl_wait();
  if (n0 >= p.N) return;  // warp-uniform
  const int nvec = p.K / 16;
  int acc[R][M];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[r][m] = 0;
  for (int v0 = lane; v0 < nvec; v0 += 32 * UNROLL) {
    int4 q[R][UNROLL];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
        q[r][u] = ld_stream(reinterpret_cast<const int4*>(w + (n0 + r) * ldw) + v0 + 32 * u,
                            v0 + 32 * u < nvec && (R == 1 || n0 + r < p.N));
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int v = v0 + 32 * u < nvec ? v0 + 32 * u : lane;  // (past the end: times 0)
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int4 x = __ldg(reinterpret_cast<const int4*>(a + m * lda) + v);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][m] = __dp4a(q[r][u].x, x.x, acc[r][m]);
          acc[r][m] = __dp4a(q[r][u].y, x.y, acc[r][m]);
          acc[r][m] = __dp4a(q[r][u].z, x.z, acc[r][m]);
          acc[r][m] = __dp4a(q[r][u].w, x.w, acc[r][m]);
        }
      }
    }
  }
  // lane r * M + m finishes channel r of row m
  float mine = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int t = __reduce_add_sync(0xffffffffu, acc[r][m]);
      if (lane == r * M + m) mine = __int2float_rn(t);
    }
  const int n = n0 + lane / M, m = lane % M;
  // (sum, row scale, channel scale, as everywhere: the product of the scales alone may leave fp32's range)
  if (lane < R * M && n < p.N)
    i8_store1(p, m, n, fmaf(mine * __ldg(p.a_scale + m), __ldg(p.w_scale + n), p.bias != nullptr ? __ldg(p.bias + n) : 0.f));
}

}  // namespace moe
