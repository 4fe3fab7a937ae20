// Host side of the int8 products (tc_gemm_i8.cuh): tensor maps, the choice of tile, launches;
// and the re-quantisation of the experts' intermediate h.
#include <cudaTypedefs.h>
#include <math_constants.h>

#include "i8_choice.h"
#include "internal.h"
#include "tc_gemm_i8.cuh"

namespace moe {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn_i8() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
  }();
  return fn;
}

// 8-bit matrix [rows, cols] with row stride ld bytes: boxes of 128 columns (one 128-byte swizzle
// row) x box_rows rows; what lies outside the matrix reads as zero and adds nothing.
bool make_tmap_i8(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
  auto fn = encode_fn_i8();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output [rows, cols] of 2- or 4-byte elements, row stride ld elements: boxes of 32 rows x 128
// bytes.  False where the rows do not start and end on 16-byte borders (the store unit clips a box
// at such a border: it was seen to write past cols); the kernel then stores element by element.
bool make_tmap_out(CUtensorMap* m, void* ptr, uint64_t rows, uint64_t cols, uint64_t ld, bool wide) {
  auto fn = encode_fn_i8();
  const uint64_t esz = wide ? 4 : 2;
  if (fn == nullptr || (reinterpret_cast<uintptr_t>(ptr) & 15u) != 0 || ld * esz % 16 != 0 || cols * esz % 16 != 0 ||
      ld * esz >= (1ull << 40))
    return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld * esz};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esz), 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, wide ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, ptr, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

long long cdiv(long long a, long long b) { return i8_cdiv(a, b); }

// A [a_rows, K] (row stride lda), B [b_rows, K] (row stride ldb; b1: SWIGLU's up weights).
template <class Cfg>
cudaError_t launch_i8(const void* A, int64_t a_rows, int64_t lda, const void* b0, const void* b1, int64_t b_rows,
                      int64_t ldb, I8Params p, long long max_items, int kid, cudaStream_t st) {
  constexpr uint32_t b_box = Cfg::SWIGLU ? Cfg::BN / 2 : Cfg::B_ROWS;
  CUtensorMap ta, ta32, tb0, tb1;
  if (!make_tmap_i8(&ta, A, a_rows, p.K, lda, 128) || !make_tmap_i8(&ta32, A, a_rows, p.K, lda, kI8SmallRows) ||
      !make_tmap_i8(&tb0, b0, b_rows, p.K, ldb, b_box))
    return cudaErrorInvalidValue;
  tb1 = tb0;  // (read by SWIGLU only)
  if (Cfg::SWIGLU && !make_tmap_i8(&tb1, b1, b_rows, p.K, ldb, b_box)) return cudaErrorInvalidValue;
  CUtensorMap tout;
  const bool wide = Cfg::SWIGLU || p.out_type == MOE_OUT_FP32;
  p.tma_store = make_tmap_out(&tout, p.out, a_rows, p.N, p.ldo, wide) ? 1 : 0;
  if (!p.tma_store) tout = ta;  // never used then
  auto kern = tc_gemm_i8_kernel<Cfg>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t err = allow_smem(kern, Cfg::SMEM_BYTES, smem_set);
  if (err != cudaSuccess) return err;
  const long long most = num_sms() / Cfg::CG;
  const long long n = max_items < most ? (max_items > 0 ? max_items : 1) : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(Cfg::CG * n), 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pdl_enabled()) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  if (Cfg::CG > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = Cfg::CG;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  trace_before(kid, st);
  err = cudaLaunchKernelEx(&cfg, kern, ta, ta32, tb0, tb1, tout, p);
  trace_after(kid, st);
  return err != cudaSuccess ? err : cudaGetLastError();
}

// One tile per cluster of ks CTAs.
template <class Cfg>
cudaError_t launch_i8_split(const void* a, int64_t lda, const void* w, int64_t ldw, const I8Params& p, int ks,
                            cudaStream_t st) {
  const int M = p.dense_rows;
  CUtensorMap ta, tb;
  if (!make_tmap_i8(&ta, a, M, p.K, lda, Cfg::ROWS) || !make_tmap_i8(&tb, w, p.N, p.K, ldw, Cfg::BN))
    return cudaErrorInvalidValue;
  auto kern = tc_gemm_i8_split_kernel<Cfg>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t err = allow_smem(kern, Cfg::SMEM_BYTES, smem_set);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ks, static_cast<unsigned>(cdiv(p.N, Cfg::BN)), static_cast<unsigned>(cdiv(M, 128)));
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  trace_before(MOE_K_LINEAR, st);
  err = cudaLaunchKernelEx(&cfg, kern, ta, tb, p);
  trace_after(MOE_K_LINEAR, st);
  return err != cudaSuccess ? err : cudaGetLastError();
}

// As many stages as shared memory holds beside scales, barriers and parts, of two K-blocks each but for
// the largest tile (128 x 4096 x 7168 in four parts of 128 columns: 11.9 us, 12.3 with two).
template <int BN, int ROWS>
constexpr int split_sub() { return BN == 128 && ROWS == 128 ? 1 : 2; }
template <int BN, int ROWS, bool LONE>
constexpr int split_stages() {
  constexpr int parts = LONE ? 0 : ROWS * BN * 4;
  constexpr int n = (221 * 1024 - 2 * BN * 4 - parts) / (split_sub<BN, ROWS>() * (ROWS + BN) * 128);
  return n < 12 ? n : 12;
}
template <int BN, int ROWS, bool LONE>
using SplitCfg = I8SplitCfg<BN, ROWS, split_sub<BN, ROWS>(), split_stages<BN, ROWS, LONE>(), LONE>;

template <int ROWS>
cudaError_t launch_i8_split_rows(const void* a, int64_t lda, const void* w, int64_t ldw, const I8Params& p, int bn, int ks,
                                 cudaStream_t st) {
  if (ks == 1) {
    if (bn == 32) return launch_i8_split<SplitCfg<32, ROWS, true>>(a, lda, w, ldw, p, 1, st);
    if (bn == 64) return launch_i8_split<SplitCfg<64, ROWS, true>>(a, lda, w, ldw, p, 1, st);
    return launch_i8_split<SplitCfg<128, ROWS, true>>(a, lda, w, ldw, p, 1, st);
  }
  if (bn == 32) return launch_i8_split<SplitCfg<32, ROWS, false>>(a, lda, w, ldw, p, ks, st);
  if (bn == 64) return launch_i8_split<SplitCfg<64, ROWS, false>>(a, lda, w, ldw, p, ks, st);
  return launch_i8_split<SplitCfg<128, ROWS, false>>(a, lda, w, ldw, p, ks, st);
}

template <int M, int R>
cudaError_t launch_i8_gemv(const void* a, int64_t lda, const void* w, int64_t ldw, I8Params p, cudaStream_t st) {
  // Up to eight blocks an SM, what it holds of the one-row kernel at once (of the others four to six),
  // and no more than L2 takes in passing: 1 x 4096 x 7168 7.2 -> 6.5 us in one session, but 2 x 14336 x 4096, where the
  // loads wait for it, 13.6 -> 15.7.
  p.prefetch = pdl_enabled() && cdiv(p.N, 8 * R) <= 8LL * num_sms() &&
               static_cast<long long>(p.N) * (p.K < 4096 ? p.K : 4096) <= (24LL << 20);
  trace_before(MOE_K_LINEAR, st);
  const cudaError_t err = launch_k(i8_gemv_kernel<M, R>, static_cast<int>(cdiv(p.N, 8 * R)), 256, 0, st,
                                   static_cast<const int8_t*>(a), lda, static_cast<const int8_t*>(w), ldw, p);
  trace_after(MOE_K_LINEAR, st);
  return err != cudaSuccess ? err : cudaGetLastError();
}

// ------------------------------------------------------------------ h -> int8
// q = rint(h / s), s = max|h| / 127 over the row (1 where the row is zero), as int8 codes and one
// fp32 scale per row.  A row with a NaN or an infinity gets codes 0 and scale NaN, so that its
// outputs are NaN.  Only the groups' real rows are read and written.
// What bounds it is HBM: 4 bytes read and 1 written per element.  A block holds one row in
// registers between its largest value and its codes, up to 32 elements a thread, all of whose
// loads are in flight at once; enough blocks share an SM that some load while others store.
// (Fewer threads with more elements and the next row prefetched into shared memory took 346 us
// for 131072 rows of 1536, and runs of rows per block instead of alternating ones 322, against
// 170.)
struct QuantParams {
  const float* h;
  const int32_t* offsets;
  const int32_t* counts;
  int E;
  int cap;
  int cols;
  int8_t* codes;
  float* scale;
};

// Numbers the real rows 0, 1, ... over the groups: pref[g] real rows lie before group g's.
struct RealRows {
  const QuantParams& p;
  int* pref;  // [E + 1], shared
  // one block-wide scan of the counts
  MOE_DEVINL RealRows(const QuantParams& params, int* shared_pref, int* warp_tot) : p(params), pref(shared_pref) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int per = (p.E + blockDim.x - 1) / blockDim.x, g0 = tid * per;
    int run = 0;
    for (int g = g0; g < g0 + per && g < p.E; ++g) run += count(g);
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int acc = incl - run;
    for (int w = 0; w < warp; ++w) acc += warp_tot[w];
    for (int g = g0; g < g0 + per && g < p.E; ++g) {
      pref[g] = acc;
      acc += per == 1 ? run : count(g);
    }
    if (warp == warps - 1 && lane == 31) pref[p.E] = acc;
    __syncthreads();
  }
  MOE_DEVINL int count(int g) const {
    return real_rows(p.offsets, p.counts, p.cap, g);
  }
  MOE_DEVINL int total() const { return pref[p.E]; }
  // where real row i lies
  MOE_DEVINL long long row(int i) const {
    int lo = 0, hi = p.E - 1;  // group with pref[g] <= i < pref[g+1]
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pref[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return (p.cap > 0 ? static_cast<long long>(lo) * p.cap : __ldg(p.offsets + lo)) + i - pref[lo];
  }
};

MOE_DEVINL uint32_t absmax4(uint32_t m, float4 v) {
  return __float_as_uint(max_abs(max_abs(max_abs(max_abs(__uint_as_float(m), v.x), v.y), v.z), v.w));
}

MOE_DEVINL uint32_t quant4(float4 v, float f) {
  const float2 ff = make_float2(f, f), magic = make_float2(kRoundMagic, kRoundMagic);
  const float2 a = fma2(make_float2(v.x, v.y), ff, magic), b = fma2(make_float2(v.z, v.w), ff, magic);
  const uint32_t c[4] = {__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
  return low_bytes(c);
}

// Scale of a row whose largest value has bits m, and what its values are multiplied with.
MOE_DEVINL float row_quant(uint32_t m, float& f, bool& bad) {
  bad = m >= 0x7f800000u;
  const float s = bad ? CUDART_NAN_F : (m == 0 ? 1.f : fmaxf(__uint_as_float(m) / 127.f, 1.1754943508222875e-38f));
  f = bad ? 0.f : 1.f / s;
  return s;
}

// The block's largest m, one barrier (`buf` alternates).
MOE_DEVINL uint32_t block_max(uint32_t m, uint32_t (*sh)[32], int buf) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  m = __reduce_max_sync(0xffffffffu, m);
  if (warps == 1) return m;
  if (lane == 0) sh[buf][threadIdx.x >> 5] = m;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < warps ? sh[buf][lane] : 0u);
}

template <int VPT>
__global__ void __launch_bounds__(512) quant_rows_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t sh[2][32];
  __shared__ int pref[kI8MaxGroups + 1], warp_tot[32];
  const int nt = blockDim.x, tid = threadIdx.x, n4 = p.cols / 4;
  const RealRows rows(p, pref, warp_tot);
  const int total = rows.total();
  for (int k = blockIdx.x, turn = 0; k < total; k += gridDim.x, turn ^= 1) {
    const long long r = rows.row(k);
    const float4* src = reinterpret_cast<const float4*>(p.h + r * p.cols);
    float4 x[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) x[i] = tid + i * nt < n4 ? __ldcs(src + tid + i * nt) : make_float4(0.f, 0.f, 0.f, 0.f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) m = absmax4(m, x[i]);
    m = block_max(m, sh, turn);
    float f;
    bool bad;
    const float s = row_quant(m, f, bad);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + r * p.cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (tid + i * nt < n4) dst[tid + i * nt] = bad ? 0u : quant4(x[i], f);
    if (tid == 0) p.scale[r] = s;
  }
}

// Rows that do not fit the registers (more than 16384 columns): two passes, the second from L2.
__global__ void __launch_bounds__(1024) quant_long_rows_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t sh[2][32];
  __shared__ int pref[kI8MaxGroups + 1], warp_tot[32];
  const int n4 = p.cols / 4;
  const RealRows rows(p, pref, warp_tot);
  const int total = rows.total();
  int b = 0;
  for (int k = blockIdx.x; k < total; k += gridDim.x, b ^= 1) {
    const long long r = rows.row(k);
    const float4* src = reinterpret_cast<const float4*>(p.h + r * p.cols);
    uint32_t m = 0;
    for (int v = threadIdx.x; v < n4; v += blockDim.x) m = absmax4(m, src[v]);
    m = block_max(m, sh, b);
    float f;
    bool bad;
    const float s = row_quant(m, f, bad);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + r * p.cols);
    for (int v = threadIdx.x; v < n4; v += blockDim.x) dst[v] = bad ? 0u : quant4(src[v], f);
    if (threadIdx.x == 0) p.scale[r] = s;
  }
}

template <int VPT>
cudaError_t launch_quant(const QuantParams& p, long long max_rows, cudaStream_t st) {
  const int n4 = p.cols / 4, threads = 32 * ((n4 + 32 * VPT - 1) / (32 * VPT));
  const int per_sm = 1024 / threads < 32 ? 1024 / threads : 32;  // (64 registers a thread)
  const long long most = static_cast<long long>(num_sms()) * per_sm;
  return launch_k(quant_rows_kernel<VPT>, static_cast<int>(max_rows < most ? max_rows : most), threads, 0, st, p);
}

// int8 codes as bf16 (exact), for the router's product.
__global__ void __launch_bounds__(256) codes_to_bf16_kernel(const uint2* __restrict__ q, long long n8,
                                                            uint4* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  for (long long v = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; v < n8;
       v += static_cast<long long>(gridDim.x) * blockDim.x) {
    const uint2 c = __ldg(q + v);
    const uint32_t w[2] = {c.x, c.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t half = w[i >> 1] >> (16 * (i & 1));
      o[i] = pack_bf16x2(static_cast<float>(static_cast<int8_t>(half & 0xffu)),
                         static_cast<float>(static_cast<int8_t>((half >> 8) & 0xffu)));
    }
    out[v] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace

cudaError_t launch_codes_to_bf16(const void* q, long long n, void* x_bf16, cudaStream_t st) {
  const long long n8 = n / 8, want = cdiv(n8, 256);
  const int grid = static_cast<int>(want < num_sms() * 8LL ? want : num_sms() * 8LL);
  trace_before(MOE_K_DEQUANT_X, st);
  const cudaError_t err = launch_k(codes_to_bf16_kernel, grid, 256, 0, st, static_cast<const uint2*>(q), n8,
                                   static_cast<uint4*>(x_bf16));
  trace_after(MOE_K_DEQUANT_X, st);
  return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_quant_rows(const float* h, long long max_rows, const int32_t* offsets, const int32_t* counts, int E,
                              int cap, int cols, void* codes, float* scale, cudaStream_t st) {
  const QuantParams p{h, offsets, counts, E, cap, cols, static_cast<int8_t*>(codes), scale};
  trace_before(MOE_K_QUANT_H, st);
  cudaError_t err;
  if (cols <= 512) {
    err = launch_quant<4>(p, max_rows, st);
  } else if (cols <= 16384) {
    err = launch_quant<8>(p, max_rows, st);
  } else {
    const long long most = num_sms();
    err = launch_k(quant_long_rows_kernel, static_cast<int>(max_rows < most ? max_rows : most), 1024, 0, st, p);
  }
  trace_after(MOE_K_QUANT_H, st);
  return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t gemm_i8_gateup_swiglu(const I8Rows& a, const void* w_gate, const void* w_up, const float* gate_scale,
                                  const float* up_scale, int N, int K, float* h, int32_t* status, int tile,
                                  cudaStream_t st) {
  I8Params p{};
  p.offsets = a.offsets;
  p.counts = a.counts;
  p.G = a.G;
  p.masked_cap = a.masked_cap;
  p.K = K;
  p.N = N;
  p.a_scale = a.scale;
  p.w_scale = gate_scale;
  p.w_scale_up = up_scale;
  p.out = h;
  p.ldo = N;
  p.status = status;
  const int64_t b_rows = static_cast<int64_t>(a.G) * N;
  const long long mt = cdiv(a.rows, 128);
  if (tile == kI8PairTile)
    return launch_i8<I8Cfg<2, 256, true, 6>>(a.codes, a.rows, K, w_gate, w_up, b_rows, K, p, mt * cdiv(N, 128), MOE_K_GATEUP, st);
  if (tile == 256)
    return launch_i8<I8Cfg<1, 256, true, 4>>(a.codes, a.rows, K, w_gate, w_up, b_rows, K, p, mt * cdiv(N, 128), MOE_K_GATEUP, st);
  if (tile == 128)
    return launch_i8<I8Cfg<1, 128, true, 3, 2>>(a.codes, a.rows, K, w_gate, w_up, b_rows, K, p, mt * cdiv(N, 64), MOE_K_GATEUP, st);
  return launch_i8<I8Cfg<1, 64, true, 4, 2>>(a.codes, a.rows, K, w_gate, w_up, b_rows, K, p, mt * cdiv(N, 32), MOE_K_GATEUP, st);
}

cudaError_t gemm_i8_down(const I8Rows& a, const void* w, const float* w_scale, int N, int K, void* y, int32_t* status,
                         int tile, cudaStream_t st) {
  I8Params p{};
  p.offsets = a.offsets;
  p.counts = a.counts;
  p.G = a.G;
  p.masked_cap = a.masked_cap;
  p.K = K;
  p.N = N;
  p.a_scale = a.scale;
  p.w_scale = w_scale;
  p.out = y;
  p.out_type = MOE_OUT_BF16;
  p.ldo = N;
  p.status = status;
  const int64_t b_rows = static_cast<int64_t>(a.G) * N;
  const long long mt = cdiv(a.rows, 128);
  if (tile == kI8PairTile)
    return launch_i8<I8Cfg<2, 256, false, 6>>(a.codes, a.rows, K, w, w, b_rows, K, p, mt * cdiv(N, 256), MOE_K_DOWN, st);
  if (tile == 256)
    return launch_i8<I8Cfg<1, 256, false, 4>>(a.codes, a.rows, K, w, w, b_rows, K, p, mt * cdiv(N, 256), MOE_K_DOWN, st);
  if (tile == 128)
    return launch_i8<I8Cfg<1, 128, false, 3, 2>>(a.codes, a.rows, K, w, w, b_rows, K, p, mt * cdiv(N, 128), MOE_K_DOWN, st);
  return launch_i8<I8Cfg<1, 64, false, 4, 2>>(a.codes, a.rows, K, w, w, b_rows, K, p, mt * cdiv(N, 64), MOE_K_DOWN, st);
}

cudaError_t gemm_i8_linear(int M, int N, int K, const void* a, int64_t lda, const float* a_scale, const void* w,
                           int64_t ldw, const float* w_scale, const float* bias, int out_type, void* out, int64_t ldo,
                           int32_t* status, cudaStream_t st) {
  I8Params p{};
  p.G = 1;
  p.dense_rows = M;
  p.K = K;
  p.N = N;
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.bias = bias;
  p.out = out;
  p.out_type = out_type;
  p.ldo = ldo;
  p.status = status;
  const I8Choice c = i8_linear_choice(M, N, K, num_sms());
  if (c.kernel == I8_DOT) {
    if (M == 1) return launch_i8_gemv<1, 1>(a, lda, w, ldw, p, st);
    if (M == 2 && c.channels == 2) return launch_i8_gemv<2, 2>(a, lda, w, ldw, p, st);
    if (M == 2) return launch_i8_gemv<2, 1>(a, lda, w, ldw, p, st);
    if (M == 3) return launch_i8_gemv<3, 1>(a, lda, w, ldw, p, st);
    return launch_i8_gemv<4, 1>(a, lda, w, ldw, p, st);
  }
  if (c.kernel == I8_PERSISTENT) {
    if (c.bn == kI8PairTile)
      return launch_i8<I8Cfg<2, 256, false, 6>>(a, M, lda, w, w, N, ldw, p, cdiv(M, 256) * cdiv(N, 256), MOE_K_LINEAR, st);
    if (c.bn == 256) return launch_i8<I8Cfg<1, 256, false, 4>>(a, M, lda, w, w, N, ldw, p, cdiv(N, 256), MOE_K_LINEAR, st);
    return launch_i8<I8Cfg<1, 128, false, 3, 2>>(a, M, lda, w, w, N, ldw, p, cdiv(N, 128), MOE_K_LINEAR, st);
  }
  if (c.rows == 32) return launch_i8_split_rows<32>(a, lda, w, ldw, p, c.bn, c.ks, st);
  if (c.rows == 64) return launch_i8_split_rows<64>(a, lda, w, ldw, p, c.bn, c.ks, st);
  return launch_i8_split_rows<128>(a, lda, w, ldw, p, c.bn, c.ks, st);
}

}  // namespace moe
