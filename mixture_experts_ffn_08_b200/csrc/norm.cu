// Residual addition and root-mean-square norm, written in the input format of a layer.
//
//   z = bf16(x + residual)                       (z = x without a residual)
//   y = z * rstd * w,   rstd = 1 / sqrt(mean(z^2) + eps)
//   out = bf16(y)                                MOE_DTYPE_BF16
//       = e4m3(y / s), s = 2^ceil(log2(amax / 448)) per 128 channels   e4m3 activations
//       = int8(y / s), s = amax / 127 per token                        MOE_DTYPE_INT8
//
// One pass over the data: a block holds its row in registers between the reduction and the
// store, as the products z * w, which are exact in fp32 (bf16 times bf16).  The sum of squares
// and the row's largest |z * w| come out of one block reduction, because the largest |y| is
// rstd times it; the int8 codes, y / s = z w 127 / max|z w|, do not depend on rstd at all.
// The sum runs in fp32 over 8 channels and in fp64 beyond, and rstd takes one Newton step in
// fp64: a scale that is a power of two, or a code, changes where the true value lies within
// 1e-7 of a border and not within 1e-6.  An int8 code is taken from two estimates of 127 / max|z w|, next
// below and above it; where they disagree, z w and the border between the codes are compared exactly,
// and a tie goes to the even code.  (One estimate alone put 166 of 8 million codes, and half of the
// ties, on the wrong side.  The second costs 1 % of 16384 x 7168 with a residual, 6 % without, 0.15 of
// 3.4 us for 128 rows.)
//
// What bounds it is HBM: it reads x and the residual and writes the sum and the output once
// each.  Blocks are persistent: while a row is reduced and stored, the block's next row is on its
// way into shared memory (cp.async; every thread copies and reads back its own 16-byte vectors,
// so nothing waits for anybody but the reduction).  Six to eight instructions per channel: the sum
// is one bf16x2 addition per pair, products and sums of squares are packed fp32 pairs, an int8
// code is the low byte of a multiply-add onto 1.5 * 2^23.
// Measured on B200, 16384 x 7168 with a residual: bf16 146 us (939 MB, 6.4 TB/s), e4m3 131 (825 MB,
// 6.3 TB/s), int8 130 (822 MB, 6.3 TB/s); a plain copy runs at 6.45 TB/s.
#include <cuda_fp8.h>
#include <math_constants.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

enum NormFmt { NORM_BF16 = 0, NORM_E4M3 = 1, NORM_INT8 = 2 };

constexpr unsigned kAll = 0xffffffffu;

struct NormParams {
  const uint4* x;        // [T, nvec] vectors of 8 bf16
  const uint4* res;      // [T, nvec] or nullptr
  const uint4* w;        // [nvec]
  uint4* res_out;        // [T, nvec] or nullptr
  void* out;             // [T, nvec] vectors of 8 bf16 (16 bytes) or of 8 codes (8 bytes)
  float* scale;          // e4m3: [T, nvec / 16]; int8: [T]
  int nvec;
  float eps;
  double inv_h;          // 1 / H
};

// (|v| as an integer keeps the order of the values, infinities above them and NaN above those)
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kSmallBits = 0x05000000u;  // 2^-117: 448 / m of what lies below may be infinite

// Biased exponent (e + 127, at least 1) of the smallest 2^e with v <= 448 * 2^e, for the value
// v = m * rstd > 0 (448 = 1.75 * 2^8: a significand above 1.75 carries into the exponent).
// Next to that border the fp32 product decides nothing, and the fp64 one does.
MOE_DEVINL int e4m3_scale_bits(float m, float rstd_f, double rstd) {
  const uint32_t b = __float_as_uint(m * rstd_f);
  int e = static_cast<int>((b + 0x1fffffu) >> 23) - 8;
  if (((b - 0x5ffff8u) & 0x7fffffu) < 16u || b < 0x00800000u) {
    const double v = static_cast<double>(m) * rstd;
    const int hi = __double2hiint(v), lo = __double2loint(v);
    const int mant = hi & 0xfffff;
    e = ((hi >> 20) & 0x7ff) - 1023 + 127 - 8 + ((mant > 0xc0000 || (mant == 0xc0000 && lo != 0)) ? 1 : 0);
  }
  return e < 1 ? 1 : e;
}

MOE_DEVINL float2 unpack2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
// bf16(a + b) of two pairs.
MOE_DEVINL uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}
MOE_DEVINL uint4 add8(uint4 a, uint4 b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}
MOE_DEVINL uint32_t codes_e4m3(const float* v) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The row's statistics in every thread: ss = sum of squares, amax = bits of max |z w|.
// `buf` alternates between two rows of the shared arrays, so one barrier per row is enough.
MOE_DEVINL void block_reduce(double& ss, uint32_t& amax, double (*sh_ss)[32], uint32_t (*sh_amax)[32], int buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
  amax = __reduce_max_sync(kAll, amax);
  if (warps == 1) return;
  if (lane == 0) {
    sh_ss[buf][warp] = ss;
    sh_amax[buf][warp] = amax;
  }
  __syncthreads();
  ss = lane < warps ? sh_ss[buf][lane] : 0.0;
  amax = lane < warps ? sh_amax[buf][lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
  amax = __reduce_max_sync(kAll, amax);
}

// 1 / sqrt(m): the fp32 estimate and one Newton step in fp64.
MOE_DEVINL double rsqrt_newton(double m) {
  const double r = rsqrtf(static_cast<float>(m));
  return m < 3.0e38 ? r * (1.5 - 0.5 * m * r * r) : r;
}

// What a row's products z w are multiplied with, and how.
struct RowScale {
  float factor;      // bf16 and e4m3: rstd; int8: 127 / max |z w|
  float rest;        // e4m3: rstd - factor, so that a code sees one rounding
  double rstd;
  bool bad;          // e4m3, int8: a NaN, an infinity or a sum past fp32 in the row: scale NaN, codes 0
  bool wide;         // int8: `factor` does not fit fp32 well, multiply in fp64
  bool clamped;      // int8: the scale stopped at 2^-126
  double factor_wide;
  float above;       // int8: 127 / max |z w| lies between `factor` and this
  float amax;        // int8: max |z w|
};

template <int FMT>
MOE_DEVINL RowScale row_scale(double ss, uint32_t amax_bits, const NormParams& p, long long row) {
  RowScale r;
  const double mean = ss * p.inv_h + static_cast<double>(p.eps);
  r.bad = false;
  r.wide = false;
  r.clamped = false;
  r.factor_wide = 0.0;
  r.amax = __uint_as_float(amax_bits);
  if constexpr (FMT != NORM_INT8) {
    r.rstd = rsqrt_newton(mean);
    r.factor = static_cast<float>(r.rstd);
    r.rest = static_cast<float>(r.rstd - static_cast<double>(r.factor));
  }
  if constexpr (FMT != NORM_BF16) r.bad = !(ss < 3.0e38);
  if constexpr (FMT == NORM_INT8) {
    constexpr double smin = 1.1754943508222875e-38;  // 2^-126: a scale is a normal number
    r.bad = r.bad || amax_bits >= kInfBits;
    r.factor = r.above = 0.f;
    if (!r.bad && r.amax > 0.f) {
      const uint32_t f = __float_as_uint(127.f / r.amax);
      r.factor = __uint_as_float(f - 1);
      r.above = __uint_as_float(f + 1);
      // (the codes of ordinary rows do not need rstd, only the scale below does)
      if (r.amax < 1e-30f || r.amax * rsqrtf(static_cast<float>(mean)) < 1e-35f) {
        r.rstd = rsqrt_newton(mean);
        r.clamped = static_cast<double>(r.amax) * r.rstd < 127.0 * smin;
        r.wide = true;
        r.factor_wide = r.clamped ? r.rstd / smin : 127.0 / static_cast<double>(r.amax);
      }
    }
    if (threadIdx.x == 0) {
      const double s = static_cast<double>(r.amax) * rsqrt_newton(mean) * (1.0 / 127.0);
      p.scale[row] = r.bad ? CUDART_NAN_F : r.amax == 0.f ? 1.f : static_cast<float>(s < smin ? smin : s);
    }
  }
  return r;
}

// e4m3: the largest |z w| of the 128 channels, of which 16 lanes hold 8 each; called by whole warps.
MOE_DEVINL float block_largest(const float2 (&zw)[4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_abs(max_abs(m, zw[i].x), zw[i].y);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(kAll, m, o));
  return m;
}

// int8: the code of z w that lies near the border between the codes a and b = a +- 1: the one on whose side
// of it 127 z w / amax lies, the even one on it.  z w and amax have 16 significant bits, so both sides of
// the comparison are exact.
template <class F>
MOE_DEVINL F code_at_border(F zw, F amax, F a, F b) {
  const F v = zw * static_cast<F>(127.0 / 256), border = static_cast<F>(0.5) * (a + b) * (amax * static_cast<F>(1.0 / 256));
  if (v == border) return 2 * rint(static_cast<F>(0.25) * (a + b));
  return (v > border) == (b > a) ? b : a;
}

// Stores the 8 outputs of vector v (products zw; m: block_largest) of a row in bf16 or e4m3, where `in`.
template <int FMT>
MOE_DEVINL void store_vec(const float2 (&zw)[4], float m, const RowScale& r, const NormParams& p, long long row, int v,
                          bool in) {
  const long long at = row * p.nvec + v;
  if constexpr (FMT == NORM_BF16) {
    const float2 f = make_float2(r.factor, r.factor);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = mul2(zw[i], f);
      w[i] = pack_bf16x2(y.x, y.y);
    }
    if (in) static_cast<uint4*>(p.out)[at] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float2 y[4];
    float s = 1.f;
    const uint32_t mb = __float_as_uint(m);
    if (!r.bad && mb - kSmallBits < kInfBits - kSmallBits) {
      const int e = e4m3_scale_bits(m, r.factor, r.rstd);
      s = __int_as_float(e << 23);
      const float inv = __int_as_float((254 - e) << 23);
      const float2 f = make_float2(r.factor * inv, r.factor * inv), g = make_float2(r.rest * inv, r.rest * inv);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fma2(zw[i], f, mul2(zw[i], g));
    } else if (r.bad || mb >= kInfBits) {
      s = CUDART_NAN_F;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = make_float2(0.f, 0.f);
    } else {
      // rstd / s, which is about 448 / m, may pass fp32's range: z w is divided by s first
      const int e = m > 0.f ? e4m3_scale_bits(m, r.factor, r.rstd) : 127;
      s = __int_as_float(e << 23);
      const float inv = __int_as_float((254 - e) << 23);
      const float2 v = make_float2(inv, inv), f = make_float2(r.factor, r.factor), g = make_float2(r.rest, r.rest);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = mul2(zw[i], v);
        y[i] = fma2(t, f, mul2(t, g));
      }
    }
    const float* yv = reinterpret_cast<const float*>(y);
    if (in) {
      static_cast<uint2*>(p.out)[at] = make_uint2(codes_e4m3(yv), codes_e4m3(yv + 4));
      if ((threadIdx.x & 15) == 0) p.scale[at >> 4] = s;
    }
  }
}

// int8 codes of the 8 products of a vector by the estimate `factor`; `differ` is set where `above` gives others.
// (NaN and infinite products are in rows whose factors are 0 and whose codes are not stored.)
MOE_DEVINL uint2 codes_int8(const float2 (&zw)[4], const RowScale& r, uint32_t& differ) {
  const float2 magic = make_float2(kRoundMagic, kRoundMagic);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = fma2(zw[i], make_float2(r.factor, r.factor), magic), hi = fma2(zw[i], make_float2(r.above, r.above), magic);
    c[2 * i] = __float_as_uint(lo.x);
    c[2 * i + 1] = __float_as_uint(lo.y);
    differ |= __float_as_uint(lo.x) ^ __float_as_uint(hi.x);
    differ |= __float_as_uint(lo.y) ^ __float_as_uint(hi.y);
  }
  return make_uint2(low_bytes(c), low_bytes(c + 4));
}

// The same for every value, next to a border and in `wide` rows.  (A branch for each value: with the 8 of a
// vector at once, or the fp64 form in a call, registers spill and 16384 x 7168 takes 159 us for 130.)
MOE_DEVINL uint32_t code_int8_exact(float zw, const RowScale& r) {
  if (!r.wide) {
    const float lo = fmaf(zw, r.factor, kRoundMagic) - kRoundMagic, hi = fmaf(zw, r.above, kRoundMagic) - kRoundMagic;
    return static_cast<uint32_t>(static_cast<int>(lo == hi ? lo : code_at_border(zw, r.amax, lo, hi)));
  }
  const double v = static_cast<double>(zw) * r.factor_wide;
  double k = rint(v);
  if (!r.clamped && fabs(v - k) > 0.5 - 1e-9)
    k = code_at_border(static_cast<double>(zw), static_cast<double>(r.amax), k, k + (v > k ? 1.0 : -1.0));
  return static_cast<uint32_t>(__double2int_rn(k));
}
MOE_DEVINL uint2 codes_int8_exact(const float2 (&zw)[4], const RowScale& r) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = code_int8_exact(zw[i].x, r);
    c[2 * i + 1] = code_int8_exact(zw[i].y, r);
  }
  return make_uint2(low_bytes(c), low_bytes(c + 4));
}

// Stores the outputs of N vectors of a row, v0, v0 + step, ...; called by whole warps.  m: block_largest.
template <int FMT, int N>
MOE_DEVINL void store_vecs(const float2 (&zw)[N][4], const float (&m)[N], const RowScale& r, const NormParams& p, long long row,
                           int v0, int step) {
  if constexpr (FMT == NORM_INT8) {
    uint2 c[N];
    uint32_t differ = r.wide;  // (one branch for all vectors, whose steps the compiler mixes)
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = codes_int8(zw[i], r, differ);
    if (differ != 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) c[i] = codes_int8_exact(zw[i], r);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (v0 + i * step < p.nvec)
        static_cast<uint2*>(p.out)[row * p.nvec + v0 + i * step] = r.bad ? make_uint2(0u, 0u) : c[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = v0 + i * step;
      if ((v & ~31) < p.nvec) store_vec<FMT>(zw[i], m[i], r, p, row, v, v < p.nvec);
    }
  }
}

// The products zw of a vector z with its weights; adds its squares to ss, its largest to amax.
template <int FMT>
MOE_DEVINL void products(uint4 zq, uint4 wq, float2 (&zw)[4], double& ss, float& amax) {
  const uint32_t z[4] = {zq.x, zq.y, zq.z, zq.w}, w[4] = {wq.x, wq.y, wq.z, wq.w};
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(z[i]);
    s = fma2(v, v, s);
    zw[i] = mul2(v, unpack2(w[i]));
    if (FMT == NORM_INT8) amax = max_abs(max_abs(amax, zw[i].x), zw[i].y);
  }
  ss += static_cast<double>(s.x + s.y);
}

// Rows of at most 8 * VPT * blockDim channels, one at a time per block.  Thread t holds vectors
// t, t + blockDim, ... (VPT of them).  Shared memory: two buffers of [x, residual][VPT][blockDim]
// vectors, each thread's own.
template <int FMT, int VPT>
__global__ void __launch_bounds__(1024) norm_rows_kernel(const NormParams p, const int T) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ uint4 buf[];
  __shared__ double sh_ss[2][32];
  __shared__ uint32_t sh_amax[2][32];
  const int nt = blockDim.x, tid = threadIdx.x;
  const int streams = p.res != nullptr ? 2 : 1;
  auto slot = [&](int b, int stream, int i) { return buf + ((b * streams + stream) * VPT + i) * nt + tid; };
  auto fetch = [&](long long row, int b) {
    if (row < T) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * nt;
        if (v < p.nvec) {
          cp_async16(slot(b, 0, i), p.x + row * p.nvec + v);
          if (streams == 2) cp_async16(slot(b, 1, i), p.res + row * p.nvec + v);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  constexpr bool HOLD_W = VPT <= 2;  // (four vectors of weights do not fit the registers beside zw)
  uint4 w[HOLD_W ? VPT : 1];
  long long row = blockIdx.x;
  fetch(row, 0);
  if constexpr (HOLD_W) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) w[i] = tid + i * nt < p.nvec ? __ldg(p.w + tid + i * nt) : make_uint4(0, 0, 0, 0);
  }
  for (int b = 0; row < T; row += gridDim.x, b ^= 1) {
    fetch(row + gridDim.x, b ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    double ss = 0.0;
    float amax = 0.f;
    float2 zw[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * nt;
      if (v < p.nvec) {
        uint4 z = *slot(b, 0, i);
        if (streams == 2) {
          z = add8(z, *slot(b, 1, i));
          if (p.res_out != nullptr) p.res_out[row * p.nvec + v] = z;
        }
        if constexpr (HOLD_W) products<FMT>(z, w[i], zw[i], ss, amax);
        else products<FMT>(z, __ldg(p.w + v), zw[i], ss, amax);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) zw[i][j] = make_float2(0.f, 0.f);
      }
    }
    float m[VPT];  // (before the reduction, whose wait hides it)
#pragma unroll
    for (int i = 0; i < VPT; ++i) m[i] = FMT == NORM_E4M3 ? block_largest(zw[i]) : 0.f;
    uint32_t amax_bits = __float_as_uint(amax);
    block_reduce(ss, amax_bits, sh_ss, sh_amax, b);
    const RowScale r = row_scale<FMT>(ss, amax_bits, p, row);
    store_vecs<FMT, VPT>(zw, m, r, p, row, tid, nt);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Longer rows: two passes, a block per row.  The second reads the sum back where it was stored
// (over the residual, it may be) and makes it again where it was not.
template <int FMT>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ double sh_ss[2][32];
  __shared__ uint32_t sh_amax[2][32];
  const long long row = blockIdx.x, base = row * p.nvec;
  double ss = 0.0;
  float amax = 0.f;
  float2 zw[1][4];
  for (int v = threadIdx.x; v < p.nvec; v += blockDim.x) {
    uint4 z = p.x[base + v];
    if (p.res != nullptr) {
      z = add8(z, p.res[base + v]);
      if (p.res_out != nullptr) p.res_out[base + v] = z;
    }
    products<FMT>(z, __ldg(p.w + v), zw[0], ss, amax);
  }
  uint32_t amax_bits = __float_as_uint(amax);
  block_reduce(ss, amax_bits, sh_ss, sh_amax, 0);
  const RowScale r = row_scale<FMT>(ss, amax_bits, p, row);
  for (int v = threadIdx.x; (v & ~31) < p.nvec; v += blockDim.x) {
    const bool in = v < p.nvec;
    uint4 z = make_uint4(0, 0, 0, 0);
    if (in) {
      if (p.res_out != nullptr) z = p.res_out[base + v];
      else z = p.res != nullptr ? add8(p.x[base + v], p.res[base + v]) : p.x[base + v];
    }
    products<FMT>(z, in ? __ldg(p.w + v) : z, zw[0], ss, amax);
    const float m[1] = {FMT == NORM_E4M3 ? block_largest(zw[0]) : 0.f};
    store_vecs<FMT, 1>(zw, m, r, p, row, v, 0);
  }
}

template <int FMT, int VPT>
cudaError_t launch_rows(const NormParams& p, int T, cudaStream_t st) {
  const int threads = 32 * ((p.nvec + 32 * VPT - 1) / (32 * VPT));
  const int smem = 2 * (p.res != nullptr ? 2 : 1) * VPT * threads * 16;
  auto kern = norm_rows_kernel<FMT, VPT>;
  constexpr int most_smem = 2 * 2 * VPT * (VPT == 4 ? 832 : 1024) * 16;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t err = allow_smem(kern, most_smem, smem_set);
  if (err != cudaSuccess) return err;
  static std::atomic<int> regs_seen{0};  // registers per thread, the same on every device
  int regs = regs_seen.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    regs = (attr.numRegs + 7) & ~7;
    regs_seen.store(regs, std::memory_order_relaxed);
  }
  // As many blocks as the SMs hold at once, by shared memory and registers (with more, of which the
  // rest starts late, 300 x 7168 in bf16 took 6.2 us against 5.4).  Long batches take several times as
  // many, whose reads and writes mix better: with a residual 8 times in bf16 (16384 x 7168 161 to
  // 143 us) and 4 times in 8 bits (16384 x 4096 int8 85 to 75), without one twice in 8 bits (e4m3 64
  // to 62) and no more in bf16 (4 times: 44 to 45).
  int per_sm = 227 * 1024 / (smem + 2048);
  const int by_regs = 65536 / (regs * threads);
  per_sm = per_sm < by_regs ? per_sm : by_regs;
  per_sm = per_sm < 1 ? 1 : (per_sm > 16 ? 16 : per_sm);
  long long most = static_cast<long long>(num_sms()) * per_sm;
  if (threads >= 64 && T >= 6 * most) {
    if (FMT == NORM_BF16) most *= p.res != nullptr ? 8 : 1;
    else if (per_sm > 1) most *= p.res != nullptr ? 4 : 2;
  }
  const int grid = static_cast<int>(T < most ? T : most);
  return launch_k(kern, grid, threads, smem, st, p, T);
}

template <int FMT>
cudaError_t launch_fmt(const NormParams& p, int T, cudaStream_t st) {
  // one vector per thread where an SM has one row at most, or a row is one warp's
  if (p.nvec <= 32 || (p.nvec <= 1024 && T <= num_sms())) return launch_rows<FMT, 1>(p, T, st);
  if (p.nvec <= 2048) return launch_rows<FMT, 2>(p, T, st);
  if (p.nvec <= 3328) return launch_rows<FMT, 4>(p, T, st);
  return launch_k(norm_long_kernel<FMT>, T, 1024, 0, st, p);
}

}  // namespace

cudaError_t launch_add_rms_norm(const moe_params_t& p, const void* x, const void* residual, const void* w, float eps,
                                void* residual_out, void* out, float* scale, cudaStream_t st) {
  if (p.T == 0) return cudaSuccess;
  NormParams np{};
  np.x = static_cast<const uint4*>(x);
  np.res = static_cast<const uint4*>(residual);
  np.w = static_cast<const uint4*>(w);
  np.res_out = static_cast<uint4*>(residual_out);
  np.out = out;
  np.scale = scale;
  np.nvec = p.H / 8;
  np.eps = eps;
  np.inv_h = 1.0 / p.H;
  trace_before(MOE_K_NORM, st);
  const cudaError_t err = p.dtype == MOE_DTYPE_INT8 ? launch_fmt<NORM_INT8>(np, p.T, st)
                          : act_e4m3(p)             ? launch_fmt<NORM_E4M3>(np, p.T, st)
                                                    : launch_fmt<NORM_BF16>(np, p.T, st);
  trace_after(MOE_K_NORM, st);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe
