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
// 1e-7 of a border and not within 1e-6.  What bounds it is HBM: it reads x and the residual and
// writes the sum and the output once each.
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

MOE_DEVINL void unpack8(uint4 q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

MOE_DEVINL uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// |v| as an integer: the order of the values, infinities above them and NaN above those.
MOE_DEVINL uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// Smallest e >= -126 with v <= 448 * 2^e, for finite v > 0 (448 = 1.75 * 2^8).
MOE_DEVINL int e4m3_exponent(double v) {
  const int hi = __double2hiint(v), lo = __double2loint(v);
  const int mant = hi & 0xfffff;
  const int e = ((hi >> 20) & 0x7ff) - 1023 - 8 + ((mant > 0xc0000 || (mant == 0xc0000 && lo != 0)) ? 1 : 0);
  return e < -126 ? -126 : (e > 127 ? 127 : e);
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

// What a row's elements are multiplied with, and how.
struct RowScale {
  float factor;      // bf16: rstd; e4m3: rstd; int8: 127 / max |z w|
  double rstd;
  bool bad;          // e4m3, int8: a NaN, an infinity or a sum past fp32 in the row: scale NaN, codes 0
  bool wide;         // int8: `factor` does not fit fp32 well, multiply in fp64
  double factor_wide;
};

template <int FMT>
MOE_DEVINL RowScale row_scale(double ss, uint32_t amax_bits, const NormParams& p, long long row) {
  RowScale r;
  r.rstd = rsqrt_newton(ss * p.inv_h + static_cast<double>(p.eps));
  r.factor = static_cast<float>(r.rstd);
  r.bad = false;
  r.wide = false;
  r.factor_wide = 0.0;
  if constexpr (FMT != NORM_BF16) r.bad = !(ss < 3.0e38) || amax_bits >= kInfBits;
  if constexpr (FMT == NORM_INT8) {
    const float amax = __uint_as_float(amax_bits);
    float s = 1.f;
    r.factor = 0.f;
    if (r.bad) {
      s = CUDART_NAN_F;
    } else if (amax > 0.f) {
      const double sd = static_cast<double>(amax) * r.rstd / 127.0;
      const double smin = 1.1754943508222875e-38;  // 2^-126: a scale is a normal number
      s = static_cast<float>(sd < smin ? smin : sd);
      r.factor = 127.f / amax;
      r.wide = amax < 1e-30f || sd < smin;
      if (r.wide) r.factor_wide = sd < smin ? r.rstd / smin : 127.0 / static_cast<double>(amax);
    }
    if (threadIdx.x == 0) p.scale[row] = s;
  }
  return r;
}

// Stores the 8 outputs of vector v (products zw) of a row; called by whole half-warps.
template <int FMT>
MOE_DEVINL void store_vec(const float (&zw)[8], const RowScale& r, const NormParams& p, long long row, int v) {
  const long long at = row * p.nvec + v;
  if constexpr (FMT == NORM_BF16) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = zw[i] * r.factor;
    static_cast<uint4*>(p.out)[at] = pack8(y);
  } else if constexpr (FMT == NORM_E4M3) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(zw[i]));
    m = __reduce_max_sync(0xffffu << (threadIdx.x & 16), m);  // 16 lanes hold the 128 channels
    float y[8];
    float s = 1.f;
    if (r.bad) {
      s = CUDART_NAN_F;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = 0.f;
    } else {
      const int e = m > 0 ? e4m3_exponent(static_cast<double>(__uint_as_float(m)) * r.rstd) : 0;
      s = m > 0 ? __int_as_float((e + 127) << 23) : 1.f;
      const float inv = ldexpf(1.f, -e);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = zw[i] * r.factor * inv;
    }
    static_cast<uint2*>(p.out)[at] = make_uint2(codes_e4m3(y), codes_e4m3(y + 4));
    if ((threadIdx.x & 15) == 0) p.scale[at >> 4] = s;
  } else {
    uint32_t q[2] = {0u, 0u};
    if (!r.bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = r.wide ? __double2int_rn(static_cast<double>(zw[i]) * r.factor_wide) : __float2int_rn(zw[i] * r.factor);
        q[i >> 2] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (i & 3));
      }
    }
    static_cast<uint2*>(p.out)[at] = make_uint2(q[0], q[1]);
  }
}

// z of vector v of a row (and its store); `again`: the second pass of a long row, where
// the sum was stored already (over the residual, it may be) and is read back.
MOE_DEVINL void load_z(const NormParams& p, long long at, float (&z)[8], bool again) {
  if (again && p.res_out != nullptr) {
    unpack8(p.res_out[at], z);
    return;
  }
  unpack8(p.x[at], z);
  if (p.res != nullptr) {
    float r[8];
    unpack8(p.res[at], r);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += r[i];
    const uint4 packed = pack8(z);
    if (p.res_out != nullptr) p.res_out[at] = packed;
    unpack8(packed, z);
  }
}

// One block per row.  VPT > 0: thread t holds vectors t, t + blockDim, ... (VPT of them) in
// registers; VPT == 0 (rows of more than 32768 channels): two passes over the row.
template <int FMT, int VPT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ double sh_ss[1][32];
  __shared__ uint32_t sh_amax[1][32];
  const long long row = blockIdx.x;
  const long long base = row * p.nvec;
  double ss = 0.0;
  uint32_t amax = 0;
  constexpr int HELD = VPT > 0 ? VPT : 1;
  float zw[HELD][8];
  auto take = [&](int v, float (&o)[8]) {
    float z[8], w[8];
    load_z(p, base + v, z, false);
    unpack8(__ldg(p.w + v), w);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s = fmaf(z[i], z[i], s);
      o[i] = z[i] * w[i];
      if (FMT == NORM_INT8) amax = max(amax, abs_bits(o[i]));
    }
    ss += static_cast<double>(s);
  };
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < p.nvec) take(v, zw[i]);
    }
  } else {
    for (int v = threadIdx.x; v < p.nvec; v += blockDim.x) take(v, zw[0]);
  }
  block_reduce(ss, amax, sh_ss, sh_amax, 0);
  const RowScale r = row_scale<FMT>(ss, amax, p, row);
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < p.nvec) store_vec<FMT>(zw[i], r, p, row, v);
    }
  } else {
    for (int v = threadIdx.x; v < p.nvec; v += blockDim.x) {
      float z[8], w[8], o[8];
      load_z(p, base + v, z, true);
      unpack8(__ldg(p.w + v), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = z[i] * w[i];
      store_vec<FMT>(o, r, p, row, v);
    }
  }
}

template <int FMT>
cudaError_t launch_fmt(const NormParams& p, int T, cudaStream_t st) {
  // threads: whole warps, as few as hold the row at VPT vectors each
  const int warps = (p.nvec + 31) / 32;
  auto threads = [&](int vpt) { return 32 * ((warps + vpt - 1) / vpt); };
  if (p.nvec <= 1024 && T <= 4 * num_sms()) return launch_k(norm_kernel<FMT, 1>, T, threads(1), 0, st, p);
  if (p.nvec <= 4096) return launch_k(norm_kernel<FMT, 4>, T, threads(4), 0, st, p);
  return launch_k(norm_kernel<FMT, 0>, T, 1024, 0, st, p);
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
