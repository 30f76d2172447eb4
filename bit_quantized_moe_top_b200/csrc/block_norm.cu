// Row-wise operators around a block: the norms before and after it fused with
// gate, residual scale and the combination of expert rows, and the per-row
// 8-bit quantiser.
//
// Both hold a whole row in registers (fp32), so each input byte is read once
// and each output byte written once; they are bound by HBM at many rows and by
// the chain load -> reduce -> reduce -> store at few.
#include "kernels.h"
#include "ops.cuh"

namespace moeq {
namespace {

// Sum over the blockDim.x threads of a row (blockDim.x a multiple of 32).
// Every thread of the block takes part.
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float* r = red + threadIdx.y * 32;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < nw; ++i) s += r[i];
  return s;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  uint32_t* r = red + threadIdx.y * 32;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t s = 0;
  for (int i = 0; i < nw; ++i) s = max(s, r[i]);
  return s;
}

// One row per threadIdx.y; element (v * blockDim.x + threadIdx.x) * VEC + i in
// register v * VEC + i.
template <typename T, typename RT, int VEC, int NV>
__global__ void block_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][256];
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = t < a.T;
  const int tx = threadIdx.x, nx = blockDim.x;
  float b[NV * VEC];
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) b[i] = 0.f;
  if (live && a.y) {
    const T* y = static_cast<const T*>(a.y);
    if (a.k == 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (v * nx + tx) * VEC;
        if (e < a.K) load_vec<T, VEC>(y + t * a.ldy + e, b + v * VEC);
      }
    } else {
      for (int j = 0; j < a.k; ++j) {
        const int p = a.inv[t * a.k + j];
        if (p < 0 || p >= a.rows) continue;
        const float w = a.pw[t * a.k + j];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = (v * nx + tx) * VEC;
          if (e >= a.K) continue;
          float f[VEC];
          load_vec<T, VEC>(y + (long long)p * a.ldy + e, f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) b[v * VEC + i] += w * f[i];
        }
      }
    }
  }
  if (a.w_post) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) ss += b[i] * b[i];
    const float inv = 1.f / sqrtf(row_sum(ss, red[0]) / a.K + a.eps);
    if (live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (v * nx + tx) * VEC;
        if (e >= a.K) continue;
        float w[VEC];
        load_vec<T, VEC>(static_cast<const T*>(a.w_post) + e, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) b[v * VEC + i] *= inv * (a.w_off + w[i]);
      }
    }
  }
  if (live) {
    const T* gate = static_cast<const T*>(a.gate);
    float gt = 1.f;
    if (gate && a.gate_c == 0) {
      gt = to_f32<T>(gate[t * a.gate_t]);
      if (a.gate_sig) gt = 1.f / (1.f + expf(-gt));
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * nx + tx) * VEC;
      if (e >= a.K) continue;
      float* bv = b + v * VEC;
      if (gate && a.gate_c != 0) {
        float g[VEC];
        load_vec<T, VEC>(gate + t * a.gate_t + e, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) bv[i] *= a.br_scale * (a.gate_sig ? 1.f / (1.f + expf(-g[i])) : g[i]);
      } else if (a.y) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) bv[i] *= a.br_scale * gt;
      }
      if (a.res) {
        float r[VEC];
        load_vec<RT, VEC>(static_cast<const RT*>(a.res) + t * a.ldr + e, r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) bv[i] += a.res_scale * r[i];
      }
    }
  }
  float inv = 0.f;
  if (a.w_pre) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) ss += b[i] * b[i];
    inv = 1.f / sqrtf(row_sum(ss, red[1]) / a.K + a.eps);
  }
  if (!live) return;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * nx + tx) * VEC;
    if (e >= a.K) continue;
    float* bv = b + v * VEC;
    if (a.r_out) store_vec<RT, VEC>(static_cast<RT*>(a.r_out) + t * a.ldro + e, bv);
    if (a.w_pre) {
      float w[VEC];
      load_vec<T, VEC>(static_cast<const T*>(a.w_pre) + e, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) bv[i] *= inv * (a.w_off + w[i]);
      store_vec<T, VEC>(static_cast<T*>(a.h) + t * a.ldh + e, bv);
    }
  }
}

// codes = round(127 x / max|x|) by the quotient itself: 127 x is exact in fp32
// for 16-bit x, and a quotient that is not a half-integer lies at least 2^-12
// from one (its denominator has at most 11 significant bits), so the rounded
// fp32 quotient rounds to the same whole number as the exact one.
template <typename T, int VEC, int NV>
__global__ void quantize_rows_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t red[256];
  const long long r = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = r < a.rows;
  const int tx = threadIdx.x, nx = blockDim.x;
  long long s = live ? (a.src ? a.src[r] : r) : -1;
  const bool have = s >= 0 && s < a.x_rows;
  float b[NV * VEC];
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) b[i] = 0.f;
  if (have) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * nx + tx) * VEC;
      if (e < a.K) load_vec<T, VEC>(static_cast<const T*>(a.x) + s * a.ldx + e, b + v * VEC);
    }
  }
  uint32_t m = 0;  // the bits of |x| order as |x| does, with NaN above infinity
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) m = max(m, __float_as_uint(b[i]) & 0x7fffffffu);
  m = row_max(m, red);
  if (!live) return;
  const bool finite = m < 0x7f800000u;
  const float top = __uint_as_float(m);
  if (tx == 0) a.s[r] = finite ? __fdiv_rn(top, 127.f) : __uint_as_float(0x7fc00000u);
  const bool zero = m == 0 || !finite;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * nx + tx) * VEC;
    if (e >= a.K) continue;
    uint32_t c[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      c[i] = zero ? 0u : (uint32_t)__float2int_rn(__fdiv_rn(127.f * b[v * VEC + i], top)) & 0xffu;
    if constexpr (VEC == 1) {
      a.q[r * a.ldq + e] = (signed char)c[0];
    } else {
      *reinterpret_cast<uint2*>(a.q + r * a.ldq + e) =
          make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    }
  }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// threads per row, rows per block and grid of a row-wise kernel with NV
// vectors of VEC elements per thread
struct RowShape {
  dim3 grid, block;
};
RowShape row_shape(long long rows, int K, int VEC, int NV) {
  const int nvec = (K + VEC - 1) / VEC;
  const int tx = ((nvec + NV - 1) / NV + 31) / 32 * 32;
  const int ty = tx < 128 ? 128 / tx : 1;
  return {dim3((unsigned)((rows + ty - 1) / ty)), dim3(tx, ty)};
}

template <typename T, typename RT>
cudaError_t norm_typed(const NormArgs& a, bool vec, cudaStream_t st) {
  auto go = [&](auto kern, int VEC, int NV) {
    const RowShape s = row_shape(a.T, a.K, VEC, NV);
    return launch_kernel(kern, s.grid, s.block, 0, st, false, a);
  };
  if (!vec) return a.K <= 2048 ? go(block_norm_kernel<T, RT, 1, 4>, 1, 4) : go(block_norm_kernel<T, RT, 1, 32>, 1, 32);
  if (a.K <= 2048) return go(block_norm_kernel<T, RT, 8, 1>, 8, 1);
  if (a.K <= 4096) return go(block_norm_kernel<T, RT, 8, 2>, 8, 2);
  return go(block_norm_kernel<T, RT, 8, 4>, 8, 4);
}

template <typename T>
cudaError_t quant_typed(const QuantArgs& a, bool vec, cudaStream_t st) {
  auto go = [&](auto kern, int VEC, int NV) {
    const RowShape s = row_shape(a.rows, a.K, VEC, NV);
    return launch_kernel(kern, s.grid, s.block, 0, st, false, a);
  };
  if (!vec) return a.K <= 2048 ? go(quantize_rows_kernel<T, 1, 4>, 1, 4) : go(quantize_rows_kernel<T, 1, 32>, 1, 32);
  if (a.K <= 2048) return go(quantize_rows_kernel<T, 8, 1>, 8, 1);
  if (a.K <= 4096) return go(quantize_rows_kernel<T, 8, 2>, 8, 2);
  return go(quantize_rows_kernel<T, 8, 4>, 8, 4);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int dtype, int res_dtype, cudaStream_t st) {
  // 16-byte accesses need every row of every tensor to start at such a boundary
  const int rmul = res_dtype == DT_FP32 ? 4 : 8;
  const bool vec = a.K % 8 == 0 && aligned(a.y, 16) && aligned(a.w_post, 16) && aligned(a.w_pre, 16) &&
                   aligned(a.res, 16) && aligned(a.r_out, 16) && aligned(a.h, 16) && a.ldy % 8 == 0 &&
                   a.ldr % rmul == 0 && a.ldro % rmul == 0 && a.ldh % 8 == 0 &&
                   (!a.gate || a.gate_c == 0 || (aligned(a.gate, 16) && a.gate_t % 8 == 0));
  if (dtype == DT_BF16)
    return res_dtype == DT_FP32 ? norm_typed<__nv_bfloat16, float>(a, vec, st)
                                : norm_typed<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
  return res_dtype == DT_FP32 ? norm_typed<__half, float>(a, vec, st) : norm_typed<__half, __half>(a, vec, st);
}

cudaError_t launch_quantize_rows(const QuantArgs& a, int dtype, cudaStream_t st) {
  const bool vec = a.K % 8 == 0 && aligned(a.x, 16) && a.ldx % 8 == 0 && aligned(a.q, 8) && a.ldq % 8 == 0;
  return dtype == DT_BF16 ? quant_typed<__nv_bfloat16>(a, vec, st) : quant_typed<__half>(a, vec, st);
}

}  // namespace moeq
