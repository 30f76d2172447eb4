// Shared pieces of the stand-alone operators: launch arguments, conversions,
// row-wide reductions and the split of ragged expert groups into row tiles.
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"

namespace moeq {

constexpr int kMaxRowWidth = 16384;  // widest row the row-wise operators hold in registers

enum : int { DT_BF16 = 0, DT_FP16 = 1, DT_FP32 = 2 };

struct NormArgs {
  int T, K;
  const void* y;          // branch rows
  long long ldy;
  int rows, k;
  const int* inv;         // [T, k]
  const float* pw;        // [T, k]
  const void* w_post;
  const void* gate;
  long long gate_t;
  int gate_c, gate_sig;
  const void* res;
  long long ldr;
  float res_scale, br_scale;
  const void* w_pre;
  float eps, w_off, inv_K;
  void* r_out;
  long long ldro;
  void* h;
  long long ldh;
};

struct QuantArgs {
  const void* x;
  long long ldx;
  int x_rows;
  const int* src;
  int rows, K;
  signed char* q;
  long long ldq;
  float* s;
};

// y[r, n] = scale * sum_k x[r, k] w[e(r), n, k]; the scales are null for 16-bit operands
struct GroupedArgs {
  const void* x;
  long long ldx;
  const void* w;
  long long ldw, ldwe;
  const float* xs;        // [rows]
  const float* ws;        // [E, N]
  const int* offsets;     // [E + 1] or null (one group of all rows)
  int rows, E, K, N;
  void* y;
  long long ldy;
  unsigned long long wait_ns;
};

cudaError_t launch_block_norm(const NormArgs& a, int dtype, int res_dtype, cudaStream_t st);
cudaError_t launch_quantize_rows(const QuantArgs& a, int dtype, cudaStream_t st);
// operand type: DT_BF16, DT_FP16, or kOpInt8
constexpr int kOpInt8 = 3;
bool grouped_tc_fits(const GroupedArgs& a, int op);
cudaError_t launch_grouped_tc(const GroupedArgs& a, int op, int y_dtype, cudaStream_t st);
// for the calls that do not fit
cudaError_t launch_grouped_loads(const GroupedArgs& a, int op, int y_dtype, cudaStream_t st);
// how many CTAs of the products have given up a wait on the current device, read once the stream is idle
cudaError_t read_op_timeouts(unsigned* out, cudaStream_t st);

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// two values packed into one 32-bit word, lo in the low half
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) { return pack_half2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// 8 elements to a 16-byte boundary
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                              pack2<T>(v[6], v[7]));
  }
}

// The row tiles of all experts in expert order, built by one block (at least
// kMaxExperts threads): first[e] = tiles before expert e, begin[e] / rows[e]
// its rows. Offsets are read as their running maximum clamped to [0, rows], so
// that no content of the array leads outside x or y. TileFn(rows) = tiles of
// a group.
struct GroupTable {
  int first[kMaxExperts + 1];
  int begin[kMaxExperts];
  int rows[kMaxExperts];
  int scratch[2][kMaxExperts / 32];
};
template <typename TileFn>
__device__ __forceinline__ void build_group_table(GroupTable& g, const int* offsets, int rows, int E, TileFn tiles_of) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (!offsets) {  // one group of all rows
    if (t == 0) {
      g.begin[0] = 0;
      g.rows[0] = rows;
      g.first[0] = 0;
      g.first[1] = tiles_of(rows);
    }
    __syncthreads();
    return;
  }
  if (E <= 32) {  // one warp, without the passes between warps
    if (warp == 0) {
      int lo = 0, hi = 0;
      if (lane < E) {
        lo = min(max(offsets[lane], 0), rows);
        hi = min(max(offsets[lane + 1], 0), rows);
      }
      int m = max(lo, hi);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, o);
      }
      const int prev = __shfl_up_sync(0xffffffffu, m, 1);
      const int start = lane == 0 ? lo : max(lo, prev);
      const int n = lane < E ? m - start : 0;
      int s = n > 0 ? tiles_of(n) : 0;
      const int own = s;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
      }
      if (lane < E) {
        g.begin[lane] = start;
        g.rows[lane] = n;
        g.first[lane] = s - own;
        if (lane == E - 1) g.first[E] = s;
      }
    }
    __syncthreads();
    return;
  }
  int lo = 0, hi = 0;
  if (t < E) {
    lo = min(max(offsets[t], 0), rows);
    hi = min(max(offsets[t + 1], 0), rows);
  }
  // running maximum up to offsets[t + 1]; lo's is the neighbour's value
  int m = max(lo, hi);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, m, d);
    if (lane >= d) m = max(m, o);
  }
  if (t < kMaxExperts && lane == 31) g.scratch[0][warp] = m;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 32; ++w) {
    const int o = g.scratch[0][w];
    if (w < warp) before = max(before, o);
  }
  int prev = __shfl_up_sync(0xffffffffu, m, 1);
  prev = lane == 0 ? before : max(prev, before);
  m = max(m, before);
  const int start = max(lo, prev);
  const int n = t < E ? m - start : 0;
  int s = n > 0 ? tiles_of(n) : 0;
  const int own = s;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (t < kMaxExperts && lane == 31) g.scratch[1][warp] = s;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 32; ++w) {
    const int o = g.scratch[1][w];
    if (w < warp) base += o;
  }
  if (t < E) {
    g.begin[t] = start;
    g.rows[t] = n;
    g.first[t] = base + s - own;
    if (t == E - 1) g.first[E] = base + s;
  }
  __syncthreads();
}
// The expert whose tiles hold tile i (first[e] <= i < first[e + 1]): the last
// one that begins no later, counted by a whole warp, 8 experts a lane and then
// those one by one.
__device__ __forceinline__ int find_group(const GroupTable& g, int E, int i) {
  static_assert(kMaxExperts <= 256, "two steps of 32 and 8");
  const int lane = threadIdx.x & 31;
  int from = 0;
  if (E > 32) from = 8 * (__popc(__ballot_sync(0xffffffffu, lane * 8 < E && g.first[min(lane * 8, E)] <= i)) - 1);
  const int e = from + lane;
  return from + __popc(__ballot_sync(0xffffffffu, e < E && g.first[min(e, E)] <= i)) - 1;
}

}  // namespace moeq
