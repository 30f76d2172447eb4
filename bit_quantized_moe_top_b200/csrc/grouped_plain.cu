// Products grouped by expert with ordinary loads: any pointer, stride, K and N.
// y[r, n] = xs[r] ws[e, n] sum_k x[r, k] w[e, n, k], 64 x 64 output tiles,
// operands staged as 32-bit values in shared memory, 4 x 4 outputs per thread.
#include "kernels.h"
#include "ops.cuh"

namespace moeq {
namespace {

constexpr int kTile = 64, kStep = 16, kThreadsPlain = 256;

struct RowTiles {
  int w;
  __device__ int operator()(int n) const { return (n + w - 1) / w; }
};

template <typename TI>
struct Acc {
  using type = float;
};
template <>
struct Acc<signed char> {
  using type = int;
};
template <typename TI>
__device__ __forceinline__ typename Acc<TI>::type widen(TI v) {
  if constexpr (sizeof(TI) == 1) return (int)v;
  else return to_f32<TI>(v);
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreadsPlain) grouped_plain_kernel(const __grid_constant__ GroupedArgs a) {
  using A = typename Acc<TI>::type;
  __shared__ GroupTable g;
  __shared__ A xt[kStep][kTile + 4], wt[kStep][kTile + 4];
  build_group_table(g, a.offsets, a.rows, a.E, RowTiles{kTile});
  const int t = threadIdx.x, tr = t / 16 * 4, tn = t % 16 * 4;
  const int nf = (a.N + kTile - 1) / kTile;
  const long long total = (long long)g.first[a.E] * nf;
  for (long long tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const int rt = (int)(tile / nf), n0 = (int)(tile % nf) * kTile;
    const int e = find_group(g, a.E, rt);
    const int in = (rt - g.first[e]) * kTile;          // first row of the tile within the group
    const long long r0 = (long long)g.begin[e] + in;
    const int live = min(kTile, g.rows[e] - in);
    const TI* x = static_cast<const TI*>(a.x) + r0 * a.ldx;
    const TI* w = static_cast<const TI*>(a.w) + e * a.ldwe;
    A acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
      for (int i = t; i < kTile * kStep; i += kThreadsPlain) {
        const int r = i / kStep, k = i % kStep;
        const bool in_k = k0 + k < a.K;
        xt[k][r] = in_k && r < live ? widen<TI>(x[r * a.ldx + k0 + k]) : A(0);
        wt[k][r] = in_k && n0 + r < a.N ? widen<TI>(w[(n0 + r) * a.ldw + k0 + k]) : A(0);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        A xv[4], wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xv[i] = xt[k][tr + i];
          wv[i] = wt[k][tn + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += xv[i] * wv[j];
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (tr + i >= live) continue;
      const long long r = r0 + tr + i;
      TO* y = static_cast<TO*>(a.y) + r * a.ldy + n0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (n0 + tn + j >= a.N) continue;
        float v = (float)acc[i][j];
        if constexpr (sizeof(TI) == 1) v *= a.xs[r] * a.ws[(long long)e * a.N + n0 + tn + j];
        y[tn + j] = from_f32<TO>(v);
      }
    }
  }
}

template <typename TI, typename TO>
cudaError_t launch_plain(const GroupedArgs& a, cudaStream_t st) {
  const long long tiles = ((long long)(a.rows + kTile - 1) / kTile + a.E) * ((a.N + kTile - 1) / kTile);
  const int grid = (int)(tiles < 8LL * device_sms() ? tiles : 8LL * device_sms());
  return launch_kernel(grouped_plain_kernel<TI, TO>, dim3(grid), dim3(kThreadsPlain), 0, st, false, a);
}
template <typename TI>
cudaError_t launch_plain_out(const GroupedArgs& a, int y_dtype, cudaStream_t st) {
  if (y_dtype == DT_BF16) return launch_plain<TI, __nv_bfloat16>(a, st);
  if (y_dtype == DT_FP16) return launch_plain<TI, __half>(a, st);
  return launch_plain<TI, float>(a, st);
}

}  // namespace

cudaError_t launch_grouped_plain(const GroupedArgs& a, int op, int y_dtype, cudaStream_t st) {
  if (op == DT_BF16) return launch_plain_out<__nv_bfloat16>(a, y_dtype, st);
  if (op == DT_FP16) return launch_plain_out<__half>(a, y_dtype, st);
  return launch_plain_out<signed char>(a, y_dtype, st);
}

}  // namespace moeq
