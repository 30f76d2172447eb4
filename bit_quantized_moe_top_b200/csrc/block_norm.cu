// Row-wise operators around a block: the norms before and after it fused with
// gate, residual scale and the combination of expert rows, and the per-row
// 8-bit quantiser.
//
// Both hold a whole row in registers (fp32), so each input byte is read once
// and each output byte written once; they are bound by HBM at many rows and by
// the chain load -> reduce -> reduce -> store at few. Next to the traffic it is
// the number of instructions per element that counts, so arithmetic goes in
// pairs of fp32 values (one instruction for two), and rows are split into 8
// elements per thread and vector even where no row starts at a 16-byte
// boundary. Measured, of HBM's 6.46 TB/s: norm of 16384 x 2048 95%, 8192 x 4096
// with two combined rows 83%; quantiser of 8192 x 4096 97%, 16384 x 14336 94%.
// Rows of more than 8192 elements take 110 to 124 registers a thread, so that one
// row at a time lives on an SM and HBM idles through its two reductions: norm of
// 4000 x 14336 67%. Rows at any alignment take two loads and a shift for every
// vector, the norms' weights among them, anew for each row: norm of 1027 x 2051
// 33%, 4096 x 9001 50%; quantiser of 8192 x 4095 60%, 4000 x 14335 60%.
#include "kernels.h"
#include "ops.cuh"

namespace moeq {
namespace {

// ---- two fp32 values per instruction
__device__ __forceinline__ uint64_t bits2(float2 v) { return *reinterpret_cast<uint64_t*>(&v); }
__device__ __forceinline__ float2 float2_of(uint64_t b) { return *reinterpret_cast<float2*>(&b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Sum (or maximum) over the blockDim.x threads of a row (blockDim.x a multiple
// of 32), in a fixed order. Every thread of the block takes part; red holds 32
// words per row.
__device__ __forceinline__ int warps_pow2() {
  const int nw = blockDim.x >> 5;
  return 1 << (32 - __clz(nw - 1));  // of the row's warps
}
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float* r = red + threadIdx.y * 32;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  const int P = warps_pow2(), i = threadIdx.x & (P - 1);
  v = i < nw ? r[i] : 0.f;
  for (int d = P >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  uint32_t* r = red + threadIdx.y * 32;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __reduce_max_sync(0xffffffffu, lane < nw ? r[lane] : 0u);
}

// Elements e .. e + 7 of a row as loaded; their conversion comes where they are
// used, so that a row's loads are all in flight together. Without SHIFT e is a
// multiple of 8 within the row and every row starts at a 16-byte boundary. With
// SHIFT neither holds (e may be negative or reach past K; absent elements read
// as zero): the 16 aligned bytes at e if it lies on a boundary, else the two
// aligned 16-byte pieces around it, shifted when used, and single elements
// where those pieces would leave the row.
template <typename T, bool SHIFT>
struct Vec8 {
  static constexpr int kWords = SHIFT || sizeof(T) == 4 ? 8 : 4;
  uint32_t w[kWords];
  int mode;  // 0: whole; 1: single elements; else the byte offset (even) within the pieces
  __device__ __forceinline__ void put(int i, uint4 u) {
    w[i] = u.x;
    w[i + 1] = u.y;
    w[i + 2] = u.z;
    w[i + 3] = u.w;
  }
  __device__ __forceinline__ void zero() {
    mode = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* row, int e, int K) {
    const T* p = row + e;
    if constexpr (!SHIFT) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) put(i, reinterpret_cast<const uint4*>(p)[i / 4]);
    } else {
      const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15);
      const int first = e - mis / (int)sizeof(T);  // of the pieces
      if (mis == 0 && e >= 0 && e + 8 <= K) {
        mode = 0;
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); i += 4) put(i, reinterpret_cast<const uint4*>(p)[i / 4]);
      } else if (sizeof(T) == 2 && first >= 0 && first + 16 <= K) {
        mode = mis;
        const uint4* q = reinterpret_cast<const uint4*>(row + first);
        put(0, q[0]);
        put(4, q[1]);
      } else {
        mode = 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = 0;
          if (e + i >= 0 && e + i < K) {
            if constexpr (sizeof(T) == 2) w[i] = reinterpret_cast<const uint16_t*>(p)[i];
            else w[i] = reinterpret_cast<const uint32_t*>(p)[i];
          }
        }
      }
    }
  }
  // 16-bit elements as pairs
  __device__ __forceinline__ void words(uint32_t (&o)[4]) const {
    if constexpr (SHIFT) {
      if (mode > 1) {
        uint32_t s[7], r[5];
        const bool one = mode & 4, two = mode & 8;
#pragma unroll
        for (int i = 0; i < 7; ++i) s[i] = one ? w[i + 1] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) r[i] = two ? s[i + 2] : s[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(r[i], r[i + 1], (mode & 2) * 8);
        return;
      }
      if (mode == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = prmt(w[2 * i], w[2 * i + 1], 0x5410u);
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = w[i];
  }
  __device__ __forceinline__ void floats(float2 (&f)[4]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
      uint32_t o[4];
      words(o);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = unpack2<T>(o[i]);
    }
  }
};
template <typename T, bool SHIFT>
__device__ __forceinline__ void store8(T* row, int e, int K, const float2 (&f)[4]) {
  T* p = row + e;
  if (!SHIFT || (e >= 0 && e + 8 <= K && (reinterpret_cast<uintptr_t>(p) & 15) == 0)) {
    store_vec<T>(p, reinterpret_cast<const float*>(f));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i >= 0 && e + i < K) p[i] = from_f32<T>(i & 1 ? f[i / 2].y : f[i / 2].x);
  }
}
// Elements by which a row's vectors are moved so that those of its output start
// at aligned addresses (8 elements of ES bytes)
template <int ES>
__device__ __forceinline__ int row_shift(const void* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) / ES) & 7;
}

// How a call's rows lie: kFull, aligned and with a vector for every thread and
// nothing over (no bounds to look at: norm of 16384 x 2048 46 -> 44 us,
// quantiser of 8192 x 4096 18 -> 16 us); kEven, aligned; kShift, any.
enum : int { kFull, kEven, kShift };

// One row per threadIdx.y, NV vectors of 8 elements per thread. Every load that
// does not wait for a reduction is issued before the first one, so that a row
// waits for HBM once; the weights, which every row reads, come from the caches.
// (Shifted rows of more than 8192 elements go two vectors at a time and read
// the residual late instead, since their loads take twice the registers, and
// keep to 56 registers, so that two blocks share an SM and one's loads run
// under the other's reductions: 4096 rows of 9001 with two combined rows 168
// -> 133 us in spite of the spills.)
template <typename T, typename RT, int NV, int FORM>
__global__ void __launch_bounds__(NV == 1 ? 1024 : NV == 4 && FORM == kShift ? 544 : 512, (NV == 4 && FORM == kShift) || (NV == 2 && FORM != kShift) ? 2 : 1)
    block_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr bool SHIFT = FORM == kShift;
  __shared__ float red[2][4 * 32];
  // Combined rows in flight, as many as the registers hold. One, two, four, eight,
  // us: 128 x 7168 with eight rows (NV = 1) 10.0, 8.5, 7.8, 8.2; 8192 x 4096 with
  // two (NV = 2) 69, 62, 74; shifted 1027 x 2051 with eight 21.7, 23.0, 40.
  constexpr int kAhead = SHIFT ? 1 : NV == 1 ? 4 : 2;
  // Vectors of a row in flight: all, but half of the four of shifted rows, whose
  // loads take twice the registers (4096 x 9001 with two rows 133 us, all four 258).
  constexpr int kGroup = SHIFT && NV == 4 ? 2 : NV;
  constexpr bool kLate = kGroup < NV;
  pdl_wait();
  pdl_trigger();
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = FORM == kFull || t < a.T;
  const int tx = threadIdx.x, nx = blockDim.x, K = a.K;
  T* h = static_cast<T*>(a.h) + t * a.ldh;
  RT* r_out = static_cast<RT*>(a.r_out) + t * a.ldro;
  const int shift = !SHIFT ? 0 : a.h ? row_shift<sizeof(T)>(h) : row_shift<sizeof(RT)>(r_out);
  auto at = [&](int v) { return (v * nx + tx) * 8 - shift; };
  auto in = [&](int v) { return FORM == kFull || (live && at(v) < K); };
  float2 b[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) b[v][i] = both(0.f);
  Vec8<RT, SHIFT> rr[NV];
  const T* y = static_cast<const T*>(a.y);
  const T* gate = static_cast<const T*>(a.gate);
  const T* w_post = static_cast<const T*>(a.w_post);
  const T* w_pre = static_cast<const T*>(a.w_pre);
  const bool gate_row = gate && a.gate_c != 0;
  auto load_residual = [&] {
    if (!a.res) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in(v)) rr[v].load(static_cast<const RT*>(a.res) + t * a.ldr, at(v), K);
  };
  if (a.k == 0) {
#pragma unroll
    for (int g = 0; g < NV; g += kGroup) {
      Vec8<T, SHIFT> yr[kGroup];
      if (y) {
#pragma unroll
        for (int v = 0; v < kGroup; ++v)
          if (in(g + v)) yr[v].load(y + t * a.ldy, at(g + v), K);
      }
      if (!kLate) load_residual();
      if (y) {
#pragma unroll
        for (int v = 0; v < kGroup; ++v)
          if (in(g + v)) yr[v].floats(b[g + v]);
      }
    }
  } else {
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
      int p[kAhead];
      float w[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool have = live && j0 + j < a.k;
        p[j] = have ? a.inv[t * a.k + j0 + j] : -1;
        w[j] = have ? a.pw[t * a.k + j0 + j] : 0.f;
        if (p[j] >= a.rows) p[j] = -1;
      }
#pragma unroll
      for (int g = 0; g < NV; g += kGroup) {
        Vec8<T, SHIFT> yr[kAhead][kGroup];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int v = 0; v < kGroup; ++v)
            if (p[j] >= 0 && in(g + v)) yr[j][v].load(y + (long long)p[j] * a.ldy, at(g + v), K);
        if (!kLate && j0 == 0) load_residual();
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int v = 0; v < kGroup; ++v)
            if (p[j] >= 0 && in(g + v)) {
              float2 f[4];
              yr[j][v].floats(f);
#pragma unroll
              for (int i = 0; i < 4; ++i) b[g + v][i] = fma2(both(w[j]), f[i], b[g + v][i]);
            }
      }
    }
  }
  float gt = a.br_scale;
  if (live && gate && !gate_row) {
    gt = to_f32<T>(gate[t * a.gate_t]);
    gt = a.br_scale * (a.gate_sig ? 1.f / (1.f + expf(-gt)) : gt);
  }
  auto sum_of_squares = [&] {
    float2 s = both(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(b[v][i], b[v][i], s);
    return s.x + s.y;
  };
  // b *= s (w_off + w)
  auto scale_by = [&](const T* w, float s) {
    const float2 s2 = both(s), o2 = both(s * a.w_off);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in(v)) {
        Vec8<T, SHIFT> wv;
        wv.load(w, at(v), K);
        float2 f[4];
        wv.floats(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[v][i] = mul2(b[v][i], fma2(f[i], s2, o2));
      }
  };
  if (w_post) {
    const float inv = rsqrtf(row_sum(sum_of_squares(), red[0]) * a.inv_K + a.eps);
    scale_by(w_post, gate_row ? inv : inv * gt);
    if (!gate_row) gt = 1.f;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!in(v)) continue;
    if (gate_row) {
      Vec8<T, SHIFT> g;
      g.load(gate + t * a.gate_t, at(v), K);
      float2 f[4];
      g.floats(f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (a.gate_sig) {
          f[i].x = __fdividef(1.f, 1.f + expf(-f[i].x));
          f[i].y = __fdividef(1.f, 1.f + expf(-f[i].y));
        }
        b[v][i] = mul2(b[v][i], mul2(f[i], both(gt)));
      }
    } else if (!w_post) {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[v][i] = mul2(b[v][i], both(gt));
    }
    if (a.res) {
      if (kLate) rr[v].load(static_cast<const RT*>(a.res) + t * a.ldr, at(v), K);
      float2 f[4];
      rr[v].floats(f);
#pragma unroll
      for (int i = 0; i < 4; ++i) b[v][i] = fma2(both(a.res_scale), f[i], b[v][i]);
    }
    if (a.r_out) store8<RT, SHIFT>(r_out, at(v), K, b[v]);
  }
  if (!w_pre) return;
  scale_by(w_pre, rsqrtf(row_sum(sum_of_squares(), red[1]) * a.inv_K + a.eps));
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (in(v)) store8<T, SHIFT>(h, at(v), K, b[v]);
}

// One code: 127 x / top rounded to the nearest whole number, halves to even, of
// the exact quotient and without dividing by it. With x = X 2^a and
// top = Y 2^(a + s), X and Y whole numbers of at most 11 bits, the quotient
// 127 X / (Y 2^s) is below 2^(8 - s), and one that is not a half-integer lies
// at least 1 / (2 Y 2^s) > 2^-(12 + s) from one. The two products with
// r = 127 / top, made larger and smaller by 2^-21 of itself, lie on either side
// of the quotient and within 2^-(13 + s) + 2^-(15 + s) of it: they round to one
// number unless the quotient is a half-integer, and then to its two neighbours,
// of which the even one is taken. The rounding is an addition of 1.5 * 2^23,
// which leaves the code in the low byte.
constexpr float kRoundBias = 12582912.f;
constexpr float kTiny = 5.4210108624275222e-20f;  // 2^-64; rows below it are scaled by its inverse, so that r is finite

template <typename T, int NV, int FORM>
__global__ void __launch_bounds__(NV == 1 ? 1024 : NV == 4 && FORM == kShift ? 544 : 512)
    quantize_rows_kernel(const __grid_constant__ QuantArgs a) {
  constexpr bool SHIFT = FORM == kShift;
  __shared__ uint32_t red[4 * 32];
  pdl_wait();
  pdl_trigger();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = FORM == kFull || row < a.rows;
  const int tx = threadIdx.x, nx = blockDim.x, K = a.K;
  const long long s = live ? (a.src ? a.src[row] : row) : -1;
  const bool have = s >= 0 && s < a.x_rows;
  signed char* q = a.q + row * a.ldq;
  const int shift = SHIFT ? row_shift<1>(q) : 0;
  auto at = [&](int v) { return (v * nx + tx) * 8 - shift; };
  Vec8<T, SHIFT> x[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (have && (FORM == kFull || at(v) < K)) x[v].load(static_cast<const T*>(a.x) + s * a.ldx, at(v), K);
    else x[v].zero();
  }
  // the bits of |x| order as |x| does, with NaN above infinity
  uint32_t w[NV][4], m = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    x[v].words(w[v]);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[v][i] & 0x7fff7fffu);
  }
  m = row_max(max(m & 0xffffu, m >> 16), red);
  if (!live) return;
  const uint16_t bits = (uint16_t)m;
  const float top = to_f32<T>(*reinterpret_cast<const T*>(&bits));
  const bool finite = top < __uint_as_float(0x7f800000u);
  if (tx == 0) a.s[row] = finite ? __fdiv_rn(top, 127.f) : __uint_as_float(0x7fc00000u);
  const bool tiny = top < kTiny;
  const uint32_t keep = m == 0 || !finite ? 0u : ~0u;
  const float r = keep ? __fdiv_rn(127.f, tiny ? top * (1.f / kTiny) : top) : 0.f;
  const float2 hi = both(r * (1.f + 0x1p-21f)), lo = both(r * (1.f - 0x1p-21f)), bias = both(kRoundBias);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = at(v);
    if (FORM != kFull && e >= K) continue;
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = unpack2<T>(w[v][i]);
    if (tiny) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], both(1.f / kTiny));
    }
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      auto pack = [&](float2 scale) {
        const float2 t = fma2(f[2 * i], scale, bias), u = fma2(f[2 * i + 1], scale, bias);
        return prmt(prmt(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040u),
                    prmt(__float_as_uint(u.x), __float_as_uint(u.y), 0x0040u), 0x5410u);
      };
      const uint32_t a4 = pack(hi), b4 = pack(lo), odd = (a4 & 0x01010101u) * 0xffu;
      c[i] = ((a4 & ~odd) | (b4 & odd)) & keep;
    }
    if (!SHIFT || (e >= 0 && e + 8 <= K)) {
      *reinterpret_cast<uint2*>(q + e) = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i >= 0 && e + i < K) q[e + i] = (signed char)(c[i >> 2] >> (8 * (i & 3)) & 0xffu);
    }
  }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// threads per row, rows per block and grid of a row-wise kernel whose rows are
// nvec vectors, NV per thread
struct RowShape {
  dim3 grid, block;
};
RowShape row_shape(long long rows, int nvec, int NV) {
  const int tx = ((nvec + NV - 1) / NV + 31) / 32 * 32;
  const int ty = tx < 128 ? 128 / tx : 1;
  return {dim3((unsigned)((rows + ty - 1) / ty)), dim3(tx, ty)};
}

int row_vectors(int K, bool shift) { return shift ? (K + 14) / 8 : K / 8; }

// Vectors per thread. Few rows: as many threads per row as can be used (a
// shorter chain). Many rows: fewer (less synchronisation per byte), as far as
// the registers leave enough rows on an SM at a time. One, two or four vectors,
// us: norm with two combined rows, 8192 x 4096 99, 62, 64; 16384 x 1024 43, 30,
// 31; without, 16384 x 256 7.8, 10.4, 16; quantiser, one or four, 8192 x 4096
// 27, 16; 16384 x 512 9.4, 6.9; 30000 x 256 8.4, 9.5. Shifted rows of the norm
// take one longer: 1027 x 2051 9.5, 15.
int norm_vectors(long long rows, int nvec, bool shift) {
  if (rows <= 2LL * device_sms()) return nvec <= 1024 ? 1 : 4;
  return nvec <= (shift ? 512 : 32) ? 1 : nvec <= 1024 ? 2 : 4;
}
int quant_vectors(long long rows, int nvec) {
  if (rows <= 2LL * device_sms()) return nvec <= 1024 ? 1 : 4;
  return nvec < 64 ? 1 : 4;
}

bool full_rows(const RowShape& s, long long rows, int nvec, int NV) {
  return rows % s.block.y == 0 && (int)s.block.x * NV == nvec;
}

template <typename T, typename RT, bool SHIFT>
cudaError_t norm_typed(const NormArgs& a, cudaStream_t st) {
  const int nvec = row_vectors(a.K, SHIFT), NV = norm_vectors(a.T, nvec, SHIFT);
  const RowShape s = row_shape(a.T, nvec, NV);
  auto go = [&](auto kern) { return launch_kernel(kern, s.grid, s.block, 0, st, true, a); };
  constexpr int kBounded = SHIFT ? kShift : kEven;
  if constexpr (!SHIFT) {
    if (full_rows(s, a.T, nvec, NV)) {
      if (NV == 1) return go(block_norm_kernel<T, RT, 1, kFull>);
      if (NV == 2) return go(block_norm_kernel<T, RT, 2, kFull>);
      return go(block_norm_kernel<T, RT, 4, kFull>);
    }
  }
  if (NV == 1) return go(block_norm_kernel<T, RT, 1, kBounded>);
  if (NV == 2) return go(block_norm_kernel<T, RT, 2, kBounded>);
  return go(block_norm_kernel<T, RT, 4, kBounded>);
}

template <typename T, bool SHIFT>
cudaError_t quant_typed(const QuantArgs& a, cudaStream_t st) {
  const int nvec = row_vectors(a.K, SHIFT), NV = quant_vectors(a.rows, nvec);
  const RowShape s = row_shape(a.rows, nvec, NV);
  auto go = [&](auto kern) { return launch_kernel(kern, s.grid, s.block, 0, st, true, a); };
  constexpr int kBounded = SHIFT ? kShift : kEven;
  if constexpr (!SHIFT) {
    if (full_rows(s, a.rows, nvec, NV)) return go(NV == 1 ? quantize_rows_kernel<T, 1, kFull> : quantize_rows_kernel<T, 4, kFull>);
  }
  return go(NV == 1 ? quantize_rows_kernel<T, 1, kBounded> : quantize_rows_kernel<T, 4, kBounded>);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int dtype, int res_dtype, cudaStream_t st) {
  // every row of every tensor starts at a 16-byte boundary
  const int rmul = res_dtype == DT_FP32 ? 4 : 8;
  const bool even = a.K % 8 == 0 && aligned(a.y, 16) && aligned(a.w_post, 16) && aligned(a.w_pre, 16) &&
                    aligned(a.res, 16) && aligned(a.r_out, 16) && aligned(a.h, 16) && a.ldy % 8 == 0 &&
                    a.ldr % rmul == 0 && a.ldro % rmul == 0 && a.ldh % 8 == 0 &&
                    (!a.gate || a.gate_c == 0 || (aligned(a.gate, 16) && a.gate_t % 8 == 0));
  auto go = [&](auto t, auto rt) {
    using T = decltype(t);
    using RT = decltype(rt);
    return even ? norm_typed<T, RT, false>(a, st) : norm_typed<T, RT, true>(a, st);
  };
  if (dtype == DT_BF16)
    return res_dtype == DT_FP32 ? go(__nv_bfloat16{}, 0.f) : go(__nv_bfloat16{}, __nv_bfloat16{});
  return res_dtype == DT_FP32 ? go(__half{}, 0.f) : go(__half{}, __half{});
}

cudaError_t launch_quantize_rows(const QuantArgs& a, int dtype, cudaStream_t st) {
  const bool even = a.K % 8 == 0 && aligned(a.x, 16) && a.ldx % 8 == 0 && aligned(a.q, 8) && a.ldq % 8 == 0;
  if (dtype == DT_BF16) return even ? quant_typed<__nv_bfloat16, false>(a, st) : quant_typed<__nv_bfloat16, true>(a, st);
  return even ? quant_typed<__half, false>(a, st) : quant_typed<__half, true>(a, st);
}

}  // namespace moeq
