// C entry points of the stand-alone operators: argument checks and launches.
#include <atomic>
#include <cmath>

#include "../../include/moe_layer.h"
#include "kernels.h"
#include "ops.cuh"

using namespace moeq;

namespace {

std::atomic<unsigned long long> g_wait_ns{kDefaultWaitNs};

bool is16(int d) { return d == MOE_BF16 || d == MOE_FP16; }
bool is_out(int d) { return is16(d) || d == MOE_FP32; }

constexpr int kMaxExtent = 1 << 29;  // rows and N: coordinates stay within an int
constexpr int kMaxSum = 1 << 24;     // K: a tile's sums take far less than the limit of the waits for them

// whether a pointer lies at a multiple of its elements' size
bool at_elements(const void* p, int es) { return reinterpret_cast<uintptr_t>(p) % es == 0; }

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// checks shared by the two products
moe_status_t check_product(const void* x, long long ldx, const void* w, long long ldw, long long ldwe,
                           int es, const int* offsets, int rows, int E, int K, int N, const void* y, long long ldy,
                           int yd) {
  if (rows < 0 || E < 1 || K < 1 || N < 1 || !is_out(yd)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || rows > kMaxExtent || K > kMaxSum || N > kMaxExtent) return MOE_ERR_TOO_LARGE;
  if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
  if (ldx < 0 || ldw < 0 || ldwe < 0 || (rows > 1 && ldy < N)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !w || !y)) return MOE_ERR_INVALID_ARG;
  if (!at_elements(x, es) || !at_elements(w, es) || !at_elements(y, yd == MOE_FP32 ? 4 : 2) ||
      !at_elements(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// What each stream has been told of its device's count of timeouts. The count only
// grows and every stream keeps its own place in it, so that no caller takes
// another's timeout. A stream gets its place with its first product, at the
// highest count that anyone had read by then (which its calls cannot be part of);
// one without a place (it only replays graphs, or the table is full) starts at 0
// and may be told of timeouts before its time, never too few. Streams are known
// by their handles: asking CUDA for a stream's number ends a capture of it.
struct Told {
  std::atomic<unsigned long long> key{0};  // 0: free
  std::atomic<unsigned> count{0};
};
constexpr int kPlaces = 4096;
Told g_told[kPlaces];
constexpr int kMaxDevices = 64;
std::atomic<unsigned> g_read[kMaxDevices];  // highest count read

unsigned long long key_of(cudaStream_t st, int dev) {
  static std::atomic<unsigned long long> threads{0};
  static thread_local const unsigned long long thread = ++threads;
  unsigned long long id = (unsigned long long)reinterpret_cast<uintptr_t>(st);
  if (st == cudaStreamPerThread) id |= thread << 12;  // another stream in every thread; no other handle ends in its bits
  return id << 8 | (unsigned)(dev + 1);
}
// the stream's place, a new one if make; null if there is none
Told* place_of(cudaStream_t st, int dev, bool make, unsigned start) {
  const unsigned long long key = key_of(st, dev);
  for (int i = 0, h = (int)(key * 0x9E3779B97F4A7C15ull >> 52); i < kPlaces; ++i, h = (h + 1) % kPlaces) {
    unsigned long long k = g_told[h].key.load(std::memory_order_acquire);
    if (k == 0) {
      if (!make) return nullptr;
      if (g_told[h].key.compare_exchange_strong(k, key)) {
        g_told[h].count.store(start);
        return &g_told[h];
      }
    }
    if (k == key) return &g_told[h];
  }
  return nullptr;
}

moe_status_t run_product(GroupedArgs& a, int op, int y_dtype, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return MOE_ERR_CUDA;
  place_of(st, dev, true, g_read[dev].load());
  a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  return cuda_status(grouped_tc_fits(a, op) ? launch_grouped_tc(a, op, y_dtype, st)
                                            : launch_grouped_loads(a, op, y_dtype, st));
}

}  // namespace

extern "C" {

moe_status_t moe_block_norm(const moe_block_norm_t* p, void* cuda_stream) {
  if (!p || p->tokens < 0 || p->width < 1 || !is16(p->dtype) ||
      (p->residual_dtype != MOE_FP32 && p->residual_dtype != p->dtype))
    return MOE_ERR_INVALID_ARG;
  if (p->width > kMaxRowWidth) return MOE_ERR_TOO_LARGE;
  const bool no_rows = p->pairs > 0 && p->branch_rows == 0;  // every pair is dropped: there may be no branch to point to
  const bool branch = p->branch || no_rows;
  if ((!branch && !p->residual) || (!p->residual_out && !p->h) || !p->h != !p->pre_weight)
    return MOE_ERR_INVALID_ARG;
  if (!branch && (p->pairs || p->post_weight || p->gate)) return MOE_ERR_INVALID_ARG;
  if (p->pairs < 0 || p->pairs > kMaxTopK || (p->pairs > 0 && (!p->inv_pos || !p->pair_weights || p->branch_rows < 0)) ||
      (p->pairs == 0 && p->branch && p->branch_rows < p->tokens))
    return MOE_ERR_INVALID_ARG;
  if (p->branch_stride < 0 || p->residual_stride < 0 || p->gate_token_stride < 0 || p->gate_channel_stride < 0 ||
      p->gate_channel_stride > 1)
    return MOE_ERR_INVALID_ARG;
  if (p->tokens > 1 && ((p->residual_out && p->residual_out_stride < p->width) || (p->h && p->h_stride < p->width)))
    return MOE_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->weight_offset) ||
      !std::isfinite(p->residual_scale) || !std::isfinite(p->branch_scale))
    return MOE_ERR_INVALID_ARG;
  const int rs = p->residual_dtype == MOE_FP32 ? 4 : 2;
  if (!at_elements(p->branch, 2) || !at_elements(p->post_weight, 2) || !at_elements(p->gate, 2) ||
      !at_elements(p->pre_weight, 2) || !at_elements(p->h, 2) || !at_elements(p->residual, rs) ||
      !at_elements(p->residual_out, rs) || !at_elements(p->inv_pos, 4) || !at_elements(p->pair_weights, 4))
    return MOE_ERR_INVALID_ARG;
  if (p->tokens == 0) return MOE_OK;
  NormArgs a{};
  a.T = p->tokens;
  a.K = p->width;
  a.y = p->branch;
  a.ldy = p->branch_stride;
  a.rows = p->branch_rows;
  a.k = p->pairs;
  a.inv = p->inv_pos;
  a.pw = p->pair_weights;
  a.w_post = p->post_weight;
  a.gate = p->gate;
  a.gate_t = p->gate_token_stride;
  a.gate_c = p->gate_channel_stride;
  a.gate_sig = p->gate_sigmoid;
  a.res = p->residual;
  a.ldr = p->residual_stride;
  a.res_scale = p->residual_scale;
  a.br_scale = p->branch_scale;
  a.w_pre = p->pre_weight;
  a.eps = p->eps;
  a.w_off = p->weight_offset;
  a.inv_K = 1.f / p->width;
  a.r_out = p->residual_out;
  a.ldro = p->residual_out_stride;
  a.h = p->h;
  a.ldh = p->h_stride;
  return cuda_status(launch_block_norm(a, p->dtype, p->residual_dtype, static_cast<cudaStream_t>(cuda_stream)));
}

moe_status_t moe_quantize_rows(const void* x, long long x_stride, int x_rows, moe_dtype_t dtype, const int* src_rows,
                               int rows, int width, signed char* codes, long long codes_stride, float* scales,
                               void* cuda_stream) {
  if (rows < 0 || x_rows < 0 || width < 1 || !is16(dtype) || x_stride < 0 || (rows > 1 && codes_stride < width) ||
      (!src_rows && rows != x_rows))
    return MOE_ERR_INVALID_ARG;
  if (width > kMaxRowWidth) return MOE_ERR_TOO_LARGE;
  if (rows > 0 && ((!x && x_rows > 0) || !codes || !scales)) return MOE_ERR_INVALID_ARG;
  if (!at_elements(x, 2) || !at_elements(src_rows, 4) || !at_elements(scales, 4)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  QuantArgs a{x, x_stride, x_rows, src_rows, rows, width, codes, codes_stride, scales};
  return cuda_status(launch_quantize_rows(a, dtype, static_cast<cudaStream_t>(cuda_stream)));
}

moe_status_t moe_int8_matmul(const signed char* x, long long x_stride, const float* row_scales, const signed char* w,
                             long long w_stride, long long expert_stride, const float* channel_scales,
                             const int* offsets, int rows, int experts, int K, int N, void* y, long long y_stride,
                             moe_dtype_t y_dtype, void* cuda_stream) {
  const moe_status_t s = check_product(x, x_stride, w, w_stride, expert_stride, 1, offsets, rows, experts, K, N, y,
                                       y_stride, y_dtype);
  if (s != MOE_OK) return s;
  if (K > 131071) return MOE_ERR_TOO_LARGE;
  if (rows > 0 && (!row_scales || !channel_scales)) return MOE_ERR_INVALID_ARG;
  if (!at_elements(row_scales, 4) || !at_elements(channel_scales, 4)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  GroupedArgs a{x, x_stride, w, w_stride, expert_stride, row_scales, channel_scales, offsets, rows, experts, K, N,
                y, y_stride, 0};
  return run_product(a, kOpInt8, y_dtype, static_cast<cudaStream_t>(cuda_stream));
}

moe_status_t moe_grouped_matmul(const void* x, long long x_stride, const void* w, long long w_stride,
                                long long expert_stride, const int* offsets, int rows, int experts, int K, int N,
                                moe_dtype_t dtype, void* y, long long y_stride, moe_dtype_t y_dtype,
                                void* cuda_stream) {
  if (!is16(dtype)) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = check_product(x, x_stride, w, w_stride, expert_stride, 2, offsets, rows, experts, K, N, y,
                                       y_stride, y_dtype);
  if (s != MOE_OK) return s;
  if (rows == 0) return MOE_OK;
  GroupedArgs a{x, x_stride, w, w_stride, expert_stride, nullptr, nullptr, offsets, rows, experts, K, N,
                y, y_stride, 0};
  return run_product(a, dtype, y_dtype, static_cast<cudaStream_t>(cuda_stream));
}

moe_status_t moe_op_sync_status(void* cuda_stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  unsigned now = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices || read_op_timeouts(&now, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  for (unsigned seen = g_read[dev].load(); seen < now && !g_read[dev].compare_exchange_weak(seen, now);) {
  }
  Told* t = place_of(st, dev, now != 0, 0);
  const unsigned before = t ? t->count.exchange(now) : 0;
  return now != before ? MOE_ERR_TIMEOUT : MOE_OK;
}

moe_status_t moe_op_set_wait_limit(unsigned long long limit_ns) {
  g_wait_ns.store(limit_ns ? limit_ns : kDefaultWaitNs, std::memory_order_relaxed);
  return MOE_OK;
}

}  // extern "C"
