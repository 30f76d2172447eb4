// Products grouped by expert on the 5th-generation tensor cores:
//   y[r, n] = xs[r] ws[e, n] sum_k x[r, k] w[e, n, k]   (8-bit, int32 sums)
//   y[r, n] = sum_k x[r, k] w[e, n, k]                  (16-bit, fp32 sums)
//
// The weights are the MMA's M operand and the rows its N operand, so that a
// group of any size fills the tensor cores' 128 (or, over a CTA pair, 256)
// lanes with output channels and only pays for its own rows: N follows the
// rows of the tile in steps of 16 or 32. Both operands are K-major tiles of
// 128-byte rows (64 fp16 or 128 int8) brought in by TMA with the 128-byte
// swizzle, zero-filled past K, N and the last row; rows of a tile that belong
// to the next group are computed and not stored (columns of D are independent).
//
// Two forms of one kernel:
//   CG = 2  CTA pair, 256 channels x up to 256 rows, persistent over the tiles
//           of all experts, accumulators double-buffered in TMEM so that the
//           epilogue of one tile runs under the MMAs of the next;
//   CG = 1  128 channels x up to 128 rows per CTA for calls with few tiles; a
//           cluster of S CTAs splits K and adds the partial sums in rank order
//           through distributed shared memory, each CTA finishing n / S rows.
// What bounds it: with many rows the tensor cores (8192 x 4096 x 4096: busy 94%
// of the cycles in 16 bits, 88% in 8, at the clock that the power limit leaves);
// with some hundred rows per expert the reads of L2, which a tile of few rows
// needs more of per MMA (24576 x 2048 x 2816 in 64 uneven experts: busy 67%, dense
// 86%, both at 12 TB/s); with a few rows per expert the weights' bytes (128 rows
// in 8 experts of 4096 x 28672: 302 us, 97% of HBM's rate); with a few rows in
// all, latency (4.5 us for 2 rows).
// Roles: warp 0 TMA producer, warp 1 MMA (of the pair's first CTA), warps 2-9
// epilogue. Every mbarrier wait is bounded; one that runs out is counted, every
// role of the CTA stops at its next wait, the cluster drains its copies and MMAs,
// frees TMEM and returns.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "grouped_form.h"
#include "kernels.h"
#include "ops.cuh"
#include "tc.cuh"

namespace moeq {

__device__ unsigned g_op_timeouts;  // CTAs of the products in which a bounded wait ran out; only ever counted up

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreadsTc = 64 + 32 * kEpiWarps;
constexpr int kRowBytes = 128;                 // K bytes per stage
constexpr int kABytes = 128 * kRowBytes;       // 128 channels
constexpr int kBoxRows = 32;                   // unit of the rows per TMA box of x
constexpr int kBoxBytes = kBoxRows * kRowBytes;
constexpr int kMaxStagesTc = 10;
// Row tiles that share a sweep over the channels: few re-read the weights, many
// the rows. One, four, eight, sixteen, thirty-two, us: 8192 x 4096 x 8192 386,
// 360, 352, 350, 388; 16384 x 14336 x 4096 1283, 1284, 1276, 1326, 1441; 2048 x
// 4096 x 28672 398, 317, 305, 305, 303.
constexpr int kBandTc = 8;
constexpr int kStagingBytes = kEpiWarps * 2048;

// The tensor cores add to their fp32 accumulators with truncation, whose error
// grows in proportion to the number of additions: relative to the output 6e-7
// over 512 values of K summed in one go, 1.2e-6 over 1024, 2.5e-6 over 2048
// (fp16; bf16 a fifth less), always towards zero. So the accumulators of 16-bit
// operands are emptied every kChunk stages and added up in fp32, rounded to
// nearest: 512 values for fp32 outputs, 1024 for 16-bit ones, whose own rounding
// is far coarser (8192 x 4096 x 8192 in bf16: 341 us in one go, 347 with 1024
// values, 351 with 512; misrounded outputs at K = 14336 0.8%, 0.07%, 0.04%,
// nearest-rounded sums 0.08%). What remains to grow with K are the roundings to
// nearest of K / 512 or K / 1024 additions: 7.7e-7 and 1.3e-6 at K = 2^20.
template <typename TO>
constexpr int kChunk = sizeof(TO) == 4 ? 8 : 16;

struct TcArgs {
  CUtensorMap map_w;   // [E][N][K], box 128 rows
  CUtensorMap map_x[4];  // [rows][K], boxes of 32, 64, 96 and 128 rows as far as nmax needs them: one copy per stage
  GroupedArgs g;
  uint32_t idesc;      // without the N field
  int NF;              // channel tiles
  uint32_t nf_inv;     // 2^32 / NF, rounded down, + 1
  int nmax;            // rows per tile
  int stages, bslot;   // ring depth, bytes of a stage's x part
  int S;               // CTAs splitting K (CG = 1)
  int vec;             // y rows start at 8-byte boundaries
};

struct RowTilesTc {
  int nmax;
  __device__ int operator()(int n) const { return (n + nmax - 1) / nmax; }
};

// ---- cluster helpers
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// takes the place of copies that were announced and never issued
__device__ __forceinline__ void complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// makes what other CTAs of the cluster wrote before their arrivals visible
__device__ __forceinline__ void fence_acquire_cluster() { asm volatile("fence.acq_rel.cluster;\n" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---- tcgen05 and TMA forms of one CTA or a CTA pair
template <int CG>
__device__ __forceinline__ void tma2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
template <int CG, bool I8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc) {
  if constexpr (CG == 1 && !I8)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
  else if constexpr (CG == 1)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
  else if constexpr (!I8)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// arrives on the barrier at this offset in every CTA of the group once the MMAs issued so far are done
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1)
    mma_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar), "h"((uint16_t)3) : "memory");
}
template <int CG>
__device__ __forceinline__ void alloc_tmem(uint32_t slot, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, cols);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(slot), "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
  }
}
template <int CG>
__device__ __forceinline__ void free_tmem(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 1) tmem_dealloc(addr, cols);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(cols));
}
// Wait of a role: the phase has usually completed; the shared abort flag is
// looked at only when it has not.
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity, unsigned* status, unsigned long long limit_ns,
                                          volatile int* aborted) {
  if (limit_ns >= kSleepLimitNs && mbar_test(bar, parity)) return true;
  return !*aborted && mbar_wait_slow(bar, parity, status, limit_ns);
}

struct Tile {
  int e, r0, live, n, f0;  // expert, first row, rows to store, rows computed, first channel
};
// Tile i of the call: experts in order; within one, bands of kBandTc row tiles
// sweep the channels together, so that the CTAs running at one time read about
// as many distinct weight rows as activation rows.
template <int CG>
__device__ __forceinline__ Tile tile_of(const GroupTable& g, const TcArgs& a, int i) {
  constexpr int kUnit = 16 * CG;  // step of a tile's rows
  // i / NF by a product that is one too large at most
  auto by_nf = [&](int v) {
    const int q = a.NF == 1 ? v : (int)__umulhi((uint32_t)v, a.nf_inv);
    return q * a.NF > v ? q - 1 : q;
  };
  Tile t;
  t.e = find_group(g, a.g.E, by_nf(i));
  const int nt = g.first[t.e + 1] - g.first[t.e], rows = g.rows[t.e];
  const int local = i - g.first[t.e] * a.NF;
  const int band = by_nf(local) / kBandTc, in = local - band * kBandTc * a.NF;
  const int bt = min(kBandTc, nt - band * kBandTc);
  const int f = bt == 1 ? in : in / bt, tk = band * kBandTc + in - f * bt;
  // widths in units that differ by one at most, so that no tile reads its
  // weights for a few rows only
  const int units = (rows + kUnit - 1) / kUnit, base = nt == 1 ? units : units / nt, more = units - base * nt;
  const int u0 = tk * base + min(tk, more);
  t.n = (base + (tk < more ? 1 : 0)) * kUnit;
  t.live = min(t.n, rows - u0 * kUnit);
  t.r0 = g.begin[t.e] + u0 * kUnit;
  t.f0 = f * 128 * CG;
  return t;
}

// A pair's work: whole tiles, then its share of the last turn's.
template <int CG>
struct Turns {
  int whole, parts, items;  // tiles of complete turns; parts of each further one; all pieces of work
  __device__ __forceinline__ Turns(int tiles, int clusters) {
    const int rest = CG == 2 ? tiles % clusters : 0;
    whole = tiles - rest;
    parts = last_turn_parts(rest, clusters);
    items = whole + rest * parts;
  }
};
// piece i of the work; false if it has no rows
template <int CG>
__device__ __forceinline__ bool piece_of(const GroupTable& g, const TcArgs& a, const Turns<CG>& w, int i, Tile& t) {
  if (CG == 1 || i < w.whole || w.parts == 1) {
    t = tile_of<CG>(g, a, i);
    return true;
  }
  constexpr int kUnit = 16 * CG;
  const int j = i - w.whole, shift = w.parts == 4 ? 2 : 1, p = j & (w.parts - 1);
  t = tile_of<CG>(g, a, w.whole + (j >> shift));
  const int units = t.n / kUnit, u0 = units * p >> shift, u1 = units * (p + 1) >> shift;
  t.n = (u1 - u0) * kUnit;
  t.live = min(t.n, t.live - u0 * kUnit);
  t.r0 += u0 * kUnit;
  return u1 > u0;
}

template <bool I8>
__device__ __forceinline__ float scaled(uint32_t v, float s) {
  if constexpr (I8) return (float)(int)v * s;
  else return __uint_as_float(v);
}

// 32 columns (rows of y from row c0 of the tile) of the accumulator into registers
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The loaded registers may be read only after this (they pass through it, so
// that no use moves ahead of the wait).
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// One warp's 32 channels (lane = channel) of 32 rows to y. 16-bit outputs
// cross the warp's 2 KiB of shared memory as pairs of rows, so that a store
// covers four rows of 32 channels, 8 bytes a lane; 32-bit outputs go out
// directly, one row of 32 channels per store.
// ws: the lane's channel's scale, xv: the scale of row c0 + lane.
template <typename TO, bool I8>
__device__ __forceinline__ void store_chunk(const TcArgs& a, const Tile& t, int c0, const uint32_t (&v)[32], float ws,
                                            float xv, uint32_t* stage, float* xs, int ch0, int lane) {
  float sc[32];
  if constexpr (I8) {
    xs[lane] = xv;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 x = *reinterpret_cast<const float4*>(xs + j);
      sc[j] = ws * x.x;
      sc[j + 1] = ws * x.y;
      sc[j + 2] = ws * x.z;
      sc[j + 3] = ws * x.w;
    }
  }
  const int rows = t.live - c0;  // rows to store, maybe more than 32
  if constexpr (sizeof(TO) == 4) {
    if (ch0 + lane < a.g.N) {
      float* y = static_cast<float*>(a.g.y) + (long long)(t.r0 + c0) * a.g.ldy + ch0 + lane;
      if (rows >= 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j * a.g.ldy] = scaled<I8>(v[j], I8 ? sc[j] : 0.f);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < rows) y[j * a.g.ldy] = scaled<I8>(v[j], I8 ? sc[j] : 0.f);
      }
    }
    __syncwarp();
  } else {
#pragma unroll
    for (int p = 0; p < 16; ++p)
      stage[p * 32 + lane] = pack2<TO>(scaled<I8>(v[2 * p], I8 ? sc[2 * p] : 0.f),
                                       scaled<I8>(v[2 * p + 1], I8 ? sc[2 * p + 1] : 0.f));
    __syncwarp();
    uint4 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const uint4*>(stage + (4 * i + (lane >> 3)) * 32 + 4 * (lane & 7));
    __syncwarp();
    const int ch = ch0 + 4 * (lane & 7), p0 = lane >> 3;
    TO* y = static_cast<TO*>(a.g.y) + (long long)(t.r0 + c0 + 2 * p0) * a.g.ldy + ch;
    if (a.vec && rows >= 32 && ch0 + 32 <= a.g.N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<uint2*>(y + 8 * i * a.g.ldy) = make_uint2(prmt(q[i].x, q[i].y, 0x5410u), prmt(q[i].z, q[i].w, 0x5410u));
        *reinterpret_cast<uint2*>(y + (8 * i + 1) * a.g.ldy) = make_uint2(prmt(q[i].x, q[i].y, 0x7632u), prmt(q[i].z, q[i].w, 0x7632u));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (8 * i + 2 * p0 + h >= rows) continue;
          uint16_t* o = reinterpret_cast<uint16_t*>(y + (8 * i + h) * a.g.ldy);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (ch + b < a.g.N) o[b] = (uint16_t)(w[b] >> (16 * h));
        }
      }
    }
  }
}

#include "grouped_loads.cuh"

template <int CG, bool I8, typename TO>
__global__ void __launch_bounds__(kThreadsTc, 1) grouped_tc_kernel(const __grid_constant__ TcArgs a) {
  extern __shared__ uint8_t raw[];
  __shared__ GroupTable g;
  __shared__ __align__(16) float xs_s[kEpiWarps][32];
  __shared__ __align__(8) uint64_t bars_s[2 * kMaxStagesTc + 6];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s, issued_s;
  __shared__ unsigned status_s;  // of this CTA's waits
  __shared__ uint32_t bytes_s[kMaxStagesTc];  // of the stage's last copies
  __shared__ uint32_t cluster_abort;
  constexpr int kUnitCols = CG == 2 ? 256 : 128;  // TMEM columns of one accumulator
  constexpr uint32_t kCols = 2 * kUnitCols;
  constexpr int kElem = I8 ? 128 : 64;            // elements per 128-byte row
  const uint32_t pad = (1024u - (smem_u32(raw) & 1023u)) & 1023u;
  uint8_t* sm = raw + pad;
  const uint32_t sbase = smem_u32(sm);
  const int stage_bytes = kABytes + a.bslot;
  uint8_t* tail = sm + a.stages * stage_bytes;    // staging (CG = 2) or partial sums (CG = 1)
  const uint32_t bars = smem_u32(bars_s);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kMaxStagesTc + s); };
  auto acc_full = [&](int b) { return bars + 8 * (2 * kMaxStagesTc + b); };
  auto acc_empty = [&](int b) { return bars + 8 * (2 * kMaxStagesTc + 2 + b); };
  const uint32_t drained = bars + 8 * (2 * kMaxStagesTc + 4), summed = bars + 8 * (2 * kMaxStagesTc + 5);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int csize = CG == 2 ? 2 : a.S;
  const int cluster = blockIdx.x / csize, nclusters = gridDim.x / csize;
  const int lead = CG == 2 ? 0 : (int)rank;       // CTA whose MMA warp consumes this CTA's stages
  volatile int* aborted = &abort_s;
  unsigned* status = &status_s;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), kEpiWarps * CG);
    }
    mbar_init(drained, 1);
    mbar_init(summed, kEpiWarps * (CG == 1 ? a.S : 1));
    abort_s = 0;
    status_s = 0;
    cluster_abort = 0;
    issued_s = 0;
    fence_barrier_init();
  }
  if (warp == 0 && elect_one()) {
    prefetch_map(&a.map_w);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (b * kBoxRows * CG < a.nmax) prefetch_map(&a.map_x[b]);
  }
  if (warp == 1) alloc_tmem<CG>(smem_u32(&tmem_slot), kCols);
  auto sync = [&] {
    if (csize > 1) cluster_sync();
    else __syncthreads();
  };
  tc_fence_before();
  sync();
  tc_fence_after();
  pdl_wait();  // what precedes touches no memory of the call
  pdl_trigger();
  build_group_table(g, a.g.offsets, a.g.rows, a.g.E, RowTilesTc{a.nmax});
  const uint32_t tmem = tmem_slot;
  const Turns<CG> work(g.first[a.g.E] * a.NF, nclusters);
  const int nk = (a.g.K + kElem - 1) / kElem;
  const int kb0 = CG == 1 ? nk * (int)rank / a.S : 0, kb1 = CG == 1 ? nk * ((int)rank + 1) / a.S : nk;

  // The copy and MMA warps run their loops whole, with warp-uniform values; one
  // elected lane issues.
  if (warp == 0) {
    // the pair's copies all count on the first CTA's barrier, which that CTA alone announces them to
    const uint32_t full0 = CG == 2 ? map_rank(full(0), 0) : full(0);
    const bool announce = CG == 1 || rank == 0;
    int slot = 0, round = 0, issued = 0;
    bool ok = true;
    for (int i = cluster; i < work.items && ok; i += nclusters) {
      Tile t;
      if (!piece_of<CG>(g, a, work, i, t)) continue;
      const int nb = (t.n / CG + kBoxRows - 1) / kBoxRows;
      const uint32_t bytes = kABytes + nb * kBoxBytes;
      const CUtensorMap* map_x = &a.map_x[nb - 1];
      const int row = t.r0 + (CG == 2 ? (int)rank * (t.n / 2) : 0), ch = t.f0 + (CG == 2 ? (int)rank * 128 : 0);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = round == 0 || role_wait(empty(slot), (round - 1) & 1, status, a.g.wait_ns, aborted);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          if (announce) mbar_expect_tx(full(slot), CG * bytes);
          bytes_s[slot] = bytes;
          const uint32_t dst = sbase + slot * stage_bytes;
          tma3<CG>(dst, &a.map_w, kb * kElem, ch, t.e, full0 + 8 * slot);
          tma2<CG>(dst + kABytes, map_x, kb * kElem, row, full0 + 8 * slot);
        }
        __syncwarp();
        ++issued;
        if (++slot == a.stages) {
          slot = 0;
          ++round;
        }
      }
    }
    if (lane == 0) issued_s = issued;
    // the last arrivals on this CTA's empty barriers land before it may exit
    for (int u = max(0, issued - a.stages); u < issued && ok; ++u)
      ok = mbar_wait_fast(empty(u % a.stages), (u / a.stages) & 1, status, kDrainLimitNs);
    if (!ok) *aborted = 1;
  } else if (warp == 1) {
    if (CG == 1 || rank == 0) {
      int slot = 0, ph = 0, u = 0;  // u: accumulators filled so far
      bool ok = true;
      for (int i = cluster; i < work.items && ok; i += nclusters) {
        Tile t;
        if (!piece_of<CG>(g, a, work, i, t)) continue;
        const uint32_t idesc = a.idesc | ((uint32_t)(t.n >> 3) << 17);
        for (int kb = kb0; kb < kb1 && ok; ++u) {
          const int first = kb, end = I8 ? kb1 : min(kb + kChunk<TO>, kb1), buf = u & 1;
          ok = u < 2 || role_wait(acc_empty(buf), ((u >> 1) - 1) & 1, status, a.g.wait_ns, aborted);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * kUnitCols;
          for (; kb < end; ++kb) {
            ok = role_wait(full(slot), ph, status, a.g.wait_ns, aborted);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t ad = sw128_desc(sbase + slot * stage_bytes), bd = sw128_desc(sbase + slot * stage_bytes + kABytes);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ss<CG, I8>(d, ad + 2 * k, bd + 2 * k, idesc, kb > first || k > 0);
              commit<CG>(empty(slot));
              if (kb == end - 1) commit<CG>(acc_full(buf));
            }
            __syncwarp();
            if (++slot == a.stages) {
              slot = 0;
              ph ^= 1;
            }
          }
        }
      }
      if (!ok) *aborted = 1;
      // every MMA completes before the cluster frees its TMEM
      if (elect_one()) {
        if constexpr (CG == 1) mma_commit(drained);
        else
          asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(drained) : "memory");
      }
      __syncwarp();
      mbar_wait(drained, 0, status, kDrainLimitNs);
    }
  } else {
    // two warps per 32 channels, taking the tile's column chunks in turn
    const int quarter = warp & 3;
    uint32_t* stage = reinterpret_cast<uint32_t*>(tail) + (warp - 2) * 512;
    float* xs = xs_s[warp - 2];
    int u = 0, it = 0;
    auto filled = [&](int buf) {
      const bool ok = role_wait(acc_full(buf), (u >> 1) & 1, status, a.g.wait_ns, aborted);
      return __all_sync(0xffffffffu, ok);
    };
    auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) arrive_cluster(map_rank(acc_empty(buf), lead));
        else mbar_arrive(acc_empty(buf));
      }
    };
    for (int i = cluster; i < work.items; i += nclusters) {
      Tile t;
      if (!piece_of<CG>(g, a, work, i, t)) continue;
      // tiles of up to 32 rows go to one half of the warps, in turn
      const int half = ((warp - 2) >> 2) ^ (it++ & 1);
      const int ch0 = t.f0 + (CG == 2 ? (int)rank * 128 : 0) + quarter * 32, ch = ch0 + lane;
      const bool split = CG == 1 && a.S > 1;
      // Of a split tile the partial sums of columns [q c, q c + c) go to CTA q,
      // slot [rank]; in a slot four columns of a channel lie together, 16 bytes
      // a lane.
      const int c = split ? t.n / a.S : t.n;
      const uint32_t part = smem_u32(tail) + (uint32_t)((int)rank * c * 512 + (quarter * 32 + lane) * 16);
      auto send = [&](int col, const uint32_t* v) {
        const int q = col / c;
        st_cluster_v4(map_rank(part + (uint32_t)(col - q * c) * 512, q), v);
      };
      // scales are on their way while the accumulators are filled
      float ws = 0.f;
      auto row_scale = [&](int c0) {
        float x = 0.f;
        if constexpr (I8)
          if (c0 + lane < t.live) x = a.g.xs[t.r0 + c0 + lane];
        return x;
      };
      if constexpr (I8)
        if (ch < a.g.N) ws = a.g.ws[(long long)t.e * a.g.N + ch];
      float xv = split ? 0.f : row_scale(half * 32);
      bool ok = true;
      if constexpr (!I8) {
        constexpr int kParts = kUnitCols / 64;
        uint32_t sum[kParts][32];
        for (int kb = kb0; kb < kb1; kb += kChunk<TO>, ++u) {
          const int buf = u & 1;
          ok = filled(buf);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * kUnitCols + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
          for (int p = 0; p < kParts; ++p) {
            const int c0 = half * 32 + p * 64;
            if (c0 >= t.n) break;
            if (kb == kb0) {
              tmem_ld32_nw(d + c0, sum[p]);
              tmem_wait_ld(sum[p]);
            } else {
              uint32_t v[32];
              tmem_ld32_nw(d + c0, v);
              tmem_wait_ld(v);
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[p][j] = __float_as_uint(__uint_as_float(sum[p][j]) + __uint_as_float(v[j]));
            }
          }
          release(buf);
        }
        if (ok) {
#pragma unroll
          for (int p = 0; p < kParts; ++p) {
            const int c0 = half * 32 + p * 64;
            if (c0 >= t.n) break;
            if (split) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                if (c0 + j < t.n) send(c0 + j, sum[p] + j);
            } else {
              store_chunk<TO, I8>(a, t, c0, sum[p], ws, 0.f, stage, xs, ch0, lane);
            }
          }
        }
      } else {
        const int buf = u & 1;
        ok = filled(buf);
        if (ok) {
          tc_fence_after();
          const uint32_t d = tmem + buf * kUnitCols + ((uint32_t)(quarter * 32) << 16);
          if (!split) {
            // the next chunk's load is in flight while a chunk is stored
            uint32_t v[2][32];
            const int c_first = half * 32;
            if (c_first < t.n) tmem_ld32_nw(d + c_first, v[0]);
#pragma unroll 1
            for (int c0 = c_first; c0 < t.n; c0 += 128) {
              tmem_wait_ld(v[0]);
              if (c0 + 64 < t.n) tmem_ld32_nw(d + c0 + 64, v[1]);
              float xn = row_scale(c0 + 64);
              store_chunk<TO, I8>(a, t, c0, v[0], ws, xv, stage, xs, ch0, lane);
              if (c0 + 64 < t.n) {
                tmem_wait_ld(v[1]);
                if (c0 + 128 < t.n) tmem_ld32_nw(d + c0 + 128, v[0]);
                xv = row_scale(c0 + 128);
                store_chunk<TO, I8>(a, t, c0 + 64, v[1], ws, xn, stage, xs, ch0, lane);
              }
            }
          } else {
            for (int c0 = half * 16; c0 < t.n; c0 += 32) {
              uint32_t v[16];
              tmem_ld16(d + c0, v);
#pragma unroll
              for (int j = 0; j < 16; j += 4) send(c0 + j, v + j);
            }
          }
          release(buf);
        }
        ++u;
      }
      if (!ok) {
        *aborted = 1;
        break;
      }
      if (split) {
        __syncwarp();
        if (lane < a.S) arrive_cluster(map_rank(summed, lane));
        ok = mbar_wait(summed, 0, status, a.g.wait_ns);
        fence_acquire_cluster();
        if (!ok) {
          *aborted = 1;
          break;
        }
        // this CTA's c columns, four at a time: added in rank order, finished, stored
        const uint4* sums = reinterpret_cast<const uint4*>(tail) + quarter * 32 + lane;
        const int slot4 = c * 32;  // 16-byte words of a slot
        for (int j = half * 4; j < c; j += 8) {
          const int col = (int)rank * c + j;
          if (col >= t.live || ch >= a.g.N) break;
          float y[4];
          if constexpr (I8) {
            int n[4] = {};
            for (int q = 0; q < a.S; q += 2) {
              const uint4 u = sums[q * slot4 + j * 32], w = sums[(q + 1) * slot4 + j * 32];
              n[0] += (int)u.x + (int)w.x;
              n[1] += (int)u.y + (int)w.y;
              n[2] += (int)u.z + (int)w.z;
              n[3] += (int)u.w + (int)w.w;
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) y[h] = col + h < t.live ? (float)n[h] * (ws * a.g.xs[t.r0 + col + h]) : 0.f;
          } else {
            float4 n = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q = 0; q < a.S; q += 2) {
              const uint4 u = sums[q * slot4 + j * 32], w = sums[(q + 1) * slot4 + j * 32];
              n.x = n.x + __uint_as_float(u.x) + __uint_as_float(w.x);
              n.y = n.y + __uint_as_float(u.y) + __uint_as_float(w.y);
              n.z = n.z + __uint_as_float(u.z) + __uint_as_float(w.z);
              n.w = n.w + __uint_as_float(u.w) + __uint_as_float(w.w);
            }
            y[0] = n.x;
            y[1] = n.y;
            y[2] = n.z;
            y[3] = n.w;
          }
          TO* out = static_cast<TO*>(a.g.y) + (long long)(t.r0 + col) * a.g.ldy + ch;
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (col + h < t.live) out[h * a.g.ldy] = from_f32<TO>(y[h]);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && abort_s)
    for (int q = 0; q < csize; ++q) st_cluster_u32(map_rank(smem_u32(&cluster_abort), q), 1u);
  tc_fence_before();
  sync();
  tc_fence_after();
  if (*(volatile uint32_t*)&cluster_abort) {
    // Wait for every copy in flight. Where one CTA of a pair filled a stage and
    // the other did not, the missing half is made up here, so that the phase
    // can complete.
    if (threadIdx.x == 0 && (CG == 1 || rank == 0)) {
      const int mine = issued_s, other = CG == 2 ? (int)ld_cluster_u32(map_rank(smem_u32(&issued_s), 1)) : mine;
      const int last = max(mine, other);
      for (int u = max(0, last - a.stages); u < last; ++u) {
        const int s = u % a.stages;
        if (u >= other) complete_tx(full(s), bytes_s[s]);
        if (u >= mine) mbar_expect_tx(full(s), ld_cluster_u32(map_rank(smem_u32(&bytes_s[s]), 1)));
        mbar_wait(full(s), (u / a.stages) & 1, status, kDrainLimitNs);
      }
    }
    cluster_sync();
  }
  if (warp == 1) free_tmem<CG>(tmem, kCols);
  if constexpr (CG == 2) cluster_sync();  // the pair's TMEM goes together
  if (threadIdx.x == 0 && status_s) atomicAdd(&g_op_timeouts, 1u);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

bool encode_rows(CUtensorMap* m, const void* base, int op, int es, long long K, long long rows, long long ld,
                 long long E, long long lde, int box_rows) {
  const CUtensorMapDataType type = op == kOpInt8   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : op == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)rows, (cuuint64_t)E};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * es), (cuuint64_t)(lde * es)};
  const cuuint32_t box[3] = {(cuuint32_t)(kRowBytes / es), (cuuint32_t)box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode_fn()(m, type, E ? 3 : 2, const_cast<void*>(base), dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSmemBudget = 221 * 1024;  // dynamic; the static tables take about 6 KiB more

// Raises a kernel's limit of dynamic shared memory once per device; set holds
// the devices done.
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<unsigned long long>& set) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev <= 63 && (set.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess && dev <= 63) set.fetch_or(1ull << dev, std::memory_order_release);
  return err;
}

template <int CG, bool I8, typename TO>
cudaError_t launch_tc(const TcArgs& a, int clusters, size_t smem, cudaStream_t st) {
  static std::atomic<unsigned long long> set{0};
  const cudaError_t err = allow_smem(grouped_tc_kernel<CG, I8, TO>, kSmemBudget, set);
  if (err != cudaSuccess) return err;
  const int csize = CG == 2 ? 2 : a.S;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * csize);
  cfg.blockDim = dim3(kThreadsTc);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = csize;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_tc_kernel<CG, I8, TO>, a);
}
template <bool I8, typename TO>
cudaError_t launch_loads(const TcArgs& a, int grid, cudaStream_t st) {
  constexpr int kSmem = kStagesLoads * (kABytes + 128 * kRowBytes) + 1024;
  static std::atomic<unsigned long long> set{0};
  const cudaError_t err = allow_smem(grouped_loads_kernel<I8, TO>, kSmem, set);
  if (err != cudaSuccess) return err;
  return launch_kernel(grouped_loads_kernel<I8, TO>, dim3(grid), dim3(kThreadsLoads), kSmem, st, true, a);
}
// go(whether the operands are 8-bit, a value of the output type)
template <typename Go>
cudaError_t by_types(int op, int y_dtype, Go go) {
  auto by_out = [&](auto i8) {
    if (y_dtype == DT_BF16) return go(i8, __nv_bfloat16{});
    if (y_dtype == DT_FP16) return go(i8, __half{});
    return go(i8, 0.f);
  };
  return op == kOpInt8 ? by_out(std::true_type{}) : by_out(std::false_type{});
}
template <int CG>
cudaError_t launch_tc_typed(const TcArgs& a, int op, int y_dtype, int clusters, size_t smem, cudaStream_t st) {
  return by_types(op, y_dtype, [&](auto i8, auto out) {
    return launch_tc<CG, decltype(i8)::value, decltype(out)>(a, clusters, smem, st);
  });
}

// what every form of the kernels needs; the instruction descriptor without its N field
TcArgs common_args(const GroupedArgs& g, int op, int cg, int width) {
  TcArgs a{};
  a.g = g;
  a.vec = reinterpret_cast<uintptr_t>(g.y) % 8 == 0 && g.ldy % 4 == 0;
  a.idesc = op == kOpInt8 ? (2u << 4) | (1u << 7) | (1u << 10)
                          : (1u << 4) | ((op == DT_BF16 ? 1u : 0u) << 7) | ((op == DT_BF16 ? 1u : 0u) << 10);
  a.idesc |= (uint32_t)(128 * cg >> 4) << 24;
  a.NF = (g.N - 1) / (128 * cg) + 1;
  a.nf_inv = (uint32_t)((1ull << 32) / a.NF + 1);
  a.nmax = width;
  a.S = 1;
  return a;
}
// ceil(r / n) summed over the groups' rows r is at most one tile for each group
// that can have rows and one for every n of the other rows
long long most_tiles(const GroupedArgs& g, int width, int NF) {
  const int groups = std::min(g.rows, g.E);
  return (long long)(groups + (g.rows - groups) / width) * NF;
}

}  // namespace

// Whether TMA can address the operands: 16-byte bases and strides, each stride a
// multiple of the one below it (a rule of tensor maps), rows that do not overlap;
// and tile counts within an int.
bool grouped_tc_fits(const GroupedArgs& a, int op) {
  const long long es = op == kOpInt8 ? 1 : 2;
  auto m16 = [](long long v) { return v % 16 == 0; };
  const long long lim = 1LL << 39;
  if (!encode_fn()) return false;
  if (!m16((long long)reinterpret_cast<uintptr_t>(a.x)) || !m16((long long)reinterpret_cast<uintptr_t>(a.w))) return false;
  if ((a.rows > 1 && (!m16(a.ldx * es) || a.ldx < a.K)) || !m16(a.ldw * es) || a.ldw < a.K) return false;
  if (a.E > 1 && (!m16(a.ldwe * es) || a.ldwe % a.ldw || a.ldwe < (a.N - 1) * a.ldw + a.K)) return false;
  if (a.ldx * es >= lim || a.ldw * es * a.N >= lim || a.ldwe * es >= lim) return false;
  return ((long long)a.rows / 16 + a.E) * (a.N / 128 + 1) < (1LL << 30);
}

cudaError_t launch_grouped_tc(const GroupedArgs& g, int op, int y_dtype, cudaStream_t st) {
  const int es = op == kOpInt8 ? 1 : 2;
  const int sms = device_sms(), pairs = sms / 2;
  const long long ldx = g.rows > 1 ? g.ldx : (g.K + 15) / 16 * 16;
  const long long ldwe = g.E > 1 ? g.ldwe : g.ldw * g.N;
  const int nk = (g.K * es + kRowBytes - 1) / kRowBytes;
  const auto [cg, width, S] = choose_form(g.rows, g.E, g.N, (long long)g.K * es, sms);
  TcArgs a = common_args(g, op, cg, width);
  a.S = S;
  const long long most = most_tiles(g, a.nmax, a.NF);
  if (!encode_rows(&a.map_w, g.w, op, es, g.K, g.N, g.ldw, g.E, ldwe, 128)) return cudaErrorInvalidValue;
  for (int b = 0; b < 4 && b * kBoxRows * cg < a.nmax; ++b)
    if (!encode_rows(&a.map_x[b], g.x, op, es, g.K, g.rows, ldx, 0, 0, (b + 1) * kBoxRows)) return cudaErrorInvalidValue;
  if (cg == 2) {
    a.bslot = 128 * kRowBytes;
    a.stages = 6;
    const size_t smem = (size_t)a.stages * (kABytes + a.bslot) + kStagingBytes + 1024;
    return launch_tc_typed<2>(a, op, y_dtype, (int)std::min<long long>(most, pairs), smem, st);
  }
  a.bslot = (a.nmax + kBoxRows - 1) / kBoxRows * kBoxBytes;
  const int fixed = (a.S > 1 ? a.nmax * 512 : kStagingBytes) + 1024;
  a.stages = std::min({kMaxStagesTc, (kSmemBudget - fixed) / (kABytes + a.bslot), std::max(2, (nk + a.S - 1) / a.S)});
  const size_t smem = (size_t)a.stages * (kABytes + a.bslot) + fixed;
  const int clusters = (int)(a.S > 1 ? most : std::min<long long>(most, sms));
  return launch_tc_typed<1>(a, op, y_dtype, clusters, smem, st);
}

cudaError_t launch_grouped_loads(const GroupedArgs& g, int op, int y_dtype, cudaStream_t st) {
  const int NF = (g.N - 1) / 128 + 1;
  int width = 128;  // narrower only where there would not be a tile for every SM
  while (width > 16 && most_tiles(g, width, NF) < device_sms()) width /= 2;
  const TcArgs a = common_args(g, op, 1, width);
  const int grid = (int)std::min<long long>(most_tiles(g, width, NF), 2LL * device_sms());
  return by_types(op, y_dtype, [&](auto i8, auto out) {
    return launch_loads<decltype(i8)::value, decltype(out)>(a, grid, st);
  });
}

cudaError_t read_op_timeouts(unsigned* out, cudaStream_t st) {
  const cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_op_timeouts, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, st);
  return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

}  // namespace moeq
