// The grouped products for operands that bulk copies cannot address: bases or
// strides that are not multiples of 16 bytes, rows that overlap. Included by
// grouped_tc.cu, whose tiles, MMAs and stores it shares; only the copies differ.
//
// One CTA per 128 channels x up to 128 rows, two CTAs per SM. Its eight warps load
// a stage with ordinary loads, 16 bytes of a row at a time, write it to shared
// memory in the swizzled layout that the MMAs read, and store the finished tile;
// warp 0 issues the MMAs of a stage while the loads of the next are under way (a
// warp of its own for them would leave the others 96 registers instead of 128, too
// few for the loads of a stage beside the sums of the chunks: 25% slower).
// 16 bytes that lie across an aligned boundary are shifted out of the two aligned
// pieces around them, or read element by element where those would leave the row.
// A tile's sums of earlier chunks wait in TMEM, beside the accumulators. Bound by
// the loads' latency, which two CTAs of three stages cover in part: 16384 rows by
// 4096 channels of 14335 in 8 experts 7.7 ms (bulk copies at 14336: 1.26), 8-bit
// 4.0 (0.59); one row of 2047 by 2816 channels 47 us, 8-bit 29.

constexpr int kLoadWarps = 8;
constexpr int kThreadsLoads = 32 * kLoadWarps;
constexpr int kStagesLoads = 3;

// Bytes b .. b + 15 of a row of len bytes, as loaded
template <int ES>
struct Chunk16 {
  uint32_t w[8];
  int mis;  // 0, or the offset within the two pieces
  __device__ __forceinline__ void load(const uint8_t* row, int b, int len, bool have) {
    mis = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0;
    if (!have || b >= len) return;
    const uint8_t* p = row + b;
    const int m = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    if (m == 0 && b + 16 <= len) {
      put(0, *reinterpret_cast<const uint4*>(p));
    } else if (b - m >= 0 && b - m + 32 <= len) {
      mis = m;
      put(0, reinterpret_cast<const uint4*>(p - m)[0]);
      put(4, reinterpret_cast<const uint4*>(p - m)[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 16 / ES; ++i) {
        if (b + i * ES >= len) break;
        if constexpr (ES == 2) w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        else w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
      }
    }
  }
  __device__ __forceinline__ void put(int i, uint4 u) {
    w[i] = u.x;
    w[i + 1] = u.y;
    w[i + 2] = u.z;
    w[i + 3] = u.w;
  }
  __device__ __forceinline__ uint4 value() const {
    if (mis == 0) return make_uint4(w[0], w[1], w[2], w[3]);
    uint32_t s[7], r[5];
    const bool one = mis & 4, two = mis & 8;
#pragma unroll
    for (int i = 0; i < 7; ++i) s[i] = one ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) r[i] = two ? s[i + 2] : s[i];
    const int bits = (mis & 3) * 8;
    return make_uint4(__funnelshift_r(r[0], r[1], bits), __funnelshift_r(r[1], r[2], bits),
                      __funnelshift_r(r[2], r[3], bits), __funnelshift_r(r[3], r[4], bits));
  }
};

template <bool I8, typename TO>
__global__ void __launch_bounds__(kThreadsLoads, 2) grouped_loads_kernel(const __grid_constant__ TcArgs a) {
  extern __shared__ uint8_t raw[];
  __shared__ GroupTable g;
  __shared__ __align__(16) float xs_s[kLoadWarps][32];
  __shared__ __align__(8) uint64_t bars_s[2 * kStagesLoads + 3];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ unsigned status_s;  // of this CTA's waits
  constexpr int ES = I8 ? 1 : 2;
  constexpr uint32_t kSums = 128;  // first TMEM column of the sums of a tile's earlier chunks
  constexpr uint32_t kCols = I8 ? kSums : 2 * kSums;
  constexpr int kStage = kABytes + 128 * kRowBytes;
  const uint32_t pad = (1024u - (smem_u32(raw) & 1023u)) & 1023u;
  uint8_t* sm = raw + pad;
  const uint32_t sbase = smem_u32(sm), bars = smem_u32(bars_s);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStagesLoads + s); };
  const uint32_t acc_full = bars + 8 * (2 * kStagesLoads), acc_empty = acc_full + 8, drained = acc_full + 16;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* aborted = &abort_s;
  unsigned* status = &status_s;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStagesLoads; ++s) {
      mbar_init(full(s), kLoadWarps);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kLoadWarps);
    mbar_init(drained, 1);
    abort_s = 0;
    status_s = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  build_group_table(g, a.g.offsets, a.g.rows, a.g.E, RowTilesTc{a.nmax});
  const uint32_t tmem = tmem_slot;
  const int total = g.first[a.g.E] * a.NF;
  const int len = a.g.K * ES, nk = (len + kRowBytes - 1) / kRowBytes;

  const int quarter = warp & 3, half = warp >> 2;
  const int lr = threadIdx.x >> 3, lc = threadIdx.x & 7;  // this thread's row (+ 32 j) and 16 bytes of a stage
  const uint32_t place = (uint32_t)(lr * kRowBytes + ((lc ^ (lr & 7)) << 4));
  // the stages are free while a tile is stored: all its MMAs are done and the next is not begun
  uint32_t* stage = reinterpret_cast<uint32_t*>(sm) + warp * 512;
  const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16);
  int slot = 0, round = 0, it = 0;  // it: accumulators filled so far
  int mslot = 0, mph = 0;           // of the next MMAs (warp 0)
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    const bool done = role_wait(bar, parity, status, a.g.wait_ns, aborted);
    return (bool)__all_sync(0xffffffffu, done);
  };
  // the MMAs of one stage, once every warp has written its part
  auto issue = [&](uint32_t idesc, bool first, bool last) {
    ok = wait(full(mslot), mph);
    if (!ok) return;
    tc_fence_after();
    if (elect_one()) {
      const uint64_t ad = sw128_desc(sbase + mslot * kStage), bd = sw128_desc(sbase + mslot * kStage + kABytes);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_ss<1, I8>(tmem, ad + 2 * k, bd + 2 * k, idesc, !first || k > 0);
      commit<1>(empty(mslot));
      if (last) commit<1>(acc_full);
    }
    __syncwarp();
    if (++mslot == kStagesLoads) {
      mslot = 0;
      mph ^= 1;
    }
  };
  for (int i = blockIdx.x; i < total && ok; i += gridDim.x) {
    const Tile t = tile_of<1>(g, a, i);
    const uint8_t* x = static_cast<const uint8_t*>(a.g.x) + (long long)t.r0 * a.g.ldx * ES;
    const uint8_t* w = static_cast<const uint8_t*>(a.g.w) + ((long long)t.e * a.g.ldwe + (long long)t.f0 * a.g.ldw) * ES;
    const uint8_t *wr[4], *xr[4];  // this thread's rows
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wr[j] = w + (long long)(lr + 32 * j) * a.g.ldw * ES;
      xr[j] = x + (long long)(lr + 32 * j) * a.g.ldx * ES;
    }
    const uint32_t idesc = a.idesc | ((uint32_t)(t.n >> 3) << 17);
    for (int kb = 0; kb < nk && ok; ++it) {
      const int first = I8 ? 0 : kb, end = I8 ? nk : min(kb + kChunk<TO>, nk);
      for (; kb < end; ++kb) {
        const int b = kb * kRowBytes + lc * 16;
        Chunk16<ES> cw[4], cx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = lr + 32 * j;
          cw[j].load(wr[j], b, len, t.f0 + r < a.g.N);
          cx[j].load(xr[j], b, len, r < t.live);
        }
        // under the loads' latency the stage before this one
        if (warp == 0 && kb > first) {
          if (kb == first + 1 && it > 0) ok = wait(acc_empty, (it - 1) & 1);
          if (ok) issue(idesc, kb == first + 1, false);
          if (!ok) break;
        }
        ok = round == 0 || wait(empty(slot), (round - 1) & 1);
        if (!ok) break;
        uint8_t* dst = sm + slot * kStage + place;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          *reinterpret_cast<uint4*>(dst + j * 32 * kRowBytes) = cw[j].value();
          if (lr + 32 * j < t.n) *reinterpret_cast<uint4*>(dst + kABytes + j * 32 * kRowBytes) = cx[j].value();
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(slot));
        if (++slot == kStagesLoads) {
          slot = 0;
          ++round;
        }
      }
      if (!ok) break;
      if (warp == 0) {
        if (end == first + 1 && it > 0) ok = wait(acc_empty, (it - 1) & 1);
        if (ok) issue(idesc, end == first + 1, true);
        if (!ok) break;
      }
      const int ch0 = t.f0 + quarter * 32;
      float ws = 0.f;
      if constexpr (I8)
        if (ch0 + lane < a.g.N) ws = a.g.ws[(long long)t.e * a.g.N + ch0 + lane];
      ok = wait(acc_full, it & 1);
      if (!ok) break;
      tc_fence_after();
      for (int c0 = half * 32; c0 < t.n; c0 += 64) {
        uint32_t v[32];
        tmem_ld32_nw(acc + c0, v);
        tmem_wait_ld(v);
        if (!I8 && first > 0) {
          uint32_t sum[32];
          tmem_ld32_nw(acc + kSums + c0, sum);
          tmem_wait_ld(sum);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(sum[j]) + __uint_as_float(v[j]));
        }
        if (!I8 && end < nk) {
          tmem_st32(acc + kSums + c0, v);
          continue;
        }
        float xv = 0.f;
        if constexpr (I8)
          if (c0 + lane < t.live) xv = a.g.xs[t.r0 + c0 + lane];
        store_chunk<TO, I8>(a, t, c0, v, ws, xv, stage, xs_s[warp], ch0, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      // no stage is written before every warp's part of a tile has left it
      if (end == nk) ok = wait(acc_empty, it & 1);
    }
  }
  if (!ok) *aborted = 1;
  if (warp == 0) {
    if (elect_one()) mma_commit(drained);
    __syncwarp();
    mbar_wait(drained, 0, status, kDrainLimitNs);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kCols);
  if (threadIdx.x == 0 && status_s) atomicAdd(&g_op_timeouts, 1u);
}
