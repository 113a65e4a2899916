// The 8-bit product for many tokens on the 5th-generation tensor cores:
// tcgen05.mma kind::i8, int32 accumulators in tensor memory, the scales of
// token and channel in the epilogue.
//   acc[m][n] = sum_k q[m][k] * wq[n][k]             (int32, exact)
//   y[m][n]   = fp32(acc) * ((1 / s[m]) * (1 / ws[n]))
// Both operands are row-major along k, as the tensor core wants them, so TMA
// brings 128-byte blocks of rows straight into the 128-byte swizzled layout.
//
// One kernel in three shapes:
//   pair   a cluster of two CTAs shares 256 tokens x 256 channels through
//          cta_group::2: each loads its 128 tokens and 128 of the channels;
//   single one CTA, 128 tokens x 32 .. 256 channels (a multiple of 16);
//   split  `single` with a cluster of up to 8 CTAs over the k-blocks of one
//          tile, whose int32 sums meet through distributed shared memory.
// Warps: 0 the TMA producer, 1 the tensor-memory owner and MMA issuer, 4-7
// the epilogue; two accumulators let the epilogue of a tile overlap the next
// tile's products (pair and single are persistent, split is one tile).
// Every mbarrier wait is bounded; one that runs out records the timeout in
// the status word, raises the abort flags and the block winds down.
//
// What bounds it: with many tokens the tensor cores (2048 tokens, 8192 ->
// 28672: 299 - 314 us by the power that is left, 3.06 - 3.22 POPS, where the
// library's 8192^3 product runs at 2.85; 2560 -> 6912: 28 us, 2.6 POPS; with
// fp32 outputs 337 and 31 us), as far as the pairs' whole tiles fill their last
// round: 2048 tokens, 2560 -> 2560 are 80 tiles on 74 pairs and take 19.0 us,
// 44% of the rate; with up to 128 tokens and large matrices the weights'
// stream (32 tokens, 8192 -> 28672: 44.4 us, 5.3 TB/s; 2560 -> 128000: 55 us,
// 6.0 TB/s), which is why the tile width is free: 448 tiles of 64 or 224 of
// 128 channels for 148 SMs leave a quarter of the time idle (the model takes
// 224 channels for 28672, 128 tiles that leave 20 SMs without one, as the
// stream bounds them all the same); and in between the latency of a tile's
// k-blocks, which the split shortens.
// An MMA of one CTA holds the tensor core for about 130 clocks whatever its
// width, so narrow tiles are only as fast as wide ones.
#include <cuda.h>
#include <cuda_bf16.h>
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace bl {

namespace {

constexpr int kBM = 128, kBK = 128;
constexpr int kThreads = 256;
constexpr int kEpiWarps = 4;
constexpr int kMaxSplit = 8;

constexpr int kMaxBN = 256;  // channels of a tile, and tensor-memory columns of an accumulator
constexpr int kMaxStages = 16;

// Shared memory: the ring, the output staging (two 32 x 32 boxes per epilogue
// warp), 1 / ws of the tile's channels (two buffers), barriers.
template <typename TY, int CG>
struct I8Cfg {
  static constexpr int kBoxBytes = 32 * 32 * static_cast<int>(sizeof(TY));
  static constexpr int kOutBytes = kEpiWarps * 2 * kBoxBytes;
  static constexpr int kNumBars = 2 * kMaxStages + 6;
  static constexpr int kTail = 2 * kMaxBN * 4 + kNumBars * 8 + 64;
  static constexpr int kPairStages = sizeof(TY) == 2 ? 6 : 5;
  static constexpr int kRingBytes = (232448 - 1024 - kOutBytes - kTail) / 1024 * 1024;
  static constexpr int kOffOut = kRingBytes;
  static constexpr int kOffRw = kOffOut + kOutBytes;
  static constexpr int kOffBar = kOffRw + 2 * kMaxBN * 4;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;  // + alignment slack
  static constexpr uint32_t kTmemCols = 2 * kMaxBN;
  static_assert(kSmemBytes <= 232448, "shared memory per block");
  static_assert(kPairStages * 32768 <= kRingBytes && kBM * kMaxBN * 4 <= kRingBytes, "ring");
  static_assert(kOffOut % 1024 == 0, "swizzled staging alignment");
};

// Set by every wait of this file that runs out on the device, whatever
// workspace its call was given: a call without one has no status word that its
// caller could read, nor has a replayed graph.
__device__ uint32_t g_status;

// Bounded wait; in the pair form giving up raises the peer's abort flag too.
template <int CG>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const WaitCtl& ctl, uint32_t peer_abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity, 200000u)) return true;
    if (*ctl.abort) return false;
    if (global_ns() - t0 > ctl.limit_ns) {
      *ctl.abort = 1;
      if (CG == 2) st_shared_cluster_u32(peer_abort, 1u);
      if (ctl.status) {
        atomicOr(ctl.status, kStatusTimeout);
        atomicOr(&g_status, kStatusTimeout);
      }
      return false;
    }
  }
}

template <int CG>
__device__ __forceinline__ void commit_both(uint32_t bar) {
  if constexpr (CG == 1) {
    tc_commit(bar);
  } else {
    tc_commit_pair_mc(bar, static_cast<uint16_t>(0x3));
  }
}

// Barrier of the four epilogue warps; true in all of them if any of them says so.
__device__ __forceinline__ bool epi_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

struct I8Tiles {
  int m_tiles, n_tiles, kblocks, split;
  int bn;      // channels per tile (a multiple of 16)
  int rows_a;  // token rows that a load of x brings (of 128; the rest of the tile is never looked at)
  int stages;
};

template <typename TY>
__device__ __forceinline__ TY to_out(float v) {
  if constexpr (sizeof(TY) == 2) {
    return __float2bfloat16_rn(v);
  } else {
    return v;
  }
}

// Byte of 16-byte piece j of row `lane` in a staged 32 x 32 box: the swizzle
// of the box's tensor map (64-byte rows for bf16, 128-byte rows for fp32), so
// that the lanes' stores meet no bank conflict.
template <typename TY>
__device__ __forceinline__ int box_at(int row, int j) {
  if constexpr (sizeof(TY) == 2) {
    return row * 64 + ((j ^ ((row >> 1) & 3)) << 4);
  } else {
    return row * 128 + ((j ^ (row & 7)) << 4);
  }
}

// The first 16 of a row's values (fp32 bits), 16-byte aligned.
template <typename TY>
__device__ __forceinline__ void store16(TY* y, const uint32_t (&r)[32]) {
  uint4* d = reinterpret_cast<uint4*>(y);
  if constexpr (sizeof(TY) == 2) {
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      p[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    d[0] = make_uint4(p[0], p[1], p[2], p[3]);
    d[1] = make_uint4(p[4], p[5], p[6], p[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
  }
}

template <typename TY, int CG>
__global__ void __launch_bounds__(kThreads) i8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x,
                                                           const __grid_constant__ CUtensorMap tmap_w,
                                                           const __grid_constant__ CUtensorMap tmap_y, int tma_out,
                                                           const I8Args P, const I8Tiles T) {
  using C = I8Cfg<TY, CG>;
  const int bn = CG == 2 ? 256 : T.bn, stages = CG == 2 ? C::kPairStages : T.stages;
  const int a_bytes = kBM * kBK, stage_bytes = a_bytes + bn / CG * kBK;
  const int load_bytes = (CG == 2 ? kBM : T.rows_a) * kBK + bn / CG * kBK;
  // Instruction descriptor: D s32, A s8, B s8, both K-major, N = bn, M = 128 * CG.
  const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(bn >> 3) << 17) | (((kBM * CG) >> 4) << 24);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto full_bar = [&](int i) { return sb + C::kOffBar + 8 * i; };
  auto empty_bar = [&](int i) { return sb + C::kOffBar + 8 * (kMaxStages + i); };
  auto tfull_bar = [&](int i) { return sb + C::kOffBar + 8 * (2 * kMaxStages + i); };
  auto tempty_bar = [&](int i) { return sb + C::kOffBar + 8 * (2 * kMaxStages + 2 + i); };
  const uint32_t done_bar = sb + C::kOffBar + 8 * (C::kNumBars - 2);
  const uint32_t done2_bar = sb + C::kOffBar + 8 * (C::kNumBars - 1);  // the split's sums of this CTA's rows
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 16);
  volatile int* never = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool split = CG == 1 && T.split > 1;
  const uint32_t crank = (CG == 2 || split) ? cluster_ctarank() : 0u;
  const uint32_t rank = CG == 2 ? crank : 0u;  // half of the pair
  const uint32_t peer_abort = CG == 2 ? mapa_shared(sb + C::kOffMisc + 16, rank ^ 1u) : 0u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full_bar(i), 1);   // the even CTA's expect-tx arrive (bytes of both CTAs)
      mbar_init(empty_bar(i), 1);  // MMA commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), kEpiWarps * CG);
    }
    mbar_init(done_bar, 1);
    mbar_init(done2_bar, 1);
    *abort_flag = 0;
    *never = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_w);
  }
  if (warp == 1) {
    if constexpr (CG == 1) {
      tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
      tmem_relinquish();
    } else {
      tmem_alloc_pair(smem_u32(tmem_slot), C::kTmemCols);
      tmem_relinquish_pair();
    }
  }
  tc_fence_before();
  if (CG == 2 || split) {
    cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();

  const WaitCtl ctl{P.status, abort_flag, kWaitLimitNs};
  const int tiles = T.m_tiles * T.n_tiles;
  const int group = CG == 2 ? 2 : T.split;
  const int first = blockIdx.x / group, stride = gridDim.x / group;
  const int pitch = (bn + 31) / 32 * 128;  // bytes of a token's sums in the split form
  // This CTA's k-blocks: all of them, or its share of the split's.
  const int kb0 = split ? T.kblocks * static_cast<int>(crank) / T.split : 0;
  const int kb1 = split ? T.kblocks * (static_cast<int>(crank) + 1) / T.split : T.kblocks;

  if (warp == 0) {
    if (lane == 0) {
      // The weights' first blocks come as far as L2 while the preceding kernel
      // (the quantisation) runs; a write by that kernel would still reach them.
      if (first < tiles) {
        const int row = (first / T.m_tiles) * bn + static_cast<int>(rank) * (bn / CG);
        for (int kb = kb0; kb < kb1 && kb < kb0 + stages; ++kb)
          asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(
                           reinterpret_cast<uint64_t>(&tmap_w)),
                       "r"(kb * kBK), "r"(row)
                       : "memory");
      }
      griddep_wait();
      int it = 0, s = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int tile = first; ok && tile < tiles; tile += stride) {
        const int mt = tile % T.m_tiles, nt = tile / T.m_tiles;
        const int arow = mt * kBM * CG + static_cast<int>(rank) * kBM;
        const int brow = nt * bn + static_cast<int>(rank) * (bn / CG);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          if (!wait_bar<CG>(empty_bar(s), ph, ctl, peer_abort)) {
            ok = false;
            break;
          }
          const uint32_t a = sb + s * stage_bytes, b = a + a_bytes;
          if constexpr (CG == 1) {
            mbar_arrive_expect_tx(full_bar(s), load_bytes);
            tma_load_2d(b, &tmap_w, kb * kBK, brow, full_bar(s));
            tma_load_2d(a, &tmap_x, kb * kBK, arow, full_bar(s));
          } else {
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * load_bytes);
            const uint32_t bar = mapa_shared(full_bar(s), 0);
            tma_load_2d_pair(a, &tmap_x, kb * kBK, arow, bar);
            tma_load_2d_pair(b, &tmap_w, kb * kBK, brow, bar);
          }
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {
        // Let copies in flight land before the block's shared memory goes away.
        const WaitCtl drain{nullptr, never, 100000000ull};
        if constexpr (CG == 1) {
          for (int i = (it > stages ? it - stages : 0); i < it; ++i)
            wait_bar<1>(full_bar(i % stages), (i / stages) & 1, drain, 0u);
        } else {
          const uint64_t t0 = global_ns();
          while (global_ns() - t0 < 1000000ull) __nanosleep(10000);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      griddep_wait();  // so that the bounded waits below begin when the copies do
      int tc = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true, issued = false;
      for (int tile = first; ok && tile < tiles; tile += stride, ++tc) {
        const int a = tc & 1;
        if (!wait_bar<CG>(tempty_bar(a), ((tc >> 1) & 1) ^ 1, ctl, peer_abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + a * kMaxBN;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bar<CG>(full_bar(s), ph, ctl, peer_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t adesc = sw128_kmajor_desc(sb + s * stage_bytes);
          const uint64_t bdesc = sw128_kmajor_desc(sb + s * stage_bytes + a_bytes);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k) {
            if constexpr (CG == 1) {
              tc_mma_i8(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, kb != kb0 || k != 0);
            } else {
              tc_mma_i8_pair(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, kb != kb0 || k != 0);
            }
          }
          issued = true;
          commit_both<CG>(empty_bar(s));
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok) commit_both<CG>(tfull_bar(a));
      }
      if (issued) {
        // Every MMA must be finished before tensor memory is released.
        if constexpr (CG == 1) {
          tc_commit(done_bar);
        } else {
          tc_commit_pair(done_bar);
        }
        const WaitCtl drain{nullptr, never, 100000000ull};
        wait_bar<1>(done_bar, 0, drain, 0u);
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3;  // tensor-memory lane quarter this warp may read
    griddep_wait();          // the scales come from the preceding kernel; y may be read by it
    if (split) {
      // The tile's reciprocal scales, for the finish: channels, then tokens.
      if (first < tiles) {
        float* rec = reinterpret_cast<float*>(smem + C::kOffRw);
        for (int i = threadIdx.x - 128; i < bn + kBM; i += 128) {
          const bool ch = i < bn;
          const int at = ch ? (first / T.m_tiles) * bn + i : (first % T.m_tiles) * kBM + i - bn;
          rec[ch ? i : kMaxBN + i - bn] =
              at < (ch ? P.N : P.M) ? __frcp_rn(__ldcg((ch ? P.wscale : P.scale) + at)) : 0.0f;
        }
      }
      // The int32 sums of this CTA's k-blocks, token rows of BN, over the ring
      // (whose copies have all been consumed once the products are done).
      if (first < tiles) {
        const bool got = wait_bar<1>(tfull_bar(0), 0, ctl, 0u);
        if (__all_sync(0xffffffffu, got)) {
          tc_fence_after();
          const int mt = first % T.m_tiles;
          const int row = q * 32 + lane;
          if (mt * kBM + q * 32 < P.M) {  // warp-uniform: some token of this warp exists
#pragma unroll 1
            for (int c = 0; c < pitch / 128; ++c) {
              uint32_t r[32];
              tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c * 32, r);
              tmem_ld_wait();
              // 16-byte pieces, rotated by the row so that the lanes' stores spread over the banks.
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(smem + row * pitch + (((8 * c + j) ^ (row & 7)) << 4)) =
                    make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            }
          }
          tc_fence_before();
        }
      }
    } else {
      float* rw = reinterpret_cast<float*>(smem + C::kOffRw);
      uint8_t* obuf = smem + C::kOffOut + (warp - 4) * 2 * C::kBoxBytes;
      if (tma_out && lane == 0) tma_prefetch_desc(&tmap_y);
      int ob = 0, tc = 0;
      bool failed = false;
      for (int tile = first; tile < tiles; tile += stride, ++tc) {
        const int mt = tile % T.m_tiles, nt = tile / T.m_tiles;
        const int a = tc & 1;
        // 1 / ws of the tile's channels: written once by the four warps.  The
        // buffer was last read two tiles ago, before the barrier of the last tile.
        float* rwt = rw + a * kMaxBN;
        for (int i = threadIdx.x - 128; i < bn; i += 128) {
          const int n = nt * bn + i;
          rwt[i] = n < P.N ? __frcp_rn(__ldcg(P.wscale + n)) : 0.0f;
        }
        // One of the four gave up: all leave together (a warp that left alone would strand the rest here).
        if (epi_any(failed)) break;
        const int m0 = mt * kBM * CG + static_cast<int>(rank) * kBM + q * 32;  // first token of this warp
        const int m = m0 + lane;
        const float rs = m < P.M ? __frcp_rn(__ldcg(P.scale + m)) : 0.0f;
        // tcgen05.ld below is warp-collective: take the wait's outcome warp-wide.
        const bool got = wait_bar<CG>(tfull_bar(a), (tc >> 1) & 1, ctl, peer_abort);
        const bool go = __all_sync(0xffffffffu, got);
        if (go) {
          tc_fence_after();
          const int n_end = min(P.N, nt * bn + bn);
#pragma unroll 1
          for (int c = 0; c < kMaxBN / 32; ++c) {
            const int n0 = nt * bn + c * 32;
            if (n0 >= n_end || m0 >= P.M) break;  // warp-uniform
            const bool boxed = n0 + 32 <= n_end || n_end == P.N;  // not the last 16 columns of a tile
            uint32_t r[32];
            tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * kMaxBN + c * 32, r);
            tmem_ld_wait();
            if (P.acc_out && m < P.M) {
              int32_t* ar = P.acc_out + static_cast<size_t>(m) * P.N + n0;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (n0 + i < n_end) ar[i] = static_cast<int32_t>(r[i]);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 w = *reinterpret_cast<const float4*>(rwt + c * 32 + i);
              const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                r[i + e] = __float_as_uint(
                    __fmul_rn(static_cast<float>(static_cast<int32_t>(r[i + e])), __fmul_rn(rs, f[e])));
            }
            if (tma_out && !boxed) {
              // Half a box: 16 columns, which the lane writes itself.
              if (m < P.M) store16<TY>(static_cast<TY*>(P.y) + static_cast<size_t>(m) * P.N + n0, r);
              continue;
            }
            uint8_t* b = obuf + ob * C::kBoxBytes;
            if (tma_out) {
              // The buffer's previous box (two groups ago) must have been read.
              if (lane == 0) bulk_wait_group_read<1>();
              __syncwarp();
            }
            if constexpr (sizeof(TY) == 2) {
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                p[i] = *reinterpret_cast<const uint32_t*>(&h);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(b + box_at<TY>(lane, j)) =
                    make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(b + box_at<TY>(lane, j)) =
                    make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            }
            if (tma_out) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmap_y, smem_u32(b), n0, m0);
                bulk_commit_group();
              }
              ob ^= 1;
            } else {
              // Rows that are no multiple of 16 bytes: the lanes take a row's columns together.
              __syncwarp();
              constexpr int kE = 16 / static_cast<int>(sizeof(TY));
              const int rows = min(32, P.M - m0);
              if (n0 + lane < n_end) {
                TY* yp = static_cast<TY*>(P.y) + static_cast<size_t>(m0) * P.N + n0 + lane;
                for (int i = 0; i < rows; ++i)
                  yp[static_cast<size_t>(i) * P.N] =
                      *reinterpret_cast<const TY*>(b + box_at<TY>(i, lane / kE) + (lane % kE) * sizeof(TY));
              }
              __syncwarp();
            }
          }
          tc_fence_before();
        }
        failed = !go;
        __syncwarp();
        if (go && lane == 0) {
          if constexpr (CG == 1) {
            mbar_arrive(tempty_bar(a));
          } else {
            mbar_arrive_cluster(mapa_shared(tempty_bar(a), 0));
          }
        }
      }
      if (tma_out && lane == 0) bulk_wait_group_all();  // stores done before shared memory goes away
    }
  }

  tc_fence_before();
  if (split) {
    // The cluster's sums meet: CTA c finishes the c-th share of the token rows.
    // Every CTA adds its rows of another's share into that CTA's shared memory
    // with one bulk reduction (single loads from a neighbour's shared memory
    // came at 7 bytes a clock); int32 sums, so their order does not matter.
    const int mt = first % T.m_tiles, nt = first / T.m_tiles;
    const int rows = min(kBM, P.M - mt * kBM), share = (rows + T.split - 1) / T.split;
    auto rows_of = [&](int c) { return max(0, min(share, rows - c * share)); };
    const int mine = rows_of(static_cast<int>(crank)), row0 = static_cast<int>(crank) * share;
    fence_proxy_async_smem();  // the sums just written are read by the bulk reductions
    if (threadIdx.x == 0 && mine > 0) mbar_arrive_expect_tx(done2_bar, (T.split - 1) * mine * pitch);
    cluster_sync_all();
    griddep_wait();  // every warp writes y here
    const bool good = !*abort_flag;
    if (threadIdx.x == 0 && good) {
      for (int i = 1; i < T.split; ++i) {
        const int c = (static_cast<int>(crank) + i) % T.split, n = rows_of(c);
        if (n > 0) {
          const uint32_t src = sb + c * share * pitch;
          asm volatile(
              "cp.reduce.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes.add.s32 [%0], [%1], %2, "
              "[%3];" ::"r"(mapa_shared(src, static_cast<uint32_t>(c))),
              "r"(src), "r"(n * pitch), "r"(mapa_shared(done2_bar, static_cast<uint32_t>(c)))
              : "memory");
        }
      }
    }
    if (good && mine > 0 && wait_bar<1>(done2_bar, 0, ctl, 0u)) {
      const int pieces = bn / 4;  // of four channels
      const float* rec = reinterpret_cast<const float*>(smem + C::kOffRw);
      const bool vec = P.N % 4 == 0;
      for (int i = threadIdx.x; i < mine * pieces; i += kThreads) {
        const int row = row0 + i / pieces, j = i % pieces;
        const int n = nt * bn + 4 * j, m = mt * kBM + row;
        if (n >= P.N) continue;
        const int4 v = *reinterpret_cast<const int4*>(smem + row * pitch + ((j ^ (row & 7)) << 4));
        const int sum[4] = {v.x, v.y, v.z, v.w};
        const float rs = rec[kMaxBN + row];
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[e] = __fmul_rn(static_cast<float>(sum[e]), __fmul_rn(rs, rec[4 * j + e]));
        const size_t o = static_cast<size_t>(m) * P.N + n;
        TY* yp = static_cast<TY*>(P.y) + o;
        if (vec) {
          if constexpr (sizeof(TY) == 2) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
            *reinterpret_cast<uint2*>(yp) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          } else {
            *reinterpret_cast<float4*>(yp) = make_float4(f[0], f[1], f[2], f[3]);
          }
          if (P.acc_out) *reinterpret_cast<int4*>(P.acc_out + o) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < P.N) {
              yp[e] = to_out<TY>(f[e]);
              if (P.acc_out) P.acc_out[o + e] = sum[e];
            }
        }
      }
    }
    if (!good && threadIdx.x == 0) {
      // Given up: what the others already sent here gets a fixed millisecond to land.
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 1000000ull) __nanosleep(10000);
    }
    cluster_sync_all();  // no CTA leaves while its sums are being read
  } else if constexpr (CG == 2) {
    cluster_sync_all();  // no CTA leaves while its peer may still signal it
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 1) {
      tmem_dealloc(tmem_base, C::kTmemCols);
    } else {
      tmem_dealloc_pair(tmem_base, C::kTmemCols);
    }
  }
}

// A wait that nothing ends (see launch_i8_wait_timeout_selftest).
__global__ void i8_wait_timeout_selftest_kernel(uint32_t* status, unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  griddep_wait();
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    fence_barrier_init();
    const WaitCtl ctl{status, &abort_flag, limit_ns};
    wait_bar<1>(smem_u32(&bar), 0, ctl, 0u);
  }
}

bool map_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t pitch, uint32_t box_inner,
            uint32_t box_outer, CUtensorMapSwizzle swz, CUtensorMapDataType type) {
  EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {pitch};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How many clusters of `size` CTAs the device holds at once (one CTA per SM;
// the SMs of a cluster share a GPC, so this is less than SMs / size), asked
// once per device.
template <typename TY, int CG>
int resident_clusters(int size) {
  static std::atomic<int> known[64][kMaxSplit + 1];
  if (size == 1) return num_sms();
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) dev = -1;
  int n = dev >= 0 ? known[dev][size].load(std::memory_order_acquire) : 0;
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() / size * size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = I8Cfg<TY, CG>::kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, i8_gemm_kernel<TY, CG>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (n < 1) n = 1;
  if (n > num_sms() / size) n = num_sms() / size;
  if (dev >= 0) known[dev][size].store(n, std::memory_order_release);
  return n;
}

template <typename TY, int CG>
cudaError_t set_attributes() {
  static std::atomic<uint64_t> attr_done{0};
  return once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(i8_gemm_kernel<TY, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                I8Cfg<TY, CG>::kSmemBytes);
  });
}

template <typename TY, int CG>
cudaError_t launch_t(const I8Args& a, int bn, int split, cudaStream_t stream, bool pdl) {
  using C = I8Cfg<TY, CG>;
  const int rows_a = a.M < kBM ? (a.M + 7) / 8 * 8 : kBM;
  CUtensorMap tx, tw, ty = {};
  if (!map_2d(&tx, a.xq, a.K, a.M, a.K, kBK, rows_a, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
      !map_2d(&tw, a.wq, a.K, a.N, a.K, kBK, bn / CG, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8))
    return cudaErrorInvalidValue;
  const uint64_t pitch = static_cast<uint64_t>(a.N) * sizeof(TY);
  const int tma_out = split == 1 && pitch % 16 == 0;
  if (tma_out && !map_2d(&ty, a.y, a.N, a.M, pitch, 32, 32,
                         sizeof(TY) == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                         sizeof(TY) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32))
    return cudaErrorInvalidValue;
  const int cluster = CG == 2 ? 2 : split;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (cluster > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = cluster;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  int stages = C::kRingBytes / ((kBM + bn / CG) * kBK);
  if (stages > kMaxStages) stages = kMaxStages;
  const I8Tiles T{(a.M + kBM * CG - 1) / (kBM * CG), (a.N + bn - 1) / bn, (a.K + kBK - 1) / kBK, split, bn, rows_a,
                  stages};
  int groups = T.m_tiles * T.n_tiles;  // the split form: one tile per cluster
  if (split == 1) groups = std::min(groups, resident_clusters<TY, CG>(CG));
  cfg.gridDim = dim3(cluster * groups);
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = na + 1;
  }
  return cudaLaunchKernelEx(&cfg, i8_gemm_kernel<TY, CG>, tx, tw, ty, tma_out, a, T);
}

template <typename TY>
cudaError_t launch_i8_gemm_t(const I8Args& a, cudaStream_t stream, bool pdl) {
  cudaError_t e = set_attributes<TY, 1>();
  if (e == cudaSuccess) e = set_attributes<TY, 2>();
  if (e != cudaSuccess) return e;
  const int sms = num_sms();
  auto ceil_div = [](int x, int y) { return (x + y - 1) / y; };
  const int kblocks = ceil_div(a.K, kBK);
  // Pairs when their tiles fill most of the SMs.
  if (a.M > kBM && 2LL * ceil_div(a.M, 256) * ceil_div(a.N, 256) >= sms * 3 / 4)
    return launch_t<TY, 2>(a, 256, 1, stream, pdl);
  // Else single CTAs, on the tile width and the split that a model of the
  // kernel's time (in ns, from sweeps of both at 24 to 512 tokens) finds best:
  //  - a k-block takes at least 277 ns: its four MMAs hold the tensor core for
  //    130 clocks each whatever the width (20 k-blocks of 2560 inputs 8.4 us
  //    at 32 channels, 9.5 us at 160); what it loads comes at 85 bytes a ns at
  //    most for one SM, and the weights at 6500 for all of them;
  //  - a tile ends in about 300 ns;
  //  - a split adds its cluster and the meeting of its sums: 47 tokens,
  //    2560 -> 2560: 8.9 us whole, 7.0 us in four; 128 tokens, 2560 -> 6912:
  //    9.6 us whole, 10.4 us in two.
  const int mt = ceil_div(a.M, kBM), rows = a.M < kBM ? (a.M + 7) / 8 * 8 : kBM;
  long long best = -1;
  int bn = 64, split = 1;
  for (int s = 1; s <= kMaxSplit && (s == 1 || 2 * s <= kblocks); ++s) {
    const int clusters = resident_clusters<TY, 1>(s);
    for (int w = 32; w <= kMaxBN; w += 16) {
      const long long tiles = static_cast<long long>(mt) * ceil_div(a.N, w);
      if (s > 1 && tiles > clusters) continue;  // the split form is one wave
      const long long rounds = (tiles * s + sms - 1) / sms;
      const long long ctas = tiles * s < sms ? tiles * s : sms;
      long long block = 277;
      block = std::max(block, (w + rows) * 128LL / 85);
      block = std::max(block, w * 128LL * ctas / 6500);
      long long cost = rounds * (ceil_div(kblocks, s) * block + 300);
      if (s > 1) cost += 1900 + 60 * s + rows * w / s * 3 / 10;
      if (best < 0 || cost < best) {
        best = cost;
        bn = w;
        split = s;
      }
    }
  }
  return launch_t<TY, 1>(a, bn, split, stream, pdl);
}

}  // namespace

cudaError_t launch_i8_wait_timeout_selftest(uint32_t* status, int limit_us, cudaStream_t stream) {
  return launch(i8_wait_timeout_selftest_kernel, dim3(1), dim3(32), 0, stream, true, status,
                static_cast<unsigned long long>(limit_us) * 1000ull);
}

cudaError_t take_i8_status(uint32_t* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(*word));
  if (e != cudaSuccess || *word == 0) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
}

cudaError_t launch_i8_gemm(const I8Args& a, cudaStream_t stream, bool pdl) {
  if (a.M <= 0) return cudaSuccess;
  return a.y_type == kOutBF16 ? launch_i8_gemm_t<__nv_bfloat16>(a, stream, pdl) : launch_i8_gemm_t<float>(a, stream, pdl);
}

}  // namespace bl
