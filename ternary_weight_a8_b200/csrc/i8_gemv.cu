// The 8-bit product for a few tokens: y = x . W^T with int8 codes on both
// sides, a scale for each token and each output channel.
//   acc[m][n] = sum_k q[m][k] * wq[n][k]             (int32, exact)
//   y[m][n]   = fp32(acc) * ((1 / s[m]) * (1 / ws[n]))
// Bound by the weights' stream, N * K bytes.  `mma.sync` m16n8k32 carries it:
// per SM the HBM rate brings about 23 weight bytes a clock, one MMA takes 512,
// so 8 tokens need a tenth of the legacy tensor path's rate and 32 tokens
// less than half.
//
// A block takes 16 weight rows; its warps split the row's 64-byte chunks
// between them and join their sums in shared memory.  The MMA's k order is
// free as long as both operands agree on it, so a lane loads 16 consecutive
// bytes of row g and of row g + 8 (g = lane / 4, 16 bytes at 16 * (lane % 4)
// of the chunk) and uses their words as the fragments of two MMAs; a token's
// codes are loaded the same way.  Nothing is staged: the loads go from L2 to
// the fragments, four chunks in flight per warp and four blocks per SM.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace bl {

namespace {

constexpr int kGvWarps = 8;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// TG: groups of 8 tokens; MT: groups of 16 rows; U: chunks in flight per warp.
template <typename TY, int TG, int MT, int U0>
__global__ void __launch_bounds__(32 * kGvWarps, TG * MT >= 8 ? 2 : TG * MT >= 4 ? 3 : 4) i8_gemv_kernel(const I8Args P, int first_wave) {
  constexpr int kRows = 16 * MT;
  __shared__ int sums[8 * TG][kRows + 1];
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < 8 * TG * (kRows + 1); i += 32 * kGvWarps) (&sums[0][0])[i] = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows;
  const int chunks = P.K >> 6;
  const int c0 = chunks * warp / kGvWarps, c1 = chunks * (warp + 1) / kGvWarps;
  // Rows past N and tokens past M repeat the last one; their sums are dropped.
  const uint8_t* wp[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i)
    wp[i] = reinterpret_cast<const uint8_t*>(P.wq) + static_cast<size_t>(min(n0 + g + 8 * i, P.N - 1)) * P.K + 16 * t;
  const uint8_t* xp[TG];
#pragma unroll
  for (int j = 0; j < TG; ++j)
    xp[j] = reinterpret_cast<const uint8_t*>(P.xq) + static_cast<size_t>(min(8 * j + g, P.M - 1)) * P.ldx + 16 * t;

  // While the preceding kernel (the quantisation) runs, the first weights
  // come as far as L2, where a write by that kernel would still reach them.
  if (blockIdx.x < first_wave) {
    if (P.K <= 4096) {
      if (threadIdx.x == 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(P.wq + static_cast<size_t>(n0) * P.K),
                     "r"(min(kRows, P.N - n0) * P.K)
                     : "memory");
    } else {
#pragma unroll
      for (int u = 0; u < U0; ++u)
        if (c0 + u < c1) {
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) prefetch_l2(wp[i] + 64 * (c0 + u));
        }
    }
  }
  griddep_wait();

  int acc[MT][TG][4] = {};
  auto step = [&](int c, auto n_tag) {
    constexpr int U = decltype(n_tag)::value;
    uint4 a[U][2 * MT], x[U][TG];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) a[u][i] = ldg_stream_u4(wp[i] + 64 * (c + u));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < TG; ++j) x[u][j] = *reinterpret_cast<const uint4*>(xp[j] + 64 * (c + u));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < TG; ++j) {
          const uint4 lo = a[u][2 * i], hi = a[u][2 * i + 1];
          mma_s8(acc[i][j], lo.x, hi.x, lo.y, hi.y, x[u][j].x, x[u][j].y);
          mma_s8(acc[i][j], lo.z, hi.z, lo.w, hi.w, x[u][j].z, x[u][j].w);
        }
  };
  int c = c0;
  for (; c + U0 <= c1; c += U0) step(c, std::integral_constant<int, U0>{});
  if constexpr (U0 > 1)
    for (; c < c1; ++c) step(c, std::integral_constant<int, 1>{});

  __syncthreads();  // the sums are zero
  // Fragment (row g or g + 8, tokens 2t and 2t + 1) of every group; integer
  // sums, so the warps' order does not matter.
#pragma unroll
  for (int r = 0; r < MT; ++r)
#pragma unroll
    for (int j = 0; j < TG; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red_shared_add(&sums[8 * j + 2 * t + (i & 1)][16 * r + g + 8 * (i >> 1)], acc[r][j][i]);
  __syncthreads();
  TY* y = static_cast<TY*>(P.y);
  for (int i = threadIdx.x; i < 8 * TG * kRows; i += 32 * kGvWarps) {
    const int m = i / kRows, r = i % kRows, n = n0 + r;
    if (m >= P.M || n >= P.N) continue;
    const int sum = sums[m][r];
    const float f = __fmul_rn(__frcp_rn(__ldg(P.scale + m)), __frcp_rn(__ldg(P.wscale + n)));
    const size_t at = static_cast<size_t>(m) * P.N + n;
    const float v = __fmul_rn(static_cast<float>(sum), f);
    if constexpr (sizeof(TY) == 2) {
      y[at] = __float2bfloat16_rn(v);
    } else {
      y[at] = v;
    }
    if (P.acc_out) P.acc_out[at] = sum;
  }
}

template <typename TY, int TG, int MT, int U>
cudaError_t launch_k(const I8Args& a, cudaStream_t stream, bool pdl) {
  const int blocks = (a.N + 16 * MT - 1) / (16 * MT);
  const int resident = (TG * MT >= 8 ? 2 : TG * MT >= 4 ? 3 : 4) * num_sms();
  int wave = blocks > resident ? resident : blocks <= 2 * num_sms() ? blocks : 0;
  return launch(i8_gemv_kernel<TY, TG, MT, U>, dim3(blocks), dim3(32 * kGvWarps), 0, stream, pdl, a, wave);
}

template <typename TY>
cudaError_t launch_i8_gemv_t(const I8Args& a, cudaStream_t stream, bool pdl) {
  if (a.M <= 8) {
    // Short rows and enough of them for several waves of twice as large blocks
    // (1 token, 2560 -> 128000: 51.7 us, 54.7 with 16 rows; 8 tokens, 8192 ->
    // 28672: 39.5 us, 36.6 with 16 rows; 2560 -> 6912: 6.8 us, 5.3).
    if (a.K <= 4096 && a.N >= 32 * 8 * num_sms()) return launch_k<TY, 1, 2, 2>(a, stream, pdl);
    return launch_k<TY, 1, 1, 4>(a, stream, pdl);
  }
  if (a.M <= 16) return launch_k<TY, 2, 1, 4>(a, stream, pdl);
  return launch_k<TY, 4, 1, 4>(a, stream, pdl);
}

}  // namespace

// Up to 8 tokens always.  More tokens read as many codes as weights or more
// through L1, which only a call short enough for its latency to count gains
// from: 16 tokens, 2560 -> 6912: 5.9 us against 8.7 on the tensor cores, 8640
// -> 3200: 9.9 against 10.4, 2560 -> 128000: 66 against 55; 32 tokens, 2560
// -> 6912: 7.1 against 8.7, 8640 -> 3200: 14.0 against 10.4, 8192 -> 28672:
// 64 against 43.
bool i8_takes_gemv(int M, int N, int K) {
  const long long weights = static_cast<long long>(N) * K;
  return M <= 8 || (M <= 16 && weights <= (64LL << 20)) || (M <= kI8GemvMaxTokens && weights <= (20LL << 20));
}

cudaError_t launch_i8_gemv(const I8Args& a, cudaStream_t stream, bool pdl) {
  if (a.M <= 0) return cudaSuccess;
  if (a.M > kI8GemvMaxTokens) return cudaErrorInvalidValue;
  return a.y_type == kOutBF16 ? launch_i8_gemv_t<__nv_bfloat16>(a, stream, pdl) : launch_i8_gemv_t<float>(a, stream, pdl);
}

}  // namespace bl
