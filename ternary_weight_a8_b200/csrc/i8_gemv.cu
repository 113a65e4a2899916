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

constexpr int kGvRows = 16;
constexpr int kGvWarps = 8;
constexpr int kGvUnroll = 4;  // chunks in flight per warp

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// TG: groups of 8 tokens.
template <typename TY, int TG>
__global__ void __launch_bounds__(32 * kGvWarps, TG <= 2 ? 4 : 3) i8_gemv_kernel(const I8Args P) {
  __shared__ int part[kGvWarps][8 * TG][kGvRows + 1];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kGvRows;
  const int chunks = P.K >> 6;
  const int c0 = chunks * warp / kGvWarps, c1 = chunks * (warp + 1) / kGvWarps;
  // Rows past N and tokens past M repeat the last one; their sums are dropped.
  const int ra = min(n0 + g, P.N - 1), rb = min(n0 + g + 8, P.N - 1);
  const uint8_t* wa = reinterpret_cast<const uint8_t*>(P.wq) + static_cast<size_t>(ra) * P.K + 16 * t;
  const uint8_t* wb = reinterpret_cast<const uint8_t*>(P.wq) + static_cast<size_t>(rb) * P.K + 16 * t;
  const uint8_t* xp[TG];
#pragma unroll
  for (int j = 0; j < TG; ++j)
    xp[j] = reinterpret_cast<const uint8_t*>(P.xq) + static_cast<size_t>(min(8 * j + g, P.M - 1)) * P.ldx + 16 * t;

  // While the preceding kernel (the quantisation) runs, the first weights
  // come as far as L2, where a write by that kernel would still reach them.
#pragma unroll
  for (int u = 0; u < kGvUnroll; ++u)
    if (c0 + u < c1) {
      prefetch_l2(wa + 64 * (c0 + u));
      prefetch_l2(wb + 64 * (c0 + u));
    }
  griddep_wait();

  int acc[TG][4] = {};
  auto step = [&](int c, auto n_tag) {
    constexpr int U = decltype(n_tag)::value;
    uint4 a[U], b[U], x[U][TG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a[u] = ldg_stream_u4(wa + 64 * (c + u));
      b[u] = ldg_stream_u4(wb + 64 * (c + u));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < TG; ++j) x[u][j] = *reinterpret_cast<const uint4*>(xp[j] + 64 * (c + u));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < TG; ++j) {
        mma_s8(acc[j], a[u].x, b[u].x, a[u].y, b[u].y, x[u][j].x, x[u][j].y);
        mma_s8(acc[j], a[u].z, b[u].z, a[u].w, b[u].w, x[u][j].z, x[u][j].w);
      }
  };
  int c = c0;
  for (; c + kGvUnroll <= c1; c += kGvUnroll) step(c, std::integral_constant<int, kGvUnroll>{});
  for (; c < c1; ++c) step(c, std::integral_constant<int, 1>{});

  // Fragment (row g or g + 8, tokens 2t and 2t + 1) of every group.
#pragma unroll
  for (int j = 0; j < TG; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][8 * j + 2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[j][i];
  __syncthreads();
  TY* y = static_cast<TY*>(P.y);
  for (int i = threadIdx.x; i < 8 * TG * kGvRows; i += 32 * kGvWarps) {
    const int m = i / kGvRows, r = i % kGvRows, n = n0 + r;
    if (m >= P.M || n >= P.N) continue;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kGvWarps; ++w) sum += part[w][m][r];
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

template <typename TY>
cudaError_t launch_i8_gemv_t(const I8Args& a, cudaStream_t stream, bool pdl) {
  const dim3 grid((a.N + kGvRows - 1) / kGvRows), block(32 * kGvWarps);
  if (a.M <= 8) return launch(i8_gemv_kernel<TY, 1>, grid, block, 0, stream, pdl, a);
  if (a.M <= 16) return launch(i8_gemv_kernel<TY, 2>, grid, block, 0, stream, pdl, a);
  return launch(i8_gemv_kernel<TY, 4>, grid, block, 0, stream, pdl, a);
}

}  // namespace

cudaError_t launch_i8_gemv(const I8Args& a, cudaStream_t stream, bool pdl) {
  if (a.M <= 0) return cudaSuccess;
  if (a.M > kI8GemvMaxTokens) return cudaErrorInvalidValue;
  return a.y_type == kOutBF16 ? launch_i8_gemv_t<__nv_bfloat16>(a, stream, pdl) : launch_i8_gemv_t<float>(a, stream, pdl);
}

}  // namespace bl
