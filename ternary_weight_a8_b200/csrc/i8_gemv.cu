// The 8-bit product for a few tokens: y = x . W^T with int8 codes on both
// sides, a scale for each token and each output channel.
//   acc[m][n] = sum_k q[m][k] * wq[n][k]             (int32, exact)
//   y[m][n]   = fp32(acc) * ((1 / s[m]) * (1 / ws[n]))
// Bound by the weights' stream, N * K bytes.  `mma.sync` m16n8k32 carries it:
// per SM the HBM rate brings about 23 weight bytes a clock, one MMA takes 512,
// so 8 tokens need a tenth of the legacy tensor path's rate and 32 tokens
// less than half.
//
// A block takes 16 (or 32) weight rows; its warps split the rows' 64-byte
// chunks between them and join their sums in shared memory.  The MMA's k order
// is free as long as both operands agree on it, so a lane loads 16 consecutive
// bytes of row g and of row g + 8 (g = lane / 4, 16 bytes at 16 * (lane % 4)
// of the chunk) and uses their words as the fragments of two MMAs; a token's
// codes are loaded the same way.  Nothing is staged: the loads go from L2 to
// the fragments, four chunks in flight per warp and four blocks per SM (32-byte
// loads, which touch half as many lines at a time, were faster on short calls
// by up to 8% and slower on the long ones by 10 to 20%).
//
// Measured: 1 token, 2560 -> 128000: 52 - 55 us (5.9 - 6.3 TB/s, 90 - 97% of
// the copy rate by box); 8 tokens, 8192 -> 28672: 36.6 - 38.7 us (93 - 98%);
// short calls are latency: 1 token, 2560 -> 6912: 5.1 us, of which the weights
// need 2.7 and an empty launch 2.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "pairs.cuh"

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

// The codes of up to 8 raw tokens, made by the whole block in shared memory
// (rows `pitch` bytes apart), and their scales: quant_act's arithmetic.
template <typename TX>
__device__ __forceinline__ void block_codes(const I8Args& P, int8_t* codes, int pitch, float* scales) {
  __shared__ uint32_t top_of[kGvWarps], number_of[kGvWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = P.M == 1 ? kGvWarps : P.M == 2 ? 4 : P.M <= 4 ? 2 : 1;  // warps of a token
  const int m = warp / per, tid = warp % per * 32 + lane, step = 32 * per, chunks = P.K / kPer<TX>;
  const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const TX*>(P.x) + static_cast<size_t>(m) * P.K);
  // A thread's first chunks stay in registers between the two passes.
  constexpr int kKeep = 4;
  uint4 keep[kKeep];
  // The largest |value| as bits, and the largest that is no NaN.
  uint32_t top = 0, number = 0;
  auto look = [&](const uint4& v) {
    const uint32_t t = absmax_bits<TX>(absmax16<TX>(0, v));
    top = max(top, t);
    number = max(number, t <= 0x7f800000u ? t : __float_as_uint(absmax_any<TX>(v)));
  };
  if (m < P.M) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (tid + i * step < chunks) keep[i] = xr[tid + i * step];
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (tid + i * step < chunks) look(keep[i]);
    for (int c = tid + kKeep * step; c < chunks; c += step) look(xr[c]);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  number = __reduce_max_sync(0xffffffffu, number);
  if (lane == 0) {
    top_of[warp] = top;
    number_of[warp] = number;
  }
  __syncthreads();
  if (m < P.M) {
    for (int i = 0; i < per; ++i) {
      top = max(top, top_of[m * per + i]);
      number = max(number, number_of[m * per + i]);
    }
    const float s = __fdiv_rn(127.0f, fmaxf(__uint_as_float(number), 1e-5f));
    const f32x2 s2 = pack2(s, s);
    int8_t* row = codes + m * pitch;
    if (top < 0x7f800000u) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int c = tid + i * step;
        if (c < chunks) store_codes<TX>(keep[i], s2, row + c * kPer<TX>);
      }
      for (int c = tid + kKeep * step; c < chunks; c += step) store_codes<TX>(xr[c], s2, row + c * kPer<TX>);
    } else {
      for (int c = tid; c < chunks; c += step) store_codes_any<TX>(xr[c], s, row + c * kPer<TX>);
    }
    if (tid == 0) scales[m] = s;
  }
  __syncthreads();
}

// TG: groups of 8 tokens; MT: groups of 16 rows; U: chunks in flight per warp.
// TX: the type of raw tokens that the block quantises itself, or int8_t for
// codes.
template <typename TX, typename TY, int TG, int MT, int U0>
__global__ void __launch_bounds__(32 * kGvWarps, sizeof(TX) > 1 || TG * MT >= 4 ? 3 : 4)
    i8_gemv_kernel(const I8Args P, int first_wave) {
  constexpr bool kRaw = sizeof(TX) > 1;
  constexpr int kRows = 16 * MT;
  extern __shared__ uint4 raw_codes[];
  __shared__ int sums[8 * TG][kRows + 1];
  __shared__ float raw_scales[8];
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
  // Raw tokens' codes lie an odd number of 64 bytes apart, so that the pieces
  // of two neighbouring tokens fall into different halves of the banks.
  const int pitch = kRaw ? P.K | 64 : P.ldx;
  const uint8_t* xp[TG];
#pragma unroll
  for (int j = 0; j < TG; ++j)
    xp[j] = reinterpret_cast<const uint8_t*>(kRaw ? reinterpret_cast<const int8_t*>(raw_codes) : P.xq) +
            static_cast<size_t>(min(8 * j + g, P.M - 1)) * pitch + 16 * t;

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
  auto fetch = [&](int c, auto& a, auto n_tag) {
    constexpr int U = decltype(n_tag)::value;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) a[u][i] = ldg_stream_u4(wp[i] + 64 * (c + u));
  };
  auto use = [&](int c, auto& a, auto n_tag) {
    constexpr int U = decltype(n_tag)::value;
    uint4 x[U][TG];
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
  const std::integral_constant<int, U0> full{};
  const std::integral_constant<int, 1> one{};
  int c = c0;
  if constexpr (kRaw) {
    // The first weights are under way while the block quantises.
    uint4 first[U0][2 * MT];
    const bool some = c0 + U0 <= c1;
    if (some) fetch(c0, first, full);
    block_codes<TX>(P, reinterpret_cast<int8_t*>(raw_codes), pitch, raw_scales);
    if (some) {
      use(c0, first, full);
      c += U0;
    }
  }
  for (; c + U0 <= c1; c += U0) {
    uint4 a[U0][2 * MT];
    fetch(c, a, full);
    use(c, a, full);
  }
  if constexpr (U0 > 1)
    for (; c < c1; ++c) {
      uint4 a[1][2 * MT];
      fetch(c, a, one);
      use(c, a, one);
    }

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
    const float f = __fmul_rn(__frcp_rn(kRaw ? raw_scales[m] : __ldg(P.scale + m)), __frcp_rn(__ldg(P.wscale + n)));
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

template <typename TX, typename TY, int TG, int MT, int U>
cudaError_t launch_k(const I8Args& a, cudaStream_t stream, bool pdl) {
  const int blocks = (a.N + 16 * MT - 1) / (16 * MT);
  const int resident = (sizeof(TX) > 1 || TG * MT >= 4 ? 3 : 4) * num_sms();
  // Blocks whose first weights are fetched into L2 ahead.  Where the grid is
  // one wave of more than two blocks per SM and nothing has to be quantised
  // first, the extra requests cost more than they hide (1 token, 2560 -> 6912:
  // 5.1 us without, 5.3 with; 2560 -> 2560: 3.8 and 3.6; 2560 -> 128000: 56.2
  // and 54.2, or 70 when later waves fetch ahead too).
  constexpr bool kRaw = sizeof(TX) > 1;
  const int wave = blocks > resident ? resident : kRaw || blocks <= 2 * num_sms() ? blocks : 0;
  const size_t smem = kRaw ? static_cast<size_t>(a.M) * (a.K | 64) : 0;
  return launch(i8_gemv_kernel<TX, TY, TG, MT, U>, dim3(blocks), dim3(32 * kGvWarps), smem, stream, pdl, a, wave);
}

template <typename TY>
cudaError_t launch_i8_gemv_t(const I8Args& a, cudaStream_t stream, bool pdl) {
  if (a.x) return a.x_bf16 ? launch_k<__nv_bfloat16, TY, 1, 1, 4>(a, stream, pdl) : launch_k<float, TY, 1, 1, 4>(a, stream, pdl);
  if (a.M <= 8) {
    // Short rows and enough of them for several waves of twice as large blocks
    // (1 token, 2560 -> 128000: 51.7 us, 54.7 with 16 rows; 8 tokens, 8192 ->
    // 28672: 39.5 us, 36.6 with 16 rows; 2560 -> 6912: 6.8 us, 5.3).
    if (a.K <= 4096 && a.N >= 32 * 8 * num_sms()) return launch_k<int8_t, TY, 1, 2, 2>(a, stream, pdl);
    return launch_k<int8_t, TY, 1, 1, 4>(a, stream, pdl);
  }
  if (a.M <= 16) return launch_k<int8_t, TY, 2, 1, 4>(a, stream, pdl);
  return launch_k<int8_t, TY, 4, 1, 4>(a, stream, pdl);
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

// One wave of blocks can afford to quantise the tokens in every block, when
// that is short: one or two tokens, or at most the four chunks a thread keeps
// in registers (1 token, 2560 -> 6912: 6.0 us, 6.6 with a launch for the
// codes; 8192 -> 2560: 8.3 and 9.7; 4 tokens, 2560 -> 2560: 5 chunks a thread,
// 5.6 and 5.4; 8 tokens, 2048 -> 4096: 8 chunks, 6.4 and 5.2).  The codes have
// to fit beside the blocks of an SM.
bool i8_gemv_quantises(int M, int N, int K, int x_bf16) {
  const int warps = M == 1 ? kGvWarps : M == 2 ? 4 : M <= 4 ? 2 : 1;
  const int chunks = K / (x_bf16 ? 8 : 4);
  return M <= 8 && static_cast<long long>(M) * K <= kI8RawMax && (N + 15) / 16 <= 3 * num_sms() &&
         (M <= 2 || chunks <= 4 * 32 * warps);
}

cudaError_t launch_i8_gemv(const I8Args& a, cudaStream_t stream, bool pdl) {
  if (a.M <= 0) return cudaSuccess;
  if (a.M > kI8GemvMaxTokens) return cudaErrorInvalidValue;
  return a.y_type == kOutBF16 ? launch_i8_gemv_t<__nv_bfloat16>(a, stream, pdl) : launch_i8_gemv_t<float>(a, stream, pdl);
}

}  // namespace bl
