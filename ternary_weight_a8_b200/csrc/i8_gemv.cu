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
// the fragments, a batch of U chunks in flight per warp and BPS blocks per SM
// (32-byte loads, which touch half as many lines at a time, were faster on
// short calls by up to 8% and slower on the long ones by 10 to 20%).
//
// Measured, the weights new in every call: 1 token, 2560 -> 128000: 50.5 us
// (6.5 TB/s, 99% of the copy rate); 8 tokens, 8192 -> 28672: 37.8 us (95%);
// 1 token, 28672 -> 8192: 37.8 us; short calls are latency: 1 token, 2560 ->
// 6912: 4.6 us, of which the weights need 2.7 and an empty launch 2.  (The
// sweeps behind the rules below were taken when a block still read its scales
// last; every form has become 1 to 8% faster since.)
#include <cuda_bf16.h>
#include <type_traits>

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
template <typename TX, typename TY, int TG, int MT, int U, int BPS>
__global__ void __launch_bounds__(32 * kGvWarps, BPS)
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
  const int pitch = kRaw ? P.K | 64 : P.K;
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
      for (int u = 0; u < U; ++u)
        if (c0 + u < c1) {
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) prefetch_l2(wp[i] + 64 * (c0 + u));
        }
    }
  }
  griddep_wait();

  int acc[MT][TG][4] = {};
  // A batch of U chunks, all in flight together; the last one is cut at c1
  // (what it lacks is zero), since chunks one by one would each wait alone.
  auto fetch = [&](int c, uint4 (&a)[U][2 * MT], auto cut) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        if (!decltype(cut)::value || c + u < c1) {
          a[u][i] = ld_stream_u4(wp[i] + 64 * (c + u));
        } else {
          a[u][i] = make_uint4(0, 0, 0, 0);
        }
      }
  };
  auto use = [&](int c, uint4 (&a)[U][2 * MT], auto cut) {
    uint4 x[U][TG];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < TG; ++j) {
        if (!decltype(cut)::value || c + u < c1) {
          x[u][j] = *reinterpret_cast<const uint4*>(xp[j] + 64 * (c + u));
        } else {
          x[u][j] = make_uint4(0, 0, 0, 0);
        }
      }
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
  const std::true_type cut{};
  const std::false_type whole{};
  int c = c0;
  if constexpr (kRaw) {
    // The first weights are under way while the block quantises.
    uint4 first[U][2 * MT];
    fetch(c0, first, cut);
    block_codes<TX>(P, reinterpret_cast<int8_t*>(raw_codes), pitch, raw_scales);
    use(c0, first, cut);
    c += U;
  }
  for (; c + U <= c1; c += U) {
    uint4 a[U][2 * MT];
    fetch(c, a, whole);
    use(c, a, whole);
  }
  if (c < c1) {
    uint4 a[U][2 * MT];
    fetch(c, a, cut);
    use(c, a, cut);
  }

  // The scales of this thread's outputs, under way while the sums meet (read
  // where they are used: 32 tokens, 4096 -> 6912 10.1 us, 9.1 here; 1 token,
  // 2560 -> 128000 52.2 and 50.3; before the loop their registers are missed
  // there: 10.5 and 51.3).
  constexpr int kOuts = (8 * TG * kRows + 32 * kGvWarps - 1) / (32 * kGvWarps);
  float sx[kOuts], sw[kOuts];
#pragma unroll
  for (int o = 0; o < kOuts; ++o) {
    const int i = threadIdx.x + o * 32 * kGvWarps, m = i / kRows, n = n0 + i % kRows;
    sx[o] = !kRaw && m < P.M ? __ldcg(P.scale + m) : 1.0f;
    sw[o] = n < P.N ? __ldcg(P.wscale + n) : 1.0f;
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
#pragma unroll
  for (int o = 0; o < kOuts; ++o) {
    const int i = threadIdx.x + o * 32 * kGvWarps, m = i / kRows, r = i % kRows, n = n0 + r;
    if (i >= 8 * TG * kRows || m >= P.M || n >= P.N) continue;
    const int sum = sums[m][r];
    const float f = __fmul_rn(__frcp_rn(kRaw ? raw_scales[m] : sx[o]), __frcp_rn(sw[o]));
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

template <typename TX, typename TY, int TG, int MT, int U, int BPS>
cudaError_t launch_k(const I8Args& a, cudaStream_t stream, bool pdl) {
  const int blocks = (a.N + 16 * MT - 1) / (16 * MT);
  const int resident = BPS * num_sms();
  // Blocks whose first weights are fetched into L2 ahead: the first wave of
  // several (1 token, 8192 -> 28672: 37.1 us, 38.2 without; 2560 -> 32000: 15.9
  // and 16.8), never more (2560 -> 128000: 70 us, 52).  Where all blocks are
  // resident they fetch at up to two per SM (1024 -> 4096: 2.2 us, 2.8 without;
  // 28672 -> 4096: 19.5 and 20.8), not at more (2560 -> 6912: 5.0 and 4.9) nor
  // for more than 8 tokens, whose codes share L2 (16 tokens, 4096 -> 4096: 5.8
  // and 5.0), unless they have to quantise first, which gives the time.
  constexpr bool kRaw = sizeof(TX) > 1;
  const int wave = blocks > resident ? resident : kRaw || (TG == 1 && blocks <= 2 * num_sms()) ? blocks : 0;
  const size_t smem = kRaw ? static_cast<size_t>(a.M) * (a.K | 64) : 0;
  return launch(i8_gemv_kernel<TX, TY, TG, MT, U, BPS>, dim3(blocks), dim3(32 * kGvWarps), smem, stream, pdl, a, wave);
}

// The zeros that batches of `u` chunks pad a warp's share of K with.
inline int padding(int K, int u) {
  const int share = (K / 64 + kGvWarps - 1) / kGvWarps;
  return (share + u - 1) / u * u - share;
}

// Batches of UA chunks, or of UB where those pad less.
template <typename TX, typename TY, int TG, int UA, int UB, int BPS>
cudaError_t launch_u(const I8Args& a, cudaStream_t stream, bool pdl) {
  return padding(a.K, UB) < padding(a.K, UA) ? launch_k<TX, TY, TG, 1, UB, BPS>(a, stream, pdl)
                                             : launch_k<TX, TY, TG, 1, UA, BPS>(a, stream, pdl);
}

// A warp waits once per batch, so a batch should be long and its last one full
// (4 tokens, U = 5 and 8, three blocks per SM: 2560 -> 6912, 5 chunks a warp,
// 4.9 and 5.1 us; 4096 -> 6912, 8 chunks, 6.4 and 6.3; 3200 -> 6912, 7 chunks,
// 6.0 and 5.4).  Registers pay for it, so a block takes as many as the grid
// leaves it: two blocks per SM where no SM gets more (4 tokens, 8192 -> 4096:
// 7.5 us, 8.7 with three; 16 tokens, 2560 -> 2560: 3.8 with two, 4.8 with
// three), four where four make one wave (1 token, 28672 -> 8192: 37.3 us, 45
// with three) and where blocks are many, for their starts and ends (4 tokens,
// 4096 -> 128000: 78 us, 83 with three; 2560 -> 32000: 16.7 and 16.0).
template <typename TY>
cudaError_t launch_i8_gemv_t(const I8Args& a, cudaStream_t stream, bool pdl) {
  using bf16 = __nv_bfloat16;
  const int per_sm = (a.N + 16 * num_sms() - 1) / (16 * num_sms());
  if (a.x) {
    // The first batch stays in registers while the block quantises, beside the
    // tokens' values, which at three blocks per SM leaves room for four chunks
    // (1 token, 8192 -> 7000: 11.9 us, 14.1 with five).
    if (per_sm <= 2)
      return a.x_bf16 ? launch_k<bf16, TY, 1, 1, 5, 2>(a, stream, pdl) : launch_k<float, TY, 1, 1, 5, 2>(a, stream, pdl);
    return a.x_bf16 ? launch_u<bf16, TY, 1, 4, 5, 3>(a, stream, pdl) : launch_u<float, TY, 1, 4, 5, 3>(a, stream, pdl);
  }
  if (a.M <= 8) {
    if (per_sm <= 2) return launch_u<int8_t, TY, 1, 5, 8, 2>(a, stream, pdl);
    if (per_sm != 4 && per_sm <= 15) return launch_u<int8_t, TY, 1, 5, 8, 3>(a, stream, pdl);
    // Two chunks a warp: twice the rows per block (8 tokens, 1024 -> 128000:
    // 23.8 us, 28.2 with 16 rows; 1536 -> 128000: 37.4 and 33.0).
    if (per_sm > 15 && a.K <= 1024) return launch_k<int8_t, TY, 1, 2, 2, 4>(a, stream, pdl);
    return launch_u<int8_t, TY, 1, 4, 5, 4>(a, stream, pdl);
  }
  if (a.M <= 16) {
    if (per_sm <= 2) return launch_u<int8_t, TY, 2, 5, 8, 2>(a, stream, pdl);
    if (per_sm <= 3) return launch_u<int8_t, TY, 2, 4, 5, 3>(a, stream, pdl);
    return launch_k<int8_t, TY, 2, 1, 4, 4>(a, stream, pdl);
  }
  // 32 tokens, 2560 -> 2560: 5.3 us with two blocks per SM, 6.5 with three;
  // 2560 -> 6912: 7.2 with three, 9.8 with two.
  return per_sm <= 2 ? launch_k<int8_t, TY, 4, 1, 5, 2>(a, stream, pdl) : launch_k<int8_t, TY, 4, 1, 3, 3>(a, stream, pdl);
}

}  // namespace

// Up to 8 tokens always.  More tokens read as many codes as weights or more
// through L1, so the blocks should be one wave, and not of few long rows, which
// the tensor cores' split of K spreads over more SMs.  16 tokens against the
// tensor cores: 2560 -> 6912: 5.5 us and 8.3, 8192 -> 8192: 13.3 and 15.8, 4096
// -> 9472: 8.5 and 11.5, but 2560 -> 12800: 11.9 and 10.5, 16384 -> 2048: 12.5
// and 11.3.  32 tokens: 2560 -> 6912: 7.2 and 8.7, 4096 -> 6912: 9.4 and 10.8,
// but 2560 -> 8640: 13.0 and 9.7, 5120 -> 5120: 10.6 and 9.7, 6912 -> 2560:
// 9.7 and 8.4.
bool i8_takes_gemv(int M, int N, int K) {
  const int per_sm = (N + 16 * num_sms() - 1) / (16 * num_sms());
  return M <= 8 || (M <= 16 && per_sm <= 4 && K <= 12288) || (M <= kI8GemvMaxTokens && per_sm <= 3 && K <= 4096);
}

// One wave of blocks can afford to quantise the tokens in every block, when
// that is short: one or two tokens, or at most the four chunks a thread keeps
// in registers, and not many values (1 token, 2560 -> 6912: 6.1 us, 6.4 with a
// launch for the codes; 2 tokens, 4096 -> 4096: 6.1 and 6.6; 4 tokens, 2560 ->
// 2560: 5 chunks a thread, 5.1 and 4.9; 2 tokens, 8192 -> 4096: 10.7 and 9.1).
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
