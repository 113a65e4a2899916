// The residual sum, the RMSNorm after it and the activation codes in one pass
// (add_rmsnorm_quant), and the gradient of the sum and the norm
// (add_rmsnorm_backward).
//
// Forward, for a token of K inputs:
//   z = T(x + residual)                       fp32 sum, rounded to the activation type T and stored
//   r = fp32(1 / sqrt(mean_k z^2 + eps))      squares summed in double, as rmsnorm_quant does
//   v = T((z * r) * g)                        fp32 products
//   s = 127 / max(max_k |v|, 1e-5),  q = clamp(rint(v * s)),  rowsum = sum_k q
// so the codes equal rmsnorm_quant's on z bit for bit, up to the order of the
// sum in double: where that is not exact its last bits differ, and once in some
// millions of tokens the fp32 root with them.
//
// Backward, with n = z * r and the quantisation as the identity
// (straight-through), for the gradient dv of v and dz_in of z:
//   dz = r * (gd - n * mean_k(gd * n)) + dz_in,  gd = dv * g
//   dg = sum over tokens of dv * n
// dz is the gradient of x and of the residual alike.
//
// Both are bound by memory: 7 bytes per bf16 input forward (x, residual, z,
// codes), 8 backward (z, dv, dz_in, dz; 10 with fp32 dv).  To get there the
// arithmetic has to stay small: sums in bf16 pairs, packed fp32 products,
// maxima as integers, codes by an addition, 1 / rms by Newton's method.
// 8192 x 8192 bf16 forward took 126 us in scalar arithmetic, 78 - 80 in pairs
// and takes 74 - 76 (94 - 96% of the copy rate, by where the tensors lie) with
// the next tokens read ahead into L2; backward 167 us, 96 and 91 (90%).  2048
// x 2560 (one wave, 5.6 us of traffic) takes 11.2 us forward and 15.9 backward,
// of which 5 are the closing kernel's boundary and its sum.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pairs.cuh"

namespace bl {

namespace {

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Memory that another token will want, from HBM as far as L2.
__device__ __forceinline__ void prefetch_l2(const void* p, size_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(static_cast<uint32_t>(bytes)));
}

template <typename V, typename Op>
__device__ __forceinline__ V warp_reduce(V v, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A token belongs to a group of W warps (at most 16); a block holds as many
// groups as fit in 256 threads, or one.
constexpr int kMaxGroupWarps = 16;
constexpr int kNormThreads = 256;
constexpr int kMaxRowBytes = 224 * 1024;  // of a long token in shared memory

// The value of every warp of the token's group, combined in warp order (the
// same in every thread).  `slot`: this group's W values in shared memory.  The
// caller uses another slot for its next reduction, so one barrier is enough.
template <typename V, typename Op>
__device__ __forceinline__ V group_reduce(V v, Op op, V* slot, int W, int wig, int lane, int bar) {
  v = warp_reduce(v, op);
  if (W == 1) return v;
  if (lane == 0) slot[wig] = v;
  group_sync(bar, 32 * W);
  V r = slot[0];
  for (int i = 1; i < W; ++i) r = op(r, slot[i]);
  return r;
}

// fp32(1 / sqrt(ss / K + eps)) exactly as the divisions and the square root
// in double give it.  Those cost hundreds of instructions, and every thread
// needs the value, so it is first taken from rsqrtf and two steps of Newton's
// method in double (y += y / 2 (1 - x y^2)), which is within 2^-50; only when
// that lies within 2^-44 of a border between two fp32 values, or outside the
// range where fp32's rsqrtf starts well, are the divisions done.
__device__ __forceinline__ float rstd_of(double ss, int K, double inv_k, float eps) {
  const double x = __fma_rn(ss, inv_k, static_cast<double>(eps));
  if (x > 1e-30 && x < 1e30) {
    double y = static_cast<double>(rsqrtf(static_cast<float>(x)));
#pragma unroll
    for (int i = 0; i < 2; ++i) y = __fma_rn(0.5 * y, __fma_rn(-x * y, y, 1.0), y);
    // The 29 bits that fp32 drops, from the middle between two values.
    const int off = static_cast<int>(__double_as_longlong(y) & 0x1fffffffll) - 0x10000000;
    if (off > 256 || off < -256) return __double2float_rn(y);
  }
  const double ms = __ddiv_rn(ss, static_cast<double>(K));
  return __double2float_rn(__ddiv_rn(1.0, __dsqrt_rn(__dadd_rn(ms, static_cast<double>(eps)))));
}

struct AddNormParams {
  const void* x;
  const void* res;
  const float* gain;  // [K] or null
  float eps;
  void* z;       // may be x or res
  void* x_norm;  // or null
  int8_t* xq;
  float* scale;
  int32_t* rowsum;  // or null
  int M, K;
  double inv_k;
};

// C: 16-byte chunks of a token per thread, held in registers from the sum to
// the codes (z's chunk is overwritten by v's).  C = 0: the token is longer
// than the registers hold, and its chunks wait in shared memory (`staged`), or,
// longer than that too, z is read back for the absmax and again for the
// codes; either way each thread reads only what it wrote.  kFull: every thread
// has all its chunks, so their instructions interleave without bounds between
// them (2048 x 2560 fp32 16.7 -> 14.6 us).  kAhead: x and residual of the
// token `ahead` tokens on come as far as L2 while this one is worked on, so
// that HBM does not stand still while the blocks of an SM, which began
// together, all compute or store.  Not before this token's own loads are in:
// asked for at the start they delay those (8192 x 2560 in four chunks 30.4 -
// 31.8 us, 29.5 after the first sum; 32.9 without).  kRoom: for blocks of at
// most 256 threads, three of which share an SM's registers.
template <typename T, int C, bool kFull, bool kAhead, bool kRoom>
__global__ void __launch_bounds__(kRoom ? 256 : 512, (C == 4 && !kRoom) || C == 0 ? 2 : 3)
    add_rmsnorm_quant_kernel(const AddNormParams P, int W, int staged, int ahead) {
  extern __shared__ uint4 row_buf[];
  constexpr int N = kPer<T>;
  __shared__ double red_d[kMaxGroupWarps];
  __shared__ uint32_t red_u[kMaxGroupWarps];
  __shared__ float red_f[kMaxGroupWarps];
  __shared__ int red_i[kMaxGroupWarps];
  griddep_launch_dependents();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wig = warp % W, groups = (blockDim.x >> 5) / W;
  const int m = blockIdx.x * groups + group;
  const int tid = wig * 32 + lane, step = 32 * W, chunks = P.K / N, bar = 1 + group;
  griddep_wait();  // the inputs may be the preceding kernel's outputs; the outputs may still be read by it
  if (m >= P.M) return;  // the whole group: its named barrier is its own

  const size_t row = static_cast<size_t>(m) * P.K;
  const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const T*>(P.x) + row);
  const uint4* rr = reinterpret_cast<const uint4*>(static_cast<const T*>(P.res) + row);
  uint4* zr = reinterpret_cast<uint4*>(static_cast<T*>(P.z) + row);
  uint4* nr = P.x_norm ? reinterpret_cast<uint4*>(static_cast<T*>(P.x_norm) + row) : nullptr;
  int8_t* qr = P.xq + row;

  // Squares in double, in two chains.
  double ss0 = 0.0, ss1 = 0.0;
  auto square = [&](const uint4& zc) {
    f32x2 p[kPairs<T>];
    to_pairs<T>(zc, p);
#pragma unroll
    for (int e = 0; e < kPairs<T>; ++e) {
      float lo, hi;
      split2(p[e], lo, hi);
      const double dl = static_cast<double>(lo), dh = static_cast<double>(hi);
      ss0 = __fma_rn(dl, dl, ss0);
      ss1 = __fma_rn(dh, dh, ss1);
    }
  };
  f32x2 r2 = 0;
  // z r g of a chunk, its gains read here or already (`g`).
  auto norm_chunk = [&](const uint4& zc, int c, const f32x2 (*g)[kPairs<T>] = nullptr) {
    f32x2 p[kPairs<T>];
    to_pairs<T>(zc, p);
#pragma unroll
    for (int e = 0; e < kPairs<T>; ++e) p[e] = mul2(p[e], r2);
    if (P.gain) {
      f32x2 own[kPairs<T>];
      if (!g) load_pairs(P.gain + static_cast<size_t>(c) * N, own);
#pragma unroll
      for (int e = 0; e < kPairs<T>; ++e) p[e] = mul2(p[e], g ? (*g)[e] : own[e]);
    }
    return from_pairs<T>(p);
  };

  constexpr int CR = C > 0 ? C : 1;
  // The gains of the first kGainFirst chunks are asked for with the token's
  // own loads, those up to kGainNext behind the first sum, and the rest where
  // they are used: as many early as the registers take without spilling (all
  // where they are used: 4096 x 1280 fp32 16.1 us, 13.3 with all first; 2048 x
  // 5120 bf16, four chunks with room, 18.1, 16.0 with 2 and 4, 17.2 with all
  // first; 2048 x 2560 bf16, five chunks, 12.5, 11.2 with 3, 12.4 with 1 and 4;
  // 64 x 8192 bf16, two chunks of 40 registers, 5.1 with none and 5.7 with any).
  constexpr int kGainFirst = sizeof(T) == 4 || C <= 1 ? C : C == 2 ? 0 : C == 4 ? (kRoom ? 2 : kFull ? 0 : 1) : 3;
  constexpr int kGainNext = kRoom && C == 4 ? 4 : kGainFirst;
  f32x2 gains[kGainNext > 0 ? kGainNext : 1][kPairs<T>];
  auto load_gains = [&](int first, int end) {
    if (!P.gain) return;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i >= first && i < end && (kFull || tid + i * step < chunks))
        load_pairs(P.gain + static_cast<size_t>(tid + i * step) * N, gains[i < kGainNext ? i : 0]);
  };
  uint4 keep[CR];
  if constexpr (C > 0) {
    uint4 other[CR];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (kFull || c < chunks) {
        keep[i] = __ldcg(xr + c);
        other[i] = __ldcg(rr + c);
      }
    }
    load_gains(0, kGainFirst);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (kFull || c < chunks) {
        keep[i] = sum16<T>(keep[i], other[i]);
        zr[c] = keep[i];
        square(keep[i]);
      }
    }
  } else {
    for (int c0 = tid; c0 < chunks; c0 += 4 * step) {
      uint4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i * step < chunks) {
          a[i] = __ldcg(xr + c0 + i * step);
          b[i] = __ldcg(rr + c0 + i * step);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i * step;
        if (c < chunks) {
          const uint4 zc = sum16<T>(a[i], b[i]);
          zr[c] = zc;
          if (staged) row_buf[c] = zc;
          square(zc);
        }
      }
    }
  }
  const double ss = group_reduce(__dadd_rn(ss0, ss1), [](double a, double b) { return __dadd_rn(a, b); },
                                 red_d + group * W, W, wig, lane, bar);
  load_gains(kGainFirst, kGainNext);
  const float r = rstd_of(ss, P.K, P.inv_k, P.eps);
  r2 = pack2(r, r);
  if (kAhead && tid == 0 && P.M - m > ahead) {
    const size_t at = row + static_cast<size_t>(ahead) * P.K;
    prefetch_l2(static_cast<const T*>(P.x) + at, P.K * sizeof(T));
    prefetch_l2(static_cast<const T*>(P.res) + at, P.K * sizeof(T));
  }

  uint32_t top = 0;
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (kFull || c < chunks) {
        keep[i] = norm_chunk(keep[i], c, i < kGainNext ? &gains[i < kGainNext ? i : 0] : nullptr);
        top = absmax16<T>(top, keep[i]);
        if (nr) nr[c] = keep[i];
      }
    }
  } else {
    for (int c = tid; c < chunks; c += step) {
      const uint4 v = norm_chunk(staged ? row_buf[c] : zr[c], c);
      top = absmax16<T>(top, v);
      if (staged) row_buf[c] = v;
    }
  }
  top = __reduce_max_sync(0xffffffffu, absmax_bits<T>(top));
  if (W > 1) {
    if (lane == 0) red_u[group * W + wig] = top;
    group_sync(bar, 32 * W);
    for (int i = 0; i < W; ++i) top = max(top, red_u[group * W + i]);
  }
  float amax = __uint_as_float(top);
  const bool finite = top < 0x7f800000u;  // the same in the whole group
  // fn(values, chunk) over the normalised chunks.
  auto for_each = [&](auto&& fn) {
    if constexpr (C > 0) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = tid + i * step;
        if (kFull || c < chunks) fn(keep[i], c);
      }
    } else {
      for (int c = tid; c < chunks; c += step) fn(staged ? row_buf[c] : norm_chunk(zr[c], c), c);
    }
  };
  int sum = 0;
  float s;
  if (finite) {
    s = __fdiv_rn(127.0f, fmaxf(amax, 1e-5f));
    const f32x2 s2 = pack2(s, s);
    for_each([&](const uint4& v, int c) {
      if (C == 0 && nr) nr[c] = v;
      sum += store_codes<T>(v, s2, qr + static_cast<size_t>(c) * N);
    });
  } else {
    // Infinities or NaN: the largest |value| that is a number or an infinity.
    amax = 0.0f;
    for_each([&](const uint4& v, int) { amax = fmaxf(amax, absmax_any<T>(v)); });
    amax = group_reduce(amax, [](float a, float b) { return fmaxf(a, b); }, red_f + group * W, W, wig, lane, bar);
    s = __fdiv_rn(127.0f, fmaxf(amax, 1e-5f));
    for_each([&](const uint4& v, int c) {
      if (C == 0 && nr) nr[c] = v;
      sum += store_codes_any<T>(v, s, qr + static_cast<size_t>(c) * N);
    });
  }
  if (P.rowsum) {
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (W > 1) {
      if (lane == 0) red_i[group * W + wig] = sum;
      group_sync(bar, 32 * W);
      if (tid == 0)
        for (int i = 1; i < W; ++i) sum += red_i[group * W + i];
    }
    if (tid == 0) P.rowsum[m] = sum;
  }
  if (tid == 0) P.scale[m] = s;
}

// How tokens are spread: n chunks per thread (over four: more than registers
// hold), W warps per token, `groups` tokens per block.
struct Groups {
  int n, W, groups;
};

Groups plan_groups(int M, int chunks) {
  // Four chunks per thread (the most that leave 32 warps to an SM) while the
  // tokens give every SM 16 warps, else fewer chunks and more warps, as far
  // as a block goes.
  Groups g{5, 0, 1};
  for (int c = 4; c >= 1; c /= 2) {
    int w = (chunks + 32 * c - 1) / (32 * c);
    if (w > 8) w = (w + 3) / 4 * 4;  // an even share of an SM's four schedulers and their registers
    if (w > kMaxGroupWarps) break;
    g.W = w;
    g.n = (chunks + 32 * w - 1) / (32 * w);
    if (static_cast<long long>(M) * w >= 16LL * num_sms()) break;
  }
  // Longer than 16 warps hold.  Up to nine chunks a thread, eight warps leave
  // room for more tokens on an SM (1021 fp32 tokens of 8640: 26.8 us, 33.0
  // with 16 warps); longer tokens want all 16 (512 bf16 tokens of 28672:
  // 28.2 us, 36.0 with 8).
  if (g.W == 0) g.W = chunks <= 9 * 32 * 8 ? 8 : kMaxGroupWarps;
  g.groups = g.W > kNormThreads / 32 ? 1 : kNormThreads / 32 / g.W;
  if (g.n > 4) g.groups = 1;
  return g;
}

using AddNormKernel = void (*)(AddNormParams, int, int, int);

cudaError_t launch_add_rmsnorm_quant_k(AddNormKernel kernel, const AddNormParams& P, const Groups& g, int ahead, size_t smem,
                                       cudaStream_t stream, bool pdl) {
  return launch(kernel, dim3((P.M + g.groups - 1) / g.groups), dim3(32 * g.W * g.groups), smem, stream, pdl, P, g.W,
                smem ? 1 : 0, ahead);
}

template <typename T, int C, bool kRoom>
cudaError_t launch_add_rmsnorm_quant_c(const AddNormParams& P, const Groups& g, bool full, int ahead, size_t smem,
                                       cudaStream_t stream, bool pdl) {
  AddNormKernel kernel = ahead ? add_rmsnorm_quant_kernel<T, C, false, true, kRoom>
                               : add_rmsnorm_quant_kernel<T, C, false, false, kRoom>;
  if constexpr (C > 0) {
    if (full)
      kernel = ahead ? add_rmsnorm_quant_kernel<T, C, true, true, kRoom> : add_rmsnorm_quant_kernel<T, C, true, false, kRoom>;
  } else {
    static std::atomic<uint64_t> attr_done{0};
    const cudaError_t e = once_per_device(attr_done, [] {
      const AddNormKernel both[] = {add_rmsnorm_quant_kernel<T, C, false, true, kRoom>,
                                    add_rmsnorm_quant_kernel<T, C, false, false, kRoom>};
      for (AddNormKernel k : both) {
        const cudaError_t e1 = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRowBytes);
        if (e1 != cudaSuccess) return e1;
      }
      return cudaSuccess;
    });
    if (e != cudaSuccess) return e;
  }
  return launch_add_rmsnorm_quant_k(kernel, P, g, ahead, smem, stream, pdl);
}

template <typename T>
cudaError_t launch_add_rmsnorm_quant_t(const AddNormParams& P, cudaStream_t stream, bool pdl) {
  const int chunks = P.K / kPer<T>;
  Groups g = plan_groups(P.M, chunks);
  int held = g.n <= 2 ? g.n : g.n <= 4 ? 4 : 0;
  // 80 registers a thread and 24 warps per SM (kRoom) in place of 64 and 32.
  // Four chunks of bf16 that every thread has: 2048 x 5120 16.6 us, 19.1 with
  // 64; 2048 x 4096 14.0 and 15.9; 700 x 4096 6.6 and 7.3; but with whole
  // schedulers per token and many waves the warps count more: 8192 x 8192 78.4
  // and 74.9, 16384 x 4096 75.6 and 72.8, 8192 x 4096 40.7 and 40.9; nor where
  // 32 warps make one wave and 24 do not: 4096 x 1024 8.7 and 7.6.  fp32 has
  // its room in 64: 4096 x 2048 19.9 and 19.1.
  const bool fills = held == 4 && chunks == 4 * 32 * g.W;
  const long long sms = num_sms(), warps = static_cast<long long>(P.M) * g.W;
  bool room = fills && sizeof(T) == 2 && g.W <= kNormThreads / 32 && (g.W % 4 != 0 || warps <= 240 * sms) &&
              (warps <= 24 * sms || warps > 32 * sms);
  // Five chunks where every thread has five and would lack some of four, or
  // where they spare more than eight warps, and 24 warps per SM have work: 8192
  // x 2560 27.3 us, 31.5 with four; 2048 x 10240 29.0 and 35.7; 4096 x 1280
  // fp32 13.3 and 17.0; 1021 x 8640 18.5 and 19.4; 1024 x 2560 6.8 and 6.6.
  const int five = (chunks + 159) / 160;
  const bool spares = g.W > kNormThreads / 32 || (held == 4 && !fills && chunks == 160 * five);
  if (spares && five <= kNormThreads / 32 && static_cast<long long>(P.M) * five >= 24 * sms) {
    held = 5;
    room = true;
    g = Groups{5, five, kNormThreads / 32 / five};
  }
  const bool full = chunks == held * 32 * g.W;  // every thread holds as many chunks as it has room for
  const size_t row = static_cast<size_t>(P.K) * sizeof(T);
  const size_t smem = held == 0 && row <= kMaxRowBytes ? row : 0;
  // Reading ahead pays where enough tokens wait behind those that what the
  // registers and the staged rows let be resident, and over a distance of half
  // to all of these (8192 x 8192 78.0 us without, 78.4, 73.2, 72.4 and 72.5 at
  // 1/4, 1/2, 3/4 and all; 1021 fp32 tokens of 8640 26.0, and 24.2, 24.1, 24.5
  // and 24.2; 700 x 4096, 1.2 waves: 7.3 without, 7.6 with; 512 x 28672, two
  // resident per SM, 1.7 waves: 28.6 and 29.1).
  int per_sm = (room ? 768 : held == 1 || held == 2 ? 1536 : 1024) / (32 * g.W * g.groups);
  if (held == 0) per_sm = smem ? std::min(per_sm, static_cast<int>(228 * 1024 / (row + 2048))) : 0;
  const long long resident = sms * per_sm * g.groups;
  int ahead = 0;
  if (per_sm > 0 && 2LL * P.M > (per_sm > 2 ? 3 : 4) * resident)
    ahead = static_cast<int>(held ? resident / 4 * 3 : resident / 2);
  if (held == 1) return launch_add_rmsnorm_quant_c<T, 1, false>(P, g, full, ahead, 0, stream, pdl);
  if (held == 2) return launch_add_rmsnorm_quant_c<T, 2, false>(P, g, full, ahead, 0, stream, pdl);
  if (held == 5) return launch_add_rmsnorm_quant_c<T, 5, true>(P, g, full, ahead, 0, stream, pdl);
  if constexpr (sizeof(T) == 2) {
    if (room)
      return launch_add_rmsnorm_quant_k(ahead ? add_rmsnorm_quant_kernel<T, 4, true, true, true>
                                              : add_rmsnorm_quant_kernel<T, 4, true, false, true>,
                                        P, g, ahead, 0, stream, pdl);
  }
  if (held == 4) return launch_add_rmsnorm_quant_c<T, 4, false>(P, g, full, ahead, 0, stream, pdl);
  return launch_add_rmsnorm_quant_c<T, 0, false>(P, g, false, ahead, smem, stream, pdl);
}

// ---------------------------------------------------------------------------
// The activation codes alone, for the 8-bit product: exactly quant_act's, on
// the norm's arithmetic (packed products, integer maxima, groups of warps per
// token).  Bound by memory: 3 bytes per bf16 input.
// ---------------------------------------------------------------------------
struct CodesParams {
  const void* x;
  int8_t* xq;
  float* scale;
  int M, K;
};

template <typename T, int C>
__global__ void __launch_bounds__(512, C == 4 || C == 0 ? 2 : 3) row_codes_kernel(const CodesParams P, int W) {
  constexpr int N = kPer<T>;
  __shared__ uint32_t red_u[kMaxGroupWarps];
  __shared__ float red_f[kMaxGroupWarps];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wig = warp % W, groups = (blockDim.x >> 5) / W;
  const int m = blockIdx.x * groups + group;
  const int tid = wig * 32 + lane, step = 32 * W, chunks = P.K / N, bar = 1 + group;
  griddep_wait();
  if (m >= P.M) return;  // the whole group: its named barrier is its own
  const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const T*>(P.x) + static_cast<size_t>(m) * P.K);
  int8_t* qr = P.xq + static_cast<size_t>(m) * P.K;

  constexpr int CR = C > 0 ? C : 1;
  uint4 keep[CR];
  uint32_t top = 0;
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (tid + i * step < chunks) keep[i] = __ldcg(xr + tid + i * step);
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (tid + i * step < chunks) top = absmax16<T>(top, keep[i]);
  } else {
#pragma unroll 4
    for (int c = tid; c < chunks; c += step) top = absmax16<T>(top, __ldcg(xr + c));
  }
  auto for_each = [&](auto&& fn) {
    if constexpr (C > 0) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (tid + i * step < chunks) fn(keep[i], tid + i * step);
    } else {
#pragma unroll 4
      for (int c = tid; c < chunks; c += step) fn(__ldcg(xr + c), c);
    }
  };
  top = __reduce_max_sync(0xffffffffu, absmax_bits<T>(top));
  if (W > 1) {
    if (lane == 0) red_u[group * W + wig] = top;
    group_sync(bar, 32 * W);
    for (int i = 0; i < W; ++i) top = max(top, red_u[group * W + i]);
  }
  float s;
  if (top < 0x7f800000u) {
    s = __fdiv_rn(127.0f, fmaxf(__uint_as_float(top), 1e-5f));
    const f32x2 s2 = pack2(s, s);
    for_each([&](const uint4& v, int c) { store_codes<T>(v, s2, qr + static_cast<size_t>(c) * N); });
  } else {
    // Infinities or NaN, as in the norm.
    float amax = 0.0f;
    for_each([&](const uint4& v, int) { amax = fmaxf(amax, absmax_any<T>(v)); });
    amax = group_reduce(amax, [](float a, float b) { return fmaxf(a, b); }, red_f + group * W, W, wig, lane, bar);
    s = __fdiv_rn(127.0f, fmaxf(amax, 1e-5f));
    for_each([&](const uint4& v, int c) { store_codes_any<T>(v, s, qr + static_cast<size_t>(c) * N); });
  }
  if (tid == 0) P.scale[m] = s;
}

template <typename T>
cudaError_t launch_row_codes_t(const CodesParams& P, cudaStream_t stream, bool pdl) {
  const Groups g = plan_groups(P.M, P.K / kPer<T>);
  const dim3 grid((P.M + g.groups - 1) / g.groups), block(32 * g.W * g.groups);
  if (g.n <= 1) return launch(row_codes_kernel<T, 1>, grid, block, 0, stream, pdl, P, g.W);
  if (g.n <= 2) return launch(row_codes_kernel<T, 2>, grid, block, 0, stream, pdl, P, g.W);
  if (g.n <= 4) return launch(row_codes_kernel<T, 4>, grid, block, 0, stream, pdl, P, g.W);
  return launch(row_codes_kernel<T, 0>, grid, block, 0, stream, pdl, P, g.W);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
struct AddNormBackParams {
  const void* z;
  const void* dv;
  const float* gain;   // [K] or null
  const void* dz_in;   // or null
  float eps;
  void* dz;            // may be dz_in
  float* part;         // [rows][K] sums of dv * n over each block's tokens, or null
  float* rstd;         // [M] (long tokens only)
  int M, K;
  double inv_k;
  float inv_kf;
  int ahead = 0;       // kAheadIn, kAheadRing
};

constexpr int kAheadIn = 1, kAheadRing = 2;

// N gradient values of type TD: 8, 16 or 32 bytes.
template <typename TD, int N>
struct GradChunk {
  static constexpr int kBytes = N * static_cast<int>(sizeof(TD));
  uint4 w[kBytes > 16 ? 2 : 1];
  __device__ __forceinline__ void load(const TD* p) {
    if constexpr (kBytes == 8) {
      const uint2 h = __ldcg(reinterpret_cast<const uint2*>(p));
      w[0] = make_uint4(h.x, h.y, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) w[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
    }
  }
  __device__ __forceinline__ void get(f32x2 (&f)[N / 2]) const {
    if constexpr (sizeof(TD) == 2) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < N / 2; ++i) f[i] = pair_of_bf16(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        f32x2 t[2];
        to_pairs<float>(w[i], t);
        f[2 * i] = t[0];
        f[2 * i + 1] = t[1];
      }
    }
  }
};

// A thread's own pieces of 16 (or 8) bytes on their way through shared memory.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  }
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// The ring of the backward's z and dv: for every stage and chunk, a piece of
// each thread after the other.  Three stages: a token's output, the next
// one's sums and the one after on its way; two with fp32 gradients of bf16
// tokens, whose pieces are half as large again, so that more blocks fit.
template <typename T, typename TD>
struct BackRing {
  static constexpr int kZ = 16, kD = kPer<T> * static_cast<int>(sizeof(TD)), kChunk = kZ + kD;
  static constexpr int kStages = kChunk > 32 ? 2 : 3;
  static constexpr int bytes(int threads, int chunks) { return kStages * chunks * threads * kChunk; }
};

template <int P2>
__device__ __forceinline__ void store_pairs(float* p, const f32x2 (&v)[P2]) {
#pragma unroll
  for (int i = 0; i < P2 / 2; ++i) {
    float f[4];
    split2(v[2 * i], f[0], f[1]);
    split2(v[2 * i + 1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[i] = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// Both sums of a token are taken again in double where fp32 may not hold them:
//  - the sum of z^2 outside this range (fp32 squares overflow above 2^128 and
//    lose bits below 2^-126);
//  - the sum of gd * z no number, or overflowing with r;
//  - that sum so small that the half steps of subnormal terms, 2^-150 each,
//    may count: 2^26 of them are 2^-24 of 1e-30.  Zero is the sum of tokens
//    without a gradient (padding, 8192 x 8192 91 us; taken again, 129), and
//    up to r = 2^10 what it may hide is below 2^-140 of gradient.
constexpr float kSquaresLow = 1e-25f, kSquaresHigh = 1e37f, kDotLow = 1e-30f, kDotZeroRstd = 1024.0f;

__device__ __forceinline__ bool dot_in_range(float dot, float r) {
  return fabsf(dot * r) < INFINITY && (fabsf(dot) > kDotLow || (dot == 0.0f && r <= kDotZeroRstd));
}

// gd * z of a pair in double, added to t.
__device__ __forceinline__ double add_products(f32x2 gd, f32x2 z, double t) {
  float g0, g1, z0, z1;
  split2(gd, g0, g1);
  split2(z, z0, z1);
  t = __fma_rn(static_cast<double>(g0), static_cast<double>(z0), t);
  return __fma_rn(static_cast<double>(g1), static_cast<double>(z1), t);
}

constexpr int kMaxCluster = 8;

__device__ __forceinline__ void st_cluster_b64(uint32_t cluster_addr, f32x2 v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(cluster_addr), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive_release() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_acquire() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// The two sums of a pair over the warp, in one butterfly.
__device__ __forceinline__ f32x2 warp_sum2(f32x2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add2(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A group of W warps takes tokens group0, group0 + groups_total, ...; a
// thread owns the same C chunks of every token (kFull: all of them exist), so
// the gain's gradient is summed in its registers and written once per block.
// The two sums over a token run as one pair of fp32, through at most 31 steps
// (16 fused ones of a thread's halves, their join, 5 shuffles, up to 4 places
// of a cluster's warps and 5 shuffles): at 16 warps a token, sums and 1 / rms
// in double were half of the kernel's instructions.
// A token of more than 1024 chunks is shared by a cluster (kCluster: C chunks
// of 32 W threads in each of its CTAs), whose sums meet in every CTA's shared
// memory.  z and dv of the next tokens are under way in shared memory, where a
// thread reads only what it copied itself, so no barrier guards them; a
// token's sums are taken while the token before is written, so that the
// reduction's chain of shuffles and its barrier wait for nobody.
template <typename T, typename TD, int C, bool kGain, bool kFull, bool kCluster>
__global__ void __launch_bounds__(C <= 2 ? 256 : 512, C == 1 ? 4 : C == 2 ? 3 : 1)
    add_rmsnorm_backward_kernel(const AddNormBackParams P, int W) {
  constexpr int N = kPer<T>, NP = kPairs<T>;
  using R = BackRing<T, TD>;
  extern __shared__ uint4 ring[];
  constexpr int kSlots = kCluster ? kMaxGroupWarps * kMaxCluster : kMaxGroupWarps;
  __shared__ f32x2 red[2][kSlots];
  __shared__ double red_d[2][kSlots];
  griddep_launch_dependents();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cl = kCluster ? static_cast<int>(cluster_nctarank()) : 1;
  const int rank = kCluster ? static_cast<int>(cluster_ctarank()) : 0;
  const int group = kCluster ? 0 : warp / W, wig = kCluster ? warp : warp % W;
  const int groups = kCluster ? 1 : (blockDim.x >> 5) / W;
  const int g0 = kCluster ? blockIdx.x / cl : blockIdx.x * groups + group;
  const int stride = kCluster ? gridDim.x / cl : gridDim.x * groups;
  // A thread's chunks are tid, tid + step, ... of its token (of its CTA's part).
  const int tid = (kCluster ? rank * C * 32 * W : 0) + wig * 32 + lane, step = 32 * W;
  const int chunks = P.K / N, bar = 1 + group;
  if constexpr (kCluster) cluster_sync_all();  // the others' shared memory is there
  griddep_wait();
  // This warp's pair of sums into its place in every CTA of the cluster.
  auto post = [&](f32x2 (&slots)[kSlots], f32x2 v) {
    if constexpr (kCluster) {
      if (lane < cl) st_cluster_b64(mapa_shared(smem_u32(&slots[rank * W + wig]), static_cast<uint32_t>(lane)), v);
    } else {
      if (lane == 0) slots[group * W + wig] = v;
    }
  };
  auto total = [&](const f32x2 (&slots)[kSlots]) {
    f32x2 v = 0;
    if constexpr (kCluster) {
      for (int i = lane; i < cl * W; i += 32) v = add2(v, slots[i]);
    } else {
      if (lane < W) v = slots[group * W + lane];
    }
    return warp_sum2(v);
  };

  // The gains and the sums of their gradient stay in registers: reading 4
  // bytes of gain for every 2 of z, twice a token, kept the kernel waiting.
  f32x2 acc[kGain ? C : 1][NP], gains[kGain ? C : 1][NP];
#pragma unroll
  for (int i = 0; i < (kGain ? C : 1); ++i) {
#pragma unroll
    for (int e = 0; e < NP; ++e) acc[i][e] = 0;
    if constexpr (kGain) {
      const int c = tid + i * step;
      if (kFull || c < chunks) load_pairs(P.gain + static_cast<size_t>(c) * N, gains[i]);
    }
  }

  // Stage s, chunk i: this thread's z, and behind every thread's z its dv (32
  // bytes as two pieces apart, so that the threads' pieces stay adjacent).
  const int threads = blockDim.x;
  uint8_t* const mine = reinterpret_cast<uint8_t*>(ring);
  auto z_at = [&](int s, int i) { return mine + (s * C + i) * threads * R::kChunk + threadIdx.x * 16; };
  auto d_at = [&](int s, int i, int j) {
    return mine + (s * C + i) * threads * R::kChunk + threads * (16 + 16 * j) + threadIdx.x * (R::kD < 16 ? R::kD : 16);
  };
  auto request = [&](int m, int s) {
    if (m < P.M) {
      const size_t row = static_cast<size_t>(m) * P.K;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = tid + i * step;
        if (kFull || c < chunks) {
          copy_async<16>(smem_u32(z_at(s, i)), reinterpret_cast<const uint4*>(static_cast<const T*>(P.z) + row) + c);
          const uint8_t* d =
              reinterpret_cast<const uint8_t*>(static_cast<const TD*>(P.dv) + row + static_cast<size_t>(c) * N);
          if constexpr (R::kD < 16) {
            copy_async<8>(smem_u32(d_at(s, i, 0)), d);
          } else {
#pragma unroll
            for (int j = 0; j < R::kD / 16; ++j) copy_async<16>(smem_u32(d_at(s, i, j)), d + 16 * j);
          }
        }
      }
    }
    copy_async_commit();  // a group for every token, also past the last
  };
  auto z_of = [&](int s, int i, f32x2 (&z)[NP]) { to_pairs<T>(*reinterpret_cast<const uint4*>(z_at(s, i)), z); };
  auto d_of = [&](int s, int i, f32x2 (&d)[NP]) {
    GradChunk<TD, N> dc;
    if constexpr (R::kD < 16) {
      const uint2 h = *reinterpret_cast<const uint2*>(d_at(s, i, 0));
      dc.w[0] = make_uint4(h.x, h.y, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < R::kD / 16; ++j) dc.w[j] = *reinterpret_cast<const uint4*>(d_at(s, i, j));
    }
    dc.get(d);
  };

  // The sums of z^2 and gd * z over this warp's part of the token in stage s.
  auto sums_of = [&](int s) {
    f32x2 sq2 = 0, dot2 = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (kFull || c < chunks) {
        f32x2 z[NP], d[NP];
        z_of(s, i, z);
        d_of(s, i, d);
        if constexpr (kGain) {
#pragma unroll
          for (int e = 0; e < NP; ++e) d[e] = mul2(d[e], gains[i][e]);
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          sq2 = fma2(z[e], z[e], sq2);
          dot2 = fma2(d[e], z[e], dot2);
        }
      }
    }
    float a0, a1, b0, b1;
    split2(sq2, a0, a1);
    split2(dot2, b0, b1);
    return warp_sum2(pack2(a0 + a1, b0 + b1));
  };

  // From HBM as far as L2: dz_in of the next token, z and dv of the one behind
  // the ring's.
  auto ahead_in = [&](size_t row) {
    prefetch_l2(static_cast<const T*>(P.dz_in) + (row + static_cast<size_t>(stride) * P.K), P.K * sizeof(T));
  };
  auto ahead_ring = [&](size_t row) {
    const size_t at = row + static_cast<size_t>(3 * stride) * P.K;
    prefetch_l2(static_cast<const T*>(P.z) + at, P.K * sizeof(T));
    prefetch_l2(static_cast<const TD*>(P.dv) + at, P.K * sizeof(TD));
  };

  request(g0, 0);
  request(g0 + stride, 1);
  copy_async_wait<1>();
  f32x2 both = 0;
  if (g0 < P.M) both = sums_of(0);
  if constexpr (kCluster) {
    post(red[0], both);
    cluster_sync_all();
  } else if (W > 1) {
    post(red[0], both);
    group_sync(bar, 32 * W);
  }
  int parity = 0, s = 0;
  for (int m = g0; m < P.M; m += stride, parity ^= 1) {
    const size_t row = static_cast<size_t>(m) * P.K;
    const int s1 = s == R::kStages - 1 ? 0 : s + 1, s2 = s1 == R::kStages - 1 ? 0 : s1 + 1;
    if constexpr (R::kStages == 3) {
      if (P.ahead && tid == 0) {
        if (P.dz_in && (P.ahead & kAheadIn) && m + stride < P.M) ahead_in(row);
        if ((P.ahead & kAheadRing) && m + 3 * stride < P.M) ahead_ring(row);
      }
    } else if constexpr (C == 4 && !kCluster) {
      if (wig == 0 && lane == 0) {
        if (P.dz_in && m + stride < P.M) ahead_in(row);
        if (m + 3 * stride < P.M) ahead_ring(row);
      }
    }
    uint4 in[C];
    if (P.dz_in) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = tid + i * step;
        if (kFull || c < chunks)
          in[i] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.dz_in) + row) + c);
      }
    }
    if constexpr (R::kStages == 3) {
      request(m + 2 * stride, s2);  // the stage of the token before: this thread has used all it read there
      copy_async_wait<1>();
    } else {
      copy_async_wait<0>();
    }
    // The next token's sums, posted a whole token ahead of their use.
    f32x2 next = 0;
    if (m + stride < P.M) next = sums_of(s1);
    if (kCluster || W > 1) {
      post(red[parity ^ 1], next);
      both = total(red[parity]);
    }
    float ss, dot;
    split2(both, ss, dot);
    both = next;
    float r = rsqrtf(fmaf(ss, P.inv_kf, P.eps));
    float mean = dot * r * P.inv_kf;
    const bool squares = !(ss > kSquaresLow && ss < kSquaresHigh);
    if (squares || !dot_in_range(dot, r)) {  // the same in the whole group
      double t = 0.0, u = 0.0;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if (kFull || tid + i * step < chunks) {
          f32x2 z[NP], d[NP];
          z_of(s, i, z);
          d_of(s, i, d);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            float lo, hi;
            split2(z[e], lo, hi);
            if (squares) {
              t = __fma_rn(static_cast<double>(lo), static_cast<double>(lo), t);
              t = __fma_rn(static_cast<double>(hi), static_cast<double>(hi), t);
            }
            if constexpr (kGain) d[e] = mul2(d[e], gains[i][e]);
            u = add_products(d[e], z[e], u);
          }
        }
      }
      auto add = [](double a, double b) { return __dadd_rn(a, b); };
      if constexpr (kCluster) {
        cluster_sync_all();  // red_d may still be read for an earlier token
        t = warp_reduce(t, add);
        u = warp_reduce(u, add);
        if (lane < cl) {
          st_cluster_b64(mapa_shared(smem_u32(&red_d[0][rank * W + wig]), static_cast<uint32_t>(lane)),
                         static_cast<f32x2>(__double_as_longlong(t)));
          st_cluster_b64(mapa_shared(smem_u32(&red_d[1][rank * W + wig]), static_cast<uint32_t>(lane)),
                         static_cast<f32x2>(__double_as_longlong(u)));
        }
        cluster_sync_all();
        t = red_d[0][0];
        u = red_d[1][0];
        for (int i = 1; i < cl * W; ++i) {
          t = add(t, red_d[0][i]);
          u = add(u, red_d[1][i]);
        }
      } else {
        if (W > 1) group_sync(bar, 32 * W);  // red_d may still be read for an earlier token
        t = group_reduce(t, add, red_d[0] + group * W, W, wig, lane, bar);
        u = group_reduce(u, add, red_d[1] + group * W, W, wig, lane, bar);
      }
      if (squares) r = rstd_of(t, P.K, P.inv_k, P.eps);
      mean = __double2float_rn(u * static_cast<double>(r) * P.inv_k);
    }
    // This token's sums are read and the next one's posted: the barrier may
    // begin, and is waited for once the token is written.
    if constexpr (kCluster) cluster_arrive_release();
    const f32x2 r2 = pack2(r, r), mean2 = pack2(-mean, -mean);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(P.dz) + row);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (kFull || c < chunks) {
        f32x2 n[NP], d[NP], o[NP];
        z_of(s, i, n);
        d_of(s, i, d);
        if (P.dz_in) {
          to_pairs<T>(in[i], o);
        } else {
#pragma unroll
          for (int e = 0; e < NP; ++e) o[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) n[e] = mul2(n[e], r2);
        if constexpr (kGain) {
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            acc[i][e] = fma2(d[e], n[e], acc[i][e]);
            d[e] = mul2(d[e], gains[i][e]);
          }
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) o[e] = fma2(r2, fma2(n[e], mean2, d[e]), o[e]);
        out[c] = from_pairs<T>(o);
      }
    }
    if constexpr (R::kStages == 2) request(m + 2 * stride, s);
    if constexpr (kCluster) {
      cluster_wait_acquire();
    } else if (W > 1) {
      group_sync(bar, 32 * W);
    }
    s = s1;
  }
  if constexpr (kGain) {
    if (P.part) {
      // One row of sums per block: its groups' rows meet in the ring, in order.
      float* out = P.part + static_cast<size_t>(kCluster ? g0 : blockIdx.x) * P.K;
      float* own = groups > 1 ? reinterpret_cast<float*>(ring) + group * P.K : out;
      if (groups > 1) {
        copy_async_wait<0>();
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = tid + i * step;
        if (kFull || c < chunks) store_pairs<NP>(own + static_cast<size_t>(c) * N, acc[i]);
      }
      if (groups > 1) {
        __syncthreads();
        for (int k = threadIdx.x; k < P.K; k += blockDim.x) {
          float t = reinterpret_cast<const float*>(ring)[k];
          for (int g = 1; g < groups; ++g) t += reinterpret_cast<const float*>(ring)[g * P.K + k];
          out[k] = t;
        }
      }
    }
  }
}

// Tokens longer than a cluster holds (131072 bf16 inputs, 65536 fp32): one
// block per token reads it twice (the second time from L2) and leaves 1 / rms
// in rstd for the gain's gradient.
template <typename T, typename TD>
__global__ void __launch_bounds__(512, 2) add_rmsnorm_backward_long_kernel(const AddNormBackParams P) {
  constexpr int N = kPer<T>, NP = kPairs<T>;
  __shared__ double red_d[kMaxGroupWarps];
  __shared__ float red_f[kMaxGroupWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = blockDim.x >> 5;
  const int chunks = P.K / N, m = blockIdx.x;
  const size_t row = static_cast<size_t>(m) * P.K;
  const uint4* zr = reinterpret_cast<const uint4*>(static_cast<const T*>(P.z) + row);
  const TD* dr = static_cast<const TD*>(P.dv) + row;
  double ss = 0.0;
  f32x2 dot2 = 0;
  auto chunk = [&](int c, f32x2 (&z)[NP], f32x2 (&gd)[NP]) {
    to_pairs<T>(__ldcg(zr + c), z);
    GradChunk<TD, N> dc;
    dc.load(dr + static_cast<size_t>(c) * N);
    dc.get(gd);
    if (P.gain) {
      f32x2 g[NP];
      load_pairs(P.gain + static_cast<size_t>(c) * N, g);
#pragma unroll
      for (int e = 0; e < NP; ++e) gd[e] = mul2(gd[e], g[e]);
    }
  };
#pragma unroll 2
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    f32x2 z[NP], gd[NP];
    chunk(c, z, gd);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      float lo, hi;
      split2(z[e], lo, hi);
      ss = __fma_rn(static_cast<double>(lo), static_cast<double>(lo), ss);
      ss = __fma_rn(static_cast<double>(hi), static_cast<double>(hi), ss);
      dot2 = fma2(gd[e], z[e], dot2);
    }
  }
  float dot, dot_hi;
  split2(dot2, dot, dot_hi);
  dot += dot_hi;
  ss = group_reduce(ss, [](double a, double b) { return __dadd_rn(a, b); }, red_d, W, warp, lane, 1);
  dot = group_reduce(dot, [](float a, float b) { return a + b; }, red_f, W, warp, lane, 1);
  const float r = rstd_of(ss, P.K, P.inv_k, P.eps);
  float mean = dot * r * P.inv_kf;
  if (!dot_in_range(dot, r)) {  // the same in the whole block
    double u = 0.0;
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
      f32x2 z[NP], gd[NP];
      chunk(c, z, gd);
#pragma unroll
      for (int e = 0; e < NP; ++e) u = add_products(gd[e], z[e], u);
    }
    u = group_reduce(u, [](double a, double b) { return __dadd_rn(a, b); }, red_d, W, warp, lane, 1);
    mean = __double2float_rn(u * static_cast<double>(r) * P.inv_k);
  }
  const f32x2 r2 = pack2(r, r), mean2 = pack2(-mean, -mean);
  if (P.rstd && threadIdx.x == 0) P.rstd[m] = r;
#pragma unroll 2
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    f32x2 z[NP], gd[NP], o[NP];
    chunk(c, z, gd);
    if (P.dz_in) {
      to_pairs<T>(__ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.dz_in) + row) + c), o);
    } else {
#pragma unroll
      for (int e = 0; e < NP; ++e) o[e] = 0;
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) o[e] = fma2(r2, fma2(mul2(z[e], r2), mean2, gd[e]), o[e]);
    reinterpret_cast<uint4*>(static_cast<T*>(P.dz) + row)[c] = from_pairs<T>(o);
  }
}

// part[p][k] = sum over tokens p, p + rows, ... of dv * (z * rstd): one
// thread per chunk of columns, block row p.
template <typename T, typename TD>
__global__ void __launch_bounds__(256) gain_grad_long_kernel(const AddNormBackParams P, int rows) {
  constexpr int N = kPer<T>, NP = kPairs<T>;
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= P.K / N) return;
  f32x2 acc[NP] = {};
#pragma unroll 4
  for (int m = blockIdx.y; m < P.M; m += rows) {
    const size_t at = static_cast<size_t>(m) * P.K + static_cast<size_t>(c) * N;
    f32x2 z[NP], d[NP];
    to_pairs<T>(__ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.z) + at)), z);
    GradChunk<TD, N> dc;
    dc.load(static_cast<const TD*>(P.dv) + at);
    dc.get(d);
    const float r = __ldcg(P.rstd + m);
    const f32x2 r2 = pack2(r, r);
#pragma unroll
    for (int e = 0; e < NP; ++e) acc[e] = fma2(d[e], mul2(z[e], r2), acc[e]);
  }
  store_pairs<NP>(P.part + static_cast<size_t>(blockIdx.y) * P.K + static_cast<size_t>(c) * N, acc);
}

// dgain[k] = the sum of the partial rows in a fixed order: 32 columns per
// block, four to a thread; 128 threads share a column's rows, so that the 592
// rows of a full grid are one batch of loads, then the warps in order.
__global__ void __launch_bounds__(1024) gain_grad_finish_kernel(const float* __restrict__ part, int rows, int K,
                                                                float* __restrict__ dgain) {
  __shared__ float sums[32][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = threadIdx.x & 7, first = threadIdx.x >> 3;
  const float* p = part + blockIdx.x * 32 + 4 * q;  // K % 64 == 0: always inside
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 5
  for (int i = first; i < rows; i += 128) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p + static_cast<size_t>(i) * K));
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
#pragma unroll
  for (int o = 8; o < 32; o *= 2) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
  }
  if (lane < 8) *reinterpret_cast<float4*>(&sums[warp][4 * q]) = a;
  __syncthreads();
  if (warp == 0) {
    float t = sums[0][lane];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += sums[i][lane];
    dgain[blockIdx.x * 32 + lane] = t;
  }
}

constexpr int kRingMax = 216 * 1024;  // of a block's shared memory, beside the static arrays

// How the backward splits its work: from the sizes and the SM count alone, so
// the workspace figure and the launch agree.
struct BackPlan {
  int W, C, threads, grid, rows;  // C = 0: the long form; rows of the partial gain gradient
  int cluster;                    // CTAs per token
};

BackPlan plan_backward(int M, int K, int per, int piece) {
  BackPlan p;
  const int chunks = K > per ? K / per : 1;  // (any K may be asked about)
  const int sms = num_sms();
  // Chunks per thread: one while a warp holds the token, two while eight do, else four.
  p.C = chunks <= 32 ? 1 : chunks <= 512 ? 2 : 4;
  // Longer than eight warps of four chunks hold: a cluster of such blocks (512
  // tokens of 28672: 34 us bf16, 50 fp32; read twice by one block each and a
  // third time for the gain 44 and 80; 1024 bf16 tokens of 8640 with fp32
  // gradients 29.5 us, 31.3 in one block of nine warps), unless 12 or 16 warps
  // hold it, an even share for an SM's four schedulers (4096 fp32 tokens of
  // 8192: 87 us, 91.8 in clusters of two); or a cluster of up to sixteen
  // warps where eight CTAs of eight are too few.
  p.cluster = 1;
  const int warps = (chunks - 1) / (32 * 4) + 1;
  if (warps > kNormThreads / 32 && (warps > kMaxGroupWarps || warps % 4 != 0)) {
    p.cluster = (chunks - 1) / (4 * kNormThreads) + 1;
    if (p.cluster > kMaxCluster) p.cluster = (chunks - 1) / (32 * 4 * kMaxGroupWarps) + 1;
  }
  p.W = (chunks - 1) / (32 * p.C * p.cluster) + 1;
  const int groups = p.cluster > 1 || p.W > kNormThreads / 32 ? 1 : kNormThreads / 32 / p.W;
  const long long ring = (piece > 32 ? 2LL : 3LL) * p.C * 32 * p.W * groups * piece;
  if (p.W > kMaxGroupWarps || p.cluster > kMaxCluster || ring > kRingMax) {
    p.C = 0;
    p.cluster = 1;
    p.W = kMaxGroupWarps;
    p.threads = 32 * kMaxGroupWarps;
    p.grid = M;
    p.rows = M < 64 ? M : 64;
    return p;
  }
  p.threads = 32 * p.W * groups;
  // What the registers (64, 80 or 128 a thread) and the ring (`piece` bytes a
  // chunk, two or three stages) let be resident.
  int resident = (p.C == 1 ? 1024 : p.C == 2 ? 768 : 512) / p.threads;
  const int by_ring = static_cast<int>(228 * 1024 / (ring + 2048));  // a block's fixed share and its other shared memory
  if (resident > by_ring) resident = by_ring;
  const int need = (M + groups - 1) / groups;
  int most = resident * sms;
  // Clusters do not use every SM: the SMs of one share a GPC (of 148 SMs, 33
  // clusters of four fit and 28 of five do not).
  if (p.cluster > 1) most = std::max(1, most / p.cluster * (p.cluster > 2 ? 7 : 8) / 8);
  p.rows = need < most ? need : most;
  p.grid = p.rows * p.cluster;
  return p;
}

template <typename T, typename TD, int C, bool kGain, bool kFull, bool kCluster>
cudaError_t launch_back_k(const AddNormBackParams& P, const BackPlan& p, cudaStream_t stream) {
  auto kernel = add_rmsnorm_backward_kernel<T, TD, C, kGain, kFull, kCluster>;
  static std::atomic<uint64_t> attr_done{0};
  const cudaError_t e = once_per_device(
      attr_done, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingMax); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(p.threads);
  cfg.dynamicSmemBytes = BackRing<T, TD>::bytes(p.threads, C);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P, p.W);
}

template <typename T, typename TD, bool kGain, bool kFull>
cudaError_t launch_back_f(const AddNormBackParams& P, const BackPlan& p, cudaStream_t stream) {
  if (p.cluster > 1) return launch_back_k<T, TD, 4, kGain, kFull, true>(P, p, stream);
  if (p.C == 1) return launch_back_k<T, TD, 1, kGain, kFull, false>(P, p, stream);
  if (p.C == 2) return launch_back_k<T, TD, 2, kGain, kFull, false>(P, p, stream);
  return launch_back_k<T, TD, 4, kGain, kFull, false>(P, p, stream);
}

template <typename T, typename TD, bool kGain>
cudaError_t launch_back_c(const AddNormBackParams& P, const BackPlan& p, cudaStream_t stream) {
  return P.K / kPer<T> == p.C * 32 * p.W * p.cluster ? launch_back_f<T, TD, kGain, true>(P, p, stream)
                                                     : launch_back_f<T, TD, kGain, false>(P, p, stream);
}

template <typename T, typename TD>
cudaError_t launch_back_t(AddNormBackParams P, float* dgain, cudaStream_t stream) {
  const BackPlan p = plan_backward(P.M, P.K, kPer<T>, BackRing<T, TD>::kChunk);
  if (!dgain) P.part = nullptr;
  // (8192 x 8192 bf16 96.1 -> 92.3 us, with dz_in alone 96.3 and with z and dv
  // alone 97.3; 8192 x 2560 51.1 -> 46.4; 8192 x 1024, many short tokens, 19.3,
  // and 20.0 with both.  fp32 tokens and clusters, which have twice and more of
  // a token under way in the ring, do best with dz_in: 512 x 28672 bf16 35.5 ->
  // 33.8, 34.8 with both; 4096 x 8192 fp32 89.7 -> 87.1 and 89.7.)
  if (sizeof(T) == 4 || p.cluster > 1) {
    P.ahead = kAheadIn;
  } else if (P.K >= 2048) {
    P.ahead = kAheadIn | kAheadRing;
  }
  cudaError_t e;
  if (p.C == 0) {
    if (!dgain) P.rstd = nullptr;
    e = launch(add_rmsnorm_backward_long_kernel<T, TD>, dim3(p.grid), dim3(p.threads), 0, stream, true, P);
    if (e != cudaSuccess || !dgain) return e;
    const int blocks = (P.K / kPer<T> + 255) / 256;
    e = launch(gain_grad_long_kernel<T, TD>, dim3(blocks, p.rows), dim3(256), 0, stream, true, P, p.rows);
  } else if (P.gain) {
    e = launch_back_c<T, TD, true>(P, p, stream);
  } else {
    e = launch_back_c<T, TD, false>(P, p, stream);
  }
  if (e != cudaSuccess || !dgain) return e;
  return launch(gain_grad_finish_kernel, dim3(P.K / 32), dim3(1024), 0, stream, true,
                static_cast<const float*>(P.part), p.rows, P.K, dgain);
}

size_t r256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_add_rmsnorm_quant(const void* x, const void* residual, int x_bf16, int M, int K, const float* gain,
                                     float eps, void* z, void* x_norm, int8_t* xq, float* scale, int32_t* rowsum,
                                     cudaStream_t stream, bool pdl) {
  if (M <= 0) return cudaSuccess;
  const AddNormParams P{x, residual, gain, eps, z, x_norm, xq, scale, rowsum, M, K, 1.0 / K};
  return x_bf16 ? launch_add_rmsnorm_quant_t<__nv_bfloat16>(P, stream, pdl)
                : launch_add_rmsnorm_quant_t<float>(P, stream, pdl);
}

cudaError_t launch_row_codes(const void* x, int x_bf16, int M, int K, int8_t* xq, float* scale, cudaStream_t stream,
                             bool pdl) {
  if (M <= 0) return cudaSuccess;
  const CodesParams P{x, xq, scale, M, K};
  return x_bf16 ? launch_row_codes_t<__nv_bfloat16>(P, stream, pdl) : launch_row_codes_t<float>(P, stream, pdl);
}

// Partial rows, then 1 / rms of the long form; for dv of either type.
static size_t part_bytes(int M, int K, int z_bf16) {
  const int per = z_bf16 ? 8 : 4;
  const BackPlan a = plan_backward(M, K, per, 16 + 2 * per), b = plan_backward(M, K, per, 16 + 4 * per);
  return r256(static_cast<size_t>(a.rows > b.rows ? a.rows : b.rows) * K * 4);
}

size_t add_rmsnorm_backward_scratch_bytes(int M, int K, int z_bf16) {
  if (M <= 0 || K <= 0) return 0;
  return part_bytes(M, K, z_bf16) + r256(static_cast<size_t>(M) * 4);
}

cudaError_t launch_add_rmsnorm_backward(const void* z, int z_bf16, const void* dnorm, int dnorm_bf16, int M, int K,
                                        const float* gain, float eps, const void* dz_in, void* dz, float* dgain,
                                        uint8_t* scratch, cudaStream_t stream) {
  if (M <= 0) return cudaSuccess;
  AddNormBackParams P{z, dnorm, gain, dz_in, eps, dz, nullptr, nullptr, M, K, 1.0 / K, static_cast<float>(1.0 / K)};
  if (scratch) {
    P.part = reinterpret_cast<float*>(scratch);
    P.rstd = reinterpret_cast<float*>(scratch + part_bytes(M, K, z_bf16));
  }
  if (z_bf16)
    return dnorm_bf16 ? launch_back_t<__nv_bfloat16, __nv_bfloat16>(P, dgain, stream)
                      : launch_back_t<__nv_bfloat16, float>(P, dgain, stream);
  return dnorm_bf16 ? launch_back_t<float, __nv_bfloat16>(P, dgain, stream)
                    : launch_back_t<float, float>(P, dgain, stream);
}

}  // namespace bl
