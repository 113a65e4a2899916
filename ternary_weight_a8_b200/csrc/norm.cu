// The residual sum, the RMSNorm after it and the activation codes in one pass
// (add_rmsnorm_quant), and the gradient of the sum and the norm
// (add_rmsnorm_backward).
//
// Forward, for a token of K inputs:
//   z = T(x + residual)                       fp32 sum, rounded to the activation type T and stored
//   r = fp32(1 / sqrt(mean_k z^2 + eps))      squares summed in double, as rmsnorm_quant does
//   v = T((z * r) * g)                        fp32 products
//   s = 127 / max(max_k |v|, 1e-5),  q = clamp(rint(v * s)),  rowsum = sum_k q
// so the codes equal rmsnorm_quant's on z bit for bit.
//
// Backward, with n = z * r and the quantisation as the identity
// (straight-through), for the gradient dv of v and dz_in of z:
//   dz = r * (gd - n * mean_k(gd * n)) + dz_in,  gd = dv * g
//   dg = sum over tokens of dv * n
// dz is the gradient of x and of the residual alike.
//
// Both are bound by memory: 7 bytes per bf16 input forward (x, residual, z,
// codes), 8 backward (z, dv, dz_in, dz).
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace bl {

namespace {

// 16 bytes of activations: 8 bf16 or 4 fp32.
template <typename T>
constexpr int kPer = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ uint32_t bf16_bits_rn(float v) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v)));
}

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& w, float (&f)[kPer<T>]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      f[2 * i] = __uint_as_float(u[i] << 16);  // bf16 -> fp32 is exact
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(u[i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&f)[kPer<T>]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      u[i] = bf16_bits_rn(f[2 * i]) | (bf16_bits_rn(f[2 * i + 1]) << 16);
    } else {
      u[i] = __float_as_uint(f[i]);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// N consecutive fp32 values (the gains of a chunk, 16-byte aligned).
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p) + i);
    f[4 * i] = q.x;
    f[4 * i + 1] = q.y;
    f[4 * i + 2] = q.z;
    f[4 * i + 3] = q.w;
  }
}

// Codes of N values (4 or 8), stored together; returns their sum.
template <int N>
__device__ __forceinline__ int store_codes(const float (&v)[N], float s, int8_t* dst) {
  uint32_t w[N / 4];
  int sum = 0;
#pragma unroll
  for (int b = 0; b < N / 4; ++b) {
    int q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = min(max(__float2int_rn(__fmul_rn(v[4 * b + e], s)), -128), 127);
    const uint32_t lo = __byte_perm(static_cast<uint32_t>(q[0]), static_cast<uint32_t>(q[1]), 0x5140);
    const uint32_t hi = __byte_perm(static_cast<uint32_t>(q[2]), static_cast<uint32_t>(q[3]), 0x5140);
    w[b] = __byte_perm(lo, hi, 0x5410);
    sum = __dp4a(static_cast<int>(w[b]), 0x01010101, sum);
  }
  if constexpr (N == 8) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
  return sum;
}

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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

__device__ __forceinline__ float rstd_of(double ss, int K, float eps) {
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
};

// C: 16-byte chunks of a token per thread, held in registers from the sum to
// the codes (z's chunk is overwritten by v's).  C = 0: the token is longer
// than the registers hold; z is read back (each thread its own chunks) for
// the absmax and again for the codes.
template <typename T, int C>
__global__ void __launch_bounds__(512) add_rmsnorm_quant_kernel(const AddNormParams P, int W) {
  constexpr int N = kPer<T>;
  __shared__ double red_d[kMaxGroupWarps];
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

  auto sum_chunk = [&](const uint4& a, const uint4& b, double& ss) {
    float fa[N], fb[N];
    unpack16<T>(a, fa);
    unpack16<T>(b, fb);
#pragma unroll
    for (int e = 0; e < N; ++e) fa[e] = round_to<T>(__fadd_rn(fa[e], fb[e]));
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double v = static_cast<double>(fa[e]);
      ss = __fma_rn(v, v, ss);
    }
    return pack16<T>(fa);
  };
  float r = 0.0f;
  auto norm_chunk = [&](const uint4& zc, int c, float (&v)[N]) {
    unpack16<T>(zc, v);
    float g[N];
    if (P.gain) load_f32<N>(P.gain + static_cast<size_t>(c) * N, g);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float t = __fmul_rn(v[e], r);
      if (P.gain) t = __fmul_rn(t, g[e]);
      v[e] = round_to<T>(t);
    }
  };

  constexpr int CR = C > 0 ? C : 1;
  uint4 keep[CR];
  double ss = 0.0;
  if constexpr (C > 0) {
    uint4 other[CR];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (c < chunks) {
        keep[i] = __ldcg(xr + c);
        other[i] = __ldcg(rr + c);
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (c < chunks) {
        keep[i] = sum_chunk(keep[i], other[i], ss);
        zr[c] = keep[i];
      }
    }
  } else {
    for (int c = tid; c < chunks; c += step) zr[c] = sum_chunk(__ldcg(xr + c), __ldcg(rr + c), ss);
  }
  ss = group_reduce(ss, [](double a, double b) { return __dadd_rn(a, b); }, red_d + group * W, W, wig, lane, bar);
  r = rstd_of(ss, P.K, P.eps);

  float amax = 0.0f;
  auto amax_of = [&](const float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) amax = fmaxf(amax, fabsf(v[e]));
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (c < chunks) {
        float v[N];
        norm_chunk(keep[i], c, v);
        amax_of(v);
        keep[i] = pack16<T>(v);  // exact: v is rounded to T
        if (nr) nr[c] = keep[i];
      }
    }
  } else {
    for (int c = tid; c < chunks; c += step) {
      float v[N];
      norm_chunk(zr[c], c, v);
      amax_of(v);
    }
  }
  amax = group_reduce(amax, [](float a, float b) { return fmaxf(a, b); }, red_f + group * W, W, wig, lane, bar);
  const float s = __fdiv_rn(127.0f, fmaxf(amax, 1e-5f));

  int sum = 0;
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (c < chunks) {
        float v[N];
        unpack16<T>(keep[i], v);
        sum += store_codes<N>(v, s, qr + static_cast<size_t>(c) * N);
      }
    }
  } else {
    for (int c = tid; c < chunks; c += step) {
      float v[N];
      norm_chunk(zr[c], c, v);
      if (nr) nr[c] = pack16<T>(v);
      sum += store_codes<N>(v, s, qr + static_cast<size_t>(c) * N);
    }
  }
  if (P.rowsum) {
    sum = group_reduce(sum, [](int a, int b) { return a + b; }, red_i + group * W, W, wig, lane, bar);
    if (tid == 0) P.rowsum[m] = sum;
  }
  if (tid == 0) P.scale[m] = s;
}

template <typename T>
cudaError_t launch_add_rmsnorm_quant_t(const AddNormParams& P, cudaStream_t stream, bool pdl) {
  const int chunks = P.K / kPer<T>;
  // Chunks per thread n and warps per token W: eight chunks per thread (the
  // fewest warps to join) while the tokens give every SM 16 warps, else fewer
  // chunks and more warps, as far as a block goes.
  int W = 0, n = 0;
  for (int c = 8; c >= 1; c /= 2) {
    const int w = (chunks + 32 * c - 1) / (32 * c);
    if (w > kMaxGroupWarps) break;
    W = w;
    n = (chunks + 32 * w - 1) / (32 * w);
    if (static_cast<long long>(P.M) * w >= 16LL * num_sms()) break;
  }
  if (W == 0) {  // longer than 16 warps hold
    W = kMaxGroupWarps;
    n = 9;
  }
  const int groups = W > kNormThreads / 32 ? 1 : kNormThreads / 32 / W;
  const int threads = 32 * W * groups;
  const dim3 grid((P.M + groups - 1) / groups);
  if (n <= 1) return launch(add_rmsnorm_quant_kernel<T, 1>, grid, dim3(threads), 0, stream, pdl, P, W);
  if (n <= 2) return launch(add_rmsnorm_quant_kernel<T, 2>, grid, dim3(threads), 0, stream, pdl, P, W);
  if (n <= 4) return launch(add_rmsnorm_quant_kernel<T, 4>, grid, dim3(threads), 0, stream, pdl, P, W);
  if (n <= 8) return launch(add_rmsnorm_quant_kernel<T, 8>, grid, dim3(threads), 0, stream, pdl, P, W);
  return launch(add_rmsnorm_quant_kernel<T, 0>, grid, dim3(threads), 0, stream, pdl, P, W);
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
  float* part;         // [rows][K] sums of dv * n over each group's tokens, or null
  float* rstd;         // [M] (long tokens only)
  int M, K;
};

// N gradient values of type TD at element offset `at` (16-byte aligned for N
// values of TD, or 8 bytes for 4 bf16 values).
template <typename TD, int N>
struct GradChunk {
  uint4 w[N * sizeof(TD) > 16 ? 2 : 1];
  __device__ __forceinline__ void load(const TD* p) {
    if constexpr (N * sizeof(TD) == 8) {
      const uint2 h = __ldcg(reinterpret_cast<const uint2*>(p));
      w[0] = make_uint4(h.x, h.y, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(N * sizeof(TD) / 16); ++i)
        w[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
    }
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (sizeof(TD) == 2) {
      float t[8];
      unpack16<__nv_bfloat16>(w[0], t);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = t[e];
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        float t[4];
        unpack16<float>(w[i], t);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * i + e] = t[e];
      }
    }
  }
};

struct SumPair {
  double ss;
  float dot;
};

// A group of W warps takes tokens group0, group0 + groups_total, ...; a
// thread owns the same C chunks of every token, so the gain's gradient is
// summed in its registers and written once per group.  The next token's z
// and dv are requested before the current token's reduction.
template <typename T, typename TD, int C, bool kGain>
__global__ void __launch_bounds__(512) add_rmsnorm_backward_kernel(const AddNormBackParams P, int W) {
  constexpr int N = kPer<T>;
  __shared__ SumPair red[2][kMaxGroupWarps];
  griddep_launch_dependents();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wig = warp % W, groups = (blockDim.x >> 5) / W;
  const int g0 = blockIdx.x * groups + group, stride = gridDim.x * groups;
  const int tid = wig * 32 + lane, step = 32 * W, chunks = P.K / N, bar = 1 + group;
  griddep_wait();

  float acc[kGain ? C : 1][N];
#pragma unroll
  for (int i = 0; i < (kGain ? C : 1); ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[i][e] = 0.0f;

  uint4 zc[C];
  GradChunk<TD, N> dc[C];
  auto fetch = [&](int m) {
    const size_t row = static_cast<size_t>(m) * P.K;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (c < chunks) {
        zc[i] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.z) + row) + c);
        dc[i].load(static_cast<const TD*>(P.dv) + row + static_cast<size_t>(c) * N);
      }
    }
  };
  int m = g0, parity = 0;
  if (m < P.M) fetch(m);
  for (; m < P.M; m += stride, parity ^= 1) {
    const size_t row = static_cast<size_t>(m) * P.K;
    uint4 in[C];
    if (P.dz_in) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = tid + i * step;
        if (c < chunks) in[i] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.dz_in) + row) + c);
      }
    }
    double ss = 0.0;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (c < chunks) {
        float z[N], d[N];
        unpack16<T>(zc[i], z);
        dc[i].get(d);
        if constexpr (kGain) {
          float g[N];
          load_f32<N>(P.gain + static_cast<size_t>(c) * N, g);
#pragma unroll
          for (int e = 0; e < N; ++e) dot = fmaf(d[e] * g[e], z[e], dot);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) dot = fmaf(d[e], z[e], dot);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const double t = static_cast<double>(z[e]);
          ss = __fma_rn(t, t, ss);
        }
      }
    }
    ss = warp_reduce(ss, [](double a, double b) { return __dadd_rn(a, b); });
    dot = warp_reduce(dot, [](float a, float b) { return a + b; });
    if (W > 1) {
      SumPair* slot = red[parity] + group * W;
      if (lane == 0) slot[wig] = SumPair{ss, dot};
      group_sync(bar, 32 * W);
      ss = slot[0].ss;
      dot = slot[0].dot;
      for (int i = 1; i < W; ++i) {
        ss = __dadd_rn(ss, slot[i].ss);
        dot += slot[i].dot;
      }
    }
    const float r = rstd_of(ss, P.K, P.eps);
    const float mean = dot * r / static_cast<float>(P.K);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(P.dz) + row);
    uint4 zo[C];
    GradChunk<TD, N> dn[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      zo[i] = zc[i];
      dn[i] = dc[i];
    }
    if (m + stride < P.M) fetch(m + stride);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = tid + i * step;
      if (c < chunks) {
        float z[N], d[N], o[N];
        unpack16<T>(zo[i], z);
        dn[i].get(d);
        if (P.dz_in) {
          unpack16<T>(in[i], o);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) o[e] = 0.0f;
        }
        float g[N];
        if constexpr (kGain) load_f32<N>(P.gain + static_cast<size_t>(c) * N, g);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float n = z[e] * r;
          if constexpr (kGain) acc[i][e] = fmaf(d[e], n, acc[i][e]);
          const float gd = kGain ? d[e] * g[e] : d[e];
          o[e] = fmaf(r, fmaf(-n, mean, gd), o[e]);
        }
        out[c] = pack16<T>(o);
      }
    }
  }
  if constexpr (kGain) {
    if (P.part) {
      float* pr = P.part + static_cast<size_t>(g0) * P.K;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = tid + i * step;
        if (c < chunks) {
#pragma unroll
          for (int e = 0; e < N / 4; ++e)
            reinterpret_cast<float4*>(pr + static_cast<size_t>(c) * N)[e] =
                make_float4(acc[i][4 * e], acc[i][4 * e + 1], acc[i][4 * e + 2], acc[i][4 * e + 3]);
        }
      }
    }
  }
}

// Tokens longer than the registers hold: one block per token reads it twice
// (the second time from L2) and leaves 1 / rms in rstd for the gain's gradient.
template <typename T, typename TD>
__global__ void __launch_bounds__(512) add_rmsnorm_backward_long_kernel(const AddNormBackParams P) {
  constexpr int N = kPer<T>;
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
  float dot = 0.0f;
  auto chunk = [&](int c, float (&z)[N], float (&d)[N], float (&gd)[N]) {
    unpack16<T>(__ldcg(zr + c), z);
    GradChunk<TD, N> dc;
    dc.load(dr + static_cast<size_t>(c) * N);
    dc.get(d);
    if (P.gain) {
      float g[N];
      load_f32<N>(P.gain + static_cast<size_t>(c) * N, g);
#pragma unroll
      for (int e = 0; e < N; ++e) gd[e] = d[e] * g[e];
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) gd[e] = d[e];
    }
  };
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    float z[N], d[N], gd[N];
    chunk(c, z, d, gd);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double t = static_cast<double>(z[e]);
      ss = __fma_rn(t, t, ss);
      dot = fmaf(gd[e], z[e], dot);
    }
  }
  ss = group_reduce(ss, [](double a, double b) { return __dadd_rn(a, b); }, red_d, W, warp, lane, 1);
  dot = group_reduce(dot, [](float a, float b) { return a + b; }, red_f, W, warp, lane, 1);
  const float r = rstd_of(ss, P.K, P.eps);
  const float mean = dot * r / static_cast<float>(P.K);
  if (P.rstd && threadIdx.x == 0) P.rstd[m] = r;
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    float z[N], d[N], gd[N], o[N];
    chunk(c, z, d, gd);
    if (P.dz_in) {
      unpack16<T>(__ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.dz_in) + row) + c), o);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = fmaf(r, fmaf(-(z[e] * r), mean, gd[e]), o[e]);
    reinterpret_cast<uint4*>(static_cast<T*>(P.dz) + row)[c] = pack16<T>(o);
  }
}

// part[p][k] = sum over tokens p, p + rows, ... of dv * (z * rstd): one
// thread per chunk of columns, block row p.
template <typename T, typename TD>
__global__ void __launch_bounds__(256) gain_grad_long_kernel(const AddNormBackParams P, int rows) {
  constexpr int N = kPer<T>;
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= P.K / N) return;
  float acc[N] = {};
  for (int m = blockIdx.y; m < P.M; m += rows) {
    const size_t at = static_cast<size_t>(m) * P.K + static_cast<size_t>(c) * N;
    float z[N], d[N];
    unpack16<T>(__ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.z) + at)), z);
    GradChunk<TD, N> dc;
    dc.load(static_cast<const TD*>(P.dv) + at);
    dc.get(d);
    const float r = __ldcg(P.rstd + m);
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = fmaf(d[e], z[e] * r, acc[e]);
  }
  float* pr = P.part + static_cast<size_t>(blockIdx.y) * P.K + static_cast<size_t>(c) * N;
#pragma unroll
  for (int e = 0; e < N / 4; ++e)
    reinterpret_cast<float4*>(pr)[e] = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
}

// dgain[k] = the sum of the partial rows in a fixed order: 32 columns per
// block, warp w rows w, w + 32, ..., then the warps in order.
__global__ void __launch_bounds__(1024) gain_grad_finish_kernel(const float* __restrict__ part, int rows, int K,
                                                                float* __restrict__ dgain) {
  __shared__ float sums[32][33];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = blockIdx.x * 32 + lane;  // K % 64 == 0: always inside
  float a = 0.0f;
#pragma unroll 4
  for (int p = warp; p < rows; p += 32) a += __ldcg(part + static_cast<size_t>(p) * K + k);
  sums[warp][lane] = a;
  __syncthreads();
  if (warp == 0) {
    float t = sums[0][lane];
    for (int i = 1; i < 32; ++i) t += sums[i][lane];
    dgain[k] = t;
  }
}

// How the backward splits its work: from the sizes and the SM count alone, so
// the workspace figure and the launch agree.
struct BackPlan {
  int W, C, threads, grid, rows;  // C = 0: the long form; rows of the partial gain gradient
};

BackPlan plan_backward(int M, int K, int per) {
  BackPlan p;
  const int chunks = K / per;
  const int sms = num_sms();
  p.W = (chunks + 31) / 32;
  if (p.W > kMaxGroupWarps) p.W = kMaxGroupWarps;
  const int n = (chunks + 32 * p.W - 1) / (32 * p.W);
  if (n > 4) {
    p.C = 0;
    p.threads = 32 * kMaxGroupWarps;
    p.grid = M;
    p.rows = M < 64 ? M : 64;
    return p;
  }
  p.C = n <= 1 ? 1 : n <= 2 ? 2 : 4;
  const int groups = p.W > kNormThreads / 32 ? 1 : kNormThreads / 32 / p.W;
  p.threads = 32 * p.W * groups;
  const int resident = p.C > 2 ? 1 : p.threads > kNormThreads ? 2 : 4;
  const int need = (M + groups - 1) / groups;
  p.grid = need < resident * sms ? need : resident * sms;
  p.rows = p.grid * groups;
  return p;
}

template <typename T, typename TD, bool kGain>
cudaError_t launch_back_c(const AddNormBackParams& P, const BackPlan& p, cudaStream_t stream) {
  const dim3 g(p.grid), b(p.threads);
  if (p.C == 1) return launch(add_rmsnorm_backward_kernel<T, TD, 1, kGain>, g, b, 0, stream, true, P, p.W);
  if (p.C == 2) return launch(add_rmsnorm_backward_kernel<T, TD, 2, kGain>, g, b, 0, stream, true, P, p.W);
  return launch(add_rmsnorm_backward_kernel<T, TD, 4, kGain>, g, b, 0, stream, true, P, p.W);
}

template <typename T, typename TD>
cudaError_t launch_back_t(AddNormBackParams P, float* dgain, cudaStream_t stream) {
  const BackPlan p = plan_backward(P.M, P.K, kPer<T>);
  if (!dgain) P.part = nullptr;
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
  const AddNormParams P{x, residual, gain, eps, z, x_norm, xq, scale, rowsum, M, K};
  return x_bf16 ? launch_add_rmsnorm_quant_t<__nv_bfloat16>(P, stream, pdl)
                : launch_add_rmsnorm_quant_t<float>(P, stream, pdl);
}

size_t add_rmsnorm_backward_scratch_bytes(int M, int K, int x_bf16) {
  if (M <= 0 || K <= 0) return 0;
  const BackPlan p = plan_backward(M, K, x_bf16 ? 8 : 4);
  return r256(static_cast<size_t>(p.rows) * K * 4) + r256(static_cast<size_t>(M) * 4);
}

cudaError_t launch_add_rmsnorm_backward(const void* z, int z_bf16, const void* dnorm, int dnorm_bf16, int M, int K,
                                        const float* gain, float eps, const void* dz_in, void* dz, float* dgain,
                                        uint8_t* scratch, cudaStream_t stream) {
  if (M <= 0) return cudaSuccess;
  AddNormBackParams P{z, dnorm, gain, dz_in, eps, dz, nullptr, nullptr, M, K};
  if (scratch) {
    const BackPlan p = plan_backward(M, K, z_bf16 ? 8 : 4);
    P.part = reinterpret_cast<float*>(scratch);
    P.rstd = reinterpret_cast<float*>(scratch + r256(static_cast<size_t>(p.rows) * K * 4));
  }
  if (z_bf16)
    return dnorm_bf16 ? launch_back_t<__nv_bfloat16, __nv_bfloat16>(P, dgain, stream)
                      : launch_back_t<__nv_bfloat16, float>(P, dgain, stream);
  return dnorm_bf16 ? launch_back_t<float, __nv_bfloat16>(P, dgain, stream)
                    : launch_back_t<float, float>(P, dgain, stream);
}

}  // namespace bl
