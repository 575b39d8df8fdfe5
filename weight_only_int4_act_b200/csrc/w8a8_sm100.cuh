// 8-bit integer linear layer on sm_100a: the per-row quantiser and the product
//   Y[t, o] = (sum_i xq[t, i] wq[o, i]) * dx[t] * dw[o] (+ bias[o])
// with one step per token (dx) and one per output channel (dw).
//
// Quantiser, row by row (rows are tokens or output channels):
//   v_i = x_i, x_i s_i (weights, W S) or x_i (1 / s_i) (activations, X S^-1);
//   top = max(max_i |v_i|, 1e-8), step = top / 127, q_i = rne(v_i (127 / top)).
// Every operation is one fp32 rounding (1 / s_i and 127 / top are correctly
// rounded quotients), so the codes are a function of the inputs alone. A row
// that holds NaN or infinity gets step NaN and codes 0: its product is NaN and
// no other row's is.
//
// The product's int32 sum is exact (d_in <= 131072: 127^2 * 131072 < 2^31), so
// neither the order of the sum nor a split of K changes a bit of the result.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "check.cuh"
#include "ptx.cuh"
#include "w4a16_sm100.cuh"

namespace awq {

enum : int { Q8_PLAIN = 0, Q8_MUL = 1, Q8_DIV = 2 };  // v = x, x s, x (1 / s)
constexpr int W8_MAX_K = 131072;

// Two 16-bit activations of a 32-bit word as floats.
template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// rne(x) of |x| < 2^22 in the low mantissa bits of the result: adding 1.5 * 2^23
// leaves a unit in the last place of 1, and the low byte is the integer's.
__device__ __forceinline__ uint32_t round_bits(float x) { return __float_as_uint(__fadd_rn(x, 12582912.0f)); }

// One block per row; 16 channels (32 bytes in, 16 bytes out) per thread and turn.
template <bool F16, int MODE>
__global__ void __launch_bounds__(256)
    quantize_int8_rows(const void* __restrict__ xv, long long ldx, const float* __restrict__ s, long long rows, int d_in,
                       int8_t* __restrict__ q, float* __restrict__ step) {
  const uint16_t* x = static_cast<const uint16_t*>(xv);
  __shared__ float red[8];
  const int n16 = d_in / 16;
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    const uint4* row = reinterpret_cast<const uint4*>(x + r * ldx);
    auto load = [&](int c, float (&v)[16]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 w = __ldg(row + 2 * c + h);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = widen2<F16>(u[i]);
          v[8 * h + 2 * i] = f.x;
          v[8 * h + 2 * i + 1] = f.y;
        }
      }
      if constexpr (MODE != Q8_PLAIN) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float si = __ldg(s + 16 * c + i);
          v[i] = __fmul_rn(v[i], MODE == Q8_MUL ? si : __frcp_rn(si));
        }
      }
    };
    float top = 0.0f;
    bool bad = false;
    for (int c = threadIdx.x; c < n16; c += blockDim.x) {
      float v[16];
      load(c, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        top = fmaxf(top, fabsf(v[i]));
        bad |= !(fabsf(v[i]) <= 3.402823466e38f);
      }
    }
    if (bad) top = __int_as_float(0x7f800000);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
    top = red[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) top = fmaxf(top, red[w]);
    const bool finite = top <= 3.402823466e38f;
    top = fmaxf(top, 1e-8f);
    const float inv = __fdiv_rn(127.0f, top);
    if (threadIdx.x == 0 && AWQ_IDX_OK(r, rows, BS_Q8_STEP))
      step[r] = finite ? __fdiv_rn(top, 127.0f) : __int_as_float(0x7fffffff);
    for (int c = threadIdx.x; c < n16; c += blockDim.x) {
      float v[16];
      load(c, v);
      uint32_t out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = round_bits(__fmul_rn(v[4 * i], inv)), b = round_bits(__fmul_rn(v[4 * i + 1], inv));
        const uint32_t e = round_bits(__fmul_rn(v[4 * i + 2], inv)), f = round_bits(__fmul_rn(v[4 * i + 3], inv));
        out[i] = finite ? __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(e, f, 0x0040), 0x5410) : 0u;
      }
      if (AWQ_SPAN_OK(r * d_in + 16 * c, 16, rows * d_in, BS_Q8_CODES))
        *reinterpret_cast<uint4*>(q + r * d_in + 16 * c) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

// Plain tile product: 64 tokens x 64 channels a block, 64 channels of K a turn.
template <bool F16>
__global__ void __launch_bounds__(256)
    w8a8_gemm_tiles(const int8_t* __restrict__ xq, const float* __restrict__ dx, const int8_t* __restrict__ wq,
                    const float* __restrict__ dw, const float* __restrict__ bias, int N, int d_out, int d_in,
                    void* __restrict__ Yv) {
  using Ty = W4Type<F16>;
  __shared__ int sx[64][17], sw[64][17];
  const long long t0 = (long long)blockIdx.y * 64, o0 = (long long)blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k = 0; k < d_in; k += 64) {
    for (int e = threadIdx.x; e < 64 * 4; e += 256) {
      const int row = e >> 2, c = e & 3;
      int4 a = make_int4(0, 0, 0, 0), b = a;
      if (k + 16 * c < d_in) {
        if (t0 + row < N) a = __ldg(reinterpret_cast<const int4*>(xq + (t0 + row) * d_in + k + 16 * c));
        if (o0 + row < d_out) b = __ldg(reinterpret_cast<const int4*>(wq + (o0 + row) * d_in + k + 16 * c));
      }
      int* pa = &sx[row][4 * c];
      int* pb = &sw[row][4 * c];
      pa[0] = a.x, pa[1] = a.y, pa[2] = a.z, pa[3] = a.w;
      pb[0] = b.x, pb[1] = b.y, pb[2] = b.z, pb[3] = b.w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      int a[4], b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        a[u] = sx[ty + 16 * u][i];
        b[u] = sw[tx + 16 * u][i];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[u][w] = __dp4a(a[u], b[w], acc[u][w]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const long long t = t0 + ty + 16 * u, o = o0 + tx + 16 * w;
      if (t >= N || o >= d_out || !AWQ_IDX_OK(t * d_out + o, (long long)N * d_out, BS_W8_Y)) continue;
      float y = __fmul_rn(__fmul_rn((float)acc[u][w], dx[t]), dw[o]);
      if (bias) y = __fadd_rn(y, bias[o]);
      static_cast<typename Ty::T*>(Yv)[t * d_out + o] = Ty::from_float(y);
    }
}

}  // namespace awq
