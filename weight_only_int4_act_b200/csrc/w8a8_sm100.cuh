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

// Kernels that come in chains (a quantiser and its product, a cache write and the
// attention) overlap each other's launch: the first one lets the next start as
// soon as all of its blocks have, and that one waits, its barriers and tensor
// memory set up, until the first has ended and its writes are there. Nothing is
// read or written before the wait. A kernel that allocates tensor memory lets the
// next one start only once it has it: all that a waiting kernel holds, it holds
// until the kernels before it have ended, and those must not need it.
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// The row's largest |v| as bits: for floats without their sign the order of the
// bits is the order of the values, infinity and NaN above all finite ones.
constexpr uint32_t Q8_INF = 0x7f800000u, Q8_FLOOR = 0x322bcc77u;  // infinity, 1e-8f

// 8 channels of a row: v = x, x s or x (1 / s).
template <bool F16, int MODE>
__device__ __forceinline__ void q8_values(const uint4& raw, const float (&f)[8], float (&v)[8]) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = widen2<F16>(u[i]);
    v[2 * i] = MODE == Q8_PLAIN ? p.x : __fmul_rn(p.x, f[2 * i]);
    v[2 * i + 1] = MODE == Q8_PLAIN ? p.y : __fmul_rn(p.y, f[2 * i + 1]);
  }
}
template <int MODE>
__device__ __forceinline__ void q8_factors(const float* __restrict__ s, int c, float (&f)[8]) {
  if constexpr (MODE != Q8_PLAIN) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(s) + 2 * c), b = __ldg(reinterpret_cast<const float4*>(s) + 2 * c + 1);
    const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = MODE == Q8_MUL ? g[i] : __frcp_rn(g[i]);
  }
}
__device__ __forceinline__ uint32_t q8_top(const float (&v)[8], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return top;
}
// 8 codes; a row that is not finite gets zeros.
__device__ __forceinline__ uint2 q8_codes(const float (&v)[8], float inv, bool finite) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = round_bits(__fmul_rn(v[i], inv));
  const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return finite ? make_uint2(lo, hi) : make_uint2(0, 0);
}
// The maximum over the block; red: 32 words, not in use by the call before.
__device__ __forceinline__ uint32_t q8_block_max(uint32_t top, uint32_t* red) {
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0u);
}

// A block takes rows blockIdx.x, + gridDim.x, ...; a thread keeps CH fixed
// chunks of 8 channels (tid + k blockDim), so 1 / s is taken once a launch and
// a row is read once: it stays in registers between its maximum and its codes,
// and the next row's loads are under way meanwhile. Bound by HBM (3 bytes a
// channel): 16384 x 8192 bf16 with 1 / s takes 74 to 87 us, 4.6 to 5.4 TB/s.
template <bool F16, int MODE, int CH>
__global__ void quantize_int8_rows(const void* __restrict__ xv, long long ldx, const float* __restrict__ s, long long rows,
                                   int d_in, int8_t* __restrict__ q, float* __restrict__ step) {
  let_next_kernel_start();
  wait_for_kernel_before();
  const uint16_t* x = static_cast<const uint16_t*>(xv);
  __shared__ uint32_t red[2][32];
  const int n8 = d_in / 8, tid = threadIdx.x, T = blockDim.x;
  float f[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k)
    if (tid + k * T < n8) q8_factors<MODE>(s, tid + k * T, f[k]);
  uint4 next[CH];
  auto load = [&](long long r) {
#pragma unroll
    for (int k = 0; k < CH; ++k)
      next[k] = r < rows && tid + k * T < n8 && AWQ_SPAN_OK(r * ldx + 8 * (tid + k * T), 8, (rows - 1) * ldx + d_in, BS_Q8_IN)
                    ? __ldcs(reinterpret_cast<const uint4*>(x + r * ldx) + tid + k * T)
                    : make_uint4(0, 0, 0, 0);
  };
  load(blockIdx.x);
  int turn = 0;
  for (long long r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
    uint4 raw[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) raw[k] = next[k];
    load(r + gridDim.x);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < CH; ++k)
      if (tid + k * T < n8) {
        float v[8];
        q8_values<F16, MODE>(raw[k], f[k], v);
        top = q8_top(v, top);
      }
    top = q8_block_max(top, red[turn]);
    const bool finite = top < Q8_INF;
    const float most = __uint_as_float(max(top, Q8_FLOOR)), inv = __fdiv_rn(127.0f, most);
    if (tid == 0 && AWQ_IDX_OK(r, rows, BS_Q8_STEP)) step[r] = finite ? __fdiv_rn(most, 127.0f) : __int_as_float(0x7fffffff);
#pragma unroll
    for (int k = 0; k < CH; ++k)
      if (tid + k * T < n8) {
        float v[8];
        q8_values<F16, MODE>(raw[k], f[k], v);
        const int c = tid + k * T;
        if (AWQ_SPAN_OK(r * d_in + 8 * c, 8, rows * d_in, BS_Q8_CODES))
          *reinterpret_cast<uint2*>(q + r * d_in + 8 * c) = q8_codes(v, inv, finite);
      }
  }
}

// Rows too long for registers: read twice (the second time mostly out of L2).
template <bool F16, int MODE>
__global__ void __launch_bounds__(1024)
    quantize_int8_long(const void* __restrict__ xv, long long ldx, const float* __restrict__ s, long long rows, int d_in,
                       int8_t* __restrict__ q, float* __restrict__ step) {
  let_next_kernel_start();
  wait_for_kernel_before();
  const uint16_t* x = static_cast<const uint16_t*>(xv);
  __shared__ uint32_t red[2][32];
  const int n8 = d_in / 8;
  int turn = 0;
  for (long long r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
    auto load = [&](int c) {
      return AWQ_SPAN_OK(r * ldx + 8 * c, 8, (rows - 1) * ldx + d_in, BS_Q8_IN)
                 ? __ldg(reinterpret_cast<const uint4*>(x + r * ldx) + c)
                 : make_uint4(0, 0, 0, 0);
    };
    uint32_t top = 0;
    for (int c = threadIdx.x; c < n8; c += blockDim.x) {
      float f[8], v[8];
      q8_factors<MODE>(s, c, f);
      q8_values<F16, MODE>(load(c), f, v);
      top = q8_top(v, top);
    }
    top = q8_block_max(top, red[turn]);
    const bool finite = top < Q8_INF;
    const float most = __uint_as_float(max(top, Q8_FLOOR)), inv = __fdiv_rn(127.0f, most);
    if (threadIdx.x == 0 && AWQ_IDX_OK(r, rows, BS_Q8_STEP))
      step[r] = finite ? __fdiv_rn(most, 127.0f) : __int_as_float(0x7fffffff);
    for (int c = threadIdx.x; c < n8; c += blockDim.x) {
      float f[8], v[8];
      q8_factors<MODE>(s, c, f);
      q8_values<F16, MODE>(load(c), f, v);
      if (AWQ_SPAN_OK(r * d_in + 8 * c, 8, rows * d_in, BS_Q8_CODES))
        *reinterpret_cast<uint2*>(q + r * d_in + 8 * c) = q8_codes(v, inv, finite);
    }
  }
}

// What a serving kernel finds wrong goes to its call's workspace and, as many
// calls leave theirs to be forgotten, to one word of the device as well: the
// first code since awq_device_error() last read it.
__device__ int g_device_err;
__device__ __forceinline__ void keep_device_error(int code) { atomicCAS(&g_device_err, 0, code); }

// mbar_wait for handshakes on the critical path: try_wait itself sleeps in
// hardware for a while, and the clock, whose read costs about a microsecond, is
// looked at only after many tries. Same bound and same effects when it gives up.
// ns > 0: sleep so long between tries, where there is time, to leave the issue slots to others.
__device__ __forceinline__ bool mbar_wait_lean(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code,
                                               uint32_t ns = 0) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (ns) __nanosleep(ns);
    if ((it & 255u) == 0) {
      if (*abort_flag) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > AWQ_WAIT_LIMIT_NS) {
        *abort_flag = 1;
        if (err) {
          atomicCAS(err, 0, code);
          keep_device_error(code);
        }
        return false;
      }
    }
  }
}

// ------------------------------------------------------------------ tensor-core product
// Output channels are the M rows of tcgen05.mma kind::i8 (128 a CTA; 256 over a
// CTA pair) and tokens the N columns (BN of them, a multiple of 16, or of 32 in
// a pair), so a few tokens still fill an instruction and a TMEM lane is an
// output channel: an epilogue warp stores 32 consecutive channels of a token.
// One K step is 128 channels (128 bytes, one swizzled row; 4 MMAs of K = 32).
//
// w8a8_gemm_tcgen05 (many tokens): G workers (CTAs, or CTA pairs) take whole
// tiles c, c + G, ... The accumulators are double, so that an epilogue runs
// under the next tile. Roles (320 threads, one CTA per SM): warp 0 TMA, warp 1
// TMEM and MMAs, warps 2..9 epilogue (two on each quarter of the TMEM lanes:
// with one a 256-token tile's epilogue took 10 us, as long as 28 K steps).
// Bound by what an SM can fetch from L2: about 80 bytes a ns were measured, so
// the plan takes the tile shape with the fewest bytes an SM. Measured, with the
// time at twice the bf16 rate: 16384 tokens of 28672 x 8192 2.44 to 2.57 ms
// under the power cap (2.32), 1000 of 4096 x 11008 32 us (27), 333 of
// 11008 x 4096 22 us (9: 129 tiles for 74 pairs are two waves, and the pipeline's
// fill and the last epilogue are 4 us of them).
//
// w8a8_small_tcgen05 (few tokens): the weights' bytes are the bound, and 128 of
// its channels a CTA are too few CTAs. So a cluster of S CTAs shares a tile,
// each over its S-th of K, several CTAs to an SM; at the end they add their
// int32 accumulators through distributed shared memory (exact in any order).
// Measured: 16 tokens of 28672 x 8192 41.5 us, 5.7 TB/s (36 us at a copy's rate);
// one of 4096 x 4096 5.3 us (2.6) behind other kernels, 6.5 alone.
constexpr int W8_BM = 128;
constexpr int W8_BK = 128;
constexpr int W8_A_STAGE = W8_BM * W8_BK;
constexpr int W8_MAX_STAGES = 12;
constexpr int W8_NBARS = 2 * W8_MAX_STAGES + 5;
constexpr int W8_SMEM_LIMIT = 232448;
constexpr int W8_SMS = 148;      // CTAs of the plan: one per SM
constexpr int W8_EPI = 8;        // epilogue warps
constexpr int W8_THREADS = 64 + 32 * W8_EPI;
constexpr int W8_SMALL_THREADS = 192;
constexpr int W8_SMALL_N = 128;  // tokens up to which the small kernel runs

__host__ __device__ constexpr int w8_stage_bytes(int b_rows) { return W8_A_STAGE + b_rows * W8_BK; }
__host__ __device__ constexpr int w8_smem_bytes(int stages, int b_rows) {
  return 1024 + stages * w8_stage_bytes(b_rows) + W8_NBARS * 8 + 64 + W8_EPI * 128 * 4;
}

__host__ __device__ constexpr int w8_small_smem(int stages, int bn) {
  return 1024 + stages * w8_stage_bytes(bn) + W8_NBARS * 8 + 64 + W8_SMALL_N * 4;
}

constexpr int ERR_W8_EMPTY = 0x501, ERR_W8_FULL = 0x502, ERR_W8_TFULL = 0x503, ERR_W8_TEMPTY = 0x504;

struct W8Args {
  int N, d_out;
  int bn;                // tokens of a tile
  int n_mb, n_nb, n_kb;  // tiles of channels and tokens, K steps
  int group_nb;          // token tiles that neighbouring workers share a weight tile over
  int stages;
  int cols;              // small kernel: TMEM columns
  int split;             // small kernel: CTAs of a cluster
  const float *dx, *dw, *bias;
  void* Y;
  int* err;
};

__host__ __device__ inline void w8_tile(const W8Args& a, long long t, int& mb, int& nb) {
  const long long per = (long long)a.n_mb * a.group_nb, grp = t / per, in = t - grp * per;
  const int first = (int)grp * a.group_nb;
  const int width = a.n_nb - first < a.group_nb ? a.n_nb - first : a.group_nb;
  nb = first + (int)(in % width);
  mb = (int)(in / width);
}

// Instruction descriptor, kind::i8: signed 8-bit A and B (K-major), int32 D.
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
template <bool PAIR>
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ float w8_scale(int acc, float dx, float dw) {
  return __fmul_rn(__fmul_rn(__int2float_rn(acc), dx), dw);
}

// One channel's sums of tokens 32 c .. of a tile (jn of them, at most 32) to Y: y is the first's place.
template <bool F16>
__device__ __forceinline__ void w8_store32(const W8Args& a, const uint32_t (&v)[32], const float* dx, float dw, float bias,
                                           bool biased, long long e0, int jn) {
  uint16_t* y = static_cast<uint16_t*>(a.Y) + e0;
  const long long ld = a.d_out, all = (long long)a.N * a.d_out;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 d4 = *reinterpret_cast<const float4*>(dx + j);
    float r[4] = {w8_scale((int)v[j], d4.x, dw), w8_scale((int)v[j + 1], d4.y, dw), w8_scale((int)v[j + 2], d4.z, dw),
                  w8_scale((int)v[j + 3], d4.w, dw)};
    if (biased) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = __fadd_rn(r[i], bias);
    }
    const uint32_t p0 = pack2<F16>(r[0], r[1]), p1 = pack2<F16>(r[2], r[3]);
    if (j < jn && AWQ_IDX_OK(e0 + j * ld, all, BS_W8_Y)) y[0] = (uint16_t)p0;
    if (j + 1 < jn && AWQ_IDX_OK(e0 + (j + 1) * ld, all, BS_W8_Y)) y[ld] = (uint16_t)(p0 >> 16);
    if (j + 2 < jn && AWQ_IDX_OK(e0 + (j + 2) * ld, all, BS_W8_Y)) y[2 * ld] = (uint16_t)p1;
    if (j + 3 < jn && AWQ_IDX_OK(e0 + (j + 3) * ld, all, BS_W8_Y)) y[3 * ld] = (uint16_t)(p1 >> 16);
    y += 4 * ld;
  }
}

template <bool PAIR, bool F16>
__device__ __forceinline__ void w8a8_body(const CUtensorMap& tmW, const CUtensorMap& tmX, const W8Args& args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int bn = args.bn, stages = args.stages;
  const int b_rows = PAIR ? bn / 2 : bn;  // token rows this CTA loads
  const uint32_t b_stage = (uint32_t)b_rows * W8_BK, stage_bytes = W8_A_STAGE + b_stage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + stages * stage_bytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + W8_NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // [epilogue warps][128] steps of the tokens; 16-byte aligned (29 barriers and 64 bytes behind a 1024-byte boundary)
  float* sdx = reinterpret_cast<float*>(tmem_slot + 14);
  static_assert((W8_NBARS * 8 + 14 * 4) % 16 == 0, "sdx is read 16 bytes at a time");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? (cluster_ctarank() & 1u) : 0u;
  const bool lead = rank == 0;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, G = PAIR ? gridDim.x >> 1 : gridDim.x;
  const long long tiles = (long long)args.n_mb * args.n_nb;
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + W8_MAX_STAGES + s); };
  auto tfull = [&](int a) { return smem_u32(bars + 2 * W8_MAX_STAGES + a); };
  auto tempty = [&](int a) { return smem_u32(bars + 2 * W8_MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = smem_u32(bars + 2 * W8_MAX_STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), PAIR ? 2 * W8_EPI : W8_EPI);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // barriers of both CTAs initialised before any remote use
  tc_fence_after();
  let_next_kernel_start();
  wait_for_kernel_before();
  // the error word of this call: only waits that give up after two seconds write it
  if (blockIdx.x == 0 && threadIdx.x == 0) *args.err = 0;
  const uint32_t tmem_base = *tmem_slot;
  constexpr int acc_stride = 256;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA: this CTA's 128 weight rows and b_rows token rows of each K step
      Ring ring;
      uint32_t issued = 0, last_parity = 0;
      bool ok = true;
      for (long long t = worker; ok && t < tiles; t += G) {
        int mb, nb;
        w8_tile(args, t, mb, nb);
        const int wrow = (mb * (PAIR ? 2 : 1) + (int)rank) * W8_BM, xrow = nb * bn + (int)rank * b_rows;
        for (int kb = 0; kb < args.n_kb; ++kb) {
          if (!mbar_wait_lean(empty(ring.stage), ring.phase ^ 1u, abort_flag, args.err, ERR_W8_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem + ring.stage * stage_bytes), sb = sa + W8_A_STAGE;
          if constexpr (PAIR) {
            const uint32_t bar = mapa_shared(full(ring.stage), 0);
            if (lead) mbar_arrive_expect_tx(full(ring.stage), 2 * stage_bytes);
            tma_load_2d_pair(sa, &tmW, bar, kb * W8_BK, wrow);
            tma_load_2d_pair(sb, &tmX, bar, kb * W8_BK, xrow);
          } else {
            mbar_arrive_expect_tx(full(ring.stage), stage_bytes);
            tma_load_2d(sa, &tmW, full(ring.stage), kb * W8_BK, wrow);
            tma_load_2d(sb, &tmX, full(ring.stage), kb * W8_BK, xrow);
          }
          issued |= 1u << ring.stage;
          last_parity = (last_parity & ~(1u << ring.stage)) | (ring.phase << ring.stage);
          ring.next(stages);
        }
      }
      if (lead) {
        for (int s = 0; s < stages; ++s)
          if (issued & (1u << s)) mbar_wait_drain(full(s), (last_parity >> s) & 1u);
      } else if (*abort_flag) {
        // on an aborted run, give this CTA's unconsumed loads time to land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && lead) {
      // ---------------- MMA issuer
      const uint32_t idesc = idesc_i8_s32(PAIR ? 2 * W8_BM : W8_BM, bn);
      const uint64_t d0 = desc_kmajor_sw128(smem_u32(smem));
      Ring ring;
      bool ok = true;
      int local = 0;
      for (long long t = worker; ok && t < tiles; t += G, ++local) {
        const int acc = local & 1;
        if (!mbar_wait_lean(tempty(acc), ((local >> 1) & 1) ^ 1u, abort_flag, args.err, ERR_W8_TEMPTY)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * acc_stride;
        for (int kb = 0; kb < args.n_kb; ++kb) {
          if (!mbar_wait_lean(full(ring.stage), ring.phase, abort_flag, args.err, ERR_W8_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = d0 + ((uint64_t)(ring.stage * stage_bytes) >> 4), db = da + (W8_A_STAGE >> 4);
#pragma unroll
          for (int k = 0; k < W8_BK / 32; ++k) mma_i8<PAIR>(d_tmem, da + 2 * k, db + 2 * k, idesc, kb != 0 || k);
          if constexpr (PAIR)
            mma_commit_pair(empty(ring.stage), 0x3);
          else
            mma_commit(empty(ring.stage));
          ring.next(stages);
        }
        if (ok) {
          if constexpr (PAIR)
            mma_commit_pair(tfull(acc), 0x3);
          else
            mma_commit(tfull(acc));
        }
      }
      if constexpr (PAIR)
        mma_commit_pair(drain_bar, 0x1);
      else
        mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0);
    }
  } else {
    // ---------------- epilogue: warp w reads TMEM lanes 32 (w % 4) .., every other 32 tokens
    const int quad = warp & 3, half = (warp - 2) >> 2;
    float* dxs = sdx + (warp - 2) * 128;
    int local = 0;
    for (long long t = worker; t < tiles; t += G, ++local) {
      int mb, nb;
      w8_tile(args, t, mb, nb);
      const int acc = local & 1;
      const int t0 = nb * bn, toks = min(bn, args.N - t0);
      const int o = (mb * (PAIR ? 2 : 1) + (int)rank) * W8_BM + quad * 32 + lane;
      const bool in = o < args.d_out;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int tok = 64 * c + 32 * half + lane;
        if (tok < toks) dxs[32 * c + lane] = __ldg(args.dx + t0 + tok);
      }
      const float dw = in ? __ldg(args.dw + o) : 0.0f;
      const float bias = in && args.bias ? __ldg(args.bias + o) : 0.0f;
      __syncwarp();
      const bool ready = mbar_wait_lean(tfull(acc), (local >> 1) & 1u, abort_flag, args.err, ERR_W8_TFULL);
      if (!__all_sync(0xffffffffu, ready)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + acc * acc_stride;
      for (int c = half; c * 32 < toks; c += 2) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c * 32, v);
        tmem_ld_wait();
        if (in)
          w8_store32<F16>(args, v, dxs + 32 * (c >> 1), dw, bias, args.bias != nullptr,
                          (long long)(t0 + c * 32) * args.d_out + o, min(32, toks - c * 32));
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (lead)
          mbar_arrive(tempty(acc));
        else
          mbar_arrive_remote(mapa_shared(tempty(acc), 0));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // all MMAs drained, all TMEM reads and remote arrivals done in both CTAs
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

template <bool F16>
__global__ void __launch_bounds__(W8_THREADS, 1)
    w8a8_gemm_tcgen05(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ W8Args args) {
  w8a8_body<false, F16>(tmW, tmX, args);
}
template <bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(W8_THREADS, 1)
    w8a8_gemm_pair_tcgen05(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                           const __grid_constant__ W8Args args) {
  w8a8_body<true, F16>(tmW, tmX, args);
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// One tile of 128 channels x bn tokens (bn <= 128, all of them) and one S-th of
// K per CTA; blockIdx.x = tile * S + rank in the cluster.
template <bool F16>
__global__ void __launch_bounds__(W8_SMALL_THREADS)
    w8a8_small_tcgen05(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ W8Args args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int bn = args.bn, stages = args.stages, S = args.split;
  const uint32_t stage_bytes = w8_stage_bytes(bn);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + stages * stage_bytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + W8_NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sdx = reinterpret_cast<float*>(tmem_slot + 14);  // [128] steps of the tokens
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mb = blockIdx.x / S, rank = blockIdx.x - mb * S;
  const int kb0 = (int)((long long)args.n_kb * rank / S), kb1 = (int)((long long)args.n_kb * (rank + 1) / S);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + W8_MAX_STAGES + s); };
  const uint32_t tfull = smem_u32(bars + 2 * W8_MAX_STAGES);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(tfull, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), args.cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  let_next_kernel_start();
  wait_for_kernel_before();
  if (blockIdx.x == 0 && threadIdx.x == 0) *args.err = 0;
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      Ring ring;
      uint32_t issued = 0, last_parity = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_lean(empty(ring.stage), ring.phase ^ 1u, abort_flag, args.err, ERR_W8_EMPTY)) break;
        const uint32_t sa = smem_u32(smem + ring.stage * stage_bytes);
        mbar_arrive_expect_tx(full(ring.stage), stage_bytes);
        tma_load_2d(sa, &tmW, full(ring.stage), kb * W8_BK, mb * W8_BM);
        tma_load_2d(sa + W8_A_STAGE, &tmX, full(ring.stage), kb * W8_BK, 0);
        issued |= 1u << ring.stage;
        last_parity = (last_parity & ~(1u << ring.stage)) | (ring.phase << ring.stage);
        ring.next(stages);
      }
      for (int s = 0; s < stages; ++s)
        if (issued & (1u << s)) mbar_wait_drain(full(s), (last_parity >> s) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_i8_s32(W8_BM, bn);
      const uint64_t d0 = desc_kmajor_sw128(smem_u32(smem));
      Ring ring;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_lean(full(ring.stage), ring.phase, abort_flag, args.err, ERR_W8_FULL)) break;
        tc_fence_after();
        const uint64_t da = d0 + ((uint64_t)(ring.stage * stage_bytes) >> 4), db = da + (W8_A_STAGE >> 4);
#pragma unroll
        for (int k = 0; k < W8_BK / 32; ++k) mma_i8<false>(tmem_base, da + 2 * k, db + 2 * k, idesc, kb != kb0 || k);
        mma_commit(empty(ring.stage));
        ring.next(stages);
      }
      // (on a wait that gave up too: what was issued ends before the block does)
      mma_commit(tfull);
      mbar_wait_drain(tfull, 0);
    }
  }
  __syncwarp();
  // ---------------- epilogue (warps 2..5; warp w reads TMEM lanes 32 (w % 4) ..)
  const int quad = warp & 3, o = mb * W8_BM + quad * 32 + lane;
  const bool in = o < args.d_out, biased = args.bias != nullptr;
  int* part = reinterpret_cast<int*>(smem);  // [bn][128] int32, over the ring
  bool ready = true;
  if (warp >= 2) {
    const int tok = threadIdx.x - 64;
    if (tok < args.N) sdx[tok] = __ldg(args.dx + tok);
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const float dw = in ? __ldg(args.dw + o) : 0.0f, bias = in && biased ? __ldg(args.bias + o) : 0.0f;
    ready = __all_sync(0xffffffffu, mbar_wait_lean(tfull, 0, abort_flag, args.err, ERR_W8_TFULL)) && !*abort_flag;
    tc_fence_after();
    for (int c = 0; c * 32 < args.N && ready; ++c) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quad * 32) << 16) + c * 32, v);
      tmem_ld_wait();
      const int jn = min(32, args.N - c * 32);
      if (S == 1) {
        if (in) w8_store32<F16>(args, v, sdx + 32 * c, dw, bias, biased, (long long)(c * 32) * args.d_out + o, jn);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < jn) part[(c * 32 + j) * 128 + quad * 32 + lane] = (int)v[j];
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  if (S > 1) {
    cluster_sync();  // every CTA's accumulators are in its shared memory
    if (warp >= 2 && ready) {
      const float dw = in ? __ldg(args.dw + o) : 0.0f, bias = in && biased ? __ldg(args.bias + o) : 0.0f;
      const uint32_t mine = smem_u32(part + quad * 32 + lane);
      for (int j = rank; j < args.N; j += S) {  // tokens go round the cluster
        int sum = 0;
        for (int r = 0; r < S; ++r) sum += ld_cluster_s32(mapa_shared(mine + j * 512, (uint32_t)r));
        float y = w8_scale(sum, sdx[j], dw);
        if (biased) y = __fadd_rn(y, bias);
        const long long e = (long long)j * args.d_out + o;
        if (in && AWQ_IDX_OK(e, (long long)args.N * args.d_out, BS_W8_Y))
          static_cast<typename W4Type<F16>::T*>(args.Y)[e] = W4Type<F16>::from_float(y);
      }
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, args.cols);
  }
}

}  // namespace awq
