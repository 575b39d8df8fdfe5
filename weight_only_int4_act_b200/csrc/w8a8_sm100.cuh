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
// channel); 16384 x 8192 bf16 with 1 / s: see the design document's table.
template <bool F16, int MODE, int CH>
__global__ void quantize_int8_rows(const void* __restrict__ xv, long long ldx, const float* __restrict__ s, long long rows,
                                   int d_in, int8_t* __restrict__ q, float* __restrict__ step) {
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
  const uint16_t* x = static_cast<const uint16_t*>(xv);
  __shared__ uint32_t red[2][32];
  const int n8 = d_in / 8;
  int turn = 0;
  for (long long r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
    const uint4* row = reinterpret_cast<const uint4*>(x + r * ldx);
    uint32_t top = 0;
    for (int c = threadIdx.x; c < n8; c += blockDim.x) {
      float f[8], v[8];
      q8_factors<MODE>(s, c, f);
      q8_values<F16, MODE>(__ldg(row + c), f, v);
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
      q8_values<F16, MODE>(__ldg(row + c), f, v);
      if (AWQ_SPAN_OK(r * d_in + 8 * c, 8, rows * d_in, BS_Q8_CODES))
        *reinterpret_cast<uint2*>(q + r * d_in + 8 * c) = q8_codes(v, inv, finite);
    }
  }
}

// ------------------------------------------------------------------ tensor-core product
// Output channels are the M rows of tcgen05.mma kind::i8 (128 a CTA; 256 over a
// CTA pair) and tokens the N columns (BN of them, a multiple of 16, or of 32 in
// a pair), so a few tokens still fill an instruction and a TMEM lane is an
// output channel: an epilogue warp stores 32 consecutive channels of a token.
// One K step is 128 channels (128 bytes, one swizzled row; 4 MMAs of K = 32).
// Roles (192 threads, one CTA per SM): warp 0 TMA, warp 1 TMEM and MMAs, warps
// 2..5 epilogue out of two accumulators, so that it runs under the next tile.
//
// Work: G workers (CTAs, or pairs) first take whole tiles c, c + G, ...; the
// last one to two waves (all tiles, where there are fewer) are cut into G equal
// contiguous ranges of (tile, K step) units. A tile that several workers touch
// leaves int32 partials in slabs which w8a8_reduce adds: the sum is exact, so
// the split changes no bit.
constexpr int W8_THREADS = 192;
constexpr int W8_BM = 128;
constexpr int W8_BK = 128;
constexpr int W8_A_STAGE = W8_BM * W8_BK;
constexpr int W8_MAX_STAGES = 12;
constexpr int W8_NBARS = 2 * W8_MAX_STAGES + 5;
constexpr int W8_TMEM_COLS = 512;
constexpr int W8_SMEM_LIMIT = 232448;
constexpr int W8_SMS = 148;  // workers of the plan: one CTA per SM

__host__ __device__ constexpr int w8_stage_bytes(int b_rows) { return W8_A_STAGE + b_rows * W8_BK; }
__host__ __device__ constexpr int w8_smem_bytes(int stages, int b_rows) {
  return 1024 + stages * w8_stage_bytes(b_rows) + W8_NBARS * 8 + 64 + 4 * 256 * 4;
}

constexpr int ERR_W8_EMPTY = 0x501, ERR_W8_FULL = 0x502, ERR_W8_TFULL = 0x503, ERR_W8_TEMPTY = 0x504;

struct W8Args {
  int N, d_out;
  int bn;                // tokens of a tile
  int n_mb, n_nb, n_kb;  // tiles of channels and tokens, K steps
  int group_nb;          // token tiles that neighbouring workers share a weight tile over
  int stages;
  int whole;             // tiles [0, whole) are taken whole, strided by the workers
  long long units;       // (tiles - whole) * n_kb, cut into ranges
  const float *dx, *dw, *bias;
  void* Y;
  int* P;                // [slots][N, d_out] partials
  long long p_stride;
  int* err;
};

__host__ __device__ inline void w8_tile(const W8Args& a, long long t, int& mb, int& nb) {
  const long long per = (long long)a.n_mb * a.group_nb, grp = t / per, in = t - grp * per;
  const int first = (int)grp * a.group_nb;
  const int width = a.n_nb - first < a.group_nb ? a.n_nb - first : a.group_nb;
  nb = first + (int)(in % width);
  mb = (int)(in / width);
}

struct W8Seg {
  int mb, nb, kb0, kb1, slot;
  bool whole;  // no other worker touches the tile
};

// The segments of worker c of G, in order; every role walks the same sequence.
struct W8Sched {
  long long t, u, u1;
  int c, G;
  __device__ W8Sched(const W8Args& a, int c_, int G_) : t(c_), c(c_), G(G_) {
    u = w4_sk_begin(c, G, a.units);
    u1 = w4_sk_begin(c + 1, G, a.units);
  }
  __device__ bool next(const W8Args& a, W8Seg& g) {
    long long tile;
    g.kb0 = 0;
    g.kb1 = a.n_kb;
    g.slot = 0;
    g.whole = true;
    if (t < a.whole) {
      tile = t;
      t += G;
    } else {
      if (u >= u1) return false;
      const long long k = u / a.n_kb, t0 = k * a.n_kb;
      tile = a.whole + k;
      g.kb0 = (int)(u - t0);
      g.kb1 = (int)min((long long)a.n_kb, (long long)g.kb0 + (u1 - u));
      const long long first = w4_sk_cta(t0, G, a.units);
      g.whole = w4_sk_cta(t0 + a.n_kb - 1, G, a.units) == first;
      g.slot = (int)(c - first);
      u += g.kb1 - g.kb0;
    }
    w8_tile(a, tile, g.mb, g.nb);
    return true;
  }
};

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

template <bool F16>
__device__ __forceinline__ float w8_scale(int acc, float dx, float dw) {
  return __fmul_rn(__fmul_rn(__int2float_rn(acc), dx), dw);
}

template <bool PAIR, bool F16>
__device__ __forceinline__ void w8a8_body(const CUtensorMap& tmW, const CUtensorMap& tmX, const W8Args& args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int bn = args.bn, stages = args.stages;
  const int b_rows = PAIR ? bn / 2 : bn;  // token rows this CTA loads
  const uint32_t b_stage = (uint32_t)b_rows * W8_BK, stage_bytes = W8_A_STAGE + b_stage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + stages * stage_bytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + W8_NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sdx = reinterpret_cast<float*>(tmem_slot + 16);  // [4 epilogue warps][256]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? (cluster_ctarank() & 1u) : 0u;
  const bool lead = rank == 0;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, G = PAIR ? gridDim.x >> 1 : gridDim.x;
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
      mbar_init(tempty(a), PAIR ? 8 : 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    // the error word of this call: only waits that give up after two seconds write it
    if (blockIdx.x == 0) *args.err = 0;
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), W8_TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), W8_TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // barriers of both CTAs initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int acc_stride = 256;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA: this CTA's 128 weight rows and b_rows token rows of each K step
      Ring ring;
      uint32_t issued = 0, last_parity = 0;
      bool ok = true;
      W8Sched sched(args, worker, G);
      W8Seg g;
      while (ok && sched.next(args, g)) {
        for (int kb = g.kb0; kb < g.kb1; ++kb) {
          if (!mbar_wait(empty(ring.stage), ring.phase ^ 1u, abort_flag, args.err, ERR_W8_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem + ring.stage * stage_bytes), sb = sa + W8_A_STAGE;
          const int wrow = (g.mb * (PAIR ? 2 : 1) + (int)rank) * W8_BM, xrow = g.nb * bn + (int)rank * b_rows;
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
      W8Sched sched(args, worker, G);
      W8Seg g;
      for (int local = 0; ok && sched.next(args, g); ++local) {
        const int acc = local & 1;
        if (!mbar_wait(tempty(acc), ((local >> 1) & 1) ^ 1u, abort_flag, args.err, ERR_W8_TEMPTY)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * acc_stride;
        for (int kb = g.kb0; kb < g.kb1; ++kb) {
          if (!mbar_wait(full(ring.stage), ring.phase, abort_flag, args.err, ERR_W8_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = d0 + ((uint64_t)(ring.stage * stage_bytes) >> 4), db = da + (W8_A_STAGE >> 4);
#pragma unroll
          for (int k = 0; k < W8_BK / 32; ++k) mma_i8<PAIR>(d_tmem, da + 2 * k, db + 2 * k, idesc, (kb != g.kb0) || k);
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
    // ---------------- epilogue (warp w reads TMEM lanes 32 (w % 4) ..)
    using Ty = W4Type<F16>;
    const int quad = warp & 3;
    float* dxs = sdx + (warp - 2) * 256;
    W8Sched sched(args, worker, G);
    W8Seg g;
    for (int local = 0; sched.next(args, g); ++local) {
      const int acc = local & 1;
      const int t0 = g.nb * bn, toks = min(bn, args.N - t0);
      const int o = (g.mb * (PAIR ? 2 : 1) + (int)rank) * W8_BM + quad * 32 + lane;
      const bool in = o < args.d_out;
      if (g.whole)
        for (int j = lane; j < toks; j += 32) dxs[j] = __ldg(args.dx + t0 + j);
      const float dw = g.whole && in ? __ldg(args.dw + o) : 0.0f;
      const float bias = g.whole && in && args.bias ? __ldg(args.bias + o) : 0.0f;
      __syncwarp();
      const bool ready = mbar_wait_sleep(tfull(acc), (local >> 1) & 1u, abort_flag, args.err, ERR_W8_TFULL, 64);
      if (!__all_sync(0xffffffffu, ready)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + acc * acc_stride;
      for (int c = 0; c * 32 < toks; ++c) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c * 32, v);
        tmem_ld_wait();
        const int jn = min(32, toks - c * 32);
        const long long e0 = (long long)(t0 + c * 32) * args.d_out + o;
        if (in && g.whole) {
          typename Ty::T* y = static_cast<typename Ty::T*>(args.Y) + e0;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float r = w8_scale<F16>((int)v[j], dxs[c * 32 + j], dw);
            if (args.bias) r = __fadd_rn(r, bias);
            if (j < jn && AWQ_IDX_OK(e0 + (long long)j * args.d_out, (long long)args.N * args.d_out, BS_W8_Y))
              y[(long long)j * args.d_out] = Ty::from_float(r);
          }
        } else if (in) {
          int* P = args.P + (long long)g.slot * args.p_stride + e0;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < jn && AWQ_IDX_OK(e0 + (long long)j * args.d_out, (long long)args.N * args.d_out, BS_W8_P))
              P[(long long)j * args.d_out] = (int)v[j];
        }
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
      tmem_dealloc_pair(tmem_base, W8_TMEM_COLS);
    else
      tmem_dealloc(tmem_base, W8_TMEM_COLS);
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

// Tiles that two or more workers touch, found on the host from the shapes.
struct W8Fixups {
  int n;
  int tile[W8_SMS];
  short ns[W8_SMS];
};

// Block (b, y) adds the partials of split tile fx.tile[b] for 1024 of its
// elements (channel fastest) and writes them scaled and rounded.
template <bool F16>
__global__ void __launch_bounds__(256) w8a8_reduce(const W8Args a, int bm, const __grid_constant__ W8Fixups fx) {
  using Ty = W4Type<F16>;
  if (!AWQ_IDX_OK(blockIdx.x, fx.n, BS_W8_P)) return;
  int mb, nb;
  w8_tile(a, fx.tile[blockIdx.x], mb, nb);
  const int ns = fx.ns[blockIdx.x];
  const int o0 = mb * bm, t0 = nb * a.bn;
  const int rows = min(bm, a.d_out - o0), toks = min(a.bn, a.N - t0);
  long long idx[4];
  bool in[4];
  int acc[4], oo[4], tt[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int e = blockIdx.y * 1024 + k * 256 + threadIdx.x;
    const int j = e / rows, r = e - j * rows;
    tt[k] = t0 + j;
    oo[k] = o0 + r;
    idx[k] = (long long)tt[k] * a.d_out + oo[k];
    in[k] = e < rows * toks && AWQ_IDX_OK(idx[k], (long long)a.N * a.d_out, BS_W8_P);
    acc[k] = 0;
  }
  for (int s = 0; s < ns; ++s) {
    const int* P = a.P + (long long)s * a.p_stride;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (in[k]) acc[k] += P[idx[k]];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (in[k]) {
      float y = w8_scale<F16>(acc[k], __ldg(a.dx + tt[k]), __ldg(a.dw + oo[k]));
      if (a.bias) y = __fadd_rn(y, __ldg(a.bias + oo[k]));
      static_cast<typename Ty::T*>(a.Y)[idx[k]] = Ty::from_float(y);
    }
}

}  // namespace awq
