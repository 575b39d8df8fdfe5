// Attention of many query rows a sequence (prompts and their chunks) over the
// 4-bit cache, on tcgen05. A block takes 256 rows (token x head of the group)
// of one kv head in two tiles of 128, and walks the context in tiles of 64
// tokens:
//   S_q = Q_q K_t^T       M = 128 rows, N = 64 tokens, K = D
//   O_q += W_q V_t        M = 128 rows, N = D channels, K = 64 tokens
// with fp16 operands and fp32 accumulators in tensor memory (S_q twice, so that
// the next tile's scores are there when a softmax ends; W_q takes the place of
// its S_q).
//
// Values are unpacked as (code - zero) step 2^(10 - e): one rounding to fp16 of
// each value, off by 2^-11 of it or, where it is far below, 2^-35 of 2^e; e joins
// the weight's exponent, w = 2^(score + e - m), and leaves the sum of the p again.
// e is the exponent of the largest step in the strip of 16 tokens where those of
// its tokens lie within KVP_SPREAD of each other, so that the softmax has one
// number a strip; in other strips each token has its own, and the softmax takes
// the way that looks at every token. A row's reference m thus follows what its
// tokens weigh, p times step, to KVP_SPREAD: a token of a huge step and no
// probability does not push the others out of fp16's range. Keys have their
// strip's largest step always (what the small ones lose there is at most 2^-20
// |q| a channel of a score): that power of two goes into the
// factor of its scores; but for fp16 queries (EXACT; one group a head), whose
// output resolves it, the codes less zeros (-15 .. 15) are the keys, exactly, and
// each score is multiplied by its token's step in fp32 (2 x 2048 queries of 8000
// tokens, 32 heads over 8 of 128: 475 us that way in fp16, 454 with folded keys in
// bf16 of the same run; one read of a step from shared memory a score, beside the MMAs' operands).
// A token one of whose groups holds NaN turns the rows that see it to NaN.
//
// Measured: 2 x 2048 queries of up to 8000 tokens, 32 heads over 8 of 128: 451 us,
// 741 TFLOP/s (202 us at the bf16 rate). A context tile takes a block about 2200
// cycles. Its MMAs are 1024 cycles' work and take 1560, as N = 64 costs what
// N = 128 does (64 to 67 cycles); beside them go the exponentials of 16384 scores
// on 8 warps and the handshakes between loader, unpacking, products and softmax,
// about 300 cycles each. Blocks of unequal contexts on 148 SMs and their starts
// are the rest.
//
// Warps (15): 0 loads packed strips (cp.async.bulk), 1 and 14 issue the MMAs of
// the two row tiles (one thread for both spent as long on its handshakes as the
// tensor cores on their work), 2..5 unpack strips into the operand tiles, 6..9
// and 10..13 are the softmax of the two row tiles, a thread a row.
#pragma once
#include "kv4_sm100.cuh"

namespace awq {

constexpr int KVP_ROWS = 256, KVP_TOK = 64, KVP_THREADS = 480, KVP_STAGES = 3, KVP_RAW = 5;
constexpr int KVP_MIN_ROWS = 64;  // sequences of at most so many rows are the split kernel's
// How far apart the exponents of the tokens' largest steps may lie in a strip that
// has one for all of them.
constexpr int KVP_SPREAD = 2;
// The reference is whole, so that what is scaled when it moves keeps its digits,
// and is set such that the row's largest weight then lies in (2^3, 2^4]: with
// KVP_SPREAD and a step's mantissa taken off, its largest p step is 1 or more, and
// what falls below fp16's 2^-24 does so beside that. It may lag behind by KVP_LAG:
// weights then reach 2^15, which fp16 holds. (2 x 2048 queries of 8000 tokens: 451
// us; with a spread of 3, and so 2^5, 458; with an exponent a token in every
// strip 478; with one a strip and 2^0, whatever the steps, 442.)
constexpr float KVP_HEAD = 4.0f, KVP_LAG = 15.0f;
constexpr int ERR_KVP_RAW = 0x601, ERR_KVP_FREE = 0x602, ERR_KVP_SCORE = 0x603, ERR_KVP_WEIGHT = 0x604, ERR_KVP_OUT = 0x605,
              ERR_KVP_TILE = 0x606;

// What the softmax knows of a strip: its keys are (code - zero) step / key, its
// values (code - zero) step 2^(10 - e), down = 2^-e. odd: tokens (by bit) that hold
// NaN, and bit 16 where each token has an e of its own (KvpSmem::e).
struct KvpStrip {
  float key, e, down;
  unsigned odd;
};

template <int D, int G>
struct KvpSmem {
  static constexpr int SUB = (D + 63) / 64;                 // 64-channel sub-tiles of 128-byte rows
  static constexpr int STRIP = kv4_strip_bytes(D, G);
  alignas(1024) uint8_t q[2][SUB][128 * 128];
  alignas(1024) uint8_t k[KVP_STAGES][SUB][KVP_TOK * 128];
  alignas(1024) uint8_t v[KVP_STAGES][D * 128];
  alignas(128) uint8_t raw[KVP_RAW][4 * STRIP];
  alignas(16) KvpStrip strip[KVP_STAGES][4];
  float step[KVP_STAGES][KVP_TOK];   // EXACT: key step of a token
  float e[KVP_STAGES][KVP_TOK];      // exponent of a token's values
  float unit[2][128];                // score (log2) per unit of a row's product
  int lost_raw[KVP_RAW], lost[KVP_STAGES];  // strips (by bit) in pages outside the cache
  uint64_t raw_full[KVP_RAW], raw_empty[KVP_RAW], tile_full[KVP_STAGES], tile_empty[KVP_STAGES];
  uint64_t q_full[2], score[2][2], weight[2][2], out_done[2][2], drain[2];  // [row tile][context tile & 1]
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// 16 columns of a thread's TMEM lane.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Codes less zero of the four pairs of a word, exact in fp16: low nibbles as
// (1024 + c) - (1024 + z), high ones as (1024 + 16 c) / 16 - (64 + z).
// lo: bytes 0 and 2, bytes 1 and 3; hi: the same of the high nibbles.
struct KvpPairs {
  __half2 lo0, lo1, hi0, hi1;
  // times a factor each for (lo0, hi0) and (lo1, hi1), rounded once
  __device__ __forceinline__ void scale(__half2 m0, __half2 m1) {
    lo0 = __hmul2(lo0, m0);
    hi0 = __hmul2(hi0, m0);
    lo1 = __hmul2(lo1, m1);
    hi1 = __hmul2(hi1, m1);
  }
};
__device__ __forceinline__ KvpPairs kvp_unpack(uint32_t w, __half2 z0, __half2 z1) {
  // z0: the zeros of lo0 and hi0, z1: of lo1 and hi1
  const uint32_t x = w >> 8;
  const __half2 k1024 = __float2half2_rn(1024.0f), k64 = __float2half2_rn(64.0f), k16 = __float2half2_rn(0.0625f);
  auto h2 = [](uint32_t u) { return *reinterpret_cast<const __half2*>(&u); };
  KvpPairs p;
  p.lo0 = __hsub2(h2((w & 0x000F000Fu) | 0x64006400u), __hadd2(k1024, z0));
  p.lo1 = __hsub2(h2((x & 0x000F000Fu) | 0x64006400u), __hadd2(k1024, z1));
  p.hi0 = __hfma2(h2((w & 0x00F000F0u) | 0x64006400u), k16, __hneg2(__hadd2(k64, z0)));
  p.hi1 = __hfma2(h2((x & 0x00F000F0u) | 0x64006400u), k16, __hneg2(__hadd2(k64, z1)));
  return p;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

template <int D, int G, bool EXACT>
__global__ void __launch_bounds__(KVP_THREADS, 1) kv4_attention_prompt(const __grid_constant__ Kv4AttnArgs a) {
  using Sm = KvpSmem<D, G>;
  constexpr int NJ = D / 32, NG = D / G, STRIP = Sm::STRIP;
  static_assert(!EXACT || NG == 1, "one step a token");
  extern __shared__ uint8_t smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.y, b = blockIdx.z;
  wait_for_kernel_before();
  const Kv4Seq seq = kv4_seq(a, b);
  const int rows = seq.n * a.share;
  auto bad_page = [&]() {
    atomicMax(a.err, ERR_KV4_PAGE);
    keep_device_error(ERR_KV4_PAGE);
  };
  if (threadIdx.x == 0 && seq.bad) bad_page();
  // the longest tiles first
  const int n_tiles = (rows + KVP_ROWS - 1) / KVP_ROWS, tile = n_tiles - 1 - (int)blockIdx.x;
  if (rows <= KVP_MIN_ROWS || tile < 0) return;
  const int r0 = tile * KVP_ROWS;
  // context tiles of the two row tiles (their last rows see the most)
  int n_ctx[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int last = min(r0 + 128 * (q + 1), rows) - 1;
    const int see = last >= r0 + 128 * q ? seq.L - seq.n + (int)((unsigned)last / (unsigned)a.share) + 1 : 0;
    n_ctx[q] = see > 0 ? (see + KVP_TOK - 1) / KVP_TOK : 0;
  }
  const int n = max(n_ctx[0], n_ctx[1]);  // (the second's, unless it is empty)

  if (threadIdx.x == 0) {
    for (int s = 0; s < KVP_RAW; ++s) {
      mbar_init(smem_u32(&sm.raw_full[s]), 1);
      mbar_init(smem_u32(&sm.raw_empty[s]), 4);
    }
    for (int s = 0; s < KVP_STAGES; ++s) {
      mbar_init(smem_u32(&sm.tile_full[s]), 4);
      mbar_init(smem_u32(&sm.tile_empty[s]), 2);
    }
    mbar_init(smem_u32(&sm.q_full[0]), 4);
    mbar_init(smem_u32(&sm.q_full[1]), 4);
    for (int q = 0; q < 2; ++q) {
      mbar_init(smem_u32(&sm.score[q][0]), 1);
      mbar_init(smem_u32(&sm.score[q][1]), 1);
      mbar_init(smem_u32(&sm.weight[q][0]), 4);
      mbar_init(smem_u32(&sm.weight[q][1]), 4);
      mbar_init(smem_u32(&sm.out_done[q][0]), 1);
      mbar_init(smem_u32(&sm.out_done[q][1]), 1);
    }
    mbar_init(smem_u32(&sm.drain[0]), 1);
    mbar_init(smem_u32(&sm.drain[1]), 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now may the next kernel start: the 8-bit product takes its tensor memory
  // before it waits for this kernel's end, and a block of it on this SM would
  // otherwise hold columns that this block still has to wait for.
  let_next_kernel_start();
  const uint32_t tmem = sm.tmem;
  volatile int* abort_flag = &sm.abort;
  auto score_col = [&](int q, int buf) { return tmem + (uint32_t)(128 * q + 64 * buf); };
  auto out_col = [&](int q) { return tmem + (uint32_t)(256 + 128 * q); };

  if (warp == 0) {
    // ---------------- packed strips
    Ring ring;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait_lean(smem_u32(&sm.raw_empty[ring.stage]), ring.phase ^ 1u, abort_flag, a.err,
                                                   ERR_KVP_RAW));
      if (!ok) break;
      const uint32_t bar = smem_u32(&sm.raw_full[ring.stage]);
      // lane i < 4: strip i of the tile (pages of 16 .. 64 tokens and more hold 1, 2 or 4 of them in a row)
      const int per = min(4, 1 << (a.c.page_shift - 4)), t0 = KVP_TOK * j + 16 * lane, p = t0 >> a.c.page_shift;
      const bool in = lane < 4 && t0 < seq.L;
      const int page = in && p < a.table_pages ? __ldg(a.table + (long long)b * a.table_pages + p) : -1;
      bool good = in && page >= 0 && page < a.c.n_pages;
      if (in && !good) bad_page();
      if (good && lane % per == 0) {
        // (a run's later strips lie in the same page: inside the cache too)
        const long long off = a.c.strip(page, head, t0 & ((1 << a.c.page_shift) - 1));
        good = AWQ_SPAN_OK(off, (long long)per * STRIP, a.c.bytes(), BS_KV4_STRIP);
        if (good) {
          mbar_expect_tx(bar, per * STRIP);
          bulk_load(smem_u32(sm.raw[ring.stage]) + lane * STRIP, a.c.base + off, per * STRIP, bar);
        }
      }
      const unsigned lost = __ballot_sync(0xffffffffu, in && !good);
      __syncwarp();
      if (lane == 0) {
        sm.lost_raw[ring.stage] = (int)lost;
        mbar_arrive(bar);
      }
      ring.next(KVP_RAW);
    }
    if (!ok) {  // copies in flight end before the block does
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
  } else if (warp == 1 || warp == 14) {
    if (lane == 0 && n > 0) {
      // ---------------- MMAs of row tile q
      const int q = warp == 1 ? 0 : 1;
      constexpr uint32_t F16_F32 = 1u << 4, M128 = (128u >> 4) << 24;
      constexpr uint32_t S_DESC = F16_F32 | ((KVP_TOK >> 3) << 17) | M128, O_DESC = F16_F32 | ((D >> 3) << 17) | M128;
      const uint64_t dq = desc_kmajor_sw128(smem_u32(sm.q[q][0]));
      auto scores = [&](int j, int st) {
        const uint64_t dk = desc_kmajor_sw128(smem_u32(sm.k[st][0]));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_bf16(score_col(q, j & 1), dq + (((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4),
                   dk + (((k >> 2) * KVP_TOK * 128 + (k & 3) * 32) >> 4), S_DESC, k != 0);
        mma_commit(smem_u32(&sm.score[q][j & 1]));
      };
      Ring now, next;  // the stages of tiles j and j + 1
      bool ok = mbar_wait_lean(smem_u32(&sm.q_full[q]), 0, abort_flag, a.err, ERR_KVP_TILE) &&
                mbar_wait_lean(smem_u32(&sm.tile_full[0]), 0, abort_flag, a.err, ERR_KVP_TILE);
      if (ok && n_ctx[q] > 0) {
        tc_fence_after();
        scores(0, 0);
      }
      next.next(KVP_STAGES);
      for (int j = 0; ok && j < n; ++j) {
        if (j + 1 < n_ctx[q]) {
          // the buffer of scores j + 1 held the weights of j - 1: their product is done
          ok = mbar_wait_lean(smem_u32(&sm.tile_full[next.stage]), next.phase, abort_flag, a.err, ERR_KVP_TILE) &&
               (j == 0 || mbar_wait_lean(smem_u32(&sm.out_done[q][(j - 1) & 1]), ((j - 1) >> 1) & 1, abort_flag, a.err,
                                         ERR_KVP_OUT));
          if (!ok) break;
          tc_fence_after();
          scores(j + 1, next.stage);
        }
        if (j < n_ctx[q]) {
          ok = mbar_wait_lean(smem_u32(&sm.weight[q][j & 1]), (j >> 1) & 1, abort_flag, a.err, ERR_KVP_WEIGHT);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = desc_kmajor_sw128(smem_u32(sm.v[now.stage]));
#pragma unroll
          for (int k = 0; k < KVP_TOK / 16; ++k)
            mma_f16_tmem_a(out_col(q), score_col(q, j & 1) + 8 * k, dv + ((k * 32) >> 4), O_DESC, j > 0 || k > 0);
          mma_commit(smem_u32(&sm.out_done[q][j & 1]));
        } else {
          // the other row tile's still: this one only hands the stage back once it is full
          ok = mbar_wait_lean(smem_u32(&sm.tile_full[now.stage]), now.phase, abort_flag, a.err, ERR_KVP_TILE);
          if (!ok) break;
        }
        mma_commit(smem_u32(&sm.tile_empty[now.stage]));
        now.next(KVP_STAGES);
        next.next(KVP_STAGES);
      }
      // what was issued ends before the block does
      mma_commit(smem_u32(&sm.drain[q]));
      mbar_wait_drain(smem_u32(&sm.drain[q]), 0);
      if (!ok) *abort_flag = 1;
    }
  } else if (warp < 6) {
    // ---------------- unpack: warp u takes strip u's values and steps, and keys of 16 tokens
    const int u = warp - 2, r = lane >> 2, q4 = lane & 3;
    Ring ring, raw;
    for (int j = 0; j < n; ++j) {
      bool ok = mbar_wait_lean(smem_u32(&sm.raw_full[raw.stage]), raw.phase, abort_flag, a.err, ERR_KVP_RAW) &&
                mbar_wait_lean(smem_u32(&sm.tile_empty[ring.stage]), ring.phase ^ 1u, abort_flag, a.err, ERR_KVP_FREE);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint8_t* s = sm.raw[raw.stage] + u * STRIP;
      const bool lost = sm.lost_raw[raw.stage] >> u & 1;
      const int t0 = KVP_TOK * j + 16 * u;
      const uint32_t* kpar = reinterpret_cast<const uint32_t*>(s + 16 * D);
      const uint32_t* vpar = kpar + 16 * NG;
      // the strip's largest steps and its tokens that hold NaN: lane l looks at token l % 16, of the keys or the values
      const int lt = lane & 15;
      float most = 0.0f;
      bool nan = false;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        const float x = __low2float(*reinterpret_cast<const __half2*>((lane < 16 ? kpar : vpar) + 16 * gi + lt));
        nan |= x != x;
        most = fmaxf(most, x);
      }
      const bool there = !lost && t0 + lt < seq.L;  // (else its bytes may hold anything)
      const bool sized = there && !nan;
      // (the quantiser's steps are 2^-24 or more; 0 is a token never written)
      int e = sized ? max((int)(__float_as_uint(most) >> 23) - 127, -24) : -24;
      // the largest e and the least (as 256 less it) over the half warp, two 16-bit numbers in a word
      uint32_t ends = (uint32_t)(e + 128) << 16 | (sized ? (uint32_t)(128 - e) : 0u);
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) ends = __vmaxu2(ends, __shfl_xor_sync(0xffffffffu, ends, d));
      const unsigned nans = __ballot_sync(0xffffffffu, there && nan);
      const uint32_t ends_v = __shfl_sync(0xffffffffu, ends, 16);
      const int ek = (int)(__shfl_sync(0xffffffffu, ends, 0) >> 16) - 128, ev = (int)(ends_v >> 16) - 128;
      const bool each = ev + (int)(ends_v & 0xffffu) > 128 + KVP_SPREAD;
      if (!each) e = ev;  // (lanes 16 .. have the values' tokens)
      if (EXACT && lane < 16) sm.step[ring.stage][16 * u + lane] = there ? most : 0.0f;
      if (lane >= 16) sm.e[ring.stage][16 * u + lt] = (float)e;
      if (lane == 0)
        sm.strip[ring.stage][u] = KvpStrip{EXACT ? 1.0f : __uint_as_float((uint32_t)(117 + ek) << 23), (float)ev,
                                           __uint_as_float((uint32_t)(127 - ev) << 23),
                                           ((nans | nans >> 16) & 0xffffu) | (each ? 0x10000u : 0u)};
      if (u == 0 && lane == 0) sm.lost[ring.stage] = sm.lost_raw[raw.stage];
      const float kup = __uint_as_float((uint32_t)(137 - ek) << 23);
      // (step times its strip's power of two, zero) of a token's group; nothing where its bytes may hold anything or NaN
      const unsigned dead = (nans | nans >> 16) | (lost ? 0xffffu : t0 + 16 > seq.L ? 0xffffu << max(seq.L - t0, 0) : 0u);
      auto param = [&](const uint32_t* par, int gi, int t, float up) -> float2 {
        const float2 p = widen2<true>(par[16 * gi + t]);
        return dead >> t & 1u ? make_float2(0.0f, 0.0f) : make_float2(p.x * up, p.y);
      };
      // keys: a lane takes the words of (token, q): chunk 4 j + q of the token's row holds channels 8 (4 j + q) + {0 4 2 6 1 5 3 7}
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int t = 8 * half + r, row = 16 * u + t;
        uint32_t w[NJ];
        load_words<NJ>(s + t * (D / 2) + 4 * q4 * NJ, w);
        __half2 kz[NG], km[NG];
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          const float2 p = param(kpar, gi, t, kup);
          km[gi] = __float2half2_rn(p.x);
          kz[gi] = __float2half2_rn(p.y);
        }
#pragma unroll
        for (int jj = 0; jj < NJ; ++jj) {
          KvpPairs c = kvp_unpack(w[jj], kz[jj * 32 / G], kz[jj * 32 / G]);
          if (!EXACT) c.scale(km[jj * 32 / G], km[jj * 32 / G]);
          const int chunk = 4 * jj + q4;
          *reinterpret_cast<uint4*>(sm.k[ring.stage][chunk >> 3] + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) =
              make_uint4(bits(c.lo0), bits(c.lo1), bits(c.hi0), bits(c.hi1));
        }
      }
      // values: rows are channels, 64 tokens of 2 bytes; a lane writes pairs of tokens
      const uint2* vw = reinterpret_cast<const uint2*>(s + 8 * D) + lane;
      const int ta = 2 * q4, tb = ta + 8;
      float vup[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) vup[i] = __uint_as_float((uint32_t)(137 - ev) << 23);
      if (each) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vup[i] = __uint_as_float((uint32_t)(137 - __shfl_sync(0xffffffffu, e, 16 + (i & 1) + (i < 2 ? ta : tb))) << 23);
      }
      uint2 w2[NJ];
      __half2 vz0[NG], vz1[NG], vm0[NG], vm1[NG];
#pragma unroll
      for (int p = 0; p < NJ; ++p) w2[p] = vw[32 * p];
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        const float2 a0 = param(vpar, gi, ta, vup[0]), a1 = param(vpar, gi, ta + 1, vup[1]), b0 = param(vpar, gi, tb, vup[2]),
                     b1 = param(vpar, gi, tb + 1, vup[3]);
        vm0[gi] = __floats2half2_rn(a0.x, a1.x);
        vz0[gi] = __floats2half2_rn(a0.y, a1.y);
        vm1[gi] = __floats2half2_rn(b0.x, b1.x);
        vz1[gi] = __floats2half2_rn(b0.y, b1.y);
      }
#pragma unroll
      for (int p = 0; p < NJ; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          KvpPairs c = kvp_unpack(h ? w2[p].y : w2[p].x, vz0[p * 32 / G], vz1[p * 32 / G]);
          c.scale(vm0[p * 32 / G], vm1[p * 32 / G]);
          const int ch = 32 * p + 8 * h + r;  // (its low three bits are r's)
          uint8_t* row = sm.v[ring.stage] + ch * 128 + 4 * q4;
          const int c0 = ((2 * u) ^ r) << 4, c1 = ((2 * u + 1) ^ r) << 4;
          *reinterpret_cast<uint32_t*>(row + c0) = bits(c.lo0);
          *reinterpret_cast<uint32_t*>(row + c1) = bits(c.lo1);
          *reinterpret_cast<uint32_t*>(row + 16 * 128 + c0) = bits(c.hi0);
          *reinterpret_cast<uint32_t*>(row + 16 * 128 + c1) = bits(c.hi1);
        }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&sm.tile_full[ring.stage]));
        mbar_arrive(smem_u32(&sm.raw_empty[raw.stage]));
      }
      ring.next(KVP_STAGES);
      raw.next(KVP_RAW);
    }
  } else {
    // ---------------- softmax: a thread a row
    const int q = (warp - 6) >> 2, quad = warp & 3, row = quad * 32 + lane, r = r0 + 128 * q + row;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const bool in = r < rows;
    // (a row behind the last, whose query is 0 and which is not written, sees all:
    // else its warp would take the long way at every tile)
    const int vis = in ? seq.L - seq.n + (int)((unsigned)r / (unsigned)a.share) + 1 : 0x7fffffff;
    {
      // The warp's 32 rows, a row by LANES lanes of 8 channels each: scaled by a
      // power of two so that the largest entry lies in [2^10, 2^11) (a row of
      // NaN or infinity: its operands become NaN or infinity too). A negative
      // scale turns the query round, so that the largest score is the largest
      // product's.
      constexpr int LANES = D > 64 ? 16 : 8, PER = 32 / LANES;
      const int chunk = lane % LANES;
      const bool used = chunk < D / 8;
      static_assert(32 / PER % 8 == 0, "rows in batches");
      constexpr int BATCH = 8;  // rows' loads under way at once
#pragma unroll 1
      for (int i0 = 0; i0 < 32 / PER; i0 += BATCH) {
        uint4 ahead[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int gr = r0 + 128 * q + quad * 32 + PER * (i0 + i) + lane / LANES;
          const bool have = gr < rows;
          const int t = have ? (int)((unsigned)gr / (unsigned)a.share) : 0, he = have ? gr - t * a.share : 0;
          const long long off = (seq.row0 + t) * a.q_tok + (long long)(head * a.share + he) * a.q_head;
          ahead[i] = make_uint4(0, 0, 0, 0);
          if (have && used && AWQ_IDX_OK(seq.row0 + t, a.T, BS_KV4_Q))
            ahead[i] = __ldg(reinterpret_cast<const uint4*>(a.q + off) + chunk);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int lr = quad * 32 + PER * (i0 + i) + lane / LANES;
          const uint4 w = ahead[i];
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          float2 f[4];
          float top = 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[k] = a.f16 ? widen2<true>(ww[k]) : widen2<false>(ww[k]);
            top = fmaxf(top, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
          }
#pragma unroll
          for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          const int ex = top > 0.0f ? min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -110), 127) : 0;
          const float up = copysignf(__uint_as_float((uint32_t)(137 - ex) << 23), a.scale_log2);
          // channels {0 4 2 6 1 5 3 7} of the eight, as the keys' codes come out of their words
          if (used)
            *reinterpret_cast<uint4*>(sm.q[q][chunk >> 3] + lr * 128 + (((chunk & 7) ^ (lr & 7)) << 4)) =
                make_uint4(pack2<true>(f[0].x * up, f[2].x * up), pack2<true>(f[1].x * up, f[3].x * up),
                           pack2<true>(f[0].y * up, f[2].y * up), pack2<true>(f[1].y * up, f[3].y * up));
          // 2^(ex - 10) |scale|: score (log2) per unit of q . k; never 0, which would make hidden scores NaN
          if (chunk == 0) sm.unit[q][lr] = fmaxf(__uint_as_float((uint32_t)(117 + ex) << 23) * fabsf(a.scale_log2), 1e-37f);
        }
      }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[q]));
    const float unit = sm.unit[q][row];
    float m = KV4_LOWEST, l = 0.0f;
    bool ok = true;
    const int n_mine = n_ctx[q];
    // Wait for the weights' product of tile j. (Scores j or j + 1 being there
    // means that the one of the same barrier before, j - 2, is done.)
    auto product_done = [&](int j) {
      return mbar_wait_lean(smem_u32(&sm.out_done[q][j & 1]), (j >> 1) & 1, abort_flag, a.err, ERR_KVP_OUT);
    };
    Ring ring;
    for (int j = 0; j < n_mine; ++j, ring.next(KVP_STAGES)) {
      const int st = j & 1, t0 = KVP_TOK * j;
      ok = mbar_wait_lean(smem_u32(&sm.score[q][st]), (j >> 1) & 1, abort_flag, a.err, ERR_KVP_SCORE) &&
           mbar_wait_lean(smem_u32(&sm.tile_full[ring.stage]), ring.phase, abort_flag, a.err, ERR_KVP_TILE);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const KvpStrip* strip = sm.strip[ring.stage];
      const float4* step = reinterpret_cast<const float4*>(sm.step[ring.stage]);
      const unsigned lost = (unsigned)sm.lost[ring.stage];
      const uint32_t col = score_col(q, st) + lanes;
      // Half a tile at a time (short code: the warps of an SM sub-partition run
      // four different loops, which together must stay in its instruction
      // cache); its 16 columns of weights go over scores read already.
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        const KvpStrip f[2] = {strip[2 * c], strip[2 * c + 1]};
        const unsigned off = lost >> (2 * c) & 3u;
        const bool odd = __any_sync(0xffffffffu, t0 + 32 * c + 32 > vis) || off || f[0].odd || f[1].odd;
        uint32_t s[32], wbits[16];
        tmem_ld_32x32b_x32(col + 32 * c, s);
        tmem_ld_wait();
        float sum = 0.0f;
        bool done = false;
        if (!odd) {
          // The usual case: weights under the reference as it stands, if all of them turn out to fit fp16.
          __half2 big = __float2half2_rn(0.0f);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 u2 = make_float2(unit * f[h].key, unit * f[h].key), m2 = make_float2(f[h].e - m, f[h].e - m);
            float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float2 y = make_float2(__uint_as_float(s[16 * h + k]), __uint_as_float(s[16 * h + k + 1]));
              if (EXACT) {
                const float4 d = step[8 * c + 4 * h + (k >> 2)];
                y = mul2(y, k & 2 ? make_float2(d.z, d.w) : make_float2(d.x, d.y));
              }
              y = fma2(y, u2, m2);
              const float2 w = make_float2(exp2_fast(y.x), exp2_fast(y.y));
              part = add2(part, w);
              wbits[8 * h + (k >> 1)] = pack2<true>(w.x, w.y);
              big = __hmax2(big, *reinterpret_cast<const __half2*>(&wbits[8 * h + (k >> 1)]));
            }
            sum = fmaf(part.x + part.y, f[h].down, sum);
          }
          const float2 top2 = __half22float2(big);
          done = !__any_sync(0xffffffffu, fmaxf(top2.x, top2.y) > 65504.0f);
        }
        if (!done) {
          // The first tokens, some that a row does not see, NaN, steps of very
          // different sizes, and scores that outgrow the reference: the row's
          // largest exponent first.
          auto score = [&](int k) {
            return __uint_as_float(s[k]) * (EXACT ? sm.step[ring.stage][32 * c + k] : 1.0f);
          };
          const float* e = sm.e[ring.stage] + 32 * c;
          auto hidden = [&](int k) { return t0 + 32 * c + k >= vis || (off >> (k >> 4) & 1u); };
          float want = -INFINITY;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!hidden(k)) want = fmaxf(want, fmaf(score(k), unit * f[k >> 4].key, e[k]));
          float scale = 1.0f;
          if (want > m + KVP_LAG) {
            const float to = ceilf(want) - KVP_HEAD, by = to - m;  // (2^-by exactly; 0 from 127 on)
            scale = __uint_as_float((uint32_t)(127 - (int)fminf(by, 127.0f)) << 23);
            m = to;
            l *= scale;
          }
          if (__any_sync(0xffffffffu, scale != 1.0f)) {
            // bring along the output, which the product of the tile before is in, and this tile's weights so far
            if (j > 0) {
              ok = __all_sync(0xffffffffu, product_done(j - 1));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < D / 16; ++i) {
                uint32_t v[16];
                __syncwarp();
                tmem_ld_32x32b_x16(out_col(q) + lanes + 16 * i, v);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * scale);
                tmem_st_32x32b_x16(out_col(q) + lanes + 16 * i, v);
              }
            }
            if (c > 0) {
              uint32_t v[16];
              tmem_st_wait();  // the first half's weights are there to be read
              __syncwarp();
              tmem_ld_32x32b_x16(col, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 w = widen2<true>(v[k]);
                v[k] = pack2<true>(w.x * scale, w.y * scale);
              }
              tmem_st_32x32b_x16(col, v);
            }
            tmem_st_wait();
          }
          sum = 0.0f;
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const KvpStrip& g = f[k >> 4];
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float et = e[k + i];
              w[i] = g.odd >> ((k + i) & 15) & 1u ? __int_as_float(0x7fffffff) : exp2_fast(fmaf(score(k + i), unit * g.key, et - m));
              if (hidden(k + i)) w[i] = 0.0f;
              sum = fmaf(w[i], __uint_as_float((uint32_t)(127 - (int)et) << 23), sum);
            }
            wbits[k >> 1] = pack2<true>(w[0], w[1]);
          }
          __syncwarp();
        }
        l += sum;
        tmem_st_32x32b_x16(col + 16 * c, wbits);
      }
      if (!ok) break;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.weight[q][st]));  // (a warp may be a tile ahead of its neighbours)
    }
    // ---------------- output
    if (ok && n_mine > 0) {
      ok = product_done(n_mine - 1);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    const long long at = in ? kv4_out_row(a, seq, head, r) : -1;
    const float inv = l == 0.0f ? 0.0f : __fdividef(0.0009765625f, l);  // (the values' 2^10)
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        uint32_t v[16];
        __syncwarp();
        if (n_mine > 0) {
          tmem_ld_32x32b_x16(out_col(q) + lanes + 16 * c, v);
          tmem_ld_wait();
        }
        if (at >= 0) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + 16 * c);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a row that sees nothing gives zeros, whatever stands in tensor memory
              const float x = l == 0.0f ? 0.0f : __uint_as_float(v[8 * k + 2 * i]) * inv;
              const float y = l == 0.0f ? 0.0f : __uint_as_float(v[8 * k + 2 * i + 1]) * inv;
              o[i] = a.f16 ? pack2<true>(x, y) : pack2<false>(x, y);
            }
            dst[k] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        __syncwarp();
      }
      if (at >= 0 && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace awq
