// The key/value cache held in 4 bits on sm_100a: write, read back, attention.
//
// Quantiser of a group of g channels of one (token, kv head), the asymmetric
// group quantiser of the weights with a range that always holds 0:
//   lo = min(0, min v), hi = max(0, max v), step = fp16((hi - lo) / 15) in [2^-24, 65504],
//   inv = 1 / step, zero = rne(-lo inv), code = clamp(rne(v inv) + zero, 0, 15);
//   the cache holds (code - zero) * step.
// A group that holds NaN or infinity gets step NaN and reads back as NaN.
//
// Layout: each (page, kv head) is one run of bytes, page_size / 16 strips of
// 16 tokens, a strip being
//   keys    [16 tokens][4 q][D/32 j][4 b]      channel 8 (4 j + q) + 2 b + n in nibble n of the byte
//   values  [D/32 p][8 r][4 q][2 h][4 b]       token 2 q + (b >> 1) + 8 (b & 1), channel 32 p + 16 n + 8 h + r in nibble n
//   key parameters, value parameters           [D/g groups][16 tokens] of (fp16 step, fp16 zero)
// which is the order in which a warp's lanes (r = lane / 4, q = lane % 4) feed
// mma.m16n8k16: with the 16 tokens (keys) or 16 channels (values) as rows of
// the A operand, a lane's words hold its own A registers. Masking a word with
// 0x000F000F (or 0x00F000F0) leaves two codes in the low mantissa bits of two
// fp16 numbers: the subnormals c 2^-24 (or c 2^-20), exactly, which the tensor
// cores multiply exactly. So a code costs half an instruction, and steps and
// zeros enter outside the product:
//   q . k_t = dk_t (sum_i q_i c_ti - zk_t sum_i q_i),
//   O_d     = sum_t w_t c_td - sum_t w_t zv_t,  w_t = p_t dv_t.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "check.cuh"
#include "ptx.cuh"
#include "w4a16_sm100.cuh"
#include "w8a8_sm100.cuh"

namespace awq {

constexpr int KV4_STRIP = 16;  // tokens of a strip
__host__ __device__ constexpr int kv4_strip_bytes(int dim, int group) { return KV4_STRIP * dim + 128 * (dim / group); }

struct Kv4Cache {
  uint8_t* base;
  long long n_pages;
  int heads, dim, group, page_shift;  // page_size = 1 << page_shift
  int strip_bytes;
  long long head_bytes;  // page_size / 16 strips
  __host__ __device__ long long bytes() const { return n_pages * heads * head_bytes; }
  // byte offset of the strip that holds token `in_page` of (page, head)
  __device__ __forceinline__ long long strip(long long page, int head, int in_page) const {
    return (page * heads + head) * head_bytes + (long long)(in_page >> 4) * strip_bytes;
  }
};

// Byte of a strip's value section that holds channels 32 p + 8 h + r (nibble 0) and 16 more (nibble 1) of token t.
__device__ __forceinline__ int kv4_value_byte(int p, int h, int r, int t) {
  return ((p * 32 + r * 4 + ((t & 7) >> 1)) << 3) + 4 * h + 2 * (t & 1) + (t >> 3);
}

struct Kv4AppendArgs {
  const uint16_t *k, *v;
  long long k_tok, k_head, v_tok, v_head;  // strides in elements
  const int* slots;
  int T;
  Kv4Cache c;
};

// A thread takes 8 consecutive channels of one (token, head) of the keys or
// the values; the g / 8 lanes of a group share its extremes by shuffles.
template <bool F16>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4AppendArgs a) {
  const int chunks = a.c.dim / 8;
  const long long units = (long long)a.T * a.c.heads * chunks;
  const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const bool live = u < 2 * units;
  const bool val = u >= units;
  const long long w = live ? (val ? u - units : u) : 0;
  const int ch = (int)(w % chunks);
  const long long th = w / chunks;
  const int head = (int)(th % a.c.heads), tok = (int)(th / a.c.heads);
  const int slot = live ? __ldg(a.slots + tok) : -1;
  const bool put = slot >= 0 && (slot >> a.c.page_shift) < a.c.n_pages;
  float x[8];
  const uint16_t* src = (val ? a.v + tok * a.v_tok + head * a.v_head : a.k + tok * a.k_tok + head * a.k_head) + 8 * ch;
  const uint4 raw = put ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
  const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
  float lo = 0.0f, hi = 0.0f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = widen2<F16>(rw[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad |= !(fabsf(x[i]) <= 3.402823466e38f);
  }
  if (bad) hi = __int_as_float(0x7f800000);
  for (int o = a.c.group / 16; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const bool finite = hi <= 3.402823466e38f;
  __half step = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
  const float sf = fminf(fmaxf(__half2float(step), 5.9604644775390625e-8f), 65504.0f);
  const float inv = __frcp_rn(sf);
  const float zf = fminf(rintf(__fmul_rn(-lo, inv)), 15.0f);
  uint32_t word = 0;
  if (finite) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(__fadd_rn(rintf(__fmul_rn(x[i], inv)), zf), 0.0f), 15.0f);
      word |= (uint32_t)c << (4 * i);
    }
  }
  const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 2);  // the 8 channels 16 away
  if (!put) return;
  const int t = slot & 15;
  const long long base = a.c.strip(slot >> a.c.page_shift, head, slot & ((1 << a.c.page_shift) - 1));
  if (!AWQ_SPAN_OK(base, a.c.strip_bytes, a.c.bytes(), BS_KV4_CACHE)) return;
  uint8_t* s = a.c.base + base;
  if (!val) {
    *reinterpret_cast<uint32_t*>(s + t * (a.c.dim / 2) + ((ch & 3) * (a.c.dim / 32) + (ch >> 2)) * 4) = word;
  } else {
    // lanes n = 0 and 1 hold channels 32 p + 8 h + r and 16 more: each writes four of the eight bytes
    const int p = ch >> 2, n = (ch >> 1) & 1, h = ch & 1;
    const uint32_t low = n ? other : word, high = n ? word : other;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * n + i;
      const uint32_t byte = ((low >> (4 * r)) & 15u) | (((high >> (4 * r)) & 15u) << 4);
      s[8 * a.c.dim + kv4_value_byte(p, h, r, t)] = (uint8_t)byte;
    }
  }
  if (ch % (a.c.group / 8) == 0) {
    const int gi = ch / (a.c.group / 8), ng = a.c.dim / a.c.group;
    const uint32_t par = finite ? (uint32_t)__half_as_ushort(__float2half_rn(sf)) |
                                      (uint32_t)__half_as_ushort(__float2half_rn(zf)) << 16
                                : 0x00007FFFu;
    *reinterpret_cast<uint32_t*>(s + 16 * a.c.dim + (val ? 64 * ng : 0) + gi * 64 + 4 * t) = par;
  }
}

// (code - zero) * step of one token of the cache, dense: a thread takes 8
// consecutive channels; slots outside the cache give zeros.
template <bool F16>
__global__ void __launch_bounds__(256)
    kv4_gather_kernel(const Kv4Cache c, const int* __restrict__ slots, int T, void* __restrict__ kv, void* __restrict__ vv) {
  const int chunks = c.dim / 8;
  const long long units = (long long)T * c.heads * chunks;
  for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < 2 * units;
       u += (long long)gridDim.x * blockDim.x) {
    const bool val = u >= units;
    const long long w = val ? u - units : u;
    const int ch = (int)(w % chunks);
    const long long th = w / chunks;
    const int head = (int)(th % c.heads), tok = (int)(th / c.heads);
    const int slot = __ldg(slots + tok);
    uint4 out = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && (slot >> c.page_shift) < c.n_pages) {
      const int t = slot & 15;
      const long long base = c.strip(slot >> c.page_shift, head, slot & ((1 << c.page_shift) - 1));
      if (AWQ_SPAN_OK(base, c.strip_bytes, c.bytes(), BS_KV4_CACHE)) {
        const uint8_t* s = c.base + base;
        const int gi = ch / (c.group / 8), ng = c.dim / c.group;
        const uint32_t par = *reinterpret_cast<const uint32_t*>(s + 16 * c.dim + (val ? 64 * ng : 0) + gi * 64 + 4 * t);
        const float step = __half2float(__ushort_as_half((unsigned short)(par & 0xFFFF)));
        const float zero = __half2float(__ushort_as_half((unsigned short)(par >> 16)));
        uint32_t codes = 0;
        if (!val) {
          codes = *reinterpret_cast<const uint32_t*>(s + t * (c.dim / 2) + ((ch & 3) * (c.dim / 32) + (ch >> 2)) * 4);
        } else {
          const int p = ch >> 2, n = (ch >> 1) & 1, h = ch & 1;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            codes |= ((uint32_t)(s[8 * c.dim + kv4_value_byte(p, h, r, t)] >> (4 * n)) & 15u) << (4 * r);
        }
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = (float)((codes >> (8 * i)) & 15u), y = (float)((codes >> (8 * i + 4)) & 15u);
          o[i] = pack2<F16>(__fmul_rn(x - zero, step), __fmul_rn(y - zero, step));
        }
        out = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    void* dst = val ? vv : kv;
    if (dst && AWQ_SPAN_OK(8 * w, 8, 8 * units, BS_KV4_OUT)) reinterpret_cast<uint4*>(dst)[w] = out;
  }
}

// ------------------------------------------------------------------ attention
struct Kv4AttnArgs {
  const uint16_t* q;
  long long q_tok, q_head;  // strides in elements
  long long T;              // rows of q
  int q_heads, share;       // query heads, query heads of a kv head
  const int* q_start;       // [batch + 1], or NULL: sequence b is row row_first + b
  int row_first;
  int max_q;
  const int* table;  // [batch, table_pages]
  int table_pages;
  const int* lens;  // [batch]
  int batch;
  float scale_log2;  // softmax scale * log2(e)
  bool f16;          // q and out are fp16 (else bf16)
  Kv4Cache c;
  void* out;   // [T, q_heads, D] contiguous
  float* lse;  // [T, q_heads] or NULL
  int* err;
};

constexpr int ERR_KV4_PAGE = 0x401, ERR_KV4_COPY = 0x402;

// One sequence's rows and context, clamped to what the arguments can hold:
// rows [row0, row0 + n), context length L. bad: something was clamped.
struct Kv4Seq {
  long long row0;
  int n, L;
  bool bad;
};
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4AttnArgs& a, int b) {
  Kv4Seq s;
  long long r0 = a.q_start ? a.q_start[b] : a.row_first + b, r1 = a.q_start ? a.q_start[b + 1] : r0 + 1;
  const long long cap = (long long)a.table_pages << a.c.page_shift;
  const int len = a.lens[b];
  s.bad = r0 < 0 || r1 < r0 || r1 > a.T || r1 - r0 > a.max_q || len < 0 || len > cap;
  r0 = r0 < 0 ? 0 : r0 > a.T ? a.T : r0;
  r1 = r1 < r0 ? r0 : r1 > a.T ? a.T : r1;
  s.row0 = r0;
  s.n = (int)(r1 - r0 < a.max_q ? r1 - r0 : a.max_q);
  s.L = len < 0 ? 0 : (int)(len < cap ? len : cap);
  return s;
}

// x rounded to the output type
__device__ __forceinline__ uint16_t kv4_narrow(const Kv4AttnArgs& a, float x) {
  return a.f16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held two a lane (lane / 4 = row).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) { return exp2f(x); }

// N consecutive words at p, aligned to the largest power of two that divides 4 N (at most 16).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 v = reinterpret_cast<const uint2*>(p)[i];
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// What a warp knows of a tile of 8 NT query rows of one (sequence, kv head).
// Column j of n-tile u is row 8 u + j of the tile; a lane works on columns
// 2 q and 2 q + 1 of each n-tile.
template <int D, int G, int NT>
struct Kv4Warp {
  static constexpr int NJ = D / 32, NG = D / G, JG = G / 32;
  uint32_t qf[NT][NJ][4];      // B operands: queries, even channels then odd ones (times 2^-4)
  float qsum[NT][NG][2];       // 2^-24 sum of the scaled query over a group, columns 2 q, 2 q + 1
  float qscale[NT][2];         // score (log2) per accumulator unit
  int vis[NT][2];              // keys [0, vis) are visible to the column's query
  int vis_min, vis_max;        // over the tile's rows
  float o[NT][NJ][2][4];       // accumulators: channels 32 p + 16 n + ..., value 2^-24 (n = 0) or 2^-20 units
  float mid[NT][NG][4];        // -8 2^-24 sum of w since the last recentre(), in every row
  float zs[NT][NG][2];         // sum of w (zero - 8) over this lane's tokens
  float m[NT][2], l[NT][2];    // reference exponent (the same in all lanes of a column), sum of p over this lane's tokens

  // Rows [r0, r0 + 8 NT) of the sequence's n * share query rows (row = token * share + head in the group).
  __device__ __forceinline__ void load_queries(const Kv4AttnArgs& a, const Kv4Seq& s, int head, long long r0, int lane) {
    const int g = lane >> 2, q = lane & 3;
    const long long rows = (long long)s.n * a.share;
    vis_min = 0x7fffffff;
    vis_max = 0;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      // this lane loads column g: 8 channels of each 32
      const long long r = r0 + 8 * u + g;
      const bool in = r < rows;
      const int tok = in ? (int)(r / a.share) : 0, e = in ? (int)(r - (long long)tok * a.share) : 0;
      const long long off = (s.row0 + tok) * a.q_tok + (long long)(head * a.share + e) * a.q_head;
      const uint16_t* src = a.q + off;
      float x[NJ][8];
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (in && AWQ_IDX_OK(s.row0 + tok, a.T, BS_KV4_Q)) w = __ldg(reinterpret_cast<const uint4*>(src + 8 * (4 * j + q)));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = a.f16 ? widen2<true>(ww[i]) : widen2<false>(ww[i]);
          x[j][2 * i] = f.x;
          x[j][2 * i + 1] = f.y;
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // Scale the row by a power of two so that its largest entry lies in
      // [2^10, 2^11): fp16 then holds every entry down to 2^-21 of it to 11
      // bits, also the odd channels' 2^-4. Exact back through the scale.
      const int ex = top > 0.0f ? min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -110), 127) : 0;
      const float f1 = __uint_as_float((uint32_t)(127 + (10 - ex) / 2) << 23);
      const float f2 = __uint_as_float((uint32_t)(127 + (10 - ex) - (10 - ex) / 2) << 23);
      float part[NG];
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) part[gi] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        __half h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[i] = __float2half_rn(x[j][i] * f1 * f2 * ((i & 1) ? 0.0625f : 1.0f));
          part[j / JG] += __half2float(h[i]) * ((i & 1) ? 16.0f : 1.0f);
        }
        auto two = [&](int lo, int hi) {
          return (uint32_t)__half_as_ushort(h[lo]) | (uint32_t)__half_as_ushort(h[hi]) << 16;
        };
        qf[u][j][0] = two(0, 4);
        qf[u][j][1] = two(2, 6);
        qf[u][j][2] = two(1, 5);
        qf[u][j][3] = two(3, 7);
      }
      const float unit = exp2f((float)(ex - 10 + 24)) * a.scale_log2;
      const int see = in ? s.L - s.n + tok + 1 : 0;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        part[gi] += __shfl_xor_sync(0xffffffffu, part[gi], 1);
        part[gi] += __shfl_xor_sync(0xffffffffu, part[gi], 2);
      }
      // columns 2 q and 2 q + 1 of this n-tile were loaded by lanes 8 q and 8 q + 4
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int from = 8 * q + 4 * c;
        qscale[u][c] = __shfl_sync(0xffffffffu, unit, from);
        vis[u][c] = __shfl_sync(0xffffffffu, see, from);
#pragma unroll
        for (int gi = 0; gi < NG; ++gi)
          qsum[u][gi][c] = __shfl_sync(0xffffffffu, part[gi], from) * 5.9604644775390625e-8f;
        m[u][c] = -INFINITY;
        l[u][c] = 0.0f;
      }
      if (in) {
        vis_min = min(vis_min, see);
        vis_max = max(vis_max, see);
      }
    }
#pragma unroll
    for (int o_ = 4; o_ < 32; o_ <<= 1) {
      vis_min = min(vis_min, __shfl_xor_sync(0xffffffffu, vis_min, o_));
      vis_max = max(vis_max, __shfl_xor_sync(0xffffffffu, vis_max, o_));
    }
    clear();
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int p = 0; p < NJ; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[u][p][n][i] = 0.0f;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        zs[u][gi][0] = zs[u][gi][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) mid[u][gi][i] = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[u][c] = -INFINITY;
        l[u][c] = 0.0f;
      }
    }
  }

  // One strip: tokens t0 .. t0 + 15 of the context, its bytes at `s`. EDGE:
  // some of the tile's queries do not see all of its tokens, whose bytes may
  // hold anything then.
  template <bool EDGE>
  __device__ __forceinline__ void strip(const uint8_t* s, int t0, int lane) {
    const int g = lane >> 2, q = lane & 3;
    uint32_t kw0[NJ], kw1[NJ];
    load_words<NJ>(s + g * (D / 2) + 4 * q * NJ, kw0);
    load_words<NJ>(s + (g + 8) * (D / 2) + 4 * q * NJ, kw1);
    const uint32_t* kpar = reinterpret_cast<const uint32_t*>(s + 16 * D);
    const uint32_t* vpar = kpar + 16 * NG;
    // scores: token rows g and g + 8, columns 2 q and 2 q + 1
    float sc[NT][4];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
      float acc[NT][4];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] = 0.0f;
#pragma unroll
      for (int jj = 0; jj < JG; ++jj) {
        const int j = gi * JG + jj;
        const uint32_t w0 = kw0[j], w1 = kw1[j], v0 = w0 >> 8, v1 = w1 >> 8;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          mma_16816(acc[u], w0 & 0x000F000Fu, w1 & 0x000F000Fu, v0 & 0x000F000Fu, v1 & 0x000F000Fu, qf[u][j][0], qf[u][j][1]);
          mma_16816(acc[u], w0 & 0x00F000F0u, w1 & 0x00F000F0u, v0 & 0x00F000F0u, v1 & 0x00F000F0u, qf[u][j][2], qf[u][j][3]);
        }
      }
      const float2 p0 = widen2<true>(kpar[16 * gi + g]), p1 = widen2<true>(kpar[16 * gi + 8 + g]);
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = i < 2 ? p0 : p1;
          const float x = p.x * fmaf(-p.y, qsum[u][gi][i & 1], acc[u][i]);
          sc[u][i] = gi == 0 ? x : sc[u][i] + x;
        }
    }
    // the exponent of the value step joins the running reference, so that
    // w = p step stays below 2^9 whatever the steps are
    float2 vp[NG][2];
    int e0 = -1000, e1 = -1000;
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
      vp[gi][0] = widen2<true>(vpar[16 * gi + g]);
      vp[gi][1] = widen2<true>(vpar[16 * gi + 8 + g]);
      e0 = max(e0, (int)(__float_as_uint(vp[gi][0].x) >> 23) - 127);
      e1 = max(e1, (int)(__float_as_uint(vp[gi][1].x) >> 23) - 127);
    }
    const float ve[2] = {(float)e0, (float)e1};
    bool grow = false;
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[u][i] *= qscale[u][i & 1];
        if (EDGE && t0 + g + 8 * (i >> 1) >= vis[u][i & 1]) sc[u][i] = -INFINITY;
        grow |= sc[u][i] + ve[i >> 1] > m[u][i & 1] + 8.0f;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(sc[u][c] + ve[0], sc[u][c + 2] + ve[1]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float mn = fmaxf(m[u][c], top);
          const float f = m[u][c] == -INFINITY ? 0.0f : exp2_fast(m[u][c] - mn);
          m[u][c] = mn;
          l[u][c] *= f;
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) {
            zs[u][gi][c] *= f;
            mid[u][gi][c] *= f;
            mid[u][gi][c + 2] *= f;
          }
#pragma unroll
          for (int p = 0; p < NJ; ++p)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              o[u][p][n][c] *= f;
              o[u][p][n][c + 2] *= f;
            }
        }
    }
    uint32_t wb[NT][NG][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ref = m[u][i & 1];
        p[i] = exp2_fast(sc[u][i] - (ref == -INFINITY ? 0.0f : ref));
      }
      l[u][0] += p[0] + p[2];
      l[u][1] += p[1] + p[3];
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = p[i] * vp[gi][i >> 1].x;
          if (EDGE && t0 + g + 8 * (i >> 1) >= vis[u][i & 1]) w[i] = 0.0f;
        }
        const uint32_t r0 = pack2<true>(w[0], w[1]), r1 = pack2<true>(w[2], w[3]);
        const float2 b0 = widen2<true>(r0), b1 = widen2<true>(r1);  // the rounded weights, which the codes meet too
        const float z0 = vp[gi][0].y - 8.0f, z1 = vp[gi][1].y - 8.0f;
        float z[4] = {b0.x * z0, b0.y * z0, b1.x * z1, b1.y * z1};
        if (EDGE) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + g + 8 * (i >> 1) >= vis[u][i & 1]) z[i] = 0.0f;
        }
        zs[u][gi][0] += z[0] + z[2];
        zs[u][gi][1] += z[1] + z[3];
        wb[u][gi][0] = transpose_8x8(r0);
        wb[u][gi][1] = transpose_8x8(r1);
        mma_16816(mid[u][gi], 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, wb[u][gi][0], wb[u][gi][1]);
      }
    }
    const uint2* vw = reinterpret_cast<const uint2*>(s + 8 * D) + lane;
#pragma unroll
    for (int p = 0; p < NJ; ++p) {
      const uint2 w = vw[32 * p];
      const uint32_t x = w.x >> 8, y = w.y >> 8;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const uint32_t b0 = wb[u][p / JG][0], b1 = wb[u][p / JG][1];
        mma_16816(o[u][p][0], w.x & 0x000F000Fu, w.y & 0x000F000Fu, x & 0x000F000Fu, y & 0x000F000Fu, b0, b1);
        mma_16816(o[u][p][1], w.x & 0x00F000F0u, w.y & 0x00F000F0u, x & 0x00F000F0u, y & 0x00F000F0u, b0, b1);
      }
    }
  }

  // Take 8 sum(w) off the accumulated codes (16 times that where codes count
  // 16-fold): they then hold sum w (c - 8), which wanders about zero, while
  // sum w c would grow with the context and the fp32 accumulators would drop
  // bits of it at every step. Measured at 131072 tokens: relative error of the
  // output against 64 bits 4.6e-3 without it, 1.7e-3 (bf16's own rounding) with it.
  __device__ __forceinline__ void recentre() {
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int p = 0; p < NJ; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[u][p][0][i] += mid[u][p / JG][i];
          o[u][p][1][i] = fmaf(16.0f, mid[u][p / JG][i], o[u][p][1][i]);
        }
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int gi = 0; gi < NG; ++gi)
#pragma unroll
        for (int i = 0; i < 4; ++i) mid[u][gi][i] = 0.0f;
  }

  // Sums over the lanes of a column.
  __device__ __forceinline__ void finish() {
    recentre();
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[u][c] += __shfl_xor_sync(0xffffffffu, l[u][c], d);
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) zs[u][gi][c] += __shfl_xor_sync(0xffffffffu, zs[u][gi][c], d);
        }
      }
  }

  // The finished state of column 2 q + c of n-tile u: channel 32 p + 16 n + 8 h + g, unnormalised.
  __device__ __forceinline__ float value(int u, int c, int p, int n, int h) const {
    return fmaf(o[u][p][n][2 * h + c], n ? 1048576.0f : 16777216.0f, -zs[u][p / JG][c]);
  }

  // This warp's finished state into part (layout [8 NT][D + 4]: unnormalised output, m, l).
  __device__ __forceinline__ void store(float* part, int lane) const {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* row = part + (8 * u + 2 * q + c) * (D + 4);
#pragma unroll
        for (int p = 0; p < NJ; ++p)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              row[32 * p + 16 * n + 8 * h + g] = value(u, c, p, n, h);
        if (g == 0) {
          row[D] = m[u][c];
          row[D + 1] = l[u][c];
        }
      }
  }
};

constexpr int KV4_RECENTRE = 8;  // strips between recentre()s
constexpr int KV4_WARPS = 4;

// One block per (tile of 8 query rows, kv head, sequence); the warps take the
// strips in turn and their states are joined at the end.
template <int D, int G>
__global__ void __launch_bounds__(32 * KV4_WARPS) kv4_attention_tiles(const Kv4AttnArgs a) {
  using W = Kv4Warp<D, G, 1>;
  __shared__ float part[KV4_WARPS][8 * (D + 4)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.y, b = blockIdx.z;
  const Kv4Seq s = kv4_seq(a, b);
  bool bad = s.bad;
  const long long r0 = 8ll * blockIdx.x, rows = (long long)s.n * a.share;
  if (bad && threadIdx.x == 0) atomicCAS(a.err, 0, ERR_KV4_PAGE);
  if (r0 >= rows) return;
  W w;
  w.load_queries(a, s, head, r0, lane);
  const int n_strips = (w.vis_max + 15) >> 4;
  int done = 0;
  for (int i = warp; i < n_strips; i += KV4_WARPS) {
    const int t0 = 16 * i;
    const int page = __ldg(a.table + (long long)b * a.table_pages + (t0 >> a.c.page_shift));
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) atomicCAS(a.err, 0, ERR_KV4_PAGE);
      continue;
    }
    const long long off = a.c.strip(page, head, t0 & ((1 << a.c.page_shift) - 1));
    if (!AWQ_SPAN_OK(off, a.c.strip_bytes, a.c.bytes(), BS_KV4_STRIP)) continue;
    if (t0 + 16 > w.vis_min)
      w.template strip<true>(a.c.base + off, t0, lane);
    else
      w.template strip<false>(a.c.base + off, t0, lane);
    if (++done % KV4_RECENTRE == 0) w.recentre();
  }
  w.finish();
  w.store(part[warp], lane);
  __syncthreads();
  for (int e = threadIdx.x; e < 8 * D; e += blockDim.x) {
    const int j = e / D, d = e - j * D;
    const long long r = r0 + j;
    if (r >= rows) break;
    float m = -INFINITY;
    for (int k = 0; k < KV4_WARPS; ++k) m = fmaxf(m, part[k][j * (D + 4) + D]);
    float o = 0.0f, l = 0.0f;
    for (int k = 0; k < KV4_WARPS; ++k) {
      const float* row = part[k] + j * (D + 4);
      if (row[D] == -INFINITY && row[D + 1] == 0.0f) continue;
      const float f = exp2_fast(row[D] - m);
      o += f * row[d];
      l += f * row[D + 1];
    }
    const long long tok = s.row0 + r / a.share;
    const int qh = head * a.share + (int)(r % a.share);
    if (!AWQ_IDX_OK(tok, a.T, BS_KV4_O)) break;
    static_cast<uint16_t*>(a.out)[(tok * a.q_heads + qh) * D + d] = kv4_narrow(a, l == 0.0f ? 0.0f : o / l);
    if (a.lse && d == 0) a.lse[tok * a.q_heads + qh] = l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
  }
}


// ------------------------------------------------------------------ attention, split evenly over the GPU
// Work is counted in units of one strip of one tile (8 NT query rows of one
// sequence and kv head), ordered by sequence, head, tile, strip. Every warp of
// the grid takes one contiguous range of equal length, whatever the contexts'
// lengths, and streams its strips through a ring of its own in shared memory
// (one cp.async.bulk a strip, issued KV4_STAGES ahead, across tiles too); no
// warp waits for another until its range is done. A tile that lies in one
// warp's range is written out by it; the at most two that it shares (its first
// and its last) go to the workspace as (unnormalised output, m, l), are joined
// within the block, and where they cross blocks by kv4_attention_join. All
// joins run in the order of the ranges, so the result is the same every time.
constexpr int KV4_MAX_BATCH = 1024;  // sequences of a launch: their unit counts sit in shared memory
constexpr int KV4_CTAS = 148;        // blocks of the grid, one per SM
constexpr int KV4_STAGES = 4;
// Warps of a block: as many as their state lets have enough registers.
constexpr int kv4_warps(int dim, int group, int nt) {
  return dim * nt > 128 ? 8 : dim / group * nt <= (dim * nt <= 64 ? 2 : 1) ? 16 : 12;
}

struct Kv4SplitArgs {
  Kv4AttnArgs a;
  int tile_rows;    // 8 NT
  float* warp_part; // [warps of the grid][2][8 NT][D + 4]
  float* cta_part;  // [KV4_CTAS][2][8 NT][D + 4]
  long long* cta_seg;  // [KV4_CTAS][2] tile of a block partial (-1: none)
  int* cta_bad;     // [KV4_CTAS]
  int clear_err;    // the first launch of a call sets the error word, later ones add to it
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

// Units of the batch: prefix[b] = units before sequence b, strips and tiles of each.
struct Kv4Plan {
  long long prefix[KV4_MAX_BATCH + 1];
  int strips[KV4_MAX_BATCH], tiles[KV4_MAX_BATCH];
  int bad;
};

// Filled by the whole block (a multiple of 32 threads, at least 32).
__device__ __forceinline__ void kv4_plan(const Kv4SplitArgs& s, Kv4Plan& p, long long* warp_sums) {
  const Kv4AttnArgs& a = s.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (threadIdx.x == 0) {
    p.prefix[0] = 0;
    p.bad = 0;
  }
  __syncthreads();
  long long before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    long long n = 0;
    if (b < a.batch) {
      const Kv4Seq q = kv4_seq(a, b);
      if (q.bad) p.bad = 1;
      const long long rows = (long long)q.n * a.share;
      // a sequence without context still has its rows to write: one unit, which reads nothing
      const int strips = q.n > 0 ? max(1, (int)(((long long)q.L + 15) >> 4)) : 0;
      const int tiles = (int)((rows + s.tile_rows - 1) / s.tile_rows);
      p.strips[b] = strips;
      p.tiles[b] = tiles;
      n = (long long)strips * tiles * a.c.heads;
    }
    long long inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += t;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += warp_sums[w];
    if (b < a.batch) p.prefix[b + 1] = before + inc;
    for (int w = 0; w < warps; ++w) before += warp_sums[w];
    __syncthreads();
  }
}

// Workers that take part: at least KV4_MIN_STRIPS units each.
constexpr int KV4_MIN_STRIPS = 4;
__device__ __forceinline__ long long kv4_workers(long long units, long long most) {
  const long long w = (units + KV4_MIN_STRIPS - 1) / KV4_MIN_STRIPS;
  return w < most ? (w > 0 ? w : 1) : most;
}
__device__ __forceinline__ long long kv4_begin(long long w, long long workers, long long units) {
  return w < workers ? w * units / workers : units;
}

// A place in the order of units.
struct Kv4Cursor {
  int b, strip, strips, tile, tiles, head;
  __device__ __forceinline__ void seek(const Kv4Plan& p, int batch, long long u) {
    int lo = 0, hi = batch;  // prefix[lo] <= u < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.prefix[mid] <= u) lo = mid;
      else hi = mid;
    }
    b = lo;
    strips = p.strips[b];
    tiles = p.tiles[b];
    const long long in = u - p.prefix[b], seg = in / strips;
    strip = (int)(in - seg * strips);
    head = (int)(seg / tiles);
    tile = (int)(seg - (long long)head * tiles);
  }
  // to the next unit; true if it begins another tile
  __device__ __forceinline__ bool step(const Kv4Plan& p, const Kv4AttnArgs& a) {
    if (++strip < strips) return false;
    strip = 0;
    if (++tile == tiles) {
      tile = 0;
      if (++head == a.c.heads) {
        head = 0;
        do ++b;
        while (b < a.batch && p.strips[b] == 0);
        if (b < a.batch) {
          strips = p.strips[b];
          tiles = p.tiles[b];
        }
      }
    }
    return true;
  }
  __device__ __forceinline__ long long id(const Kv4AttnArgs& a) const {
    return ((long long)b * a.c.heads + head) << 32 | (unsigned)tile;
  }
};

// Query row r (in the sequence's n * share) of a kv head: its element offset in out, and in lse; -1 if there is none.
__device__ __forceinline__ long long kv4_out_row(const Kv4AttnArgs& a, const Kv4Seq& s, int head, long long r) {
  if (r >= (long long)s.n * a.share) return -1;
  const long long tok = s.row0 + r / a.share;
  if (!AWQ_IDX_OK(tok, a.T, BS_KV4_O)) return -1;
  return tok * a.q_heads + head * a.share + (int)(r % a.share);
}

// Joins entries part(e), e in [e0, e1), of row `row` of a tile by one warp:
// lane's channels 4 lane + 128 k. Returns m and l; v holds the unnormalised sums.
template <int D>
struct Kv4Joined {
  static constexpr int K = (D + 127) / 128;
  float4 v[K];
  float m, l;
  template <typename Part>
  __device__ __forceinline__ void join(Part part, int e0, int e1, int row, int lane) {
    m = -INFINITY;
    for (int e = e0; e < e1; ++e) m = fmaxf(m, part(e)[row * (D + 4) + D]);
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int e = e0; e < e1; ++e) {
      const float* r = part(e) + row * (D + 4);
      const float me = r[D], le = r[D + 1];
      // a part that saw nothing holds m = -inf and zeros; NaN in l passes on
      const float f = me == -INFINITY ? (le == 0.0f ? 0.0f : le) : exp2_fast(me - m);
      l = fmaf(f, le, l);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = 4 * lane + 128 * k;
        if (c < D) {
          const float4 x = *reinterpret_cast<const float4*>(r + c);
          v[k].x = fmaf(f, x.x, v[k].x);
          v[k].y = fmaf(f, x.y, v[k].y);
          v[k].z = fmaf(f, x.z, v[k].z);
          v[k].w = fmaf(f, x.w, v[k].w);
        }
      }
    }
  }
  __device__ __forceinline__ void store(float* r, int lane) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (4 * lane + 128 * k < D) *reinterpret_cast<float4*>(r + 4 * lane + 128 * k) = v[k];
    if (lane == 0) {
      r[D] = m;
      r[D + 1] = l;
    }
  }
  __device__ __forceinline__ void write(const Kv4AttnArgs& a, long long at, int lane) const {
    if (at < 0) return;
    const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = 4 * lane + 128 * k;
      if (c < D)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + c) =
            a.f16 ? make_uint2(pack2<true>(v[k].x * inv, v[k].y * inv), pack2<true>(v[k].z * inv, v[k].w * inv))
                  : make_uint2(pack2<false>(v[k].x * inv, v[k].y * inv), pack2<false>(v[k].z * inv, v[k].w * inv));
    }
    if (a.lse && lane == 0) a.lse[at] = l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
  }
};

template <int D, int G, int NT>
struct Kv4SplitSmem {
  static constexpr int W = kv4_warps(D, G, NT);
  static constexpr int STRIP = kv4_strip_bytes(D, G);
  alignas(128) uint8_t ring[W][KV4_STAGES][STRIP];
  alignas(8) uint64_t bar[W][KV4_STAGES];
  Kv4Plan plan;
  long long sums[W];
  long long seg[W][2];   // tile of a warp's first and last part (-1: none)
  int flags[W][2];       // bit 0: the part begins its tile, bit 1: it ends it
  int chain[2 * W + 1], chains, bad;
  int abort;
};

template <int D, int G, int NT>
__global__ void __launch_bounds__(32 * kv4_warps(D, G, NT), 1) kv4_attention_split(const __grid_constant__ Kv4SplitArgs s) {
  using Sm = Kv4SplitSmem<D, G, NT>;
  using St = Kv4Warp<D, G, NT>;
  constexpr int W = Sm::W, PART = 8 * NT * (D + 4);
  extern __shared__ uint8_t smem_raw[];
  // (offset, not address, arithmetic keeps the accesses shared-memory ones)
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u));
  const Kv4AttnArgs& a = s.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < KV4_STAGES; ++i) mbar_init(smem_u32(&sm.bar[warp][i]), 1);
    fence_barrier_init();
    sm.seg[warp][0] = sm.seg[warp][1] = -1;
  }
  if (threadIdx.x == 0) {
    sm.bad = 0;
    sm.abort = 0;
  }
  kv4_plan(s, sm.plan, sm.sums);
  const long long units = sm.plan.prefix[a.batch];
  const long long workers = kv4_workers(units, (long long)gridDim.x * W);
  const long long me = (long long)blockIdx.x * W + warp;
  const long long u0 = kv4_begin(me, workers, units), u1 = kv4_begin(me + 1, workers, units);
  float* my_part = s.warp_part + me * 2 * PART;
  if (u0 < u1) {
    Kv4Cursor cur, ahead;
    cur.seek(sm.plan, a.batch, u0);
    ahead = cur;
    const int page_mask = (1 << a.c.page_shift) - 1;
    int left = (int)(u1 - u0), to_load = left;
    unsigned have = 0;  // stages whose strip is there to be read
    int win_b = -1, win_p = 0, win = 0;  // lane i: page win_p + i of sequence win_b
    int ahead_len = a.lens[ahead.b];
    auto issue = [&](int stage) {
      const int t0 = 16 * ahead.strip, p = t0 >> a.c.page_shift;
      if (ahead.b != win_b || p < win_p || p >= win_p + 32) {
        win_b = ahead.b;
        win_p = p;
        win = p + lane < a.table_pages ? __ldg(a.table + (long long)ahead.b * a.table_pages + p + lane) : -1;
        ahead_len = a.lens[ahead.b];
      }
      const int page = __shfl_sync(0xffffffffu, win, p - win_p);
      const bool in = t0 < ahead_len, good = in && page >= 0 && page < a.c.n_pages;
      bool copied = false;
      if (good) {
        const long long off = a.c.strip(page, ahead.head, t0 & page_mask);
        if (AWQ_SPAN_OK(off, Sm::STRIP, a.c.bytes(), BS_KV4_STRIP)) {
          copied = true;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&sm.bar[warp][stage]);
            mbar_arrive_expect_tx(bar, Sm::STRIP);
            bulk_load(smem_u32(sm.ring[warp][stage]), a.c.base + off, Sm::STRIP, bar);
          }
        }
      } else if (in && lane == 0) {
        sm.bad = ERR_KV4_PAGE;
      }
      have = copied ? have | (1u << stage) : have & ~(1u << stage);
      --to_load;
      if (to_load > 0) ahead.step(sm.plan, a);
    };
    for (int i = 0; i < KV4_STAGES && to_load > 0; ++i) issue(i);
    St w;
    int stage = 0;
    unsigned phases = 0;
    bool ok = true, begins = cur.strip == 0, first = true;
    Kv4Seq seq = kv4_seq(a, cur.b);
    w.load_queries(a, seq, cur.head, (long long)cur.tile * s.tile_rows, lane);
    int done = 0;
    while (ok) {
      const int t0 = 16 * cur.strip;
      if (have >> stage & 1u) {
        ok = mbar_wait(smem_u32(&sm.bar[warp][stage]), phases >> stage & 1u, &sm.abort, nullptr, 0);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        phases ^= 1u << stage;
        have &= ~(1u << stage);
        if (t0 < w.vis_max) {
          if (t0 + 16 > w.vis_min)
            w.template strip<true>(sm.ring[warp][stage], t0, lane);
          else
            w.template strip<false>(sm.ring[warp][stage], t0, lane);
          if (++done % KV4_RECENTRE == 0) w.recentre();
        }
      }
      __syncwarp();
      if (to_load > 0) issue(stage);
      if (++stage == KV4_STAGES) stage = 0;
      --left;
      const bool ends = cur.strip + 1 == cur.strips;
      if (ends || left == 0) {
        w.finish();
        if (begins && ends) {
          // the whole tile: write it
          const int g = lane >> 2, q = lane & 3;
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const long long at = kv4_out_row(a, seq, cur.head, (long long)cur.tile * s.tile_rows + 8 * u + 2 * q + c);
              if (at < 0) continue;
              const float inv = w.l[u][c] == 0.0f ? 0.0f : __fdividef(1.0f, w.l[u][c]);
              uint16_t* o = static_cast<uint16_t*>(a.out) + at * D + g;
#pragma unroll
              for (int p = 0; p < D / 32; ++p)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                  for (int h = 0; h < 2; ++h) o[32 * p + 16 * n + 8 * h] = kv4_narrow(a, w.value(u, c, p, n, h) * inv);
              if (a.lse && g == 0)
                a.lse[at] = w.l[u][c] == 0.0f ? -INFINITY : 0.69314718055994531f * (w.m[u][c] + log2f(w.l[u][c]));
            }
          __syncwarp();
        } else {
          const int k = first ? 0 : 1;
          w.store(my_part + k * PART, lane);
          if (lane == 0) {
            sm.seg[warp][k] = cur.id(a);
            sm.flags[warp][k] = (begins ? 1 : 0) | (ends ? 2 : 0);
          }
        }
        first = false;
        if (left == 0) break;
      }
      if (cur.step(sm.plan, a)) {
        const int b = cur.b;
        begins = true;
        seq = kv4_seq(a, b);
        w.load_queries(a, seq, cur.head, (long long)cur.tile * s.tile_rows, lane);
        done = 0;
      }
    }
    if (!ok) {
      // a copy that never came: wait (bounded) for the others, report, write nothing
      if (lane == 0) {
        sm.bad = ERR_KV4_COPY;
        for (int i = 0; i < KV4_STAGES; ++i)
          if (have >> i & 1u) mbar_wait_drain(smem_u32(&sm.bar[warp][i]), phases >> i & 1u);
      }
      __syncwarp();
    }
  }
  __threadfence_block();
  __syncthreads();
  // ---------------- join the warps' parts: chains of consecutive parts of one tile
  if (threadIdx.x == 0) {
    int n = 0;
    long long last = -1;
    for (int e = 0; e < 2 * W; ++e) {
      const long long g = sm.seg[e >> 1][e & 1];
      if (g < 0) continue;
      if (g != last) sm.chain[n++] = e;
      last = g;
    }
    sm.chain[n] = 2 * W;
    sm.chains = n;
    s.cta_bad[blockIdx.x] = sm.bad ? sm.bad : sm.plan.bad ? ERR_KV4_PAGE : 0;
    s.cta_seg[2 * blockIdx.x] = s.cta_seg[2 * blockIdx.x + 1] = -1;
  }
  __syncthreads();
  const float* base = s.warp_part + (long long)blockIdx.x * W * 2 * PART;
  for (int it = warp; it < sm.chains * 8 * NT; it += W) {
    const int ch = it / (8 * NT), row = it - ch * 8 * NT;
    const int e0 = sm.chain[ch];
    int entries = 0;
    const long long seg = sm.seg[e0 >> 1][e0 & 1];
    // a chain's parts: the first one, then the slot 0 of the following warps (a warp's slot 1 begins another tile)
    int flags = 0;
    for (int e = e0; e < sm.chain[ch + 1]; ++e)
      if (sm.seg[e >> 1][e & 1] >= 0) {
        flags |= sm.flags[e >> 1][e & 1];
        ++entries;
      }
    Kv4Joined<D> j;
    auto part = [&](int i) {
      // the i-th part of the chain: e0, then warp (e0 / 2 + i), slot 0
      const int e = i == 0 ? e0 : 2 * ((e0 >> 1) + i);
      return base + (long long)e * PART;
    };
    j.join(part, 0, entries, row, lane);
    if (flags == 3) {
      const int head_b = (int)(seg >> 32), b = head_b / a.c.heads, head = head_b - b * a.c.heads;
      const Kv4Seq seq = kv4_seq(a, b);
      j.write(a, kv4_out_row(a, seq, head, (long long)(int)(seg & 0xffffffff) * s.tile_rows + row), lane);
    } else {
      // shared with other blocks: slot 1 if it begins here, else 0
      const int k = flags & 1;
      j.store(s.cta_part + ((long long)blockIdx.x * 2 + k) * PART + row * (D + 4), lane);
      if (row == 0 && lane == 0) s.cta_seg[2 * blockIdx.x + k] = seg;
    }
  }
}

// Block c joins the tile that block c of the split began and did not end:
// its slot 1, then slot 0 of the following blocks while they hold that tile.
// Block 0 sets the call's error word.
template <int D, int NT>
__global__ void __launch_bounds__(256) kv4_attention_join(const __grid_constant__ Kv4SplitArgs s, int ctas) {
  constexpr int PART = 8 * NT * (D + 4);
  const Kv4AttnArgs& a = s.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  if (c == 0 && threadIdx.x < 32) {
    int bad = 0;
    for (int i = lane; i < ctas; i += 32) bad = max(bad, s.cta_bad[i]);
    bad = __reduce_max_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (s.clear_err) *a.err = bad;
      else if (bad) *a.err = bad;
    }
  }
  const long long seg = s.cta_seg[2 * c + 1];
  if (seg < 0) return;
  int n = 1;
  while (c + n < ctas && s.cta_seg[2 * (c + n)] == seg) ++n;
  const int head_b = (int)(seg >> 32), b = head_b / a.c.heads, head = head_b - b * a.c.heads;
  const Kv4Seq seq = kv4_seq(a, b);
  for (int row = warp; row < 8 * NT; row += 8) {
    const long long at = kv4_out_row(a, seq, head, (long long)(int)(seg & 0xffffffff) * s.tile_rows + row);
    if (at < 0) continue;
    Kv4Joined<D> j;
    j.join([&](int i) { return s.cta_part + ((long long)(c + i) * 2 + (i == 0)) * PART; }, 0, n, row, lane);
    j.write(a, at, lane);
  }
}

}  // namespace awq
