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

// Tokens that fill a strip in order (slots 16 i .. 16 i + 15 one behind the
// other), as those of a prompt do, are taken together by one warp a head, the
// others alone: a strip's values lie four tokens to a word, and one token alone
// touches every one of its sectors.
//
// A block has the tokens [first, first + span), span <= 16, and the strips that
// begin there. All lanes of a warp call this: lane l < span gets its token's slot,
// and the masks have the tokens that begin a whole strip (one at most) and those
// that are written alone. Bit i of a warp's view is token first - 16 + i; a bit of
// `breaks` is set where a token does not follow the one before.
struct Kv4Tokens {
  int slot;
  uint32_t strips, alone;
};
__device__ __forceinline__ Kv4Tokens kv4_tokens(const int* __restrict__ slots, int T, int first, int span, int lane) {
  const int i0 = first - 16 + lane, i1 = first + 16 + lane;
  const int a = i0 >= 0 && i0 < T ? __ldg(slots + i0) : 0, b = lane < 16 && i1 < T ? __ldg(slots + i1) : 0;
  const int a_up = __shfl_up_sync(0xffffffffu, a, 1), b_up = __shfl_up_sync(0xffffffffu, b, 1);
  const int last = __shfl_sync(0xffffffffu, a, 31);
  const uint64_t breaks = (uint64_t)__ballot_sync(0xffffffffu, i0 < 1 || i0 >= T || lane == 0 || (unsigned)a - (unsigned)a_up != 1u) |
                          (uint64_t)__ballot_sync(0xffffffffu, i1 >= T || (unsigned)b - (unsigned)(lane ? b_up : last) != 1u) << 32;
  const int at = lane - (a & 15);  // where this token's strip would begin: 1 or more for lanes 16 ..
  const bool mine = lane >= 16 && lane < 16 + span && i0 < T;
  const bool whole = mine && ((breaks >> (at + 1)) & 0x7FFFu) == 0;
  Kv4Tokens r;
  r.slot = __shfl_sync(0xffffffffu, a, (lane & 15) + 16);
  r.strips = __ballot_sync(0xffffffffu, whole && (a & 15) == 0) >> 16;
  r.alone = __ballot_sync(0xffffffffu, mine && !whole) >> 16;
  return r;
}
// Few tokens take a block each; more of them share blocks by strips.
constexpr int KV4_APPEND_WARPS = 8;
inline int kv4_span(long long T) { return T <= 1024 ? 1 : 16; }

// a[j]'s nibble r to a[r]'s nibble j: halves, bytes, nibbles
__device__ __forceinline__ void kv4_transpose(uint32_t (&a)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = a[j], y = a[j + 4];
    a[j] = __byte_perm(x, y, 0x5410);
    a[j + 4] = __byte_perm(x, y, 0x7632);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = (k & 1) + 4 * (k >> 1);
    const uint32_t x = a[j], y = a[j + 2];
    a[j] = __byte_perm(x, y, 0x6240);
    a[j + 2] = __byte_perm(x, y, 0x7351);
  }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint32_t x = a[j], y = a[j + 1];
    a[j] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
    a[j + 1] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
  }
}
// The chunk (8 channels of a token) that is row j of the transposition of lane
// item (p, q, h): token and chunk. Its word r is then that of lane (r, q).
__device__ __forceinline__ int kv4_row_token(int j, int q) { return 2 * q + ((j >> 2) & 1) + 8 * ((j >> 1) & 1); }
__device__ __forceinline__ int kv4_row_chunk(int j, int p, int h) { return 4 * p + 2 * (j & 1) + h; }

struct Kv4AppendArgs {
  const uint16_t *k, *v;
  long long k_tok, k_head, v_tok, v_head;  // strides in elements
  const int* slots;
  int T;
  Kv4Cache c;
};

// 8 NC channels of a token: their codes as words (channel i of 8 in nibble i) and
// the group's step and zero as stored. A group's lanes (neighbours; all lanes of
// a warp call this) share its extremes by shuffles: (-min, max) as a
// pair of the inputs' own type, whose order and sign are exact.
template <bool F16>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (F16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool F16, int NC>
__device__ __forceinline__ void kv4_quantize(const uint4 (&raw)[NC], int group, uint32_t (&word)[NC], uint32_t& par) {
  uint32_t low = 0, high = 0;  // 0 is always in the range
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const uint32_t rw[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      low = max2_nan<F16>(low, rw[i] ^ 0x80008000u);
      high = max2_nan<F16>(high, rw[i]);
    }
  }
  uint32_t both = max2_nan<F16>(__byte_perm(low, high, 0x5410), __byte_perm(low, high, 0x7632));
  for (int o = group / (16 * NC); o; o >>= 1) both = max2_nan<F16>(both, __shfl_xor_sync(0xffffffffu, both, o));
  const float2 ends = widen2<F16>(both);  // (-min, max); infinite or NaN if one of the inputs is
  if (!(fabsf(ends.x) <= 3.402823466e38f && fabsf(ends.y) <= 3.402823466e38f)) {  // step NaN, codes and zero 0
    par = 0x00007E00u;
#pragma unroll
    for (int k = 0; k < NC; ++k) word[k] = 0;
    return;
  }
  const __half step = __float2half_rn(__fdiv_rn(__fadd_rn(ends.y, ends.x), 15.0f));
  const float sf = fminf(fmaxf(__half2float(step), 5.9604644775390625e-8f), 65504.0f);
  const float inv = __frcp_rn(sf);
  // rint by a sum with 1.5 * 2^23, which has it in its low bits too. clamp(rint(v)
  // + z, 0, 15) = rint(clamp(v, -z, 15 - z)) + z, as z is whole; and eight such
  // sums, each four bits further up, add to the word and a known constant.
  const float zero = __fadd_rn(fminf(__fmul_rn(ends.x, inv), 15.0f), 12582912.0f);
  const float zf = __fsub_rn(zero, 12582912.0f), most = 15.0f - zf;
  par = (uint32_t)__half_as_ushort(__float2half_rn(sf)) | (uint32_t)__half_as_ushort(__float2half_rn(zf)) << 16;
  const uint32_t start = (__float_as_uint(zero) - 2u * 0x4B400000u) * 0x11111111u;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const uint32_t rw[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    uint32_t w = start;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = widen2<F16>(rw[i]);
      const float v0 = fminf(fmaxf(__fmul_rn(f.x, inv), -zf), most), v1 = fminf(fmaxf(__fmul_rn(f.y, inv), -zf), most);
      w += __float_as_uint(__fadd_rn(v0, 12582912.0f)) << (8 * i);
      w += __float_as_uint(__fadd_rn(v1, 12582912.0f)) << (8 * i + 4);
    }
    word[k] = w;
  }
}

// 16411 tokens of 8 heads of 128 in groups of 32, fp16: 30 us for 67 MB read and
// 21 written (13.5 at a copy's rate); 64 single tokens 2.5 us, a launch. A token at
// a time took 74 us: bytes of the value words written one by one, a rint, a
// conversion and two divisions' worth of slow instructions for every 8 channels
// (16 now), a block a token. Issue slots and the loads of eight warps a block, each
// one pass behind the other, share the rest about equally.
template <bool F16>
__global__ void __launch_bounds__(32 * KV4_APPEND_WARPS) kv4_append_kernel(const Kv4AppendArgs a, const int span) {
  let_next_kernel_start();
  wait_for_kernel_before();
  __shared__ uint32_t codes[KV4_APPEND_WARPS][16][33];  // a strip's value codes, a word a chunk; padded rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, begin = blockIdx.x * span;
  const Kv4Tokens own = kv4_tokens(a.slots, a.T, begin, span, lane);
  const int D = a.c.dim, chunks = D / 8, ng = D / a.c.group, per = a.c.group / 8, per_bits = __ffs(per) - 1, in_mask = (1 << a.c.page_shift) - 1;

  for (uint32_t m = own.alone; m; m &= m - 1) {
    const int i = __ffs(m) - 1, tok = begin + i, slot = __shfl_sync(0xffffffffu, own.slot, i);
    const long long page = slot >> a.c.page_shift;
    if (slot < 0 || page >= a.c.n_pages) continue;
    // units of 8 channels: keys of all heads, then values (whole warps run, for the shuffles)
    const int t = slot & 15, half = a.c.heads * chunks;
    for (int u0 = 0; u0 < 2 * half; u0 += blockDim.x) {
      const int u = u0 + threadIdx.x;
      const bool live = u < 2 * half, val = u >= half;
      const int w = live ? (val ? u - half : u) : 0, head = w / chunks, ch = w - head * chunks;
      const uint16_t* src = (val ? a.v + (long long)tok * a.v_tok + (long long)head * a.v_head
                                 : a.k + (long long)tok * a.k_tok + (long long)head * a.k_head) + 8 * ch;
      const uint4 raw[1] = {live ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0)};
      uint32_t words[1], par;
      kv4_quantize<F16>(raw, a.c.group, words, par);
      const uint32_t word = words[0];
      const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 2);  // the 8 channels 16 away
      const long long base = a.c.strip(page, head, slot & in_mask);
      if (!live || !AWQ_SPAN_OK(base, a.c.strip_bytes, a.c.bytes(), BS_KV4_CACHE)) continue;
      uint8_t* s = a.c.base + base;
      if (!val) {
        *reinterpret_cast<uint32_t*>(s + t * (D / 2) + ((ch & 3) * (D / 32) + (ch >> 2)) * 4) = word;
      } else {
        // lanes n = 0 and 1 hold channels 32 p + 8 h + r and 16 more: each writes four of the eight bytes
        const int p = ch >> 2, n = (ch >> 1) & 1, h = ch & 1;
        const uint32_t low = n ? other : word, high = n ? word : other;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 4 * n + k;
          s[8 * D + kv4_value_byte(p, h, r, t)] = (uint8_t)(((low >> (4 * r)) & 15u) | (((high >> (4 * r)) & 15u) << 4));
        }
      }
      if ((ch & (per - 1)) == 0) *reinterpret_cast<uint32_t*>(s + 16 * D + (val ? 64 * ng : 0) + (ch >> per_bits) * 64 + 4 * t) = par;
    }
  }

  if (!own.strips) return;
  const int i = __ffs(own.strips) - 1, tok = begin + i, slot = __shfl_sync(0xffffffffu, own.slot, i);
  const long long page = slot >> a.c.page_shift;
  if (slot < 0 || page >= a.c.n_pages) return;
  uint32_t(&cw)[16][33] = codes[warp];
  // Items: a head, 128 channels of it at most, its keys and then its values; with few
  // heads keys and values apart, for more warps. (3 x 4439 tokens of two heads of 256
  // and their read-back take 30 us so, 50 with a whole head an item; 9000 tokens of 4
  // heads of 128 21.3, 21.8 with keys and values apart.) The warp's lanes go over
  // (token, two chunks), tokens outermost: chunks of a group stay neighbours.
  const int apart = a.c.heads < 4, slices = D > 128 ? 2 : 1, width = D / slices, pairs = width / 16;
  const int t0 = lane / pairs, pair0 = lane - t0 * pairs, dt = 32 / pairs, dp = 32 - dt * pairs;
  for (int it = warp; it < slices * a.c.heads << apart; it += KV4_APPEND_WARPS) {
    const int slice = slices == 2 ? it & 1 : 0, hv = slices == 2 ? it >> 1 : it, head = apart ? hv >> 1 : hv;
#pragma unroll 1
    for (int val = apart ? hv & 1 : 0, end = apart ? val + 1 : 2; val < end; ++val) {
      const long long base = a.c.strip(page, head, slot & in_mask);
      if (!AWQ_SPAN_OK(base, a.c.strip_bytes, a.c.bytes(), BS_KV4_CACHE)) continue;
      uint8_t* s = a.c.base + base;
      const uint16_t* src = (val ? a.v + (long long)tok * a.v_tok + (long long)head * a.v_head
                                 : a.k + (long long)tok * a.k_tok + (long long)head * a.k_head) + slice * width;
      const long long ld = val ? a.v_tok : a.k_tok;
      uint8_t* pars = s + 16 * D + (val ? 64 * ng : 0);
      int t = t0, pair = pair0;
#pragma unroll 1
      for (int u0 = 0; u0 < 16 * pairs; u0 += 32) {  // width / 32 turns
        const uint4* from = reinterpret_cast<const uint4*>(src + t * ld + 16 * pair);
        const uint4 raw[2] = {__ldg(from), __ldg(from + 1)};
        const int ch = slice * (width / 8) + 2 * pair;
        uint32_t word[2], par;
        kv4_quantize<F16>(raw, a.c.group, word, par);
        if (val) {
          cw[t][2 * pair] = word[0];
          cw[t][2 * pair + 1] = word[1];
        } else {
          uint8_t* to = s + t * (D / 2) + ((ch & 3) * (D / 32) + (ch >> 2)) * 4;
          *reinterpret_cast<uint32_t*>(to) = word[0];
          *reinterpret_cast<uint32_t*>(to + D / 8) = word[1];
        }
        if ((ch & (per - 1)) == 0) *reinterpret_cast<uint32_t*>(pars + (ch >> per_bits) * 64 + 4 * t) = par;
        t += dt;
        pair += dp;
        if (pair >= pairs) pair -= pairs, ++t;
      }
      if (!val) continue;
      __syncwarp();
      if (lane < width / 4) {  // items (p, q, h) of the transposition
        const int h = lane & 1, q = (lane >> 1) & 3, p = lane >> 3;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = cw[kv4_row_token(j, q)][kv4_row_chunk(j, p, h)];
        kv4_transpose(w);
        uint8_t* to = s + 8 * D + ((slice * (width / 32) + p) * 32 + q) * 8 + 4 * h;
#pragma unroll
        for (int r = 0; r < 8; ++r) *reinterpret_cast<uint32_t*>(to + 32 * r) = w[r];
      }
      __syncwarp();
    }
  }
}

// (code - zero) * step of tokens of the cache, dense; slots outside it give
// zeros. Blocks, strips and warps as in the write. The same 16411 tokens: 26 us
// (45 a token at a time; 13.5 at a copy's rate), waiting for the strips' words.
template <bool F16>
__device__ __forceinline__ uint4 kv4_values(uint32_t word, uint32_t par) {
  const float2 f = widen2<true>(par);  // (step, zero)
  const float off = 8388608.0f + f.y;  // zero <= 15: exact, as is the difference
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack2<F16>(__fmul_rn(__fsub_rn(__uint_as_float(((word >> (8 * i)) & 15u) | 0x4B000000u), off), f.x),
                      __fmul_rn(__fsub_rn(__uint_as_float(((word >> (8 * i + 4)) & 15u) | 0x4B000000u), off), f.x));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool F16>
__global__ void __launch_bounds__(32 * KV4_APPEND_WARPS)
    kv4_gather_kernel(const Kv4Cache c, const int* __restrict__ slots, int T, void* __restrict__ kv, void* __restrict__ vv,
                      const int span) {
  __shared__ uint32_t codes[KV4_APPEND_WARPS][16][33];
  let_next_kernel_start();
  wait_for_kernel_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, begin = blockIdx.x * span;
  const Kv4Tokens own = kv4_tokens(slots, T, begin, span, lane);
  const int D = c.dim, chunks = D / 8, ng = D / c.group, per_bits = __ffs(c.group / 8) - 1, in_mask = (1 << c.page_shift) - 1;
  const long long all = (long long)T * c.heads * D;
  bool in = true;
  if (own.strips) {  // a strip outside the cache: its tokens are zeros
    const int slot = __shfl_sync(0xffffffffu, own.slot, __ffs(own.strips) - 1);
    in = slot >= 0 && (slot >> c.page_shift) < c.n_pages;
  }

  for (uint32_t m = own.alone; m; m &= m - 1) {
    const int i = __ffs(m) - 1, tok = begin + i, slot = __shfl_sync(0xffffffffu, own.slot, i);
    const long long page = slot >> c.page_shift;
    const bool here = slot >= 0 && page < c.n_pages;
    const int t = slot & 15, half = c.heads * chunks;
    for (int u = threadIdx.x; u < 2 * half; u += blockDim.x) {
      const bool val = u >= half;
      const int w = val ? u - half : u, head = w / chunks, ch = w - head * chunks;
      uint4 out = make_uint4(0, 0, 0, 0);
      const long long base = here ? c.strip(page, head, slot & in_mask) : 0;
      if (here && AWQ_SPAN_OK(base, c.strip_bytes, c.bytes(), BS_KV4_CACHE)) {
        const uint8_t* s = c.base + base;
        uint32_t word = 0;
        if (!val) {
          word = *reinterpret_cast<const uint32_t*>(s + t * (D / 2) + ((ch & 3) * (D / 32) + (ch >> 2)) * 4);
        } else {
          const int p = ch >> 2, n = (ch >> 1) & 1, h = ch & 1;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            word |= ((uint32_t)(s[8 * D + kv4_value_byte(p, h, r, t)] >> (4 * n)) & 15u) << (4 * r);
        }
        out = kv4_values<F16>(word, *reinterpret_cast<const uint32_t*>(s + 16 * D + (val ? 64 * ng : 0) + (ch >> per_bits) * 64 + 4 * t));
      }
      uint16_t* dst = static_cast<uint16_t*>(val ? vv : kv);
      const long long at = ((long long)tok * c.heads + head) * D + 8 * ch;
      if (dst && AWQ_SPAN_OK(at, 8, all, BS_KV4_OUT)) *reinterpret_cast<uint4*>(dst + at) = out;
    }
  }

  if (!own.strips) return;
  const int i = __ffs(own.strips) - 1, tok = begin + i, slot = __shfl_sync(0xffffffffu, own.slot, i);
  const long long page = slot >> c.page_shift;
  uint32_t(&cw)[16][33] = codes[warp];
  const int apart = c.heads < 4, slices = D > 128 ? 2 : 1, width = D / slices, row = width / 8;  // items as in the write
  const int t0 = lane / row, ch0 = lane - t0 * row, dt = 32 / row, dch = 32 - dt * row;
  for (int it = warp; it < slices * c.heads << apart; it += KV4_APPEND_WARPS) {
    const int slice = slices == 2 ? it & 1 : 0, hv = slices == 2 ? it >> 1 : it, head = apart ? hv >> 1 : hv;
#pragma unroll 1
    for (int val = apart ? hv & 1 : 0, end = apart ? val + 1 : 2; val < end; ++val) {
      uint16_t* dst = static_cast<uint16_t*>(val ? vv : kv);
      if (!dst) continue;
      const long long base = in ? c.strip(page, head, slot & in_mask) : 0;
      const bool ok = in && AWQ_SPAN_OK(base, c.strip_bytes, c.bytes(), BS_KV4_CACHE);
      const uint8_t* s = c.base + base;
      if (val && ok) {
        if (lane < width / 4) {
          const int h = lane & 1, q = (lane >> 1) & 3, p = lane >> 3;
          const uint8_t* from = s + 8 * D + ((slice * (width / 32) + p) * 32 + q) * 8 + 4 * h;
          uint32_t w[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) w[r] = *reinterpret_cast<const uint32_t*>(from + 32 * r);
          kv4_transpose(w);
#pragma unroll
          for (int j = 0; j < 8; ++j) cw[kv4_row_token(j, q)][kv4_row_chunk(j, p, h)] = w[j];
        }
        __syncwarp();
      }
      const uint8_t* pars = s + 16 * D + (val ? 64 * ng : 0);
      int t = t0, c0 = ch0;
#pragma unroll 2
      for (int u0 = 0; u0 < 16 * row; u0 += 32) {
        const int ch = slice * row + c0;
        uint4 out = make_uint4(0, 0, 0, 0);
        if (ok) {
          const uint32_t word =
              val ? cw[t][c0] : *reinterpret_cast<const uint32_t*>(s + t * (D / 2) + ((ch & 3) * (D / 32) + (ch >> 2)) * 4);
          out = kv4_values<F16>(word, *reinterpret_cast<const uint32_t*>(pars + (ch >> per_bits) * 64 + 4 * t));
        }
        const long long at = ((long long)(tok + t) * c.heads + head) * D + 8 * ch;
        if (AWQ_SPAN_OK(at, 8, all, BS_KV4_OUT)) *reinterpret_cast<uint4*>(dst + at) = out;
        t += dt;
        c0 += dch;
        if (c0 >= row) c0 -= row, ++t;
      }
      __syncwarp();
    }
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

// 2^x, at most 2 units off; -inf gives 0
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr int KV4_UNIT = 32;       // tokens a warp takes at a time: two strips
constexpr int KV4_RECENTRE = 4;    // units between recentre()s
constexpr float KV4_HEAD = 6.0f;   // the largest weight's exponent where a reference is taken
constexpr float KV4_LOWEST = -1.7e38f;  // reference exponent of a part that saw no token

// What a warp knows of a tile of 8 NT query rows of one (sequence, kv head).
// Column j of n-tile u is row 8 u + j of the tile; a lane works on columns
// 2 q and 2 q + 1 of each n-tile.
template <int D, int G, int NT>
struct Kv4Warp {
  static constexpr int NJ = D / 32, NG = D / G, JG = G / 32;
  static constexpr int STRIP = kv4_strip_bytes(D, G);
  // strips worked on at once: two hide each other's latencies where there are registers for it
  static constexpr int NS = D * NT <= 128 && NG * NT <= 3 ? 2 : 1;
  uint32_t qf[NT][NJ][4];      // B operands: queries, even channels then odd ones (times 2^-4)
  float qsum[NT][NG][2];       // 2^-24 sum of the scaled query over a group, columns 2 q, 2 q + 1
  float qscale[NT][2];         // score (log2) per accumulator unit
  int vis[NT][2];              // keys [0, vis) are visible to the column's query
  int vis_min, vis_max;        // over the tile's rows
  bool fresh;                  // no tokens yet: the first ones set the reference
  float o[NT][NJ][2][4];       // accumulators: channels 32 p + 16 n + ..., value 2^-24 (n = 0) or 2^-20 units
  float mid[NT][NG][4];        // -2^-24 sum of w zero since the last recentre(), in every row
  float m[NT][2], l[NT][2];    // reference exponent (the same in all lanes of a column), sum of p over this lane's tokens

  // Rows [r0, r0 + 8 NT) of the sequence's n * share query rows (row = token * share + head in the group).
  __device__ __forceinline__ void load_queries(const Kv4AttnArgs& a, const Kv4Seq& s, int head, int r0, int lane) {
    const int g = lane >> 2, q = lane & 3;
    const int rows = s.n * a.share;
    vis_min = 0x7fffffff;
    vis_max = 0;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      // this lane loads column g: 8 channels of each 32
      const int r = r0 + 8 * u + g;
      const bool in = r < rows;
      const int tok = in ? (int)((unsigned)r / (unsigned)a.share) : 0, e = in ? r - tok * a.share : 0;
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
      // [2^10, 2^11): fp16 then holds every entry down to 2^-20 of it to 11
      // bits, also the odd channels' 2^-4. Exact back through the scale.
      const int ex = top > 0.0f ? min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -110), 127) : 0;
      const float even = __uint_as_float((uint32_t)(137 - ex) << 23), odd = even * 0.0625f;
      float part[NG];
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) part[gi] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float(&y)[8] = x[j];
        part[j / JG] += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
        qf[u][j][0] = pack2<true>(y[0] * even, y[4] * even);
        qf[u][j][1] = pack2<true>(y[2] * even, y[6] * even);
        qf[u][j][2] = pack2<true>(y[1] * odd, y[5] * odd);
        qf[u][j][3] = pack2<true>(y[3] * odd, y[7] * odd);
      }
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) part[gi] *= even;
      // 2^(ex + 14): through two factors, as 2^14 more than a float's largest may be meant
      const float unit = __uint_as_float((uint32_t)(117 + ex) << 23) * (16777216.0f * a.scale_log2);
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
        m[u][c] = 0.0f;
        l[u][c] = 0.0f;
      }
      if (in) {
        vis_min = min(vis_min, see);
        vis_max = max(vis_max, see);
      }
    }
    fresh = true;
    vis_min = __reduce_min_sync(0xffffffffu, vis_min);
    vis_max = __reduce_max_sync(0xffffffffu, vis_max);
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int p = 0; p < NJ; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[u][p][n][i] = 0.0f;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi)
#pragma unroll
        for (int i = 0; i < 4; ++i) mid[u][gi][i] = 0.0f;
    }
  }

  // Reference exponents that admit these scores (d: score - m; dv: value
  // steps of the lane's two tokens a strip): the largest score plus the
  // exponent of its token's value step, less KV4_HEAD, so that the largest
  // w = p step lies in [2^6, 2^7) whatever the steps are. Moves d along. Taken for
  // a tile's first tokens and then only when a weight passes 2^15, so the largest
  // weight of a row is never below 2^6: groups whose steps are 2^20 below the
  // loudest one's have weights of fp16's full precision still. (A column that sees
  // none of a tile's first tokens sees none of the later ones either: rows see a
  // prefix of the context.)
  template <int N>
  __device__ __forceinline__ void raise(float (&d)[N][NT][4], const float (&dv)[N][NG][2]) {
    float e[N][2];
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = dv[s][0][h];
#pragma unroll
        for (int gi = 1; gi < NG; ++gi) x = fmaxf(x, dv[s][gi][h]);
        // (the quantiser's steps are 2^-24 or more; 0 is a token never written)
        e[s][h] = (float)max((int)(__float_as_uint(x) >> 23) - 127, -24);
      }
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float up = fresh ? -INFINITY : 0.0f;
#pragma unroll
        for (int s = 0; s < N; ++s) up = fmaxf(up, fmaxf(d[s][u][c] + e[s][0], d[s][u][c + 2] + e[s][1]) - KV4_HEAD);
        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 4));
        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 8));
        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 16));
        if (up == -INFINITY) up = 0.0f;
        // (d moves by what m really moved; a fresh state holds zeros, and its
        // reference may fall by any amount)
        const float mn = m[u][c] + up, by = mn - m[u][c], f = fresh ? 1.0f : exp2_fast(-by);
        m[u][c] = mn;
        l[u][c] *= f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
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
#pragma unroll
        for (int s = 0; s < N; ++s) {
          d[s][u][c] -= by;
          d[s][u][c + 2] -= by;
        }
      }
    fresh = false;
  }

  // N strips at `base`, tokens t0 .. of the context. EDGE: some of the tile's
  // queries do not see all of the tokens, whose bytes may hold anything then;
  // drop: strips (by bit) that are left out.
  template <bool EDGE, int N>
  __device__ __forceinline__ void strips(const uint8_t* base, int t0, unsigned drop, int lane) {
    const int g = lane >> 2, q = lane & 3;
    // scores: token rows g and g + 8 of a strip, columns 2 q and 2 q + 1
    float d[N][NT][4];
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint8_t* b = base + s * STRIP;
      uint32_t kw0[NJ], kw1[NJ];
      load_words<NJ>(b + g * (D / 2) + 4 * q * NJ, kw0);
      load_words<NJ>(b + (g + 8) * (D / 2) + 4 * q * NJ, kw1);
      const uint32_t* kpar = reinterpret_cast<const uint32_t*>(b + 16 * D) + g;
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
        const float2 p0 = widen2<true>(kpar[16 * gi]), p1 = widen2<true>(kpar[16 * gi + 8]);
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 p = i < 2 ? p0 : p1;
            const float x = fmaf(-p.y, qsum[u][gi][i & 1], acc[u][i]);
            d[s][u][i] = gi == 0 ? (NG == 1 ? fmaf(x, p.x * qscale[u][i & 1], -m[u][i & 1]) : x * p.x)
                                 : fmaf(x, p.x, d[s][u][i]);
          }
      }
      if (NG > 1) {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[s][u][i] = fmaf(d[s][u][i], qscale[u][i & 1], -m[u][i & 1]);
      }
    }
    // value steps of tokens g and g + 8, zeros (as codes, negative) of tokens
    // 2 q, 2 q + 1 and 2 q + 8, 2 q + 9: an A operand whose 16 rows are alike
    float dv[N][NG][2];
    uint32_t zc[N][NG][2];
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t* vpar = reinterpret_cast<const uint32_t*>(base + s * STRIP + 16 * D) + 16 * NG;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (a token never written has step 0; the 2^-60, which is lost in any other
          // step, lets it outgrow the reference too, as its probability counts)
          dv[s][gi][h] = __low2float(*reinterpret_cast<const __half2*>(vpar + 16 * gi + 8 * h + g)) + 8.673617379884035e-19f;
          const uint2 pz = *reinterpret_cast<const uint2*>(vpar + 16 * gi + 8 * h + 2 * q);
          uint32_t z = __byte_perm(pz.x, pz.y, 0x7632);
          if (EDGE) {
            const __half2 ok = __hmin2(__hmax2(*reinterpret_cast<const __half2*>(&z), __float2half2_rn(0.0f)),
                                       __float2half2_rn(15.0f));
            z = *reinterpret_cast<const uint32_t*>(&ok);
          }
          const uint32_t unit = 0x80018001u;  // -2^-24 twice
          const __half2 zz = __hmul2(*reinterpret_cast<const __half2*>(&z), *reinterpret_cast<const __half2*>(&unit));
          zc[s][gi][h] = *reinterpret_cast<const uint32_t*>(&zz);
        }
    }
    bool hidden[N][NT][4];
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hidden[s][u][i] = EDGE && (t0 + 16 * s + g + 8 * (i >> 1) >= vis[u][i & 1] || (drop >> s & 1u));
          if (hidden[s][u][i]) d[s][u][i] = -INFINITY;
        }
    float w[N][NT][NG][4];
    float p[N][NT][4];
    auto weigh = [&]() {
      bool big = false;
#pragma unroll
      for (int s = 0; s < N; ++s)
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[s][u][i] = exp2_fast(d[s][u][i]);
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
              const float x = p[s][u][i] * dv[s][gi][i >> 1];
              w[s][u][gi][i] = hidden[s][u][i] ? 0.0f : x;
              big |= w[s][u][gi][i] > 32768.0f;
            }
          }
      return fresh || __any_sync(0xffffffffu, big);
    };
    if (weigh()) {
      raise<N>(d, dv);
      weigh();
    }
    uint32_t wb[N][NT][NG][2];
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        l[u][0] += p[s][u][0] + p[s][u][2];
        l[u][1] += p[s][u][1] + p[s][u][3];
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          const float(&x)[4] = w[s][u][gi];
          wb[s][u][gi][0] = transpose_8x8(pack2<true>(x[0], x[1]));
          wb[s][u][gi][1] = transpose_8x8(pack2<true>(x[2], x[3]));
          mma_16816(mid[u][gi], zc[s][gi][0], zc[s][gi][0], zc[s][gi][1], zc[s][gi][1], wb[s][u][gi][0], wb[s][u][gi][1]);
        }
      }
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint2* vw = reinterpret_cast<const uint2*>(base + s * STRIP + 8 * D) + lane;
#pragma unroll
      for (int pp = 0; pp < NJ; ++pp) {
        const uint2 c = vw[32 * pp];
        const uint32_t x = c.x >> 8, y = c.y >> 8;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          const uint32_t b0 = wb[s][u][pp / JG][0], b1 = wb[s][u][pp / JG][1];
          mma_16816(o[u][pp][0], c.x & 0x000F000Fu, c.y & 0x000F000Fu, x & 0x000F000Fu, y & 0x000F000Fu, b0, b1);
          mma_16816(o[u][pp][1], c.x & 0x00F000F0u, c.y & 0x00F000F0u, x & 0x00F000F0u, y & 0x00F000F0u, b0, b1);
        }
      }
    }
  }

  // One unit (two strips) at `base`, tokens t0 .. t0 + 31.
  __device__ __forceinline__ void unit(const uint8_t* base, int t0, unsigned drop, int lane) {
    if constexpr (NS == 2) {
      if (t0 + 32 > vis_min || drop)
        strips<true, 2>(base, t0, drop, lane);
      else
        strips<false, 2>(base, t0, 0, lane);
    } else {
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        if (t0 + 16 * s >= vis_max) break;
        if (drop >> s & 1u) continue;  // (it would set the reference to nothing)
        if (t0 + 16 * s + 16 > vis_min)
          strips<true, 1>(base + s * STRIP, t0 + 16 * s, 0, lane);
        else
          strips<false, 1>(base + s * STRIP, t0 + 16 * s, 0, lane);
      }
    }
  }

  // Take sum(w zero) off the accumulated codes (16 times that where codes count
  // 16-fold): they then hold sum w (c - zero), which wanders about zero, while
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
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[u][c] += __shfl_xor_sync(0xffffffffu, l[u][c], d);
  }

  // The finished state of column 2 q + c of n-tile u: channel 32 p + 16 n + 8 h + g, unnormalised.
  __device__ __forceinline__ float value(int u, int c, int p, int n, int h) const {
    return o[u][p][n][2 * h + c] * (n ? 1048576.0f : 16777216.0f);
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
            for (int h = 0; h < 2; ++h) row[32 * p + 16 * n + 8 * h + g] = value(u, c, p, n, h);
        if (g == 0) {
          row[D] = l[u][c] == 0.0f ? KV4_LOWEST : m[u][c];
          row[D + 1] = l[u][c];
        }
      }
  }
};

// ------------------------------------------------------------------ attention, split evenly over the GPU
// Work is counted in units of two strips of one tile (8 NT query rows of one
// sequence and kv head), ordered by sequence, head, tile, tokens. Every working
// warp of the grid takes one contiguous range of equal length, whatever the
// contexts' lengths, out of a ring of its own in shared memory that the block's
// producer warp keeps filled (lane i serves working warp i: one cp.async.bulk a
// unit, two with pages of 16, on across tiles); no working warp waits for
// another until its range is done. A tile that lies in one warp's range is
// written out by it; the at most two that it shares (its first and its last) go
// to shared memory as (unnormalised output, m, l), are joined within the block,
// and where they cross blocks, through the workspace, by kv4_attention_join. All
// joins run in the order of the ranges, so the result is the same every time.
// A tile's queries, its first reference and its end cost a warp about as much
// as KV4_EDGE units, so the ranges are cut in a count that has that many more
// at the front of each tile.
// With short contexts (the page tables bound them) the blocks' ranges begin and
// end with tiles instead (`solo`): some blocks then have more to do, but there
// is nothing to join between blocks and the second launch falls away.
//
// Bound by HBM while it runs: 64 sequences of up to 8192 tokens (8 kv heads of 128,
// 293 MB) take 62 us where a copy of as many bytes takes 45, four contexts of
// 131072 (604 MB) 119 us (92). The strips arrive at 6.9 TB/s; the rest is the
// launch and the plan (4 us until the first copies are asked for), the slowest
// warp of a block (2 to 3 us behind the mean) and the two joins (2 and 4 us). A
// sequence of 777 tokens with 32 kv heads takes 8.7 us; 16 sequences with 5
// queries each, 16 rows a tile, 24 us, of which the same ends are half.
constexpr int KV4_EDGE = 2;
constexpr int KV4_MAX_BATCH = 512;  // sequences of a launch: what the block needs of them sits in shared memory
constexpr int KV4_CTAS = 148;       // blocks of the grid, one per SM
// Working warps of a block: as many as their state leaves registers for.
constexpr int kv4_warps(int dim, int group, int nt) {
  return dim * nt > 128 ? 7 : dim / group * nt == 1 || (dim == 64 && nt == 1) ? 15 : 11;
}
constexpr int KV4_STAGES = 2;       // units in a warp's ring

struct Kv4SplitArgs {
  Kv4AttnArgs a;
  int tile_rows;    // 8 NT
  float* cta_part;  // [KV4_CTAS][2][8 NT][D + 4]
  long long* cta_seg;  // [KV4_CTAS][2] tile of a block partial (-1: none)
  int* cta_bad;     // [KV4_CTAS]
  int max_rows;     // sequences of more query rows are another kernel's
  int solo;         // blocks take whole tiles
  int clear_err;    // the first launch of a call sets the error word, later ones add to it
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The batch: count[b] = counted units before sequence b, real[b] = units before
// it; units of a tile (span) and tiles of a head of each, its rows and context.
struct Kv4Plan {
  long long count[KV4_MAX_BATCH + 1], real[KV4_MAX_BATCH + 1];
  int span[KV4_MAX_BATCH], tiles[KV4_MAX_BATCH], row0[KV4_MAX_BATCH], n[KV4_MAX_BATCH], len[KV4_MAX_BATCH];
  int bad;
  __device__ __forceinline__ Kv4Seq seq(int b) const {
    Kv4Seq s;
    s.row0 = row0[b];
    s.n = n[b];
    s.L = len[b];
    s.bad = false;
    return s;
  }
};

// Filled by the whole block.
__device__ __forceinline__ void kv4_plan(const Kv4SplitArgs& s, Kv4Plan& p, longlong2* warp_sums) {
  const Kv4AttnArgs& a = s.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (threadIdx.x == 0) p.count[0] = p.real[0] = 0;
  long long count0 = 0, real0 = 0;
  bool bad = false;
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    long long count = 0, real = 0;
    if (b < a.batch) {
      const Kv4Seq q = kv4_seq(a, b);
      bad |= q.bad;
      const int rows = q.n * a.share;
      // a sequence without context still has its rows to write: one unit, which reads nothing
      const int span = q.n > 0 && rows <= s.max_rows ? max(1, (int)(((long long)q.L + KV4_UNIT - 1) / KV4_UNIT)) : 0;
      const int tiles = (rows + s.tile_rows - 1) / s.tile_rows;
      p.span[b] = span;
      p.tiles[b] = tiles;
      p.row0[b] = (int)q.row0;
      p.n[b] = q.n;
      p.len[b] = q.L;
      const long long all = (long long)tiles * a.c.heads;
      real = all * span;
      count = real + all * (span ? KV4_EDGE : 0);
    }
#pragma unroll 1
    for (int d = 1; d < min(32, a.batch); d <<= 1) {  // (what lies behind the batch is 0)
      const long long x = __shfl_up_sync(0xffffffffu, count, d), y = __shfl_up_sync(0xffffffffu, real, d);
      if (lane >= d) {
        count += x;
        real += y;
      }
    }
    if (a.batch > 32) {
      if (lane == 31) warp_sums[warp] = make_longlong2(count, real);
      __syncthreads();
    }
    if (b < a.batch) {
      for (int w = 0; w < warp; ++w) {
        count += warp_sums[w].x;
        real += warp_sums[w].y;
      }
      p.count[b + 1] = count0 + count;
      p.real[b + 1] = real0 + real;
    }
    if (b0 + (int)blockDim.x < a.batch) {
      for (int w = 0; w < warps; ++w) {
        count0 += warp_sums[w].x;
        real0 += warp_sums[w].y;
      }
      __syncthreads();
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.bad = any;
}

// A place in the order of units.
struct Kv4Cursor {
  int b, at, span, tile, tiles, head;  // unit `at` of `span` of a tile
  // Counted place u (inside the batch): the unit there, or the tile's first
  // where u counts its edge. Returns how far u lies behind the tile's begin.
  __device__ __forceinline__ int seek(const Kv4Plan& p, int batch, long long u) {
    int lo = 0, hi = batch;  // count[lo] <= u < count[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.count[mid] <= u) lo = mid;
      else hi = mid;
    }
    b = lo;
    span = p.span[b];
    tiles = p.tiles[b];
    const long long in = u - p.count[b];
    const int wide = span + KV4_EDGE;
    const int seg = in >> 32 ? (int)(in / wide) : (int)((unsigned)in / (unsigned)wide);
    const int off = (int)(in - (long long)seg * wide);
    at = max(0, off - KV4_EDGE);
    head = (int)((unsigned)seg / (unsigned)tiles);
    tile = seg - head * tiles;
    return off;
  }
  // units before this place
  __device__ __forceinline__ long long index(const Kv4Plan& p) const {
    return p.real[b] + (long long)(head * tiles + tile) * span + at;
  }
  // to the next unit; true if it begins another tile
  __device__ __forceinline__ bool step(const Kv4Plan& p, const Kv4AttnArgs& a) {
    if (++at < span) return false;
    at = 0;
    if (++tile == tiles) {
      tile = 0;
      if (++head == a.c.heads) {
        head = 0;
        do ++b;
        while (b < a.batch && p.span[b] == 0);
        if (b < a.batch) {
          span = p.span[b];
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

// all * i / n, i <= n <= 256
__device__ __forceinline__ long long kv4_share(long long all, int i, int n) {
  // (a 64-bit quotient takes some 200 cycles)
  return all < (1 << 24) ? (long long)((unsigned)all * (unsigned)i / (unsigned)n) : all * i / n;
}

// The ranges of the W working warps of this block, found by the producer warp:
// lane w gets the first unit and the number of units of working warp w.
__device__ __forceinline__ int kv4_ranges(const Kv4SplitArgs& s, const Kv4Plan& p, int W, int lane, Kv4Cursor& cur) {
  const int batch = s.a.batch;
  // Where there are fewer counted units than takers, the last takers get none,
  // so that the parts of a tile always are with neighbours.
  const long long all = p.count[batch];
  const int blocks = (int)min((long long)gridDim.x, all), c = blockIdx.x;
  if (c >= blocks) return 0;
  long long mine = kv4_share(all, c + (lane & 1), blocks);  // even lanes: the block's begin, odd ones: its end
  if (s.solo && mine < all)                                // up to the begin of a tile
    if (const int off = cur.seek(p, batch, mine)) mine += cur.span + KV4_EDGE - off;
  const long long c0 = __shfl_sync(0xffffffffu, mine, 0), c1 = __shfl_sync(0xffffffffu, mine, 1);
  const int warps = (int)min((long long)W, c1 - c0);
  long long at = p.real[batch];
  if (lane <= warps) {
    const long long u = c0 + (warps ? kv4_share(c1 - c0, lane, warps) : 0);
    if (u < all) {
      cur.seek(p, batch, u);
      at = cur.index(p);
    }
  }
  const long long next = __shfl_down_sync(0xffffffffu, at, 1);
  return lane < warps ? (int)(next - at) : 0;
}

// Query row r (in the sequence's n * share) of a kv head: its row in out and lse; -1 if there is none.
__device__ __forceinline__ long long kv4_out_row(const Kv4AttnArgs& a, const Kv4Seq& s, int head, int r) {
  if (r >= s.n * a.share) return -1;
  const int t = (int)((unsigned)r / (unsigned)a.share);
  const long long tok = s.row0 + t;
  if (!AWQ_IDX_OK(tok, a.T, BS_KV4_O)) return -1;
  return tok * a.q_heads + head * a.share + (r - t * a.share);
}

// Row `row` of a tile joined by one warp out of n parts part(0), part(1), ...:
// the lane's channels 4 lane + 128 k, unnormalised, and m and l.
template <int D>
struct Kv4Joined {
  static constexpr int K = (D + 127) / 128;
  float4 v[K];
  float m, l;
  template <typename Part>
  __device__ __forceinline__ void join(Part part, int n, int row, int lane) {
    m = KV4_LOWEST;
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int e0 = 0; e0 < n; e0 += 32) {  // 32 parts at a time: lane i takes the i-th one's m and l
      const int cnt = min(32, n - e0);
      float2 ml = make_float2(KV4_LOWEST, 0.0f);
      if (lane < cnt) ml = *reinterpret_cast<const float2*>(part(e0 + lane) + row * (D + 4) + D);
      float top = fmaxf(m, ml.x);
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float old = exp2_fast(m - top), f = exp2_fast(ml.x - top);  // (NaN in a part's sums passes on)
      m = top;
      float add = f * ml.y;
#pragma unroll
      for (int d = 16; d; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
      l = fmaf(l, old, add);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k].x *= old;
        v[k].y *= old;
        v[k].z *= old;
        v[k].w *= old;
      }
#pragma unroll 4
      for (int e = 0; e < cnt; ++e) {
        const float* r = part(e0 + e) + row * (D + 4);
        const float fe = __shfl_sync(0xffffffffu, f, e);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int c = 4 * lane + 128 * k;
          if (c < D) {
            const float4 x = *reinterpret_cast<const float4*>(r + c);
            v[k].x = fmaf(fe, x.x, v[k].x);
            v[k].y = fmaf(fe, x.y, v[k].y);
            v[k].z = fmaf(fe, x.z, v[k].z);
            v[k].w = fmaf(fe, x.w, v[k].w);
          }
        }
      }
    }
  }
  // behind m and l: the row of out that this becomes
  __device__ __forceinline__ void store(float* r, long long at, int lane) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (4 * lane + 128 * k < D) *reinterpret_cast<float4*>(r + 4 * lane + 128 * k) = v[k];
    if (lane == 0)
      *reinterpret_cast<float4*>(r + D) = make_float4(m, l, __int_as_float((int)(at & 0xffffffff)), __int_as_float((int)(at >> 32)));
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
  static constexpr int STAGES = KV4_STAGES;
  static constexpr int PART = 8 * NT * (D + 4);
  static_assert(PART * (int)sizeof(float) <= STAGES * 2 * STRIP, "a warp's last part lies in its ring");
  alignas(128) uint8_t ring[W][STAGES][2 * STRIP];
  float part[W][PART];   // a warp's first part
  alignas(8) uint64_t full[W][STAGES];
  uint64_t empty[W][STAGES];
  Kv4Plan plan;
  longlong2 sums[W + 1];
  Kv4Cursor begin[W];    // a working warp's first unit
  int units[W];          // and how many it has
  long long seg[W][2];   // tile of a warp's first and last part (-1: none)
  int flags[W][2];       // bit 0: the part begins its tile, bit 1: it ends it
  uint8_t lost[W][4];    // strips of a stage's unit that are not there to be read (by bit)
  int bad;
  int abort;
};

// Lane i of the producer warp: the units of working warp i.
template <int D, int G, int NT>
__device__ __forceinline__ void kv4_produce(const Kv4SplitArgs& s, Kv4SplitSmem<D, G, NT>& sm, int lane) {
  using Sm = Kv4SplitSmem<D, G, NT>;
  constexpr int W = Sm::W, STAGES = Sm::STAGES, STRIP = Sm::STRIP;
  const Kv4AttnArgs& a = s.a;
  Kv4Cursor cur{};
  int left = kv4_ranges(s, sm.plan, W, lane, cur), stage = 0, sent = 0;
  if (lane < W) {
    sm.begin[lane] = cur;
    sm.units[lane] = left;
  }
  __syncthreads();  // (the working warps are there for it at once)
  uint32_t phase = 1;  // a fresh ring is empty
  int page[2] = {-1, -1};
  // pages of 16 tokens hold one strip of the unit each, larger ones both, one behind the other
  const bool two = a.c.page_shift == 4;
  auto look = [&]() {
    const int p = KV4_UNIT * cur.at >> a.c.page_shift;
    const int* row = a.table + (long long)cur.b * a.table_pages;
    page[0] = p < a.table_pages ? __ldg(row + p) : -1;
    if (two) page[1] = p + 1 < a.table_pages ? __ldg(row + p + 1) : -1;
  };
  if (left > 0) look();
  uint64_t idle_since = 0;
  while (__any_sync(0xffffffffu, left > 0)) {
    bool moved = false;
    if (left > 0 && mbar_test(smem_u32(&sm.empty[lane][stage]), phase)) {
      moved = true;
      const uint32_t bar = smem_u32(&sm.full[lane][stage]), dst = smem_u32(sm.ring[lane][stage]);
      const int t0 = KV4_UNIT * cur.at, len = sm.plan.len[cur.b];
      unsigned lost = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !two) break;
        const uint32_t n = two ? STRIP : 2 * STRIP;
        const bool in = t0 + 16 * h < len;
        bool good = in && page[h] >= 0 && page[h] < a.c.n_pages;
        if (in && !good) sm.bad = ERR_KV4_PAGE;
        const long long off = good ? a.c.strip(page[h], cur.head, t0 & ((1 << a.c.page_shift) - 1)) : 0;
        good = good && AWQ_SPAN_OK(off, n, a.c.bytes(), BS_KV4_STRIP);
        if (good) {
          mbar_expect_tx(bar, n);
          bulk_load(dst + h * STRIP, a.c.base + off, n, bar);
        } else {
          lost |= two ? 1u << h : 3u;
        }
      }
      sm.lost[lane][stage] = (uint8_t)lost;
      mbar_arrive(bar);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      ++sent;
      if (--left > 0) {
        cur.step(sm.plan, a);
        look();
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
      idle_since = 0;
    } else {
      // nothing to fill: a unit takes a warp over a microsecond
      __nanosleep(64);
      if (*(volatile int*)&sm.abort) break;
      const uint64_t now = globaltimer_ns();
      if (idle_since == 0) idle_since = now;
      if (__any_sync(0xffffffffu, now - idle_since > 2 * AWQ_WAIT_LIMIT_NS)) break;
    }
  }
  // copies in flight end before the block does (their units are waited for by
  // the working warps, unless a wait there gave up)
  __syncwarp();
  if (*(volatile int*)&sm.abort && lane < W && sent > 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  __syncwarp();
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(32 * (kv4_warps(D, G, NT) + 1), 1)
    kv4_attention_split(const __grid_constant__ Kv4SplitArgs s) {
  using Sm = Kv4SplitSmem<D, G, NT>;
  using St = Kv4Warp<D, G, NT>;
  constexpr int W = Sm::W, STAGES = Sm::STAGES, PART = Sm::PART;
  extern __shared__ uint8_t smem_raw[];
  // (offset, not address, arithmetic keeps the accesses shared-memory ones)
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u));
  const Kv4AttnArgs& a = s.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0 && warp < W) {
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&sm.full[warp][i]), 1);
      mbar_init(smem_u32(&sm.empty[warp][i]), 1);
    }
    fence_barrier_init();
    sm.seg[warp][0] = sm.seg[warp][1] = -1;
  }
  if (threadIdx.x == 0) {
    sm.bad = 0;
    sm.abort = 0;
  }
  wait_for_kernel_before();
  kv4_plan(s, sm.plan, sm.sums);
  if (warp == W) {
    kv4_produce<D, G, NT>(s, sm, lane);
    if (s.solo && blockIdx.x == 0) {
      // no second kernel gathers what the blocks found: this warp looks at all
      // pages of the batch (few, or the call would not be solo)
      int bad = sm.plan.bad ? ERR_KV4_PAGE : 0;
      for (int i = lane; i < a.batch * a.table_pages; i += 32) {
        const int b = i / a.table_pages, p = i - b * a.table_pages, page = __ldg(a.table + i);
        if (sm.plan.span[b] > 0 && (long long)p << a.c.page_shift < sm.plan.len[b] && (page < 0 || page >= a.c.n_pages))
          bad = ERR_KV4_PAGE;
      }
      bad = __reduce_max_sync(0xffffffffu, bad);
      if (lane == 0 && (s.clear_err || bad)) *a.err = bad;
      if (lane == 0 && bad) keep_device_error(bad);
    }
  } else {
    __syncthreads();
    Kv4Cursor cur = sm.begin[warp];
    int left = sm.units[warp], stage = 0;
    uint32_t phase = 0;
    bool fresh_tile = true, first = true, begins = cur.at == 0;
    St w;
    int done = 0;
    while (left > 0) {
      if (fresh_tile) {
        w.load_queries(a, sm.plan.seq(cur.b), cur.head, cur.tile * s.tile_rows, lane);
        fresh_tile = false;
        done = 0;
      }
      const bool here = mbar_wait_lean(smem_u32(&sm.full[warp][stage]), phase, &sm.abort, nullptr, 0);
      if (!__all_sync(0xffffffffu, here)) {
        // a copy that never came (the wait took two seconds): report, write nothing
        if (lane == 0) {
          sm.bad = ERR_KV4_COPY;
          keep_device_error(ERR_KV4_COPY);
          if (s.solo) *a.err = ERR_KV4_COPY;
        }
        break;
      }
      const unsigned lost = sm.lost[warp][stage];
      if (lost != 3u && KV4_UNIT * cur.at < w.vis_max) {
        w.unit(sm.ring[warp][stage], KV4_UNIT * cur.at, lost, lane);
        if (++done % KV4_RECENTRE == 0) w.recentre();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.empty[warp][stage]));
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      --left;
      const bool ends = cur.at + 1 == cur.span;
      if (ends || left == 0) {
        w.finish();
        if (begins && ends) {
          // the whole tile: write it
          const Kv4Seq seq = sm.plan.seq(cur.b);
          const int g = lane >> 2, q = lane & 3;
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const long long at = kv4_out_row(a, seq, cur.head, cur.tile * s.tile_rows + 8 * u + 2 * q + c);
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
          // (a last part that is not the first follows the warp's last unit: its ring is free)
          const int k = first ? 0 : 1;
          __syncwarp();
          w.store(k ? reinterpret_cast<float*>(sm.ring[warp][0]) : sm.part[warp], lane);
          if (lane == 0) {
            sm.seg[warp][k] = cur.id(a);
            sm.flags[warp][k] = (begins ? 1 : 0) | (ends ? 2 : 0);
          }
        }
        first = false;
        if (left > 0) {
          cur.step(sm.plan, a);
          begins = true;
          fresh_tile = true;
        }
      } else {
        ++cur.at;
      }
    }
  }
  let_next_kernel_start();
  __syncthreads();
  // ---------------- join the warps' parts: chains of consecutive parts of one tile
  // lane e of every warp looks at part e (2 W <= 32): which parts begin a chain
  static_assert(2 * W <= 32, "parts of a block");
  const long long my_seg = lane < 2 * W ? sm.seg[lane >> 1][lane & 1] : -1;
  const int my_flags = lane < 2 * W ? sm.flags[lane >> 1][lane & 1] : 0;
  const unsigned valid = __ballot_sync(0xffffffffu, my_seg >= 0);
  const unsigned below = valid & ((1u << lane) - 1u);
  const long long prev = __shfl_sync(0xffffffffu, my_seg, below ? 31 - __clz(below) : 0);
  unsigned heads = __ballot_sync(0xffffffffu, my_seg >= 0 && (!below || prev != my_seg));
  if (threadIdx.x == 0) {
    if (!s.solo) s.cta_bad[blockIdx.x] = sm.bad ? sm.bad : sm.plan.bad ? ERR_KV4_PAGE : 0;
    // slot 0: a tile that an earlier block began, slot 1: one that a later block ends
    if (!s.solo) s.cta_seg[2 * blockIdx.x] = s.cta_seg[2 * blockIdx.x + 1] = -1;
  }
  __syncthreads();
  for (int turn = 0; heads; ++turn) {
    const int e0 = __ffs(heads) - 1;
    heads &= heads - 1;
    const long long seg = __shfl_sync(0xffffffffu, my_seg, e0);
    const unsigned mine = __ballot_sync(0xffffffffu, my_seg == seg);
    const int flags = __reduce_or_sync(0xffffffffu, (unsigned)(my_seg == seg ? my_flags : 0));
    const int b = (int)(seg >> 32) / a.c.heads, head = (int)(seg >> 32) - b * a.c.heads;
    // rows go round the warps, on from where the last chain's stopped
    for (int row = (warp + (W + 1) * 8 * NT - turn * 8 * NT % (W + 1)) % (W + 1); row < 8 * NT; row += W + 1) {
      const long long at = kv4_out_row(a, sm.plan.seq(b), head, (int)(seg & 0xffffffff) * s.tile_rows + row);
      Kv4Joined<D> j;
      // the i-th part of the chain: e0, then the first parts of the warps behind
      j.join(
          [&](int i) -> const float* {
            return i == 0 && (e0 & 1) ? reinterpret_cast<const float*>(sm.ring[e0 >> 1][0]) : sm.part[(e0 >> 1) + i];
          },
          __popc(mine), row, lane);
      if (flags == 3) {
        j.write(a, at, lane);
      } else if (!s.solo) {
        // shared with other blocks: slot 1 if it begins here, else 0
        const int k = flags & 1;
        j.store(s.cta_part + ((long long)blockIdx.x * 2 + k) * PART + row * (D + 4), at, lane);
        if (row == 0 && lane == 0) s.cta_seg[2 * blockIdx.x + k] = seg;
      }
    }
  }
}

constexpr int KV4_JOIN_WARPS = 16;

// Block c joins the tile that block c of the split began and did not end:
// its slot 1, then slot 0 of the following blocks while they hold that tile.
// Block 0 sets the call's error word. Launched to overlap the split's end.
template <int D, int NT>
__global__ void __launch_bounds__(32 * KV4_JOIN_WARPS) kv4_attention_join(const __grid_constant__ Kv4SplitArgs s, int ctas) {
  constexpr int PART = 8 * NT * (D + 4);
  const Kv4AttnArgs& a = s.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  wait_for_kernel_before();
  if (c == 0 && warp == 0) {
    int bad = 0;
    for (int i = lane; i < ctas; i += 32) bad = max(bad, s.cta_bad[i]);
    bad = __reduce_max_sync(0xffffffffu, bad);
    if (lane == 0 && (s.clear_err || bad)) *a.err = bad;
    if (lane == 0 && bad) keep_device_error(bad);
  }
  const long long seg = s.cta_seg[2 * c + 1];
  int n = 1;
  for (int i = c + 1; i < ctas; i += 32) {  // how many blocks behind hold the tile
    const bool same = i + lane < ctas && s.cta_seg[2 * (i + lane)] == seg;
    const unsigned run = __ballot_sync(0xffffffffu, same);
    const int k = run == 0xffffffffu ? 32 : __ffs(~run) - 1;
    n += k;
    if (k < 32) break;
  }
  if (seg < 0) return;
  for (int row = warp; row < 8 * NT; row += KV4_JOIN_WARPS) {
    const float* first = s.cta_part + ((long long)c * 2 + 1) * PART + row * (D + 4) + D;
    const long long at = (long long)__float_as_int(first[3]) << 32 | (unsigned)__float_as_int(first[2]);
    Kv4Joined<D> j;
    j.join([&](int i) -> const float* { return s.cta_part + ((long long)(c + i) * 2 + (i == 0)) * PART; }, n, row, lane);
    j.write(a, at, lane);
  }
}

}  // namespace awq
