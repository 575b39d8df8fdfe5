// C ABI of the serving-side operators: the 8-bit integer linear layer and the
// 4-bit key/value cache with its attention (declared in include/awq.h).
// Included after awq_api.cu, whose host helpers it uses.
#pragma once
#include <atomic>

#include "kv4_prompt_sm100.cuh"
#include "kv4_sm100.cuh"
#include "w8a8_sm100.cuh"

namespace {

// Shared memory of a kernel, set once a context (an attribute call costs about
// a microsecond, as much as a small launch's share of it). All kernels of a
// chain ask for the largest split of L1, so that the SMs are not reconfigured
// between them. `once` belongs to the one kernel.
template <typename K>
bool kernel_smem(K kernel, int smem, std::atomic<unsigned long long>& once) {
  const unsigned long long ctx = current_context_id();
  if (ctx != 0 && once.load(std::memory_order_relaxed) == ctx) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
          cudaSuccess)
    return false;
  once.store(current_context_id(), std::memory_order_relaxed);
  return true;
}

// Launch that may start while the kernel before it on the stream still runs
// (programmatic dependent launch): the kernel waits for that one's end before it
// touches memory. cluster: CTAs of a cluster whose size the kernel leaves open.
template <typename... P, typename... A>
awq_status launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t cs, unsigned cluster, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = cs;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...) == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

bool dtype_ok(awq_dtype d) { return d == AWQ_DTYPE_BF16 || d == AWQ_DTYPE_F16; }

// ------------------------------------------------------------------ 8-bit integer linear layer
constexpr double W8_EPILOGUE_BYTES = 80.0 * 10;  // a token's part of an epilogue: about 10 ns, at 80 bytes a ns

awq_status check_w8(int64_t N, int64_t d_out, int64_t d_in) {
  if (N < 1 || d_out < 1 || d_in < 16 || d_in % 16 != 0 || d_in > W8_MAX_K) return AWQ_ERR_SHAPE;
  if (d_out > (1 << 24) || N > (1 << 24)) return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

struct W8Plan {
  bool small, pair;
  int b_rows, ctas, smem;
  W8Args a;
};

W8Plan w8_plan(int64_t N, int64_t d_out, int64_t d_in) {
  W8Plan p{};
  W8Args& a = p.a;
  a.N = (int)N;
  a.d_out = (int)d_out;
  a.n_kb = (int)cdiv(d_in, W8_BK);
  p.small = N <= W8_SMALL_N;
  if (p.small) {
    a.bn = (int)(cdiv(N, 16) * 16);
    p.b_rows = a.bn;
    a.n_mb = (int)cdiv(d_out, W8_BM);
    a.n_nb = 1;
    a.cols = a.bn <= 32 ? 32 : a.bn <= 64 ? 64 : 128;
    // three CTAs to an SM (two of the widest tiles): the ring covers the loads'
    // latency together with the neighbours', and holds [bn][128] int32
    const int per_sm = a.bn <= 64 ? 3 : 2;
    a.stages = (W8_SMEM_LIMIT / per_sm - 1024 - w8_small_smem(0, a.bn)) / w8_stage_bytes(a.bn);
    p.smem = w8_small_smem(a.stages, a.bn);
    // as many CTAs share a tile as fill the SMs once, at least four K steps each
    a.split = 1;
    while (a.split < 8 && (int64_t)a.n_mb * a.split * 2 <= (int64_t)W8_SMS * per_sm && a.n_kb / (a.split * 2) >= 4) a.split *= 2;
    p.ctas = a.n_mb * a.split;
    return p;
  }
  // The tile shape whose workers have the fewest bytes to fetch into an SM: the
  // waves of tiles times a tile's K steps, and an epilogue in plain sight at
  // the end, about as long as one byte a ns and token.
  double best = 0.0;
  for (int pair = 0; pair < 2; ++pair)
    for (int bn = 64; bn <= 256; bn += 32) {
      const int bm = pair ? 2 * W8_BM : W8_BM, rows = pair ? bn / 2 : bn, G = pair ? W8_SMS / 2 : W8_SMS;
      const double waves = (double)cdiv(cdiv(d_out, bm) * cdiv(N, bn), G);
      const double cost = waves * a.n_kb * w8_stage_bytes(rows) + W8_EPILOGUE_BYTES * bn;
      if (best == 0.0 || cost < best) {
        best = cost;
        p.pair = pair != 0;
        a.bn = bn;
      }
    }
  p.b_rows = p.pair ? a.bn / 2 : a.bn;
  a.n_mb = (int)cdiv(d_out, p.pair ? 2 * W8_BM : W8_BM);
  a.n_nb = (int)cdiv(N, a.bn);
  a.group_nb = a.n_nb < 8 ? a.n_nb : 8;
  const int st = (W8_SMEM_LIMIT - w8_smem_bytes(0, p.b_rows)) / w8_stage_bytes(p.b_rows);
  a.stages = st < W8_MAX_STAGES ? st : W8_MAX_STAGES;
  p.smem = w8_smem_bytes(a.stages, p.b_rows);
  const int64_t tiles = (int64_t)a.n_mb * a.n_nb, G = p.pair ? W8_SMS / 2 : W8_SMS;
  p.ctas = (int)(tiles < G ? tiles : G) * (p.pair ? 2 : 1);
  return p;
}

// 2-D map of bytes over a row-major [rows, cols] matrix, box of 128 columns (one swizzled row) x box_rows.
bool make_map_u8(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols};
  cuuint32_t box[2] = {W8_BK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// ------------------------------------------------------------------ 4-bit cache
awq_status check_kv4(const awq_kv4cfg* c) {
  if (!c) return AWQ_ERR_INVALID_ARG;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024) return AWQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 256) return AWQ_ERR_INVALID_ARG;
  if (c->group != 32 && c->group != 64 && c->group != 128) return AWQ_ERR_INVALID_ARG;
  if (c->head_dim % c->group != 0) return AWQ_ERR_INVALID_ARG;
  const int p = c->page_size;
  if (p < 16 || p > 256 || (p & (p - 1)) != 0) return AWQ_ERR_INVALID_ARG;
  return AWQ_OK;
}

size_t kv4_head_bytes(const awq_kv4cfg* c) {
  return (size_t)(c->page_size / KV4_STRIP) * kv4_strip_bytes(c->head_dim, c->group);
}

awq_status check_kv4_cache(const awq_kv4cfg* c, const void* cache, int64_t n_pages) {
  if (!cache || !aligned(cache, 16)) return AWQ_ERR_INVALID_ARG;
  if (n_pages < 1 || n_pages > INT32_MAX / c->page_size) return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

Kv4Cache kv4_cache(const awq_kv4cfg* c, const void* cache, int64_t n_pages) {
  Kv4Cache k{};
  k.base = static_cast<uint8_t*>(const_cast<void*>(cache));
  k.n_pages = n_pages;
  k.heads = c->n_kv_heads;
  k.dim = c->head_dim;
  k.group = c->group;
  while ((1 << k.page_shift) < c->page_size) ++k.page_shift;
  k.strip_bytes = kv4_strip_bytes(c->head_dim, c->group);
  k.head_bytes = (long long)kv4_head_bytes(c);
  return k;
}

bool strides_ok(int64_t tok, int64_t head) {
  const int64_t lim = (int64_t)1 << 40;
  return tok % 8 == 0 && head % 8 == 0 && tok >= 0 && head >= 0 && tok < lim && head < lim;
}

awq_status check_kv4_attention(int64_t batch, int64_t n_q_heads, int64_t max_q, const awq_kv4cfg* c) {
  awq_status st = check_kv4(c);
  if (st != AWQ_OK) return st;
  if (batch < 1 || batch > 65535 || n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % c->n_kv_heads != 0)
    return AWQ_ERR_SHAPE;
  if (max_q < 1 || max_q > (1 << 24) || max_q * (n_q_heads / c->n_kv_heads) > (1 << 30)) return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

// Contexts of at most this many tokens (as the page tables bound them) are not
// split between blocks, if the tables are small enough for one warp to check.
constexpr int64_t KV4_SOLO_TOKENS = 2048, KV4_SOLO_PAGES = 4096;

// The prompt kernel takes the sequences of more than KVP_MIN_ROWS rows where it
// has blocks for a good part of the SMs; else all go to the split kernel.
constexpr int64_t KVP_CTAS = 40;
bool kvp_used(int64_t batch, int64_t share, int64_t max_q, const awq_kv4cfg* c, bool f16) {
  // (fp16 with several groups a head would be rounded more than its output resolves)
  return c->head_dim <= 128 && (!f16 || c->head_dim == c->group) && max_q * share > KVP_MIN_ROWS &&
         batch * c->n_kv_heads * cdiv(max_q * share, KVP_ROWS) >= KVP_CTAS;
}

// Workspace of the attention: [0, kAlign) error word, then the block flags and
// tiles and the blocks' partial outputs.
struct Kv4Layout {
  int nt;
  size_t off_bad, off_seg, off_cta, total;
};

Kv4Layout kv4_layout(int64_t n_q_heads, int64_t max_q, const awq_kv4cfg* c) {
  Kv4Layout L{};
  const long long rows = max_q * (n_q_heads / c->n_kv_heads);
  L.nt = rows > 8 && c->head_dim <= 128 ? 2 : 1;
  const size_t part = (size_t)8 * L.nt * (c->head_dim + 4) * sizeof(float);
  size_t off = kAlign;
  L.off_bad = off;   off += align_up(KV4_CTAS * sizeof(int));
  L.off_seg = off;   off += align_up(KV4_CTAS * 2 * sizeof(long long));
  L.off_cta = off;   off += align_up(KV4_CTAS * 2 * part);
  L.total = off;
  return L;
}

// One launch per (head dimension, group); f is called with the two as constants.
template <typename F>
awq_status kv4_shapes(int dim, int group, F f) {
  auto go = [&](auto d, auto g) { return f(d, g); };
#define AWQ_KV4_SHAPE(D, G) \
  if (dim == D && group == G) return go(std::integral_constant<int, D>{}, std::integral_constant<int, G>{})
  AWQ_KV4_SHAPE(64, 32);
  AWQ_KV4_SHAPE(64, 64);
  AWQ_KV4_SHAPE(96, 32);
  AWQ_KV4_SHAPE(128, 32);
  AWQ_KV4_SHAPE(128, 64);
  AWQ_KV4_SHAPE(128, 128);
  AWQ_KV4_SHAPE(256, 32);
  AWQ_KV4_SHAPE(256, 64);
  AWQ_KV4_SHAPE(256, 128);
#undef AWQ_KV4_SHAPE
  return AWQ_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" awq_status awq_quantize_int8(const void* x, awq_dtype dtype, int64_t ldx, const float* s,
                                        awq_scale_mode mode, int64_t rows, int64_t d_in, int8_t* q, float* step,
                                        awq_stream_t stream) {
  if (!dtype_ok(dtype) || mode < AWQ_SCALE_NONE || mode > AWQ_SCALE_DIV) return AWQ_ERR_INVALID_ARG;
  if (!x || !q || !step || (mode != AWQ_SCALE_NONE && !s)) return AWQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(step, 4) || (mode != AWQ_SCALE_NONE && !aligned(s, 16)))
    return AWQ_ERR_INVALID_ARG;
  if (rows < 1 || rows > INT32_MAX / 2 || d_in < 16 || d_in % 16 != 0 || d_in > W8_MAX_K) return AWQ_ERR_SHAPE;
  if (ldx < d_in || ldx % 8 != 0) return AWQ_ERR_SHAPE;
  int sms = 0;
  awq_status st = check_device(&sms);
  if (st != AWQ_OK) return st;
  cudaStream_t cs = as_stream(stream);
  // Few rows: as many threads as a row has chunks of 8 channels, for its
  // latency. Many: up to four chunks a thread, so that several blocks fit an SM
  // and one row's reduction hides under another's loads.
  const int64_t n8 = d_in / 8;
  const int ch = rows <= 2 * sms ? (n8 <= 1024 ? 1 : 2) : n8 <= 256 ? 1 : n8 <= 512 ? 2 : 4;
  const unsigned threads = (unsigned)(cdiv(cdiv(n8, ch), 32) * 32);
  const int64_t resident = (int64_t)sms * (threads <= 64 ? 16 : threads <= 128 ? 8 : threads <= 256 ? 3 : 1);
  const unsigned grid = (unsigned)(rows < resident ? rows : resident);
  auto launch = [&](auto f16, auto m) {
    constexpr bool F = decltype(f16)::value;
    constexpr int M = decltype(m)::value;
    const void* in = x;
    // Blocks of a row each overlap the launch with the kernel before (333 rows of
    // 4096 and their product: 28.8 -> 27.3 us). Blocks that stay for several rows
    // would share the SMs with the waiting blocks of the kernels around them: 4096
    // rows, 1000 more and the product took 102 us that way, 78 without.
    auto behind = [&](auto kernel, unsigned blocks, unsigned block) {
      if (blocks == rows)
        return launch_behind(kernel, dim3(blocks), dim3(block), 0, cs, 0, in, ldx, s, rows, (int)d_in, q, step);
      kernel<<<blocks, block, 0, cs>>>(in, ldx, s, rows, (int)d_in, q, step);
      return launch_status();
    };
    if (threads > (ch == 4 ? 512u : 1024u))
      return behind(quantize_int8_long<F, M>, (unsigned)(rows < 2 * sms ? rows : 2 * sms), 1024u);
    if (ch == 1) return behind(quantize_int8_rows<F, M, 1>, grid, threads);
    if (ch == 2) return behind(quantize_int8_rows<F, M, 2>, grid, threads);
    return behind(quantize_int8_rows<F, M, 4>, grid, threads);
  };
  auto modes = [&](auto f16) {
    if (mode == AWQ_SCALE_MUL) return launch(f16, std::integral_constant<int, Q8_MUL>{});
    if (mode == AWQ_SCALE_DIV) return launch(f16, std::integral_constant<int, Q8_DIV>{});
    return launch(f16, std::integral_constant<int, Q8_PLAIN>{});
  };
  return dtype == AWQ_DTYPE_F16 ? modes(std::true_type{}) : modes(std::false_type{});
}

extern "C" awq_status awq_device_error(awq_stream_t stream) {
  cudaStream_t cs = as_stream(stream);
  int word = 0;
  if (cudaMemcpyFromSymbolAsync(&word, g_device_err, sizeof(int), 0, cudaMemcpyDeviceToHost, cs) != cudaSuccess ||
      cudaStreamSynchronize(cs) != cudaSuccess)
    return AWQ_ERR_CUDA;
  if (word == 0) return AWQ_OK;
  const int zero = 0;
  if (cudaMemcpyToSymbolAsync(g_device_err, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, cs) != cudaSuccess ||
      cudaStreamSynchronize(cs) != cudaSuccess)
    return AWQ_ERR_CUDA;
  return AWQ_ERR_DEVICE;
}

extern "C" size_t awq_w8a8_workspace_size(int64_t N, int64_t d_out, int64_t d_in) {
  if (check_w8(N, d_out, d_in) != AWQ_OK) return 0;
  return kAlign;
}

extern "C" awq_status awq_w8a8_gemm(const int8_t* xq, const float* x_step, const int8_t* wq, const float* w_step,
                                    const float* bias, awq_dtype dtype, int64_t N, int64_t d_out, int64_t d_in, void* Y,
                                    void* ws, size_t ws_bytes, awq_stream_t stream) {
  awq_status st = check_w8(N, d_out, d_in);
  if (st != AWQ_OK) return st;
  if (!dtype_ok(dtype) || !xq || !x_step || !wq || !w_step || !Y || !ws) return AWQ_ERR_INVALID_ARG;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(Y, 16) || !aligned(x_step, 4) || !aligned(w_step, 4) ||
      !aligned(bias, 4) || !aligned(ws, 256))
    return AWQ_ERR_INVALID_ARG;
  if (ws_bytes < kAlign) return AWQ_ERR_WORKSPACE;
  if ((st = check_device(nullptr)) != AWQ_OK) return st;
  W8Plan p = w8_plan(N, d_out, d_in);
  cudaStream_t cs = as_stream(stream);
  W8Args& a = p.a;
  a.dx = x_step;
  a.dw = w_step;
  a.bias = bias;
  a.Y = Y;
  a.err = at<int>(ws, 0);
  CUtensorMap tw, tx;
  if (!make_map_u8(&tw, wq, d_out, d_in, W8_BM) || !make_map_u8(&tx, xq, N, d_in, p.b_rows)) return AWQ_ERR_CUDA;
  const bool f16 = dtype == AWQ_DTYPE_F16;
  static std::atomic<unsigned long long> once[6];
  if (p.small) {
    auto launch = [&](auto kernel) -> awq_status {
      if (!kernel_smem(kernel, W8_SMEM_LIMIT / 2, once[f16 ? 1 : 0])) return AWQ_ERR_CUDA;
      return launch_behind(kernel, dim3((unsigned)p.ctas), dim3(W8_SMALL_THREADS), p.smem, cs, (unsigned)a.split, tw, tx, a);
    };
    return f16 ? launch(w8a8_small_tcgen05<true>) : launch(w8a8_small_tcgen05<false>);
  }
  auto launch = [&](auto kernel) -> awq_status {
    if (!kernel_smem(kernel, W8_SMEM_LIMIT, once[(p.pair ? 4 : 2) + (f16 ? 1 : 0)])) return AWQ_ERR_CUDA;
    return launch_behind(kernel, dim3((unsigned)p.ctas), dim3(W8_THREADS), p.smem, cs, 0, tw, tx, a);
  };
  return p.pair ? (f16 ? launch(w8a8_gemm_pair_tcgen05<true>) : launch(w8a8_gemm_pair_tcgen05<false>))
                : (f16 ? launch(w8a8_gemm_tcgen05<true>) : launch(w8a8_gemm_tcgen05<false>));
}

extern "C" size_t awq_kv4_page_bytes(const awq_kv4cfg* cfg) {
  return check_kv4(cfg) == AWQ_OK ? kv4_head_bytes(cfg) : 0;
}

extern "C" awq_status awq_kv4_append(const void* k, const void* v, awq_dtype dtype, int64_t T, int64_t k_tok,
                                     int64_t k_head, int64_t v_tok, int64_t v_head, const int32_t* slots, void* cache,
                                     int64_t n_pages, const awq_kv4cfg* cfg, awq_stream_t stream) {
  awq_status st = check_kv4(cfg);
  if (st != AWQ_OK) return st;
  if (T < 0 || T > (1 << 28)) return AWQ_ERR_SHAPE;
  if ((st = check_kv4_cache(cfg, cache, n_pages)) != AWQ_OK) return st;
  if (!dtype_ok(dtype) || !strides_ok(k_tok, k_head) || !strides_ok(v_tok, v_head)) return AWQ_ERR_INVALID_ARG;
  if (T == 0) return AWQ_OK;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return AWQ_ERR_INVALID_ARG;
  if ((st = check_device(nullptr)) != AWQ_OK) return st;
  Kv4AppendArgs a{};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_tok = k_tok;
  a.k_head = k_head;
  a.v_tok = v_tok;
  a.v_head = v_head;
  a.slots = slots;
  a.T = (int)T;
  a.c = kv4_cache(cfg, cache, n_pages);
  const int span = kv4_span(T);
  const unsigned blocks = (unsigned)((T + span - 1) / span);
  auto kernel = dtype == AWQ_DTYPE_F16 ? kv4_append_kernel<true> : kv4_append_kernel<false>;
  return launch_behind(kernel, dim3(blocks), dim3(32 * KV4_APPEND_WARPS), 0, as_stream(stream), 0, a, span);
}

extern "C" awq_status awq_kv4_gather(const void* cache, int64_t n_pages, const int32_t* slots, int64_t T,
                                     const awq_kv4cfg* cfg, void* k, void* v, awq_dtype dtype, awq_stream_t stream) {
  awq_status st = check_kv4(cfg);
  if (st != AWQ_OK) return st;
  if (T < 0 || T > (1 << 28)) return AWQ_ERR_SHAPE;
  if ((st = check_kv4_cache(cfg, cache, n_pages)) != AWQ_OK) return st;
  if (!dtype_ok(dtype)) return AWQ_ERR_INVALID_ARG;
  if (T == 0 || (!k && !v)) return AWQ_OK;
  if (!slots || !aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16)) return AWQ_ERR_INVALID_ARG;
  if ((st = check_device(nullptr)) != AWQ_OK) return st;
  const Kv4Cache c = kv4_cache(cfg, cache, n_pages);
  const int span = kv4_span(T);
  const unsigned blocks = (unsigned)((T + span - 1) / span);
  auto kernel = dtype == AWQ_DTYPE_F16 ? kv4_gather_kernel<true> : kv4_gather_kernel<false>;
  return launch_behind(kernel, dim3(blocks), dim3(32 * KV4_APPEND_WARPS), 0, as_stream(stream), 0, c, slots, (int)T, k, v, span);
}

extern "C" size_t awq_kv4_attention_workspace_size(int64_t batch, int64_t n_q_heads, int64_t max_q,
                                                   const awq_kv4cfg* cfg) {
  if (check_kv4_attention(batch, n_q_heads, max_q, cfg) != AWQ_OK) return 0;
  return kv4_layout(n_q_heads, max_q, cfg).total;
}

extern "C" awq_status awq_kv4_attention(const void* q, awq_dtype dtype, int64_t q_tok, int64_t q_head, int64_t T,
                                        int64_t n_q_heads, const int32_t* q_start, int64_t max_q, const void* cache,
                                        int64_t n_pages, const int32_t* table, int64_t table_pages, const int32_t* lens,
                                        int64_t batch, float scale, const awq_kv4cfg* cfg, void* out, float* lse,
                                        void* ws, size_t ws_bytes, awq_stream_t stream) {
  awq_status st = check_kv4_attention(batch, n_q_heads, max_q, cfg);
  if (st != AWQ_OK) return st;
  if ((st = check_kv4_cache(cfg, cache, n_pages)) != AWQ_OK) return st;
  // (the kernels' token indices run on to the end of a tile of 64 and its neighbour in 32 bits)
  if (T < 0 || T > (1 << 28) || table_pages < 1 || table_pages > (INT32_MAX - 128) / cfg->page_size)
    return AWQ_ERR_SHAPE;
  if (!q_start && (T < batch || max_q != 1)) return AWQ_ERR_SHAPE;
  if (!dtype_ok(dtype) || !strides_ok(q_tok, q_head) || !std::isfinite(scale)) return AWQ_ERR_INVALID_ARG;
  if (!q || !table || !lens || !out || !ws) return AWQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_start, 4) ||
      !aligned(lse, 4) || !aligned(ws, 256))
    return AWQ_ERR_INVALID_ARG;
  const Kv4Layout L = kv4_layout(n_q_heads, max_q, cfg);
  if (ws_bytes < L.total) return AWQ_ERR_WORKSPACE;
  if ((st = check_device(nullptr)) != AWQ_OK) return st;
  cudaStream_t cs = as_stream(stream);
  Kv4AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_tok = q_tok;
  a.q_head = q_head;
  a.T = T;
  a.q_heads = (int)n_q_heads;
  a.share = (int)(n_q_heads / cfg->n_kv_heads);
  a.q_start = q_start;
  a.max_q = (int)max_q;
  a.table = table;
  a.table_pages = (int)table_pages;
  a.lens = lens;
  a.batch = (int)batch;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.f16 = dtype == AWQ_DTYPE_F16;
  a.c = kv4_cache(cfg, cache, n_pages);
  a.out = out;
  a.lse = lse;
  a.err = at<int>(ws, 0);
  const bool prompt = kvp_used(batch, a.share, max_q, cfg, a.f16);
  Kv4SplitArgs sa{};
  sa.tile_rows = 8 * L.nt;
  sa.max_rows = prompt ? KVP_MIN_ROWS : INT32_MAX;
  sa.cta_part = at<float>(ws, L.off_cta);
  sa.cta_seg = at<long long>(ws, L.off_seg);
  sa.cta_bad = at<int>(ws, L.off_bad);
  for (int64_t first = 0; first < batch; first += KV4_MAX_BATCH) {
    sa.a = a;
    sa.a.batch = (int)(batch - first < KV4_MAX_BATCH ? batch - first : KV4_MAX_BATCH);
    sa.a.table += first * table_pages;
    sa.a.lens += first;
    if (q_start) sa.a.q_start += first;
    sa.a.row_first = (int)first;
    sa.clear_err = first == 0;
    sa.solo = table_pages * cfg->page_size <= KV4_SOLO_TOKENS && sa.a.batch * table_pages <= KV4_SOLO_PAGES;
    st = kv4_shapes(cfg->head_dim, cfg->group, [&](auto d, auto g) -> awq_status {
      constexpr int D = decltype(d)::value, G = decltype(g)::value;
      auto launch = [&](auto nt) -> awq_status {
        constexpr int NT = decltype(nt)::value;
        constexpr int smem = (int)sizeof(Kv4SplitSmem<D, G, NT>) + 128;
        static_assert(smem <= 232448, "shared memory of the split attention");
        auto k = kv4_attention_split<D, G, NT>;
        auto j = kv4_attention_join<D, NT>;
        static std::atomic<unsigned long long> once_k{0}, once_j{0};
        if (!kernel_smem(k, smem, once_k) || !kernel_smem(j, 0, once_j)) return AWQ_ERR_CUDA;
        st = launch_behind(k, dim3(KV4_CTAS), dim3(32 * (kv4_warps(D, G, NT) + 1)), smem, cs, 0, sa);
        if (st != AWQ_OK || sa.solo) return st;
        return launch_behind(j, dim3(KV4_CTAS), dim3(32 * KV4_JOIN_WARPS), 0, cs, 0, sa, KV4_CTAS);
      };
      return L.nt == 2 ? launch(std::integral_constant<int, D <= 128 ? 2 : 1>{}) : launch(std::integral_constant<int, 1>{});
    });
    if (st != AWQ_OK) return st;
  }
  if (!prompt) return AWQ_OK;
  const dim3 grid((unsigned)cdiv(max_q * a.share, KVP_ROWS), (unsigned)cfg->n_kv_heads, (unsigned)batch);
  return kv4_shapes(cfg->head_dim, cfg->group, [&](auto d, auto g) -> awq_status {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    if constexpr (D <= 128) {
      constexpr int smem = (int)sizeof(KvpSmem<D, G>) + 1024;
      static_assert(smem <= 232448, "shared memory of the prompt attention");
      auto launch = [&](auto k, std::atomic<unsigned long long>& once) -> awq_status {
        if (!kernel_smem(k, smem, once)) return AWQ_ERR_CUDA;
        return launch_behind(k, grid, dim3(KVP_THREADS), smem, cs, 0, a);
      };
      static std::atomic<unsigned long long> once[2];
      if constexpr (D == G)
        if (a.f16) return launch(kv4_attention_prompt<D, G, true>, once[1]);
      return launch(kv4_attention_prompt<D, G, false>, once[0]);
    }
    return AWQ_ERR_UNSUPPORTED;  // (kvp_used keeps them with the split kernel)
  });
}
