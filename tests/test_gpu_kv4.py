"""The 4-bit key/value cache on the GPU: written and read back byte for byte
against the oracle, and the attention over it against the float64 softmax on
the same codes.

Tolerance of the attention, for a row with visible tokens t, weights p_t (sum
1), values v_t = (c_t - z_t) D_t (oracle, float64), u the output type's half
step, n the number of visible tokens:
- a score is a sum of head_dim + D/g products (codes times fp16 queries, exact)
  in fp32 and a few fp32 operations; with tensor-core accumulation taken as 2^-22
  an operation its error is at most ds_t = (head_dim + 16) 2^-22 * scale * sum_i
  |q_i| Dk (c_i + z) (the products before the zero is taken off, so c + z, not
  |c - z|), and the base-2 exponent adds (|s_t| + |max s| + 40) 2^-22: a relative
  error e_t = 1.01 (ds_t + (|s_t| + |smax| + 40) 2^-22) + 2^-20 of p_t (the last
  for the exponential itself, a few units);
- the query is held in fp16 scaled by a power of two: exact for both types up to
  entries 2^-21 below the row's largest, so 2^-30 |q|max a channel: in ds_t;
- the weight p_t D_t is rounded to fp16: 2^-11 relative, and half the smallest
  subnormal where it is tiny; the largest weight is at least 1 in the kernel's
  units, so that is at most 2^-25 max_t(p_t D_t) a token;
- numerator and denominator are fp32 sums: (n/8 + 64) 2^-22 of the terms' sizes.
So |O - O_ref| <= u |O| + sum_t p_t (e_t + 2^-11) (c_t + z_t) D_t + sum_t p_t e_t |O|
  + 2^-25 max(p D) sum_t (c_t + z_t) + (n/8 + 64) 2^-22 (sum_t p_t (c_t + z_t) D_t + |O|), times 1.1.
- The kernel for prompts holds values, and for bf16 also keys, as (code - zero) step in fp16, rounded once: 2^-11 |v| a
  value, so sum_t p_t 2^-11 |v_t| more, and 2^-11 scale sum_i |q_i| |k_ti| more in ds_t. (Steps far below the strip's
  largest: half of fp16's smallest subnormal, 2^-25, of 2^10 over it: 2^-35 of the largest, below the terms above.)"""
import zlib

import numpy as np
import pytest

from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import weight_only_int4_act_b200 as awq  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SHAPES = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def _f64(t):
    return t.double().cpu().numpy()


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def _bytes(cache):
    return cache.cpu().numpy().view(np.uint8)


# ---------------------------------------------------------------- write and read back
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", SHAPES)
def test_append_byte_for_byte(dim, group, dtype):
    """Tokens in scattered order, some skipped, into a cache that holds other bytes: exactly their own bytes change."""
    heads, page, pages, T = 3, 32, 5, 41
    cfg = awq.make_kv4(heads, dim, page, group)
    cache = awq.kv4_new_cache(pages, cfg)
    cache.random_(-2 ** 31, 2 ** 31 - 1, generator=torch.Generator(device="cuda").manual_seed(2))
    want = _bytes(cache).copy()
    fused = _rand((T, 3 * heads, dim), dtype, dim + group, 3.0)
    k, v = fused[:, heads:2 * heads], fused[:, 2 * heads:]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:T].int()
    slots[5], slots[6], slots[7] = -1, pages * page, 2 ** 31 - 1
    awq.kv4_append(k, v, slots.cuda(), cache, cfg)
    for kind, x in ((0, k), (1, v)):
        code, step, zero = S.four_bit(_f64(x), group)
        for t in range(T):
            if 0 <= slots[t] < pages * page:
                for h in range(heads):
                    S.write_token(want, int(slots[t]), h, page, dim, group, kind, code[t, h], step[t, h], zero[t, h])
    assert np.array_equal(_bytes(cache), want)
    back = awq.kv4_gather(cache, slots.cuda(), cfg, dtype=DT[dtype])
    for x, y in ((k, back[0]), (v, back[1])):
        ref = torch.from_numpy(S.four_bit_values(*S.four_bit(_f64(x), group))).to(DT[dtype])
        out = (slots < 0) | (slots >= pages * page)
        ref[out] = 0
        assert torch.equal(y.cpu(), ref)


def _awkward(x, seed):
    """Some groups' worth of x replaced by infinities, NaN, zeros, the least and the largest values."""
    g = torch.Generator().manual_seed(seed)
    flat, f = x.view(-1), torch.finfo(x.dtype)
    for v in (float("inf"), -float("inf"), float("nan"), 0.0, -0.0, f.max, f.min, f.tiny, f.tiny * f.eps, -f.tiny):
        at = torch.randint(0, flat.numel(), (3,), generator=g)
        flat[at.cuda()] = v
    x[0], x[-1, :, ::2] = 0, -0.0
    return x


def _runs(T, page, pages, seed):
    """T slots: runs of following tokens that begin and end anywhere, some backwards, some outside the cache."""
    r = np.random.default_rng(seed)
    at, out = list(r.permutation(pages * page // 64) * 64), []
    while len(out) < T:
        base, skip, n = int(at.pop()), int(r.integers(0, 20)), int(r.integers(1, 45))
        run = np.arange(base + skip, base + skip + n)
        kind = r.integers(0, 8)
        if kind == 0:
            run = run[::-1]
        elif kind == 1:
            run = run + pages * page * 3
        elif kind == 2:
            run = run - 64 * (pages * page // 64 + 2)
        elif kind == 3:
            run = run[:1]
        out += list(run)
    return np.array(out[:T], dtype=np.int32)


@pytest.mark.parametrize("T,dim,group,page,dtype", [(500, 64, 32, 16, "bf16"), (1024, 128, 128, 64, "f16"),
                                                    (1025, 96, 32, 32, "bf16"), (1300, 128, 32, 16, "f16"),
                                                    (1100, 256, 64, 256, "bf16"), (1040, 64, 64, 128, "f16")])
def test_append_runs_of_tokens(T, dim, group, page, dtype):
    """Runs of following slots (whole strips are taken together), broken, reversed and partly outside; awkward values."""
    heads, pages = 3, 12800 // page
    cfg = awq.make_kv4(heads, dim, page, group)
    cache = awq.kv4_new_cache(pages, cfg)
    cache.random_(-2 ** 31, 2 ** 31 - 1, generator=torch.Generator(device="cuda").manual_seed(2))
    want = _bytes(cache).copy()
    k, v = (_awkward(_rand((T, heads + 1, dim), dtype, T + i, 3.0), i)[:, 1:] for i in (0, 1))
    slots = _runs(T, page, pages, T)
    awq.kv4_append(k, v, torch.from_numpy(slots).cuda(), cache, cfg)
    for kind, x in ((0, k), (1, v)):
        code, step, zero = S.four_bit(_f64(x), group)
        for t in range(T):
            if 0 <= slots[t] < pages * page:
                for h in range(heads):
                    S.write_token(want, int(slots[t]), h, page, dim, group, kind, code[t, h], step[t, h], zero[t, h])
    assert np.array_equal(_bytes(cache), want)
    back = awq.kv4_gather(cache, torch.from_numpy(slots).cuda(), cfg, dtype=DT[dtype])
    out = torch.from_numpy((slots < 0) | (slots >= pages * page))
    for x, y in ((k, back[0]), (v, back[1])):
        ref = torch.from_numpy(S.four_bit_values(*S.four_bit(_f64(x), group))).to(DT[dtype])
        ref[out] = 0
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=-77.0), torch.nan_to_num(ref, nan=-77.0))


def _fill(lens, heads, dim, group, page, dtype, seed, kscale=1.0, vscale=1.0, spare=2, scale_k=None):
    """A cache with shuffled pages: (cfg, cache, table, lens, k, v as written)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).int()
    table = torch.full((len(lens), max(max(need), 1)), -7, dtype=torch.int32)  # never read beyond a context
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cfg = awq.make_kv4(heads, dim, page, group)
    cache = awq.kv4_new_cache(total, cfg)
    cache.fill_(-1)  # stale bytes: codes 15, steps and zeros NaN
    slots = [int(table[b, i // page]) * page + i % page for b, n in enumerate(lens) for i in range(n)]
    T = len(slots)
    k = _rand((T, heads, dim), dtype, seed + 1, kscale)
    v = _rand((T, heads, dim), dtype, seed + 2, vscale)
    if scale_k is not None:
        k = (k.float() * scale_k).to(DT[dtype])
    if T:
        awq.kv4_append(k, v, torch.tensor(slots, dtype=torch.int32).cuda(), cache, cfg)
    return cfg, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), np.array(slots, dtype=np.int64)


def _read(cache, cfg, slots):
    """float64 (code, step, zero) per kind of the slots: [T, H, D], [T, H, D/g] twice."""
    page = cfg.page_size
    out = []
    for code, step, zero in S.unpack_pages(_bytes(cache), cfg.head_dim, cfg.group):
        at = (slots // page, slice(None), slots % page)
        out.append(tuple(a[at].astype(np.float64) for a in (code, step, zero)))
    return out


def _check(out, lse, q, cfg, parts, lens, starts, share, scale, dtype, prompt=False):
    """Every row of every sequence against the oracle; parts: _read() of all tokens in order; prompt: the prompts' kernel
    may have run."""
    rk, rv = (2.0 ** -11 if dtype == "bf16" else 0.0, 2.0 ** -11) if prompt else (0.0, 0.0)
    g, D = cfg.group, cfg.head_dim
    rep = lambda a: np.repeat(a, g, axis=-1)  # noqa: E731
    (kc, ks, kz), (vc, vs, vz) = parts
    got, qq = _f64(out), _f64(q)
    at = 0
    for b, L in enumerate(lens):
        sl = slice(at, at + L)
        at += L
        r0, r1 = starts[b], starts[b + 1]
        n = r1 - r0
        if n == 0:
            continue
        k = (kc[sl] - rep(kz[sl])) * rep(ks[sl])
        v = (vc[sl] - rep(vz[sl])) * rep(vs[sl])
        ref, ref_lse, p = S.attention(qq[r0:r1], k, v, share, scale, L - n + 1)
        ksize, vsize = (kc[sl] + rep(kz[sl])) * rep(ks[sl]), (vc[sl] + rep(vz[sl])) * rep(vs[sl])
        for e in range(qq.shape[1]):
            h = e // share
            q_e = qq[r0:r1, e]
            s = scale * q_e @ k[:, h].T
            qa = np.abs(q_e) + 2.0 ** -8 * np.abs(q_e).max(axis=1, keepdims=True)  # 2^-8 * 2^-22: the fp16 query
            ds = (D + 16) * 2.0 ** -22 * scale * qa @ ksize[:, h].T + rk * scale * qa @ np.abs(k[:, h]).T
            vis = p[:, e] > 0
            smax = np.where(vis, np.abs(s), 0).max(axis=1, keepdims=True) if L else np.zeros((n, 1))
            err = np.where(p[:, e] > 0, 1.01 * (ds + (np.abs(s) + smax + 40) * 2.0 ** -22) + 2.0 ** -20, 0)
            pe = p[:, e]
            seen = vis.sum(axis=1, keepdims=True)
            pd = (pe[:, :, None] * vs[sl][:, h].max(axis=-1)[None, :, None]).max(axis=1) if L else np.zeros((n, 1))
            size = pe @ vsize[:, h]
            o = np.abs(ref[:, e])
            codes = vis.astype(np.float64) @ (vc[sl] + rep(vz[sl]))[:, h]
            tol = 1.1 * (UNIT[dtype] * o + (pe * (err + 2.0 ** -11)) @ vsize[:, h] + (pe * err).sum(1, keepdims=True) * o
                         + rv * pe @ np.abs(v[:, h])                         + 2.0 ** -25 * pd * codes + (seen / 8 + 64) * 2.0 ** -22 * (size + o)) + 2.0 ** -25
            d = np.abs(got[r0:r1, e] - ref[:, e])
            bad = ~(d <= tol)
            assert not bad.any(), (b, e, np.argwhere(bad)[:4], d[bad][:4], tol[bad][:4])
            if lse is not None:
                w = _f64(lse)[r0:r1, e]
                empty = ~vis.any(axis=1)
                assert np.array_equal(np.isneginf(w), empty)
                lt = err.max(axis=1, initial=0) + (np.abs(ref_lse[:, e]) + seen[:, 0] / 8 + 64) * 2.0 ** -22
                assert (np.abs(w[~empty] - ref_lse[~empty, e]) <= 1.1 * lt[~empty]).all()


def _run(lens, new, heads, share, dim, group, page, dtype, seed, lse=True, prompt=False, **kw):
    """Build, attend (q a strided slice, output and workspace given), check. new: rows of each sequence."""
    cfg, cache, table, lens_t, slots = _fill(lens, heads, dim, group, page, dtype, seed, **kw)
    starts = np.concatenate([[0], np.cumsum(new)])
    T = int(starts[-1])
    q = _rand((T + 3, heads * share + 2, dim), dtype, seed + 5, 2.0)[:T, 1:-1]
    work = awq.workspace(awq.kv4_attention_workspace_size(len(lens), heads * share, max(max(new), 1), cfg))
    work.fill_(0xA5)
    buf = torch.full((T + 2, heads * share, dim), 9.0, dtype=DT[dtype], device="cuda")
    args = dict(q_start=torch.tensor(starts, dtype=torch.int32).cuda(), max_q=max(max(new), 1))
    r = awq.kv4_attention(q, cache, table, lens_t, cfg, lse=lse, ws=work, out=buf[1:T + 1], **args)
    awq.workspace_error(work)
    out, l = r if lse else (r, None)
    assert (buf[0] == 9).all() and (buf[-1] == 9).all()
    _check(out, l, q, cfg, _read(cache, cfg, slots), lens, starts, share, dim ** -0.5, dtype, prompt)
    again = awq.kv4_attention(q, cache, table, lens_t, cfg, ws=work, **args)
    rows = np.concatenate([np.arange(a, b) for a, b in zip(starts[:-1], starts[1:])]) if T else []
    assert torch.equal(again[rows], out[rows])  # the same bits on every call
    return cfg, cache, table, lens_t, q, out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", SHAPES)
def test_attention_shapes(dim, group, dtype):
    _run([130, 1, 47, 0, 16, 15, 17, 300], [1] * 8, 2, 3, dim, group, 32, dtype, dim + group)


@pytest.mark.parametrize("share", [1, 2, 5, 8, 12, 16, 17, 33, 71])
def test_attention_shared_heads(share):
    _run([97, 200], [1, 1], 2, share, 64, 64, 16, "f16", share)


@pytest.mark.parametrize("page", [16, 64, 128, 256])
def test_attention_pages(page):
    _run([page, page - 1, page + 1, 5 * page + 3, 1], [1] * 5, 2, 4, 128, 128, page, "bf16", page)


@pytest.mark.parametrize("new,share", [([1, 2, 0, 3], 4), ([5, 5, 5, 5], 3), ([8, 1, 8, 1], 8), ([40, 3, 17, 64], 2),
                                       ([130, 1, 0, 257], 1)])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
def test_attention_several_queries(new, share, dim, group):
    """Causal at the end of the context: ragged rows, sequences without rows, more rows than context (rows that see nothing)."""
    lens = [300, 33, 64, 2 if new[3] > 2 else 70]
    if new[3] == 257:
        lens[3] = 255  # the first two rows see nothing
    _run(lens, new, 2, share, dim, group, 32, "bf16" if share % 2 else "f16", 11 + sum(new))


@pytest.mark.parametrize("lens", [[4096], [1], [16], [5000, 3], [777] * 7, [1] * 300, [33] * 200, [20000, 1, 64, 9000]])
def test_attention_lengths(lens):
    """One long context, many tiny ones, and mixtures: the split over the GPU joins what it cuts."""
    _run(lens, [1] * len(lens), 2, 4, 128, 128, 64, "bf16", len(lens), lse=len(lens) < 10)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_prompt_chunk(dtype):
    """A chunk long enough for tiles of queries, behind an older context, and a whole prompt."""
    _run([700, 260], [300, 260], 2, 4, 128, 128, 64, dtype, 77)


# the batches below give enough blocks of 256 query rows for the tensor-memory kernel (head_dim <= 128; fp16: one group a head)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_prompt_pages_and_mixed_rows(dim, page, dtype):
    """Chunks behind older contexts, a whole prompt, single tokens and a sequence without rows in one batch."""
    _run([700, 260, 90, 333, 64, 129, 40], [300, 260, 1, 70, 0, 129, 3], 8, 2, dim, dim, page, dtype, 7 * page + dim, prompt=True)


@pytest.mark.parametrize("share,heads,new", [(1, 16, 700), (3, 7, 201), (8, 5, 260), (16, 40, 5), (71, 10, 15)])
def test_prompt_shared_heads(share, heads, new):
    """Row tiles that cut a token's heads anywhere; few and many rows a token."""
    _run([new + 77, new], [new, new], heads, share, 64, 64, 64, "bf16", share, prompt=True)


@pytest.mark.parametrize("dim,group", [(64, 32), (96, 32), (128, 32), (128, 64)])
def test_prompt_groups(dim, group):
    """Several groups a head, of very different sizes; fp16 stays with the exact kernel."""
    _run([400, 333], [300, 290], 8, 3, dim, group, 32, "bf16", dim + group, prompt=True)
    loud = torch.exp(torch.arange(dim, device="cuda") // group * 2.0)
    _run([400, 333], [300, 290], 8, 3, dim, group, 32, "bf16", dim + group, prompt=True, scale_k=loud.reciprocal())
    _run([200, 133], [100, 90], 8, 3, dim, group, 32, "f16", dim + group)


def test_prompt_more_rows_than_context():
    """Rows that see nothing: zeros and -inf."""
    _run([100, 40, 0], [300, 129, 70], 16, 2, 128, 128, 16, "f16", 3, prompt=True)


def test_prompt_large_values_and_steps():
    loud = torch.ones(128, device="cuda")
    loud[3], loud[77] = 40.0, 25.0
    _run([500, 390], [300, 290], 10, 4, 128, 128, 32, "bf16", 5, prompt=True, kscale=2.0, vscale=100.0, scale_k=loud)
    _run([500, 390], [300, 290], 10, 4, 128, 128, 32, "f16", 6, prompt=True, kscale=0.01, vscale=1e-3)


def test_prompt_long_context():
    _run([6000, 5001], [260, 130], 10, 2, 128, 128, 64, "bf16", 8, lse=False, prompt=True)


def test_prompt_masked_tokens_may_hold_anything():
    """NaN in a token does not reach the rows before it, does reach all from it on."""
    heads, n = 20, 300
    cfg, cache, table, lens, slots = _fill([400, 350], heads, 128, 128, 32, "bf16", 60)
    q = _rand((2 * n, 2 * heads, 128), "bf16", 61)
    start = torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda()
    good = awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=n)
    bad = torch.full((1, heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    awq.kv4_append(bad, bad, torch.tensor([slots[290]], dtype=torch.int32).cuda(), cache, cfg)
    out = awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=n)
    first = 290 - (400 - n)  # the first row that sees token 290
    assert torch.equal(out[:first], good[:first]) and torch.equal(out[n:], good[n:])
    assert torch.isnan(out[first:n]).all()
    work = awq.workspace(awq.kv4_attention_workspace_size(2, 2 * heads, n, cfg))
    table[1, 3] = cache.shape[0]  # a page outside the cache: left out of the second sequence, and reported
    out, lse = awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=n, ws=work, lse=True)
    with pytest.raises(awq.AwqError, match="DEVICE"):
        awq.workspace_error(work)
    assert torch.equal(out[:first], good[:first])
    assert torch.equal(out[n:n + 96 - 50], good[n:n + 96 - 50])  # rows that see only the first three pages
    keep = np.concatenate([slots[400:400 + 96], slots[400 + 128:]])
    (kc, ks, kz), (vc, vs, vz) = _read(cache, cfg, keep)
    k, v = S.four_bit_values(kc, ks, kz), S.four_bit_values(vc, vs, vz)
    ref, ref_lse, _ = S.attention(_f64(q[2 * n - 1:]), k, v, 2, 128 ** -0.5, 318)
    assert np.abs(_f64(out[2 * n - 1:]) - ref).max() <= 2.0 ** -7 * np.abs(v).max()
    assert np.abs(_f64(lse[2 * n - 1:]) - ref_lse).max() <= 2.0 ** -10


@pytest.mark.parametrize("n", [1, 150])
def test_scale_zero_and_negative(n):
    """scale 0: the mean of the visible values; scale below 0: the softmax turned round."""
    cfg, cache, table, lens, slots = _fill([200, 170], 20, 64, 64, 16, "f16", 33)
    q = _rand((2 * n, 40, 64), "f16", 34, 2.0)
    start = torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda()
    parts = _read(cache, cfg, slots)
    for scale in (0.0, -0.2):
        out, lse = awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=n, scale=scale, lse=True)
        _check(out, lse, q if scale >= 0 else -q, cfg, parts, [200, 170], [0, n, 2 * n], 2, abs(scale), "f16", n > 1)


def test_attention_large_values_and_steps():
    """Peaked softmax, values of very different sizes, loud key channels, large queries."""
    loud = torch.ones(128, device="cuda")
    loud[3], loud[77] = 40.0, 25.0
    _run([500, 90], [1, 4], 2, 4, 128, 32, 32, "bf16", 5, kscale=2.0, vscale=100.0, scale_k=loud)
    _run([500, 90], [1, 4], 2, 4, 128, 128, 32, "f16", 6, kscale=0.01, vscale=1e-3)


def test_attention_first_value_huge_and_unlikely():
    """A token with a value step 2^14 times the others' whose probability is about nothing, before and after the likely ones."""
    for where in (0, 40, 79):
        cfg, cache, table, lens, slots = _fill([80], 1, 64, 64, 16, "f16", 50)
        k = torch.full((1, 1, 64), -4.0, dtype=torch.float16, device="cuda")
        v = _rand((1, 1, 64), "f16", 51, 16384.0)
        awq.kv4_append(k, v, torch.tensor([slots[where]], dtype=torch.int32).cuda(), cache, cfg)
        q = torch.full((1, 2, 64), 1.5, dtype=torch.float16, device="cuda")
        out, lse = awq.kv4_attention(q, cache, table, lens, cfg, lse=True)
        _check(out, lse, q, cfg, _read(cache, cfg, slots), [80], [0, 1], 2, 64 ** -0.5, "f16")


def test_masked_tokens_may_hold_anything():
    """NaN in tokens that a row does not see (later ones, and stale bytes behind the context) does not reach it; in one that it sees it does."""
    cfg, cache, table, lens, slots = _fill([50], 2, 128, 64, 32, "bf16", 60)
    q = _rand((4, 4, 128), "bf16", 61)
    start = torch.tensor([0, 4], dtype=torch.int32).cuda()
    good = awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=4)
    bad = torch.full((1, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    awq.kv4_append(bad, bad, torch.tensor([slots[48]], dtype=torch.int32).cuda(), cache, cfg)
    out, lse = awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=4, lse=True)
    assert torch.equal(out[:2], good[:2]) and torch.isfinite(lse[:2]).all()
    assert torch.isnan(out[2:]).all()
    k, v = awq.kv4_gather(cache, torch.tensor([slots[48]], dtype=torch.int32).cuda(), cfg)
    assert torch.isnan(k).all() and torch.isnan(v).all()


def test_bad_pages_lengths_and_rows_are_reported():
    """Pages outside the cache are left out, lengths are cut to the table, rows to max_q: all reported, nothing else read or written."""
    cfg, cache, table, lens, slots = _fill([96, 40], 2, 64, 64, 32, "f16", 70)
    q = _rand((2, 4, 64), "f16", 71)
    work = awq.workspace(awq.kv4_attention_workspace_size(2, 4, 1, cfg))
    for wrong in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = wrong
        out, lse = awq.kv4_attention(q, cache, t, lens, cfg, ws=work, lse=True)
        with pytest.raises(awq.AwqError, match="DEVICE"):
            awq.workspace_error(work)
        awq.workspace_error(work)  # reading cleared it
        keep = np.concatenate([slots[:32], slots[64:]])
        _check(out, lse, q, cfg, _read(cache, cfg, keep), [64, 40], [0, 1, 2], 2, 64 ** -0.5, "f16")
    for n in (-5, 97, 2 ** 31 - 1):
        out = awq.kv4_attention(q, cache, table, torch.tensor([n, 40], dtype=torch.int32).cuda(), cfg, ws=work)
        with pytest.raises(awq.AwqError, match="DEVICE"):
            awq.workspace_error(work)
        if n < 0:
            assert not out[0].any()
        else:
            assert torch.equal(out, awq.kv4_attention(q, cache, table, lens, cfg))
    for start in ([0, 2, 2], [0, -1, 2], [0, 5, 9], [1, 0, 2]):
        out = torch.full((2, 4, 64), 3.0, dtype=torch.float16, device="cuda")
        awq.kv4_attention(q, cache, table, lens, cfg, q_start=torch.tensor(start, dtype=torch.int32).cuda(), max_q=1,
                          ws=work, out=out)
        with pytest.raises(awq.AwqError, match="DEVICE"):
            awq.workspace_error(work)


def test_rows_behind_the_last_sequence_stay():
    cfg, cache, table, lens, slots = _fill([40, 20], 2, 64, 32, 16, "bf16", 80)
    q = _rand((9, 4, 64), "bf16", 81)
    out = torch.full((9, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([1, 3, 6], dtype=torch.int32).cuda()
    awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=3, out=out)
    assert (out[0] == 5).all() and (out[6:] == 5).all()
    _check(out, None, q, cfg, _read(cache, cfg, slots), [40, 20], [1, 3, 6], 2, 64 ** -0.5, "bf16")


def test_token_strides_of_one_row_and_no_tokens():
    cfg = awq.make_kv4(2, 64, 16, 64)
    cache = awq.kv4_new_cache(2, cfg)
    before = cache.clone()
    none = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    awq.kv4_append(none, none, empty, cache, cfg)
    k, v = awq.kv4_gather(cache, empty, cfg)
    assert k.shape == (0, 2, 64) and torch.equal(cache, before)


def test_python_refusals():
    cfg, cache, table, lens, slots = _fill([40, 20], 2, 64, 32, 16, "bf16", 90)
    q = _rand((2, 4, 64), "bf16", 91)
    with pytest.raises(ValueError, match="cache must be"):
        awq.kv4_attention(q, cache[:, :, :-1].contiguous(), table, lens, cfg)
    with pytest.raises(ValueError, match="q must have shape"):
        awq.kv4_attention(q[..., :32], cache, table, lens, cfg)
    with pytest.raises(ValueError, match="one row a sequence"):
        awq.kv4_attention(q[:1], cache, table, lens, cfg)
    with pytest.raises(ValueError, match="max_q"):
        awq.kv4_attention(q, cache, table, lens, cfg, q_start=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(awq.AwqError, match="SHAPE"):
        awq.kv4_attention(q[:, :3], cache, table, lens, cfg)  # 3 query heads over 2
    with pytest.raises(ValueError, match="int32"):
        awq.kv4_append(q[:, :2], q[:, 2:], torch.zeros(2, dtype=torch.int64, device="cuda"), cache, cfg)
    with pytest.raises(ValueError, match="one dtype"):
        awq.kv4_append(q[:, :2], q[:, 2:].half(), torch.zeros(2, dtype=torch.int32, device="cuda"), cache, cfg)


@pytest.mark.parametrize("lens", [[(7 * i) % 41 for i in range(700)], [3000 if i in (100, 650) else 5 for i in range(1100)]])
def test_more_sequences_than_a_launch(lens):
    """Batches above one launch's plan; with and without row starts, and contexts of no tokens."""
    _run(lens, [1 if n else 0 for n in lens], 2, 3, 64, 32, 16, "bf16", 120)
    cfg, cache, table, lens_t, slots = _fill(lens, 2, 64, 32, 16, "bf16", 121)
    q = _rand((len(lens), 6, 64), "bf16", 122, 2.0)
    out, lse = awq.kv4_attention(q, cache, table, lens_t, cfg, lse=True)
    _check(out, lse, q, cfg, _read(cache, cfg, slots), lens, range(len(lens) + 1), 3, 64 ** -0.5, "bf16")


def test_cache_beyond_32_bits():
    """The last pages of a cache of more than 2^32 bytes: written, read and attended as those of a small one."""
    heads, dim, page, group, pages = 32, 256, 256, 128, 2000
    cfg = awq.make_kv4(heads, dim, page, group)
    big, small = awq.kv4_new_cache(pages, cfg), awq.kv4_new_cache(4, cfg)
    assert big.numel() * 4 > 2 ** 32
    where = [pages - 1, 3, pages - 3, 1000]
    n = 4 * page - 37
    k, v, q = _rand((n, heads, dim), "bf16", 1), _rand((n, heads, dim), "bf16", 2), _rand((1, heads, dim), "bf16", 3)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    results = []
    for cache, ids in ((big, where), (small, [2, 0, 3, 1])):
        slots = torch.tensor([ids[i // page] * page + i % page for i in range(n)], dtype=torch.int32).cuda()
        awq.kv4_append(k, v, slots, cache, cfg)
        table = torch.tensor([ids], dtype=torch.int32).cuda()
        results.append((*awq.kv4_gather(cache, slots, cfg), awq.kv4_attention(q, cache, table, lens, cfg)))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][0].any()
    assert not big[[0, 1, 2, 4, 999, 1001, pages - 2]].any()


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, over one cache; a prompt and single tokens."""
    cfg, cache, table, lens, slots = _fill([900, 2300, 700], 4, 128, 128, 64, "bf16", 130)
    one, many = _rand((3, 16, 128), "bf16", 131), _rand((600, 16, 128), "bf16", 132)
    start = torch.tensor([0, 200, 400, 600], dtype=torch.int32).cuda()
    want = (awq.kv4_attention(one, cache, table, lens, cfg),
            awq.kv4_attention(many, cache, table, lens, cfg, q_start=start, max_q=200))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            got[0].append(awq.kv4_attention(one, cache, table, lens, cfg))
        with torch.cuda.stream(streams[1]):
            got[1].append(awq.kv4_attention(many, cache, table, lens, cfg, q_start=start, max_q=200))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_captured_between_other_work():
    """Calls captured behind copies, fills and another stream's work, whose launches overlap the kernel before them: every
    kernel sees what the ones before wrote."""
    cfg, cache, table, lens, slots = _fill([300, 41, 2500], 4, 128, 128, 32, "bf16", 150)
    X, W = _rand((9, 512), "bf16", 151), _rand((1024, 512), "bf16", 152, 0.1)
    wq, w_step = awq.quantize_int8(W)
    new = torch.from_numpy(slots[np.cumsum([300, 41, 2500]) - 1]).int().cuda()
    x_in, q_in = torch.zeros_like(X[:3]), torch.zeros((3, 1024), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            twice = x_in + x_in
        xq, x_step = awq.quantize_int8(x_in)
        here.wait_stream(side)
        y = awq.w8a8_gemm(xq, x_step, wq, w_step)  # behind an event as well as a kernel
        q_in.copy_(y)
        kv = q_in.view(3, 8, 128)[:, :4].contiguous()
        awq.kv4_append(kv, kv, new, cache, cfg)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            z = awq.quantize_int8(twice)[1]
        out = awq.kv4_attention(q_in.view(3, 8, 128), cache, table, lens, cfg)
        here.wait_stream(side)
        k, _ = awq.kv4_gather(cache, new, cfg)
        q_in.zero_()
        many = awq.kv4_attention(out.repeat(40, 1, 1), cache, table[2:], lens[2:], cfg,
                                 q_start=start, max_q=120)
        return y, z, out, k, many
    start = torch.tensor([0, 120], dtype=torch.int32, device="cuda")
    x_in.copy_(X[:3])
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(3):
        x_in.copy_(X[3 * i:3 * i + 3])
        want = step()
        torch.cuda.synchronize()
        for t in got:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b) and b.any()


def test_short_and_long_calls_agree():
    """Calls that leave outputs and workspace to the library (one compiled call) and calls that bring their own."""
    cfg, cache, table, lens, slots = _fill([300, 41, 77], 4, 128, 64, 32, "f16", 140)
    q = _rand((3, 12, 136), "f16", 141)[:, 2:10, :128]  # strided
    start = torch.tensor([0, 1, 1, 3], dtype=torch.int32).cuda()
    work = awq.workspace(awq.kv4_attention_workspace_size(3, 8, 2, cfg))
    out = torch.zeros((3, 8, 128), dtype=torch.float16, device="cuda")
    for args in (dict(), dict(scale=0.3), dict(lse=True), dict(q_start=start, max_q=2), dict(max_q=1)):
        a = awq.kv4_attention(q, cache, table, lens, cfg, **args)
        b = awq.kv4_attention(q, cache, table, lens, cfg, ws=work, out=out, **args)
        for x, y in zip(a if args.get("lse") else (a,), b if args.get("lse") else (b,)):
            assert x.dtype == y.dtype and x.is_contiguous() and torch.equal(x, y)
    s = torch.from_numpy(slots[:50]).int().cuda()
    for dt in (None, torch.bfloat16, torch.float16):
        a = awq.kv4_gather(cache, s, cfg, dtype=dt)
        own = tuple(torch.empty((50, 4, 128), dtype=dt or torch.bfloat16, device="cuda") for _ in range(2))
        b = awq.kv4_gather(cache, s, cfg, outputs=own)
        assert a[0].dtype == (dt or torch.bfloat16) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    k = _rand((50, 4, 256), "bf16", 142)
    one, two = cache.clone(), cache.clone()
    assert awq.kv4_append(k[..., :128], k[..., 128:], s, one, cfg) is one
    awq.kv4_append(k[..., :128].clone(), k[..., 128:].clone(), s, two, cfg)
    assert torch.equal(one, two) and not torch.equal(one, cache)
    with pytest.raises(awq.AwqError, match="SHAPE"):
        awq.kv4_attention(q[:, :6], cache, table, lens, cfg)  # 6 query heads over 4
    with pytest.raises(awq.AwqError, match="INVALID"):
        awq.kv4_attention(q, cache, table, lens, cfg, scale=float("nan"))
    with pytest.raises(ValueError, match="one row a sequence"):
        awq.kv4_attention(q[:2], cache, table, lens, cfg)


def test_decode_step_captured_and_replayed():
    """append + attend of one decode step in a graph, replayed as the contexts grow (lengths, slots and inputs change in
    place), beside a second graph with a workspace of its own."""
    heads, share, dim, page = 2, 4, 128, 16
    lens0 = [30, 64, 5]
    cfg, cache, table, lens, slots = _fill([n + 20 for n in lens0], heads, dim, 128, page, "bf16", 95)
    k = _rand((3, heads, dim), "bf16", 1)
    v = _rand((3, heads, dim), "bf16", 2)
    q = _rand((3, heads * share, dim), "bf16", 3)
    slot = torch.zeros(3, dtype=torch.int32, device="cuda")
    outs, graphs, works = [], [], []  # a graph's workspace lives as long as the graph
    for _ in range(2):
        out = torch.zeros((3, heads * share, dim), dtype=torch.bfloat16, device="cuda")
        work = awq.workspace(awq.kv4_attention_workspace_size(3, heads * share, 1, cfg))
        awq.kv4_attention(q, cache, table, lens, cfg, ws=work, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            awq.kv4_append(k, v, slot, cache, cfg)
            awq.kv4_attention(q, cache, table, lens, cfg, ws=work, out=out)
        outs.append(out)
        graphs.append(g)
        works.append(work)
    first = np.concatenate([[0], np.cumsum([n + 20 for n in lens0])])[:-1]
    for i in range(18):
        now = [n + i + 1 for n in lens0]
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        mine = slots[first + np.array(now) - 1]
        slot.copy_(torch.from_numpy(mine).int())
        for t, seed in ((k, 100), (v, 200), (q, 300)):
            t.copy_(_rand(t.shape, "bf16", seed + i))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        every = np.concatenate([slots[f:f + n] for f, n in zip(first, now)])
        _check(outs[0], None, q, cfg, _read(cache, cfg, every), now, [0, 1, 2, 3], share, dim ** -0.5, "bf16")


def test_attention_block_in_8_and_4_bits():
    """The operators together, as a decoder layer's attention runs them: int8 projections, cache write, attention over the
    cache, int8 output projection; a prompt, then single tokens: the same cache bytes as all at once, and every stage within
    its own bound of float64."""
    hidden, heads, share, dim, page = 512, 2, 4, 64, 16
    q_heads = heads * share
    wqkv = _rand(((q_heads + 2 * heads) * dim, hidden), "bf16", 1, hidden ** -0.5)
    wo = _rand((hidden, q_heads * dim), "bf16", 2, (q_heads * dim) ** -0.5)
    s = torch.exp(0.3 * _rand((hidden,), "bf16", 3).float())
    qkv_w, o_w = awq.quantize_int8(wqkv, s), awq.quantize_int8(wo)
    cfg = awq.make_kv4(heads, dim, page, 32)
    x = _rand((40, hidden), "bf16", 4)
    table = torch.tensor([[4, 0, 2]], dtype=torch.int32, device="cuda")
    slot_of = [int(table[0, i // page]) * page + i % page for i in range(40)]

    def layer(cache, rows, upto):
        xq = awq.quantize_int8(rows, s, inverse=True)
        qkv = awq.w8a8_gemm(*xq, *qkv_w).view(len(rows), q_heads + 2 * heads, dim)
        slots = torch.tensor(slot_of[upto - len(rows):upto], dtype=torch.int32, device="cuda")
        awq.kv4_append(qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:], slots, cache, cfg)
        o = awq.kv4_attention(qkv[:, :q_heads], cache, table, torch.tensor([upto], dtype=torch.int32, device="cuda"),
                              cfg, q_start=torch.tensor([0, len(rows)], dtype=torch.int32, device="cuda"),
                              max_q=len(rows))
        return awq.w8a8_gemm(*awq.quantize_int8(o.view(len(rows), -1)), *o_w), o, qkv

    one = awq.kv4_new_cache(5, cfg)
    y_all, o_all, qkv_all = layer(one, x, 40)
    steps = awq.kv4_new_cache(5, cfg)
    parts = [layer(steps, x[:33], 33)] + [layer(steps, x[i:i + 1], i + 1) for i in range(33, 40)]
    assert torch.equal(one, steps)  # the cache does not depend on how the tokens came
    _check(o_all, None, qkv_all[:, :q_heads], cfg, _read(one, cfg, np.array(slot_of)), [40], [0, 40], share, dim ** -0.5, "bf16")
    o_parts = torch.cat([p[1] for p in parts])
    _check(o_parts, None, qkv_all[:, :q_heads], cfg, _read(one, cfg, np.array(slot_of)), [40], [0, 40], share, dim ** -0.5, "bf16")
    # the output projection's own two roundings: its operands' codes, then the product
    o_q, o_s = awq.quantize_int8(o_all.view(40, -1))
    ref = S.int8_product(*(t.cpu().numpy() for t in (o_q, o_s, *o_w)))
    assert (np.abs(_f64(y_all) - ref) <= (UNIT["bf16"] + 1.01 * 2.0 ** -22) * np.abs(ref)).all()
