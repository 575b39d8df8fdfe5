"""The serving-side entry points without a GPU: sizes, refusals before anything
is enqueued, and the oracle's statements of the formats. No test here enqueues
GPU work."""
import ctypes

import numpy as np
import pytest

import weight_only_int4_act_b200 as awq
from oracle import serve_oracle as S

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10008)
OK, ARG, SHAPE, WORKSPACE = 0, 1, 2, 3


def test_quantize_int8_refusals():
    f = awq.lib().awq_quantize_int8

    def call(x=FAKE, dt=0, ldx=64, s=FAKE, mode=1, rows=4, d_in=64, q=FAKE, step=FAKE):
        return f(x, dt, ldx, s, mode, rows, d_in, q, step, None)
    assert call(x=None) == ARG and call(q=None) == ARG and call(step=None) == ARG
    assert call(s=None) == ARG and call(s=None, mode=2) == ARG
    assert call(dt=2) == ARG and call(mode=3) == ARG and call(mode=-1) == ARG
    assert call(x=ODD) == ARG and call(q=ODD) == ARG and call(s=ODD) == ARG
    for d in (0, 8, 24, 131088):
        assert call(d_in=d, ldx=1 << 20) == SHAPE
    assert call(rows=0) == SHAPE and call(ldx=56) == SHAPE and call(ldx=68) == SHAPE


def test_w8a8_refusals_and_workspace():
    f = awq.lib().awq_w8a8_gemm
    big = 1 << 40

    def call(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, bias=None, dt=0, N=4, d_out=64, d_in=64, Y=FAKE, work=FAKE, n=big):
        return f(xq, xs, wq, ws, bias, dt, N, d_out, d_in, Y, work, n, None)
    for name in ("xq", "xs", "wq", "ws", "Y", "work"):
        assert call(**{name: None}) == ARG
    for name in ("xq", "wq", "Y", "work"):
        assert call(**{name: ODD}) == ARG
    assert call(dt=2) == ARG and call(bias=ctypes.c_void_p(0x10002)) == ARG
    for bad in (dict(N=0), dict(d_out=0), dict(d_in=0), dict(d_in=24), dict(d_in=131088), dict(d_out=(1 << 24) + 1)):
        assert call(**bad) == SHAPE
        assert awq.w8a8_workspace_size(bad.get("N", 4), bad.get("d_out", 64), bad.get("d_in", 64)) == 0
    for shape in ((1, 1, 16), (16, 28672, 8192), (4096, 4096, 4096)):
        need = awq.w8a8_workspace_size(*shape)
        assert need >= 1024
        assert call(N=shape[0], d_out=shape[1], d_in=shape[2], n=need - 1) == WORKSPACE


@pytest.mark.parametrize("bad", [dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(head_dim=80), dict(head_dim=0),
                                 dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(group=16),
                                 dict(group=256), dict(head_dim=96, group=64)])
def test_kv4_bad_config(bad):
    cfg = awq.make_kv4(4, 128, 64, 128)
    for k, v in bad.items():
        setattr(cfg, k, v)
    c = ctypes.byref(cfg)
    L = awq.lib()
    assert awq.kv4_page_bytes(cfg) == 0 and awq.kv4_attention_workspace_size(1, 1, 1, cfg) == 0
    assert L.awq_kv4_append(FAKE, FAKE, 0, 1, 512, 128, 512, 128, FAKE, FAKE, 4, c, None) == ARG
    assert L.awq_kv4_gather(FAKE, 4, FAKE, 1, c, FAKE, FAKE, 0, None) == ARG
    assert L.awq_kv4_attention(FAKE, 0, 512, 128, 1, 4, None, 1, FAKE, 4, FAKE, 2, FAKE, 1, 0.1, c, FAKE, None, FAKE,
                               1 << 40, None) == ARG
    with pytest.raises(awq.AwqError):
        awq.kv4_new_cache(4, cfg)


def test_kv4_cache_calls_refusals():
    cfg = awq.make_kv4(4, 128, 64)
    assert cfg.group == 128 and awq.make_kv4(1, 96).group == 32 and awq.make_kv4(1, 64).group == 64
    c = ctypes.byref(cfg)
    L = awq.lib()

    def put(k=FAKE, v=FAKE, dt=0, T=4, st=(512, 128, 512, 128), slots=FAKE, cache=FAKE, pages=4, c_=c):
        return L.awq_kv4_append(k, v, dt, T, *st, slots, cache, pages, c_, None)
    assert put(k=None) == ARG and put(v=None) == ARG and put(slots=None) == ARG and put(cache=None) == ARG
    assert put(c_=None) == ARG and put(dt=7) == ARG and put(k=ODD) == ARG and put(v=ODD) == ARG and put(cache=ODD) == ARG
    for i in range(4):
        st = [512, 128, 512, 128]
        st[i] += 4
        assert put(st=st) == ARG
        st[i] = -128
        assert put(st=st) == ARG
    assert put(T=-1) == SHAPE and put(pages=0) == SHAPE and put(pages=(1 << 25)) == SHAPE
    for pages in (1 << 58, 1 << 62):  # (times the page size: past 64 bits)
        assert put(pages=pages) == SHAPE
    assert put(T=0, k=None, v=None, slots=None) == OK

    def get(cache=FAKE, pages=4, slots=FAKE, T=4, k=FAKE, v=FAKE, dt=1):
        return L.awq_kv4_gather(cache, pages, slots, T, c, k, v, dt, None)
    assert get(cache=None) == ARG and get(slots=None) == ARG and get(k=ODD) == ARG and get(v=ODD) == ARG and get(dt=2) == ARG
    assert get(pages=0) == SHAPE and get(T=-1) == SHAPE
    assert get(T=0) == OK and get(k=None, v=None) == OK


def test_kv4_attention_refusals():
    cfg = awq.make_kv4(4, 128, 64)
    c = ctypes.byref(cfg)
    L = awq.lib()
    big = 1 << 40

    def call(q=FAKE, dt=0, st=(1024, 128), T=3, heads=8, start=None, max_q=1, cache=FAKE, pages=9, table=FAKE, tp=5,
             lens=FAKE, batch=3, scale=0.1, out=FAKE, lse=None, ws=FAKE, n=big):
        return L.awq_kv4_attention(q, dt, *st, T, heads, start, max_q, cache, pages, table, tp, lens, batch, scale, c, out,
                                   lse, ws, n, None)
    for name in ("q", "cache", "table", "lens", "out", "ws"):
        assert call(**{name: None}) == ARG
    for name in ("q", "cache", "out", "ws"):
        assert call(**{name: ODD}) == ARG
    assert call(dt=2) == ARG and call(scale=float("inf")) == ARG and call(scale=float("nan")) == ARG
    assert call(st=(1028, 128)) == ARG and call(st=(1024, 124)) == ARG
    assert call(heads=6) == SHAPE and call(heads=0) == SHAPE and call(batch=0) == SHAPE and call(batch=65536) == SHAPE
    assert call(max_q=0) == SHAPE and call(tp=0) == SHAPE and call(tp=1 << 26) == SHAPE and call(pages=0) == SHAPE
    assert call(tp=1 << 58) == SHAPE and call(tp=1 << 62) == SHAPE and call(pages=1 << 62) == SHAPE
    assert call(T=2) == SHAPE and call(max_q=2) == SHAPE and call(T=-1, start=FAKE) == SHAPE
    need = awq.kv4_attention_workspace_size(3, 8, 1, cfg)
    assert need >= 1024 and call(n=need - 1) == WORKSPACE
    assert awq.kv4_attention_workspace_size(3, 6, 1, cfg) == 0


def test_python_binding_refuses_cpu_tensors():
    import torch
    cfg = awq.make_kv4(2, 64)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    i = torch.zeros((4, 64), dtype=torch.int8)
    for call in (lambda: awq.quantize_int8(x), lambda: awq.w8a8_gemm(i, x[:, 0], i, x[:, 0]),
                 lambda: awq.kv4_append(x.view(2, 2, 64), x.view(2, 2, 64), i[0], i, cfg),
                 lambda: awq.kv4_gather(i, i[0], cfg), lambda: awq.kv4_attention(x.view(2, 2, 64), i, i, i, cfg)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_short_calls_leave_what_they_do_not_know():
    """The compiled calls return None for arguments that the binding has to look at, and never reach the library."""
    import torch
    from weight_only_int4_act_b200 import binding as B
    c = B._calls(B._active)
    cfg = awq.make_kv4(2, 64)
    at = ctypes.addressof(cfg)
    x, i = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 64), dtype=torch.int8)
    for bad in (x, None, 3, "x", np.zeros(4)):
        assert c.quantize_int8(bad, None, 1) is None and c.quantize_int8(x, bad, 1) is None
        assert c.w8a8_gemm(i, x, i, x, bad, False, bad) is None
        assert c.kv4_append(bad, x, i, i, at) is None and c.kv4_gather(bad, i, at, True) is None
        assert c.kv4_attention(bad, i, i, i, at, None, None, None, False) is None
    for f in vars(c).values():
        with pytest.raises(TypeError):
            f(1)
    with pytest.raises((TypeError, ValueError)):
        awq.quantize_int8([1.0])


# ---------------------------------------------------------------- the oracle's own statements
@pytest.mark.parametrize("D,g", [(64, 32), (96, 32), (128, 128), (256, 64)])
def test_strip_layout_places_every_code_once(D, g):
    seen = set()
    for kind in range(2):
        for t in range(16):
            for ch in range(D):
                byte, sh = S.place(D, g, kind, t, ch)
                assert kind * 8 * D <= byte < (kind + 1) * 8 * D and sh in (0, 4)
                seen.add((byte, sh))
            for j in range(D // g):
                at = S.place_params(D, g, kind, t, j)
                assert 16 * D <= at <= S.strip_bytes(D, g) - 4
                seen.add((at, None))
    assert len(seen) == 2 * 16 * (D + D // g)
    cfg = awq.make_kv4(3, D, 32, g)
    assert awq.kv4_page_bytes(cfg) == 2 * S.strip_bytes(D, g)


def test_strips_round_trip_and_single_tokens():
    rng = np.random.default_rng(1)
    D, g, page = 96, 32, 32
    x = rng.standard_normal((2, 2, page, D)) * 3
    y = rng.standard_normal((2, 2, page, D))
    k, v = S.four_bit(x, g), S.four_bit(y, g)
    whole = S.pack_pages(*k, *v, page)
    for kind, want in enumerate((k, v)):
        for a, b in zip(S.unpack_pages(whole, D, g)[kind], want):
            assert np.array_equal(a, b)
    single = np.full_like(whole, 0xEE)
    for p in range(2):
        for h in range(2):
            for t in rng.permutation(page):
                for kind, (c, s, z) in enumerate((k, v)):
                    S.write_token(single, p * page + t, h, page, D, g, kind, c[p, h, t], s[p, h, t], z[p, h, t])
    assert np.array_equal(single, whole)


def test_four_bit_error_is_half_a_step():
    """|value - v| <= half the ideal step and what fp16 takes off the stored one: (1/2 + 15 2^-11) step."""
    rng = np.random.default_rng(2)
    v = rng.standard_normal((500, 64)) * np.exp(rng.standard_normal((500, 1)) * 2)
    v = v.astype(np.float32).astype(np.float64)
    v[0], v[1], v[2, :32] = 0.0, 2.5, -1.25  # all equal groups are exact up to the step's rounding
    c, s, z = S.four_bit(v, 32)
    err = np.abs(S.four_bit_values(c, s, z) - v)
    assert (err <= (0.5 + 16 * 2.0 ** -11) * np.repeat(s.astype(np.float64), 32, -1)).all()
    assert not S.four_bit_values(c, s, z)[0].any()
    c, s, z = S.four_bit(np.array([[np.nan] + [1.0] * 31, [np.inf] + [0.0] * 31]), 32)
    assert np.isnan(s).all() and not c.any()


def test_int8_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 128)) * np.exp(rng.standard_normal((50, 1)) * 3)).astype(np.float32).astype(np.float64)
    x[0] = 0
    q, step = S.int8_rows(x)
    assert (np.abs(q * step.astype(np.float64)[:, None] - x) <= (0.5 + 127 * 2.0 ** -22) * step[:, None]).all()
    s = np.exp(rng.standard_normal(128)).astype(np.float32)
    qm, sm = S.int8_rows(x, s)
    assert (np.abs(qm * sm.astype(np.float64)[:, None] - x * s) <= (0.5 + 127 * 2.0 ** -21) * sm[:, None]).all()


def test_oracle_attention_by_hand():
    q = np.array([[[1.0, 0.0]], [[0.0, 2.0]]])
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[1.0, 1.0]]])
    v = np.array([[[1.0, 2.0]], [[3.0, 4.0]], [[5.0, 6.0]]])
    out, lse, p = S.attention(q, k, v, 1, 1.0, 2)
    e = np.e
    assert np.allclose(out[0, 0], (e * v[0, 0] + v[1, 0]) / (e + 1)) and np.isclose(lse[0, 0], np.log(e + 1))
    w = np.array([1.0, e * e, e * e])
    assert np.allclose(out[1, 0], w @ v[:, 0] / w.sum()) and np.isclose(p[1, 0].sum(), 1)
    out, lse, _ = S.attention(q, k, v, 1, 1.0, 0)
    assert not out[0].any() and np.isneginf(lse[0, 0]) and np.array_equal(out[1, 0], v[0, 0])
