"""The 8-bit integer linear layer on the GPU: awq_quantize_int8 code for code
against its float32 statement, and awq_w8a8_gemm against the float64 product
of the same codes.

Tolerance of the product: the integer sum is exact, so Y is the float64 value
through at most four fp32 roundings (int32 to fp32, two steps, the bias; each
half a unit, 2^-24 relative, the bias' relative to the larger of the sum's
terms) and one to Y's type (u = 2^-8 bf16, 2^-11 fp16; half the smallest
subnormal, 2^-25, below fp16's normal range):
|Y_gpu - Y| <= u |Y| + 1.01 * (4 * 2^-24) (|Y - bias| + |bias|) + 2^-25."""
import zlib

import numpy as np
import pytest

from oracle import awq_oracle as O
from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import weight_only_int4_act_b200 as awq  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * scale
    return x.to(DT[dtype])


def _f64(t):
    return t.double().cpu().numpy()


def _check_rows(X, s, inverse, q, step):
    qr, sr = S.int8_rows(_f64(X), None if s is None else s.cpu().numpy(), inverse)
    assert np.array_equal(q.cpu().numpy(), qr)
    assert np.array_equal(step.cpu().numpy(), sr, equal_nan=True)


ROWS = [(1, 16), (1, 4096), (3, 32), (5, 48), (17, 1040), (2, 4112), (64, 8192), (130, 11008), (3, 16384), (2, 16400),
        (2, 40000), (1, 131072), (1000, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("mode", ["plain", "mul", "div"])
@pytest.mark.parametrize("rows,d_in", ROWS)
def test_rows_code_for_code(rows, d_in, mode, dtype):
    X = _rand((rows, d_in), dtype, rows + d_in)
    s = None if mode == "plain" else torch.exp(_rand((d_in,), "bf16", 7).float())
    q, step = awq.quantize_int8(X, s, inverse=mode == "div")
    _check_rows(X, s, mode == "div", q, step)


def test_rows_special_values():
    """Zero rows, the floor, halves, the largest values, NaN and infinity in
    single rows, infinity that only the scaling makes."""
    d = 256
    X = torch.zeros((10, d), dtype=torch.bfloat16)
    X[1, 3] = 1e-30
    X[2] = torch.arange(d) % 255 - 127.0           # every code, step 1
    X[3, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])  # ties go to even
    X[4] = 3e38
    X[5, 17] = float("nan")
    X[6, 200] = float("-inf")
    X[7, 0] = -5.0
    X[8, 1] = 3e38
    X = X.cuda()
    q, step = awq.quantize_int8(X)
    _check_rows(X, None, False, q, step)
    assert torch.isnan(step[[5, 6]]).all() and not q[[5, 6]].any() and int(torch.isnan(step).sum()) == 2
    assert q[3, :4].tolist() == [127, 0, 2, -2]
    s = torch.ones(d, device="cuda")
    s[1] = 0.5
    q, step = awq.quantize_int8(X, s, inverse=True)  # 3e38 / 0.5 overflows: row 8 (and row 4) not finite
    _check_rows(X, s, True, q, step)
    assert torch.isnan(step[8]) and torch.isnan(step[4])


def test_rows_strided_views_and_given_outputs():
    big = _rand((37, 1024), "f16", 3)
    X = big[:, 256:768]
    q = torch.full((39, 512), 55, dtype=torch.int8, device="cuda")
    step = torch.full((39,), 7.0, device="cuda")
    awq.quantize_int8(X, outputs=(q[1:38], step[1:38]))
    _check_rows(X, None, False, q[1:38], step[1:38])
    for edge in (0, 38):  # nothing outside the outputs is touched
        assert (q[edge] == 55).all() and step[edge] == 7.0
    every = big[::3]
    q2, s2 = awq.quantize_int8(every)
    _check_rows(every, None, False, q2, s2)


# N, d_out, d_in
PRODUCTS = [(1, 1, 16), (1, 8, 16), (1, 130, 4096), (1, 4096, 4096), (2, 257, 528), (7, 96, 1040), (8, 1000, 512),
            (9, 640, 2048), (16, 4096, 4096), (17, 333, 352), (33, 128, 16384), (64, 512, 1024), (65, 200, 144),
            (100, 384, 48), (128, 257, 4096), (129, 1023, 656), (255, 128, 256), (300, 130, 272), (333, 11008, 1024),
            (512, 512, 512), (777, 640, 1152), (1025, 2049, 400), (2048, 4096, 2048), (3, 128, 131072)]


def _operands(N, d_out, d_in, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    xq = torch.randint(-127, 128, (N, d_in), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (d_out, d_in), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(N, generator=g, device="cuda") * 0.02 + 1e-3
    ws = torch.rand(d_out, generator=g, device="cuda") * 0.002 + 1e-4
    bias = torch.randn(d_out, generator=g, device="cuda")
    return xq, xs, wq, ws, bias


def _check_product(Y, xq, xs, wq, ws, bias=None):
    ref = S.int8_product(xq.cpu().numpy(), xs.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy(),
                         None if bias is None else bias.cpu().numpy())
    b = 0.0 if bias is None else np.abs(bias.cpu().numpy().astype(np.float64))
    u = UNIT["bf16" if Y.dtype == torch.bfloat16 else "f16"]
    tol = u * np.abs(ref) + 1.01 * 2.0 ** -22 * (np.abs(ref) + 2 * b) + 2.0 ** -25
    err = np.abs(_f64(Y) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], _f64(Y)[bad][:5], ref[bad][:5])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,d_out,d_in", PRODUCTS)
def test_product_against_float64(N, d_out, d_in, dtype):
    xq, xs, wq, ws, bias = _operands(N, d_out, d_in, zlib.crc32(f"{N} {d_out} {d_in}".encode()))
    work = awq.workspace(awq.w8a8_workspace_size(N, d_out, d_in))
    work.fill_(0xA5)  # a workspace holds anything before the call
    Y = awq.w8a8_gemm(xq, xs, wq, ws, dtype=DT[dtype], ws=work)
    awq.workspace_error(work)
    _check_product(Y, xq, xs, wq, ws)
    Yb = awq.w8a8_gemm(xq, xs, wq, ws, dtype=DT[dtype], bias=bias, ws=work)
    awq.workspace_error(work)
    _check_product(Yb, xq, xs, wq, ws, bias)
    assert torch.equal(Y, awq.w8a8_gemm(xq, xs, wq, ws, dtype=DT[dtype], ws=work))


def test_product_extreme_sums_are_exact():
    """127 * 127 * 131072, the largest sum, of either sign, and steps that make it 1."""
    K = 131072
    xq = torch.full((3, K), 127, dtype=torch.int8, device="cuda")
    wq = torch.full((160, K), 127, dtype=torch.int8, device="cuda")
    wq[1::2] = -127
    one = torch.ones(3, device="cuda")
    ws = torch.full((160,), 1.0 / (127 * 127 * K), dtype=torch.float32, device="cuda")
    Y = awq.w8a8_gemm(xq, one, wq, ws, dtype=torch.float16)
    want = torch.ones(160, device="cuda")
    want[1::2] = -1
    assert torch.equal(Y.float(), want.expand(3, -1))


@pytest.mark.parametrize("N", [5, 300, 4097])
def test_product_writes_its_rows_only(N):
    xq, xs, wq, ws, _ = _operands(N, 264, 160, 5)
    buf = torch.full((N + 2, 264), 3.0, dtype=torch.bfloat16, device="cuda")
    awq.w8a8_gemm(xq, xs, wq, ws, out=buf[1:N + 1])
    assert (buf[0] == 3).all() and (buf[-1] == 3).all()
    _check_product(buf[1:N + 1], xq, xs, wq, ws)


def test_product_nan_row_stays_alone():
    X = _rand((6, 512), "bf16", 9)
    X[2, 100] = float("inf")
    W = _rand((140, 512), "bf16", 10, 0.02)
    xq, xs = awq.quantize_int8(X)
    wq, ws = awq.quantize_int8(W)
    Y = awq.w8a8_gemm(xq, xs, wq, ws)
    assert torch.isnan(Y[2]).all() and torch.isfinite(Y[[0, 1, 3, 4, 5]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_layer_error_is_the_quantisers(dtype):
    """W S and X S^-1 quantised, multiplied: within the sum of the half steps of
    the float64 layer W X. |Y - Y0| <= sum_i (|v| dw/2 + |w| dx/2 + dx dw/4), dx
    and dw the rows' steps, v = X S^-1, w = W S, plus the product's roundings."""
    N, d_out, d_in = 70, 200, 768
    X, W = _rand((N, d_in), dtype, 21), _rand((d_out, d_in), "bf16", 22, 0.02)
    s = torch.exp(0.5 * _rand((d_in,), "bf16", 23).float())
    wq, ws = awq.quantize_int8(W, s)
    xq, xs = awq.quantize_int8(X, s, inverse=True)
    Y = awq.w8a8_gemm(xq, xs, wq, ws, dtype=DT[dtype])
    s64 = _f64(s)
    v, w = _f64(X) / s64, _f64(W) * s64
    ref = v @ w.T
    dx, dw = _f64(xs)[:, None], _f64(ws)
    half = 0.5 * (np.abs(v).sum(1)[:, None] * dw + dx * np.abs(w).sum(1)) + 0.25 * d_in * dx * dw
    tol = 1.001 * half + 1.01 * (UNIT[dtype] + 2.0 ** -22) * (np.abs(ref) + half)
    assert (np.abs(_f64(Y) - ref) <= tol).all()


def test_python_refusals():
    xq, xs, wq, ws, bias = _operands(4, 32, 64, 1)
    with pytest.raises(ValueError, match="torch.int8"):
        awq.w8a8_gemm(xq.float(), xs, wq, ws)
    with pytest.raises(ValueError, match="wq"):
        awq.w8a8_gemm(xq, xs, wq[:, :48].contiguous(), ws)
    with pytest.raises(ValueError, match="x_step"):
        awq.w8a8_gemm(xq, xs[:3], wq, ws)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        awq.w8a8_gemm(xq, xs, wq, ws, dtype=torch.float32)
    with pytest.raises(awq.AwqError, match="WORKSPACE"):
        awq.w8a8_gemm(xq, xs, wq, ws, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(awq.AwqError, match="SHAPE"):
        awq.quantize_int8(torch.zeros((2, 24), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="last axis"):
        awq.quantize_int8(torch.zeros((32, 64), dtype=torch.float16, device="cuda").t())


def test_side_stream_and_graph_replay():
    """The layer on a stream of its own, then captured once and replayed on new data."""
    N, d_out, d_in = 24, 512, 1024
    W = _rand((d_out, d_in), "bf16", 31, 0.02)
    wq, ws = awq.quantize_int8(W)
    X = _rand((N, d_in), "bf16", 32)
    Y = torch.empty((N, d_out), dtype=torch.bfloat16, device="cuda")
    work = awq.workspace(awq.w8a8_workspace_size(N, d_out, d_in))
    outs = (torch.empty((N, d_in), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda"))

    def layer():
        awq.quantize_int8(X, outputs=outs)
        awq.w8a8_gemm(*outs, wq, ws, ws=work, out=Y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    _check_product(Y, *outs, wq, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for seed in (33, 34):
        X.copy_(_rand((N, d_in), "bf16", seed))
        g.replay()
        torch.cuda.synchronize()
        _check_rows(X, None, False, *outs)
        _check_product(Y, *outs, wq, ws)


def test_short_and_long_calls_agree():
    """Calls that leave outputs and workspace to the library (one compiled call) and calls that bring their own."""
    X, W = _rand((37, 272), "bf16", 50), _rand((45, 272), "f16", 51)
    s = torch.rand(272, device="cuda") + 0.5
    work = awq.workspace(awq.w8a8_workspace_size(37, 45, 272))
    for sc, inv in ((None, False), (s, False), (s, True)):
        a = awq.quantize_int8(X[::2], sc, inverse=inv)
        b = awq.quantize_int8(X[::2], sc, inverse=inv, outputs=tuple(torch.empty_like(t) for t in a))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    x, w, bias = awq.quantize_int8(X, s, inverse=True), awq.quantize_int8(W, s), torch.randn(45, device="cuda")
    for dt in (None, torch.bfloat16, torch.float16):
        for bi in (None, bias):
            a = awq.w8a8_gemm(*x, *w, dtype=dt, bias=bi)
            out = torch.empty((37, 45), dtype=dt or torch.bfloat16, device="cuda")
            assert a.dtype == out.dtype and torch.equal(a, awq.w8a8_gemm(*x, *w, bias=bi, ws=work, out=out))
    with pytest.raises(ValueError):
        awq.w8a8_gemm(*x, *w, dtype=torch.float32)
    with pytest.raises(ValueError):
        awq.w8a8_gemm(*x, w[0], w[1][:-1])
    with pytest.raises(awq.AwqError, match="SHAPE"):
        awq.quantize_int8(X[:, :200])
