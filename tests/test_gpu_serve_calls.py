"""The serving calls from Python where arguments are not what a kernel can take: errors, never a crash."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import weight_only_int4_act_b200 as awq  # noqa: E402


@pytest.fixture(autouse=True)
def _no_error_from_before():
    try:
        awq.device_error()
    except awq.AwqError:
        pass


def test_tensors_without_storage_are_refused():
    """Inside torch.func's transforms a tensor is a plain torch.Tensor of the right device and type whose data_ptr() throws:
    a RuntimeError for every call, and the interpreter and the library go on."""
    cfg = awq.make_kv4(2, 64, 16)
    cache = awq.kv4_new_cache(4, cfg)
    x = torch.zeros((3, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((3, 4, 64), dtype=torch.int8, device="cuda")
    step = torch.ones(4, device="cuda")
    table, lens = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    calls = [(lambda t: awq.quantize_int8(t[0]), x),
             (lambda t: awq.w8a8_gemm(t, step, codes[0], step), codes),
             (lambda t: awq.kv4_append(t[:, :2], t[:, 2:], slots, cache, cfg), x),
             (lambda t: awq.kv4_gather(cache, t[:, 0, 0].int(), cfg), x),
             (lambda t: awq.kv4_attention(t, cache, table, lens, cfg), x)]
    for f, arg in calls:
        with pytest.raises(RuntimeError):
            torch.func.vmap(f)(arg)
        assert awq.quantize_int8(x[0, 0])[0].shape == (4, 64)  # as before


def test_strides_of_axes_of_one():
    """The stride of an axis with one entry means nothing: a token's slice out of rows of an odd pitch, a lone head."""
    cfg = awq.make_kv4(1, 64, 16)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn((1, 1, 64), generator=g, device="cuda").bfloat16() for _ in range(3))
    odd = [torch.empty_strided((1, 1, 64), (205, 77, 1), dtype=torch.bfloat16, device="cuda").copy_(t) for t in (k, v, q)]
    assert odd[0].stride() == (205, 77, 1)
    one, two = awq.kv4_new_cache(1, cfg), awq.kv4_new_cache(1, cfg)
    awq.kv4_append(k, v, slot, one, cfg)
    awq.kv4_append(odd[0], odd[1], slot, two, cfg)
    assert torch.equal(one, two) and one.any()
    out = torch.empty_like(q)
    want = awq.kv4_attention(q, one, table, lens, cfg)
    assert torch.equal(awq.kv4_attention(odd[2], one, table, lens, cfg), want) and want.any()
    assert torch.equal(awq.kv4_attention(odd[2], one, table, lens, cfg, out=out), want)  # (the long way)
    assert torch.equal(awq.quantize_int8(odd[0][0])[0], awq.quantize_int8(k[0])[0])


def _attention(new, context=40):
    """Arguments of an attention call of `new` rows in each of 5 sequences, whose tables are good."""
    cfg = awq.make_kv4(8, 64, 16)
    cache = awq.kv4_new_cache(5 * context // 16 + 5, cfg)
    pages = -(-context // 16)
    table = torch.arange(5 * pages, dtype=torch.int32, device="cuda").view(5, pages)
    lens = torch.full((5,), context, dtype=torch.int32, device="cuda")
    q = torch.ones((5 * new, 16, 64), dtype=torch.bfloat16, device="cuda")
    start = torch.arange(6, dtype=torch.int32, device="cuda") * new
    return q, cache, table, lens, cfg, dict(q_start=start, max_q=new)


@pytest.mark.parametrize("new,context", [(1, 40), (1, 4000), (90, 200)])
def test_device_errors_are_kept(new, context):
    """Calls without a workspace of their own: what the device finds is told by device_error(), once; short contexts, split
    ones, prompts; a page outside the cache, a length past the table, rows past max_q, and a replayed graph."""
    q, cache, table, lens, cfg, args = _attention(new, context)
    good = awq.kv4_attention(q, cache, table, lens, cfg, **args)
    awq.device_error()
    bad_page, bad_len = table.clone(), lens.clone()
    bad_page[3, 1] = cache.shape[0]
    bad_len[4] = table.shape[1] * 16 + 1
    short = dict(args, max_q=new - 1) if new > 1 else dict(args, q_start=args["q_start"] + 1)
    for a in ((bad_page, lens, args), (table, bad_len, args), (table, lens, short)):
        awq.kv4_attention(q, cache, a[0], a[1], cfg, **a[2])
        assert torch.equal(awq.kv4_attention(q, cache, table, lens, cfg, **args), good)  # (does not clear it)
        with pytest.raises(awq.AwqError, match="DEVICE"):
            awq.device_error()
        awq.device_error()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = awq.kv4_attention(q, cache, table, lens, cfg, **args)
    g.replay()
    awq.device_error()
    table.copy_(bad_page)
    g.replay()
    with pytest.raises(awq.AwqError, match="DEVICE"):
        awq.device_error()
    assert torch.isfinite(out).all()


def test_workspaces_still_tell_of_their_own_call():
    q, cache, table, lens, cfg, args = _attention(1)
    works = [awq.workspace(awq.kv4_attention_workspace_size(5, 16, 1, cfg)) for _ in range(2)]
    bad = table.clone()
    bad[0, 0] = -1
    awq.kv4_attention(q, cache, bad, lens, cfg, ws=works[0], **args)
    awq.kv4_attention(q, cache, table, lens, cfg, ws=works[1], **args)
    awq.workspace_error(works[1])
    for check in (lambda: awq.workspace_error(works[0]), awq.device_error):
        with pytest.raises(awq.AwqError, match="DEVICE"):
            check()
        check()


def test_no_rows_is_no_work():
    """A step without tokens: empty results from every call, with and without outputs of the caller's; shapes that the
    library does not take are refused all the same."""
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.ones(64, device="cuda")
    for args in (dict(), dict(s=s), dict(s=s, inverse=True)):
        q, step = awq.quantize_int8(x, **args)
        assert q.shape == (0, 64) and q.dtype == torch.int8 and step.shape == (0,)
    assert awq.quantize_int8(x, outputs=(q, step))[0] is q
    w = awq.quantize_int8(torch.ones((48, 64), dtype=torch.bfloat16, device="cuda"))
    y = awq.w8a8_gemm(q, step, *w, dtype=torch.float16)
    assert y.shape == (0, 48) and y.dtype == torch.float16 and awq.w8a8_gemm(q, step, *w, out=y) is y
    with pytest.raises(awq.AwqError):
        awq.quantize_int8(torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"))
    cfg = awq.make_kv4(2, 64, 16)
    cache = awq.kv4_new_cache(2, cfg)
    none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for batch, args in ((0, dict()), (0, dict(q_start=torch.zeros(1, **i32), max_q=1)), (3, dict(q_start=torch.zeros(4, **i32), max_q=5))):
        table, lens = torch.zeros((batch, 2), **i32), torch.zeros(batch, **i32)
        out, lse = awq.kv4_attention(none, cache, table, lens, cfg, lse=True, **args)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
        assert awq.kv4_attention(none, cache, table, lens, cfg, out=out, **args) is out
    with pytest.raises(awq.AwqError):
        awq.kv4_attention(none[:, :3], cache, table, lens, cfg, **args)  # 3 heads over 2
