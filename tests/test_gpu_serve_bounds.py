"""The serving kernels on the debug build with index checks: on small ragged shapes, next to unusual arguments that the
kernels themselves turn away, their results equal the release build's bit for bit and no check fires."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import weight_only_int4_act_b200 as awq  # noqa: E402
from test_gpu_bounds import _using  # noqa: E402


def _rand(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _quantiser():
    """Rows in registers (1, 2 and 4 chunks a thread), rows read twice, strided rows; all ways of scaling."""
    out = []
    for rows, d in ((1, 16), (3, 4096), (5, 16400), (700, 272), (601, 6000), (650, 9008), (330, 20000), (3, 66000)):
        x = _rand((rows, d + 24), rows + d)[:, 8:8 + d]
        s = _rand((d,), 7, torch.float32).abs() + 0.5
        out += [*awq.quantize_int8(x), *awq.quantize_int8(x.half(), s), *awq.quantize_int8(x, s, inverse=True)]
    return out


def _product():
    """Few tokens (one CTA a tile and clusters), single-CTA and pair tiles, ragged in every direction, with and without bias."""
    out = []
    for n, o, i in ((1, 1, 16), (17, 130, 4112), (100, 300, 2048), (128, 129, 64), (129, 64, 48), (200, 1000, 528),
                    (999, 333, 1040), (1500, 4100, 256)):
        x, w = (awq.quantize_int8(_rand((r, i), r + i + k)) for k, r in enumerate((n, o)))
        for dtype in (torch.bfloat16, torch.float16):
            out.append(awq.w8a8_gemm(*x, *w, dtype=dtype, bias=_rand((o,), 3, torch.float32) if n % 2 else None))
    return out


def _cache(dim, group):
    """Write, read back and attend: tokens alone and whole strips, slots outside, short and long contexts, several rows,
    prompts; lengths, rows and pages that have to be left out."""
    out = []
    heads, page = 3, 32
    cfg = awq.make_kv4(heads, dim, page, group)
    cache = awq.kv4_new_cache(60, cfg)
    for n, at in ((40, 1), (1100, 64)):
        kv = _rand((n, 2 * heads, dim), n)
        slots = torch.arange(at, at + n, dtype=torch.int32, device="cuda")
        slots[3], slots[9] = -1, 60 * page
        awq.kv4_append(kv[:, :heads], kv[:, heads:], slots, cache, cfg)
        out += [cache.clone(), *awq.kv4_gather(cache, slots, cfg), *awq.kv4_gather(cache, slots[5:6], cfg, dtype=torch.float16)]
    order = torch.randperm(60, generator=torch.Generator().manual_seed(1)).int().cuda()
    for lens, pages, new in (([33, 1, 0], 2, 1), ([1100, 5, 640], 30, 1), ([1100, 40, 300], 30, 5), ([900, 300, 260], 30, 130)):
        table = order[:3 * pages].view(3, pages) if 3 * pages <= 60 else order[torch.arange(3 * pages, device="cuda") % 60].view(3, pages)
        for dtype in (torch.bfloat16, torch.float16):
            for wrong in (False, True):
                t, n = table.clone(), torch.tensor(lens, dtype=torch.int32).cuda()
                if wrong:
                    t[0, 1], n[1] = 60, 10 ** 6
                q = _rand((3 * new, 18 * heads, dim), new, dtype)
                start = torch.arange(4, dtype=torch.int32, device="cuda") * new
                o, lse = awq.kv4_attention(q, cache, t, n, cfg, q_start=start, max_q=new, lse=True)
                out += [o, lse]
    return out


CHAINS = {"quantiser": _quantiser, "product": _product}
for _d, _g in ((64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)):
    CHAINS[f"cache {_d} {_g}"] = lambda d=_d, g=_g: _cache(d, g)


@pytest.mark.parametrize("name", CHAINS)
def test_check_build_matches_release_and_no_check_fires(name):
    results = []
    for variant in ("release", "check"):
        with _using(variant):
            results.append([t.cpu() for t in CHAINS[name]()])
            assert awq.bounds_error() == (0, 0)
    assert len(results[0]) == len(results[1])
    for i, (a, b) in enumerate(zip(*results)):
        assert a.dtype == b.dtype and np.array_equal(a.view(torch.uint8).numpy(), b.view(torch.uint8).numpy()), i
