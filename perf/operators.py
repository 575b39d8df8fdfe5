"""Cases of the serving-side operators next to the W4A16 product: the 8-bit
integer linear layer (per-row quantiser, product with a scale per token and
per output channel) and the paged key/value cache held in 4 bits (write, read
back, attention over it).

`run` computes a case in its plain form (elementary torch operations in 32
bits, rounded once) or, where `own` is true, through the package's entry
points; `exact` is the definition in 64 bits.

The 4-bit cache. int32 [n_pages, n_kv_heads, page_size/16 * strip words]: each
(page, head) holds page_size/16 strips of 16 tokens, a strip being, in bytes,
  keys    [16 tokens][4 q][D/32 j][4 b]   channel 8 (4 j + q) + 2 b + n in nibble n of the byte
  values  [D/32 p][8 r][4 q][2 h][4 b]    token 2 q + (b >> 1) + 8 (b & 1), channel 32 p + 16 n + 8 h + r in nibble n
  key parameters, then value parameters   [D/g groups][16 tokens] of (fp16 step, fp16 zero)
and a value stands for (code - zero) * step.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token through an attention projection: latency of the two launches
        dict(name="int8 1 token 4096x4096", op="int8", tokens=1, d_out=4096, d_in=4096, dtype="bf16", scaled=True, held=True),
        # a small decode batch through the 70B MLP layer: the int8 weights' bytes
        dict(name="int8 16 tokens 28672x8192", op="int8", tokens=16, d_out=28672, d_in=8192, dtype="f16", scaled=False, held=True),
        # a ragged mixed batch through the MLP up projection
        dict(name="int8 333 tokens 11008x4096", op="int8", tokens=333, d_out=11008, d_in=4096, dtype="bf16", scaled=True, held=True),
        # a trial of one scale vector: the weights are quantised in the pass too
        dict(name="int8 trial 1000 4096x11008", op="int8", tokens=1000, d_out=4096, d_in=11008, dtype="bf16", scaled=True, held=False),
        # a large prompt batch through the 70B MLP layer: the tensor cores
        dict(name="int8 16384 tokens 28672x8192", op="int8", tokens=16384, d_out=28672, d_in=8192, dtype="bf16", scaled=True, held=True),
        # one decode step's keys and values of 64 sequences, and their last pages read back
        dict(name="kv4 write 64 sequences", op="write", batch=64, new=1, len=513, heads=8, dim=128, group=128, page=64, dtype="bf16"),
        # a prompt's keys and values in fine groups, read back dense
        dict(name="kv4 write prompt 16411", op="write", batch=1, new=16411, len=16411, heads=8, dim=128, group=32, page=16, dtype="f16"),
        # one short conversation: latency
        dict(name="kv4 attend 1 x 777", op="attend", batch=1, new=1, len=777, low=1.0, q_heads=32, heads=32, dim=128, group=128, page=64, dtype="f16"),
        # a serving batch of mixed lengths, grouped queries
        dict(name="kv4 attend 64 x 8192 ragged", op="attend", batch=64, new=1, len=8192, low=0.02, q_heads=64, heads=8, dim=128, group=128, page=64, dtype="bf16"),
        # a few very long contexts
        dict(name="kv4 attend 4 x 131072", op="attend", batch=4, new=1, len=131072, low=1.0, q_heads=32, heads=8, dim=128, group=64, page=128, dtype="bf16"),
        # drafted tokens checked: 5 queries a sequence, a narrow head
        dict(name="kv4 attend 16 x 5 of 4001", op="attend", batch=16, new=5, len=4001, low=0.1, q_heads=24, heads=8, dim=64, group=32, page=32, dtype="f16"),
        # a prompt's later chunk over what the cache holds already
        dict(name="kv4 attend 2 x 2048 of 8000", op="attend", batch=2, new=2048, len=8000, low=0.5, q_heads=32, heads=8, dim=128, group=128, page=64, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int8", "int8", "write", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "int8":
        d_in = 16 * _spread(rng, 16, 700)
        d_out = _spread(rng, 64, 28672)
        tokens = min(_spread(rng, 1, 16384), 2 ** 39 // (d_in * d_out) + 1)
        return dict(op=op, tokens=tokens, d_out=d_out, d_in=d_in, dtype=dtype, scaled=rng.random() < 0.6,
                    held=rng.random() < 0.8)
    dim = rng.choice([64, 96, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if dim % g == 0])
    page = rng.choice([16, 32, 64, 128, 256])
    heads = rng.choice([1, 2, 4, 5, 8, 16, 32])
    if op == "write":
        batch = _spread(rng, 1, 64)
        length = _spread(rng, 1, max(2, 16384 * 8 * 128 // (batch * heads * dim)))
        new = rng.choice([1, 1, length, rng.randint(1, length)])
        return dict(op=op, batch=batch, new=new, len=length, heads=heads, dim=dim, group=group, page=page, dtype=dtype)
    kind = rng.choice(["token", "token", "draft", "chunk"])
    shared = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if kind == "chunk":
        batch, heads = rng.choice([1, 2]), min(heads, 8)
        shared = min(shared, 4)
        length = _spread(rng, 64, 8000)
        new = rng.randint(8, min(length, 2048))
    else:
        batch = _spread(rng, 1, 128)
        length = _spread(rng, 1, max(2, min(131072, 2 ** 22 * 128 // (batch * heads * dim))))
        new = 1 if kind == "token" else min(length, rng.randint(2, 8))
    return dict(op=op, batch=batch, new=new, len=length, low=rng.choice([1.0, 0.5, 0.05]), q_heads=heads * shared,
                heads=heads, dim=dim, group=group, page=page, dtype=dtype)


def _lengths(case):
    """Context length of each sequence: from `len` down to `low` of it, long and short ones mixed."""
    n, b, low = case["len"], case["batch"], case.get("low", 1.0)
    if b == 1:
        return [n]
    return [max(case["new"], 1, int(round(n * (1.0 - (1.0 - low) * ((i * 37) % b) / (b - 1))))) for i in range(b)]


def work(case):
    if case["op"] == "int8":
        t, o, i = case["tokens"], case["d_out"], case["d_in"]
        weights = o * i + 4 * o if case["held"] else 2 * o * i
        return {"bytes": 2 * t * i + 2 * t * o + weights + (4 * i if case["scaled"] else 0), "flops": 2 * t * o * i}
    h, d, ng = case["heads"], case["dim"], case["dim"] // case["group"]
    token = h * (d + 8 * ng)  # keys and values of one token: codes and parameters
    if case["op"] == "write":
        n = sum(_read_back(case))
        new = case["batch"] * case["new"]
        return {"bytes": new * (4 * h * d + 2 * token + 4) + (n - new) * token + n * (4 * h * d + 4), "flops": 0}
    pairs = sum(case["new"] * (n - case["new"]) + case["new"] * (case["new"] + 1) // 2 for n in _lengths(case))
    rows = case["batch"] * case["new"]
    return {"bytes": sum(_lengths(case)) * token + 4 * rows * case["q_heads"] * d,
            "flops": 4 * pairs * case["q_heads"] * d}


def _read_back(case):
    """Tokens of each sequence that a write case reads back: the pages that the new tokens lie in."""
    first = (case["len"] - case["new"]) // case["page"] * case["page"]
    return [case["len"] - first] * case["batch"]


# ------------------------------------------------------------------ inputs
def _strip_bytes(dim, group):
    return 16 * dim + 128 * (dim // group)


def _tables(case, gen, lengths, device):
    """Pages of each sequence, in shuffled order, a few of the pool unused: int32 [batch, most pages], padded with 0."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device=device).int()
    table = torch.zeros((len(need), max(need)), dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"] == "int8":
        t, o, i = case["tokens"], case["d_out"], case["d_in"]
        spread = torch.exp(0.7 * normal(i))  # some input channels carry large activations
        x = torch.empty((t, i), dtype=dt, device=dev)
        for r in range(0, t, 4096):
            x[r:r + 4096] = (normal(min(4096, t - r), i) * spread).to(dt)
        w = torch.empty((o, i), dtype=torch.bfloat16, device=dev)
        for r in range(0, o, 4096):
            w[r:r + 4096] = (0.02 * normal(min(4096, o - r), i)).to(torch.bfloat16)
        s = spread.sqrt().contiguous() if case["scaled"] else None
        st = dict(case=case, x=x, s=s)
        if case["held"]:
            parts = [_quantize_rows(w[r:r + 4096], s, False) for r in range(0, o, 4096)]
            st["wq"] = torch.cat([p[0].to(torch.int8) for p in parts])
            st["w_step"] = torch.cat([p[1] for p in parts])
        else:
            st["w"] = w
        return st

    h, d, g, page = case["heads"], case["dim"], case["group"], case["page"]
    lengths = _lengths(case)
    table, total = _tables(case, gen, lengths, dev)
    words = page // 16 * _strip_bytes(d, g) // 4
    lens = torch.tensor(lengths, dtype=torch.int32, device=dev)
    loud = torch.exp(0.5 * normal(h, d))  # keys have a few loud channels in every head
    if case["op"] == "write":
        new = case["batch"] * case["new"]
        cache = torch.zeros((total, h, words), dtype=torch.int32, device=dev)
        pos = torch.arange(case["len"], device=dev)
        slots = (table.long()[:, pos // page] * page + pos % page).int()  # [batch, len]
        # keys and values as the projection leaves them: slices of one [tokens, 3 parts of heads x dim] product
        kv = torch.empty((new, 3 * h, d), dtype=dt, device=dev)
        kv[:, :h] = 0
        kv[:, h:2 * h] = (normal(new, h, d) * loud).to(dt)
        kv[:, 2 * h:] = normal(new, h, d).to(dt)
        first = case["len"] - _read_back(case)[0]
        return dict(case=case, k=kv[:, h:2 * h], v=kv[:, 2 * h:], cache=cache,
                    slots=slots[:, case["len"] - case["new"]:].reshape(-1).contiguous(),
                    read=slots[:, first:].reshape(-1).contiguous())
    cache = torch.empty((total, h, words), dtype=torch.int32, device=dev)
    step = max(1, (1 << 26) // (page * h * d))
    for r in range(0, total, step):
        n = min(step, total - r)
        k = (normal(n, h, page, d) * loud[:, None]).to(dt)
        v = normal(n, h, page, d).to(dt)
        cache[r:r + n] = _pack(*_quantize4(k, g), *_quantize4(v, g)).view(n, h, words)
    n = case["new"]
    q = (2.0 * normal(case["batch"] * n, case["q_heads"], d)).to(dt)
    q_start = torch.arange(case["batch"] + 1, dtype=torch.int32, device=dev) * n
    return dict(case=case, q=q, q_start=q_start, cache=cache, table=table, lens=lens)


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    return {"int8": _run_int8, "write": _run_write, "attend": _run_attend}[case["op"]](case, state)


def _run_int8(case, st):
    dt = DTYPES[case["dtype"]]
    if own:
        import weight_only_int4_act_b200 as awq
        wq, w_step = (st["wq"], st["w_step"]) if case["held"] else awq.quantize_int8(st["w"], st["s"])
        xq, x_step = awq.quantize_int8(st["x"], st["s"], inverse=True)
        return {"y": awq.w8a8_gemm(xq, x_step, wq, w_step, dtype=dt)}
    wq, w_step = (st["wq"], st["w_step"]) if case["held"] else _quantize_rows(st["w"], st["s"], False)
    xq, x_step = _quantize_rows(st["x"], st["s"], True)
    return {"y": ((xq @ wq.float().t()) * x_step[:, None] * w_step).to(dt)}


def _run_write(case, st):
    dt = DTYPES[case["dtype"]]
    if own:
        import weight_only_int4_act_b200 as awq
        cfg = awq.make_kv4(case["heads"], case["dim"], case["page"], case["group"])
        awq.kv4_append(st["k"], st["v"], st["slots"], st["cache"], cfg)
        k, v = awq.kv4_gather(st["cache"], st["read"], cfg, dtype=dt)
        return {"k": k, "v": v}
    d, g, page = case["dim"], case["group"], case["page"]
    cache = st["cache"].view(torch.uint8).view(st["cache"].shape[0], case["heads"], page // 16, _strip_bytes(d, g))
    slot = st["slots"].long()
    at = slot // page, slice(None), slot % page // 16
    t = slot % 16
    kc, kp = _quantize4(st["k"], g)  # [new, heads, dim], [new, heads, groups, 2]
    vc, vp = _quantize4(st["v"], g)
    dev = slot.device
    # keys: the token's own D/2 bytes, in [q][j][b] order
    kb = (kc[..., 0::2] | kc[..., 1::2] << 4).view(-1, case["heads"], d // 32, 4, 4).transpose(2, 3).reshape(len(slot), -1, d // 2)
    _put(cache, at, t[:, None] * (d // 2) + torch.arange(d // 2, device=dev), kb)
    # values: one byte for each pair of channels 16 apart, in [p][r][h] order
    vv = vc.view(-1, case["heads"], d // 32, 2, 2, 8)
    vb = (vv[:, :, :, 0] | vv[:, :, :, 1] << 4).transpose(3, 4).reshape(len(slot), -1, d // 2)
    q, b = t % 8 // 2, 2 * (t % 2) + t // 8
    lane = torch.arange(d // 4, device=dev)[:, None] * 32 + torch.arange(2, device=dev) * 4  # (p, r), h
    _put(cache, at, 8 * d + (lane.view(1, -1) + (q * 8 + b)[:, None]), vb)
    for k, pp in ((0, kp), (1, vp)):
        ng = d // g
        off = 16 * d + 64 * ng * k + torch.arange(ng, device=dev)[:, None] * 64 + torch.arange(4, device=dev)
        _put(cache, at, off.view(1, -1) + 4 * t[:, None], pp.contiguous().view(torch.uint8).view(len(slot), -1, 4 * ng))
    strip = st["read"].long()
    blob = cache[strip // page, :, strip % page // 16]  # [tokens, heads, strip]
    kd, vd = _unpack(blob, d, g)
    row = torch.arange(len(strip), device=dev), slice(None), strip % 16
    return {"k": kd[row].to(dt), "v": vd[row].to(dt)}


def _put(cache, at, offset, byte):
    """cache[page, head, strip, offset[token, i]] = byte[token, head, i]"""
    heads = torch.arange(cache.shape[1], device=cache.device)[None, :, None]
    cache[at[0][:, None, None], heads, at[2][:, None, None], offset[:, None, :]] = byte


def _run_attend(case, st):
    if own:
        import weight_only_int4_act_b200 as awq
        cfg = awq.make_kv4(case["heads"], case["dim"], case["page"], case["group"])
        return {"o": awq.kv4_attention(st["q"], st["cache"], st["table"], st["lens"], cfg, q_start=st["q_start"],
                                       max_q=case["new"])}
    h, d, n = case["heads"], case["dim"], case["new"]
    b, most = st["table"].shape
    blob = st["cache"][st["table"].long()].view(torch.uint8)  # [b, pages, h, strips of the page]
    k, v = _unpack(blob.view(b, most, h, -1, _strip_bytes(d, case["group"])), d, case["group"])
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(b, h, -1, d)
    v = v.permute(0, 2, 1, 3, 4, 5).reshape(b, h, -1, d)
    share = case["q_heads"] // h
    q = st["q"].float().view(b, n, h, share, d).permute(0, 2, 3, 1, 4).reshape(b, h, share * n, d)
    logit = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    key = torch.arange(k.shape[2], device=q.device)
    last = st["lens"][:, None] - n + torch.arange(n, device=q.device)  # the newest key that each query sees
    seen = (key <= last[..., None]).repeat(1, share, 1)[:, None]  # [b, 1, share * n, keys]
    logit = logit.masked_fill(~seen, -math.inf)
    top = logit.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(logit - top)
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    return {"o": o.view(b, h, share, n, d).permute(0, 3, 1, 2, 4).reshape(st["q"].shape).to(st["q"].dtype)}


# ------------------------------------------------------------------ plain forms of the formats
def _quantize_rows(x, s, inverse):
    """Codes (as float32) and steps of the symmetric 8-bit quantiser, one step a row."""
    v = x.float()
    if s is not None:
        v = v * (torch.ones_like(s) / s if inverse else s)
    top = v.abs().amax(1).clamp_min(1e-8)
    full = torch.full_like(top, 127.0)
    return (v * (full / top)[:, None]).round(), top / full


def _quantize4(x, g):
    """Codes uint8 [..., D] and (step, zero) fp16 [..., D/g, 2] of the 4-bit quantiser, groups of g channels."""
    v = x.float().unflatten(-1, (-1, g))
    lo, hi = v.amin(-1).clamp_max(0.0), v.amax(-1).clamp_min(0.0)
    step = ((hi - lo) / torch.full_like(lo, 15.0)).to(torch.float16).clamp(2.0 ** -24, 65504.0)
    inv = torch.ones_like(lo) / step.float()
    zero = (-lo * inv).round().clamp(0, 15)
    code = ((v * inv[..., None]).round() + zero[..., None]).clamp(0, 15)
    return code.to(torch.uint8).flatten(-2), torch.stack([step, zero.to(torch.float16)], -1)


def _pack(kc, kp, vc, vp):
    """Strips of bytes [..., tokens/16, strip] of codes [..., tokens, D] and parameters [..., tokens, D/g, 2]."""
    d = kc.shape[-1]
    lead = kc.shape[:-2] + (-1,)
    k = kc.reshape(lead + (16, d // 32, 4, 4, 2))  # tokens, j, q, b, n
    k = (k[..., 0] | k[..., 1] << 4).transpose(-2, -3)
    v = vc.reshape(lead + (2, 4, 2, d // 32, 2, 2, 8))  # y, q, x (token 8 y + 2 q + x), p, n, h, r
    v = v[..., 0, :, :] | v[..., 1, :, :] << 4  # y, q, x, p, h, r
    n = v.dim() - 6
    v = v.permute(*range(n), n + 3, n + 5, n + 1, n + 4, n + 2, n + 0)  # p, r, q, h, x, y
    par = [p.reshape(lead + (16,) + p.shape[-2:]).transpose(-2, -3).contiguous().view(torch.uint8) for p in (kp, vp)]
    parts = [k, v] + par
    flat = [p.reshape(p.shape[:n] + (-1,)) for p in parts]
    return torch.cat(flat, -1).view(torch.int32)


def _unpack(blob, d, g):
    """Keys and values, float32 [..., 16, D], of strips of bytes [..., strip]."""
    lead = blob.shape[:-1]
    n = len(lead)
    k = blob[..., :8 * d].reshape(lead + (16, 4, d // 32, 4)).transpose(-2, -3)
    k = torch.stack([k & 15, k >> 4], -1).reshape(lead + (16, d))
    v = blob[..., 8 * d:16 * d].reshape(lead + (d // 32, 8, 4, 2, 2, 2))  # p, r, q, h, x, y
    v = torch.stack([v & 15, v >> 4], -1)  # p, r, q, h, x, y, n
    v = v.permute(*range(n), n + 5, n + 2, n + 4, n + 0, n + 6, n + 3, n + 1).reshape(lead + (16, d))
    par = blob[..., 16 * d:].contiguous().view(torch.float16).view(lead + (2, d // g, 16, 2)).float()

    def value(code, pp):
        pp = pp.transpose(-2, -3)  # 16, groups, 2
        return ((code.float().unflatten(-1, (-1, g)) - pp[..., 1:]) * pp[..., :1]).flatten(-2)

    return value(k, par[..., 0, :, :, :]), value(v, par[..., 1, :, :, :])


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"int8": _exact_int8, "write": _exact_write, "attend": _exact_attend}[case["op"]](case, st)


def _exact_rows8(x, scale):
    y = x.double()
    if scale is not None:
        y = y * scale
    most = torch.maximum(y.abs().max(dim=1).values, torch.tensor(1e-8, dtype=torch.float64, device=y.device))
    step = most / 127.0
    return torch.round(y / step.unsqueeze(1)), step


def _exact_int8(case, st):
    s = None if st["s"] is None else st["s"].double()
    out = torch.empty((case["tokens"], case["d_out"]), dtype=torch.float64, device=st["x"].device)
    for o in range(0, case["d_out"], 4096):
        if case["held"]:
            w = st["wq"][o:o + 4096].double() * st["w_step"][o:o + 4096].double().unsqueeze(1)
        else:
            code, step = _exact_rows8(st["w"][o:o + 4096], s)
            w = code * step.unsqueeze(1)
        for t in range(0, case["tokens"], 4096):
            code, step = _exact_rows8(st["x"][t:t + 4096], None if s is None else 1.0 / s)
            out[t:t + 4096, o:o + 4096] = torch.mm(code * step.unsqueeze(1), w.t())
    return {"y": out}


def _exact_four(x, g):
    """What the 4-bit groups of x read back as."""
    y = x.double()
    parts = []
    for c in range(0, y.shape[-1], g):
        part = y[..., c:c + g]
        lo = torch.minimum(part.min(dim=-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=y.device))
        hi = torch.maximum(part.max(dim=-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=y.device))
        step = ((hi - lo) / 15.0).to(torch.float16).double().clamp(2.0 ** -24, 65504.0)
        zero = torch.round(-lo / step)
        parts.append((torch.clamp(torch.round(part / step) + zero, 0, 15) - zero) * step)
    return torch.cat(parts, dim=-1)


def _exact_write(case, st):
    new = {int(s): i for i, s in enumerate(st["slots"].tolist())}
    where = torch.tensor([new.get(int(s), -1) for s in st["read"].tolist()], device=st["k"].device)
    out = []
    for x in (st["k"], st["v"]):
        full = _exact_four(x, case["group"])
        out.append(torch.where(where[:, None, None] >= 0, full[where.clamp(min=0)], torch.zeros_like(full[:1])))
    return {"k": out[0], "v": out[1]}


def _exact_dense(case, strips):
    """float64 keys and values [tokens, dim] of one head's strips [n, strip bytes], byte by byte from the format."""
    d, g, dev = case["dim"], case["group"], strips.device
    t = torch.arange(16, device=dev).unsqueeze(1)
    c = torch.arange(d, device=dev).unsqueeze(0)
    word = c // 8
    key = t * (d // 2) + ((word % 4) * (d // 32) + word // 4) * 4 + (c % 8) // 2
    lane = (c % 8) * 4 + (t % 8) // 2
    val = 8 * d + ((c // 32) * 32 + lane) * 8 + ((c // 8) % 2) * 4 + 2 * (t % 2) + t // 8
    out = []
    for off, shift, base in ((key, 4 * (c % 2), 0), (val, 4 * ((c // 16) % 2), 1)):
        code = (strips[:, off.expand(16, d)].int() >> shift) & 15
        at = (16 * d + 64 * (d // g) * base + (c // g) * 64 + 4 * t).expand(16, d)
        halves = [(strips[:, at + k].int() | strips[:, at + k + 1].int() << 8).to(torch.int16).view(torch.float16).double()
                  for k in (0, 2)]
        out.append(((code - halves[1]) * halves[0]).reshape(-1, d))
    return out


def _exact_attend(case, st):
    n, share = case["new"], case["q_heads"] // case["heads"]
    lengths = _lengths(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    for b, length in enumerate(lengths):
        pages = st["table"][b, :-(-length // case["page"])].long()
        for h in range(case["heads"]):
            strips = st["cache"][pages, h].contiguous().view(torch.uint8).view(-1, _strip_bytes(case["dim"], case["group"]))
            k, v = (x[:length] for x in _exact_dense(case, strips))
            for e in range(share):
                q = st["q"][b * n:(b + 1) * n, h * share + e].double()
                z = torch.mm(q, k.t()) / math.sqrt(case["dim"])
                if n > 1:
                    z = z + torch.full((n, length), -math.inf, dtype=torch.float64, device=z.device).triu(length - n + 1)
                out[b * n:(b + 1) * n, h * share + e] = torch.mm(torch.softmax(z, dim=1), v)
    return {"o": out}
