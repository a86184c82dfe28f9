"""Cases for the attention operators that stand between a layer's QKV and output projections:
the per-head norm with rotation, the quantised paged KV cache (append, read back) and the
attention of drafted tokens over it.

Each case is one pass through one operator (quantised appends also read the rows back, so that
their outputs are values).  ``own`` False computes the plain form in elementary torch operations;
``own`` True calls the library.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 16 sequences behind the Llama-7B QKV projection (32 heads of 128)
        dict(name="qk_decode_16", op="qk", tokens=16, q_heads=32, kv_heads=32, dim=128, rotary=128,
             interleaved=False, norm=True),
        # the 2048-token prefill that the layer benchmark runs, Llama-7B heads
        dict(name="qk_prefill_2048", op="qk", tokens=2048, q_heads=32, kv_heads=32, dim=128, rotary=128,
             interleaved=False, norm=True),
        # an odd token count, shared heads of 64, half of each head rotated in adjacent pairs
        dict(name="qk_ragged_1021_d64", op="qk", tokens=1021, q_heads=64, kv_heads=8, dim=64, rotary=32,
             interleaved=True, norm=True),
        # a decode step's new rows into the INT4 cache, one padded row
        dict(name="append_decode_16_int4", op="append", tokens=16, heads=32, dim=128, page=64, bits=4,
             rotary=128, interleaved=False, padded=1),
        # a prefill's rows into an fp16 cache
        dict(name="append_prefill_2048_fp16", op="append", tokens=2048, heads=32, dim=128, page=64, bits=16,
             rotary=128, interleaved=False, padded=0),
        # shared heads, INT8, a packed batch with padding behind it
        dict(name="append_4093_int8_gqa", op="append", tokens=4093, heads=8, dim=128, page=32, bits=8,
             rotary=128, interleaved=False, padded=29),
        # the largest append: 4096 tokens of the Llama-7B heads into the INT4 cache
        dict(name="append_4096_int4", op="append", tokens=4096, heads=32, dim=128, page=64, bits=4,
             rotary=128, interleaved=False, padded=0),
        # one sequence, one token, short context: the call's latency
        dict(name="attend_one_short", op="attend", sequences=1, draft=1, context=200, q_heads=32, kv_heads=32,
             dim=128, page=64, bits=8, tree=False, ragged=0.0),
        # a decode batch over the INT4 cache, Llama-7B heads, unequal lengths
        dict(name="attend_decode_16_int4", op="attend", sequences=16, draft=1, context=2048, q_heads=32,
             kv_heads=32, dim=128, page=64, bits=4, tree=False, ragged=0.5),
        # one long sequence: 64 query heads (Llama-65B) on 8 shared heads, fp16 cache
        dict(name="attend_long_65536_fp16", op="attend", sequences=1, draft=1, context=65536, q_heads=64,
             kv_heads=8, dim=128, page=128, bits=16, tree=False, ragged=0.0),
        # trees of 64 drafted tokens over an INT8 cache: the tensor cores' case
        dict(name="attend_tree_64_int8", op="attend", sequences=8, draft=64, context=4096, q_heads=32,
             kv_heads=8, dim=128, page=64, bits=8, tree=True, ragged=0.25),
        # small odd trees, heads of 64, short pages, fp16
        dict(name="attend_tree_13_d64", op="attend", sequences=5, draft=13, context=1531, q_heads=16,
             kv_heads=4, dim=64, page=16, bits=16, tree=True, ragged=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 200  # flops at the rate the card makes of them while it moves a byte


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(["qk", "append", "attend", "attend"])
        dim = rng.choice([64, 128])
        if op == "qk":
            kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
            c = dict(op=op, tokens=_log(rng, 1, 8192), q_heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv,
                     dim=dim, rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3,
                     norm=rng.random() < 0.8)
        elif op == "append":
            tokens = _log(rng, 1, 8192)
            c = dict(op=op, tokens=tokens, heads=rng.choice([1, 2, 4, 5, 8, 16, 32]), dim=dim,
                     page=rng.choice([16, 32, 64, 128]), bits=rng.choice([16, 8, 4]),
                     rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3,
                     padded=rng.randrange(0, max(1, tokens // 8)))
        else:
            kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
            tree = rng.random() < 0.6
            c = dict(op=op, sequences=_log(rng, 1, 32), draft=_log(rng, 2, 64) if tree else rng.choice([1, 1, 7]),
                     context=_log(rng, 1, 65536), q_heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv, dim=dim,
                     page=rng.choice([16, 32, 64, 128]), bits=rng.choice([16, 8, 4]), tree=tree,
                     ragged=round(rng.random(), 3))
        if _cost(c) <= most[op]:
            return c


def _lengths(case):
    """Context length and drafted tokens of each sequence: the first has the most, the others fall
    short of it by a fraction of `ragged` that does not repeat."""
    ctx, draft = [], []
    for b in range(case["sequences"]):
        f = (b * 0.6180339887) % 1.0 * case["ragged"]
        ctx.append(int(case["context"] * (1 - f)))
        draft.append(max(1, int(round(case["draft"] * (1 - f)))) if case["draft"] > 1 else 1)
    return ctx, draft


def work(case):
    if case["op"] == "qk":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * n + case["tokens"] * (4 * case["rotary"] + 4), "flops": 8 * n}
    if case["op"] == "append":
        live = case["tokens"] - case["padded"]
        rows = 2 * live * case["heads"]
        b = rows * case["dim"] * (2 + case["bits"] / 8) + live * (4 * case["rotary"] + 12)
        if case["bits"] < 16:  # scales, and the values read back
            b += rows * (4 + 2 * case["dim"])
        return {"bytes": b, "flops": 6 * rows * case["dim"]}
    ctx, draft = _lengths(case)
    D, kv, qh = case["dim"], case["kv_heads"], case["q_heads"]
    row = 2 * (D * case["bits"] / 8 + (4 if case["bits"] < 16 else 0))
    b = sum((c + t) * kv * row + t * qh * (4 * D + 4) for c, t in zip(ctx, draft))
    f = sum(4 * t * qh * D * (c + (t + 1) / 2) for c, t in zip(ctx, draft))
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs
def _tables(rows, rotary, dev):
    """cos and sin [rows, rotary / 2] in fp32, from angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=dev) / rotary)
    a = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * freq
    return a.cos().float(), a.sin().float()


def _seeded(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _pool(case, heads, pages, dev):
    """Empty cache buffers: codes [pages, heads, page, row] and, below 16 bits, scales."""
    bits, dim = case["bits"], case["dim"]
    dtype, row = {16: (torch.float16, dim), 8: (torch.int8, dim), 4: (torch.uint8, dim // 2)}[bits]
    k = torch.zeros((pages, heads, case["page"], row), dtype=dtype, device=dev)
    ks = torch.zeros((pages, heads, case["page"]), dtype=torch.float32, device=dev) if bits < 16 else None
    return k, k.clone(), ks, None if ks is None else ks.clone()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _seeded(seed, dev)
    r = np.random.default_rng(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    D = case["dim"]
    if case["op"] in ("qk", "append"):
        tokens = case["tokens"]
        kv = case["kv_heads"] if case["op"] == "qk" else case["heads"]
        qh = case["q_heads"] if case["op"] == "qk" else kv
        # the QKV projection's output: rows of q heads, k heads, v heads; a few channels are large
        qkv = randn(tokens, (qh + 2 * kv) * D)
        qkv.mul_(1 + 7 * (torch.rand((1, qkv.shape[1]), generator=g, device=dev) < 0.02))
        qkv = qkv.half()
        rows = max(8192, tokens)
        cos, sin = _tables(rows, case["rotary"], dev)
        s = dict(case=case, q=qkv[:, :qh * D].unflatten(1, (qh, D)),
                 k=qkv[:, qh * D:(qh + kv) * D].unflatten(1, (kv, D)),
                 v=qkv[:, (qh + kv) * D:].unflatten(1, (kv, D)), cos=cos, sin=sin,
                 positions=torch.randint(0, rows, (tokens,), generator=g, device=dev, dtype=torch.int32))
        if case["op"] == "qk":
            for n in ("q_weight", "k_weight"):
                s[n] = (1 + 0.25 * randn(D)).abs().clamp(0.02, 4).half() if case["norm"] else None
            return s
        pages = -(-tokens // case["page"]) + 2
        s["kc"], s["vc"], s["ks"], s["vs"] = _pool(case, kv, pages, dev)
        # runs of page slots in a shuffled order of pages; padded rows have no slot
        order = torch.from_numpy(r.permutation(pages)).to(dev)
        i = torch.arange(tokens, device=dev)
        slots = order[i // case["page"]] * case["page"] + i % case["page"]
        slots[tokens - case["padded"]:] = -1
        s["slots"] = slots
        return s
    ctx, draft = _lengths(case)
    page, kv = case["page"], case["kv_heads"]
    need = [-(-(c + t) // page) for c, t in zip(ctx, draft)]
    pages = sum(need) + 3
    order = r.permutation(pages)
    table = np.zeros((len(ctx), max(need)), dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kc, vc, ks, vs = _pool(case, kv, pages, dev)
    large = 1 + 3 * (torch.rand((1, kv, 1, D), generator=g, device=dev) < 0.03)
    for p in range(0, pages, 256):
        n = min(256, pages - p)
        for c, sc, big in ((kc, ks, large), (vc, vs, None)):
            x = randn(n, kv, page, D)
            x = (x if big is None else x * big).half().float()
            codes, scale = _plain_quantise(x, case["bits"])
            c[p:p + n] = codes
            if sc is not None:
                sc[p:p + n] = scale
    total = sum(draft)
    words = -(-max(draft) // 32)
    mask = None
    if case["tree"]:
        bits = np.zeros((total, words * 32), dtype=np.uint8)
        at = 0
        for t in draft:
            for i in range(t):  # each drafted token hangs on an earlier one, or on the context
                parent = int(r.integers(-1, i)) if i else -1
                if parent >= 0:
                    bits[at + i] = bits[at + parent]
                bits[at + i, i] = 1
            at += t
        mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).to(dev)
    return dict(case=case, q=randn(total, case["q_heads"], D).half(), kc=kc, vc=vc, ks=ks, vs=vs,
                table=torch.from_numpy(table).to(dev), mask=mask,
                context=torch.tensor(ctx, dtype=torch.int32, device=dev),
                cu=torch.tensor(np.concatenate([[0], np.cumsum(draft)]), dtype=torch.int32, device=dev),
                max_draft=max(draft), max_context=max(ctx), scale=D ** -0.5)


# ------------------------------------------------------------------ plain forms
def _plain_rotate(x, cos, sin, rotary, interleaved):
    """The first `rotary` channels of x [tokens, heads, D] fp32, turned by cos, sin [tokens, rotary / 2]."""
    c, s = cos[:, None], sin[:, None]
    t = x[..., :rotary]
    a, b = (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., :rotary // 2], t[..., rotary // 2:])
    u, w = a * c - b * s, b * c + a * s
    t = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((t, x[..., rotary:]), -1)


def _plain_quantise(x, bits):
    """Codes as the cache stores them, and one scale per row, of x [..., D] fp32."""
    if bits == 16:
        return x.half(), None
    top = 7 if bits == 4 else 127
    m = x.abs().amax(-1)
    scale = m / torch.full_like(m, top)  # a tensor divisor: the division is rounded once
    code = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    code = code.round().clamp(-top, top).to(torch.int8)
    if bits == 4:
        u = code.view(torch.uint8) & 15
        code = u[..., 0::2] | (u[..., 1::2] << 4)
    return code, scale


def _plain_values(codes, scale):
    """fp32 values of stored rows."""
    if scale is None:
        return codes.float()
    if codes.dtype == torch.uint8:
        n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
        codes = n - 16 * (n > 7)
    return codes.float() * scale[..., None]


def _plain_qk(s):
    c = s["case"]
    at = s["positions"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_plain_rotate(y, cos, sin, c["rotary"], c["interleaved"]).half())
    return tuple(out)


def _plain_append(s):
    c = s["case"]
    at = s["positions"].long()
    k = _plain_rotate(s["k"].float(), s["cos"][at], s["sin"][at], c["rotary"], c["interleaved"])
    live = s["slots"] >= 0
    slot = s["slots"][live]
    page, off = slot // c["page"], slot % c["page"]
    back = []
    for x, codes, scales in ((k, s["kc"], s["ks"]), (s["v"].float(), s["vc"], s["vs"])):
        q, sc = _plain_quantise(x[live], c["bits"])
        codes[page, :, off] = q
        if c["bits"] < 16:
            scales[page, :, off] = sc
            v = torch.zeros(x.shape, dtype=torch.float16, device=x.device)
            v[live] = _plain_values(codes[page, :, off], scales[page, :, off]).half()
            back.append(v)
    return (s["kc"], s["vc"]) if c["bits"] == 16 else tuple(back)


def _plain_attend(s):
    c = s["case"]
    dev, D, kv, qh, page = s["q"].device, c["dim"], c["kv_heads"], c["q_heads"], c["page"]
    B, T, S, G = c["sequences"], s["max_draft"], s["max_context"] + s["max_draft"], qh // kv
    ctx, cu = s["context"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    pos = torch.arange(S, device=dev)[None].expand(B, S)
    have = pos < (ctx + n)[:, None]
    p = torch.where(have, s["table"].long().gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1)), 0)
    # [B, kv, S, D]
    K, V = ((_plain_values(x[p, :, pos % page], None if sc is None else sc[p, :, pos % page])).transpose(1, 2)
            for x, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
    V = V.where(have[:, None, :, None], torch.zeros((), device=dev))
    # rows of each sequence, padded to T
    t = torch.arange(T, device=dev)
    real = t[None] < n[:, None]
    row = (cu[:-1, None] + t[None]).clamp(max=s["q"].shape[0] - 1)
    Q = s["q"].float()[row].view(B, T, kv, G, D).permute(0, 2, 1, 3, 4).reshape(B, kv, T * G, D)
    j = pos - ctx[:, None]
    if s["mask"] is None:
        bit = j[:, None] <= t[None, :, None]
    else:
        m = s["mask"].long()[row]  # [B, T, words]
        jj = j.clamp(0, T - 1)
        bit = (m.gather(2, (jj // 32)[:, None].expand(B, T, S)) >> (jj % 32)[:, None]) & 1 > 0
    see = (have[:, None] & ((j < 0)[:, None] | bit))[:, None, :, None].expand(B, 1, T, G, S).reshape(B, 1, T * G, S)
    sc = (Q @ K.transpose(2, 3)) * s["scale"]
    sc = torch.where(see, sc, torch.full((), -math.inf, device=dev))
    top = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    z = e.sum(-1, keepdim=True)
    o = (e @ V) / torch.where(z > 0, z, torch.ones_like(z))
    lse = top + torch.log(z)
    o = o.view(B, kv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, qh, D)
    lse = lse.view(B, kv, T, G).permute(0, 2, 1, 3).reshape(B, T, qh)
    return o[real].half(), lse[real]


# ------------------------------------------------------------------ a pass
def run(s):
    c = s["case"]
    if own:
        import mixed_precision_quantized_quantize_b200 as q
        if c["op"] == "qk":
            return q.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], EPS, s["cos"], s["sin"],
                                  s["positions"], interleaved=c["interleaved"])
        cache = s.get("cache")
        if cache is None:  # the handle that a program keeps beside its buffers
            cache = s["cache"] = q.QuikKVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        if c["op"] == "append":
            cache.append(s["k"], s["v"], s["slots"], s["cos"], s["sin"], s["positions"],
                         interleaved=c["interleaved"])
            return (s["kc"], s["vc"]) if c["bits"] == 16 else cache.gather(s["slots"])
        return q.tree_attention(s["q"], cache, s["table"], s["context"], s["cu"], s["max_draft"],
                                s["max_context"], mask=s["mask"], scale=s["scale"], return_lse=True)
    return {"qk": _plain_qk, "append": _plain_append, "attend": _plain_attend}[c["op"]](s)


# ------------------------------------------------------------------ the definition in 64 bits
def _turn64(x, cos, sin, rotary, interleaved):
    y = x.clone()
    half = rotary // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, i, None], sin[:, i, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def exact(case, seed):
    s = prepare(case, seed)
    D = case["dim"]
    if case["op"] == "qk":
        at = s["positions"].long()
        cos, sin = s["cos"].double()[at], s["sin"].double()[at]
        out = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w.double()
            out.append(_turn64(x, cos, sin, case["rotary"], case["interleaved"]))
        return tuple(out)
    if case["op"] == "append":
        at = s["positions"].long()
        k = _turn64(s["k"].double(), s["cos"].double()[at], s["sin"].double()[at], case["rotary"],
                    case["interleaved"])
        out = []
        live = case["tokens"] - case["padded"]
        for x, codes in ((k, s["kc"]), (s["v"].double(), s["vc"])):
            x[live:] = 0
            if case["bits"] == 16:
                cache = codes.double().transpose(1, 2).flatten(0, 1)  # [slot, heads, D]
                cache[s["slots"][:live]] = x[:live]
                out.append(cache.unflatten(0, (-1, case["page"])).transpose(1, 2).contiguous())
            else:
                top = 2 ** (case["bits"] - 1) - 1
                step = x.abs().amax(-1, keepdim=True) / top
                out.append(torch.round(x / step.clamp(min=1e-300)) * step)
        return tuple(out)
    out, lse = [], []
    cu, ctx = s["cu"].tolist(), s["context"].tolist()
    G = case["q_heads"] // case["kv_heads"]
    for b in range(case["sequences"]):
        n = ctx[b] + cu[b + 1] - cu[b]
        pages = s["table"][b, :-(-n // case["page"])].long()
        kv = []
        for x, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
            x = x[pages].transpose(0, 1).flatten(1, 2)[:, :n]  # [heads, n, row]
            if case["bits"] == 4:
                low, high = (x % 16).double(), torch.div(x, 16, rounding_mode="floor").double()
                x = torch.empty((*x.shape[:2], D), dtype=torch.float64, device=x.device)
                x[..., 0::2], x[..., 1::2] = low, high
                x[x >= 8] -= 16
            x = x.double()
            if sc is not None:
                x = x * sc[pages].transpose(0, 1).flatten(1, 2)[:, :n, None].double()
            kv.append(x)
        T = cu[b + 1] - cu[b]
        see = torch.ones((T, n), dtype=torch.bool, device=x.device)
        if s["mask"] is None:
            see[:, ctx[b]:] = torch.ones((T, T), dtype=torch.bool, device=x.device).tril()
        else:
            m = s["mask"][cu[b]:cu[b + 1]].cpu().numpy().view(np.uint8)
            m = np.unpackbits(m, axis=1, bitorder="little")[:, :T]
            see[:, ctx[b]:] = torch.from_numpy(m > 0).to(x.device)
        q = s["q"][cu[b]:cu[b + 1]].double().transpose(0, 1)  # [q heads, T, D]
        o, z = [], []
        for h in range(case["q_heads"]):
            a = q[h] @ kv[0][h // G].T * s["scale"]
            a = a.masked_fill(~see, -math.inf)
            z.append(torch.logsumexp(a, -1))
            o.append(torch.softmax(a, -1) @ kv[1][h // G])
        out.append(torch.stack(o, 1))
        lse.append(torch.stack(z, 1))
    return torch.cat(out), torch.cat(lse)
