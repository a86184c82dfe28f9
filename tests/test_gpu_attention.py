"""The attention operators on a B200 against the 64-bit implementations of
attention_ref: the per-head norm with rotation, the paged cache (append and
read-back, bit for bit) and the attention of drafted tokens over it, at the
sizes, masks and lengths where they can go wrong."""
import numpy as np
import pytest
import torch

import attention_ref as ref
import mixed_precision_quantized_quantize_b200 as q
from mixed_precision_quantized_quantize_b200 import workloads as wl

pytestmark = pytest.mark.gpu
BITS = [16, 8, 4]


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return t.to("cuda") if dtype is None else t.to("cuda", dtype)


def checked():
    torch.cuda.synchronize()
    assert q.quik_sync_check() == q.QUIK_OK


def within(got, want, bound, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
    off = np.where((got == want) | (np.isnan(got) & np.isnan(want)), 0, off)
    worst = np.unravel_index(np.argmax(off - bound), off.shape)
    assert (off <= bound).all(), (f"{what}: off by {off[worst]:.3e} at {worst}, bound {bound[worst]:.3e}, got "
                                  f"{got[worst]}, want {want[worst]}")


# ------------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens,qh,kh", [(1, 1, 1), (1, 32, 8), (7, 5, 0), (3, 0, 3), (33, 32, 32), (700, 12, 4)])
@pytest.mark.parametrize("rotary,inter", [("full", False), ("full", True), ("half", False), ("part", True),
                                          ("none", False)])
def test_qk_norm_rope(D, tokens, qh, kh, rotary, inter):
    r = np.random.default_rng(tokens * 100 + qh)
    rot = {"full": D, "half": D // 2, "part": 16, "none": 0}[rotary]
    x = r.standard_normal((tokens, (qh + 2 * kh + 1) * D)) * np.exp(r.uniform(-3, 3, (tokens, 1)))
    X = dev(x.astype(np.float16))
    Q, K = X[:, :qh * D].unflatten(1, (qh, D)) if qh else X[:, :0].reshape(tokens, 0, D), None
    if kh:
        K = X[:, qh * D:(qh + kh) * D].unflatten(1, (kh, D))
    cos, sin = ref.tables(500, rot) if rot else (None, None)
    pos = r.integers(0, 500, tokens).astype(np.int32) if rot else None
    for weights in (True, False):
        w = [np.abs(1 + 0.3 * r.standard_normal(D)).astype(np.float16) if weights else None for _ in "qk"]
        got = q.qk_norm_rope(Q, K, *(None if u is None else dev(u) for u in w), 1e-5,
                             *(None if u is None else dev(u) for u in (cos, sin, pos)), interleaved=inter)
        checked()
        for g, a, u in zip(got, (Q, K), w):
            if a is not None and a.numel():
                want, bound = ref.norm_rotate(a.cpu().numpy(), u, 1e-5, cos, sin, pos, inter)
                within(g, want, bound)


def test_qk_norm_rope_one_weight_extremes_and_in_place():
    """A zero head stays zero, the largest fp16 values do not overflow the sum of
    squares, a weight may be given for q alone, and the outputs may be the inputs."""
    D, n = 128, 9
    r = np.random.default_rng(1)
    x = r.standard_normal((n, 6, D)).astype(np.float16)
    x[0] = 0
    x[1] = 65504
    x[2] = 6e-8
    cos, sin = ref.tables(64, D)
    pos = np.arange(n, dtype=np.int32) * 7
    w = (1 + 0.1 * r.standard_normal(D)).astype(np.float16)
    X = dev(x)
    Q, K = X[:, :4], X[:, 4:]
    x[1, 4:] = 30000  # the rotated pair without a norm stays within fp16
    X.copy_(dev(x))
    wq, bq = ref.norm_rotate(x[:, :4], w, 1e-6, cos, sin, pos, False)
    wk, bk = ref.norm_rotate(x[:, 4:], None, 1e-6, cos, sin, pos, False)
    out = q.qk_norm_rope(Q, K, dev(w), None, 1e-6, dev(cos), dev(sin), dev(pos), q_out=Q, k_out=K)
    checked()
    assert out[0].data_ptr() == X.data_ptr()
    within(Q, wq, bq)
    within(K, wk, bk)


def test_no_tokens():
    D = 64
    e = torch.empty((0, 4, D), dtype=torch.float16, device="cuda")
    a, b = q.qk_norm_rope(e, e)
    assert a.shape == b.shape == (0, 4, D)
    c = q.QuikKVCache.empty(2, 4, D, 16, 8)
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    c.append(e, e, slots)
    assert c.gather(slots)[0].shape == (0, 4, D)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = q.tree_attention(e, c, torch.zeros((0, 1), dtype=torch.int32, device="cuda"), z[:0], z, 0, 0)
    assert o.shape == (0, 4, D)
    checked()


# ------------------------------------------------------------------ cache
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D,heads,tokens,page", [(128, 8, 1, 16), (64, 1, 37, 32), (128, 5, 300, 64),
                                                 (64, 3, 2500, 16), (128, 32, 700, 256)])
@pytest.mark.parametrize("rot,inter", [("full", False), ("half", True), ("none", False)])
def test_append_and_gather_bit_exact(bits, D, heads, tokens, page, rot, inter):
    r = np.random.default_rng(tokens + D)
    x = (r.standard_normal((tokens, 2 * heads * D + 8)) * np.exp(r.uniform(-4, 4, (tokens, 1)))).astype(np.float16)
    x[tokens // 2, :D] = 0  # a zero row
    X = dev(x)
    K = X[:, :heads * D].unflatten(1, (heads, D))
    V = X[:, heads * D:2 * heads * D].unflatten(1, (heads, D))
    rotary = {"full": D, "half": D // 2, "none": 0}[rot]
    cos, sin = ref.tables(300, rotary) if rotary else (None, None)
    pos = r.integers(0, 300, tokens).astype(np.int32) if rotary else None
    pages = -(-tokens // page) + 2
    slots = r.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 4:
        slots[r.permutation(tokens)[:tokens // 5]] = -1
    c = q.QuikKVCache.empty(pages, heads, D, page, bits)
    for t in (c.k, c.v):
        t.fill_(3)
    c.append(K, V, dev(slots), *(None if u is None else dev(u) for u in (cos, sin, pos)), interleaved=inter)
    checked()
    live = slots >= 0
    for src, buf, sc, turned in ((K, c.k, c.k_scale, True), (V, c.v, c.v_scale, False)):
        a = src.cpu().numpy()
        y = ref.rotate(a, cos if turned else None, sin, pos, inter, np.float32)[live]
        want = np.full(buf.shape, 3, buf.cpu().numpy().dtype)
        at = (slots[live] // page, slice(None), slots[live] % page)
        if bits == 16:
            want[at] = y.astype(np.float16)
            assert np.array_equal(buf.cpu().numpy().view(np.uint16), want.view(np.uint16))
            back = want[at]
        else:
            codes, scale = ref.quantise(y, bits)
            want[at] = ref.pack4(codes) if bits == 4 else codes
            assert np.array_equal(buf.cpu().numpy(), want)
            ws = np.zeros(sc.shape, np.float32)
            ws[at] = scale
            assert np.array_equal(sc.cpu().numpy().view(np.uint32), ws.view(np.uint32))
            back = (codes.astype(np.float32) * scale[..., None]).astype(np.float16)
        got = c.gather(dev(slots))[0 if turned else 1].cpu().numpy()
        assert np.array_equal(got[live].view(np.uint16), back.view(np.uint16))
        assert not got[~live].any()
    checked()


@pytest.mark.parametrize("bits", [8, 4])
def test_append_ties_and_tiny_and_non_finite_rows(bits):
    """Quotients at half-integers round to even, magnitudes near fp32's smallest
    keep the IEEE rule, and a row with an infinity or NaN reads as NaN."""
    D, top = 64, 127 if bits == 8 else 7
    x = np.zeros((6, 1, D), np.float16)
    x[0, 0] = np.resize([0.5, 1.5, -2.5, 3.5, -0.5, 2.5], D)
    x[0, 0, 7] = top            # scale 1: the others are exact ties
    x[1, 0] = 6e-8              # smallest subnormal
    x[2, 0, 3] = np.inf
    x[3, 0, 5] = np.nan
    x[4, 0, :8] = [65504, -65504, 1, 0, 516, -516, 257.875, 32752]
    x[5, 0] = np.linspace(-1, 1, D)
    cos = np.full((1, D // 2), 1e-32, np.float32)  # tiny but finite quotients
    sin = np.full((1, D // 2), 3e-33, np.float32)
    pos = np.zeros(6, np.int32)
    for rotated in (False, True):
        c = q.QuikKVCache.empty(1, 1, D, 16, bits)
        t = [dev(u) for u in (cos, sin, pos)] if rotated else [None] * 3
        c.append(dev(x), dev(x), torch.arange(6, device="cuda"), *t)
        checked()
        with np.errstate(invalid="ignore", over="ignore"):
            y = ref.rotate(x, cos if rotated else None, sin, pos, False, np.float32)
            codes, scale = ref.quantise(y[:2], bits)
            codes2, scale2 = ref.quantise(y[4:], bits)
        got, gs = c.k[0, 0, :6].cpu().numpy(), c.k_scale[0, 0, :6].cpu().numpy()
        got = ref.unpack4(got) if bits == 4 else got
        assert np.array_equal(got[:2], codes[:, 0]) and np.array_equal(got[4:], codes2[:, 0])
        assert np.array_equal(gs[:2], scale[:, 0]) and np.array_equal(gs[4:], scale2[:, 0])
        assert not np.isfinite(gs[2]) and np.isnan(gs[3]) and not got[2:4].any()
        k, _ = c.gather(torch.arange(6, device="cuda"))
        assert torch.isnan(k[2:4]).all()


# ------------------------------------------------------------------ attention
class Case:
    """A filled cache with a shuffled page table, and drafted tokens over it."""

    def __init__(self, bits, D, heads, G, page, ctx, draft, tree, seed=0, before=0, after=0, spread=1.0):
        r = self.r = np.random.default_rng(seed)
        self.bits, self.D, self.heads, self.G, self.page = bits, D, heads, G, page
        self.ctx, self.draft = np.array(ctx, np.int32), np.array(draft, np.int32)
        self.cu = (before + np.concatenate([[0], np.cumsum(draft)])).astype(np.int32)
        self.rows = int(self.cu[-1]) + after
        need = [-(-(int(a) + int(b)) // page) for a, b in zip(ctx, draft)]
        pages = sum(need) + 2
        order = r.permutation(pages)
        self.table = np.zeros((len(ctx), max(need + [1])), np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = q.QuikKVCache.empty(pages, heads, D, page, bits)
        x = [(r.standard_normal((pages, heads, page, D)) * np.exp(spread * r.standard_normal((pages, heads, page, 1))))
             .astype(np.float16) for _ in "kv"]
        for y, buf, sc in zip(x, (self.cache.k, self.cache.v), (self.cache.k_scale, self.cache.v_scale)):
            if bits == 16:
                buf.copy_(dev(y))
            else:
                c, s = ref.quantise(y, bits)
                buf.copy_(dev(ref.pack4(c) if bits == 4 else c))
                sc.copy_(dev(s))
        self.q = r.standard_normal((self.rows, heads * G, D)).astype(np.float16)
        self.mask = None
        if tree:
            words = max(1, -(-max(draft) // 32))
            self.mask = np.zeros((self.rows, words), np.uint32)
            for b, n in enumerate(draft):
                self.mask[self.cu[b]:self.cu[b + 1]] = ref.tree_mask(int(n), r, words)
        self.scale = D ** -0.5

    def run(self, max_context=None, **more):
        m = None if self.mask is None else dev(self.mask.view(np.int32))
        return q.tree_attention(dev(self.q), self.cache, dev(self.table), dev(self.ctx), dev(self.cu),
                                int(max(self.draft)), int(max(self.ctx)) if max_context is None else max_context,
                                mask=m, scale=self.scale, return_lse=True, **more)

    def reference(self):
        c = self.cache
        kv = [ref.values(b.cpu().numpy(), None if s is None else s.cpu().numpy(), self.bits)
              for b, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
        return ref.attention(self.q, *kv, self.page, self.table, self.ctx, self.cu, self.mask, self.scale)

    def check(self, max_context=None):
        out, lse = self.run(max_context)
        checked()
        o, z, bo, bz = self.reference()
        live = slice(self.cu[0], self.cu[-1])
        within(out[live], o[live], bo[live], "out")
        within(lse[live], z[live], bz[live], "lse")
        return out, lse


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,G,page,ctx,draft,tree", [
    (1, 1, 16, [1], [1], False),                    # one token, one cached
    (2, 1, 64, [0, 0], [1, 1], False),              # an empty context: the token sees itself
    (3, 5, 16, [31, 32, 33, 0], [1, 1, 1, 1], False),
    (2, 4, 32, [100, 0, 257], [5, 0, 3], True),     # a sequence without new tokens
    (1, 8, 16, [63, 7], [17, 33], True),            # a tree past one mask word
    (2, 2, 64, [130], [64], True),
    (1, 1, 128, [5, 700], [40, 1], False),          # a chunk of a prompt beside a single token
    (1, 16, 256, [300], [2], True),
    (1, 3, 16, [17], [70], True),                   # three words of mask, 210 rows
    (1, 1, 16, [0], [150], False),                  # a whole prompt
])
def test_attention(bits, D, heads, G, page, ctx, draft, tree):
    Case(bits, D, heads, G, page, ctx, draft, tree, seed=len(ctx) + G).check()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("ctx,draft,G", [([2000, 1], [1, 1], 1), ([1500, 40, 333], [3, 20, 9], 4),
                                         ([900], [64], 2), ([1100, 5], [70, 100], 4)])
def test_attention_split_over_the_context(bits, ctx, draft, G):
    """A large hint splits the cached tokens over many CTAs, more than some
    sequences have tiles; with no hint there is one.  Both are right."""
    c = Case(bits, 128, 1, G, 64, ctx, draft, True, seed=3)
    a = c.check(max_context=1 << 20)
    b = c.check(max_context=0)
    assert torch.allclose(a[0].float(), b[0].float(), rtol=4 * ref.HALF_F16, atol=2e-3)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,draft", [(3, [3, 2]), (4, [5, 1]), (1, [24, 30]), (2, [16, 9]), (4, [16, 3]), (5, [13, 1])])
def test_attention_for_long_and_for_short_contexts(bits, D, G, draft):
    """9 to 65 rows of a key head: the longest context that the call names chooses the
    kernel and the number of pieces, not the result."""
    c = Case(bits, D, 1, G, 64, [2100, 70], draft, True, seed=17)
    for hint in (None, 100, 1 << 17):
        c.check(hint)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [90, 230])
def test_many_short_sequences(bits, D, most):
    """More (sequence, key head) pairs than the GPU holds CTAs: contexts that a warp
    takes whole and ones that a CTA takes; some sequences without new tokens."""
    r = np.random.default_rng(most)
    ctx, draft = r.integers(0, most, 200), r.integers(0, 3, 200)
    ctx[7], draft[:9] = most, [2, 1, 0, 0, 1, 2, 1, 2, 0]
    c = Case(bits, D, 4, 2, 32, ctx.tolist(), draft.tolist(), True, seed=29)
    c.check()
    c.check(1 << 14)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128])
def test_one_visible_token_is_its_value(bits, D):
    """A row that sees one token alone: the weight's own rounding cancels, and the output
    is that token's value, rounded once.  (The sums and the quotient take a few steps of
    2^-24, so it may fall on the other side of a tie: one step of fp16 at most.)"""
    c = Case(bits, D, 4, 1, 16, [0] * 40, [1] * 40, False, seed=37)
    out, _ = c.run()
    checked()
    v = ref.values(c.cache.v.cpu().numpy(), c.cache.v_scale.cpu().numpy(), bits)
    want = np.stack([v[c.table[b, 0], :, 0] for b in range(40)])
    got = out.cpu().numpy().astype(np.float64)
    step = np.spacing(np.abs(want).astype(np.float16)).astype(np.float64)
    assert (np.abs(got - want) <= step * (0.5 + 2.0 ** -9)).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("ctx", [0, 40, 150, 260, 500, 765])
def test_one_sequence_by_the_warps_of_a_cta(bits, ctx):
    """One token over contexts that a CTA's warps share, some with less than a tile each."""
    for D in (64, 128):
        Case(bits, D, 3, 4, 16, [ctx], [1], False, seed=31).check()
        Case(bits, D, 2, 2, 64, [ctx, 1], [3, 4], True, seed=31).check()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D,G,ctx,draft", [(128, 2, [100, 0], [413, 7]), (64, 3, [70], [301]), (128, 1, [0], [257])])
def test_chunks_of_a_prompt(bits, D, G, ctx, draft):
    """Several blocks of rows, each of which sees the tokens up to its own last one."""
    c = Case(bits, D, 2, G, 16, ctx, draft, False, seed=23)
    c.check()
    c.check(1 << 16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,draft", [(2, 5), (3, 12), (4, 16), (2, 64)])
def test_infinity_in_values_of_a_long_context(D, G, draft):
    """Infinities and NaN among the drafted tokens' fp16 values, over a context for
    which other kernels are taken than for a short one."""
    c = Case(16, D, 1, G, 32, [2070], [draft], True, seed=19)
    clean, _ = c.run()
    seen = torch.zeros(draft, dtype=torch.bool)
    for bad, x in ((1, float("inf")), (draft - 2, float("nan")), (draft // 2, -float("inf"))):
        pos = 2070 + bad
        c.cache.v[int(c.table[0, pos // 32]), 0, pos % 32, bad % D] = x
        seen |= torch.from_numpy((c.mask[:, bad // 32] >> np.uint32(bad % 32)) & 1 > 0)
    out, _ = c.run()
    checked()
    assert torch.equal(out[~seen], clean[~seen])
    chan = sorted({1, draft - 2, draft // 2})
    assert not torch.isfinite(out[seen][..., chan].float()).all(-1).any()
    rest = [i for i in range(D) if i not in chan]
    assert torch.equal(out[..., rest], clean[..., rest])


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("hint", [0, 1 << 18])
def test_attention_rows_that_see_nothing(bits, hint):
    """No context and no bits: zeros and lse = -inf; a row that sees one token
    gives that token's value."""
    c = Case(bits, 64, 2, 2, 16, [0, 40], [6, 4], True, seed=5)
    c.mask[:] = 0
    c.mask[3, 0] = 1 << 5
    out, lse = c.check(hint)
    assert not out[:3].any() and torch.isinf(lse[:3]).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("draft", [3, 24, 70])
def test_unseen_rows_have_no_influence(bits, draft):
    """Infinities, NaN and the types' largest values in the rest of a page, in
    pages of nobody and in drafted tokens that a row does not see; the rows that
    see such a token get what the formula gives."""
    c = Case(bits, 128, 1, 2, 32, [45, 9], [draft, 5], True, seed=7)
    clean, _ = c.check()
    bad = 1  # drafted token 1 of each sequence
    seen = (c.mask[:, 0] >> bad) & 1 > 0
    k, v, ks, vs = c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale
    used = {(int(c.table[b, p // 32]), p % 32) for b in range(2) for p in range(c.ctx[b] + c.draft[b])
            if p != c.ctx[b] + bad}
    junk = [(p, o) for p in range(k.shape[0]) for o in range(32) if (p, o) not in used]
    for n, (p, o) in enumerate(junk):
        if bits == 16:
            k[p, :, o] = (float("nan"), float("inf"), -float("inf"), 65504.0)[n % 4]
            v[p, :, o] = (float("inf"), float("nan"), 65504.0, -float("inf"))[n % 4]
        else:
            ks[p, :, o] = (float("nan"), float("inf"), 3e38)[n % 3]
            vs[p, :, o] = (float("inf"), float("nan"), float("inf"))[n % 3]
    out, lse = c.run()
    checked()
    assert torch.equal(out[~dev(seen)], clean[~dev(seen)])
    if bits != 16:  # its scale is infinite or NaN in every channel
        assert not torch.isfinite(out[dev(seen)].float()).any()


# (query heads a key head, new tokens, context, hint): a warp an item, a CTA an item, the stream
# and its join; 16 and 32 rows by the warps, with and without splits; one and two blocks of
# 128 rows by the tensor cores, with and without splits, several blocks of two
FORMS = [(2, 3, 45, 0), (1, 8, 200, 200), (2, 4, 45, 1 << 16), (2, 8, 45, 0), (3, 5, 45, 1 << 17), (2, 16, 45, 0),
         (2, 64, 45, 0), (1, 100, 2100, None), (2, 100, 45, 0), (4, 60, 2100, 1 << 17), (3, 200, 45, 0)]


def place(c, b, i):
    """Page and offset of new token i of sequence b."""
    p = int(c.ctx[b]) + i
    return int(c.table[b, p // c.page]), p % c.page


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,draft,ctx,hint", FORMS)
@pytest.mark.parametrize("tree", [False, True])
def test_unseen_value_scales_have_no_influence(bits, D, G, draft, ctx, hint, tree):
    """A finite scale of any size at a token that a row does not see (a sibling branch, a
    later token of a chunk, a slot that was never written) leaves that row as it was."""
    c = Case(bits, D, 1, G, 32, [ctx, 9], [draft, 2], tree, seed=41, spread=0.3)
    clean, clean_lse = c.run(hint)
    checked()
    bad = draft // 2  # a new token of the first sequence, unseen by the rows before it at least
    if tree:
        seen = (c.mask[:, bad // 32] >> np.uint32(bad % 32)) & 1 > 0
        seen[c.cu[1]:] = False
    else:
        seen = np.zeros(c.rows, bool)
        seen[bad:draft] = True
    blind = dev(~seen)
    page, at = place(c, 0, bad)
    for scale in (1e3, 1e6, 1e9, 1e30, 3e38):
        c.cache.v_scale[page, :, at] = scale
        out, lse = c.run(hint)
        checked()
        assert torch.equal(out[blind], clean[blind]), scale
        assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [60, 230])
def test_unseen_value_scales_in_many_short_sequences(bits, D, most):
    """The same where a warp takes an item whole, or one stream crosses many of them: the
    second of three drafted tokens in each of 200 sequences."""
    r = np.random.default_rng(most)
    c = Case(bits, D, 4, 2, 32, r.integers(0, most, 200).tolist(), [3] * 200, True, seed=61)
    clean, _ = c.run()
    seen = dev((c.mask[:, 0] >> 1) & 1 > 0)
    for b in range(200):
        page, at = place(c, b, 1)
        c.cache.v_scale[page, :, at] = (1e3, 1e9, 1e30)[b % 3]
    for hint in (None, 1 << 14):
        out, _ = c.run(hint)
        checked()
        if hint is None:
            assert torch.equal(out[~seen], clean[~seen])
        assert torch.allclose(out[~seen].float(), clean[~seen].float(), rtol=8 * ref.HALF_F16, atol=2e-3)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("G,draft,ctx,hint", FORMS)
@pytest.mark.parametrize("tree", [False, True])
def test_appended_values_of_any_size_beside_small_ones(bits, G, draft, ctx, hint, tree):
    """Values around 1e-4 and, as a new token that some rows do not see, the largest fp16
    ones, all through append: every row within the bound of the tokens that it sees."""
    D = 128
    c = Case(bits, D, 1, G, 32, [ctx], [draft], tree, seed=43)
    n = ctx + draft
    x = 1e-4 * c.r.standard_normal((n, 2, 1, D))
    x[:, 0] *= 1e4
    bad = ctx + draft // 2
    x[bad, 1] = 65504 * np.sign(c.r.standard_normal((1, D)))
    slots = [int(c.table[0, p // 32]) * 32 + p % 32 for p in range(n)]
    X = dev(x.astype(np.float16))
    c.cache.append(X[:, 0], X[:, 1], dev(np.array(slots, np.int64)))
    out, lse = c.run(hint)
    checked()
    kv = [ref.values(b.cpu().numpy(), s.cpu().numpy(), bits)
          for b, s in ((c.cache.k, c.cache.k_scale), (c.cache.v, c.cache.v_scale))]
    o, z, bo, bz = ref.attention(c.q, *kv, 32, c.table, c.ctx, c.cu, c.mask, c.scale, seen_only=True)
    within(out, o, bo, "out")
    within(lse, z, bz, "lse")


@pytest.mark.parametrize("draft", [8, 15, 90])
def test_seen_infinity_in_fp16_values(draft):
    """An infinity in a value that some rows see: those rows get it, in its channel only."""
    c = Case(16, 64, 1, 1, 16, [20], [draft], True, seed=9)
    pos = 20 + 2
    c.cache.v[int(c.table[0, pos // 16]), 0, pos % 16, 5] = float("inf")
    seen = torch.from_numpy((c.mask[:, 0] >> 2) & 1 > 0)
    out, _ = c.run()
    checked()
    assert torch.isinf(out[seen, :, 5]).all() and torch.isfinite(out[~seen]).all()
    assert torch.isfinite(out[seen][..., :5]).all() and torch.isfinite(out[seen][..., 6:]).all()
    o, _, bo, _ = c.reference()
    rest = [i for i in range(64) if i != 5]
    within(out[..., rest], o[..., rest], bo[..., rest])


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("hint", [0, 1 << 18])
def test_rows_of_no_sequence_are_left(bits, hint):
    c = Case(bits, 64, 2, 3, 16, [50, 3], [4, 2], True, seed=11, before=3, after=5)
    out = torch.full((c.rows, 6, 64), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((c.rows, 6), 7.0, device="cuda")
    c.run(hint, out=out, lse=lse)
    checked()
    o, z, bo, bz = c.reference()
    live = slice(3, 9)
    within(out[live], o[live], bo[live])
    within(lse[live], z[live], bz[live])
    for t in (out, lse):
        assert (t[:3] == 7).all() and (t[9:] == 7).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_value_scales_of_very_different_size(bits):
    """Rows whose scales lie 2^20 apart within and across tiles: the result
    follows the softmax weights, not the order of the scales."""
    c = Case(bits, 128, 1, 1, 64, [500], [4], False, seed=13)
    s = 2.0 ** c.r.uniform(-12, 8, c.cache.v_scale.shape)
    c.cache.v_scale.copy_(dev(s.astype(np.float32)))
    c.check()
    c.check(1 << 18)
    c.cache.v_scale[:, :, :] = dev(np.sort(s.reshape(-1)).reshape(s.shape).astype(np.float32))
    c.check()


@pytest.mark.parametrize("bits", BITS)
def test_large_scores(bits):
    """Scores of thousands: the maximum is taken off before the exponential."""
    c = Case(bits, 64, 1, 2, 16, [90], [5], True, seed=15)
    c.scale = 40.0
    c.check()
    c.scale = -40.0
    c.check()


def test_offsets_past_32_bits():
    """A cache of 4.5 GB of codes each for K and V: its last pages lie past 2^32 bytes."""
    D, heads, page = 128, 8, 256
    pages = (9 << 29) // (D * heads * page)
    k, v = (torch.zeros((pages, heads, page, D), dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros((pages, heads, page), dtype=torch.float32, device="cuda") for _ in "kv")
    cache = q.QuikKVCache(k, v, ks, vs)
    r = np.random.default_rng(17)
    n = 300
    x = r.standard_normal((n, 2, heads, D)).astype(np.float16)
    table = np.array([[pages - 1, pages - 2]], np.int32)
    slots = np.array([int(table[0, i // page]) * page + i % page for i in range(n)], np.int64)
    X = dev(x)
    cache.append(X[:, 0], X[:, 1], dev(slots))
    back = cache.gather(dev(slots))
    Q = r.standard_normal((1, heads, D)).astype(np.float16)
    out, lse = q.tree_attention(dev(Q), cache, dev(table), dev(np.array([n - 1], np.int32)),
                                dev(np.array([0, 1], np.int32)), 1, n, return_lse=True)
    checked()
    kv = []
    for i in range(2):
        c, s = ref.quantise(x[:, i], 8)
        assert np.array_equal(back[i].cpu().numpy(), (c.astype(np.float32) * s[..., None]).astype(np.float16))
        y = np.zeros((2, heads, page, D))
        full = c.astype(np.float64) * s[..., None]
        for t in range(n):
            y[t // page, :, t % page] = full[t]
        kv.append(y)
    o, z, bo, bz = ref.attention(Q, *kv, page, np.array([[0, 1]]), [n - 1], [0, 1], None, D ** -0.5)
    within(out, o, bo)
    within(lse, z, bz)


def test_indices_out_of_range_are_reported():
    """Bad pages, lengths, slots and positions are never used as addresses: the
    call completes, the rest of its results stand, and the check reports it."""
    c = Case(8, 64, 2, 1, 16, [40, 20], [2, 2], False, seed=19)
    c.check()
    o, _, bo, _ = c.reference()
    # the other sequence's rows: right whatever this one holds (their last bits
    # go by how all the tokens of the call are shared out)
    stands = lambda out: within(out[:2], o[:2], bo[:2])  # noqa: E731
    want = c.table.copy()
    for bad in (-1, c.cache.pages, 1 << 30):
        c.table = want.copy()
        c.table[1, 0] = bad
        out, _ = c.run()
        assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG
        stands(out)
        assert torch.isfinite(out).all()
    c.table = want
    for field, value in (("ctx", -5), ("ctx", 1 << 30)):
        keep = c.ctx.copy()
        c.ctx[1] = value
        out, _ = c.run(max_context=64)
        assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG
        stands(out)
        c.ctx = keep
    for cu in ([0, 2, 1], [-3, 2, 4], [0, 2, 900], [0, 4, 4]):
        keep = c.cu.copy()
        c.cu = np.array(cu, np.int32)
        c.run()
        assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG, cu
        c.cu = keep
    x = torch.randn((3, 2, 64), device="cuda").half()
    before = c.cache.k.clone()
    limit = c.cache.pages * 16
    c.cache.append(x, x, torch.tensor([limit, 1 << 40, -1], device="cuda"))
    assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG
    assert torch.equal(before, c.cache.k)
    k, v = c.cache.gather(torch.tensor([limit, 1 << 40, -7], device="cuda"))
    assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG and not k.any() and not v.any()
    cos, sin = (dev(t) for t in ref.tables(8, 64))
    for p in (-1, 8):
        pos = torch.tensor([0, p, 0], dtype=torch.int32, device="cuda")
        a, _ = q.qk_norm_rope(x, None, None, None, 1e-5, cos, sin, pos)
        assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG
        assert torch.equal(a, x)  # row 0 of the tables: no turn
    checked()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("G,draft,ctx,hint", FORMS)
@pytest.mark.parametrize("tree", [False, True])
def test_a_bad_page_is_reported_by_every_form(bits, G, draft, ctx, hint, tree):
    """A page number out of range, in the context or among the last new tokens of a chunk
    of several row blocks: never used as an address, counted, and nothing to the rows
    that see none of its tokens."""
    c = Case(bits, 64, 1, G, 32, [ctx, 9], [draft, 2], tree, seed=47)
    clean, clean_lse = c.run(hint)
    checked()
    keep = c.table.copy()
    for column in (0, (ctx + draft - 1) // 32):
        tokens = np.arange(32 * column, 32 * column + 32) - ctx  # as new tokens
        sees = np.zeros(c.rows, bool)
        for i in range(draft):
            bits_of = ref.visible(None if c.mask is None else c.mask[i], i, draft)
            sees[i] = (tokens < 0).any() or any(bits_of[j] for j in tokens if 0 <= j < draft)
        for bad in (-1, c.cache.pages, 1 << 30):
            c.table = keep.copy()
            c.table[0, column] = bad
            out, lse = c.run(hint)
            assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG, (column, bad)
            assert torch.equal(out[dev(~sees)], clean[dev(~sees)])
            assert torch.equal(lse[dev(~sees)], clean_lse[dev(~sees)])
            assert torch.isfinite(out).all()
    checked()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("draft,hint", [(1, 0), (1, 1 << 16), (20, 0), (40, 0), (150, 0), (150, 1 << 16)])
@pytest.mark.parametrize("tree", [False, True])
def test_no_pages_and_lengths_past_all_pages(bits, draft, hint, tree):
    """A page table without columns, and a context of 2^31 - 1: every token past the
    pages is unseen and counted, in each form of the kernel; nothing else changes."""
    c = Case(bits, 64, 1, 2, 16, [33, 20], [draft, draft], tree, seed=21)
    o, _, bo, _ = c.reference()
    c.ctx[1] = 2**31 - 1
    out, lse = c.run(hint)
    assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG
    within(out[:draft], o[:draft], bo[:draft])
    assert not torch.isnan(out).any()
    c.ctx[1] = 20
    c.table = c.table[:, :0]
    out, lse = c.run(hint)
    assert q.quik_sync_check() == q.QUIK_ERR_INVALID_ARG
    assert not out.any() and torch.isneginf(lse).all()
    checked()


def test_same_result_twice_and_on_another_stream():
    c = Case(4, 128, 4, 4, 64, [900, 333], [9, 2], True, seed=21)
    a, la = c.run(1 << 18)
    b, lb = c.run(1 << 18)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    d, ld = c.run(1 << 18, stream=s)
    s.synchronize()
    checked()
    for x, y in ((a, b), (la, lb), (a, d), (la, ld)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits", BITS)
def test_raw_entry_points_give_the_same_bits(bits):
    """The C calls with their structs, rows by their strides, on another stream."""
    D, heads, G, n, page = 64, 2, 3, 70, 32
    r = np.random.default_rng(53)
    X = dev(r.standard_normal((n, (heads * G + 2 * heads) * D + 8)).astype(np.float16))
    Y = X[:, :-8].unflatten(1, (-1, D))
    Q, K, V = Y.split([heads * G, heads, heads], dim=1)
    w = dev(np.abs(1 + 0.2 * r.standard_normal(D)).astype(np.float16))
    cos, sin = (dev(t) for t in ref.tables(n, D))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, device="cuda")
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    ctx, cu = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([n - 5], [n - 5, n]))
    mask = torch.from_numpy(np.concatenate([np.zeros((n - 5, 1), np.uint32), ref.tree_mask(5, r)]).view(np.int32)).cuda()
    a, b = (q.QuikKVCache.empty(3, heads, D, page, bits) for _ in "ab")
    out, lse = (torch.zeros(s, dtype=t, device="cuda") for s, t in (((n, heads * G, D), torch.float16),
                                                                  ((n, heads * G), torch.float32)))
    qa, ka = q.qk_norm_rope(Q, K, w, None, 1e-5, cos, sin, pos)
    a.append(ka, V, slots)
    back = a.gather(slots)
    q.tree_attention(qa, a, table, ctx, cu, 5, n - 5, mask=mask, out=out, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qb, kb, back_k, back_v = (torch.empty_like(t) for t in (qa, ka, *back))
    out_b, lse_b = torch.zeros_like(out), torch.zeros_like(lse)
    shape = q.quik_heads(n, heads * G, heads, D, D, 0, n)
    q.quik_qk_norm_rope(shape, Q, K, w, None, 1e-5, cos, sin, pos, qb, kb, stream=side)
    q.quik_kv_append(q.quik_heads(n, 0, heads, D, 0, 0, 0), b.struct, kb, V, None, None, None, slots, stream=side)
    q.quik_kv_gather(b.struct, slots, back_k, back_v, stream=side)
    call = q.quik_attention(n, 1, heads * G, 5, 3, n - 5, 1, D ** -0.5)
    ws = torch.empty(max(1, q.quik_attention_workspace_size(call, b.struct)), dtype=torch.uint8, device="cuda")
    q.quik_tree_attention(call, b.struct, qb, table, ctx, cu, mask, out_b, lse_b, ws, stream=side)
    side.synchronize()
    checked()
    for x, y in zip((qa, ka, *back, out, lse), (qb, kb, back_k, back_v, out_b, lse_b)):
        assert torch.equal(x, y)
    with pytest.raises(ValueError, match="heads of a token"):
        q.quik_kv_gather(b.struct, slots, back_k.transpose(1, 2).contiguous().transpose(1, 2), back_v)
    call.mask_words = 0  # fewer than five drafted tokens need
    with pytest.raises(q.QuikError):
        q.quik_tree_attention(call, b.struct, qb, table, ctx, cu, mask, out_b, lse_b, ws)


class Guarded:
    """Tensors with 4 KB of a pattern before and after each."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((4096 + -(-n // 16) * 16 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((buf, n))
        return buf[4096:4096 + n].view(dtype).view(shape)

    def untouched(self):
        return all((b[:4096] == 0xA5).all() and (b[4096 + n:] == 0xA5).all() for b, n in self.all)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,draft,ctx,hint", FORMS)
def test_guards_around_every_output_are_untouched(bits, D, G, draft, ctx, hint):
    """Guard bytes around the cache, its scales, the outputs and the workspace of one step:
    norm and rotation, append into all of the cache, read-back, attention."""
    heads, page, g = 3, 16, Guarded()
    n = ctx + draft
    pages = -(-n // page)
    r = np.random.default_rng(59)
    X = dev(r.standard_normal((n, heads * G + 2 * heads, D)).astype(np.float16))
    Q, K, V = X.split([heads * G, heads, heads], dim=1)
    row, dtype = {16: (D, torch.float16), 8: (D, torch.int8), 4: (D // 2, torch.uint8)}[bits]
    cache = q.QuikKVCache(*(g((pages, heads, page, row), dtype) for _ in "kv"),
                          *((g((pages, heads, page), torch.float32) for _ in "kv") if bits < 16 else (None, None)))
    cos, sin = (dev(t) for t in ref.tables(n, D))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qo, ko = g((n, heads * G, D), torch.float16), g((n, heads, D), torch.float16)
    q.qk_norm_rope(Q, K, None, None, 1e-5, cos, sin, pos, q_out=qo, k_out=ko)
    slots = torch.arange(n, device="cuda")
    cache.append(ko, V, slots)
    cache.gather(slots, *(g((n, heads, D), torch.float16) for _ in "kv"))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    context, cu = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([ctx], [0, draft]))
    out, lse = g((draft, heads * G, D), torch.float16), g((draft, heads * G), torch.float32)
    for words in (0, -(-draft // 32)):
        call = q.quik_attention(draft, 1, heads * G, draft, pages, ctx if hint is None else hint, words, D ** -0.5)
        mask = dev(ref.tree_mask(draft, r, words).view(np.int32)) if words else None
        ws = g((q.quik_attention_workspace_size(call, cache.struct),), torch.uint8)
        q.quik_tree_attention(call, cache.struct, qo[ctx:], table, context, cu, mask, out, lse, ws)
    checked()
    assert g.untouched()


def test_captured_and_replayed_with_other_lengths():
    """A captured call follows the lengths, pages and masks that its tensors hold
    at replay."""
    c = Case(8, 128, 2, 2, 16, [200, 100], [4, 4], True, seed=23)
    t = [dev(x) for x in (c.q, c.table, c.ctx, c.cu, c.mask.view(np.int32))]
    call = lambda: q.tree_attention(t[0], c.cache, t[1], t[2], t[3], 4, 200, mask=t[4], scale=c.scale,  # noqa: E731
                                    return_lse=True)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call()
    for ctx, cu, hint in (([200, 100], [0, 4, 8], 0), ([3, 77], [0, 1, 5], 0), ([0, 150], [0, 4, 4], 0)):
        c.ctx[:], c.cu[:] = ctx, cu
        c.q[:] = c.r.standard_normal(c.q.shape).astype(np.float16)
        for d, x in zip(t, (c.q, c.table, c.ctx, c.cu, c.mask.view(np.int32))):
            d.copy_(dev(x))
        g.replay()
        checked()
        o, z, bo, bz = c.reference()
        live = slice(0, cu[-1])
        within(out[live], o[live], bo[live])
        within(lse[live], z[live], bz[live])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("bits", BITS)
def test_attention_block_between_two_quantised_linears(bits):
    """QKV projection (RMS norm folded in), per-head norm and rotation in place,
    append, attention, output projection: a prompt chunk and then drafted
    trees, as a model's attention block runs them; then the same captured."""
    qh, kh, D, hidden, page = 4, 2, 64, 256, 16
    r = np.random.default_rng(25)
    cfg = wl.custom_config(16, (qh + 2 * kh) * D, hidden, 32)
    d = wl.make_layer(cfg)
    gamma = wl.make_norm_weight(hidden)
    qkv_layer = q.QuikLinear(d["W"].cuda(), d["perm"].cuda(), 32, norm_weight=gamma.cuda(), norm_eps=1e-5)
    cfg2 = wl.custom_config(16, hidden, qh * D, 32)
    d2 = wl.make_layer(cfg2)
    o_layer = q.QuikLinear(d2["W"].cuda(), d2["perm"].cuda(), 32)
    qn, kn = (dev(np.abs(1 + 0.2 * r.standard_normal(D)).astype(np.float16)) for _ in "qk")
    cos, sin = (dev(t) for t in ref.tables(128, D))
    cache = q.QuikKVCache.empty(8, kh, D, page, bits)
    table = np.array([[5, 1, 7], [2, 6, 0]], np.int32)

    def block(X, ctx, cu, pos, slots, mask, most):
        Y = qkv_layer(X)
        Q, K, V = Y.unflatten(1, (-1, D)).split([qh, kh, kh], dim=1)
        q.qk_norm_rope(Q, K, qn, kn, 1e-5, cos, sin, pos, q_out=Q, k_out=K)
        cache.append(K, V, slots)
        O = q.tree_attention(Q, cache, dev_table, ctx, cu, most, 32, mask=mask)
        return Y, O, o_layer(O.flatten(1))

    dev_table = dev(table)
    steps = []  # (context, new tokens, tree)
    steps.append(([0, 0], [9, 5], False))
    steps.append(([9, 5], [6, 11], True))
    for ctx, n, tree in steps:
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        X = torch.from_numpy(r.standard_normal((cu[-1], hidden)).astype(np.float16)).cuda()
        pos = np.concatenate([c + np.arange(m) for c, m in zip(ctx, n)]).astype(np.int32)
        slots = np.concatenate([table[b, (c + np.arange(m)) // page] * page + (c + np.arange(m)) % page
                                for b, (c, m) in enumerate(zip(ctx, n))]).astype(np.int64)
        mask = np.concatenate([ref.tree_mask(m, r, 1) for m in n]) if tree else None
        args = (X, dev(np.array(ctx, np.int32)), dev(cu), dev(pos), dev(slots),
                None if mask is None else dev(mask.view(np.int32)), max(n))
        Y, O, Z = block(*args)
        checked()
        # Y holds the normalised, rotated q and k in place now
        Qn = Y.cpu().numpy().reshape(cu[-1], -1, D)[:, :qh]
        kv = [ref.values(b.cpu().numpy(), None if s is None else s.cpu().numpy(), bits)
              for b, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        o, _, bo, _ = ref.attention(Qn, *kv, page, table, ctx, cu, mask, D ** -0.5)
        within(O, o, bo)
        raw = qkv_layer(X).cpu().numpy().reshape(cu[-1], -1, D)
        want, bound = ref.norm_rotate(raw[:, qh:qh + kh], kn.cpu().numpy(), 1e-5, cos.cpu().numpy(),
                                      sin.cpu().numpy(), pos, False)
        within(Y.unflatten(1, (-1, D))[:, qh:qh + kh], want, bound)
        assert torch.equal(Z, o_layer(O.flatten(1).clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y2, O2, Z2 = block(*args)
        Y2.zero_(), O2.zero_(), Z2.zero_()
        g.replay()
        checked()
        assert torch.equal(Y, Y2) and torch.equal(O, O2) and torch.equal(Z, Z2)
