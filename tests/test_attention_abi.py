"""Argument checks of the attention entry points, without a GPU: every refusal
comes before anything is launched (the addresses are made up and never
dereferenced)."""
import ctypes

import pytest
import torch

import mixed_precision_quantized_quantize_b200 as q
from mixed_precision_quantized_quantize_b200 import build as qbuild

G = 0x10000   # an aligned address
ODD = 0x10008  # not 16-byte aligned


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return q.lib()


def heads(tokens=4, q_heads=8, kv_heads=2, head_dim=128, rotary_dim=128, interleaved=0, table_rows=64):
    return q.quik_heads(tokens, q_heads, kv_heads, head_dim, rotary_dim, interleaved, table_rows)


def cache(kv_type=q.QUIK_KV_INT8, heads=2, head_dim=128, page_size=64, pages=9, reserved=0, k=G, v=G,
          k_scale=G, v_scale=G):
    return q.quik_kv_cache(kv_type, heads, head_dim, page_size, pages, reserved, k, v, k_scale, v_scale)


def attention(tokens=4, sequences=2, q_heads=8, max_tokens=3, max_pages=4, max_context=100, mask_words=1,
              scale=0.1):
    return q.quik_attention(tokens, sequences, q_heads, max_tokens, max_pages, max_context, mask_words, scale)


BAD_HEADS = [(dict(tokens=-1), "I"), (dict(q_heads=-1), "I"), (dict(kv_heads=-1), "I"),
             (dict(head_dim=0), "I"), (dict(head_dim=96), "U"), (dict(head_dim=256), "U"),
             (dict(rotary_dim=-16), "I"), (dict(rotary_dim=24), "I"), (dict(rotary_dim=144), "I"),
             (dict(interleaved=2), "I"), (dict(table_rows=0), "I"), (dict(q_heads=5000), "U")]
STATUS = {"I": q.QUIK_ERR_INVALID_ARG, "U": q.QUIK_ERR_UNSUPPORTED}


def qk(L, h, qp=G, qs=1024, kp=G, ks=256, qg=None, kg=None, eps=1e-6, cos=G, sin=G, pos=G, qo=G, qos=1024,
       ko=G, kos=256):
    return L.quik_qk_norm_rope(None if h is None else ctypes.byref(h), qp, qs, kp, ks, qg, kg, eps, cos, sin,
                               pos, qo, qos, ko, kos, None)


def test_qk_norm_rope_refusals(L):
    assert qk(L, None) == q.QUIK_ERR_INVALID_ARG
    for bad, st in BAD_HEADS:
        assert qk(L, heads(**bad)) == STATUS[st], bad
    assert qk(L, heads(q_heads=0, kv_heads=0)) == q.QUIK_ERR_INVALID_ARG
    for bad in (dict(qp=None), dict(qp=ODD), dict(kp=None), dict(qo=None), dict(ko=ODD), dict(qs=1023),
                dict(qs=1020), dict(qs=512), dict(ks=-256), dict(qos=1028), dict(kos=128), dict(cos=None),
                dict(sin=ODD), dict(pos=None), dict(pos=G + 2), dict(qg=ODD), dict(kg=ODD),
                dict(qg=G, eps=0.0), dict(kg=G, eps=-1.0), dict(qg=G, eps=float("nan")),
                dict(qg=G, eps=float("inf")),
                dict(qs=2048)):  # in place with another stride
        assert qk(L, heads(), **bad) == q.QUIK_ERR_INVALID_ARG, bad


def test_qk_norm_rope_looks_at_nothing_of_no_heads(L):
    """Without query or key heads that side's pointers are not used: neither checked
    (nor, in the kernel, read)."""
    for none, bad in ((dict(kv_heads=0), dict(kp=ODD, ks=3, kg=ODD, ko=ODD, kos=-1)),
                      (dict(q_heads=0), dict(qp=ODD, qs=3, qg=ODD, qo=ODD, qos=-1))):
        # eps belongs to the weights in use: there are none
        assert qk(L, heads(tokens=0, **none), eps=0.0, **bad) == q.QUIK_OK
    assert qk(L, heads(kv_heads=0), kg=ODD, qp=ODD) == q.QUIK_ERR_INVALID_ARG
    assert qk(L, heads(kv_heads=0), qg=G, kg=ODD, eps=0.0) == q.QUIK_ERR_INVALID_ARG


def append(L, h, c, kp=G, ks=256, vp=G, vs=256, cos=G, sin=G, pos=G, slots=G):
    return L.quik_kv_append(None if h is None else ctypes.byref(h), None if c is None else ctypes.byref(c), kp, ks,
                            vp, vs, cos, sin, pos, slots, None)


BAD_CACHE = [(dict(kv_type=3), "I"), (dict(kv_type=-1), "I"), (dict(heads=0), "I"), (dict(head_dim=-64), "I"),
             (dict(head_dim=80), "U"), (dict(page_size=8), "I"), (dict(page_size=48), "I"),
             (dict(page_size=512), "I"), (dict(pages=0), "I"), (dict(reserved=1), "I"), (dict(heads=5000), "U")]
BAD_BUFFERS = [dict(k=None), dict(k=ODD), dict(v=None), dict(k_scale=None), dict(v_scale=ODD)]


def test_kv_append_refusals(L):
    assert append(L, None, cache()) == append(L, heads(), None) == q.QUIK_ERR_INVALID_ARG
    for bad, st in BAD_HEADS:
        if "q_heads" not in bad:
            assert append(L, heads(**bad), cache()) == STATUS[st], bad
    for bad, st in BAD_CACHE:
        assert append(L, heads(), cache(**bad)) == STATUS[st], bad
    for bad in BAD_BUFFERS:
        assert append(L, heads(), cache(**bad)) == q.QUIK_ERR_INVALID_ARG, bad
    assert append(L, heads(kv_heads=3), cache()) == q.QUIK_ERR_INVALID_ARG
    assert append(L, heads(head_dim=64, rotary_dim=64), cache()) == q.QUIK_ERR_INVALID_ARG
    for bad in (dict(kp=None), dict(vp=ODD), dict(ks=255), dict(vs=128), dict(cos=None), dict(slots=None),
                dict(slots=G + 4), dict(pos=None)):
        assert append(L, heads(), cache(), **bad) == q.QUIK_ERR_INVALID_ARG, bad


def gather(L, c, tokens=4, slots=G, kp=G, ks=256, vp=G, vs=256):
    return L.quik_kv_gather(None if c is None else ctypes.byref(c), tokens, slots, kp, ks, vp, vs, None)


def test_kv_gather_refusals(L):
    assert gather(L, None) == q.QUIK_ERR_INVALID_ARG
    for bad, st in BAD_CACHE:
        assert gather(L, cache(**bad)) == STATUS[st], bad
    for bad in BAD_BUFFERS:
        assert gather(L, cache(**bad)) == q.QUIK_ERR_INVALID_ARG, bad
    for bad in (dict(tokens=-1), dict(slots=None), dict(slots=G + 4), dict(kp=ODD), dict(vp=None), dict(ks=250),
                dict(vs=8)):
        assert gather(L, cache(), **bad) == q.QUIK_ERR_INVALID_ARG, bad


def attend(L, a, c, qp=G, qs=1024, table=G, ctx=G, cu=G, mask=G, out=G, os_=1024, lse=None, ws=G, n=1 << 40):
    return L.quik_tree_attention(None if a is None else ctypes.byref(a), None if c is None else ctypes.byref(c), qp,
                                 qs, table, ctx, cu, mask, out, os_, lse, ws, n, None)


BAD_ATTENTION = [(dict(tokens=-1), "I"), (dict(sequences=-1), "I"), (dict(q_heads=0), "I"), (dict(q_heads=9), "I"),
                 (dict(max_tokens=-1), "I"), (dict(max_pages=-1), "I"), (dict(max_context=-1), "I"),
                 (dict(mask_words=-1), "I"), (dict(scale=float("nan")), "I"), (dict(scale=float("inf")), "I"),
                 (dict(sequences=65536), "U"), (dict(q_heads=8192), "U")]


def test_tree_attention_refusals(L):
    assert attend(L, None, cache()) == attend(L, attention(), None) == q.QUIK_ERR_INVALID_ARG
    for bad, st in BAD_ATTENTION:
        assert attend(L, attention(**bad), cache()) == STATUS[st], bad
        assert L.quik_attention_workspace_size(ctypes.byref(attention(**bad)), ctypes.byref(cache())) == 0
    for bad, st in BAD_CACHE:
        assert attend(L, attention(), cache(**bad)) == STATUS[st], bad
    for bad in BAD_BUFFERS:
        assert attend(L, attention(), cache(**bad)) == q.QUIK_ERR_INVALID_ARG, bad
    for bad in (dict(qp=None), dict(qp=ODD), dict(qs=1000), dict(qs=1028), dict(table=None), dict(ctx=None),
                dict(cu=G + 1), dict(mask=G + 2), dict(out=None), dict(os_=512), dict(lse=G + 1)):
        assert attend(L, attention(), cache(), **bad) == q.QUIK_ERR_INVALID_ARG, bad
    # a mask too narrow for the drafted tokens
    assert attend(L, attention(tokens=80, max_tokens=33, mask_words=1), cache()) == q.QUIK_ERR_INVALID_ARG


def test_attention_workspace(L):
    """Few rows are shared out among workers and need a workspace; without it, or
    with less of it, the call is refused.  Many rows over a short context need none."""
    a = attention(tokens=1, sequences=1, max_tokens=1, max_context=100000, mask_words=0)
    need = L.quik_attention_workspace_size(ctypes.byref(a), ctypes.byref(cache()))
    assert need > 0
    for ws, n in ((None, 1 << 40), (G, need - 1), (ODD, 1 << 40)):
        assert attend(L, a, cache(), mask=None, ws=ws, n=n) == q.QUIK_ERR_INVALID_ARG
    a = attention(tokens=64, sequences=1, max_tokens=64, max_context=20, mask_words=2)
    assert L.quik_attention_workspace_size(ctypes.byref(a), ctypes.byref(cache())) == 0


def test_no_tokens_is_no_launch(L):
    assert qk(L, heads(tokens=0), qp=None, kp=None, qo=None, ko=None) == q.QUIK_OK
    assert append(L, heads(tokens=0), cache(), kp=None, vp=None, slots=None) == q.QUIK_OK
    assert gather(L, cache(), tokens=0, slots=None, kp=None, vp=None) == q.QUIK_OK
    for none in (dict(tokens=0), dict(sequences=0), dict(max_tokens=0)):
        assert attend(L, attention(**none), cache(), qp=None, out=None) == q.QUIK_OK


def test_python_checks():
    """The Python calls refuse what the C structs cannot express."""
    h = torch.zeros((4, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        q.qk_norm_rope(h, h)
    with pytest.raises(ValueError, match="k must be"):
        q.qk_norm_rope(h, torch.zeros((3, 2, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match="needs cos, sin and positions"):
        q.qk_norm_rope(h, h, cos=torch.zeros(4, 32))
    with pytest.raises(ValueError, match="both alike"):
        q.qk_norm_rope(h, h, cos=torch.zeros(4, 32), sin=torch.zeros(5, 32),
                       positions=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="bits"):
        q.QuikKVCache.empty(1, 1, 64, 16, 5, device="cpu")
    with pytest.raises(TypeError):
        q.QuikKVCache(torch.zeros((1, 1, 16, 64)), torch.zeros((1, 1, 16, 64)))
    c8 = torch.zeros((1, 1, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError, match="scale"):
        q.QuikKVCache(c8, c8)
    with pytest.raises(ValueError, match="scales must be"):
        q.QuikKVCache(c8, c8, torch.zeros((1, 1, 8)), torch.zeros((1, 1, 8)))
