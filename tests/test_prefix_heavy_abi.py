"""The normed append, the attention behind shared prefixes and the calls on a heavy-hitter draft cache refuse bad
arguments on the host, before anything is enqueued (CPU only: every call here fails validation first)."""
import ctypes
import math

import pytest
import torch

from long_context_self_gb300 import binding
from long_context_self_gb300 import build as lbuild

P = ctypes.c_void_p
FAKE, OTHER, ODD, NULL = P(0x10000), P(0x20000), P(0x10008), P(0)
NULL_, SHAPE, ALIGN, WS, UNSUPPORTED = -1, -2, -3, -4, -5
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return binding.lib()


def paged(**kw):
    s = dict(B=2, H_q=8, H_kv=2, d=128, page_size=16, n_pages=20, max_pages=10)
    s.update(kw)
    return binding.paged_shape(**s)


def dense(**kw):
    s = dict(B=2, H_q=8, H_kv=2, d=128, L_cap=100)
    s.update(kw)
    return binding.kv_shape(**s)


BAD_PAGED = [dict(B=0), dict(B=4097), dict(H_q=0), dict(H_kv=0), dict(H_q=9), dict(d=96), dict(page_size=0),
             dict(n_pages=0), dict(max_pages=0), dict(page_size=1 << 16, max_pages=1 << 15), dict(H_q=65536)]
BAD_DENSE = [dict(B=0), dict(B=4097), dict(H_q=0), dict(H_kv=0), dict(H_q=9), dict(d=96), dict(L_cap=0), dict(L_cap=-4)]


def test_append_refusals(lib):
    def call(s=None, n=4, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, qw=FAKE, kw=FAKE, eps=1e-6, length=FAKE,
             n_new=NULL, parent=NULL, pos=NULL, axes=0, axis=NULL, inv=FAKE, rot=128, inter=0, table=FAKE, q_out=FAKE,
             kp=FAKE, vp=FAKE):
        return lib.magicdec_norm_append(s or paged(), n, q, qs, k, ks, v, vs, qw, kw, eps, length, n_new, parent, pos,
                                        axes, axis, inv, rot, inter, table, q_out, kp, vp, NULL)
    for name in ("k", "v", "length", "table", "kp", "vp", "inv", "q", "q_out"):
        assert call(**{name: NULL}) == NULL_, name
    assert call(pos=FAKE, axes=2) == NULL_
    for bad in BAD_PAGED:
        assert call(s=paged(**bad)) == SHAPE, bad
    for bad in (dict(n=0), dict(rot=-2), dict(rot=130), dict(rot=7), dict(ks=255), dict(vs=128), dict(qs=1016),
                dict(eps=0.0), dict(eps=-1e-6), dict(eps=math.inf), dict(eps=math.nan), dict(eps=0.0, qw=NULL),
                dict(pos=FAKE, axes=1, parent=FAKE), dict(pos=FAKE, axes=0), dict(pos=FAKE, axes=-1), dict(axis=FAKE)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(rot=8), dict(rot=24), dict(n=257, parent=FAKE), dict(pos=FAKE, axes=65, axis=FAKE)):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("q", "k", "v", "q_out", "kp", "vp", "qw", "kw"):
        assert call(**{name: ODD}) == ALIGN, name
    for name in ("qs", "ks", "vs"):
        assert call(**{name: 1028}) == ALIGN, name


def test_prefix_attention_refusals(lib):
    def call(s=None, prefixes=1, most=10, n=4, q=FAKE, kp=FAKE, vp=FAKE, ptable=FAKE, plen=FAKE, first=NULL, table=FAKE,
             length=FAKE, out=FAKE, ws=FAKE, nbytes=1 << 50):
        return lib.magicdec_prefix_attn(s or paged(), prefixes, most, n, q, kp, vp, ptable, plen, first, table, length,
                                        NULL, NULL, out, ws, nbytes, NULL)
    size = lib.magicdec_prefix_attn_workspace_size
    for name in ("q", "kp", "vp", "ptable", "plen", "table", "length", "out", "ws"):
        assert call(**{name: NULL}) == NULL_, name
    assert call(prefixes=2) == NULL_
    for bad in BAD_PAGED:
        assert call(s=paged(**bad)) == SHAPE, bad
        assert size(paged(**bad), 1, 4) == 0
    for bad in (dict(n=0), dict(prefixes=0), dict(prefixes=-1), dict(most=0), dict(most=1 << 27)):
        assert call(**bad) == SHAPE, bad
    assert size(paged(), 0, 4) == size(paged(), 1, 0) == size(paged(), 4097, 4) == 0
    for s, n in ((paged(), 257), (paged(H_q=129, H_kv=1), 1), (paged(page_size=1, n_pages=(1 << 31) - 1), 4)):
        assert call(s=s, n=n) == UNSUPPORTED
        assert size(s, 1, n) == 0
    assert call(prefixes=4097, first=FAKE) == UNSUPPORTED
    # more tiles of a prefix, counted for every KV head and block of rows, than 32 bits hold
    assert call(s=paged(B=4096, H_q=1024, H_kv=8), n=256, most=1 << 20) == UNSUPPORTED
    for name in ("q", "kp", "vp", "out", "ws"):
        assert call(**{name: ODD}) == ALIGN, name
    for prefixes, n in ((1, 1), (2, 4), (2, 100)):
        need = size(paged(), prefixes, n)
        assert need > 0
        assert call(prefixes=prefixes, n=n, first=FAKE, nbytes=need - 1) == WS


def test_heavy_attention_refusals(lib):
    def call(s=None, n=1, q=FAKE, kc=FAKE, vc=FAKE, length=FAKE, next_pos=FAKE, weight=FAKE, pos=FAKE, out=FAKE):
        return lib.magicdec_heavy_attn(s or dense(), n, q, kc, vc, length, next_pos, weight, pos, out, NULL)
    for name in ("q", "kc", "vc", "length", "weight", "pos", "out"):
        assert call(**{name: NULL}) == NULL_, name
    for bad in BAD_DENSE:
        assert call(s=dense(**bad)) == SHAPE, bad
    assert call(n=0) == call(n=-1) == SHAPE
    for s, n in ((dense(), 9), (dense(H_q=33, H_kv=1), 1), (dense(), 1 << 30), (dense(H_q=65536, H_kv=65536), 1)):
        assert call(s=s, n=n) == UNSUPPORTED, (s.L_cap, n)
    for name in ("q", "kc", "vc", "out"):
        assert call(**{name: ODD}) == ALIGN, name


def test_eviction_refusals(lib):
    def call(s=None, layers=1, length=FAKE, total=FAKE, budget=50, sink=4, recent=10, kc=FAKE, vc=FAKE, weight=FAKE,
             pos=FAKE, out=OTHER):
        return lib.magicdec_heavy_evict(s or dense(), layers, length, total, budget, sink, recent, kc, vc, weight, pos,
                                        out, NULL)
    for name in ("length", "total", "kc", "vc", "weight", "pos", "out"):
        assert call(**{name: NULL}) == NULL_, name
    for bad in BAD_DENSE:
        assert call(s=dense(**bad)) == SHAPE, bad
    for bad in (dict(layers=0), dict(budget=0), dict(budget=-1), dict(sink=-1), dict(recent=-1), dict(sink=41),
                dict(recent=(1 << 31) - 1, sink=(1 << 31) - 1), dict(out=FAKE)):
        assert call(**bad) == SHAPE, bad
    assert call(layers=65536) == UNSUPPORTED
    assert call(s=dense(L_cap=(1 << 20) + 1)) == UNSUPPORTED
    for name in ("kc", "vc"):
        assert call(**{name: ODD}) == ALIGN, name


@pytest.fixture
def stand_in(monkeypatch):
    """Tensors without storage pass for CUDA ones of the current device, so that a call's own checks run."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(binding, "_current_device", lambda: None)


def empty(*shape, t=I32):
    return torch.empty(shape, dtype=t, device="meta")


def calls(B=2, n=4, **kw):
    """Each call on tensors of these shapes, of which `kw` replaces some."""
    x = dict(q=empty(B, n, 8, 128, t=BF16), k=empty(B, n, 2, 128, t=BF16), p=empty(20, 16, 2, 128, t=BF16),
             table=empty(B, 10), lens=empty(B), inv=empty(64, t=F32), w=empty(128, t=BF16), ptable=empty(1, 10),
             plen=empty(1), kc=empty(B, 2, 100, 128, t=BF16), weight=empty(B, 2, 100, t=F32), pos=empty(B, 2, 100),
             stream=None, **{a: None for a in ("first", "at", "axis", "next_pos")})
    x.update(kw)
    return dict(
        append=lambda: binding.magicdec_norm_append(x["k"], x["k"], x["p"], x["p"], x["table"], x["lens"], x["inv"],
                                                    q=x["q"], q_weight=x["w"], k_weight=x["w"], pos=x["at"],
                                                    axis=x["axis"], stream=x["stream"]),
        prefix=lambda: binding.magicdec_prefix_attn(x["q"], x["p"], x["p"], x["ptable"], x["plen"], x["table"],
                                                    x["lens"], first=x["first"], stream=x["stream"]),
        heavy=lambda: binding.magicdec_heavy_attn(x["q"], x["kc"], x["kc"], x["weight"], x["lens"], pos=x["pos"],
                                                  next_pos=x["next_pos"], stream=x["stream"]),
        evict=lambda: binding.magicdec_heavy_evict(x["kc"], x["kc"], x["weight"], x["pos"], x["lens"], x["lens"], 50,
                                                   stream=x["stream"]))


@pytest.mark.parametrize("name,kw,match", [
    ("append", dict(w=empty(64, t=BF16)), "q_weight"), ("append", dict(w=empty(128, t=F32)), "q_weight"),
    ("append", dict(at=empty(2, 4, 3, 1)), "pos must be"), ("append", dict(at=empty(2, 3, 3), axis=empty(64)), "pos"),
    ("append", dict(at=empty(2, 4, 3), axis=empty(63)), "axis"),
    ("append", dict(k=empty(2, 4, 3, 128, t=BF16)), "k and k_pages disagree"),
    ("prefix", dict(ptable=empty(2, 10), plen=empty(2)), "several prefixes need first"),
    ("prefix", dict(ptable=empty(10)), "prefix_table must be"), ("prefix", dict(plen=empty(3)), "prefix_len"),
    ("prefix", dict(first=empty(3)), "first"), ("prefix", dict(q=empty(2, 4, 8, 64, t=BF16)), "disagree"),
    ("prefix", dict(ptable=empty(1, 1 << 31)), "max_prefix_pages"),
    ("heavy", dict(weight=empty(2, 2, 99, t=F32)), "weight"), ("heavy", dict(pos=empty(2, 2, 99)), "pos"),
    ("heavy", dict(kc=empty(3, 2, 100, 128, t=BF16), weight=empty(3, 2, 100, t=F32), pos=empty(3, 2, 100)), "disagree"),
    ("heavy", dict(pos=None, next_pos=empty(2)), "next_pos without pos"),
    ("evict", dict(pos=empty(2, 2, 99)), "pos"), ("evict", dict(kc=empty(2, 100, 128, t=BF16)), "kc must be"),
    ("evict", dict(pos=None), "pos must be"),
])
def test_binding_refuses_what_it_cannot_pass_on(stand_in, name, kw, match):
    with pytest.raises((ValueError, TypeError), match=match):
        calls(**kw)[name]()


def test_binding_refuses_a_stream_of_another_device(stand_in):
    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 1)

    for call in calls(stream=Stream()).values():
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_binding_refuses_tensors_of_the_host(lib):
    x = torch.zeros((2, 4, 8, 128), dtype=BF16)
    for call in calls(q=x, k=x, kc=x).values():
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_append_refuses_an_eps_that_squares_in_fp32_cannot_tell_from_others(lib):
    """Squares of some 2^-126 and less lose their last bits, so that beside a smaller eps the root would be off."""
    def call(eps, weight=FAKE):                        # 65 axes are refused behind this check
        return lib.magicdec_norm_append(paged(), 4, FAKE, 1024, FAKE, 256, FAKE, 256, weight, weight, eps, FAKE, NULL, NULL,
                                        FAKE, 65, FAKE, FAKE, 128, 0, FAKE, FAKE, FAKE, FAKE, NULL)
    for eps in (2.0 ** -127, 1e-40, 2.0 ** -149):
        assert call(eps) == SHAPE
    assert call(2.0 ** -126) == call(1e-6) == call(0.0, NULL) == UNSUPPORTED
