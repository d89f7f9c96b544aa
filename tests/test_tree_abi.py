"""The paged-cache and tree calls refuse bad arguments on the host, before anything is
enqueued (CPU only: every call here fails validation first)."""
import ctypes

import pytest

from long_context_self_gb300 import binding
from long_context_self_gb300 import build as lbuild

P = ctypes.c_void_p
FAKE, ODD, NULL = P(0x10000), P(0x10008), P(0)
NULL_, SHAPE, ALIGN, WS, UNSUPPORTED = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return binding.lib()


def shape(**kw):
    s = dict(B=2, H_q=8, H_kv=2, d=128, page_size=16, n_pages=20, max_pages=10)
    s.update(kw)
    return binding.paged_shape(**s)


BAD_SHAPES = [dict(B=0), dict(B=4097), dict(H_q=0), dict(H_kv=0), dict(H_q=9), dict(d=96), dict(page_size=0),
              dict(n_pages=0), dict(max_pages=0), dict(page_size=1 << 16, max_pages=1 << 15), dict(H_q=65536, H_kv=65536),
              dict(page_size=(1 << 31) - 255, max_pages=1), dict(H_q=65536)]


def append(lib, s=None, n=4, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, length=FAKE, n_new=NULL, parent=NULL,
           inv=FAKE, rot=128, inter=0, table=FAKE, q_out=FAKE, kp=FAKE, vp=FAKE):
    return lib.magicdec_paged_append(s or shape(), n, q, qs, k, ks, v, vs, length, n_new, parent, inv, rot, inter, table,
                                     q_out, kp, vp, NULL)


def test_append_refusals(lib):
    for name in ("k", "v", "length", "table", "kp", "vp", "inv", "q", "q_out"):
        assert append(lib, **{name: NULL}) == NULL_, name
    for bad in BAD_SHAPES:
        assert append(lib, s=shape(**bad)) == SHAPE, bad
    for bad in (dict(n=0), dict(n=-1), dict(rot=-2), dict(rot=130), dict(rot=7), dict(ks=255), dict(vs=128),
                dict(qs=1016)):
        assert append(lib, **bad) == SHAPE, bad
    for bad in (dict(rot=8), dict(rot=24), dict(n=257, parent=FAKE)):
        assert append(lib, **bad) == UNSUPPORTED, bad
    for name in ("q", "k", "v", "q_out", "kp", "vp"):
        assert append(lib, **{name: ODD}) == ALIGN, name
    for name in ("qs", "ks", "vs"):
        assert append(lib, **{name: 1028}) == ALIGN, name


def attn(lib, s=None, n=4, q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, length=FAKE, out=FAKE, ws=FAKE, nbytes=1 << 40):
    return lib.magicdec_tree_attn(s or shape(), n, q, kp, vp, table, length, NULL, NULL, out, ws, nbytes, NULL)


def test_attention_refusals(lib):
    for name in ("q", "kp", "vp", "table", "length", "out", "ws"):
        assert attn(lib, **{name: NULL}) == NULL_, name
    for bad in BAD_SHAPES:
        assert attn(lib, s=shape(**bad)) == SHAPE, bad
        assert lib.magicdec_tree_attn_workspace_size(shape(**bad), 4) == 0
    assert attn(lib, n=0) == SHAPE
    for s, n in ((shape(), 257), (shape(H_q=129, H_kv=1), 1)):
        assert attn(lib, s=s, n=n) == UNSUPPORTED
        assert lib.magicdec_tree_attn_workspace_size(s, n) == 0
    for name in ("q", "kp", "vp", "out", "ws"):
        assert attn(lib, **{name: ODD}) == ALIGN, name
    need = lib.magicdec_tree_attn_workspace_size(shape(), 4)
    assert need > 0
    assert attn(lib, nbytes=need - 1) == WS


def test_accept_refusals(lib):
    def accept(B=2, n=4, V=100, target=FAKE, tok=FAKE, n_acc=FAKE, path=FAKE, out=FAKE):
        return lib.magicdec_tree_accept(B, n, V, target, tok, NULL, NULL, n_acc, path, out, NULL)
    for name in ("target", "tok", "n_acc", "path", "out"):
        assert accept(**{name: NULL}) == NULL_, name
    for bad in (dict(B=0), dict(n=0), dict(V=0), dict(B=-1)):
        assert accept(**bad) == SHAPE, bad
    assert accept(n=257) == UNSUPPORTED
    assert accept(B=65537) == UNSUPPORTED
    assert accept(target=ODD) == ALIGN


def test_commit_refusals(lib):
    def commit(s=None, n=4, layers=1, length=FAKE, path=FAKE, n_acc=FAKE, table=FAKE, kp=FAKE, vp=FAKE):
        return lib.magicdec_tree_commit(s or shape(), n, layers, length, path, n_acc, table, kp, vp, NULL)
    for name in ("length", "path", "n_acc", "table", "kp", "vp"):
        assert commit(**{name: NULL}) == NULL_, name
    for bad in BAD_SHAPES:
        assert commit(s=shape(**bad)) == SHAPE, bad
    for bad in (dict(n=0), dict(layers=0)):
        assert commit(**bad) == SHAPE, bad
    for bad in (dict(n=257), dict(layers=65536)):
        assert commit(**bad) == UNSUPPORTED, bad
    for name in ("kp", "vp"):
        assert commit(**{name: ODD}) == ALIGN, name


def test_binding_refuses_tensors_of_the_host(lib):
    import torch
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i = torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        binding.magicdec_paged_append(z(2, 4, 2, 128), z(2, 4, 2, 128), z(20, 16, 2, 128), z(20, 16, 2, 128),
                                      z(2, 10, t=i), z(2, t=i))
    with pytest.raises(ValueError, match="CUDA"):
        binding.magicdec_tree_attn(z(2, 4, 8, 128), z(20, 16, 2, 128), z(20, 16, 2, 128), z(2, 10, t=i), z(2, t=i))
    with pytest.raises(ValueError, match="CUDA"):
        binding.magicdec_tree_accept(z(2, 4, 100, t=torch.float32), z(2, 4, t=i))
    with pytest.raises(ValueError, match="CUDA"):
        binding.magicdec_tree_commit(z(20, 16, 2, 128), z(20, 16, 2, 128), z(2, 10, t=i), z(2, t=i), z(2, 4, t=i),
                                     z(2, t=i))
    with pytest.raises(TypeError, match="target"):
        binding.magicdec_tree_accept(z(2, 4, 100), z(2, 4, t=i))


def test_binding_refuses_layouts_it_cannot_pass_on(lib, monkeypatch):
    """Token rows need dense heads and one stride; shapes have to agree."""
    import torch
    cpu = torch.device("cpu")
    x = torch.zeros((3, 5, 6, 64), dtype=torch.bfloat16)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)   # the device check comes first
    assert binding._tokens(x, "x", cpu, 3, 5, 64) == (6, 384)
    assert binding._tokens(x[:, :, 2:4], "x", cpu, 3, 5, 64) == (2, 384)
    assert binding._tokens(x[:1, :1], "x", cpu, 1, 1, 64) == (6, 384)
    assert binding._tokens(x[:, :1], "x", cpu, 3, 1, 64) == (6, 5 * 384)
    for bad in (x[:, :4], x.transpose(0, 1).contiguous().transpose(0, 1), x[..., ::2, :], x[..., :32]):
        with pytest.raises(ValueError):
            binding._tokens(bad, "x", cpu, bad.shape[0], bad.shape[1], 64)
    with pytest.raises(TypeError):
        binding._tokens(x.float(), "x", cpu, 3, 5, 64)
    i = torch.int32
    with pytest.raises(ValueError, match="block_table"):
        binding._paged_cache(x, x, torch.zeros((2, 4), dtype=i), 3, cpu)
    with pytest.raises(ValueError, match="v_pages"):
        binding._paged_cache(x, x[1:], torch.zeros((3, 4), dtype=i), 3, cpu)
    with pytest.raises(ValueError, match="k_pages"):
        binding._paged_cache(x[None], x[None], torch.zeros((3, 4), dtype=i), 3, cpu)
    assert binding._paged_cache(x[None], x[None], torch.zeros((3, 4), dtype=i), 3, cpu, 5)[3:] == (5, 3, 4, 6, 64)


def test_binding_refuses_sizes_that_ctypes_would_cut_short(monkeypatch):
    import torch
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    cpu = torch.device("cpu")
    x = torch.zeros((3, 5, 6, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="max_pages is 4294967299"):
        binding._paged_cache(x, x, torch.empty((3, (1 << 32) + 3), dtype=torch.int32, device="meta"), 3, cpu)
    binding._fits("V", (1 << 31) - 1)
    with pytest.raises(ValueError, match="V is 2147483648"):
        binding._fits("V", 1 << 31)
