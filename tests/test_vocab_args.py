"""Argument checks of the embedding and the head that the host makes before it
touches a device, and the 64-bit formulas the GPU tests compare with."""
import ctypes as C

import pytest
import torch

import vocab_util as vu


@pytest.fixture(scope="module")
def gr():
    import trie_constrained_beam_step_amd as gr
    gr.lib()
    return gr


def _embed_cfg(gr, **kw):
    base = dict(vocab=48, dim=64, max_tokens=16, dtype=0, scale=1.0)
    base.update(kw)
    return gr._lib.EmbedConfig(**base)


def _head_cfg(gr, **kw):
    base = dict(vocab=48, dim=64, max_rows=16, dtype=0, scale=1.0, score_only=0)
    base.update(kw)
    return gr._lib.HeadConfig(**base)


BAD = [dict(vocab=0), dict(vocab=-1), dict(vocab=(1 << 30) + 1), dict(dim=0), dict(dim=65537), dict(dtype=2),
       dict(dtype=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD + [dict(max_tokens=0), dict(max_tokens=-5), dict(max_tokens=(1 << 24) + 1)])
def test_embed_config_refused(gr, bad):
    h = C.c_void_p()
    assert gr.lib().gr_embed_init(C.byref(_embed_cfg(gr, **bad)), None, C.byref(h)) == gr._lib.GR_ERR_INVALID_ARG
    assert h.value is None and gr.lib().gr_last_error()


@pytest.mark.parametrize("bad", BAD + [dict(max_rows=0), dict(max_rows=-5), dict(max_rows=(1 << 20) + 1)])
def test_head_config_refused(gr, bad):
    h = C.c_void_p()
    assert gr.lib().gr_head_init(C.byref(_head_cfg(gr, **bad)), None, C.byref(h)) == gr._lib.GR_ERR_INVALID_ARG
    assert h.value is None and gr.lib().gr_last_error()


def test_null_arguments(gr):
    L, h, p = gr.lib(), C.c_void_p(), C.c_void_p(64)
    assert L.gr_embed_init(None, None, C.byref(h)) == 1
    assert L.gr_embed_init(C.byref(_embed_cfg(gr)), None, None) == 1
    assert L.gr_head_init(None, None, C.byref(h)) == 1
    assert L.gr_head_init(C.byref(_head_cfg(gr)), None, None) == 1
    assert L.gr_embed_lookup(None, p, 1, p, 0, p, 0, None) == 1
    assert L.gr_embed_backward(None, p, 1, p, 0, p, 0, 0, None) == 1
    assert L.gr_head_loss(None, p, 0, p, 0, p, 1, p, p, None) == 1
    assert L.gr_head_backward(None, p, 0, p, 0, p, 1, p, p, p, 0, p, 0, 0, None) == 1
    L.gr_embed_free(None)  # NULL-safe
    L.gr_head_free(None)


@pytest.mark.parametrize("cls", ["Embedding", "Head"])
def test_unknown_dtype_refused(gr, cls):
    with pytest.raises(ValueError):
        getattr(gr, cls)(48, 64, 16, dtype="f16")


def test_formulas_agree_with_autograd():
    """The 64-bit gradients the GPU tests use are autograd's of the plain loss."""
    gen = torch.Generator().manual_seed(3)
    h = torch.randn(7, 5, generator=gen, dtype=torch.float64, requires_grad=True)
    w = torch.randn(11, 5, generator=gen, dtype=torch.float64, requires_grad=True)
    t = torch.tensor([0, 3, -1, 10, 11, 3, 2])
    g = torch.randn(7, generator=gen, dtype=torch.float64)
    r = vu.head(h.detach(), w.detach(), t, 1.5, "f32", g)
    z = h @ w.T * 1.5
    ok = (t >= 0) & (t < 11)
    loss = torch.where(ok, torch.logsumexp(z, 1) - z.gather(1, t.clamp(0, 10)[:, None])[:, 0], 0.0)
    (loss * g).sum().backward()
    assert torch.allclose(r["loss"], loss.detach(), atol=1e-12)
    assert torch.allclose(r["gh"], h.grad, atol=1e-12) and torch.allclose(r["gw"], w.grad, atol=1e-12)
    tok = torch.tensor([[1, 4, 1], [-1, 11, 0]])
    up = torch.randn(2, 3, 5, generator=gen, dtype=torch.float64)
    w.grad = None
    y = torch.where(((tok >= 0) & (tok < 11))[..., None], w[tok.clamp(0, 10)] * 2.5, 0.0)
    (y * up).sum().backward()
    assert torch.allclose(vu.scatter(tok, up, 11, 2.5, "f32")[0], w.grad, atol=1e-12)
