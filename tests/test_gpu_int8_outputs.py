"""Given outputs of the 8-bit head: refused where they reach into what else a call
touches, before anything is enqueued."""

import pytest
import torch

import rollout_logprob_consistency_amd as lp

from .gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture
def operands():
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(6, 48, generator=g, device=DEV)
    w = torch.randn(20, 48, generator=g, device=DEV)
    return (*lp.quantize_int8(x), *lp.quantize_int8(w))


def test_quantise():
    x = torch.randn(6, 40, device=DEV)
    before = x.clone()
    scale = torch.empty(6, device=DEV)
    buf = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    codes = buf[:6 * 48].view(torch.int8).view(6, 48)[:, :40]
    with pytest.raises(ValueError, match="scale must lie apart from x"):
        lp.quantize_int8(x, scale=x[2, 3:9])
    with pytest.raises(ValueError, match="out must lie apart from scale"):
        lp.quantize_int8(x, out=codes, scale=buf[240:264].view(torch.float32))
    # The last row's padding is written too.
    with pytest.raises(ValueError, match="out must lie apart from scale"):
        lp.quantize_int8(x, out=codes, scale=buf[284:308].view(torch.float32))
    inside = buf[280:280 + 6 * 160].view(torch.float32).view(6, 40)
    with pytest.raises(ValueError, match="out must lie apart from x"):
        lp.quantize_int8(inside, out=codes, scale=scale)
    assert torch.equal(x, before) and not buf.any()
    # Side by side is apart.
    beside = buf[288:312].view(torch.float32)
    lp.quantize_int8(x, out=codes, scale=beside)
    q, s = lp.quantize_int8(x)
    assert torch.equal(codes, q) and torch.equal(beside, s)


def test_logits(operands):
    x, xs, w, ws = operands
    buf = torch.zeros(6 * 20 + 40, device=DEV)
    out = buf[:120].view(6, 20)
    a, b = buf[118:124], buf[110:130]
    a.copy_(xs)
    with pytest.raises(ValueError, match="out must lie apart from x_scale"):
        lp.logits_int8(x, a, w, ws, out=out)
    b.copy_(ws)
    with pytest.raises(ValueError, match="out must lie apart from w_scale"):
        lp.logits_int8(x, xs, w, b, out=out)
    beside = buf[120:140].copy_(ws)
    want = lp.logits_int8(x, xs, w, ws, dtype=torch.float32)
    assert torch.equal(lp.logits_int8(x, xs, w, beside, out=out), want)


def test_scores(operands):
    x, xs, w, ws = operands
    ids = torch.arange(6, device=DEV)
    one = torch.empty(6, device=DEV)
    inside = {"x": x.view(torch.float32)[0, :6], "w": w.view(torch.float32)[19, 6:12],
              "x_scale": xs, "w_scale": ws[7:13], "ids": ids.view(torch.float32)[3:9]}
    for name, t in inside.items():
        with pytest.raises(ValueError, match=f"out must lie apart from {name}$"):
            lp.score_int8(x, xs, w, ws, ids, out=t)
        with pytest.raises(ValueError, match=f"lse must lie apart from {name}$"):
            lp.score_int8(x, xs, w, ws, ids, lse=t)
    with pytest.raises(ValueError, match="lse must lie apart from out"):
        lp.score_int8(x, xs, w, ws, ids, out=one, lse=one)
    both = torch.empty(12, device=DEV)
    got = lp.score_int8(x, xs, w, ws, ids, out=both[:6], lse=both[6:])
    lse = torch.empty(6, device=DEV)
    assert torch.equal(got, lp.score_int8(x, xs, w, ws, ids, lse=lse))
    assert torch.equal(both[6:], lse)


def test_outputs_that_require_gradients(operands):
    """Their values would be written over behind autograd's back."""
    x, xs, w, ws = operands
    ids = torch.arange(6, device=DEV)
    leaf = torch.ones(6, device=DEV, requires_grad=True)
    for name, call in (("scale", lambda: lp.quantize_int8(torch.randn(6, 40, device=DEV), scale=leaf)),
                       ("out", lambda: lp.score_int8(x, xs, w, ws, ids, out=leaf)),
                       ("lse", lambda: lp.score_int8(x, xs, w, ws, ids, lse=leaf)),
                       ("out", lambda: lp.logits_int8(x, xs, w[:1], ws[:1], out=leaf.view(6, 1)))):
        with pytest.raises(ValueError, match=f"{name} must not require gradients"):
            call()
    assert (leaf == 1).all() and leaf._version == 0
