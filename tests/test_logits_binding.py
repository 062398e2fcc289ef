"""The binding of the operators on rows of logits, with the library's calls
replaced (CPU only): what it does around them."""

import pytest
import torch
from torch.autograd import forward_ad

import rollout_logprob_consistency_amd as lp
from rollout_logprob_consistency_amd import logits as binding


@pytest.fixture
def no_launch(monkeypatch):
    def forward(logits, *args, **kw):
        n = logits.shape[0]
        return torch.zeros(n), torch.zeros(n, 4, dtype=torch.float64)
    monkeypatch.setattr(binding, "distill_forward", forward)


def data():
    return torch.randn(3, 5), torch.zeros(3, 2, dtype=torch.int64), torch.randn(3, 2)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("which", ["logits", "teacher"])
@pytest.mark.parametrize("no_grad", [False, True])
def test_a_tangent_is_refused_and_not_dropped(no_launch, grad, which, no_grad):
    """Forward-mode differentiation has no formula here: a loss without a
    tangent would be a derivative of zero."""
    z, ids, x = data()
    z.requires_grad_(grad)
    with forward_ad.dual_level():
        if which == "logits":
            z = forward_ad.make_dual(z, torch.ones_like(z))
        else:
            x = forward_ad.make_dual(x, torch.ones_like(x))
        with torch.set_grad_enabled(not no_grad), pytest.raises(NotImplementedError):
            lp.distill(z, ids, x)


def test_forward_mode_transform_is_refused(no_launch):
    z, ids, x = data()
    with pytest.raises(NotImplementedError):
        torch.func.jvp(lambda a: lp.distill(a, ids, x), (z,), (torch.ones_like(z),))


def test_tensors_without_a_tangent_pass(no_launch):
    z, ids, x = data()
    assert not lp.distill(z, ids, x).requires_grad
    assert lp.distill(z.clone().requires_grad_(), ids, x).requires_grad
    with forward_ad.dual_level():
        forward_ad.make_dual(torch.ones(2), torch.ones(2))
        assert lp.distill(z, ids, x).shape == (3,)
        assert lp.distill(z.clone().requires_grad_(), ids, x).requires_grad


@pytest.mark.parametrize("earlier", [0, 5])
def test_a_checked_call_counts_apart_from_the_callers_counter(earlier):
    """A counter that holds earlier calls' rows neither raises for them nor
    loses a checked call's."""
    cpu = torch.device("cpu")
    bad = torch.full((1,), earlier, dtype=torch.int32)
    count = binding._bad_rows(bad, True, cpu)
    assert count is not bad and count.item() == 0
    binding._raise_bad(count, bad, "are bad")             # a clean call
    assert bad.item() == earlier
    count = binding._bad_rows(bad, True, cpu)
    count += 2                                            # a call with two
    with pytest.raises(ValueError, match="^2 row"):
        binding._raise_bad(count, bad, "are bad")
    assert bad.item() == earlier + 2
    assert binding._bad_rows(bad, False, cpu) is bad      # unchecked: counted there
    assert binding._bad_rows(None, False, cpu) is None
