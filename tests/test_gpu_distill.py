"""lp_distill_* against the fp64 oracle, by difference, and against themselves.

Loss: teacher terms are fp64; ln S carries the fp32 exponentials. Their
argument (z - m) * (log2 e / tau) has three roundings (3 * 2^-24 |x| relative
to its value x), so a weight is off by ln2 * 3 * 2^-24 |x|; weighted by the
weights, |x| averages at most the entropy in bits, at most log2 V <= 17.3: 36
* 2^-24. The exponential adds 2^-23, a thread's sum (of at most 64 terms) at most 63 *
2^-24. In total 102 * 2^-24 of S, times Q in the loss; the result is rounded
to fp32 once.

Gradient: the dense part c * exp2(x) carries the same error of S, 3 roundings
in c and the product, and for |x| <= 126 an argument error of ln2 * 3 * 126 *
2^-24: (102 + 4 + 263) * 2^-24 < 2.3e-5 of Q p |g| / tau, below that nothing
but underflow (2^-126 |c|); then one rounding to the logits' type."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import logit_rows as ol

from .gpu_helpers import DEV
from .logits_helpers import TYPES, dev, place, rows

pytestmark = pytest.mark.gpu
S_ERR = 102 * 2.0 ** -24
DENSE_ERR = 369 * 2.0 ** -24


def teacher(seed, z, k, absent=0.2, logprobs=False, tau=1.0):
    """Ids [T, k] (some -1) and the teacher's logits, or logprobs at tau."""
    rng = np.random.default_rng(seed)
    T, v = z.shape
    base = np.where(np.isfinite(z), z, -30.0) + rng.normal(size=z.shape) * 0.7
    ids = np.argsort(-base, axis=1)[:, :k].astype(np.int64)
    x = np.take_along_axis(base, ids, 1)
    if logprobs:
        s = base / tau
        m = s.max(1, keepdims=True)
        x = x / tau - (m + np.log(np.exp(s - m).sum(1, keepdims=True)))
    ids[rng.random((T, k)) < absent] = -1
    x = x.astype(np.float32)
    return ids, x


def compare(z, ids, x, tau, renorm, loss, grad=None, weight=None, dtype="fp32"):
    r_loss, r_grad = ol.distill(z, ids, x.astype(np.float64), tau, renorm, weight)
    loss = loss.detach().cpu().numpy().astype(np.float64)
    there = ids != -1
    q = np.where(there, np.exp(x.astype(np.float64)), 0.0).sum(1) if not renorm else np.ones(len(z))
    assert np.array_equal(np.isnan(loss), np.isnan(r_loss)), (loss, r_loss)
    inf = np.isinf(r_loss)
    assert np.array_equal(loss[inf], r_loss[inf])
    ok = np.isfinite(r_loss)
    tol = S_ERR * q + 2.0 ** -24 * np.abs(r_loss) + 1e-12
    err = np.abs(np.where(inf, 0.0, loss) - np.where(inf, 0.0, r_loss))
    print("loss error / tolerance", np.max((err / tol)[ok], initial=0.0))
    assert np.all(err[ok] <= tol[ok])
    if grad is None:
        return
    got = grad.double().cpu().numpy()
    fi = torch.finfo(TYPES[dtype])
    g = np.ones(len(z)) if weight is None else weight
    assert np.array_equal(np.isnan(got), np.isnan(r_grad))
    for t in range(len(z)):
        if np.isnan(r_grad[t]).any() or g[t] == 0:
            assert np.array_equal(got[t], r_grad[t], equal_nan=True)
            continue
        s = z[t] / tau
        p = np.exp(s - s.max()) / np.exp(s - s.max()).sum()
        scale = abs(g[t]) / tau * q[t]
        tol = (fi.eps / 2 * np.abs(r_grad[t]) + DENSE_ERR * (1 + fi.eps) * scale * p
               + fi.tiny * fi.eps / 2 + 2.0 ** -120 * scale)
        err = np.abs(got[t] - r_grad[t])
        assert np.all(err <= tol), (t, np.argmax(err - tol), np.max(err / tol))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,v,k,pad,lead", [(1, 1, 1, 0, 0), (3, 2, 2, 1, 1), (5, 17, 6, 0, 3),
                                            (7, 1000, 32, 24, 0), (4, 1025, 1024, 3, 5),
                                            (3, 8192, 64, 0, 0), (3, 8193, 64, 0, 1),
                                            (2, 16385, 257, 7, 0), (6, 50021, 100, 3, 2)])
@pytest.mark.parametrize("renorm,tau", [(True, 1.0), (True, 2.0), (False, 0.75)])
def test_loss_and_gradient(dtype, T, v, k, pad, lead, renorm, tau):
    t, z = rows(v + k, T, v, dtype, pad=pad, lead=lead)
    ids, x = teacher(1, z, k, logprobs=not renorm, tau=tau)
    w = np.random.default_rng(2).normal(size=T).astype(np.float32)
    di, dx, dw = dev(ids, torch.int64), dev(x, torch.float32), dev(w, torch.float32)
    loss, state = lp.distill_forward(t, di, dx, tau, renorm)
    grad = lp.distill_backward(t, di, dx, state, dw, tau, renorm)
    compare(z, ids, x, tau, renorm, loss, grad, w, dtype)
    loss2, grad2 = lp.distill_step(t, di, dx, dw, tau, renorm)
    assert torch.equal(loss, loss2) and torch.equal(grad.view(torch.uint8), grad2.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_language_models_vocabulary(dtype):
    t, z = rows(5, 3, 151936, dtype)
    ids, x = teacher(4, z, 64)
    w = np.float32([0.25, 0.0, -3.0])
    loss, grad = lp.distill_step(t, dev(ids, torch.int64), dev(x, torch.float32),
                                 dev(w, torch.float32))
    compare(z, ids, x, 1.0, True, loss, grad, w, dtype)
    assert not grad[1].any()


@pytest.mark.parametrize("T", [3, 300])
def test_the_smallest_temperature(T):
    """Loss and gradient scaled by it: the gradient stays in fp32's range."""
    tau = 2.0 ** -126
    rng = np.random.default_rng(12)
    z = rng.normal(size=(T, 25001)) * 3 * tau
    z[2] = rng.normal(size=25001) * 1e20       # the maximum alone is left
    t, z = place(z, "fp32")
    ids, x = teacher(1, np.clip(z / tau, -50, 50), 30)
    x = (x.astype(np.float64) * tau).astype(np.float32)
    ids[2, 0], ids[2, 1:], x[2, 0] = z[2].argmax(), -1, z[2].max()
    w = rng.random(T).astype(np.float32)
    di, dx, dw = dev(ids, torch.int64), dev(x, torch.float32), dev(w, torch.float32)
    loss, grad = lp.distill_step(t, di, dx, dw, tau)
    compare(z, ids, x, tau, True, loss, grad, w)
    assert torch.isfinite(loss).all() and torch.isfinite(grad).all()
    assert loss[2] == 0 and not grad[2].any()


def test_autograd_and_differences():
    t, z = rows(9, 6, 700, "fp32")
    ids, x = teacher(3, z, 20)
    di, dx = dev(ids, torch.int64), dev(x, torch.float32)
    w = np.random.default_rng(0).random(6).astype(np.float32)
    leaf = t.clone().requires_grad_(True)
    loss = lp.distill(leaf, di, dx, 1.5)
    (loss * dev(w, torch.float32)).sum().backward()
    compare(z, ids, x, 1.5, True, loss, leaf.grad, w)
    # A broadcast upstream gradient (the sum's) and a second use of the leaf.
    leaf2 = t.clone().requires_grad_(True)
    (lp.distill(leaf2, di, dx, 1.5).sum() + lp.distill(leaf2, di, dx, 1.5).sum()).backward()
    compare(z, ids, x, 1.5, True, loss, leaf2.grad, np.full(6, 2.0))
    # Differences along a direction: h = 2^-5; the third-order term is
    # h^2 / 6 |f'''| <= h^2 / 6 * (|d|_inf / tau)^3, the loss error 2 S_ERR / (2 h).
    d = np.random.default_rng(7).normal(size=z.shape)
    d /= np.abs(d).max()
    h = 2.0 ** -5
    up = place(z + h * d)[0]
    dn = place(z - h * d)[0]
    lu, ld = (lp.distill(a, di, dx, 1.5).double().cpu().numpy() for a in (up, dn))
    grad = torch.autograd.grad(lp.distill(leaf, di, dx, 1.5).sum(), leaf)[0].double().cpu().numpy()
    lhs, rhs = (lu - ld) / (2 * h), (grad * d).sum(1)
    tol = h * h / 6 / 1.5 ** 3 + (S_ERR + 2.0 ** -23 * 20) / h
    assert np.all(np.abs(lhs - rhs) <= tol), (lhs, rhs)
    # Differentiable once; nothing to differentiate without a leaf.
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(lp.distill(leaf, di, dx).sum(), leaf, create_graph=True)
        g.sum().backward()
    assert not lp.distill(t, di, dx).requires_grad


def test_absent_repeated_and_outside_ids():
    t, z = rows(2, 8, 5000, "bf16")
    ids, x = teacher(6, z, 12, absent=0.0)
    ids[0, 3:7] = ids[0, 2]        # the same id five times
    ids[1] = ids[1, 0]             # one id only
    ids[2] = -1                    # nothing
    ids[3, 4], ids[4, 0] = 5000, -2
    x[3, 0] = np.nan               # (a row that is bad anyway)
    x[5, 3] = -np.inf              # an entry that weighs nothing
    x[6, 1] = np.nan
    x[7] = -np.inf
    w = np.random.default_rng(3).random(8).astype(np.float32)
    args = (dev(ids, torch.int64), dev(x, torch.float32), dev(w, torch.float32))
    for renorm in (True, False):
        loss, grad = lp.distill_step(t, *args, renormalize=renorm)
        compare(z, ids, x, 1.0, renorm, loss, grad, w, "bf16")
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    lp.distill_forward(t, *args[:2], bad_rows=bad)
    assert bad.item() == 2
    with pytest.raises(ValueError, match="2 row"):
        lp.distill_step(t, *args, check=True)


def test_masked_logits_and_rows_of_no_weight():
    """-inf logits (also under a teacher's entry), rows that are all masked,
    NaN and +inf logits; rows of weight 0 are zeros whatever they hold."""
    t, z = rows(12, 9, 3000, "fp32", masked=0.4)
    z[1] = -np.inf
    z[2, 7], z[3, 8] = np.nan, np.inf
    z[4], z[5] = z[1], z[2]
    t, z = place(z, "fp32")
    ids, x = teacher(8, z, 16, absent=0.1)
    finite = np.isfinite(z)
    for r in range(9):             # entries on tokens that are not masked, but in row 8
        alive = np.flatnonzero(finite[r])
        if r != 8 and alive.size:
            ids[r] = np.where(ids[r] < 0, -1, alive[:16])
    ids[8, 0] = np.flatnonzero(~finite[8])[0]
    x[8, 0] = 3.0
    w = np.float32([1, 1, 1, 1, 0, 0, 1, 0, 0.5])
    loss, grad = lp.distill_step(t, dev(ids, torch.int64), dev(x, torch.float32),
                                 dev(w, torch.float32))
    compare(z, ids, x, 1.0, True, loss, grad, w)
    assert np.isinf(loss[8].item()) and torch.isfinite(grad[8]).all()
    # Rows without an entry: zeros, whatever the logits are.
    none = torch.full((9, 16), -1, dtype=torch.int64, device=DEV)
    loss, grad = lp.distill_step(t, none, dev(x, torch.float32), torch.ones(9, device=DEV))
    assert not loss.any() and not grad.any()


def test_padding_columns_and_rows_behind():
    """Columns behind the vocabulary get zeros, memory between and behind the
    rows is left alone."""
    t, z = rows(13, 5, 2000, "bf16", pad=8)
    t[:, 1900:] = float("nan")
    ids, x = teacher(5, z[:, :1900], 30)
    buf = torch.full((7, 2016), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[:5, :2000]
    w = torch.ones(5, device=DEV)
    args = (dev(ids, torch.int64), dev(x, torch.float32))
    loss, grad = lp.distill_step(t, *args, w, v_true=1900, out=out)
    assert grad.data_ptr() == buf.data_ptr()
    compare(z[:, :1900], ids, x, 1.0, True, loss, grad[:, :1900], np.ones(5), "bf16")
    assert not grad[:, 1900:].any()
    assert (buf[5:] == 7.0).all() and (buf[:, 2000:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("v", [1000, 40000])
def test_gradient_over_the_logits_own_buffer(dtype, v):
    t, z = rows(14, 9, v, dtype, pad=3, lead=1)
    ids, x = teacher(5, z, 50)
    args = (dev(ids, torch.int64), dev(x, torch.float32))
    w = torch.rand(9, device=DEV)
    loss, grad = lp.distill_step(t, *args, w)
    keep = t.clone()
    loss2, grad2 = lp.distill_step(t, *args, w, out=t)
    assert grad2.data_ptr() == t.data_ptr()
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)
    t.copy_(keep)
    _, state = lp.distill_forward(t, *args)
    assert torch.equal(lp.distill_backward(t, *args, state, w, out=t), grad)
    # Saved logits that were overwritten are noticed by autograd.
    leaf = keep.clone().requires_grad_(True)
    mid = leaf * 1.0
    loss = lp.distill(mid, *args)
    lp.distill_step(mid.detach(), *args, w, out=mid.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()


def test_batch_invariance_and_alignment():
    t, z = rows(31, 40, 20011, "bf16")
    ids, x = teacher(5, z, 64)
    di, dx = dev(ids, torch.int64), dev(x, torch.float32)
    w = torch.rand(40, device=DEV)
    loss, grad = lp.distill_step(t, di, dx, w)
    t2, _ = place(z, "bf16", pad=5, lead=3)
    l2, g2 = lp.distill_step(t2, di, dx, w)
    assert torch.equal(loss, l2) and torch.equal(grad, g2)
    for i in (0, 13, 39):
        l1, g1 = lp.distill_step(t2[i:i + 1], di[i:i + 1], dx[i:i + 1], w[i:i + 1])
        assert torch.equal(loss[i:i + 1], l1) and torch.equal(grad[i:i + 1], g1)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("v,pad,lead", [(5, 0, 0), (4099, 5, 1), (40007, 0, 3)])
def test_many_rows_give_the_bits_of_few(dtype, v, pad, lead):
    """300 rows (one workgroup each) and the same rows in batches of 100
    (slices): forward, backward and step, also over the logits' own buffer."""
    T = 300
    t, z = rows(17, T, v, dtype, pad=pad, lead=lead, masked=0.1)
    z[5] = -np.inf
    z[6, v // 2] = np.nan
    t, z = place(z, dtype, pad, lead)
    ids, x = teacher(5, z, min(v, 70))
    ids[7] = -1
    ids[8, 0] = v
    ids[9, :] = ids[9, 0]
    w = np.random.default_rng(3).normal(size=T).astype(np.float32)
    w[10:40] = 0
    di, dx, dw = dev(ids, torch.int64), dev(x, torch.float32), dev(w, torch.float32)
    vt = max(1, v - 3)
    di[di >= vt] = -1
    bad, bad2 = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
    loss, state = lp.distill_forward(t, di, dx, v_true=vt, bad_rows=bad)
    grad = lp.distill_backward(t, di, dx, state, dw, v_true=vt)
    loss2, grad2 = lp.distill_step(t, di, dx, dw, v_true=vt, bad_rows=bad2)
    parts = []
    for a in range(0, T, 100):
        b = slice(a, a + 100)
        parts.append(lp.distill_step(t[b], di[b], dx[b], dw[b], v_true=vt))
    loss3, grad3 = (torch.cat(p) for p in zip(*parts))
    loss4, grad4 = lp.distill_step(t, di, dx, dw, v_true=vt, out=t)
    assert grad4.data_ptr() == t.data_ptr() and torch.equal(bad, bad2)

    def same(a, b):
        return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    for other in (loss2, loss3, loss4):
        assert torch.equal(loss.nan_to_num(-9.0), other.nan_to_num(-9.0))
    for other in (grad2, grad3, grad4):
        assert torch.equal(grad.isnan(), other.isnan())
        assert same(grad.nan_to_num(0.0), other.nan_to_num(0.0))
    assert not grad[:, vt:].any() and not grad[10:40].any()


def test_many_rows():
    """More rows than fit any cache: every row against torch in fp64."""
    T, v, k = 3000, 30000, 16
    g = torch.Generator(device=DEV).manual_seed(3)
    t = (torch.randn(T, v, generator=g, device=DEV) * 2).to(torch.bfloat16)
    ids = torch.randint(0, v, (T, k), generator=g, device=DEV)
    x = torch.randn(T, k, generator=g, device=DEV)
    w = (torch.arange(T, device=DEV) % 5 != 0).float()
    loss, grad = lp.distill_step(t, ids, x, w)
    for a in range(0, T, 500):
        s = t[a:a + 500].double()
        logp = torch.log_softmax(s, 1)
        q = torch.softmax(x[a:a + 500].double(), 1)
        ref = (q * (q.log() - logp.gather(1, ids[a:a + 500]))).sum(1)
        assert ((loss[a:a + 500] - ref).abs() <= S_ERR + 2.0 ** -24 * ref.abs()).all()
        p = logp.exp()
        r = (p.scatter_add(1, ids[a:a + 500], -q)) * w[a:a + 500, None]
        err = (grad[a:a + 500].double() - r).abs()
        assert (err <= 2.0 ** -8 * r.abs() + DENSE_ERR * 1.01 * p).all()


def test_wrong_arguments():
    z = torch.zeros(4, 10, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    x, w = torch.zeros(4, 2, device=DEV), torch.zeros(4, device=DEV)
    state = torch.zeros(4, 4, dtype=torch.float64, device=DEV)
    flat = torch.zeros(100, device=DEV)
    for bad in (lambda: lp.distill(z, ids.int(), x), lambda: lp.distill(z, ids, x.double()),
                lambda: lp.distill(z, ids, x[:, :1]), lambda: lp.distill(z, ids[:3], x[:3]),
                lambda: lp.distill(z, ids[:, :0], x[:, :0]), lambda: lp.distill(z, ids, x.cpu()),
                lambda: lp.distill(z.t(), ids, x), lambda: lp.distill(z.int(), ids, x),
                lambda: lp.distill(z, ids, x, v_true=11),
                lambda: lp.distill_step(z, ids, x, w[:3]),
                lambda: lp.distill_step(z, ids, x, w, out=z[:, :9]),
                lambda: lp.distill_step(z, ids, x, w, out=z.bfloat16()),
                lambda: lp.distill_step(flat[:40].view(4, 10), ids, x, w,
                                        out=flat[20:60].view(4, 10)),
                lambda: lp.distill_backward(z, ids, x, state.float(), w),
                lambda: lp.distill_backward(z, ids, x, state, w, out=z.requires_grad_(True))):
        with pytest.raises(ValueError):
            bad()
    z = z.detach()
    with pytest.raises(lp.LpError):
        lp.distill(z, ids, x, temperature=0.0)
    assert lp.distill(z[:0], ids[:0], x[:0]).shape == (0,)
