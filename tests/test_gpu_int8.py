"""The 8-bit head on the GPU (lp_quantize_int8, lp_logits_int8, lp_score_int8)
against its fp64 oracle. Codes, scales and logits are held bit for bit: the
definition names every rounding. Scores have a bound from their arithmetic."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import int8_head as oracle

from .gpu_helpers import DEV
from .logits_helpers import TYPES, dev, place

pytestmark = pytest.mark.gpu

LP_INT8_BLOCK = 128


def bits(t):
    t = t.contiguous()
    return t.view({8: torch.int64, 4: torch.int32, 2: torch.int16, 1: torch.int8}[t.element_size()])


def same_bits(a, b):
    return torch.equal(bits(a), bits(b))


# ---- The quantiser ------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("r,h,pad,lead", [(1, 1, 0, 0), (3, 15, 1, 1), (5, 16, 0, 0), (2, 17, 3, 5),
                                          (7, 511, 0, 3), (64, 1000, 7, 0), (9, 4096, 0, 0),
                                          (2, 8200, 5, 2), (300, 64, 0, 0), (2, 16384, 0, 0),
                                          (3, 16400, 8, 0), (2, 40003, 1, 3), (1, 3000001, 0, 0)])
def test_codes_and_scales(dtype, r, h, pad, lead):
    rng = np.random.default_rng(r * 1000 + h)
    z = rng.normal(size=(r, h)) * np.exp(rng.normal(size=(r, 1)))
    z[rng.random((r, h)) < 0.05] *= 20
    x, exact = place(z, dtype, pad, lead)
    q, s = lp.quantize_int8(x, check=True)
    rq, rs = oracle.quantize(exact)
    assert q.stride(0) % 16 == 0 and q.data_ptr() % 16 == 0
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_halves_go_to_the_even_code():
    """Rows whose scale is 1 (or a power of two), and every half between codes,
    with the neighbouring floats on either side."""
    half = np.arange(-126.5, 127.0, 1.0, dtype=np.float32)
    row = np.concatenate([[np.float32(127)], half, np.nextafter(half, np.float32(200)),
                          np.nextafter(half, np.float32(-200))])
    x = np.stack([row * np.float32(2.0 ** e) for e in (0, -20, 30, -110, -126)])
    q, s = lp.quantize_int8(dev(x, torch.float32))
    rq, rs = oracle.quantize(x)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


def test_borders_under_awkward_scales():
    """Quotients as near a half as fp32 values come, under scales that are no
    powers of two: a rounded quotient would go to the other code."""
    rng = np.random.default_rng(3)
    rows = []
    for _ in range(64):
        top = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-100, 100))
        s = np.float64(top * (np.float32(1) / np.float32(127)))
        near = ((rng.integers(-126, 126, 255) + 0.5) * s).astype(np.float32)
        near = np.where(rng.random(255) < 0.5, near, np.nextafter(near, np.float32(0)))
        rows.append(np.concatenate([[top], near]))
    x = np.array(rows, np.float32)
    q, s = lp.quantize_int8(dev(x, torch.float32))
    rq, rs = oracle.quantize(x)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


def test_rows_without_codes():
    tiny = 2.0 ** -149
    x = np.array([[0, 0, 0], [1, np.nan, 2], [1, -np.inf, 2], [tiny, 0, 0], [64 * tiny, tiny, 0],
                  [200 * tiny, -199 * tiny, 3 * tiny], [3e38, -3.4e38, 1.0], [1, 2, 3]], np.float32)
    bad = torch.full((1,), 5, dtype=torch.int32, device=DEV)
    q, s = lp.quantize_int8(dev(x, torch.float32), bad_rows=bad)
    rq, rs = oracle.quantize(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert bad.item() == 7
    with pytest.raises(ValueError, match="^2 row"):
        lp.quantize_int8(dev(x, torch.float32), check=True)


def test_quantise_into_given_rows():
    x, exact = place(np.random.default_rng(1).normal(size=(5, 21)), "bf16", 3)
    buf = torch.full((5, 48), 77, dtype=torch.int8, device=DEV)
    scale = torch.empty(5, device=DEV)
    q, s = lp.quantize_int8(x, out=buf[:, :21], scale=scale)
    assert s is scale and q.data_ptr() == buf.data_ptr()
    rq, _ = oracle.quantize(exact)
    got = buf.cpu().numpy()
    assert np.array_equal(got[:, :21], rq) and (got[:, 21:32] == 0).all() and (got[:, 32:] == 77).all()
    with pytest.raises(ValueError, match="multiples of 16"):
        lp.quantize_int8(x, out=torch.empty(5, 21, dtype=torch.int8, device=DEV))
    short = torch.empty(4 * 32 + 21, dtype=torch.int8, device=DEV).as_strided((5, 21), (32, 1))
    with pytest.raises(ValueError, match="last row"):
        lp.quantize_int8(x, out=short)


def test_no_rows():
    q, s = lp.quantize_int8(torch.empty(0, 33, device=DEV))
    assert q.shape == (0, 33) and s.shape == (0,)
    w, ws = lp.quantize_int8(torch.randn(7, 33, device=DEV))
    assert lp.logits_int8(q, s, w, ws).shape == (0, 7)
    assert lp.score_int8(q, s, w, ws, torch.empty(0, dtype=torch.int64, device=DEV)).shape == (0,)


# ---- Products -------------------------------------------------------------------

def codes(rng, rows, h, pad=0, lead=0, low=-127):
    """Codes in rows of a padded buffer (multiples of 16 bytes with pad 0), what
    lies around them filled with other codes, and their scales."""
    ld = (h + 15) // 16 * 16 + pad
    buf = torch.full((lead + rows * ld + 16,), 99, dtype=torch.int8, device=DEV)
    q = rng.integers(low, 128, (rows, h)).astype(np.int8)
    t = buf[lead:lead + rows * ld].view(rows, ld)[:, :h]
    t.copy_(torch.from_numpy(q))
    s = (np.exp(rng.normal(size=rows)) * 0.02).astype(np.float32)
    return t, dev(s, torch.float32), q, s


SIZES = [(1, 1, 1), (1, 128, 64), (2, 127, 129), (3, 257, 33), (16, 300, 256), (17, 129, 100),
         (31, 515, 1001), (33, 1000, 384), (64, 640, 128), (65, 700, 130), (100, 1025, 640),
         (129, 384, 17), (257, 513, 256), (300, 2049, 72), (513, 1300, 200)]
# Tiles of 64, 128, 160, 192 and 256 tokens, one, two and three of them, rows of one
# stage and more, ends inside a tile and a block.
SIZES += [(17, 33000, 33), (64, 32897, 200), (100, 17000, 129), (150, 11100, 128),
          (190, 11009, 300), (200, 8300, 16), (256, 8321, 257), (300, 6600, 385),
          (384, 6001, 100), (513, 4000, 520), (700, 3001, 72), (2000, 1152, 500),
          (100, 33001, 129), (250, 40000, 130), (300, 33100, 70), (390, 32900, 40),
          (160, 33000, 256), (180, 65700, 64), (64, 65700, 256), (100, 140000, 64), (33, 140000, 140)]
# Streams: few tokens, rows of 16 stages and more, and enough of them.
SIZES += [(1, 8321, 2000), (16, 8321, 2048), (5, 10001, 4100), (17, 8400, 1921), (32, 32700, 2050),
          (9, 33000, 1930), (32, 32800, 2000)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("t,v,h", SIZES)
def test_logits_bit_for_bit(dtype, t, v, h):
    rng = np.random.default_rng(t + v + h)
    x, xs, qx, sx = codes(rng, t, h)
    w, ws, qw, sw = codes(rng, v, h)
    got = lp.logits_int8(x, xs, w, ws, dtype=TYPES[dtype])
    want = torch.from_numpy(oracle.logits_f32(qx, sx, qw, sw)).to(TYPES[dtype])
    assert got.shape == (t, v) and got.dtype == TYPES[dtype]
    assert same_bits(got.cpu(), want)


@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (5, 3), (16, 16), (112, 0)])
@pytest.mark.parametrize("t,v,h", [(5, 300, 128), (40, 260, 256), (150, 400, 300), (300, 300, 512),
                                   (50, 33000, 128), (140, 11111, 200)])
def test_hidden_states_lie_anywhere(t, v, h, pad, lead):
    rng = np.random.default_rng(7)
    x, xs, qx, sx = codes(rng, t, h, pad, lead)
    w, ws, qw, sw = codes(rng, v, h, pad=32, lead=16)
    want = oracle.logits_f32(qx, sx, qw, sw)
    assert np.array_equal(lp.logits_int8(x, xs, w, ws, dtype=torch.float32).cpu().numpy(), want)


@pytest.mark.parametrize("t,v", [(3, 333), (40, 333), (200, 333), (70, 17005), (135, 11205),
                                 (180, 11205), (520, 4101)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_logits_into_a_wider_buffer(t, v, dtype):
    """Rows of any stride and alignment; the columns around them stay."""
    rng = np.random.default_rng(t)
    x, xs, qx, sx = codes(rng, t, 96)
    w, ws, qw, sw = codes(rng, v, 96)
    want = torch.from_numpy(oracle.logits_f32(qx, sx, qw, sw)).to(TYPES[dtype])
    for columns, lead in ((v, 0), (v + 7, 0), (v + 18, 1), (v + 51, 5)):
        buf = torch.full((lead + t * columns + 64,), -7.0, dtype=TYPES[dtype], device=DEV)
        rows = buf[lead:lead + t * columns].view(t, columns)
        got = lp.logits_int8(x, xs, w, ws, out=rows[:, :v])
        assert got.data_ptr() == rows.data_ptr()
        assert same_bits(rows[:, :v].cpu(), want)
        assert (rows[:, v:] == -7).all() and (buf[:lead] == -7).all()
        assert (buf[lead + t * columns:] == -7).all()


def test_the_widest_rows():
    """Rows 2^22 fp32 columns apart: a wave's 128 tokens span 2 GiB."""
    rng = np.random.default_rng(22)
    t, v, ld = 250, 8500, 1 << 22
    x, xs, qx, sx = codes(rng, t, 64)
    w, ws, qw, sw = codes(rng, v, 64)
    rows = torch.empty(t, ld, device=DEV)
    rows[:, v:v + 200].fill_(-7)
    lp.logits_int8(x, xs, w, ws, out=rows[:, :v])
    assert np.array_equal(rows[:, :v].cpu().numpy(), oracle.logits_f32(qx, sx, qw, sw))
    assert (rows[:, v:v + 200] == -7).all()
    lp.logits_int8(x[:5], xs[:5], w, ws, out=rows[7:12, 100:v + 100])
    assert np.array_equal(rows[7:12, 100:v + 100].cpu().numpy(),
                          oracle.logits_f32(qx[:5], sx[:5], qw, sw))


def test_the_largest_sums():
    """-128 times -128 over the longest rows: 2^31 - 2^14."""
    h = 131071
    x = torch.full((17, 131072), -128, dtype=torch.int8, device=DEV)[:, :h]
    w = torch.full((3, 131072), -128, dtype=torch.int8, device=DEV)[:, :h]
    w[1] = 127
    one = torch.ones(17, device=DEV)
    got = lp.logits_int8(x, one, w, one[:3], dtype=torch.float32)
    want = np.array([h * 2 ** 14, -h * 128 * 127, h * 2 ** 14], np.int64).astype(np.float32)
    assert np.array_equal(got.cpu().numpy(), np.broadcast_to(want, (17, 3)))


def test_scales_that_are_no_numbers():
    rng = np.random.default_rng(5)
    for t, v in ((4, 300), (70, 300), (200, 300), (70, 16500), (140, 11100), (200, 8301)):
        x, xs, qx, sx = codes(rng, t, 64)
        w, ws, qw, sw = codes(rng, v, 64)
        xs[1], ws[7], ws[200] = float("nan"), float("inf"), 0.0
        sx[1], sw[7], sw[200] = np.nan, np.inf, 0.0
        got = lp.logits_int8(x, xs, w, ws, dtype=torch.float32).cpu().numpy()
        z = oracle.logits_f32(qx, sx, qw, sw)
        assert np.array_equal(got, z, equal_nan=True)
        ids = torch.zeros(t, dtype=torch.int64, device=DEV)
        # The infinite scale's logits: +inf has no score, -inf is probability 0.
        gone = (np.isnan(z) | np.isposinf(z)).any(axis=1)
        assert 1 < gone.sum() < t
        out = lp.score_int8(x, xs, w, ws, ids).cpu().numpy()
        assert np.array_equal(np.isnan(out), gone)
        # A row's own scale is that row's matter alone.
        ws[7] = 1e-3
        out = lp.score_int8(x, xs, w, ws, ids)
        assert torch.isnan(out).nonzero().flatten().tolist() == [1]


def score_bound(z, temperature, v, scores):
    """|error| of a score in nats. With e = 2^-24: the logit has three roundings
    and log2(e) / temperature and its product two more (5 e |z| / tau, for the
    target and for the sum's terms); a term of the sum is one exponential
    (2 e, and e of its argument, at most |2 z| / tau) and a block's 31 + 2 sums;
    joining takes 4 roundings and an exponential a step, over ceil(blocks / 64)
    blocks of a segment, two pairs of segments and 15 more, of which those without
    a block cost nothing (at most ceil(blocks / 16) + 16 in all); logarithm,
    difference and the last product 4 e of the scores' size."""
    e = 2.0 ** -24
    size = np.abs(z).max() / temperature
    steps = -(-(-(-v // LP_INT8_BLOCK)) // 16) + 16
    return e * (12 * size + 36 + 6 * steps + 4 * (np.abs(scores).max() + size + 12))


@pytest.mark.parametrize("t,v,h", SIZES + [(8, 20000, 64), (70, 20000, 64)])
@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_scores(t, v, h, temperature):
    rng = np.random.default_rng(t + v + h)
    x, xs, qx, sx = codes(rng, t, h)
    w, ws, qw, sw = codes(rng, v, h)
    sx *= np.float32(0.3 / np.sqrt(h))
    xs.mul_(np.float32(0.3 / np.sqrt(h)))
    ids = rng.integers(0, v, t)
    lse = torch.empty(t, device=DEV)
    got = lp.score_int8(x, xs, w, ws, dev(ids, torch.int64), temperature, lse=lse, check=True)
    z = oracle.logits(qx, xs.cpu().numpy(), qw, sw)
    want, want_lse = oracle.log_softmax_at(z, ids, temperature)
    bound = score_bound(z, temperature, v, want)
    assert np.abs(got.cpu().numpy() - want).max() <= bound
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= bound


@pytest.mark.parametrize("t,v,h", [(5, 1000, 64), (40, 700, 256), (300, 1500, 128), (60, 32900, 64),
                                   (150, 11300, 300), (520, 4001, 128)])
def test_scores_of_bf16_logits(t, v, h):
    rng = np.random.default_rng(t)
    x, xs, qx, sx = codes(rng, t, h)
    w, ws, qw, sw = codes(rng, v, h)
    ids = rng.integers(0, v, t)
    got = lp.score_int8(x, xs, w, ws, dev(ids, torch.int64), bf16_logits=True)
    z = torch.from_numpy(oracle.logits_f32(qx, sx, qw, sw)).bfloat16().double().numpy()
    want, _ = oracle.log_softmax_at(z, ids)
    assert np.abs(got.cpu().numpy() - want).max() <= score_bound(z, 1.0, v, want)


def test_padding_rows_of_the_head_do_not_count():
    rng = np.random.default_rng(2)
    x, xs, qx, _ = codes(rng, 20, 64)
    w, ws, _, _ = codes(rng, 500, 64)
    ids = dev(rng.integers(0, 300, 20), torch.int64)
    part = lp.score_int8(x, xs, w[:300], ws[:300], ids)
    assert same_bits(part, lp.score_int8(x, xs, w, ws, ids, v_true=300))


def test_targets_outside_the_vocabulary():
    rng = np.random.default_rng(2)
    for t in (5, 80):
        x, xs, _, _ = codes(rng, t, 64)
        w, ws, _, _ = codes(rng, 300, 64)
        ids = torch.zeros(t, dtype=torch.int64, device=DEV)
        ids[0], ids[2], ids[3], ids[4] = -1, 300, 2 ** 40, -2 ** 40
        bad = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = lp.score_int8(x, xs, w, ws, ids, bad_rows=bad)
        assert torch.isnan(out).nonzero().flatten().tolist() == [0, 2, 3, 4] and bad.item() == 4
        with pytest.raises(ValueError, match="^4 row"):
            lp.score_int8(x, xs, w, ws, ids, check=True)


def test_negative_scales():
    """Scales are any numbers: the smallest sum then is the largest logit."""
    rng = np.random.default_rng(8)
    for t, v in ((9, 400), (100, 400), (150, 11100)):
        x, xs, qx, sx = codes(rng, t, 64)
        w, ws, qw, sw = codes(rng, v, 64)
        xs[::2] *= -1
        xs[3] = 0
        ws[::3] *= -1
        sx, sw = xs.cpu().numpy(), ws.cpu().numpy()
        got = lp.logits_int8(x, xs, w, ws, dtype=torch.float32).cpu().numpy()
        assert np.array_equal(got, oracle.logits_f32(qx, sx, qw, sw))
        ids = rng.integers(0, v, t)
        for rounded in (False, True):
            z = torch.from_numpy(oracle.logits_f32(qx, sx, qw, sw))
            z = z.bfloat16().double().numpy() if rounded else oracle.logits(qx, sx, qw, sw)
            out = lp.score_int8(x, xs, w, ws, dev(ids, torch.int64), bf16_logits=rounded)
            want, _ = oracle.log_softmax_at(z, ids)
            assert np.abs(out.cpu().numpy() - want).max() <= score_bound(z, 1.0, v, want)


def test_a_rows_bits_do_not_depend_on_its_batch():
    rng = np.random.default_rng(11)
    v = 20011
    x, xs, _, _ = codes(rng, 700, 384)
    w, ws, _, _ = codes(rng, v, 384)
    ids = dev(rng.integers(0, v, 700), torch.int64)
    z = lp.logits_int8(x, xs, w, ws, dtype=torch.float32)
    s = lp.score_int8(x, xs, w, ws, ids)
    for lo, hi in ((0, 1), (5, 12), (3, 19), (10, 40), (100, 164), (0, 65), (50, 200), (10, 300),
                   (0, 513), (2, 140), (30, 190), (17, 700), (699, 700)):
        assert same_bits(lp.logits_int8(x[lo:hi], xs[lo:hi], w, ws, dtype=torch.float32), z[lo:hi])
        assert same_bits(lp.score_int8(x[lo:hi], xs[lo:hi], w, ws, ids[lo:hi]), s[lo:hi])


def test_given_outputs_count_as_written():
    rng = np.random.default_rng(4)
    x, xs, _, _ = codes(rng, 4, 48)
    w, ws, _, _ = codes(rng, 9, 48)
    out, lse, z = torch.empty(4, device=DEV), torch.empty(4, device=DEV), torch.empty(4, 9, device=DEV)
    q, s = torch.empty(4, 16, dtype=torch.int8, device=DEV), torch.empty(4, device=DEV)
    lp.score_int8(x, xs, w, ws, torch.zeros(4, dtype=torch.int64, device=DEV), out=out, lse=lse)
    lp.logits_int8(x, xs, w, ws, out=z)
    lp.quantize_int8(z, out=q[:, :9], scale=s)
    assert [t._version for t in (out, lse, z, q, s)] == [1] * 5


def test_refusals_on_the_device():
    rng = np.random.default_rng(1)
    x, xs, _, _ = codes(rng, 4, 48)
    w, ws, _, _ = codes(rng, 9, 48)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    for args, text in (((x, xs, w[:, :32], ws), "one H"), ((x, xs[:3], w, ws), "x_scale"),
                       ((x, xs, w, ws.double()), "w_scale"), ((x.float(), xs, w, ws), "int8"),
                       ((x, xs, w[:, 1:], ws), "multiples of 16|one H"),
                       ((x, xs, w[:0], ws[:0]), "must have a row")):
        with pytest.raises(ValueError, match=text):
            lp.logits_int8(*args)
        with pytest.raises(ValueError, match=text):
            lp.score_int8(*args, ids)
    wide = torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError, match="apart from x"):
        lp.quantize_int8(wide, out=wide.view(torch.int8)[:, :64])
    with pytest.raises(ValueError, match="apart from x"):
        lp.logits_int8(wide.view(torch.int8)[:, :48], xs, w, ws, out=wide[:, 40:49])
    short = torch.zeros(33, dtype=torch.int8, device=DEV).view(1, 33)
    with pytest.raises(ValueError, match="last row"):
        lp.logits_int8(codes(rng, 4, 33)[0], xs, short, ws[:1])
    with pytest.raises(ValueError, match="dtype"):
        lp.logits_int8(x, xs, w, ws, dtype=torch.float64)
    with pytest.raises(ValueError, match="out"):
        lp.logits_int8(x, xs, w, ws, out=torch.empty(4, 8, device=DEV))
    with pytest.raises(ValueError, match="v_true"):
        lp.score_int8(x, xs, w, ws, ids, v_true=10)
    with pytest.raises(lp.LpError):
        lp.score_int8(x, xs, w, ws, ids, temperature=0.0)
    with pytest.raises(lp.LpError):
        lp.logits_int8(x, xs, w, ws, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
