"""Norms and rotary positions of queries and keys (forward, backward, on the way
into a paged cache) against the 64-bit model (tests/_gradient_model.py).

Tolerances, per element, with A the sum of the absolute terms that the model
gives. Outputs are rounded once to bf16: 2^-8 of the value. In 32 bits, a mean
of d <= 128 squares is off by less than 2^-17 of itself and its root by half of
that, the angle's fraction of a turn has 24 bits (pi 2^-24 at most), cosines
and products add a few 2^-24: 2^-17 A in all. Backward there are two such
means: 2^-16 A. The weights' gradients sum terms that carry 2^-16 each, in
chains of less than 2^8 additions (2^-16 of the terms): 2^-15 A.
"""
import copy
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import gqa_attention_softmax_gb300 as sa
from gqa_attention_softmax_gb300 import _build
from gqa_attention_softmax_gb300._binding import BAD_LENGTHS, INVALID_ARG, UNSUPPORTED
from _gradient_model import (Rotation, attention, attention_gradients, hnd_rows, norm, rotated,
                             rotated_gradients)

gpu = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    yield
    if torch.cuda.is_available():
        assert sa.sinkattn_debug_status() == 0


# ----------------------------------------------------------------------------
# frequencies (host)
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("r", [0, 2, 64, 70, 128])
def test_plain_frequencies(r):
    inv, a = sa.sinkattn_rope_frequencies(r, 10000.0)
    assert a == 1.0 and np.allclose(inv, [10000.0 ** (-2.0 * i / r) for i in range(r // 2)], rtol=1e-14)


def test_scaled_frequencies():
    plain, _ = sa.sinkattn_rope_frequencies(64, 10000.0)
    lin, a = sa.sinkattn_rope_frequencies(64, 10000.0, "linear", 4.0)
    assert a == 1.0 and np.allclose(lin, np.array(plain) / 4, rtol=1e-14)
    ntk, a = sa.sinkattn_rope_frequencies(64, 10000.0, "ntk", 4.0)
    # the fastest pair stays, the slowest is divided by the factor
    assert a == 1.0 and ntk[0] == plain[0] and math.isclose(ntk[-1], plain[-1] / 4, rel_tol=1e-12)
    yarn, a = sa.sinkattn_rope_frequencies(64, 10000.0, "yarn", 8.0, 4096)
    assert math.isclose(a, 0.1 * math.log(8.0) + 1.0, rel_tol=1e-7)
    ratio = np.array(yarn) / np.array(plain)
    turns = 4096 * np.array(plain) / (2 * math.pi)   # within the original length
    assert np.allclose(ratio[turns > 32], 1.0) and np.allclose(ratio[turns < 1], 1 / 8)
    assert (np.diff(ratio) <= 1e-15).all() and ((ratio > 1 / 8 + 1e-9) & (ratio < 1 - 1e-9)).any()


def test_yarn_between_the_borders():
    """gpt-oss's constants: the borders are the indices 8.0927791 and 17.398024, the shares
    between them written out."""
    plain, _ = sa.sinkattn_rope_frequencies(64, 150000.0)
    yarn, a = sa.sinkattn_rope_frequencies(64, 150000.0, "yarn", 32.0, 4096)
    kept = {0: 1.0, 8: 1.0, 9: 0.9055510956043724, 10: 0.80144314790322064, 11: 0.69733520020206889,
            12: 0.59322725250091713, 13: 0.48911930479976537, 14: 0.38501135709861361,
            15: 0.28090340939746185, 16: 0.17679546169631009, 17: 0.072687513995158332,
            18: 0.03125, 31: 0.03125}
    for i, share in kept.items():
        assert math.isclose(yarn[i] / plain[i], share, rel_tol=1e-12), i
    assert math.isclose(yarn[10], 0.019335001126540358, rel_tol=1e-12)
    assert math.isclose(a, 1.3465735902799727, rel_tol=1e-7)


@pytest.mark.parametrize("r", [2, 64])
def test_yarn_of_pairs_that_all_turn_less_than_the_slow_border(r):
    """Five positions, of which the fastest pair makes 0.8 turns: every frequency is divided."""
    plain, _ = sa.sinkattn_rope_frequencies(r, 10000.0)
    yarn, _ = sa.sinkattn_rope_frequencies(r, 10000.0, "yarn", 8.0, 5)
    assert np.allclose(np.array(yarn) / np.array(plain), 1 / 8, rtol=1e-12)


def test_turns():
    """Turns are the frequency over 2 pi modulo 1 (of doubles: 2^-52 of the quotient)."""
    freq = [1.0, 0.5, 1e-4, 2 * math.pi * 3.25, -0.25 * 2 * math.pi, 0.0]
    for f, t in zip(freq, sa.sinkattn_rope_turns(freq)):
        want = (f / (2 * math.pi)) % 1.0
        got = t / 2.0 ** 64
        off = abs(got - want)
        assert min(off, 1 - off) <= 2.0 ** -50 * max(1.0, abs(f)), f


def test_turns_are_rounded_to_the_nearest_word():
    """Against 1 / (2 pi) to 60 digits: half a unit of 2^-64, and where the frequency has f
    turns a position 2^-100 f of them for the two-double product (2^-30 of a unit up to 2^6)."""
    inv_2pi = Fraction("0.159154943091895335768883763372514362034459645740456448747667")
    freq = [1.0, 0.3, -0.01, 1e-4, 7.5, -7.5, 0.0, 1e-18, 1e-30, 2 * math.pi, 63.9, -1e-19]
    for scaling in ("none", "linear", "ntk", "yarn"):
        freq += sa.sinkattn_rope_frequencies(128, 150000.0, scaling, 32.0, 4096)[0]
    for f, t in zip(freq, sa.sinkattn_rope_turns(freq)):
        assert 0 <= t < 2 ** 64
        off = (Fraction(f) * inv_2pi * 2 ** 64 - t) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 30), f
    # (whole turns and more are modulo 1, without an overflow on the way)
    for f in (1e15, -3e18, 1e300, 1.7e308):
        assert 0 <= sa.sinkattn_rope_turns([f])[0] < 2 ** 64


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=7), dict(rotary_dim=-2), dict(base=1.0), dict(base=float("nan")),
    dict(scaling="other"), dict(scaling=9), dict(scaling="linear", factor=0.5),
    dict(scaling="ntk", factor=float("inf")), dict(scaling="yarn", factor=2.0, original_len=0),
    dict(scaling="yarn", factor=2.0, original_len=9, beta_fast=1.0, beta_slow=2.0)])
def test_frequencies_refusals(kw):
    with pytest.raises(sa.SinkAttnError) as e:
        sa.sinkattn_rope_frequencies(**{"rotary_dim": 64, **kw})
    assert e.value.status == INVALID_ARG


def test_turns_refusals():
    for bad in (float("nan"), float("inf")):
        with pytest.raises(sa.SinkAttnError):
            sa.sinkattn_rope_turns([1.0, bad])


@pytest.mark.parametrize("name", ["rotary_dim", "interleaved", "attention_factor", "inv_freq", "turns",
                                  "device"])
def test_a_rope_does_not_change(name):
    """(A rotary_dim that grew would send the kernels past the end of the words.)"""
    rope = sa.Rope.__new__(sa.Rope)   # (a whole one needs a device)
    with pytest.raises(AttributeError):
        setattr(rope, name, 128)


@gpu
def test_rope_attributes():
    rope = sa.Rope(64, base=150000.0, interleaved=True, scaling="yarn", factor=32.0, original_len=4096)
    inv, a = sa.sinkattn_rope_frequencies(64, 150000.0, "yarn", 32.0, 4096)
    assert rope.rotary_dim == 64 and rope.interleaved is True and rope.attention_factor == a
    assert rope.inv_freq == tuple(inv) and rope.device == torch.device("cuda", torch.cuda.current_device())
    assert [t % 2 ** 64 for t in rope.turns.tolist()] == sa.sinkattn_rope_turns(inv)
    # a copy, as of a model that holds one, has words of its own
    x, rot, cu, T = make([20], 8, 2, 64, 64)
    want = forward(x)
    twin = copy.deepcopy(x["rope"])
    assert twin.turns.data_ptr() != x["rope"].turns.data_ptr()
    x["rope"].turns.zero_()
    x["rope"] = twin
    for a, b in zip(want, forward(x)):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def make(lens, hq, hkv, d, rotary, interleaved=False, q_norm=True, k_norm=True, positions=None,
         scaling="yarn", seed=0, behind=0):
    gen = torch.Generator().manual_seed(seed)
    cu = np.cumsum([0] + list(lens)).tolist()
    T = cu[-1]
    width = (hq + 2 * hkv) * d
    rows = torch.randn((T + behind, width), generator=gen).to(torch.bfloat16).cuda()
    w = [(1 + 0.3 * torch.randn(d, generator=gen)).cuda() for _ in range(2)]
    kw = dict(base=150000.0, scaling=scaling, factor=1.0 if scaling == "none" else 32.0,
              original_len=4096)
    rope = sa.Rope(rotary, interleaved=interleaved, **kw)
    pos = torch.cat([torch.arange(n) for n in lens]) if positions is None else torch.tensor(positions)
    x = dict(q=rows[:, :hq * d].view(-1, hq, d), k=rows[:, hq * d:(hq + hkv) * d].view(-1, hkv, d),
             v=rows[:, (hq + hkv) * d:].view(-1, hkv, d),
             q_weight=w[0] if q_norm else None, k_weight=w[1] if k_norm else None, rope=rope,
             cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             positions=None if positions is None else pos.int().cuda())
    rot = Rotation(rope.inv_freq, rope.attention_factor, interleaved, pos.cuda())
    return x, rot, cu, T


def forward(x, **kw):
    return sa.sinkattn_rope_qkv(x["q"], x["k"], x["v"], x["cu"], x["rope"], x["q_weight"],
                                x["k_weight"], EPS, x["positions"], **kw)


def close(got, want, size, what, rel=2.0 ** -8, of=2.0 ** -17):
    assert torch.isfinite(got).all(), what
    err = (got.double() - want).abs()
    tol = rel * want.abs() + of * size + 1e-30
    assert (err <= tol).all(), "%s: %g of the tolerance" % (what, (err / tol).max().item())


def check_forward(got, x, rot, cu, T):
    hkv = x["k"].shape[1]
    rows = hnd_rows(cu, hkv, "cuda")
    close(got[0][:T], *rotated(x["q"][:T], x["q_weight"], EPS, rot), "q")
    close(got[1][rows], *rotated(x["k"][:T], x["k_weight"], EPS, rot), "k")
    assert torch.equal(got[2][rows], x["v"][:T])


SHAPES = [(64, 8, 64), (64, 4, 128), (24, 8, 64), (5, 1, 64), (1, 1, 128), (300, 3, 64)]
ROTARY = [(64, False), (64, True), (32, False), (32, True), (2, False), (6, True), (38, False),
          (0, False), (62, False), (62, True)]


@gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rotary", ROTARY)
@pytest.mark.parametrize("norms", [(True, True), (False, False)])
def test_forward(shape, rotary, norms):
    x = make([17, 0, 1, 40], *shape, *rotary, *norms)
    check_forward(forward(x[0]), *x)


@gpu
@pytest.mark.parametrize("rotary", [(128, False), (128, True), (96, False), (100, False), (126, True)])
@pytest.mark.parametrize("norms", [(True, False), (False, True)])
def test_forward_128(rotary, norms):
    x = make([3, 250], 20, 4, 128, *rotary, *norms)
    check_forward(forward(x[0]), *x)


@gpu
@pytest.mark.parametrize("T", [1, 1300, 2500, 5000])
def test_forward_of_many_tokens(T):
    x = make([T], 8, 2, 64, 64)
    check_forward(forward(x[0]), *x)


@gpu
def test_far_positions():
    """Angles keep their accuracy at any 32-bit position, negative ones too (the
    model's own angles, in doubles, are off by 2^-52 of 2^31 radians: 2^-21)."""
    pos = [0, 1, -1, 131071, 1000003, -77777, 2 ** 31 - 1, -2 ** 31]
    for inter in (False, True):
        x, rot, cu, T = make([8], 8, 2, 64, 64, inter, positions=pos, scaling="none")
        got = forward(x)
        y, size = rotated(x["q"], x["q_weight"], EPS, rot)
        close(got[0], y, size, "q", of=2.0 ** -17 + 2.0 ** -19)


@gpu
def test_given_frequencies():
    inv = [1.0, 0.3, -0.01, 7.5]
    x, _, cu, T = make([30], 4, 2, 64, 8)
    x["rope"] = sa.Rope(8, inv_freq=inv, attention_factor=0.5)
    rot = Rotation(inv, 0.5, False, torch.arange(30, device="cuda"))
    check_forward(forward(x), x, rot, cu, T)


@gpu
def test_rows_behind_the_last_sequence_stay():
    x, rot, cu, T = make([33, 20], 8, 2, 64, 64, behind=11)
    n = T + 11
    outs = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")
            for s in ((n, 8, 64), (2 * n, 64), (2 * n, 64))]
    got = forward(x, q_out=outs[0], k_out=outs[1], v_out=outs[2])
    check_forward(got, x, rot, cu, T)
    assert (got[0][T:] == 7.0).all() and (got[1][2 * T:] == 7.0).all() and (got[2][2 * T:] == 7.0).all()
    rows = torch.full((n, 12, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    sa.sinkattn_rope_qkv_backward(outs[0], outs[1], outs[2], x["cu"], x["rope"], q=x["q"], k=x["k"],
                                  q_weight=x["q_weight"], k_weight=x["k_weight"], dq_in=rows[:, :8],
                                  dk_in=rows[:, 8:10], dv_in=rows[:, 10:])
    assert (rows[T:] == 7.0).all() and (rows[:T] != 7.0).any()


@gpu
def test_no_tokens():
    x, rot, cu, T = make([0, 0], 8, 2, 64, 64)
    q, k, v = forward(x)
    assert q.shape == (0, 8, 64) and k.shape == (0, 64) and v.shape == (0, 64)
    got = sa.sinkattn_rope_qkv_backward(q, k, v, x["cu"], x["rope"], q=x["q"], k=x["k"],
                                        q_weight=x["q_weight"], k_weight=x["k_weight"])
    assert got[0].shape == (0, 8, 64) and got[1].shape == (0, 2, 64)
    assert (got[3] == 0).all() and (got[4] == 0).all()


@gpu
def test_zero_rows():
    """A row of zeros has norm eps: no division by zero, forward or backward."""
    x, rot, cu, T = make([6], 8, 2, 64, 64)
    x["q"][2:4] = 0
    got = forward(x)
    check_forward(got, x, rot, cu, T)
    g = grads(x, cu)
    check_backward(backward(x, g), g, x, rot, cu)


@gpu
@pytest.mark.parametrize("d,r,inter", [(64, 32, False), (64, 38, False), (64, 0, False), (64, 6, True),
                                       (128, 64, False), (128, 100, True), (128, 126, False)])
@pytest.mark.parametrize("q_norm", [False, True])
def test_elements_that_are_not_rotated_stay_as_they_are(d, r, inter, q_norm):
    """Bit for bit without a norm, whatever stands beside them: infinities, NaN, both zeros.
    (q with a norm, k without: the second path of the same launches.)"""
    x, rot, cu, T = make([40, 23], 8, 3, d, r, inter, q_norm, False)
    gen = torch.Generator().manual_seed(6)
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0, 0.0, 1.0, -2.0], dtype=torch.bfloat16)
    mix = lambda *s: odd[torch.randint(0, 7, s, generator=gen)].cuda()   # noqa: E731

    def same(a, b):
        return bool(((a.view(torch.int16) == b.view(torch.int16)) | (a.isnan() & b.isnan())).all())

    x["k"][..., r:] = mix(T, 3, d - r)
    if not q_norm:
        x["q"][..., r:] = mix(T, 8, d - r)
    rows = hnd_rows(cu, 3, "cuda")
    q, k, v = forward(x)
    assert same(k[rows][..., r:], x["k"][..., r:])
    assert torch.isfinite(k[rows][..., :r]).all() and torch.isfinite(q[..., :r]).all()
    if not q_norm:
        assert same(q[..., r:], x["q"][..., r:])
    pools = [torch.zeros((4, 3, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    sa.sinkattn_rope_append_paged(x["q"], x["k"], x["v"], pos, slots, x["rope"], *pools, x["q_weight"], None, EPS)
    assert same(pools[0].transpose(1, 2).reshape(-1, 3, d)[:T, :, r:].contiguous(), x["k"][..., r:].contiguous())
    g = [t.clone() for t in grads(x, cu)]
    g[1][..., r:] = mix(3 * T, d - r)
    got = backward(x, g)
    assert same(got[1][..., r:], g[1][rows][..., r:]) and torch.isfinite(got[1][..., :r]).all()


# ----------------------------------------------------------------------------
# backward
# ----------------------------------------------------------------------------
def grads(x, cu, seed=9):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()   # noqa: E731
    T, hq, d = x["q"].shape
    hkv = x["k"].shape[1]
    return r(T, hq, d), r(hkv * T, d), r(hkv * T, d)


def backward(x, g, **kw):
    return sa.sinkattn_rope_qkv_backward(*g, x["cu"], x["rope"], q=x["q"], k=x["k"],
                                         q_weight=x["q_weight"], k_weight=x["k_weight"], eps=EPS,
                                         positions=x["positions"], **kw)


def check_backward(got, g, x, rot, cu):
    rows = hnd_rows(cu, x["k"].shape[1], "cuda")
    for name, dx, dw, dy in (("q", got[0], got[3], g[0]), ("k", got[1], got[4], g[1][rows])):
        w = x[name + "_weight"]
        val, size, wval, wsize = rotated_gradients(dy, x[name], w, EPS, rot)
        close(dx, val, size, "d" + name, of=2.0 ** -16)
        if w is None:
            assert dw is None
        else:
            close(dw, wval, wsize, "weight of " + name, rel=0.0, of=2.0 ** -15)
    assert torch.equal(got[2], g[2][rows])


@gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rotary", ROTARY)
@pytest.mark.parametrize("norms", [(True, True), (False, False)])
def test_backward(shape, rotary, norms):
    x, rot, cu, T = make([17, 0, 1, 40], *shape, *rotary, *norms)
    g = grads(x, cu)
    check_backward(backward(x, g), g, x, rot, cu)


@gpu
@pytest.mark.parametrize("rotary", [(128, False), (128, True), (96, False), (100, False)])
@pytest.mark.parametrize("norms", [(True, False), (False, True), (True, True)])
def test_backward_128(rotary, norms):
    x, rot, cu, T = make([3, 250], 20, 4, 128, *rotary, *norms, positions=list(range(5000, 5253)))
    g = grads(x, cu)
    check_backward(backward(x, g), g, x, rot, cu)


@gpu
@pytest.mark.parametrize("T", [1, 2500, 9000])
def test_backward_of_many_tokens(T):
    x, rot, cu, _ = make([T], 8, 2, 64, 64)
    g = grads(x, cu)
    got = backward(x, g)
    check_backward(got, g, x, rot, cu)
    again = backward(x, g)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("shape,lens", [((24, 8, 64), [70]), ((5, 1, 64), [70]), ((20, 4, 128), [70]),
                                        ((64, 8, 64), [17, 40]), ((64, 8, 64), [1300]),
                                        ((1, 1, 128), [5]), ((1, 1, 64), [3000])])
@pytest.mark.parametrize("norms", [(True, True), (True, False), (False, True)])
def test_eps_of_zero(shape, lens, norms, monkeypatch):
    """Rows that are not zero have gradients without eps, the weights' among them, wherever a
    token's heads do not fill the rows that a warp takes at once."""
    monkeypatch.setitem(globals(), "EPS", 0.0)
    x, rot, cu, T = make(lens, *shape, 64, False, *norms)
    assert (x["q"] != 0).any(-1).all() and (x["k"] != 0).any(-1).all()
    check_forward(forward(x), x, rot, cu, T)
    g = grads(x, cu)
    check_backward(backward(x, g), g, x, rot, cu)


@gpu
@pytest.mark.parametrize("norms", [(True, True), (False, False)])
def test_backward_against_differences(norms):
    """sum(g * y) along random directions of the inputs: the slack is the sum of the elements'
    tolerances, and 1e-6 of the value for the step."""
    x, rot, cu, T = make([9, 4], 6, 2, 64, 48, True, *norms)
    g = grads(x, cu)
    got = backward(x, g)
    rows = hnd_rows(cu, 2, "cuda")
    gen = torch.Generator().manual_seed(2)
    for name, dx, dw, dy in (("q", got[0], got[3], g[0]), ("k", got[1], got[4], g[1][rows])):
        w = x[name + "_weight"]
        _, size, _, wsize = rotated_gradients(dy, x[name], w, EPS, rot)
        for of_weight in (False, True) if w is not None else (False,):
            at = (w if of_weight else x[name]).double()
            way = torch.randn(at.shape, generator=gen, dtype=torch.float64).cuda()
            grad = (dw if of_weight else dx).double()
            tol = 2.0 ** -15 * wsize if of_weight else 2.0 ** -8 * grad.abs() + 2.0 ** -16 * size
            vals = []
            for t in (1e-4, -1e-4):
                moved = at + t * way
                y = rot(norm(x[name].double() if of_weight else moved,
                             moved if of_weight else w, EPS))
                vals.append((y * dy.double()).sum().item())
            diff = (vals[0] - vals[1]) / 2e-4
            slack = (tol * way.abs()).sum().item() + 1e-6 * abs(diff) + 1e-6
            assert abs((grad * way).sum().item() - diff) <= slack


# ----------------------------------------------------------------------------
# on the way into a paged cache
# ----------------------------------------------------------------------------
def slots_of(T, pages, page, seed=4):
    gen = torch.Generator().manual_seed(seed)
    return torch.randperm(pages * page, generator=gen)[:T].int().cuda()


@gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rotary", [(64, False), (64, True), (38, False), (0, False)])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_append(shape, rotary, page, fp8):
    hq, hkv, d = shape
    T, pages = 41, 9
    x, rot, _, _ = make([T], *shape, *rotary, positions=list(range(3000, 3000 + T)))
    slots = slots_of(T, pages, page)
    slots[5], slots[40], slots[7] = -1, pages * page, -2 ** 31   # left out
    keep = torch.tensor([i for i in range(T) if i not in (5, 40, 7)], device="cuda")
    at = slots[keep].long()
    fill = 0x31 if fp8 else 7.0
    dtype = torch.uint8 if fp8 else torch.bfloat16
    pools = [torch.full((pages, hkv, page, d), fill, dtype=dtype, device="cuda") for _ in range(2)]
    args = (x["q"], x["k"], x["v"], x["positions"], slots, x["rope"])
    if fp8:
        gen = torch.Generator().manual_seed(8)
        scales = [((0.8 + 0.4 * torch.rand(hkv, generator=gen)) * 5 / 448).cuda() for _ in range(2)]
        q = sa.sinkattn_rope_append_paged_fp8(*args, *scales, *pools, x["q_weight"], x["k_weight"], EPS)
    else:
        q = sa.sinkattn_rope_append_paged(*args, *pools, x["q_weight"], x["k_weight"], EPS)
    close(q, *rotated(x["q"], x["q_weight"], EPS, rot), "q")
    want, size = rotated(x["k"], x["k_weight"], EPS, rot)
    got = [p[at // page, :, at % page] for p in pools]
    if fp8:
        s = scales[0].double()[None, :, None]
        val = got[0].view(torch.float8_e4m3fn).double()
        q_want, q_size = (want[keep] / s).clamp(-448, 448), size[keep] / s
        # half a step of the quotient (2^-4 of it, 2^-10 where e4m3 is subnormal), and 32-bit errors
        tol = torch.maximum(2.0 ** -4 * q_want.abs(), torch.full_like(q_want, 2.0 ** -10))
        assert ((val - q_want).abs() <= tol + 2.0 ** -16 * q_size).all()
        ref = [torch.full_like(p, fill) for p in pools]
        sa.sinkattn_append_paged_fp8(x["k"], x["v"], slots, *scales, *ref)
        assert torch.equal(pools[1], ref[1])   # v: as appended without the rotation
    else:
        close(got[0], want[keep], size[keep], "k")
        assert torch.equal(got[1], x["v"][keep])
    # the other slots are as they were
    for p in pools:
        rest = torch.ones((pages, page), dtype=torch.bool, device="cuda")
        rest[at // page, at % page] = False
        assert (p.transpose(1, 2)[rest] == fill).all()


@gpu
def test_append_agrees_with_the_packed_form():
    """q, k bit for bit as sinkattn_rope_qkv gives them, at sizes that split the heads otherwise."""
    for T in (1, 64, 700):
        x, _, cu, _ = make([T], 64, 4, 128, 128, positions=list(range(100, 100 + T)))
        q, k, v = forward(x)
        pools = [torch.zeros((T // 16 + 1, 4, 16, 128), dtype=torch.bfloat16, device="cuda")
                 for _ in range(2)]
        slots = torch.arange(T, dtype=torch.int32, device="cuda")
        q2 = sa.sinkattn_rope_append_paged(x["q"], x["k"], x["v"], x["positions"], slots, x["rope"],
                                           *pools, x["q_weight"], x["k_weight"], EPS)
        assert torch.equal(q, q2)
        rows = hnd_rows(cu, 4, "cuda")
        for pool, want in zip(pools, (k, v)):
            assert torch.equal(pool.transpose(1, 2).reshape(-1, 4, 128)[:T], want[rows])


@gpu
def test_serving_step_together():
    """A prompt and one more token of each sequence: reserve, rotate and append, list, attend."""
    hq, hkv, d, page = 64, 8, 64, 16
    lens = [37, 5, 64]
    n = len(lens)
    all_lens = [x + 1 for x in lens]
    x, rot, cu, T = make(all_lens, hq, hkv, d, 64)
    rope_kw = dict(q_weight=x["q_weight"], k_weight=x["k_weight"], eps=EPS)
    first = [i for a, b in zip(cu[:-1], cu[1:]) for i in range(a, b - 1)]
    last = [b - 1 for b in cu[1:]]
    pos = torch.cat([torch.arange(m) for m in all_lens]).int().cuda()
    pools = [torch.zeros((20, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = sa.PageTable(None, 20, page, n, 8)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    for rows, new in ((first, lens), (last, [1] * n)):
        t = torch.tensor(rows, device="cuda")
        cu_new = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
        slots = sa.sinkattn_pages_reserve(table, ids, cu_new, sum(new), *pools)
        q = sa.sinkattn_rope_append_paged(*[x[m][t].contiguous() for m in "qkv"], pos[t], slots,
                                          x["rope"], *pools, **rope_kw)
    kv, ptr, idx = sa.sinkattn_pages_lists(table, ids)
    sinks = torch.zeros(hq, device="cuda")
    out, lse = sa.sinkattn_decode_paged(q, *pools, kv, ptr, idx, sinks, 1, max(all_lens))
    # the whole sequences at once, as a prefill
    qa, ka, va = forward(x)
    want, wlse = attention(qa.double(), ka.double(), va.double(), sinks.double(), cu, cu, hkv,
                           d ** -0.5, True, 0)
    want, wlse = want[last], wlse[last]
    bound = attention(qa.double(), ka.double(), va.double().abs(), sinks.double(), cu, cu, hkv,
                      d ** -0.5, True, 0)[0][last]
    # weights rounded to bf16, the output too, 2^-10 for 32-bit logits
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * bound).all()
    assert (lse.double() - wlse).abs().max() <= 1e-3


@gpu
def test_training_step_together():
    """rope_qkv, prefill, their backward passes, as one graph; against differences of the
    whole in 64 bits. Slack: bf16 roundings of the intermediate q, k, v, out (2^-8 each) act
    through smooth functions; as they are independent over 10^4 elements, 2^-6 of the
    root of the sum of squared terms is several times what they add up to."""
    hq, hkv, d = 8, 2, 64
    x, rot, cu, T = make([40, 23], hq, hkv, d, 64)
    gen = torch.Generator().manual_seed(3)
    dout = torch.randn((T, hq, d), generator=gen).to(torch.bfloat16).cuda()
    sinks = torch.randn(hq, generator=gen).cuda()

    def step():
        q, k, v = forward(x)
        out, lse = sa.sinkattn_prefill(q, k, v, sinks, x["cu"], x["cu"], 40, 40, hkv)
        dq, dk, dv, ds = sa.sinkattn_prefill_backward(dout, q, k, v, out, lse, sinks, x["cu"],
                                                      x["cu"], 40, 40, hkv)
        return (*backward(x, (dq, dk, dv)), ds)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    rows = hnd_rows(cu, hkv, "cuda").view(-1)

    def loss(p):
        y = {}
        for n in "qk":
            y[n] = rot(p[n + "_weight"] * p[n] * torch.rsqrt((p[n] ** 2).mean(-1, keepdim=True) + EPS))
        y["v"] = p["v"]
        hnd = {n: torch.zeros((hkv * T, d), dtype=torch.float64, device="cuda").index_put(
            (rows,), y[n].reshape(-1, d)) for n in "kv"}
        out, _ = attention(y["q"], hnd["k"], hnd["v"], p["sinks"], cu, cu, hkv, d ** -0.5, True, 0)
        return (out * dout.double()).sum()

    at = {n: x[n].double() for n in ("q", "k", "v", "q_weight", "k_weight")}
    at["sinks"] = sinks.double()
    for name, grad in zip(("q", "k", "v", "q_weight", "k_weight", "sinks"), got):
        way = torch.randn(at[name].shape, generator=gen, dtype=torch.float64).cuda()
        vals = [loss(dict(at, **{name: at[name] + t * way})).item() for t in (1e-4, -1e-4)]
        diff = (vals[0] - vals[1]) / 2e-4
        terms = grad.double() * way
        slack = 2.0 ** -6 * terms.square().sum().sqrt().item()
        assert abs(terms.sum().item() - diff) <= slack, name


@gpu
def test_streams():
    x, rot, cu, T = make([300], 64, 8, 64, 64)
    want = forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = forward(x, stream=side)
    g = grads(x, cu)
    side.wait_stream(torch.cuda.current_stream())
    back = backward(x, g, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    check_backward(back, g, x, rot, cu)


@gpu
def test_lengths_beyond_the_tokens_are_recorded():
    x, rot, cu, T = make([30, 10], 8, 2, 64, 64)
    want = forward(x)
    for bad in ([0, 30, 90], [0, 50, 40], [-5, 30, 40]):
        x["cu"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        forward(x)
        assert sa.sinkattn_debug_status() == BAD_LENGTHS
    x["cu"] = torch.tensor([0, 30, 90], dtype=torch.int32, device="cuda")
    got = forward(x)
    assert sa.sinkattn_debug_status() == BAD_LENGTHS
    assert torch.equal(got[0][:30], want[0][:30])
    assert torch.equal(got[1][:60], want[1][:60])


def in_a_field(n):
    """n bytes, 256-byte aligned, between bytes of a pattern, and a check that these are as they were."""
    whole = torch.full((n + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    at = 4096 - whole.data_ptr() % 256
    mine = whole[at:at + n]
    assert mine.data_ptr() % 256 == 0

    def untouched():
        return bool((whole[:at] == 0x5a).all() and (whole[at + n:] == 0x5a).all())
    return mine, untouched


@gpu
@pytest.mark.parametrize("T", [1, 5, 303, 304, 305, 5000])
@pytest.mark.parametrize("shape", [(64, 8, 64), (20, 4, 128)])
def test_backward_needs_no_more_workspace_than_it_says(T, shape):
    x, rot, cu, _ = make([T], *shape, 64)
    g = grads(x, cu)
    need = sa.sinkattn_rope_qkv_backward_workspace_bytes(T, shape[2])
    mine, untouched = in_a_field(need)
    got = backward(x, g, workspace=mine)
    assert untouched()
    check_backward(got, g, x, rot, cu)
    for a, b in zip(got, backward(x, g)):
        assert torch.equal(a, b)
    with pytest.raises(sa.SinkAttnError) as e:
        backward(x, g, workspace=mine[:-1])
    assert e.value.status == INVALID_ARG and "too small" in str(e.value)


@gpu
@pytest.mark.parametrize("norms", [(True, True), (False, False)])
def test_rows_past_32_bit_offsets(norms):
    """Every array of the packed form and of its backward pass has more than 2^31 elements
    (540,000 tokens of 3 x 32 heads of 128: 40 GB)."""
    T, hq, d = 540000, 32, 128
    assert T * hq * d > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.empty((T, 3 * hq, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = [1 + 0.3 * torch.randn(d, generator=gen, device="cuda") if n else None for n in norms]
    rope = sa.Rope(d, base=150000.0)
    cu = [0, T - 130, T - 3, T]
    x = dict(q=rows[:, :hq], k=rows[:, hq:2 * hq], v=rows[:, 2 * hq:], q_weight=w[0], k_weight=w[1],
             rope=rope, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), positions=None)
    at = torch.cat([torch.arange(20), torch.arange(T - 150, T)]).cuda()
    pos = torch.cat([torch.arange(20), torch.arange(T - 150, T - 130), torch.arange(127),
                     torch.arange(3)]).cuda()
    rot = Rotation(rope.inv_freq, 1.0, False, pos)
    # ragged HND rows of those tokens' heads
    start = torch.tensor(cu, device="cuda")
    b = torch.searchsorted(start, at, right=True) - 1
    hnd = (hq * start[b] + at - start[b])[:, None] + torch.arange(hq, device="cuda")[None, :] * (
        start[b + 1] - start[b])[:, None]
    assert hnd.max() * d > 2 ** 31
    q, k, v = forward(x)
    close(q[at], *rotated(x["q"][at], w[0], EPS, rot), "q")
    close(k[hnd], *rotated(x["k"][at], w[1], EPS, rot), "k")
    assert torch.equal(v[hnd], x["v"][at])
    got = backward(x, (q, k, v))
    for name, dx, dy in (("q", got[0], q[at]), ("k", got[1], k[hnd])):
        val, size, _, _ = rotated_gradients(dy, x[name][at], x[name + "_weight"], EPS, rot)
        close(dx[at], val, size, "d" + name, of=2.0 ** -16)
    assert torch.equal(got[2][at], x["v"][at])


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_pools_past_32_bit_offsets(fp8):
    """The last pages of pools of more than 2^31 elements (bf16: 2 x 4.4 GB)."""
    hq, hkv, d, page, T = 8, 4, 128, 64, 70
    pages = 2 ** 31 // (hkv * page * d) + 70
    x, rot, _, _ = make([T], hq, hkv, d, 128, positions=list(range(T)))
    slots = (torch.arange(T) * page + torch.arange(T) % page + (pages - T) * page).int().cuda()
    pools = [torch.zeros((pages, hkv, page, d), dtype=torch.uint8 if fp8 else torch.bfloat16,
                         device="cuda") for _ in range(2)]
    args = (x["q"], x["k"], x["v"], x["positions"], slots, x["rope"])
    if fp8:
        scales = [torch.full((hkv,), 5 / 448, device="cuda") for _ in range(2)]
        sa.sinkattn_rope_append_paged_fp8(*args, *scales, *pools, x["q_weight"], x["k_weight"], EPS)
    else:
        sa.sinkattn_rope_append_paged(*args, *pools, x["q_weight"], x["k_weight"], EPS)
    # as into a small pool
    small = [torch.zeros((T, hkv, page, d), dtype=p.dtype, device="cuda") for p in pools]
    low = slots - (pages - T) * page
    args = (*args[:4], low, x["rope"])
    if fp8:
        sa.sinkattn_rope_append_paged_fp8(*args, *scales, *small, x["q_weight"], x["k_weight"], EPS)
    else:
        sa.sinkattn_rope_append_paged(*args, *small, x["q_weight"], x["k_weight"], EPS)
    for p, want in zip(pools, small):
        assert want.any() and torch.equal(p[-T:], want)
        assert not p[:-T].any()


@gpu
@pytest.mark.parametrize("bad", [[0, 40, 90], [0, 40, 90, 40], [-5, 30, 40], [50, 60, 70], [0, 30, 10, 40],
                                 [0, -3], [-9, -3], [0] * 3000 + [41], [-1] + [0] * 3000 + [40]])
def test_bad_lengths_that_no_token_meets_are_recorded(bad):
    """Entries outside [0, 40], and ones that decrease, wherever they stand."""
    x, rot, cu, T = make([30, 10], 8, 2, 64, 64)
    g = grads(x, cu)
    x["cu"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for step in (lambda: forward(x), lambda: backward(x, g),
                 lambda: backward(dict(x, q_weight=None, k_weight=None), g)):
        step()
        assert sa.sinkattn_debug_status() == BAD_LENGTHS
        assert sa.sinkattn_debug_status() == 0


@gpu
@pytest.mark.parametrize("good", [[0, 40], [0, 0, 17, 17, 40, 40], [3, 20], [0, 0], [40, 40], [0] * 3000 + [40]])
def test_lengths_in_order_are_not_recorded(good):
    x, rot, cu, T = make([30, 10], 8, 2, 64, 64)
    g = grads(x, cu)
    x["cu"] = torch.tensor(good, dtype=torch.int32, device="cuda")
    forward(x), backward(x, g), backward(dict(x, q_weight=None, k_weight=None), g)
    assert sa.sinkattn_debug_status() == 0


# ----------------------------------------------------------------------------
# refusals: nothing launches
# ----------------------------------------------------------------------------
A = 0x1000   # fake, aligned, never dereferenced
ROPE = dict(turns=A, r=64, inter=0, factor=1.0, qw=A, kw=A, eps=1e-6)


def raw_forward(**kw):
    a = dict(q=A, k=A, v=A, qs=256, ks=64, vs=64, cu=A, pos=None, batch=1, tokens=9, hq=4, hkv=1,
             d=64, **ROPE, qo=A, ko=A, vo=A)
    a.update(kw)
    return sa.lib().sinkattn_rope_qkv(*a.values(), None)


def raw_backward(**kw):
    a = dict(dq=A, dk=A, dv=A, q=A, k=A, qs=256, ks=64, cu=A, pos=None, batch=1, tokens=9, hq=4,
             hkv=1, d=64, **ROPE, qo=A, ko=A, vo=A, dqs=256, dks=64, dvs=64, dqw=A, dkw=A, ws=0x10000,
             n=1 << 20)
    a.update(kw)
    return sa.lib().sinkattn_rope_qkv_backward(*a.values(), None)


def raw_append(fp8, **kw):
    a = dict(q=A, k=A, v=A, qs=256, ks=64, vs=64, pos=A, slots=A, tokens=9, hq=4, hkv=1, d=64, **ROPE)
    if fp8:
        a.update(k_scale=A, v_scale=A)
    a.update(qo=A, kp=A, vp=A, pages=4, page=16)
    a.update(kw)
    L = sa.lib()
    return (L.sinkattn_rope_append_paged_fp8 if fp8 else L.sinkattn_rope_append_paged)(
        *a.values(), None)


COMMON = [
    (dict(tokens=-1), INVALID_ARG), (dict(hq=0), INVALID_ARG), (dict(hkv=0), INVALID_ARG),
    (dict(d=96), UNSUPPORTED), (dict(r=65), INVALID_ARG), (dict(r=66), INVALID_ARG),
    (dict(r=-2), INVALID_ARG), (dict(turns=None), INVALID_ARG), (dict(turns=A + 4), INVALID_ARG),
    (dict(inter=2), INVALID_ARG), (dict(factor=float("nan")), INVALID_ARG),
    (dict(eps=-1.0), INVALID_ARG), (dict(eps=float("inf")), INVALID_ARG), (dict(qw=A + 2), INVALID_ARG),
    (dict(q=None), INVALID_ARG), (dict(k=A + 8), INVALID_ARG), (dict(qs=200), INVALID_ARG),
    (dict(ks=68), INVALID_ARG), (dict(qo=None), INVALID_ARG), (dict(hq=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(v=None), INVALID_ARG), (dict(vs=8), INVALID_ARG), (dict(cu=None), INVALID_ARG),
    (dict(batch=-1), INVALID_ARG), (dict(pos=A + 1), INVALID_ARG), (dict(ko=A + 8), INVALID_ARG),
    (dict(vo=None), INVALID_ARG)])
def test_forward_refusals(kw, status):
    assert raw_forward(**kw) == status and sa.sinkattn_last_error() != ""


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dq=None), INVALID_ARG), (dict(dk=A + 4), INVALID_ARG), (dict(dv=None), INVALID_ARG),
    (dict(cu=None), INVALID_ARG), (dict(batch=-1), INVALID_ARG), (dict(ko=None), INVALID_ARG),
    (dict(dqs=8), INVALID_ARG), (dict(dvs=68), INVALID_ARG), (dict(dqw=None), INVALID_ARG),
    (dict(dkw=A + 2), INVALID_ARG), (dict(ws=None), INVALID_ARG), (dict(ws=A + 16), INVALID_ARG),
    (dict(n=16), INVALID_ARG)])
def test_backward_refusals(kw, status):
    assert raw_backward(**kw) == status and sa.sinkattn_last_error() != ""


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(v=None), INVALID_ARG), (dict(pos=None), INVALID_ARG), (dict(slots=None), INVALID_ARG),
    (dict(slots=A + 2), INVALID_ARG), (dict(kp=None), INVALID_ARG), (dict(vp=A + 8), INVALID_ARG),
    (dict(pages=0), INVALID_ARG), (dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
    (dict(page=512), UNSUPPORTED), (dict(pages=1 << 27), UNSUPPORTED)])
def test_append_refusals(kw, status, fp8):
    assert raw_append(fp8, **kw) == status and sa.sinkattn_last_error() != ""


def test_append_fp8_needs_scales():
    assert raw_append(True, k_scale=None) == INVALID_ARG
    assert raw_append(True, v_scale=A + 2) == INVALID_ARG


def test_empty_calls_are_no_ops():
    assert raw_forward(tokens=0, q=None) == 0 and raw_forward(batch=0) == 0
    assert raw_append(False, tokens=0, q=None) == 0 and raw_append(True, tokens=0) == 0
    assert raw_backward(tokens=0, qw=None, kw=None, dqw=None, dkw=None) == 0


def test_workspace_bytes():
    assert sa.sinkattn_rope_qkv_backward_workspace_bytes(5000, 64) >= 2 * 64 * 4
    with pytest.raises(sa.SinkAttnError):
        sa.sinkattn_rope_qkv_backward_workspace_bytes(5, 96)


@gpu
def test_wrapper_refusals():
    x, rot, cu, T = make([20], 8, 2, 64, 64)
    for bad in (dict(q=x["q"].float()), dict(k=x["k"][:-1]), dict(v=x["v"].cpu()),
                dict(q=x["q"].transpose(1, 2).contiguous().transpose(1, 2)),
                dict(q_weight=x["q_weight"][:10]), dict(k_weight=x["k_weight"].half()),
                dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(rope=None), dict(rope=sa.Rope(128)), dict(cu=x["cu"].long())):
        with pytest.raises(sa.SinkAttnError) as e:
            forward(dict(x, **bad))
        assert e.value.status == INVALID_ARG
    with pytest.raises(sa.SinkAttnError):
        sa.Rope(64, inv_freq=[1.0])
    with pytest.raises(sa.SinkAttnError):
        sa.Rope(64, attention_factor=float("nan"))
