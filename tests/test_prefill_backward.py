"""The prefill's backward pass against the 64-bit formula (tests/_gradient_model.py,
which derives the tolerances), against differences, and its refusals."""
import numpy as np
import pytest
import torch

import gqa_attention_softmax_gb300 as sa
from gqa_attention_softmax_gb300 import _build
from gqa_attention_softmax_gb300._binding import (BAD_LENGTHS, INVALID_ARG, TIMEOUT,
                                                  UNSUPPORTED)
from _gradient_model import attention, attention_gradients

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    yield
    if torch.cuda.is_available():
        assert sa.sinkattn_debug_status() == 0


def make(q_lens, k_lens, hq, hkv, d, sinks=True, seed=0, causal=True, window=0, dev="cuda", q_scale=1.0):
    """Inputs of a backward call on `dev`, out and lse from the 64-bit forward."""
    gen = torch.Generator().manual_seed(seed)
    cu_q, cu_k = [np.cumsum([0] + list(x)).tolist() for x in (q_lens, k_lens)]
    r = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).to(dev)   # noqa: E731
    x = dict(q=(r(cu_q[-1], hq, d) * q_scale).to(torch.bfloat16), k=r(hkv * cu_k[-1], d),
             v=r(hkv * cu_k[-1], d), dout=r(cu_q[-1], hq, d),
             sinks=(torch.rand(hq, generator=gen) * 4 - 2).to(dev) if sinks else None)
    h = dict(cu_q=cu_q, cu_k=cu_k, hkv=hkv, scale=d ** -0.5, causal=causal, window=window)
    out, lse = attention(x["q"].double(), x["k"].double(), x["v"].double(),
                         None if x["sinks"] is None else x["sinks"].double(), **h)
    x["out"], x["lse"] = out.to(torch.bfloat16), lse.float().contiguous()
    return x, h


def call(x, h, **kw):
    dev = x["q"].device
    cu = [torch.tensor(h[n], dtype=torch.int32, device=dev) for n in ("cu_q", "cu_k")]
    longest = [max([b - a for a, b in zip(h[n][:-1], h[n][1:])], default=0) for n in ("cu_q", "cu_k")]
    return sa.sinkattn_prefill_backward(
        x["dout"], x["q"], x["k"], x["v"], x["out"], x["lse"], x["sinks"], *cu, *longest, h["hkv"],
        sm_scale=h["scale"], causal=h["causal"], window=h["window"], **kw)


def check(got, x, h, dlse=None):
    want = attention_gradients(x["dout"], x["q"], x["k"], x["v"], x["out"], x["lse"], x["sinks"],
                               dlse=dlse, **h)
    for name, t in zip(("dq", "dk", "dv", "dsinks"), got):
        if name not in want:
            assert t is None
            continue
        val, tol = want[name]
        assert torch.isfinite(t).all(), name
        err = (t.double() - val).abs()
        assert (err <= tol).all(), "%s: %g of the tolerance at %d of %d" % (
            name, (err / tol).max().item(), int((err > tol).sum()), err.numel())


SHAPES = [(64, 8, 64), (16, 1, 64), (24, 8, 64), (64, 4, 128), (4, 4, 128), (32, 8, 128), (5, 1, 64),
          (3, 1, 128)]


@gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens", [([1], [1]), ([16], [128]), ([130, 0, 1, 257], [130, 9, 300, 257]),
                                  ([127, 128, 129], [127, 128, 500])])
def test_causal(shape, lens):
    x, h = make(*lens, *shape)
    check(call(x, h), x, h)


@gpu
@pytest.mark.parametrize("shape", [(64, 8, 64), (24, 8, 64), (32, 8, 128), (128, 1, 64), (70, 1, 128)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 17), (True, 128), (True, 1000)])
@pytest.mark.parametrize("sinks", [False, True])
def test_masks(shape, causal, window, sinks):
    x, h = make([200, 3, 65], [200, 410, 65], *shape, sinks=sinks, causal=causal, window=window)
    check(call(x, h), x, h)


@gpu
@pytest.mark.parametrize("shape", [(64, 8, 64), (64, 4, 128), (2, 1, 128)])
def test_long(shape):
    x, h = make([1100, 700], [1100, 1500], *shape, sinks=False)
    check(call(x, h), x, h)


@gpu
def test_forward_and_backward_together():
    """out and lse as sinkattn_prefill leaves them."""
    for hq, hkv, d, window in ((64, 8, 64, 0), (64, 8, 64, 128), (64, 4, 128, 0)):
        x, h = make([300, 77], [300, 333], hq, hkv, d, window=window)
        cu = [torch.tensor(h[n], dtype=torch.int32, device="cuda") for n in ("cu_q", "cu_k")]
        x["out"], x["lse"] = sa.sinkattn_prefill(x["q"], x["k"], x["v"], x["sinks"], *cu, 300, 333,
                                                 hkv, window=window)
        check(call(x, h), x, h)


@gpu
def test_gradient_of_lse():
    x, h = make([70, 129], [90, 129], 24, 8, 64)
    dlse = torch.randn(x["lse"].shape, generator=torch.Generator().manual_seed(3)).cuda()
    check(call(x, h, dlse=dlse), x, h, dlse)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_peaked_weights(d):
    """Logits of tens: weights of nearly one and of nearly nothing. (The logit's
    32-bit error then moves a weight by less than d 2^-24 2^7 = 2^-10.)"""
    x, h = make([257], [257], 8, 2, d, q_scale=4.0)
    check(call(x, h), x, h)


@gpu
@pytest.mark.parametrize("shape", [(8, 2, 64), (8, 2, 128)])
def test_maxima_far_above_the_lengths(shape):
    """max_seqlen_* only bound the lengths: the largest int32 gives what the exact ones give."""
    for window in (0, 40):
        x, h = make([33, 200], [50, 200], *shape, window=window)
        cu = [torch.tensor(h[n], dtype=torch.int32, device="cuda") for n in ("cu_q", "cu_k")]
        got = sa.sinkattn_prefill_backward(
            x["dout"], x["q"], x["k"], x["v"], x["out"], x["lse"], x["sinks"], *cu, 2 ** 31 - 1,
            2 ** 31 - 1, h["hkv"], window=window)
        for a, b in zip(got, call(x, h)):
            assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("shape", [(16, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("window", [1, 20, 200])
def test_many_tokens_in_short_windows(shape, window):
    """Several query tiles a CTA: as many tokens as give each SM a few of them, of sequences
    of every length."""
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 400, (64,), generator=gen).tolist() + [0, 1, 3000]
    x, h = make(lens, lens, *shape, window=window)
    check(call(x, h), x, h)


@gpu
@pytest.mark.parametrize("shape", [(16, 2, 64), (16, 2, 128)])
def test_many_keys_that_no_query_sees(shape):
    """A short window at the end of long sequences: key tiles without work before, between
    and behind those with some, several of them a CTA."""
    gen = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 400, (64,), generator=gen).tolist() + [0, 1, 700]
    more = torch.randint(0, 900, (67,), generator=gen).tolist()
    x, h = make(lens, [a + b for a, b in zip(lens, more)], *shape, window=30)
    check(call(x, h), x, h)


@gpu
@pytest.mark.parametrize("shape", [(64, 8, 64), (16, 2, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_tokens(shape, causal):
    """Several query tiles a CTA without a window, and keys behind sequences of fewer queries."""
    gen = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 300, (50,), generator=gen).tolist() + [0, 1, 1000]
    more = torch.randint(0, 100, (53,), generator=gen).tolist()
    x, h = make(lens, [a + b for a, b in zip(lens, more)], *shape, causal=causal)
    check(call(x, h), x, h)


@gpu
@pytest.mark.parametrize("shape", [(8, 2, 64), (8, 2, 128)])
def test_sinks_of_minus_infinity(shape):
    """Heads whose sink is -inf have none: dsinks 0. A row with lse -inf has no
    weights: no gradient of its own and none for others, as if its dout were 0."""
    x, h = make([50, 70], [50, 90], *shape)
    x["sinks"][::3] = -torch.inf
    out, lse = attention(x["q"].double(), x["k"].double(), x["v"].double(), x["sinks"].double(), **h)
    x["out"], x["lse"] = out.to(torch.bfloat16), lse.float().contiguous()
    got = call(x, h)
    assert (got[3][::3] == 0).all()
    for a, b in zip(got[:3], call(dict(x, sinks=None), h)):
        assert torch.equal(a, b)
    check(got, x, h)
    for token, head in ((0, 0), (49, 2), (110, 7), (110, 3)):
        x["dout"][token, head] = 0
    want = call(x, h)
    assert (want[0][110, 3] == 0).all()
    for token, head in ((0, 0), (49, 2), (110, 7), (110, 3)):
        x["dout"][token, head] = 1
        x["lse"][token, head] = -torch.inf
    for a, b in zip(call(x, h), want):
        assert torch.equal(a, b)


def _differences(x, h, name, direction, step):
    """d/dt of sum(dout * out) at x[name] + t direction, by central differences in 64 bits."""
    vals = []
    for t in (step, -step):
        y = {n: (None if x[n] is None else x[n].double()) for n in ("q", "k", "v", "sinks")}
        y[name] = y[name] + t * direction
        out, _ = attention(y["q"], y["k"], y["v"], y["sinks"], **h)
        vals.append((out * x["dout"].double()).sum().item())
    return (vals[0] - vals[1]) / (2 * step)


def test_model_agrees_with_differences():
    """The formula itself (CPU): exact out and lse, so only the step's error is left,
    O(step^2) of third derivatives, below 1e-6 of the sum of the terms here."""
    x, h = make([5, 3], [9, 3], 4, 2, 64, dev="cpu", window=4)
    out, lse = attention(x["q"].double(), x["k"].double(), x["v"].double(), x["sinks"].double(), **h)
    got = attention_gradients(x["dout"], x["q"], x["k"], x["v"], out, lse, x["sinks"], **h)
    gen = torch.Generator().manual_seed(1)
    for name in ("q", "k", "v", "sinks"):
        way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        grad = got["d" + name][0]
        want = _differences(x, h, name, way, 1e-4)
        assert abs((grad * way).sum().item() - want) <= 1e-6 * (grad * way).abs().sum().item()


@gpu
@pytest.mark.parametrize("shape", [(8, 2, 64), (8, 1, 128)])
def test_differences(shape):
    """The kernel's gradients along random directions. Each element is off by its
    tolerance at most, and by what the rounding of out (2^-8 of it) does
    through delta: 2^-8 sum |dout out| instead of the 2^-16 that the formula's inputs leave."""
    x, h = make([40, 7], [40, 20], *shape)
    got = dict(zip(("dq", "dk", "dv", "dsinks"), call(x, h)))
    wide = attention_gradients(x["dout"], x["q"], x["k"], x["v"], x["out"], x["lse"], x["sinks"], **h)
    out, lse = attention(*[x[n].double() for n in ("q", "k", "v", "sinks")], **h)
    exact = attention_gradients(x["dout"], x["q"], x["k"], x["v"], out, lse, x["sinks"], **h)
    gen = torch.Generator().manual_seed(1)
    for name in ("q", "k", "v", "sinks"):
        g = got["d" + name].double()
        way = torch.randn(g.shape, generator=gen, dtype=torch.float64).to(g.device)
        slack = (wide["d" + name][1] + (wide["d" + name][0] - exact["d" + name][0]).abs()) * way.abs()
        diff = _differences(x, h, name, way, 1e-4)
        assert abs((g * way).sum().item() - diff) <= slack.sum().item() + 1e-6 * abs(diff)


@gpu
def test_no_visible_keys_and_no_queries():
    # (a sequence without queries: its keys get zeros; keys before every window too)
    x, h = make([0, 4], [33, 200], 8, 2, 64, window=8)
    got = call(x, h)
    check(got, x, h)
    assert (got[1][:2 * 33] == 0).all() and (got[2][:2 * 33] == 0).all()
    x, h = make([0, 0], [33, 0], 8, 2, 64)
    got = call(x, h, dk=torch.full((66, 64), 7.0, dtype=torch.bfloat16, device="cuda"))
    assert (got[1] == 0).all() and (got[2] == 0).all() and (got[3] == 0).all()
    for empty in ([], [0]):
        x, h = make(empty + [0], empty + [0], 8, 2, 64)
        h = dict(h, cu_q=[0] * (len(empty) + 1), cu_k=[0] * (len(empty) + 1))
        got = call(x, h)
        assert (got[3] == 0).all()


@gpu
@pytest.mark.parametrize("shape", [(64, 8, 64), (24, 8, 64), (64, 4, 128)])
def test_rows_behind_the_last_sequence_stay(shape):
    x, h = make([70, 60], [70, 100], *shape)
    hq, hkv, d = shape
    pad = {}
    for n, rows in (("q", 9), ("dout", 9), ("out", 9), ("lse", 9), ("k", 5 * hkv), ("v", 5 * hkv)):
        more = torch.full((rows,) + x[n].shape[1:], float("nan"), dtype=x[n].dtype, device="cuda")
        pad[n] = torch.cat([x[n], more])
    pad["sinks"] = x["sinks"]
    outs = {n: torch.full(pad[s].shape, 7.0, dtype=torch.bfloat16, device="cuda")
            for n, s in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    got = call(pad, h, **outs)
    for t, s in zip(got, ("q", "k", "v")):
        assert (t[x[s].shape[0]:] == 7.0).all()
    check([g[:x[s].shape[0]] for g, s in zip(got, ("q", "k", "v"))] + [got[3]], x, h)


@gpu
@pytest.mark.parametrize("shape", [(64, 8, 64), (64, 4, 128), (24, 8, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sequence_keeps_its_nan(shape, bad):
    """Another sequence's NaN or infinity, in any input, reaches no other gradient."""
    lens = ([100, 61, 140], [100, 90, 140])
    x, h = make(*lens, *shape)
    want = call(x, h)
    hkv = shape[1]
    y = {n: (t if t is None else t.clone()) for n, t in x.items()}
    for n in ("q", "dout", "out"):
        y[n][100:161] = bad
    for n in ("k", "v"):
        y[n][hkv * 100:hkv * 190] = bad
    got = call(y, h)
    for a, b, cu, heads in ((want[0], got[0], h["cu_q"], 1), (want[1], got[1], h["cu_k"], hkv),
                            (want[2], got[2], h["cu_k"], hkv)):
        assert torch.equal(a[:heads * cu[1]], b[:heads * cu[1]])
        assert torch.equal(a[heads * cu[2]:], b[heads * cu[2]:])


@gpu
def test_same_call_same_bits():
    x, h = make([500, 300], [500, 700], 64, 8, 64)
    first = [t.clone() for t in call(x, h)]
    for _ in range(3):
        for a, b in zip(first, call(x, h)):
            assert torch.equal(a, b)


@gpu
def test_streams_and_graphs():
    x, h = make([90, 300], [90, 310], 64, 8, 64)
    want = [t.clone() for t in call(x, h)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(x, h, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # two calls captured one after the other, each with its own workspace
    y, g = make([33], [64], 64, 8, 64, seed=5)
    want2 = [t.clone() for t in call(y, g)]
    cu = {}
    for n, hh in (("x", h), ("y", g)):
        cu[n] = [torch.tensor(hh[c], dtype=torch.int32, device="cuda") for c in ("cu_q", "cu_k")]
    outs = {}

    def both():
        for n, z, hh, most in (("x", x, h, (300, 310)), ("y", y, g, (33, 64))):
            outs[n] = sa.sinkattn_prefill_backward(
                z["dout"], z["q"], z["k"], z["v"], z["out"], z["lse"], z["sinks"], *cu[n], *most,
                hh["hkv"], sm_scale=hh["scale"])

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in outs["x"] + outs["y"]:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want + want2, outs["x"] + outs["y"]):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("shape", [(64, 8, 64), (3, 1, 128), (24, 8, 64)])
@pytest.mark.parametrize("tokens", [[1], [127], [128], [130, 3], [700, 1, 333]])
def test_needs_no_more_workspace_than_it_says(tokens, shape):
    """The queried bytes, between bytes of a pattern that stay as they are (blocks of
    128, 2730 and 341 tokens sum the sinks' gradients)."""
    x, h = make(tokens, tokens, *shape)
    need = sa.sinkattn_prefill_backward_workspace_bytes(sum(tokens), shape[0])
    whole = torch.full((need + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    at = 4096 - whole.data_ptr() % 256
    mine = whole[at:at + need]
    assert mine.data_ptr() % 256 == 0
    got = call(x, h, workspace=mine)
    assert (whole[:at] == 0x5a).all() and (whole[at + need:] == 0x5a).all()
    check(got, x, h)
    for a, b in zip(got, call(x, h)):
        assert torch.equal(a, b)
    with pytest.raises(sa.SinkAttnError) as e:
        call(x, h, workspace=mine[:-1])
    assert e.value.status == INVALID_ARG and "needs %d" % need in str(e.value)


@gpu
@pytest.mark.parametrize("shape", [(8, 2, 64), (8, 2, 128)])
def test_no_queries_need_no_workspace(shape):
    """(The query says 0 bytes, for which a caller may have no address.)"""
    x, h = make([0, 0], [33, 200], *shape)
    assert sa.sinkattn_prefill_backward_workspace_bytes(0, shape[0]) == 0
    outs = {n: torch.full_like(x[n[1:]], 7.0) for n in ("dk", "dv")}
    got = call(x, h, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"), **outs)
    assert all((t == 0).all() for t in got[1:])


@gpu
@pytest.mark.parametrize("shape", [(34, 34, 64), (64, 2, 128)])
def test_rows_past_32_bit_offsets(shape):
    """Sequences of 64 tokens, the last ones' rows past 2^31 elements of q, dout, out and dq, and of
    k, v, dk and dv too in the first shape (35 GB), against the 64-bit formula."""
    hq, hkv, d = shape
    n = 2 ** 31 // (64 * hq * d) + 12
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)   # noqa: E731
    T = 64 * n
    x = dict(q=r(T, hq, d), k=r(hkv * T, d), v=r(hkv * T, d), dout=r(T, hq, d),
             sinks=torch.rand(hq, generator=gen, device="cuda") * 4 - 2)
    h = dict(cu_q=list(range(0, T + 1, 64)), hkv=hkv, scale=d ** -0.5, causal=True, window=0)
    h["cu_k"] = h["cu_q"]
    assert x["q"].numel() > 2 ** 31 + 8 * 64 * hq * d
    cu = torch.tensor(h["cu_q"], dtype=torch.int32, device="cuda")
    x["out"], x["lse"] = sa.sinkattn_prefill(x["q"], x["k"], x["v"], x["sinks"], cu, cu, 64, 64, hkv)
    got = call(x, h)
    for a, b in ((0, 64), (T - 192, T)):
        part = {m: x[m][a:b] for m in ("q", "dout", "out", "lse")}
        part.update({m: x[m][hkv * a:hkv * b] for m in ("k", "v")}, sinks=None)
        cut = list(range(0, b - a + 1, 64))
        check((got[0][a:b], got[1][hkv * a:hkv * b], got[2][hkv * a:hkv * b], None), part,
              dict(h, cu_q=cut, cu_k=cut))
    weight = torch.exp(x["sinks"].double() - x["lse"].double())
    want = torch.zeros(hq, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for a in range(0, T, 1 << 16):
        terms = x["dout"][a:a + (1 << 16)].double() * x["out"][a:a + (1 << 16)].double()
        want -= (weight[a:a + (1 << 16)] * terms.sum(-1)).sum(0)
        size += (weight[a:a + (1 << 16)] * terms.abs().sum(-1)).sum(0)
    # terms as in tests/_gradient_model.py; up to 240 rows a block and 4,116 blocks, each in 20
    # slices: chains of at most 12 + 20 + 206 + 20 additions, 2^-15 of the terms
    assert ((got[3].double() - want).abs() <= (2.0 ** -12 + 2.0 ** -15) * size).all()


@gpu
def test_lengths_that_contradict_the_sizes_are_recorded():
    x, h = make([50, 60], [50, 60], 8, 2, 64)
    cu = torch.tensor(h["cu_q"], dtype=torch.int32, device="cuda")
    args = [x[n] for n in ("dout", "q", "k", "v", "out", "lse", "sinks")]
    want = call(x, h)
    # the second sequence is longer than the stated maximum: the first keeps its gradients
    got = sa.sinkattn_prefill_backward(*args, cu, cu, 55, 55, 2)
    assert sa.sinkattn_debug_status() == BAD_LENGTHS
    assert torch.equal(got[0][:50], want[0][:50]) and torch.equal(got[1][:100], want[1][:100])
    # sequences that reach past the tensors
    far = torch.tensor([0, 50, 900], dtype=torch.int32, device="cuda")
    sa.sinkattn_prefill_backward(*args, far, far, 1000, 1000, 2)
    assert sa.sinkattn_debug_status() == BAD_LENGTHS
    back = torch.tensor([0, 50, 10], dtype=torch.int32, device="cuda")
    sa.sinkattn_prefill_backward(*args, back, back, 60, 60, 2)
    assert sa.sinkattn_debug_status() == BAD_LENGTHS
    assert sa.sinkattn_debug_status() == 0


@gpu
@pytest.mark.parametrize("shape", [(8, 2, 64), (8, 2, 128)])
def test_maxima_of_zero(shape):
    """Sequences that have keys, or queries, although the bound says that there are none, are
    recorded; without queries dsinks is zero whatever the workspace holds."""
    x, h = make([50, 60], [50, 60], *shape)
    cu = torch.tensor(h["cu_q"], dtype=torch.int32, device="cuda")
    none = torch.zeros_like(cu)
    args = [x[n] for n in ("dout", "q", "k", "v", "out", "lse", "sinks")]
    for most in ((0, 0), (0, 60)):
        ws = torch.full((1 << 20,), 0x40, dtype=torch.uint8, device="cuda")
        got = sa.sinkattn_prefill_backward(*args, cu, cu, *most, 2, workspace=ws)
        assert sa.sinkattn_debug_status() == BAD_LENGTHS
        assert (got[3] == 0).all()
    # nothing but rows behind the last sequence
    outs = {n: torch.full_like(x[n[1:]], 7.0) for n in ("dq", "dk", "dv")}
    got = sa.sinkattn_prefill_backward(*args, none, none, 0, 0, 2, **outs)
    assert sa.sinkattn_debug_status() == 0
    assert all((t == 7.0).all() for t in got[:3]) and (got[3] == 0).all()


@gpu
@pytest.mark.parametrize("shape", [(8, 1, 64), (8, 1, 128)])
@pytest.mark.parametrize("tile", [0, 3])
@pytest.mark.parametrize("sinks", [False, True])
def test_a_wait_that_runs_out_is_recorded(shape, tile, sinks):
    """A test hook shortens the waits to about 10 ms and leaves one tile's copies out."""
    x, h = make([700], [700], *shape, sinks=sinks)
    want = [t.clone() for t in call(x, h) if t is not None]
    assert sa.sinkattn_debug_status() == 0
    sa.sinkattn_debug_set_hooks(20_000_000, tile)
    try:
        call(x, h)
        assert sa.sinkattn_debug_status() == TIMEOUT
    finally:
        sa.sinkattn_debug_set_hooks(0, -1)
    for a, b in zip(want, call(x, h)):
        assert torch.equal(a, b)
    assert sa.sinkattn_debug_status() == 0


@gpu
@pytest.mark.parametrize("shape", [(16, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("tile", [0, 5, 12])
def test_a_wait_that_runs_out_among_several_tiles(shape, tile):
    """As above, in CTAs that go through several tiles: the first CTA of dq has 7 query
    tiles of one tile of keys each at d 64 and 14 at d 128, that of dk and dv key tiles of
    159 and 128 queries, 10 and 8 tiles at d 64, 20 and 16 at d 128."""
    x, h = make([256] * 64, [256] * 64, *shape, window=32)
    want = [t.clone() for t in call(x, h)]
    assert sa.sinkattn_debug_status() == 0
    sa.sinkattn_debug_set_hooks(20_000_000, tile)
    try:
        call(x, h)
        assert sa.sinkattn_debug_status() == TIMEOUT
    finally:
        sa.sinkattn_debug_set_hooks(0, -1)
    for a, b in zip(want, call(x, h)):
        assert torch.equal(a, b)
    assert sa.sinkattn_debug_status() == 0


@gpu
@pytest.mark.parametrize("d,limit", [(64, 100_000), (128, 160_000)])
def test_no_wait_runs_out_while_the_first_pass_runs(d, limit):
    """150 query tiles, one an SM: as the short ones end, CTAs of dk and dv come and have to
    wait for the longest, 300 tiles of keys (100 us and more). The limit, half of that, is
    that of a wait within a pass, whose tiles take about 1 us each."""
    T = 19200
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)   # noqa: E731
    x = dict(q=r(T, 1, d), k=r(T, d), v=r(T, d), dout=r(T, 1, d), sinks=torch.zeros(1, device="cuda"))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    x["out"], x["lse"] = sa.sinkattn_prefill(x["q"], x["k"], x["v"], x["sinks"], cu, cu, T, T, 1)
    h = dict(cu_q=[0, T], cu_k=[0, T], hkv=1, scale=d ** -0.5, causal=True, window=0)
    want = call(x, h)
    assert sa.sinkattn_debug_status() == 0
    sa.sinkattn_debug_set_hooks(limit, -1)
    try:
        got = call(x, h)
        assert sa.sinkattn_debug_status() == 0
    finally:
        sa.sinkattn_debug_set_hooks(0, -1)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------
# refusals: nothing launches
# ----------------------------------------------------------------------------
A = 0x1000   # fake, aligned, never dereferenced


def raw(**kw):
    a = dict(dout=A, q=A, k=A, v=A, out=A, lse=A, sinks=A, dlse=None, cu_q=A, cu_k=A, batch=1,
             total_q=16, total_k=128, max_q=16, max_k=128, hq=4, hkv=1, d=64, scale=0.125, causal=1,
             window=0, dq=A, dk=A, dv=A, dsinks=A, ws=0x10000, n=1 << 20)
    a.update(kw)
    return sa.lib().sinkattn_prefill_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID_ARG), (dict(k=None), INVALID_ARG), (dict(dout=None), INVALID_ARG),
    (dict(out=None), INVALID_ARG), (dict(lse=None), INVALID_ARG), (dict(dq=None), INVALID_ARG),
    (dict(dk=None), INVALID_ARG), (dict(dv=None), INVALID_ARG), (dict(cu_q=None), INVALID_ARG),
    (dict(cu_k=None), INVALID_ARG), (dict(dout=A + 8), INVALID_ARG), (dict(dv=A + 8), INVALID_ARG),
    (dict(lse=A + 2), INVALID_ARG), (dict(dlse=A + 2), INVALID_ARG), (dict(ws=None), INVALID_ARG),
    (dict(ws=0x10010), INVALID_ARG), (dict(n=64), INVALID_ARG), (dict(dsinks=None), INVALID_ARG),
    (dict(sinks=None), INVALID_ARG), (dict(d=96), UNSUPPORTED), (dict(hq=5, hkv=2), UNSUPPORTED),
    (dict(hq=129), UNSUPPORTED), (dict(scale=0.0), INVALID_ARG), (dict(scale=float("nan")), INVALID_ARG),
    (dict(causal=2), INVALID_ARG), (dict(causal=0, window=4), UNSUPPORTED),
    (dict(batch=-1), INVALID_ARG), (dict(total_q=-1), INVALID_ARG), (dict(total_k=-1), INVALID_ARG),
    (dict(max_q=200), INVALID_ARG), (dict(batch=70000), UNSUPPORTED),
    (dict(total_k=1 << 30, hkv=2), UNSUPPORTED), (dict(total_q=1 << 30), UNSUPPORTED),
])
def test_refusals(kw, status):
    assert raw(**kw) == status
    assert sa.sinkattn_last_error() != ""


@pytest.mark.parametrize("name", ["cu_q", "cu_k"])
def test_misaligned_lengths_are_refused(name):
    """(A kernel would read a word across its boundary.)"""
    assert raw(**{name: A + 2}) == INVALID_ARG and "aligned" in sa.sinkattn_last_error()


def test_no_queries_need_no_workspace_address():
    """The call gets past it, as far as the work items, of which these sizes have too many."""
    assert raw(total_q=0, max_q=0, ws=None, n=0, batch=65535, hkv=4, hq=4, total_k=1 << 24,
               max_k=1 << 24) == UNSUPPORTED


def test_workspace_bytes():
    n = sa.sinkattn_prefill_backward_workspace_bytes(100, 64)
    assert n >= 100 * 64 * 4 and n % 4 == 0
    assert sa.sinkattn_prefill_backward_workspace_bytes(0, 64) == 0
    with pytest.raises(sa.SinkAttnError):
        sa.sinkattn_prefill_backward_workspace_bytes(-1, 64)


@gpu
def test_wrapper_refusals():
    x, h = make([20], [30], 8, 2, 64)
    for bad in (dict(dout=x["dout"].float()), dict(out=x["out"][:, :4]), dict(lse=x["lse"].half()),
                dict(k=x["k"][:-1]), dict(v=x["v"][:-2]), dict(q=x["q"].cpu()),
                dict(sinks=x["sinks"][:4]), dict(dout=x["dout"].transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(sa.SinkAttnError) as e:
            call(dict(x, **bad), h)
        assert e.value.status == INVALID_ARG
    with pytest.raises(sa.SinkAttnError):
        call(x, h, dq=torch.empty_like(x["q"])[:10])
    with pytest.raises(sa.SinkAttnError):
        call(x, h, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
