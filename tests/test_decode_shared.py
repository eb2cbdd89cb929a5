"""Shared-prefix decode over a paged cache, against the float64 oracle.

The oracle attends each sequence's whole key range, contiguous; the CUDA path
reads pages in random order in which the sequences of a group share their
first pages, with unused slots and spare pages full of large finite values.

Tolerances, per element. Every bf16 weight p_j is off by at most half a step
(2^-8 of it), so sum p_j v_j / D by at most 2^-8 A with A = sum p_j |v_j| / D
(the oracle's output for |v|), and the output's own rounding adds 2^-8 |out|.
e4m3 caches use f16 weights (2^-11, and 2^-25 below f16's normal range). fp32
sums of up to d products add, to each logit, at most d 2^-24 sum |q k| scale:
below 6e-5 for unit normals at d 128; weights move by that much relatively.
That bounds the log-sum-exp too (1e-4, with the exponential's 2^-21), times
the scale that a case multiplies q with.
"""
import math
import random

import numpy as np
import pytest
import torch

import oracle
import gqa_attention_softmax_gb300 as sa
from gqa_attention_softmax_gb300._binding import (BAD_LENGTHS, INVALID_ARG, TIMEOUT,
                                                  UNSUPPORTED)
from _helpers import compare

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_softmax_gb300 import _build
    _build.build()
    oracle.build()
    yield
    if torch.cuda.is_available():
        assert sa.sinkattn_debug_status() == 0


def make(groups, q_len, Hq, Hkv, d, page, seed=0, q_scale=1.0, fp8=False):
    """groups: [(prefix pages, [own keys of each sequence])]. CPU tensors: the
    paged inputs, and the contiguous k, v the oracle reads."""
    rng = random.Random(seed)
    gen = torch.Generator().manual_seed(seed)
    own = [n for _, lens in groups for n in lens]
    lens = [pre * page + n for pre, ls in groups for n in ls]
    B = len(own)
    need = sum(pre for pre, _ in groups) + sum(-(-n // page) for n in own)
    total = need + 3
    ids = list(range(total))
    rng.shuffle(ids)
    shape = (total, Hkv, page, d)
    if fp8:
        # finite codes in every slot; the unused ones hold the largest values
        pools = [torch.full(shape, 0x7e, dtype=torch.uint8) for _ in range(2)]
    else:
        pools = [(torch.randn(shape, generator=gen) * 100).to(torch.bfloat16) for _ in range(2)]

    def draw(n):
        x = torch.randn((Hkv, n, d), generator=gen)
        if not fp8:
            return x.to(torch.bfloat16)
        return (x * 90.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def place(pool, x, pages):
        for e, p in enumerate(pages):
            part = x[:, e * page:(e + 1) * page]
            pool[p, :, :part.shape[1]] = part

    lists, flat, at = [], [[], []], 0
    for pre, ls in groups:
        shared = ids[at:at + pre]
        at += pre
        common = [draw(pre * page) for _ in range(2)]
        for x, pool in zip(common, pools):
            place(pool, x, shared)
        for n in ls:
            mine = ids[at:at + -(-n // page)]
            at += len(mine)
            for i in range(2):
                x = draw(n)
                place(pools[i], x, mine)
                flat[i].append(torch.cat([common[i], x], dim=1).reshape(-1, d))
            lists.append(shared + mine)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32)   # noqa: E731
    q = (torch.randn((B * q_len, Hq, d), generator=gen) * q_scale).to(torch.bfloat16)
    out = dict(q=q, k_pages=pools[0], v_pages=pools[1],
               kv_indptr=i32(np.cumsum([0] + lens)),
               page_indptr=i32(np.cumsum([0] + [len(x) for x in lists])),
               page_indices=i32([p for x in lists for p in x]),
               group_indptr=i32(np.cumsum([0] + [len(ls) for _, ls in groups])),
               prefix_lens=i32([pre * page for pre, _ in groups]),
               sinks=torch.rand(Hq, generator=gen) * 4 - 2,
               cu_q=i32([b * q_len for b in range(B + 1)]),
               k=torch.cat(flat[0]) if B else torch.zeros((0, d), dtype=pools[0].dtype),
               v=torch.cat(flat[1]) if B else torch.zeros((0, d), dtype=pools[0].dtype))
    if fp8:
        out["k_scale"] = (0.8 + 0.4 * torch.rand(Hkv, generator=gen)) / 90.0
        out["v_scale"] = (0.8 + 0.4 * torch.rand(Hkv, generator=gen)) / 90.0
    host = dict(q_len=q_len, max_prefix=max((p for p, _ in groups), default=0) * page,
                max_suffix=max(own, default=q_len), Hq=Hq, Hkv=Hkv, d=d, q_scale=q_scale, fp8=fp8,
                keys=max(lens, default=1))
    return out, host


def call(x, h, sinks=True, **kw):
    s = x["sinks"] if sinks else None
    kw.setdefault("prefix_splits", 4)   # (by default calls this small do not share)
    if h["fp8"]:
        return sa.sinkattn_decode_shared_paged_fp8(
            x["q"], x["k_pages"], x["v_pages"], x["k_scale"], x["v_scale"], x["kv_indptr"],
            x["page_indptr"], x["page_indices"], x["group_indptr"], x["prefix_lens"], s,
            h["q_len"], h["max_prefix"], h["max_suffix"], **kw)
    return sa.sinkattn_decode_shared_paged(
        x["q"], x["k_pages"], x["v_pages"], x["kv_indptr"], x["page_indptr"], x["page_indices"],
        x["group_indptr"], x["prefix_lens"], s, h["q_len"], h["max_prefix"], h["max_suffix"], **kw)


def want(x, h, window=0, causal=True, sinks=True):
    """(out, lse, A) of the oracle; A: its output with |v| in the place of v."""
    s = x["sinks"] if sinks else None
    scales = {n: x[n] for n in ("k_scale", "v_scale") if n in x}
    got = []
    for absolute in (False, True):
        v = x["v"]
        if absolute:
            v = v & 0x7f if h["fp8"] else v.abs()
        got.append(oracle.attend(x["q"], x["k"], v, s, x["cu_q"], x["kv_indptr"], h["Hq"],
                                 h["Hkv"], h["d"], 1.0 / math.sqrt(h["d"]), causal, window,
                                 **scales))
    return got[0][0], got[0][1], got[1][0]


def check(out, lse, x, h, **kw):
    o, l, A = want(x, h, **kw)
    got = out.float().cpu().numpy().reshape(o.shape)
    assert np.isfinite(got).all()
    weight = 2.0 ** -11 if h["fp8"] else 2.0 ** -8
    low = 2.0 ** -25 * h["keys"] * 6.0 if h["fp8"] else 0.0
    logit = 1e-4 * h["q_scale"]
    err = np.abs(got - o)
    room = 2.0 ** -8 * np.abs(o) + (weight + 2 * logit) * A + low + 1e-6
    assert (err <= room).all(), "off by %.3g of the room" % (err / room).max()
    if lse is not None:
        g = lse.cpu().numpy().reshape(l.shape)
        both = np.isneginf(g) & np.isneginf(l)
        assert np.where(both, 0.0, np.abs(g - l)).max() <= logit


CASES = [
    # groups, q_len, Hq, Hkv, d, page, window, prefix_splits, num_splits, q_scale
    ([(4, [1, 40, 7])], 1, 64, 8, 64, 16, 0, 0, 0, 1.0),
    ([(1, [1])], 1, 8, 8, 64, 16, 0, 1, 1, 1.0),                       # smallest: one sequence, MHA
    ([(3, [3, 130, 64, 5])], 3, 64, 4, 128, 64, 0, 2, 3, 1.0),
    ([(2, [5, 9]), (0, [33, 1, 70]), (7, [1, 2, 3, 4])], 1, 64, 8, 64, 32, 0, 3, 2, 1.0),
    ([(0, [20, 30]), (0, [7])], 2, 32, 8, 128, 16, 0, 0, 0, 1.0),      # nothing is shared
    ([(2, [4, 4]), (5, []), (1, [9])], 4, 16, 1, 128, 128, 0, 2, 2, 1.0),   # a group without sequences
    ([(20, [1 + 5 * i for i in range(40)])], 1, 64, 8, 64, 16, 0, 4, 1, 1.0),   # 320 rows per head
    ([(5, [3 + i for i in range(30)])], 3, 64, 4, 128, 64, 0, 3, 1, 3.0),   # 1440 rows, peaky
    ([(9, [10, 300, 40])], 2, 24, 4, 64, 32, 100, 2, 2, 1.0),          # window: some see no prefix
    ([(9, [10, 500, 40]), (4, [4, 4])], 4, 64, 4, 128, 16, 150, 3, 2, 1.0),
    ([(2, [1, 1, 1, 1])], 1, 64, 1, 64, 256, 0, 9, 1, 1.0),            # 64 heads per KV head, empty chunks
    ([(1, [7] * 5), (3, [2] * 150)], 2, 8, 2, 64, 16, 0, 1, 1, 1.0),   # 1200 rows of one short prefix
    ([(33, [90, 91])], 1, 14, 2, 128, 16, 0, 5, 1, 1.0),               # 7 heads per KV head, odd tiles
    ([(11, [6, 20, 300, 31, 8])], 6, 40, 2, 128, 64, 0, 2, 4, 1.0),    # 20 heads x 6 drafts
]
IDS = ["b%d_g%d_q%d_h%d-%d_d%d_p%d_w%d_s%d-%d" % (sum(len(g[1]) for g in c[0]), len(c[0]), *c[1:6],
                                                 *c[6:9]) for c in CASES]


@gpu
@pytest.mark.parametrize("kernel", ["auto", "warp"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_shared_decode_matches_oracle(case, fp8, kernel):
    groups, q_len, Hq, Hkv, d, page, window, ps, ss, qs = case
    x, h = make(groups, q_len, Hq, Hkv, d, page, seed=page + q_len, q_scale=qs, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    sa.sinkattn_set_decode_kernel(kernel)
    try:
        out, lse = call(g, h, window=window, prefix_splits=ps, num_splits=ss)
    finally:
        sa.sinkattn_set_decode_kernel("auto")
    check(out, lse, x, h, window=window)


@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_row_blocks_and_tiles_of_every_page_size(fp8, d, page):
    """Groups that fill whole row blocks, one tile of a block, and a part of one; prefixes
    that end inside a K/V tile; more items than SMs."""
    G = 8 if d == 64 else 16
    per = 128 // G   # tokens of a tile
    n = max(1, 512 // page)
    groups = [(n, [1] * (2 * per)), (n + 1, [2] * (per - 1)), (2 * n, [1] * (4 * per + 3)),
              (1, [5] * per)]
    x, h = make(groups, 1, 2 * G, 2, d, page, seed=page, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    for ps in (1, 3, 40):
        out, lse = call(g, h, prefix_splits=ps, num_splits=1)
        check(out, lse, x, h)


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_a_wait_that_runs_out_is_recorded(fp8):
    """The first block's producer leaves one tile's copies out: its waits give up after about
    10 ms, the call ends with SINKATTN_TIMEOUT, and the next one is right."""
    x, h = make([(20, [5] * 40)], 1, 64, 8, 64, 16, seed=9, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    assert sa.sinkattn_debug_status() == 0
    sa.sinkattn_debug_set_hooks(20_000_000, 1)
    try:
        call(g, h, prefix_splits=1, num_splits=1)
        assert sa.sinkattn_debug_status() == TIMEOUT
    finally:
        sa.sinkattn_debug_set_hooks(0, -1)
    out, lse = call(g, h)
    check(out, lse, x, h)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_without_sinks_and_without_causal_masking(d):
    x, h = make([(3, [5, 70]), (1, [4])], 3, 16, 2, d, 32, seed=3)
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = call(g, h, sinks=False)
    check(out, lse, x, h, sinks=False)
    out, lse = call(g, h, causal=False)
    check(out, lse, x, h, causal=False)
    out, lse = call(g, h, return_lse=False)
    assert lse is None
    check(out, None, x, h)


@gpu
def test_prefix_of_a_row_that_sees_only_its_own_keys():
    """A window shorter than every sequence's own keys: the prefix is read by nobody."""
    x, h = make([(4, [100, 90, 200])], 1, 64, 8, 64, 16, seed=8)
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = call(g, h, window=64)
    check(out, lse, x, h, window=64)


@gpu
def test_agrees_with_the_paged_decode():
    x, h = make([(6, [3, 50, 12]), (2, [300, 3])], 3, 64, 4, 128, 64, seed=5)
    g = {k: v.cuda() for k, v in x.items()}
    o1, l1 = call(g, h)
    o2, l2 = sa.sinkattn_decode_paged(g["q"], g["k_pages"], g["v_pages"], g["kv_indptr"],
                                      g["page_indptr"], g["page_indices"], g["sinks"], 3,
                                      h["keys"])
    assert (o1.float() - o2.float()).abs().max().item() <= 1e-2
    assert (l1 - l2).abs().max().item() <= 2e-4


@gpu
@pytest.mark.parametrize("share", [2, 0])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_call_replays_on_new_inputs(fp8, share):
    """One graph, two inputs with other lengths and groups of the same sizes."""
    first, h = make([(3, [5, 70, 9]), (1, [4, 30])], 2, 64, 8, 64, 16, seed=1, fp8=fp8)
    other, h2 = make([(2, [33, 6]), (2, [8, 2, 60])], 2, 64, 8, 64, 16, seed=2, fp8=fp8)
    rows = max(first["k_pages"].shape[0], other["k_pages"].shape[0])
    n = max(first["page_indices"].numel(), other["page_indices"].numel())

    def padded(x):
        x = dict(x)
        for name in ("k_pages", "v_pages"):
            p = x[name]
            x[name] = torch.cat([p, torch.zeros((rows - p.shape[0], *p.shape[1:]), dtype=p.dtype)])
        i = x["page_indices"]
        x["page_indices"] = torch.cat([i, torch.zeros(n - i.numel(), dtype=torch.int32)])
        return x

    h["max_prefix"], h["max_suffix"], h["keys"] = 48, 70, 118
    a, b = padded(first), padded(other)
    g = {k: v.cuda() for k, v in a.items() if k not in ("k", "v", "cu_q")}
    bufs = dict(out=torch.empty_like(g["q"]),
                lse=torch.empty(g["q"].shape[:2], dtype=torch.float32, device="cuda"),
                workspace=torch.empty(sa.sinkattn_decode_shared_workspace_bytes(
                    5, 2, 64, 64, 2, 2, 2), dtype=torch.uint8, device="cuda"))
    call(g, h, num_splits=2, prefix_splits=share, **bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(g, h, num_splits=2, prefix_splits=share, **bufs)
    for x in (b, a, b):
        for k in g:
            g[k].copy_(x[k])
        bufs["out"].fill_(float("nan"))
        bufs["workspace"].fill_(0xff)   # NaN in every partial of the last replay
        graph.replay()
        torch.cuda.synchronize()
        check(bufs["out"], bufs["lse"], x, h)


@gpu
def test_two_streams_with_their_own_workspaces():
    x, h = make([(12, [1 + i for i in range(24)])], 1, 64, 8, 64, 16, seed=4)
    y, hy = make([(5, [9 + i for i in range(7)])], 2, 64, 4, 128, 64, seed=6)
    gx, gy = ({k: v.cuda() for k, v in z.items()} for z in (x, y))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for st, g, hh in ((streams[0], gx, h), (streams[1], gy, hy)):
            with torch.cuda.stream(st):
                got.append(call(g, hh))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        check(o, l, *((y, hy) if i % 2 else (x, h)))


@gpu
def test_outputs_of_an_empty_batch_are_left():
    x, h = make([(1, [])], 1, 8, 1, 64, 16, seed=1)
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = call(g, h)
    assert out.shape[0] == 0 and lse.shape[0] == 0


@gpu
@pytest.mark.parametrize("share", [4, 0])
@pytest.mark.parametrize("bad", ["prefix_unaligned", "prefix_too_long", "suffix_short",
                                 "suffix_long", "groups_end", "groups_back", "pages_few"])
def test_wrong_lengths_are_recorded(bad, share):
    """Device arrays that break a rule: recorded, and nothing is read outside
    the pools or the lists (the plan turns the part into an empty one)."""
    x, h = make([(3, [5, 70, 9]), (1, [4, 30])], 2, 16, 2, 64, 16, seed=1)
    if bad == "prefix_unaligned":
        x["prefix_lens"][0] = 40
    elif bad == "prefix_too_long":
        x["prefix_lens"][1] = 64     # past max_prefix_len
    elif bad == "suffix_short":
        x["prefix_lens"][1] = 32     # sequence 3 keeps no room for its two drafts
    elif bad == "suffix_long":
        h["max_suffix"] = 60
    elif bad == "groups_end":
        x["group_indptr"][2] = 4
    elif bad == "groups_back":
        x["group_indptr"][1] = 9
    elif bad == "pages_few":
        x["page_indptr"][1:] -= 1    # the first list is one page short
        x["page_indices"] = x["page_indices"][1:].clone()
    g = {k: v.cuda() for k, v in x.items()}
    assert sa.sinkattn_debug_status() == 0
    call(g, h, prefix_splits=share)
    assert sa.sinkattn_debug_status() == BAD_LENGTHS
    assert sa.sinkattn_debug_status() == 0


# ---------------------------------------------------------------------- host
A16, WS = 0x1000, 0x10000


def raw(**kw):
    a = dict(q=A16, k=A16, v=A16, kv=A16, pp=A16, pi=A16, gp=A16, pl=A16, ng=2, npg=8, ps=16, B=4,
             ql=1, mp=64, ms=40, Hq=8, Hkv=2, d=64, scale=0.125, causal=1, window=0, psp=2, ss=2,
             sinks=None, ws=WS, wsb=1 << 30, out=A16, lse=None)
    a.update(kw)
    L = sa.lib()
    return L.sinkattn_decode_shared_paged(
        a["q"], a["k"], a["v"], a["kv"], a["pp"], a["pi"], a["gp"], a["pl"], a["ng"], a["npg"],
        a["ps"], a["B"], a["ql"], a["mp"], a["ms"], a["Hq"], a["Hkv"], a["d"], a["scale"],
        a["causal"], a["window"], a["psp"], a["ss"], a["sinks"], a["ws"], a["wsb"], a["out"],
        a["lse"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(gp=None), 1), (dict(pl=None), 1), (dict(pp=None), 1),
    (dict(kv=None), 1), (dict(out=None), 1), (dict(out=A16 + 2), 1), (dict(lse=A16 + 2), 1),
    (dict(ws=None), 1), (dict(ws=WS + 16), 1), (dict(wsb=1000), 1),
    (dict(ng=0), 1), (dict(ng=70000), 2), (dict(mp=-1), 1), (dict(ms=0), 1), (dict(ql=41), 1),
    (dict(ps=24), 2), (dict(ps=8), 2), (dict(d=96), 2), (dict(Hq=9), 2), (dict(Hq=130), 2),
    (dict(window=8, causal=0), 2), (dict(psp=4000, ss=200), 2), (dict(B=-1), 1),
    (dict(mp=2 ** 31 - 1), 2), (dict(scale=0.0), 1), (dict(npg=1 << 27), 2),
])
def test_rejects_bad_arguments(kw, status):
    assert raw(**kw) == status
    assert sa.sinkattn_last_error() != ""


def test_empty_batch_is_a_no_op():
    assert raw(B=0) == 0


def test_fp8_rejects_missing_scales():
    L = sa.lib()
    for ks, vs in ((None, A16), (A16, None), (A16 + 2, A16)):
        rc = L.sinkattn_decode_shared_paged_fp8(
            A16, A16, A16, ks, vs, A16, A16, A16, A16, A16, 2, 8, 16, 4, 1, 64, 40, 8, 2, 64,
            0.125, 1, 0, 2, 2, None, WS, 1 << 30, A16, None, None)
        assert rc == INVALID_ARG and "scale" in sa.sinkattn_last_error()


def test_workspace_holds_plan_and_partials():
    n = sa.sinkattn_decode_shared_workspace_bytes(64, 2, 64, 64, 3, 4, 2)
    parts = sa.sinkattn_decode_workspace_bytes(64, 2, 64, 64, 6)
    assert n - parts >= 4 * (2 * 65 + 3 * 4 + 128)
    with pytest.raises(sa.SinkAttnError):
        sa.sinkattn_decode_shared_workspace_bytes(64, 2, 64, 64, 3, 4, 0)
    with pytest.raises(sa.SinkAttnError):
        sa.sinkattn_decode_shared_workspace_bytes(64, 2, 64, 96, 3, 4, 2)


def test_default_splits_are_positive():
    for B, ql, ng, mp, ms in ((1, 1, 1, 0, 1), (64, 1, 1, 8192, 512), (256, 3, 5, 4096, 9000)):
        ps, ss = sa.sinkattn_decode_shared_default_splits(B, ql, 64, 8, 64, ng, mp, ms)
        assert ps >= (0 if B == 1 else 1) and ss >= 1 and ps + ss <= 4096


def test_refuses_tensors_of_another_kind():
    x, h = make([(1, [3])], 1, 8, 1, 64, 16)
    with pytest.raises(sa.SinkAttnError) as e:
        call(x, h)   # CPU tensors
    assert e.value.status == INVALID_ARG
    assert UNSUPPORTED == 2


@gpu
@pytest.mark.parametrize("name,change", [
    ("q", lambda t: t.float()), ("kv_indptr", lambda t: t.long()),
    ("page_indptr", lambda t: t[:-1]), ("group_indptr", lambda t: torch.cat([t, t])),
    ("prefix_lens", lambda t: t.long()), ("v_pages", lambda t: t[:-1]),
    ("k_pages", lambda t: t.transpose(1, 2)), ("sinks", lambda t: t[:-1]),
    ("page_indices", lambda t: t.cpu()), ("q", lambda t: torch.cat([t, t])),
])
def test_refuses_tensors_that_would_be_misread(name, change):
    x, h = make([(2, [3, 9])], 1, 8, 2, 64, 16)
    g = {k: v.cuda() for k, v in x.items()}
    g[name] = change(g[name])
    with pytest.raises(sa.SinkAttnError) as e:
        call(g, h)
    assert e.value.status == INVALID_ARG


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_many_short_items_repeat_bit_for_bit(d, fp8):
    """Row blocks cut into items of two or three key tiles, several per thread block: every
    repetition gives the same bits as the first (a partial read before its last product
    shows here as rows that change)."""
    G = 8 if d == 64 else 16
    per = 128 // G
    groups = [(32, [1] * (2 * per)), (33, [2] * (per - 1)), (64, [1] * (4 * per + 3)), (1, [5] * per)]
    x, h = make(groups, 1, 2 * G, 2, d, 16, seed=16, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    first = {}
    for rep in range(40):
        for ps in (2, 3, 5, 16):
            out, lse = call(g, h, prefix_splits=ps, num_splits=1)
            if rep == 0:
                check(out, lse, x, h)
                first[ps] = out, lse
            assert torch.equal(out, first[ps][0]) and torch.equal(lse, first[ps][1])


@gpu
@pytest.mark.parametrize("kernel", ["auto", "warp"])
@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (64, True)])
def test_more_groups_than_are_staged(d, fp8, kernel):
    """700 groups, a third of them without a prefix, more row blocks than groups in some."""
    rng = random.Random(3)
    groups = [(rng.choice([0, 1, 2]), [rng.randint(1, 20) for _ in range(rng.randint(0, 3))])
              for _ in range(690)] + [(3, [2] * 40)] + [(1, [3])] * 9
    x, h = make(groups, 1, 16, 2, d, 16, seed=2, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    sa.sinkattn_set_decode_kernel(kernel)
    try:
        out, lse = call(g, h, prefix_splits=2)
    finally:
        sa.sinkattn_set_decode_kernel("auto")
    check(out, lse, x, h)


@gpu
def test_more_sequences_than_are_staged():
    """3000 sequences at d 128: the own pass reads lengths from memory, not from its copy."""
    rng = random.Random(5)
    x, h = make([(2, [rng.randint(1, 9) for _ in range(1700)]), (0, [rng.randint(1, 30) for _ in range(1300)])],
                1, 2, 1, 128, 16, seed=4)
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = call(g, h)
    check(out, lse, x, h)


@gpu
def test_call_on_another_stream_keeps_its_workspace():
    """The workspace that a call on a side stream allocates is not handed out to the current
    stream while the side stream still runs."""
    x, h = make([(40, [5] * 30)], 1, 64, 8, 64, 16, seed=9)
    g = {k: v.cuda() for k, v in x.items()}
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = []
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)   # the call waits behind this on its stream
    for _ in range(4):
        got.append(call(g, h, stream=st))
        # the same sizes on the current stream, at once overwritten
        n = sa.sinkattn_decode_shared_workspace_bytes(
            30, 1, 64, 64, 1, 4, sa.sinkattn_decode_shared_default_splits(30, 1, 64, 8, 64, 1, 640, 5)[1])
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xff)
    st.synchronize()
    torch.cuda.synchronize()
    for o, l in got:
        check(o, l, x, h)


@gpu
@pytest.mark.parametrize("kernel", ["auto", "warp"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("groups,q_len,Hq,Hkv,d,page", [
    ([(1, [20] + [5] * 9)], 1, 16, 2, 64, 16),            # tiles end behind the prefix
    ([(3, [64] + [5] * 9), (4, [30, 7])], 1, 64, 8, 64, 32),
    ([(1, [200, 3, 4])], 3, 64, 4, 128, 64),
    ([(5, [17] * 12), (1, [40] * 6)], 2, 32, 4, 128, 16),
    ([(1, [9, 8])], 1, 8, 8, 64, 16),
    ([(1, [300, 8])], 1, 8, 8, 64, 16),
])
@pytest.mark.parametrize("where", ["k_pages", "v_pages"])
def test_a_sequence_with_nan_keys_spoils_no_other(groups, q_len, Hq, Hkv, d, page, fp8, kernel,
                                                  where):
    """The own keys and values of each group's first sequence lie behind the prefix in the list
    that the prefix is read from: NaN there are that sequence's alone, and its answer is NaN."""
    x, h = make(groups, q_len, Hq, Hkv, d, page, seed=3, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    firsts = [int(b) for b in x["group_indptr"][:-1]]
    spoilt = []
    for b, (pre, _) in zip(firsts, groups):
        lo, hi = int(x["page_indptr"][b]) + pre, int(x["page_indptr"][b + 1])
        spoilt += x["page_indices"][lo:hi].tolist()
    g[where][torch.tensor(spoilt, device="cuda").long()] = 0x7f if fp8 else float("nan")
    sa.sinkattn_set_decode_kernel(kernel)
    try:
        out, lse = call(g, h)
    finally:
        sa.sinkattn_set_decode_kernel("auto")
    assert sa.sinkattn_debug_status() == 0
    o, l, A = want(x, h)
    o, A, got = (t.reshape(out.shape) for t in (o, A, out.float().cpu().numpy()))
    l, gl = l.reshape(lse.shape), lse.cpu().numpy()
    rest = np.ones(o.shape[0], dtype=bool)
    for b in firsts:
        rest[b * q_len:(b + 1) * q_len] = False
        assert np.isnan(got[b * q_len:(b + 1) * q_len]).all()
    o, l, A, got, gl = (t[rest] for t in (o, l, A, got, gl))
    assert np.isfinite(got).all()
    weight = 2.0 ** -11 if fp8 else 2.0 ** -8
    low = 2.0 ** -25 * h["keys"] * 6.0 if fp8 else 0.0
    room = 2.0 ** -8 * np.abs(o) + (weight + 2e-4) * A + low + 1e-6
    assert (np.abs(got - o) <= room).all()
    assert np.abs(gl - l).max() <= 1e-4


@gpu
@pytest.mark.parametrize("splits", [(2, 1), (30, 9)])   # several rows a warp; one row of many slots
def test_a_sink_of_all_weight(splits):
    x, h = make([(3, [9, 8, 1])], 1, 8, 2, 64, 16, seed=4)
    x["sinks"][2] = float("inf")
    x["sinks"][5] = float("-inf")
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = call(g, h, prefix_splits=splits[0], num_splits=splits[1])
    assert (out[:, 2] == 0).all() and (lse[:, 2] == float("inf")).all()
    x["sinks"][2] = 0.0
    o, l, A = want(x, h)
    o, A, got = (t.reshape(out.shape) for t in (o, A, out.float().cpu().numpy()))
    keep = [0, 1, 3, 4, 5, 6, 7]
    assert (np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2e-4) * A + 1e-6)[:, keep].all()
    assert np.abs(lse.cpu().numpy() - l.reshape(lse.shape))[:, keep].max() <= 1e-4


@gpu
@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (64, True), (128, True)])
def test_a_loose_bound_on_the_prefixes_changes_nothing(d, fp8):
    x, h = make([(20, [5] * 12), (3, [9] * 7)], 1, 64, 8, d, 16, seed=6, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    got = []
    for bound in (h["max_prefix"], 1 << 20):
        got.append(call(g, dict(h, max_prefix=bound), prefix_splits=4, num_splits=1))
    check(*got[0], x, h)
    assert all(torch.equal(a, b) for a, b in zip(*got))


@gpu
@pytest.mark.parametrize("kernel", ["auto", "warp"])
@pytest.mark.parametrize("d", [64, 128])
def test_groups_that_do_not_cut_the_batch_share_nothing(d, kernel):
    x, h = make([(0, [5 + 3 * i for i in range(20)])], 1, 64, 8, d, 16, seed=8)
    g = {k: v.cuda() for k, v in x.items()}
    sa.sinkattn_set_decode_kernel(kernel)
    try:
        for cut in ([0, 21], [0, 7, 5, 20], [1, 20]):
            g["group_indptr"] = torch.tensor(cut, dtype=torch.int32, device="cuda")
            g["prefix_lens"] = torch.full((len(cut) - 1,), 16, dtype=torch.int32, device="cuda")
            work = torch.full((1 << 23,), 0x7f, dtype=torch.uint8, device="cuda")
            out, lse = call(g, dict(h, max_prefix=64), workspace=work)
            assert sa.sinkattn_debug_status() == BAD_LENGTHS
            check(out, lse, x, h)
    finally:
        sa.sinkattn_set_decode_kernel("auto")


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_calls_of_few_keys_read_each_sequence_alone(case, fp8):
    groups, q_len, Hq, Hkv, d, page, window, _, ss, qs = case
    x, h = make(groups, q_len, Hq, Hkv, d, page, seed=page + q_len + 1, q_scale=qs, fp8=fp8)
    B = x["kv_indptr"].numel() - 1
    alone = B * (h["max_prefix"] + h["max_suffix"]) * Hkv * d <= 10 << 20   # (all but one or two)
    ps, _ = sa.sinkattn_decode_shared_default_splits(B, q_len, Hq, Hkv, d, len(groups),
                                                     h["max_prefix"], h["max_suffix"])
    assert (ps == 0) == alone
    g = {k: v.cuda() for k, v in x.items()}
    for splits in (0, ss):
        out, lse = call(g, h, window=window, prefix_splits=0, num_splits=splits)
        check(out, lse, x, h, window=window)
    assert sa.sinkattn_debug_status() == 0


@gpu
@pytest.mark.parametrize("d,q_len,fp8", [(64, 1, False), (64, 2, True), (128, 3, False), (128, 1, True)])
def test_calls_of_many_keys_share_by_default(d, q_len, fp8):
    groups = [(150, [3 + 7 * i for i in range(30)]), (40, [9] * 11), (0, [50, 4])]
    x, h = make(groups, q_len, 16, 4, d, 16, seed=d + q_len, fp8=fp8)
    assert sa.sinkattn_decode_shared_default_splits(43, q_len, 16, 4, d, 3, h["max_prefix"],
                                                    8 << 20)[0] > 0
    g = {k: v.cuda() for k, v in x.items()}
    for bound in (h["max_suffix"], 100000):
        out, lse = call(g, dict(h, max_suffix=bound), prefix_splits=0)
        check(out, lse, x, h)


@gpu
@pytest.mark.parametrize("at", [0, 300, 1249])
def test_wrong_lengths_of_many_short_sequences_are_recorded(at):
    """1250 sequences in 417 groups, read alone: each one's length counts."""
    x, h = make([(i % 2, [3, 5, 2]) for i in range(416)] + [(1, [4, 4])], 1, 2, 1, 64, 16, seed=7)
    assert x["kv_indptr"].numel() == 1251
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = call(g, h, prefix_splits=0)
    assert sa.sinkattn_debug_status() == 0
    check(out, lse, x, h)
    own = int(x["kv_indptr"][at + 1] - x["kv_indptr"][at]) % 16   # (prefixes of 0 or 16 keys)
    g["kv_indptr"][at + 1:] -= own   # no key of its own left, the others as they were
    call(g, h, prefix_splits=0)
    assert sa.sinkattn_debug_status() == BAD_LENGTHS


def one_late_key(d, fp8, seed):
    """40 sequences behind 768 shared keys, 8 rows per KV head each. All keys are zero but two of the
    prefix: key 5, whose logit is 2^20 in weight, and key 700, whose weight is another 2^6 to 2^7.7 times
    that. So a row's output is key 700's value but for less than 2^-6, and its weight, relative to a
    reference maximum that stayed at key 5, is no power of two. Returns (x, h, mass outside key 700)."""
    x, h = make([(48, [2] * 40)], 1, 64, 8, d, 16, seed=seed, fp8=fp8)
    one = 0x70 if fp8 else 1.0   # (the code of 128)
    x["k"].zero_()
    x["k_pages"].zero_()
    for key, dim in ((5, 0), (700, 1)):
        x["k"].view(40, 8, 770, d)[:, :, key, dim] = one
        x["k_pages"][x["page_indices"][key // 16].item(), :, key % 16, dim] = one
    value = 128.0 * x["k_scale"] if fp8 else torch.ones(8)
    unit = (math.log(2) * math.sqrt(d) / value).repeat_interleave(8)   # q of one bit of logit, by head
    gen = torch.Generator().manual_seed(seed)
    bits = 6.0 + 1.7 * torch.rand((40, 64), generator=gen)
    x["q"].zero_()
    x["q"][:, :, 0] = (20.0 * unit).to(torch.bfloat16)
    x["q"][:, :, 1] = ((20.0 + bits) * unit).to(torch.bfloat16)
    logits = x["q"][:, :, :2].double() / unit.double()[None, :, None]   # in bits
    rest = torch.exp2(logits[..., 0] - logits[..., 1]) + 768 * torch.exp2(-logits[..., 1])
    assert ((logits[..., 1] - logits[..., 0]) < 8).all() and (rest < 2.0 ** -5.8).all()
    return x, h, rest.numpy().reshape(-1)


@gpu
@pytest.mark.parametrize("kernel", ["auto", "warp"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_weight_that_is_most_of_a_row_is_not_rounded_into_the_output(d, fp8, kernel):
    """Rounded weights w (1 + r), |r| <= 2^-8, over a divisor that counts the dominant one as rounded leave
    sum p_j r_j (v_j - out) for the counted weights and sum p_j r_j v_j for the rest: with e the mass outside
    the dominant key and V the largest |v|, at most 2^-8 e 2 V + 2^-8 e 2 V, and e V 2^-7 more for logits
    that are off by 2^-8 at most (products of one term, exact to 2^-22 of 28 bits). The output's own
    rounding adds 2^-8 |out|; no 2^-8 |out| of the weight's own."""
    x, h, rest = one_late_key(d, fp8, seed=d)
    g = {k: v.cuda() for k, v in x.items()}
    sa.sinkattn_set_decode_kernel(kernel)
    try:
        out, lse = call(g, h, sinks=False, prefix_splits=1, num_splits=1)
    finally:
        sa.sinkattn_set_decode_kernel("auto")
    o, l, _ = want(x, h, sinks=False)
    v = x["v"].view(torch.float8_e4m3fn).float() * x["v_scale"].max() if fp8 else x["v"].float()
    room = 2.0 ** -8 * np.abs(o) + rest.reshape(*o.shape[:-1], 1) * (2.0 ** -6 + 2.0 ** -7) * v.abs().max().item()
    err = np.abs(out.float().cpu().numpy().reshape(o.shape) - o)
    assert (err <= room + 1e-6).all(), "off by %.3g of the room" % (err / (room + 1e-6)).max()
    assert np.abs(lse.cpu().numpy().reshape(l.shape) - l).max() <= 1e-4


@gpu
@pytest.mark.parametrize("q_scale", [3.0, 6.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_peaky_rows_meet_the_bounds_of_the_other_paths(fp8, d, q_scale):
    """max-abs 1e-2, mean-abs 1e-3, as for prefill and decode, with |v| up to 1/2: a weight's half step
    and the output's are below 2^-8 / 2 + 2^-10 together, their means a quarter of that."""
    x, h = make([(40, [3, 17] * 16)], 1, 64, 8, d, 32, seed=d, q_scale=q_scale, fp8=fp8)
    for name in ("v", "v_pages"):
        if fp8:
            f = x[name].view(torch.float8_e4m3fn).float().clamp(-90.0, 90.0) * 0.4
            x[name] = f.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x[name] = (x[name].float().clamp(-2.0, 2.0) * 0.25).to(torch.bfloat16)
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = call(g, h, prefix_splits=2, num_splits=1)
    o, l, _ = want(x, h)
    compare(out, lse, o, l, "shared prefix, logits spread by %g" % q_scale)


def test_split_counts_of_sizes_beyond_64_bits():
    """batch x KV heads x head_dim of these wraps to zero in 64 bits."""
    for B, ql, Hq, Hkv, ng in ((1 << 30, 1, 1 << 30, 1 << 30, 1),
                               (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1),
                               (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1, 2 ** 31 - 1),
                               (2 ** 31 - 1, 2 ** 31 - 1, 64, 1, 2 ** 31 - 1)):
        for mp in (0, 2 ** 31 - 1):
            for d in (64, 128):
                ps, ss = sa.sinkattn_decode_shared_default_splits(B, ql, Hq, Hkv, d, ng, mp, 2 ** 31 - 1)
                assert 1 <= ps <= 16 and 1 <= ss <= 4096
    assert raw(B=1 << 30, Hq=1 << 30, Hkv=1 << 30) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(),                                       # head_dim 64
    dict(d=128, fp8=True),                        # codes, whose own keys have the warp-level kernel only
    dict(fp8=True),
])
def test_forced_tcgen05_is_refused_before_any_launch(kw):
    """(Without a GPU a launch is a CUDA error, so the status says which came first.)"""
    kw = dict(kw)
    fp8 = kw.pop("fp8", False)
    sa.sinkattn_set_decode_kernel("tcgen05")
    try:
        if fp8:
            rc = sa.lib().sinkattn_decode_shared_paged_fp8(
                A16, A16, A16, A16, A16, A16, A16, A16, A16, A16, 2, 8, 16, 4, 1, 64, 40, 8, 2,
                kw.get("d", 64), 0.125, 1, 0, 2, 2, None, WS, 1 << 30, A16, None, None)
        else:
            rc = raw(**kw)
        text = sa.sinkattn_last_error()
    finally:
        sa.sinkattn_set_decode_kernel("auto")
    assert rc == UNSUPPORTED and "tcgen05" in text


@pytest.mark.parametrize("kw", [
    # units of the tcgen05 prefix pass (8191 full row blocks of 8 KV heads x 32768 tiles of 96)
    dict(B=65535, ql=4, ng=1, Hq=64, Hkv=8, mp=32768 * 96, ms=4),
    dict(B=65535, ql=2048, ng=65535, Hq=16, Hkv=16, mp=32000, ms=2048, psp=2, ss=1),
    dict(B=1, Hq=65536, Hkv=65536, mp=16, ms=1),
])
def test_calls_of_too_many_items_are_refused_before_any_launch(kw):
    assert raw(npg=8, ps=256 if kw["Hkv"] < 100 else 16, wsb=1 << 62, **kw) == UNSUPPORTED


@gpu
@pytest.mark.parametrize("d,fp8", [(64, False), (64, True), (128, True)])
def test_a_refused_call_leaves_its_buffers(d, fp8):
    x, h = make([(20, [5] * 40)], 1, 64, 8, d, 16, seed=2, fp8=fp8)
    g = {k: v.cuda() for k, v in x.items()}
    bufs = dict(out=torch.full_like(g["q"], 7.0), lse=torch.full(g["q"].shape[:2], 7.0, device="cuda"),
                workspace=torch.full((sa.sinkattn_decode_shared_workspace_bytes(40, 1, 64, d, 1, 4, 2),),
                                     7, dtype=torch.uint8, device="cuda"))
    sa.sinkattn_set_decode_kernel("tcgen05")
    try:
        with pytest.raises(sa.SinkAttnError) as e:
            call(g, h, num_splits=2, **bufs)
    finally:
        sa.sinkattn_set_decode_kernel("auto")
    assert e.value.status == UNSUPPORTED
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in bufs.values())


@gpu
@pytest.mark.parametrize("case", [i for i, c in enumerate(CASES) if c[4] == 128],
                         ids=[n for n, c in zip(IDS, CASES) if c[4] == 128])
def test_forced_tcgen05_matches_oracle(case):
    groups, q_len, Hq, Hkv, d, page, window, ps, ss, qs = CASES[case]
    x, h = make(groups, q_len, Hq, Hkv, d, page, seed=page, q_scale=qs)
    g = {k: v.cuda() for k, v in x.items()}
    sa.sinkattn_set_decode_kernel("tcgen05")
    try:
        out, lse = call(g, h, window=window, prefix_splits=ps, num_splits=ss)
    finally:
        sa.sinkattn_set_decode_kernel("auto")
    check(out, lse, x, h, window=window)


def test_sizes_beyond_32_bits_are_refused():
    """(As 32-bit arguments they would be other sizes: 2^32 + 64 keys would be 64.)"""
    with pytest.raises(sa.SinkAttnError) as e:
        sa.sinkattn_decode_shared_workspace_bytes(2 ** 32 + 4, 1, 8, 64, 1, 2, 2)
    assert e.value.status == INVALID_ARG
    with pytest.raises(sa.SinkAttnError) as e:
        sa.sinkattn_decode_shared_default_splits(4, 1, 8, 2, 64, 1, 2 ** 32 + 64, 40)
    assert e.value.status == INVALID_ARG


@gpu
@pytest.mark.parametrize("name", ["max_prefix", "max_suffix"])
def test_key_bounds_beyond_32_bits_are_refused(name):
    x, h = make([(4, [5, 9])], 1, 8, 1, 64, 16)
    g = {k: v.cuda() for k, v in x.items()}
    for n in (2 ** 32 + h[name], 2 ** 31):
        with pytest.raises(sa.SinkAttnError) as e:
            call(g, dict(h, **{name: n}))
        assert e.value.status == INVALID_ARG


@gpu
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5])
def test_a_window_wider_than_any_sequence_hides_nothing(window):
    x, h = make([(4, [5, 9, 60])], 2, 64, 8, 64, 16, seed=4)
    g = {k: v.cuda() for k, v in x.items()}
    for share in (4, 0):
        out, lse = call(g, h, window=window, prefix_splits=share)
        check(out, lse, x, h)


@pytest.mark.parametrize("kernel", ["auto", "warp", "tcgen05"])
def test_empty_batch_is_a_no_op_under_any_kernel(kernel):
    sa.sinkattn_set_decode_kernel(kernel)
    try:
        assert raw(B=0) == 0
    finally:
        sa.sinkattn_set_decode_kernel("auto")
