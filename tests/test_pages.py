"""Page tables, page copies and appends, held bit for bit to a plain Python
model (_page_model.py); e4m3 codes to torch's conversion of the fp32 quotient
and to the format's definition in 64 bits."""
import math
import random

import numpy as np
import pytest
import torch

import oracle
import gqa_attention_softmax_gb300 as sa
from gqa_attention_softmax_gb300._binding import (BAD_LENGTHS, BAD_PAGES, INVALID_ARG,
                                                  OUT_OF_PAGES, UNSUPPORTED)
from _page_model import PageModel

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_softmax_gb300 import _build
    _build.build()
    oracle.build()
    yield
    if torch.cuda.is_available():
        assert sa.sinkattn_debug_status() == 0


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).reshape(-1), dtype=torch.int32, device="cuda")


class Pair:
    """A table and its model, with pools of `layers` layers."""

    def __init__(self, N, P, S, M, layers=1, Hkv=2, d=64, dtype=torch.bfloat16, seed=0):
        self.table = sa.PageTable(None, N, P, S, M)
        self.model = PageModel(N, P, S, M)
        gen = torch.Generator().manual_seed(seed)
        shape = (layers, N, Hkv, P, d)
        if dtype is torch.uint8:
            pools = [torch.randint(0, 127, shape, generator=gen, dtype=torch.uint8) for _ in range(2)]
        else:
            pools = [torch.randn(shape, generator=gen).to(dtype) for _ in range(2)]
        self.want = [p.clone() for p in pools]
        self.k, self.v = (p.cuda() for p in pools)

    def used(self):
        t, m = self.table, self.model
        return t.state[:16 + m.S * (1 + m.M) + 2 * m.N].cpu().numpy()

    def check(self):
        got, (count, words) = self.used(), self.model.words()
        assert got[0] == count
        np.testing.assert_array_equal(got[16:], words)
        for a, b in zip((self.k, self.v), self.want):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))

    def reserve(self, ids, new):
        want = self.model.reserve(ids, new, self.want)
        slots = sa.sinkattn_pages_reserve(self.table, i32(ids), i32(np.cumsum([0] + list(new))),
                                          sum(new), self.k, self.v)
        got = slots.cpu().tolist()
        assert got == (want if want is not None else [-1] * sum(new))
        return want

    def fork(self, src, dst):
        sa.sinkattn_pages_fork(self.table, i32(src), i32(dst))
        return self.model.fork(src, dst)

    def truncate(self, ids, new=None):
        sa.sinkattn_pages_truncate(self.table, i32(ids), None if new is None else i32(new))
        return self.model.truncate(ids, [0] * len(ids) if new is None else new)

    def compact(self):
        got = sa.sinkattn_pages_compact(self.table, self.k, self.v).cpu().tolist()
        assert got == self.model.compact(self.want)

    def lists(self, ids):
        m = self.model
        kv, ptr, idx = (t.cpu().tolist() for t in sa.sinkattn_pages_lists(self.table, i32(ids)))
        assert kv == np.cumsum([0] + [m.lens[i] for i in ids]).tolist()
        assert ptr == np.cumsum([0] + [m.pages(m.lens[i]) for i in ids]).tolist()
        assert idx[:ptr[-1]] == [p for i in ids for p in m.list[i][:m.pages(m.lens[i])]]


@gpu
def test_a_new_table_is_empty():
    p = Pair(37, 16, 5, 9)
    p.check()
    p.lists([4, 0, 2])
    p.compact()
    p.check()


@gpu
@pytest.mark.parametrize("seed,N,P,S,M,layers,dtype", [
    (0, 40, 16, 6, 9, 1, torch.bfloat16),       # little room: calls that cannot be served
    (1, 300, 32, 20, 12, 2, torch.bfloat16),
    (2, 900, 64, 33, 40, 1, torch.uint8),
    (3, 5000, 16, 90, 128, 1, torch.uint8),     # more entries than one block takes
    (4, 257, 256, 12, 5, 3, torch.bfloat16),
    (5, 9000, 16, 1500, 10, 1, torch.uint8),    # more sequences than a block has threads
])
def test_random_calls_follow_the_model(seed, N, P, S, M, layers, dtype):
    rng = random.Random(seed)
    p = Pair(N, P, S, M, layers, dtype=dtype, seed=seed)
    m = p.model
    failed = 0
    for step in range(60):
        op = rng.choice(["reserve"] * 4 + ["fork", "fork", "truncate", "truncate", "free", "lists",
                                           "compact"])
        ids = rng.sample(range(S), rng.randint(1, S))
        if op == "reserve":
            top = rng.choice([1, 1, 3, P, 3 * P])
            new = [rng.randint(0, top) for _ in ids]
            failed += p.reserve(ids, new) is None
        elif op == "fork":
            empty = [i for i in range(S) if m.lens[i] == 0]
            full = [i for i in range(S) if m.lens[i] > 0]
            if not empty or not full:
                continue
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            assert p.fork([rng.choice(full) for _ in dst], dst)
        elif op == "truncate":
            p.truncate(ids, [rng.randint(0, m.lens[i]) for i in ids])
        elif op == "free":
            p.truncate(ids[:max(1, len(ids) // 2)])
        elif op == "lists":
            p.lists(ids)
        else:
            p.compact()
        p.check()
    status = sa.sinkattn_debug_status()
    assert (status in (OUT_OF_PAGES, BAD_PAGES)) == (failed > 0)


@gpu
def test_copy_on_write_of_every_kind():
    p = Pair(60, 16, 8, 6, layers=3)
    p.reserve([0], [37])
    assert p.fork([0, 0, 0], [1, 2, 3])
    p.check()
    p.reserve([2, 1], [1, 20])        # two of four holders write: both copy
    p.check()
    p.reserve([3, 0], [11, 12])       # both that are left write: the first keeps the page
    p.check()
    p.truncate([1], [20])             # back into a page that three others hold whole
    p.reserve([1], [5])
    p.check()
    p.truncate([0, 1, 2, 3])
    p.check()
    assert p.model.count == 60


@gpu
def test_reserve_then_truncate_gives_the_pages_back_in_place():
    p = Pair(64, 16, 4, 20)
    p.reserve([1, 3], [30, 100])
    before = p.used().copy()
    p.reserve([3, 0, 1], [17, 40, 3])
    p.truncate([3, 0, 1], [100, 0, 30])
    p.check()
    after = p.used()
    before[1:16] = after[1:16] = 0   # scratch
    np.testing.assert_array_equal(after, before)


@gpu
@pytest.mark.parametrize("bad", ["id_twice", "id_low", "id_high", "too_long", "no_pages",
                                 "fork_full", "fork_twice", "fork_chain", "fork_id",
                                 "grow_by_truncate", "truncate_twice", "truncate_below",
                                 "cu_total", "cu_back", "lists_id", "lists_room"])
def test_calls_that_cannot_be_served_change_nothing(bad):
    p = Pair(12, 16, 4, 8)
    p.reserve([0, 2], [50, 16])
    want = BAD_PAGES
    t, one = p.table, i32([0, 1])
    if bad == "id_twice":
        assert p.reserve([1, 1], [2, 2]) is None
    elif bad == "id_low":
        assert p.reserve([-1, 1], [2, 2]) is None
    elif bad == "id_high":
        assert p.reserve([1, 4], [2, 2]) is None
    elif bad == "too_long":
        assert p.reserve([0], [79]) is None
    elif bad == "no_pages":
        assert p.reserve([1, 3], [60, 61]) is None
        want = OUT_OF_PAGES
    elif bad == "fork_full":
        assert not p.fork([0], [2])
    elif bad == "fork_twice":
        assert not p.fork([0, 2], [1, 1])
    elif bad == "fork_chain":
        assert not p.fork([0, 1], [1, 3])
    elif bad == "fork_id":
        assert not p.fork([0, 9], [1, 3])
    elif bad == "grow_by_truncate":
        assert not p.truncate([0, 2], [51, 3])
    elif bad == "truncate_twice":
        assert not p.truncate([0, 0], [3, 3])
    elif bad == "truncate_below":
        assert not p.truncate([0], [-1])
    elif bad in ("cu_total", "cu_back"):
        cu = [0, 3, 6] if bad == "cu_total" else [0, 9, 5]
        s = sa.sinkattn_pages_reserve(t, one, i32(cu), 5, p.k, p.v)
        assert s.cpu().tolist() == [-1] * 5
        want = BAD_LENGTHS if bad == "cu_total" else BAD_PAGES
    elif bad == "lists_id":
        kv, ptr, idx = sa.sinkattn_pages_lists(t, i32([0, 7, 2]))
        assert kv.cpu().tolist() == [0, 50, 50, 66] and ptr.cpu().tolist() == [0, 4, 4, 5]
    elif bad == "lists_room":
        room = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        kv, ptr, idx = sa.sinkattn_pages_lists(t, i32([2, 0]), page_indices=room)
        assert kv.cpu().tolist() == [0, 16, 66] and ptr.cpu().tolist() == [0, 1, 4]
        assert idx.cpu().tolist() == [p.model.list[2][0], -7, -7, -7]
        want = BAD_LENGTHS
    p.check()
    assert sa.sinkattn_debug_status() == want
    p.reserve([1], [3])   # the table is still usable
    p.check()


@gpu
def test_pools_of_layers_with_a_stride():
    """K and V interleaved layer by layer in one buffer."""
    p = Pair(30, 32, 5, 4, layers=3)
    both = torch.stack([p.k, p.v], dim=1)   # [layers, 2, N, Hkv, P, d]
    p.k, p.v = both[:, 0], both[:, 1]
    p.reserve([0, 1], [40, 70])
    p.fork([0, 1, 1], [2, 3, 4])
    p.reserve([2, 3, 4], [1, 1, 30])
    p.check()
    p.truncate([0, 3])
    p.compact()
    p.check()


@gpu
def test_captured_draft_steps_replay():
    """Reserve, append and roll back as one graph, replayed while the table grows."""
    p = Pair(80, 16, 3, 20)
    p.reserve([0, 1, 2], [15, 3, 60])
    ids, cu, keep = i32([2, 0, 1]), i32([0, 4, 8, 12]), i32([0, 0, 0])
    k = torch.randn((12, 2, 64), device="cuda").to(torch.bfloat16)
    slots = torch.empty(12, dtype=torch.int32, device="cuda")

    def step():
        sa.sinkattn_pages_reserve(p.table, ids, cu, 12, p.k, p.v, slots=slots)
        sa.sinkattn_append_paged(k, k, slots, p.k[0], p.v[0])
        sa.sinkattn_pages_truncate(p.table, ids, keep)

    def model(accepted):
        got = p.model.reserve([2, 0, 1], [4, 4, 4], p.want)
        for t, s in enumerate(got):
            for pool in p.want:
                pool[0, s // 16, :, s % 16] = k[t].cpu()
        p.model.truncate([2, 0, 1], accepted)

    lens = [60, 15, 3]
    lens = [n + 2 for n in lens]
    keep.copy_(i32(lens))
    step()
    model(lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for more in (1, 4, 3, 2):
        lens = [n + more for n in lens]
        keep.copy_(i32(lens))
        graph.replay()
        model(lens)
        p.check()


@gpu
def test_other_streams_and_empty_calls():
    p = Pair(30, 16, 3, 8)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        p.reserve([1], [20])
        p.fork([1], [0])
    st.synchronize()
    p.check()
    none = i32([])
    assert sa.sinkattn_pages_reserve(p.table, none, i32([0]), 0, p.k, p.v).numel() == 0
    assert sa.sinkattn_pages_reserve(p.table, i32([2]), i32([0, 0]), 0, p.k, p.v).numel() == 0
    sa.sinkattn_pages_fork(p.table, none, none)
    sa.sinkattn_pages_truncate(p.table, none)
    kv, ptr, _ = sa.sinkattn_pages_lists(p.table, none)
    assert kv.cpu().tolist() == [0] and ptr.cpu().tolist() == [0]
    p.check()


@gpu
@pytest.mark.parametrize("count", [-1, 31, 2 ** 31 - 1, -2 ** 31])
def test_a_buffer_that_holds_no_table_is_refused(count):
    """A free count that no table has would index before or behind the free list."""
    p = Pair(30, 16, 4, 8)
    p.reserve([1], [40])
    free = p.table.free_count.item()
    p.table.free_count.fill_(count)
    before = p.used().copy()
    slots = sa.sinkattn_pages_reserve(p.table, i32([2]), i32([0, 20]), 20, p.k, p.v)
    assert sa.sinkattn_debug_status() == BAD_PAGES
    assert (slots == -1).all()
    sa.sinkattn_pages_truncate(p.table, i32([1]))
    assert sa.sinkattn_debug_status() == BAD_PAGES
    np.testing.assert_array_equal(np.delete(p.used(), range(1, 16)), np.delete(before, range(1, 16)))
    p.table.free_count.fill_(free)
    p.check()


@gpu
def test_lists_whose_lengths_pass_32_bits():
    M = 1 << 20
    table = sa.PageTable(None, 64, 256, 9, M)
    table.page_list.fill_(7)
    table.seq_lens.fill_(M * 256)
    kv, ptr, pages = sa.sinkattn_pages_lists(table, torch.arange(9, dtype=torch.int32, device="cuda"))
    assert sa.sinkattn_debug_status() == BAD_LENGTHS
    assert kv.tolist() == [min(i * M * 256, 2 ** 31 - 1) for i in range(10)]
    assert ptr.tolist() == [i * M for i in range(10)]
    assert (pages[:7 * M] == 7).all()   # (the eighth and ninth are left out)


@gpu
def test_results_of_a_call_on_another_stream_come_from_its_memory():
    """What a call on a side stream allocates does not lie where the current stream still
    reads, and is not handed out again while the current stream still uses it."""
    p = Pair(600, 16, 8, 80)
    st = torch.cuda.Stream()
    ids, cu = i32([0]), i32([0, 1000])
    torch.cuda.synchronize()
    old = torch.full((1000,), 5, dtype=torch.int32, device="cuda")
    torch.cuda._sleep(20_000_000)
    late = old + 1       # waits behind the sleep, reads what is given back next
    del old
    slots = sa.sinkattn_pages_reserve(p.table, ids, cu, 1000, p.k, p.v, stream=st)
    st.synchronize()
    assert (late == 6).all()
    assert slots.tolist() == list(range(1000))
    torch.cuda._sleep(20_000_000)
    kept = slots + 0     # on the current stream, behind the sleep
    del slots
    with torch.cuda.stream(st):
        torch.full((1000,), -9, dtype=torch.int32, device="cuda")
    st.synchronize()
    assert kept.tolist() == list(range(1000))


def test_a_table_keeps_its_buffer_and_sizes():
    for name in ("state", "num_pages", "page_size", "max_seqs", "max_pages"):
        with pytest.raises(AttributeError):
            setattr(sa.PageTable.__new__(sa.PageTable), name, 1)


# -------------------------------------------------------------------- append
@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("tokens", [0, 1, 7, 301])
def test_append_places_every_row(d, Hkv, tokens):
    P, N = 16, 40
    gen = torch.Generator(device="cuda").manual_seed(tokens + d)
    qkv = torch.randn((tokens, (2 * Hkv + 3) * d), generator=gen, device="cuda").to(torch.bfloat16)
    k = qkv[:, 3 * d:(3 + Hkv) * d].view(tokens, Hkv, d)
    v = qkv[:, (3 + Hkv) * d:].view(tokens, Hkv, d)
    pools = [torch.randn((N, Hkv, P, d), generator=gen, device="cuda").to(torch.bfloat16)
             for _ in range(2)]
    want = [x.clone() for x in pools]
    slots = torch.randperm(N * P, generator=gen, device="cuda")[:tokens].to(torch.int32)
    if tokens > 3:   # padding, and slots behind the pool
        slots[1], slots[3] = -1, N * P
    ok = ((slots >= 0) & (slots < N * P)).nonzero().view(-1)
    at = slots[ok].long()
    for w, x in zip(want, (k, v)):
        w[at // P, :, at % P] = x[ok]
    sa.sinkattn_append_paged(k, v, slots, *pools)
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


@gpu
@pytest.mark.parametrize("d,Hkv", [(64, 8), (128, 1)])
def test_append_fp8_rounds_to_the_nearest_code(d, Hkv):
    P, N, tokens = 32, 20, 333
    gen = torch.Generator(device="cuda").manual_seed(d)
    k = (torch.randn((tokens, Hkv, d), generator=gen, device="cuda") * 3).to(torch.bfloat16)
    v = torch.randn((tokens, Hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
    # ties, subnormal codes, both zeros, saturation, infinities, NaN
    edge = torch.tensor([1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 0.0, -0.0,
                         448.0, 464.0, 480.0, -1e30, math.inf, -math.inf, math.nan, 0.0146],
                        device="cuda").to(torch.bfloat16)
    k[5, 0, :16] = edge
    scale = [0.25 + torch.rand(Hkv, generator=gen, device="cuda") for _ in range(2)]
    scale[0][0] = 1.0
    pools = [torch.randint(0, 255, (N, Hkv, P, d), generator=gen, device="cuda",
                           dtype=torch.uint8) for _ in range(2)]
    want = [x.clone() for x in pools]
    slots = torch.randperm(N * P, generator=gen, device="cuda")[:tokens].to(torch.int32)
    at = slots.long()
    sa.sinkattn_append_paged_fp8(k, v, slots, *scale, *pools)
    for w, x, s, got in zip(want, (k, v), scale, pools):
        quot = (x.float() / s[None, :, None]).clamp(-448.0, 448.0)
        w[at // P, :, at % P] = quot.to(torch.float8_e4m3fn).view(torch.uint8)
        a = got.view(torch.float8_e4m3fn).float()
        b = w.view(torch.float8_e4m3fn).float()
        assert torch.equal(a.isnan(), b.isnan())
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
        # the format's definition in 64 bits: no code is nearer than the one taken (2^-24: the
        # quotient's own rounding)
        q64 = (x.double() / s.double()[None, :, None]).clamp(-448.0, 448.0)
        step = torch.exp2(torch.floor(torch.log2(q64.abs().clamp(min=2.0 ** -6))) - 3)
        off = (a[at // P, :, at % P].double() - q64).abs()
        fine = ~q64.isnan()
        assert (off[fine] <= (step / 2 + 2.0 ** -24 * q64.abs())[fine]).all()


# --------------------------------------------------- the operators together
@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_samples_of_one_prompt_end_to_end(fp8):
    """A prompt is appended, forked into samples, each sample grows by its own
    tokens, one is dropped, the pool is packed; every decode matches the
    oracle over the tokens that the model says each sequence holds."""
    Hq, Hkv, d, P = 16, 2, 64, 16
    gen = torch.Generator().manual_seed(7)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    p = Pair(64, P, 6, 12, layers=1, Hkv=Hkv, d=d, dtype=dtype)
    k_pool, v_pool = p.k[0], p.v[0]
    scale = [torch.full((Hkv,), 1 / 64.0), torch.full((Hkv,), 1 / 32.0)]
    scale_d = [s.cuda() for s in scale]
    held = {i: [] for i in range(6)}   # what each sequence holds: (k, v) rows of one token

    def codes(x, s):
        return (x.float() / s[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def grow(ids, new):
        n = sum(new)
        k, v = (torch.randn((n, Hkv, d), generator=gen).to(torch.bfloat16) for _ in range(2))
        slots = sa.sinkattn_pages_reserve(p.table, i32(ids), i32(np.cumsum([0] + new)), n, p.k, p.v)
        if fp8:
            sa.sinkattn_append_paged_fp8(k.cuda(), v.cuda(), slots, *scale_d, k_pool, v_pool)
            k, v = codes(k, scale[0]), codes(v, scale[1])
        else:
            sa.sinkattn_append_paged(k.cuda(), v.cuda(), slots, k_pool, v_pool)
        at = 0
        for i, m in zip(ids, new):
            held[i] = held[i] + [(k[t], v[t]) for t in range(at, at + m)]
            at += m

    def decode(ids, prefix):
        q = torch.randn((len(ids), Hq, d), generator=gen).to(torch.bfloat16)
        sinks = torch.randn(Hq, generator=gen)
        kv, ptr, idx = sa.sinkattn_pages_lists(p.table, i32(ids))
        own = max(len(held[i]) for i in ids) - prefix
        args = (kv, ptr, idx, i32([0, len(ids)]), i32([prefix]), sinks.cuda(), 1, prefix, own)
        if fp8:
            out, lse = sa.sinkattn_decode_shared_paged_fp8(q.cuda(), k_pool, v_pool, *scale_d, *args)
        else:
            out, lse = sa.sinkattn_decode_shared_paged(q.cuda(), k_pool, v_pool, *args)
        flat = [torch.cat([torch.stack([r[j] for r in held[i]], dim=1).reshape(-1, d) for i in ids])
                for j in range(2)]
        extra = dict(k_scale=scale[0], v_scale=scale[1]) if fp8 else {}
        o, l = oracle.attend(q, flat[0], flat[1], sinks,
                             torch.arange(len(ids) + 1, dtype=torch.int32), kv.cpu(), Hq, Hkv, d,
                             1 / math.sqrt(d), True, 0, **extra)
        # weights and output each off by half a bf16 step, values below 5
        assert np.abs(out.float().cpu().numpy().reshape(o.shape) - o).max() <= 2 * 5 * 2.0 ** -8
        assert np.abs(lse.cpu().numpy().reshape(l.shape) - l).max() <= 1e-4

    grow([0], [53])
    sa.sinkattn_pages_fork(p.table, i32([0, 0, 0]), i32([1, 2, 3]))
    for i in (1, 2, 3):
        held[i] = list(held[0])
    grow([0, 1, 2, 3], [1, 2, 3, 30])
    decode([0, 1, 2, 3], 48)
    sa.sinkattn_pages_truncate(p.table, i32([1]))
    held[1] = []
    grow([4], [20])
    grow([3, 0, 2], [1, 1, 1])
    decode([0, 2, 3], 48)
    sa.sinkattn_pages_compact(p.table, p.k, p.v)
    grow([0, 2, 3], [1, 1, 1])
    decode([3, 0, 2], 48)
    decode([4, 0], 0)
    assert sa.sinkattn_debug_status() == 0


# ---------------------------------------------------------------------- host
A = 0x1000


def reserve(**kw):
    a = dict(t=A, N=8, P=16, S=4, M=4, ids=A, cu=A, n=2, T=3, k=A, v=A, L=1, st=0, H=2, row=128,
             slots=A)
    a.update(kw)
    return sa.lib().sinkattn_pages_reserve(a["t"], a["N"], a["P"], a["S"], a["M"], a["ids"],
                                           a["cu"], a["n"], a["T"], a["k"], a["v"], a["L"], a["st"],
                                           a["H"], a["row"], a["slots"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=None), 1), (dict(t=A + 4), 1), (dict(N=0), 1), (dict(S=0), 1), (dict(M=0), 1),
    (dict(P=8), 2), (dict(P=48), 2), (dict(N=1 << 27), 2), (dict(M=1 << 27), 2),
    (dict(S=1 << 16, M=1 << 16), 2), (dict(ids=None), 1), (dict(n=-1), 1), (dict(n=5), 1),
    (dict(T=-1), 1), (dict(n=0, ids=None), 1), (dict(cu=None), 1), (dict(slots=None), 1),
    (dict(slots=A + 2), 1), (dict(k=None), 1), (dict(v=A + 8), 1), (dict(L=0), 1), (dict(H=0), 1),
    (dict(row=8), 1), (dict(row=136), 1), (dict(L=2, st=1000), 1), (dict(L=2, st=32776), 1),
    (dict(N=1 << 26, H=4), 2),
])
def test_reserve_rejects_bad_arguments(kw, status):
    assert reserve(**kw) == status
    assert sa.sinkattn_last_error() != ""


def test_calls_without_work_launch_nothing():
    assert reserve(n=0, T=0, ids=None) == 0
    assert reserve(T=0) == 0
    L = sa.lib()
    assert L.sinkattn_pages_fork(A, 8, 16, 4, 4, None, None, 0, None) == 0
    assert L.sinkattn_pages_truncate(A, 8, 16, 4, 4, None, None, 0, None) == 0
    assert L.sinkattn_pages_lists(A, 8, 16, 4, 4, None, 0, None, None, None, 0, None) == 0
    assert L.sinkattn_append_paged(None, None, 0, 0, None, 0, A, A, 8, 16, 2, 64, None) == 0


def test_other_table_calls_reject_bad_arguments():
    L = sa.lib()
    assert L.sinkattn_pages_init(None, 8, 16, 4, 4, None) == 1
    assert L.sinkattn_pages_fork(A, 8, 16, 4, 4, A, None, 2, None) == 1
    assert L.sinkattn_pages_fork(A, 8, 16, 4, 4, A, A, 5, None) == 1
    assert L.sinkattn_pages_truncate(A, 8, 16, 4, 4, A, A + 2, 2, None) == 1
    assert L.sinkattn_pages_truncate(A, 8, 17, 4, 4, A, A, 2, None) == 2
    assert L.sinkattn_pages_compact(A, 8, 16, 4, 4, A, A, 1, 0, 2, 128, None, None) == 1
    assert L.sinkattn_pages_compact(A, 8, 16, 4, 4, A, None, 1, 0, 2, 128, A, None) == 1
    assert L.sinkattn_pages_lists(A, 8, 16, 4, 4, A, 2, A, None, A, 8, None) == 1
    assert L.sinkattn_pages_lists(A, 8, 16, 4, 4, A, 2, A, A, A, -1, None) == 1
    with pytest.raises(sa.SinkAttnError):
        sa.sinkattn_pages_table_ints(0, 4, 4)


def test_table_ints():
    assert sa.sinkattn_pages_table_ints(100, 7, 9) == 16 + 7 * (1 + 9 + 7) + 4 * 100


def append(fp8=False, **kw):
    a = dict(k=A, v=A, ks=128, vs=128, slots=A, T=3, kp=A, vp=A, N=8, P=16, H=2, d=64, sk=A, sv=A)
    a.update(kw)
    L = sa.lib()
    if fp8:
        return L.sinkattn_append_paged_fp8(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["T"],
                                           a["sk"], a["sv"], a["kp"], a["vp"], a["N"], a["P"],
                                           a["H"], a["d"], None)
    return L.sinkattn_append_paged(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["T"], a["kp"],
                                   a["vp"], a["N"], a["P"], a["H"], a["d"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(k=A + 2), 1), (dict(v=A + 8), 1), (dict(ks=120), 1),
    (dict(vs=132), 1), (dict(slots=None), 1), (dict(slots=A + 2), 1), (dict(T=-1), 1),
    (dict(kp=None), 1), (dict(vp=A + 4), 1), (dict(N=0), 1), (dict(H=0), 1), (dict(d=32), 2),
    (dict(P=20), 2), (dict(N=1 << 27), 2),
])
def test_append_rejects_bad_arguments(kw, status):
    assert append(**kw) == status
    assert append(fp8=True, **kw) == status
    assert sa.sinkattn_last_error() != ""


def test_append_fp8_rejects_missing_scales():
    assert append(fp8=True, sk=None) == INVALID_ARG
    assert append(fp8=True, sv=A + 2) == INVALID_ARG
    assert UNSUPPORTED == 2


@gpu
def test_refuses_tensors_that_would_be_misread():
    p = Pair(8, 16, 4, 4)
    ids, cu = i32([0, 1]), i32([0, 1, 2])
    bad = [
        lambda: sa.sinkattn_pages_reserve(p.table, ids.long(), cu, 2, p.k, p.v),
        lambda: sa.sinkattn_pages_reserve(p.table, ids, cu[:-1], 2, p.k, p.v),
        lambda: sa.sinkattn_pages_reserve(p.table, ids, cu, 2, p.k[:, :-1], p.v[:, :-1]),
        lambda: sa.sinkattn_pages_reserve(p.table, ids, cu, 2, p.k, p.v[0]),
        lambda: sa.sinkattn_pages_reserve(p.table, ids, cu, 2, p.k.transpose(2, 3), p.v.transpose(2, 3)),
        lambda: sa.sinkattn_pages_reserve(p.table, ids, cu, 2, p.k, p.v, slots=i32([0])),
        lambda: sa.sinkattn_pages_fork(p.table, ids, ids[:1]),
        lambda: sa.sinkattn_pages_truncate(p.table, ids.cpu()),
        lambda: sa.sinkattn_pages_truncate(p.table, ids, cu),
        lambda: sa.sinkattn_pages_compact(p.table, p.k, p.v, page_map=ids),
        lambda: sa.sinkattn_pages_lists(p.table, ids, kv_indptr=ids),
        lambda: sa.PageTable(p.table.state[:-1], 8, 16, 4, 4),
        lambda: sa.PageTable(p.table.state.long(), 8, 16, 4, 4),
    ]
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    bad += [
        lambda: sa.sinkattn_append_paged(x.float(), x, ids, p.k[0], p.v[0]),
        lambda: sa.sinkattn_append_paged(x[:1], x, ids, p.k[0], p.v[0]),
        lambda: sa.sinkattn_append_paged(x.transpose(0, 1), x, ids, p.k[0], p.v[0]),
        lambda: sa.sinkattn_append_paged(x, x, ids.long(), p.k[0], p.v[0]),
        lambda: sa.sinkattn_append_paged(x, x, ids, p.k, p.v),
        lambda: sa.sinkattn_append_paged_fp8(x, x, ids, ids, ids, p.k[0], p.v[0]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(sa.SinkAttnError) as e:
            f()
            pytest.fail("call %d was taken" % i)
        assert e.value.status == INVALID_ARG
    p.check()


@gpu
def test_pools_past_32_bit_offsets():
    """Pools of more than 2^31 elements (2^32 bytes): appends, copies on write, the attention
    and moves at their far end."""
    N, P, Hkv, d = 40000, 64, 8, 128
    k = torch.zeros((N, Hkv, P, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    table = sa.PageTable(None, N, P, 4, N)
    sa.sinkattn_pages_reserve(table, i32([0]), i32([0, (N - 4) * P]), (N - 4) * P, k, v)
    gen = torch.Generator(device="cuda").manual_seed(1)
    new = [torch.randn((100, Hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
           for _ in range(2)]
    slots = sa.sinkattn_pages_reserve(table, i32([1]), i32([0, 100]), 100, k, v)
    assert slots.min().item() == (N - 4) * P
    sa.sinkattn_append_paged(*new, slots, k, v)
    sa.sinkattn_pages_truncate(table, i32([0]))
    sa.sinkattn_pages_fork(table, i32([1]), i32([2]))
    more = [torch.randn((2, Hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
            for _ in range(2)]
    # both write behind the shared 100 tokens: the second gets a copy of the last page
    slots = sa.sinkattn_pages_reserve(table, i32([1, 2]), i32([0, 1, 2]), 2, k, v)
    sa.sinkattn_append_paged(*more, slots, k, v)

    q = torch.randn((2, 16, d), generator=gen, device="cuda").to(torch.bfloat16)

    def look(share):
        kv, ptr, pages = sa.sinkattn_pages_lists(table, i32([1, 2]), page_indices=i32([0] * 8))
        return sa.sinkattn_decode_shared_paged(
            q, k, v, kv, ptr, pages, i32([0, 2]), i32([P]), None, 1, P, P, prefix_splits=share)

    def want(i):
        x, y = (torch.cat([a, b[i:i + 1]]).double().transpose(0, 1) for a, b in zip(new, more))
        l = torch.einsum("hgd,hjd->hgj", q[i].double().view(Hkv, 2, d), x) / math.sqrt(d)
        return torch.einsum("hgj,hjd->hgd", l.softmax(-1), y).reshape(16, d), l.logsumexp(-1).reshape(16)

    def held():
        for share in (1, 0):
            out, lse = look(share)
            for i in range(2):
                o, l = want(i)
                # weights to bf16, then the output: half a step each, relative to |v| <= 6
                assert (out[i].double() - o).abs().max().item() <= 2 * 2.0 ** -8 * 6
                assert (lse[i].double() - l).abs().max().item() <= 1e-4

    held()
    page_map = sa.sinkattn_pages_compact(table, k, v)
    assert table.page_list[1:3, :2].max().item() == 2 and table.free_count.item() == N - 3
    assert (page_map >= 0).sum().item() == 3
    held()
    assert sa.sinkattn_debug_status() == 0


def codes_of(x, scale):
    """The e4m3 codes of x / scale, by torch: [tokens, Hkv, d] under one scale per head."""
    quot = (x.float() / scale[None, :, None]).clamp(-448.0, 448.0)
    return quot.to(torch.float8_e4m3fn).view(torch.uint8)


def appended(x, scale):
    """The codes that the append writes for x, in the order of x."""
    tokens, Hkv, d = x.shape
    pools = [torch.full((-(-tokens // 16), Hkv, 16, d), 0x55, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    slots = torch.arange(tokens, dtype=torch.int32, device="cuda")
    sa.sinkattn_append_paged_fp8(x, x, slots, scale, scale, *pools)
    got = [p.transpose(1, 2).reshape(-1, Hkv, d)[:tokens] for p in pools]
    assert torch.equal(*got)
    return got[0]


@gpu
@pytest.mark.parametrize("scale", [1.0, 0.7, -0.7, 2.0 ** -99, 2.0 ** -110])
def test_append_fp8_keeps_the_sign_of_a_zero(scale):
    x = torch.tensor([0.0, -0.0] * 32, device="cuda").to(torch.bfloat16).view(1, 1, 64)
    s = torch.tensor([scale], device="cuda")
    want = codes_of(x, s)
    assert sorted(set(want.reshape(-1).tolist())) == [0x00, 0x80]
    assert torch.equal(appended(x, s), want)


@gpu
@pytest.mark.parametrize("bits", [-127, -104, -101, -100, -99, -97, -95, -93, -92, -91, -90, -89, -60,
                                  0, 60, 99, 100, 101, 110])
def test_append_fp8_codes_under_scales_of_any_size(bits):
    """Bit for bit the codes of the fp32 quotient, ties and their neighbours among them: x / s next
    to the borders between codes for scales of every mantissa end, where the residual step would be
    one bit short of exact. (s = (2 - 2^-23) 2^-97, x = 2^-106: the quotient is one step above the
    border 2^-10, so its code is 1 and not 0.)"""
    gen = torch.Generator().manual_seed(abs(bits))
    ends = torch.tensor([1.0, 1.0 + 2.0 ** -23, 2.0 - 2.0 ** -23, 2.0 - 2.0 ** -22, 1.5, 1.0 / 0.7])
    s = torch.cat([ends, 1.0 + torch.rand(10, generator=gen)]).double() * 2.0 ** bits
    s = s.float()
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    border = torch.cat([(codes[1:] + codes[:-1]) / 2, codes])[:252]
    x = (border[:, None] * s.double()[None, :]).to(torch.bfloat16)          # [252, 16 heads]
    x = torch.stack([x, -x, x * 1.0078125, x * 0.99609375], dim=-1).to(torch.bfloat16)
    two = torch.exp2(torch.arange(-11, 4).double() + bits).to(torch.bfloat16)   # powers of two at s
    x = torch.cat([x, two.view(15, 1, 1).expand(15, 16, 4)])                   # [267, 16, 4]
    x = x.repeat_interleave(16, dim=-1).contiguous().cuda()
    s = s.cuda()
    got, want = appended(x, s), codes_of(x, s)
    nan = (want & 0x7f) == 0x7f
    assert torch.equal((got & 0x7f) == 0x7f, nan)
    assert torch.equal(got[~nan], want[~nan])


@gpu
def test_lists_of_no_sequences_write_their_zeros():
    p = Pair(8, 16, 4, 4)
    kv, ptr, idx = i32([9]), i32([9]), i32([9, 9])
    got = sa.sinkattn_pages_lists(p.table, i32([]), kv_indptr=kv, page_indptr=ptr, page_indices=idx)
    assert got[0] is kv and kv.tolist() == [0] and ptr.tolist() == [0] and idx.tolist() == [9, 9]
    kv, ptr, idx = sa.sinkattn_pages_lists(p.table, i32([]))
    assert kv.tolist() == [0] and ptr.tolist() == [0] and idx.numel() == 0
    L, none = sa.lib(), i32([9])
    args = p.table._args
    assert L.sinkattn_pages_lists(*args, None, 0, none.data_ptr(), None, None, 0, None) == 0
    torch.cuda.synchronize()
    assert none.tolist() == [0]
    p.check()


def test_lists_of_more_sequences_than_a_table_can_have_are_refused():
    """(Each sequence's block sums the lengths before its own: 2^31 ids would keep a GPU for days.)"""
    for n in ((1 << 18) + 1, 2 ** 31 - 1):
        assert sa.lib().sinkattn_pages_lists(A, 8, 16, 4, 4, A, n, A, A, A, 8, None) == UNSUPPORTED
        assert "2^18" in sa.sinkattn_last_error()


def test_sizes_beyond_32_bits_are_refused():
    """(As 32-bit arguments they would be other sizes: 2^32 + 8 pages would be 8.)"""
    for call in (lambda: sa.sinkattn_pages_table_ints(2 ** 32 + 8, 4, 4),
                 lambda: sa.sinkattn_pages_table_ints(8, 4, -2 ** 31 - 1),
                 lambda: sa.PageTable(None, 2 ** 32 + 8, 16, 4, 4),
                 lambda: sa.PageTable(None, 8, 2 ** 32 + 16, 4, 4)):
        with pytest.raises(sa.SinkAttnError) as e:
            call()
        assert e.value.status == INVALID_ARG and "32-bit" in str(e.value)


@gpu
def test_a_reserve_of_2_to_the_32_tokens_is_refused():
    p = Pair(8, 16, 4, 4)
    with pytest.raises(sa.SinkAttnError) as e:
        sa.sinkattn_pages_reserve(p.table, i32([0]), i32([0, 0]), 2 ** 32, p.k, p.v)
    assert e.value.status == INVALID_ARG
    p.check()


@gpu
def test_a_table_of_the_most_sequences():
    """2^18 sequences of one table in every call, one token each at first."""
    S, N = 1 << 18, (1 << 18) + 8
    table = sa.PageTable(None, N, 16, S, 4)
    k, v = (torch.zeros((N, 1, 16, 8), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.arange(S, dtype=torch.int32, device="cuda")
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    low, high = ids[:S // 2], ids[S // 2:]
    assert torch.equal(sa.sinkattn_pages_reserve(table, ids, cu, S, k, v), 16 * ids)
    kv, ptr, pages = sa.sinkattn_pages_lists(table, ids)
    assert torch.equal(kv, cu) and torch.equal(ptr, cu) and torch.equal(pages[:S], ids)
    sa.sinkattn_pages_truncate(table, high)
    assert table.free_count.item() == S // 2 + 8
    sa.sinkattn_pages_fork(table, low, high)
    assert (table.refcount[:S // 2] == 2).all() and torch.equal(table.page_list[S // 2:, 0], low)
    # every holder writes: the first keeps its page, the other takes a copy
    slots = sa.sinkattn_pages_reserve(table, ids, cu, S, k, v)
    assert torch.equal(slots[:S // 2], 16 * low + 1) and (slots[S // 2:] % 16 == 1).all()
    assert table.free_count.item() == 8 and (table.seq_lens == 2).all()
    sa.sinkattn_pages_truncate(table, ids)
    assert table.free_count.item() == N and (table.page_list == -1).all()
    assert torch.equal(table.free_list.sort().values, torch.arange(N, dtype=torch.int32, device="cuda"))
