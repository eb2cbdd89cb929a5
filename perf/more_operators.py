"""Cases, plain forms and work of the operators around the attention: the norm
and position rotation of queries and keys (forward, backward, and on the way
into a paged cache), and the attention's backward pass.

Layouts. A fused projection's rows are [q | k | v], [tokens, (Hq + 2 Hkv) d]
bf16. The attention reads q [tokens, Hq, d] and k, v as ragged HND: sequence b
is the block [Hkv, L_b, d] at row Hkv cu[b] of [Hkv tokens, d]. Page pools are
[num_pages, Hkv, page, d], bf16 or uint8 e4m3 codes; a slot is page * page size
+ position in the page, -1 for a padded row.

The attention's gradients are taken as functions of what the forward pass left:
out (bf16) and lse (fp32) are inputs.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"

# gpt-oss-shaped (64 query / 8 KV heads, d 64, YaRN) and Qwen3-shaped (64 / 4, d 128, norms of
# queries and keys) attention: this repository's own workloads.
GPTOSS = dict(hq=64, hkv=8, d=64)
QWEN = dict(hq=64, hkv=4, d=128)
YARN = dict(rotary=64, base=150000.0, scaling="yarn", factor=32.0, original=4096,
            interleaved=False, norm=False)
PLAIN = dict(rotary=128, base=1000000.0, scaling="none", factor=1.0, original=0,
             interleaved=False, norm=True)


def listed():
    return [
        # one short prompt of a small model: the smallest call, latency counts
        dict(name="back_tiny", op="attn_back", q_lens="16", k_lens="128", hq=4, hkv=1, d=64,
             causal=True, window=0, sinks=True),
        # a packed batch of odd lengths, continued prompts (more keys than queries) and an empty one
        dict(name="back_ragged", op="attn_back", q_lens="333 1 0 77 640 129 255 901",
             k_lens="333 513 40 205 640 1029 255 901", hq=24, hkv=8, d=64, causal=True,
             window=0, sinks=True),
        # full causal attention of a training batch, sinks
        dict(name="back_gptoss", op="attn_back", q_lens="4096 3000 2048 1024",
             k_lens="4096 3000 2048 1024", causal=True, window=0, sinks=True, **GPTOSS),
        # the same batch in a layer with a sliding window of 128 keys
        dict(name="back_gptoss_w128", op="attn_back", q_lens="4096 3000 2048 1024",
             k_lens="4096 3000 2048 1024", causal=True, window=128, sinks=True, **GPTOSS),
        # long prompts with 16 query heads for each KV head
        dict(name="back_qwen", op="attn_back", q_lens="6000 6000", k_lens="6000 6000",
             causal=True, window=0, sinks=True, **QWEN),
        # a short prompt's projection on its way to the attention: latency counts
        dict(name="rope_prompt_37", op="rope", lens="37", first=0, **GPTOSS, **YARN),
        # a batch of long prompts, norms of queries and keys in the same pass
        dict(name="rope_qwen_norm", op="rope", lens="6000 6000", first=0, **QWEN, **PLAIN),
        # the gradients of the same two kinds of layers
        dict(name="rope_back_gptoss", op="rope_back", lens="4096 3000 2048 1024", first=0,
             **GPTOSS, **YARN),
        dict(name="rope_back_qwen_norm", op="rope_back", lens="6000 6000", first=0, **QWEN, **PLAIN),
        # one decode step of 64 sequences, four rows of the batch are padding
        dict(name="append_decode_b64", op="append", tokens=64, pad=4, each=1, far=8192, fp8=False,
             page=16, **GPTOSS, **YARN),
        # three drafts of 256 sequences far into long contexts
        dict(name="append_mtp_b256", op="append", tokens=768, pad=0, each=3, far=131072, fp8=False,
             page=64, **QWEN, **PLAIN),
        # chunks of eight prompts written to an e4m3 cache
        dict(name="append_prompt_fp8", op="append", tokens=21800, pad=0, each=2725, far=4000,
             fp8=True, page=64, **QWEN, **PLAIN),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(lens):
    return " ".join(str(n) for n in lens)


def _lens(case, name):
    """The lengths of a case's sequences, which it holds as text."""
    return [int(n) for n in case[name].split()]


def draw(rng):
    op = rng.choice(["attn_back", "attn_back", "attn_back", "rope", "rope_back", "append"])
    hq, hkv, d = rng.choice([(64, 8, 64), (64, 4, 128), (32, 8, 128), (16, 1, 64), (24, 8, 64),
                             (4, 4, 128)])
    case = dict(op=op, hq=hq, hkv=hkv, d=d)
    if op == "attn_back":
        q_lens, k_lens = [], []
        batch = _log(rng, 1, 8)
        top = min(2500, 10000 // batch)
        for _ in range(batch):
            n = rng.choice([0, 1, _log(rng, 1, top), _log(rng, 1, top), _log(rng, 1, top)])
            q_lens.append(n)
            k_lens.append(n + rng.choice([0, 0, 0, _log(rng, 1, 1000)]))
        if sum(q_lens) == 0:
            q_lens[0] += 3
            k_lens[0] += 3
        causal = rng.random() < 0.85
        window = rng.choice([0, 0, 0, 128, _log(rng, 1, 1000)]) if causal else 0
        return dict(case, q_lens=_text(q_lens), k_lens=_text(k_lens), causal=causal, window=window,
                    sinks=rng.random() < 0.7)
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "yarn"])
    case.update(rotary=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                base=rng.choice([10000.0, 150000.0, 1000000.0]), scaling=scaling,
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 32.0]),
                original=rng.choice([2048, 4096]), interleaved=rng.random() < 0.4,
                norm=rng.random() < 0.5)
    if op == "append":
        each = rng.choice([1, 1, 2, 3, _log(rng, 4, 1000)])
        n = _log(rng, 1, max(2, 8000 // each))
        return dict(case, tokens=n * each, pad=rng.choice([0, rng.randint(0, min(9, n))]),
                    each=each, far=_log(rng, 2000, 1000000), fp8=rng.random() < 0.5,
                    page=rng.choice([16, 32, 64, 128]))
    return dict(case, lens=_text(_log(rng, 1, 2400) for _ in range(_log(rng, 1, 5))),
                first=rng.choice([0, 0, _log(rng, 1, 1000000)]))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def _cu(lens):
    return _i32(np.concatenate([[0], np.cumsum(lens)]))


def _frequencies(case):
    """Angle per position of each pair (float64), and the factor of cos and sin."""
    r, base, kind, f = case["rotary"], case["base"], case["scaling"], case["factor"]
    i = np.arange(r // 2, dtype=np.float64)
    if kind == "ntk":
        # the base grows so that the lowest frequency shrinks by the factor
        base = base * f ** (r / (r - 2)) if r > 2 else base
    inv = base ** (-2.0 * i / r)
    if kind == "linear":
        return inv / f, 1.0
    if kind == "yarn":
        # pairs that turn fewer than beta times within the original length: low .. high
        def border(beta):
            return r * math.log(case["original"] / (beta * 2.0 * math.pi)) / (2.0 * math.log(base))
        low, high = max(border(32.0), 0.0), min(border(1.0), r - 1.0)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        return inv / f * ramp + inv * (1.0 - ramp), 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _normal(gen, *shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    if op == "attn_back":
        q_lens, k_lens = _lens(case, "q_lens"), _lens(case, "k_lens")
        tq, tk = sum(q_lens), sum(k_lens)
        s = dict(case, q_lens=q_lens, k_lens=k_lens, q=_normal(gen, tq, hq, d), k=_normal(gen, hkv * tk, d),
                 v=_normal(gen, hkv * tk, d), dout=_normal(gen, tq, hq, d),
                 sinks_t=(torch.rand(hq, generator=gen, device=DEV) * 4.0 - 2.0
                          if case["sinks"] else None),
                 cu_q=_cu(q_lens), cu_k=_cu(k_lens), max_q=max(q_lens), max_k=max(k_lens))
        s["out"], s["lse"] = _forward(s)
        return s
    rng = random.Random(seed * 1000003 + 17)
    width = (hq + 2 * hkv) * d
    inv, factor = _frequencies(case)
    s = dict(case, inv=torch.from_numpy(inv).to(DEV), attention_factor=factor)
    if own:
        import gqa_attention_softmax_gb300 as sa
        s["rope"] = sa.Rope(case["rotary"], base=case["base"], interleaved=case["interleaved"],
                            scaling=case["scaling"], factor=case["factor"],
                            original_len=case["original"])
    if op != "append":
        s["lens"] = _lens(case, "lens")
    tokens = case["tokens"] if op == "append" else sum(s["lens"])
    rows = _normal(gen, tokens, width)
    s["q"] = rows[:, :hq * d].view(tokens, hq, d)
    s["k"] = rows[:, hq * d:(hq + hkv) * d].view(tokens, hkv, d)
    s["v"] = rows[:, (hq + hkv) * d:].view(tokens, hkv, d)
    s["q_weight"] = s["k_weight"] = None
    if case["norm"]:
        s["q_weight"], s["k_weight"] = [
            1.0 + 0.2 * torch.randn(d, generator=gen, device=DEV) for _ in range(2)]
    if op == "append":
        runs, page = tokens // case["each"], case["page"]
        starts = [rng.randint(0, case["far"]) for _ in range(runs)]
        s["positions"] = _i32([p + i for p in starts for i in range(case["each"])])
        # as a page table gives them: runs of slots inside pages that lie anywhere in the pool
        per = case["each"] // page + 2
        pages = list(range(runs * per + 3))
        rng.shuffle(pages)
        slots = []
        for b, p in enumerate(starts):
            at = p % page
            slots += [pages[b * per + (at + i) // page] * page + (at + i) % page
                      for i in range(case["each"])]
        if case["pad"]:
            slots[-case["pad"]:] = [-1] * case["pad"]
        s["slots"] = _i32(slots)
        shape = (len(pages), hkv, page, d)
        dtype = torch.uint8 if case["fp8"] else torch.bfloat16
        s["k_pages"], s["v_pages"] = [torch.zeros(shape, dtype=dtype, device=DEV) for _ in range(2)]
        if case["fp8"]:
            s["k_scale"], s["v_scale"] = [
                (0.8 + 0.4 * torch.rand(hkv, generator=gen, device=DEV)) * (5.0 / 448.0)
                for _ in range(2)]
        return s
    s["cu"] = _cu(s["lens"])
    s["positions"] = None
    if case["first"]:
        s["positions"] = _i32([case["first"] + i for n in s["lens"] for i in range(n)])
    if op == "rope_back":
        s["dq"] = _normal(gen, tokens, hq, d)
        s["dk"], s["dv"] = [_normal(gen, hkv * tokens, d) for _ in range(2)]
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _blocks(s):
    """(rows of q, rows of k, Lq, Lk, KV heads taken at once) of each sequence."""
    at_q = at_k = 0
    for lq, lk in zip(s["q_lens"], s["k_lens"]):
        at = max(1, min(s["hkv"], 2 ** 30 // max(1, lq * lk * (s["hq"] // s["hkv"]))))
        yield at_q, at_k, lq, lk, at
        at_q, at_k = at_q + lq, at_k + lk


def _hidden(s, lq, lk):
    if not s["causal"]:
        return None
    pos = lk - lq + torch.arange(lq, device=DEV)
    j = torch.arange(lk, device=DEV)
    hide = j[None, :] > pos[:, None]
    if s["window"] > 0:
        hide |= j[None, :] <= pos[:, None] - s["window"]
    return hide


def _forward(s):
    """The attention's out and lse, which the backward pass takes."""
    hq, hkv, d, G = s["hq"], s["hkv"], s["d"], s["hq"] // s["hkv"]
    out, lse = torch.zeros_like(s["q"]), torch.zeros(s["q"].shape[:2], device=DEV)
    for a, b, lq, lk, step in _blocks(s):
        if lq == 0:
            continue
        hide = _hidden(s, lq, lk)
        for h in range(0, hkv, step):
            n = min(step, hkv - h)
            q = s["q"][a:a + lq, h * G:(h + n) * G].float().permute(1, 0, 2).reshape(n, G, lq, d)
            rows = slice(hkv * b + h * lk, hkv * b + (h + n) * lk)
            k, v = [s[x][rows].float().view(n, 1, lk, d) for x in ("k", "v")]
            l = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
            if hide is not None:
                l.masked_fill_(hide, -math.inf)
            m = l.amax(-1, keepdim=True)
            if s["sinks"]:
                sink = s["sinks_t"][h * G:(h + n) * G].view(n, G, 1, 1)
                m = torch.maximum(m, sink)
            l.sub_(m).exp_()
            den = l.sum(-1, keepdim=True)
            if s["sinks"]:
                den = den + torch.exp(sink - m)
            o = torch.matmul(l, v) / den
            out[a:a + lq, h * G:(h + n) * G] = o.reshape(n * G, lq, d).permute(1, 0, 2).bfloat16()
            lse[a:a + lq, h * G:(h + n) * G] = (m + den.log()).reshape(n * G, lq).t()
    return out, lse


def _plain_attn_back(s):
    hq, hkv, d, G = s["hq"], s["hkv"], s["d"], s["hq"] // s["hkv"]
    scale = 1.0 / math.sqrt(d)
    dq = torch.zeros_like(s["q"])
    dk, dv = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    delta = (s["dout"].float() * s["out"].float()).sum(-1)
    for a, b, lq, lk, step in _blocks(s):
        if lq == 0:
            continue
        hide = _hidden(s, lq, lk)
        for h in range(0, hkv, step):
            n = min(step, hkv - h)
            rows = slice(hkv * b + h * lk, hkv * b + (h + n) * lk)
            heads = slice(h * G, (h + n) * G)

            def q_rows(x):
                return x[a:a + lq, heads].float().transpose(0, 1).reshape(n, G, lq, -1)

            q, do = q_rows(s["q"]), q_rows(s["dout"])
            k, v = [s[x][rows].float().view(n, 1, lk, d) for x in ("k", "v")]
            p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
            p.sub_(q_rows(s["lse"][..., None])).exp_()
            if hide is not None:
                p.masked_fill_(hide, 0.0)
            dv[rows] = torch.matmul(p.transpose(-1, -2), do).sum(1).reshape(n * lk, d).bfloat16()
            ds = torch.matmul(do, v.transpose(-1, -2)).sub_(q_rows(delta[..., None])).mul_(p)
            del p
            got = torch.matmul(ds, k).mul_(scale).reshape(n * G, lq, d)
            dq[a:a + lq, heads] = got.transpose(0, 1).bfloat16()
            got = torch.matmul(ds.transpose(-1, -2), q).sum(1).mul_(scale)
            dk[rows] = got.reshape(n * lk, d).bfloat16()
    res = {"dq": dq, "dk": dk, "dv": dv}
    if s["sinks"]:
        res["dsinks"] = -(torch.exp(s["sinks_t"] - s["lse"]) * delta).sum(0)
    return res


def _places(s):
    """Each token's position, and the ragged HND rows [tokens, Hkv] of its heads."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    i, n = t - cu[b], cu[b + 1] - cu[b]
    h = torch.arange(s["hkv"], device=DEV)
    rows = (s["hkv"] * cu[b] + i)[:, None] + h[None, :] * n[:, None]
    return (i if s["positions"] is None else s["positions"].long()), rows


def _pairs(s, x):
    """The two members of each rotated pair, and the rest of the head."""
    r = s["rotary"]
    if s["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _unpair(s, a, b, rest):
    if s["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _cos_sin(s, positions):
    angle = positions.double()[:, None] * s["inv"][None, :]   # far positions: 64 bits
    return [(f(angle) * s["attention_factor"]).float()[:, None, :] for f in (torch.cos, torch.sin)]


EPS = 1e-6


def _rotated(s, x, weight, cos, sin):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    a, b, rest = _pairs(s, x)
    return _unpair(s, a * cos - b * sin, b * cos + a * sin, rest)


def _plain_rope(s):
    positions, rows = _places(s)
    cos, sin = _cos_sin(s, positions)
    q = _rotated(s, s["q"], s["q_weight"], cos, sin).bfloat16()
    k, v = [torch.empty((rows.numel(), s["d"]), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    k[rows] = _rotated(s, s["k"], s["k_weight"], cos, sin).bfloat16()
    v[rows] = s["v"]
    return {"q": q, "k": k, "v": v}


def _plain_rope_back(s):
    positions, rows = _places(s)
    cos, sin = _cos_sin(s, positions)
    res = {}
    for name, g, x, w in (("q", s["dq"], s["q"], s["q_weight"]),
                          ("k", s["dk"][rows], s["k"], s["k_weight"])):
        a, b, rest = _pairs(s, g.float())
        g = _unpair(s, a * cos + b * sin, b * cos - a * sin, rest)
        if w is not None:
            x = x.float()
            inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            xh = x * inv
            res["d%s_weight" % name] = (g * xh).sum((0, 1))
            u = g * w
            g = inv * (u - xh * (u * xh).mean(-1, keepdim=True))
        res["d" + name] = g.bfloat16()
    res["dv"] = s["dv"][rows]
    return res


def _plain_append(s):
    cos, sin = _cos_sin(s, s["positions"])
    q = _rotated(s, s["q"], s["q_weight"], cos, sin).bfloat16()
    at = s["slots"].long()
    keep = s["slots"].shape[0] - s["pad"]   # padded rows are the last ones
    at, P = at[:keep], s["page"]
    for pool, x, scale in (("k_pages", _rotated(s, s["k"], s["k_weight"], cos, sin), "k_scale"),
                           ("v_pages", s["v"].float(), "v_scale")):
        if s["fp8"]:
            x = (x / s[scale][None, :, None]).clamp(-448.0, 448.0)
            x = x.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = x.bfloat16()
        s[pool][at // P, :, at % P] = x[:keep]
    return q


# ----------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        import gqa_attention_softmax_gb300 as sa
        norm = {} if s.get("q_weight") is None else dict(q_weight=s["q_weight"],
                                                         k_weight=s["k_weight"], eps=EPS)
    if op == "attn_back":
        if not own:
            return _plain_attn_back(s)
        dq, dk, dv, dsinks = sa.sinkattn_prefill_backward(
            s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["sinks_t"], s["cu_q"],
            s["cu_k"], s["max_q"], s["max_k"], s["hkv"], causal=s["causal"], window=s["window"])
        res = {"dq": dq, "dk": dk, "dv": dv}
        if s["sinks"]:
            res["dsinks"] = dsinks
        return res
    if op == "rope":
        if not own:
            return _plain_rope(s)
        q, k, v = sa.sinkattn_rope_qkv(s["q"], s["k"], s["v"], s["cu"], s["rope"],
                                       positions=s["positions"], **norm)
        return {"q": q, "k": k, "v": v}
    if op == "rope_back":
        if not own:
            return _plain_rope_back(s)
        dq, dk, dv, dqw, dkw = sa.sinkattn_rope_qkv_backward(
            s["dq"], s["dk"], s["dv"], s["cu"], s["rope"], q=s["q"], k=s["k"],
            positions=s["positions"], **norm)
        res = {"dq": dq, "dk": dk, "dv": dv}
        if s["norm"]:
            res.update(dq_weight=dqw, dk_weight=dkw)
        return res
    if not own:
        q = _plain_append(s)
    elif s["fp8"]:
        q = sa.sinkattn_rope_append_paged_fp8(
            s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], s["k_scale"],
            s["v_scale"], s["k_pages"], s["v_pages"], **norm)
    else:
        q = sa.sinkattn_rope_append_paged(s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                          s["rope"], s["k_pages"], s["v_pages"], **norm)
    res = {"q": q}
    for name in ("k_pages", "v_pages"):
        res[name] = s[name].view(torch.float8_e4m3fn) if s["fp8"] else s[name]
    return res


def _seen(lq, lk, causal, window):
    """Visible (query, key) pairs of one sequence and head."""
    if not causal:
        return lq * lk
    if window <= 0:
        window = lk
    # query i sees min(window, lk - lq + i + 1) keys
    full = max(0, min(lq, lk + 1 - window))           # queries that see `window` keys
    rest = lq - full
    return full * window + rest * (lk - lq) + rest * (rest + 1) // 2


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "attn_back":
        q_lens, k_lens = _lens(case, "q_lens"), _lens(case, "k_lens")
        tq, tk = sum(q_lens), sum(k_lens)
        pairs = sum(_seen(lq, lk, case["causal"], case["window"])
                    for lq, lk in zip(q_lens, k_lens))
        # q, out, dout in and dq out; k, v in and dk, dv out; lse
        return {"bytes": 8.0 * tq * hq * d + 8.0 * tk * hkv * d + 4.0 * tq * hq,
                "flops": 10.0 * pairs * hq * d}
    tokens = case["tokens"] if case["op"] == "append" else sum(_lens(case, "lens"))
    if case["op"] == "append":
        kept = tokens - case["pad"]
        el = 1 if case["fp8"] else 2
        return {"bytes": tokens * (hq * d * 4.0 + 8) + kept * 2 * hkv * d * (2.0 + el), "flops": 0.0}
    total = tokens * (hq + 2 * hkv) * d * 4.0 + (tokens * 4.0 if case["first"] else 0.0)
    if case["op"] == "rope_back" and case["norm"]:
        total += tokens * (hq + hkv) * d * 2.0   # the inputs of the norms
    return {"bytes": total, "flops": 0.0}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_attn_back(s):
    hq, hkv, d, G = s["hq"], s["hkv"], s["d"], s["hq"] // s["hkv"]
    c = d ** -0.5
    q, do, o, lse = [s[x].double() for x in ("q", "dout", "out", "lse")]
    dq = torch.zeros_like(q)
    dk, dv = [torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
    delta = torch.einsum("thd,thd->th", do, o)
    at_q = at_k = 0
    for lq, lk in zip(s["q_lens"], s["k_lens"]):
        for h in range(hkv):
            at = hkv * at_k + h * lk
            k, v = s["k"][at:at + lk].double(), s["v"][at:at + lk].double()
            # blocks of queries, over the keys that some query of the block sees
            for i0 in range(0, lq, 1024):
                i1 = min(i0 + 1024, lq)
                j0, j1 = 0, lk
                if s["causal"]:
                    j1 = lk - lq + i1
                    if s["window"] > 0:
                        j0 = max(0, lk - lq + i0 - s["window"] + 1)
                i = torch.arange(i0, i1, device=DEV)[:, None] + (lk - lq)
                j = torch.arange(j0, j1, device=DEV)[None, :]
                see = torch.ones((i1 - i0, j1 - j0), dtype=torch.bool, device=DEV)
                if s["causal"]:
                    see = j <= i
                    if s["window"] > 0:
                        see = see & (i - j < s["window"])
                t = slice(at_q + i0, at_q + i1)
                for g in range(h * G, h * G + G):
                    w = torch.where(see, torch.exp(c * (q[t, g] @ k[j0:j1].T) - lse[t, g, None]), 0.0)
                    e = w * (do[t, g] @ v[j0:j1].T - delta[t, g, None])
                    dq[t, g] = c * (e @ k[j0:j1])
                    dk[at + j0:at + j1] += c * (e.T @ q[t, g])
                    dv[at + j0:at + j1] += w.T @ do[t, g]
        at_q, at_k = at_q + lq, at_k + lk
    res = {"dq": dq, "dk": dk, "dv": dv}
    if s["sinks"]:
        res["dsinks"] = -(torch.exp(s["sinks_t"].double()[None] - lse) * delta).sum(0)
    return res


def _matrix_rotation(s, x, positions, back=False):
    """x [tokens, heads, d] in 64 bits, each pair as a complex number times e^{i angle}."""
    r = s["rotary"]
    first = torch.arange(0, r, 2) if s["interleaved"] else torch.arange(r // 2)
    second = first + (1 if s["interleaved"] else r // 2)
    first, second = first.to(DEV), second.to(DEV)
    turns = positions.double()[:, None] * s["inv"][None, :]
    turn = torch.polar(torch.full_like(turns, s["attention_factor"]), -turns if back else turns)
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_layout(s):
    pos, rows = [], []
    for b, n in enumerate(s["lens"]):
        at = sum(s["lens"][:b])
        for_heads = [torch.arange(n) + s["hkv"] * at + h * n for h in range(s["hkv"])]
        rows.append(torch.stack(for_heads, 1))
        pos.append(torch.arange(n) + s["first"])
    return torch.cat(pos).to(DEV), torch.cat(rows).to(DEV)


def _exact_norm(x, w):
    x = x.double()
    if w is None:
        return x
    return w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn_back":
        return _exact_attn_back(s)
    if op == "append":
        pos = s["positions"].long()
        q = _matrix_rotation(s, _exact_norm(s["q"], s["q_weight"]), pos)
        k = _matrix_rotation(s, _exact_norm(s["k"], s["k_weight"]), pos)
        res = {"q": q}
        n = case["tokens"] - case["pad"]
        at = s["slots"][:n].long()
        for name, x, scale in (("k_pages", k, "k_scale"), ("v_pages", s["v"].double(), "v_scale")):
            pool = torch.zeros(s[name].shape, dtype=torch.float64, device=DEV)
            if case["fp8"]:
                # the nearest e4m3 value, to even at ties, from the format's definition
                x = (x / s[scale].double()[None, :, None]).clamp(-448.0, 448.0)
                step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
                x = torch.round(x / step) * step
            pool[at // case["page"], :, at % case["page"]] = x[:n]
            res[name] = pool
        return res
    pos, rows = _exact_layout(s)
    if op == "rope":
        res = {"q": _matrix_rotation(s, _exact_norm(s["q"], s["q_weight"]), pos)}
        for name, x in (("k", _matrix_rotation(s, _exact_norm(s["k"], s["k_weight"]), pos)),
                        ("v", s["v"].double())):
            res[name] = torch.empty((rows.numel(), case["d"]), dtype=torch.float64, device=DEV)
            res[name][rows] = x
        return res
    res = {}
    for name, g, x, w in (("dq", s["dq"], s["q"], s["q_weight"]),
                          ("dk", s["dk"][rows], s["k"], s["k_weight"])):
        g = _matrix_rotation(s, g.double(), pos, back=True)
        if w is not None:
            x, w = x.double(), w.double()
            rms = torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS)
            dw = (g * x / rms).sum(1).sum(0)
            g = g * w / rms - x * (g * w * x).sum(-1, keepdim=True) / (case["d"] * rms ** 3)
        res[name] = g
        if w is not None:
            res[name + "_weight"] = dw
    res["dv"] = s["dv"][rows].double()
    return res
