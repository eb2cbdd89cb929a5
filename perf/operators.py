"""Cases, plain forms and work of the paged-cache operators: decode over a
cache whose sequences share prefixes, appending to the pages, forking,
truncating and compacting the page table.

Layouts. Page pools: [num_pages, Hkv, page, d] (one layer) or [layers,
num_pages, Hkv, page, d], bf16 or uint8 e4m3 codes. Page table: one int32
buffer, in this order: a header of 16 words (word 0: the number of free
pages), seq_lens [max_seqs], page_list [max_seqs, max_pages] (-1 where
unused), refcount [num_pages], free_list [num_pages], and the library's
scratch. The j-th page that a call takes is free_list[count - 1 - j]; the
j-th of K pages that it gives back goes to free_list[count + K - 1 - j].
"""
import math
import random
import zlib

import numpy as np
import torch

own = False

HEADER = 16
DEV = "cuda"

# gpt-oss-shaped (64 query / 8 KV heads, d 64, pages of 16) and Qwen3-shaped
# (64 / 4, d 128, pages of 64) attention: this repository's own workloads.
GPTOSS = dict(hq=64, hkv=8, d=64, page=16)
QWEN = dict(hq=64, hkv=4, d=128, page=64)


def listed():
    return [
        # four samples of one short prompt: the smallest decode, latency counts
        dict(name="shared_samples_b4", op="shared", fp8=False, batch=4, q_len=1, groups=1,
             prefix=1024, suffix_lo=1, suffix_hi=40, window=0, **GPTOSS),
        # a serving batch behind one long system prompt
        dict(name="shared_prompt_b64", op="shared", fp8=False, batch=64, q_len=1, groups=1,
             prefix=8192, suffix_lo=17, suffix_hi=1024, window=0, **GPTOSS),
        # speculative decode, three drafts, one prompt for the whole batch
        dict(name="shared_mtp_b256", op="shared", fp8=False, batch=256, q_len=3, groups=1,
             prefix=4032, suffix_lo=3, suffix_hi=1000, window=0, **QWEN),
        # several prompts of other lengths at once (one of them empty), e4m3 cache
        dict(name="shared_fp8_groups_b96", op="shared", fp8=True, batch=96, q_len=1, groups=5,
             prefix=8192, suffix_lo=1, suffix_hi=700, window=0, **GPTOSS),
        # one decode step's cache update: a token for each of 64 sequences
        dict(name="append_decode_b64", op="append", fp8=False, n=64, len_lo=1024, len_hi=8192,
             new_lo=1, new_hi=1, **GPTOSS),
        # chunks of eight prompts written to an e4m3 cache
        dict(name="append_prompt_fp8", op="append", fp8=True, n=8, len_lo=0, len_hi=4000,
             new_lo=1500, new_hi=4000, **QWEN),
        # four samples of one prompt start: the tail page is copied for three of them
        dict(name="fork_samples", op="fork", parents=1, children=3, len_lo=1000, len_hi=1100,
             layers=1, **GPTOSS),
        # eight samples of each of 16 prompts, all layers of a four-layer slice
        dict(name="fork_batch", op="fork", parents=16, children=8, len_lo=4000, len_hi=8000,
             layers=4, **QWEN),
        # rejected drafts of a batch are rolled back
        dict(name="truncate_drafts_b256", op="truncate", n=256, held=256, len_lo=4000,
             len_hi=8000, drop_lo=0, drop_hi=3, **QWEN),
        # half of the sequences have finished and are freed, prompts shared by eight stay
        dict(name="free_half_b512", op="truncate", n=256, held=512, len_lo=1024, len_hi=8192,
             drop_lo=8192, drop_hi=8192, **GPTOSS),
        # a small pool is packed after a few sequences left it
        dict(name="compact_small", op="compact", held=8, len_lo=100, len_hi=900, spare=0.5,
             layers=1, **GPTOSS),
        # a four-layer slice of a large pool, half of it free
        dict(name="compact_pool", op="compact", held=48, len_lo=4000, len_hi=8000, spare=1.0,
             layers=4, **QWEN),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "append", "fork", "truncate", "compact"])
    hq, hkv, d = rng.choice([(64, 8, 64), (64, 4, 128), (32, 8, 128), (16, 1, 64), (24, 8, 64)])
    shape = dict(hq=hq, hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]))
    if op == "shared":
        fp8 = rng.random() < 0.4
        batch, q_len = _log(rng, 2, 200), rng.choice([1, 1, 2, 3, 4])
        lo = rng.choice([q_len, _log(rng, q_len, 300)])
        return dict(op=op, fp8=fp8, batch=batch, q_len=q_len, groups=rng.randint(1, min(6, batch)),
                    prefix=_log(rng, 128, 4000), suffix_lo=lo, suffix_hi=lo + _log(rng, 1, 600),
                    window=rng.choice([0, 0, 0, 128]), **shape)
    if op == "append":
        lo = rng.choice([1, 1, 2, 3, _log(rng, 4, 1000)])
        return dict(op=op, fp8=rng.random() < 0.5, n=_log(rng, 1, 64), len_lo=rng.choice([0, 500]),
                    len_hi=_log(rng, 501, 4000), new_lo=lo, new_hi=lo + rng.choice([0, lo // 2]),
                    **shape)
    if op == "fork":
        lo = _log(rng, 1, 4000)
        return dict(op=op, parents=_log(rng, 1, 16), children=rng.randint(1, 8), len_lo=lo,
                    len_hi=lo + _log(rng, 1, 1000), layers=rng.randint(1, 4), **shape)
    if op == "truncate":
        held, lo = _log(rng, 2, 512), _log(rng, 1, 4000)
        drop = rng.choice([3, 40, 8192])
        return dict(op=op, n=rng.randint(1, held), held=held, len_lo=lo,
                    len_hi=lo + _log(rng, 1, 2000), drop_lo=rng.choice([0, drop]), drop_hi=drop,
                    **shape)
    lo = _log(rng, 1, 2000)
    return dict(op=op, held=_log(rng, 2, 48), len_lo=lo, len_hi=lo + _log(rng, 1, 2000),
                spare=round(rng.uniform(0.05, 1.2), 2), layers=rng.randint(1, 4), **shape)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _plan(case, seed):
    """The sequences of a case: host lists of lengths, groups and pages."""
    rng = random.Random(seed * 1000003 + 17)
    P, op = case["page"], case["op"]
    if op == "shared":
        B, ng, q = case["batch"], case["groups"], case["q_len"]
        cuts = sorted(rng.sample(range(1, B), ng - 1)) if ng > 1 else []
        group = [0] + cuts + [B]
        top = max(1, case["prefix"] // P)
        # one group has the stated prefix; with several, one has none at all
        pages = [top] + [rng.randint(1, top) for _ in range(ng - 1)]
        if ng > 2:
            pages[rng.randint(1, ng - 1)] = 0
        suffix = [rng.randint(max(q, case["suffix_lo"]), max(q, case["suffix_hi"])) for _ in range(B)]
        prefix = [p * P for p in pages]
        gid = [g for g in range(ng) for _ in range(group[g], group[g + 1])]
        return dict(group=group, prefix=prefix, lens=[prefix[gid[b]] + suffix[b] for b in range(B)],
                    share=[pages[gid[b]] for b in range(B)], gid=gid, suffix=suffix, rng=rng)
    # the lengths go by the case alone, so that a pool and the outputs have one size for all seeds
    sizes = random.Random(zlib.crc32(repr(sorted((k, case[k]) for k in case if k != "name")).encode()))
    held = case.get("held") or case.get("n") or case["parents"]
    lens = [sizes.randint(case["len_lo"], case["len_hi"]) for _ in range(held)]
    if op in ("truncate", "compact"):   # every eight sequences share half of the shortest prompt
        gid = [b // 8 for b in range(held)]
        half = [min(lens[g * 8:g * 8 + 8]) // 2 // P for g in range((held + 7) // 8)]
        share = [half[g] for g in gid]
    else:
        gid, share = list(range(held)), [0] * held
    return dict(lens=lens, gid=gid, share=share, rng=rng, sizes=sizes)


def _pages(plan, P, num_pages=None):
    """Page lists (random page ids) of the plan's sequences, and a permutation of the free ids."""
    rng = plan["rng"]
    need, first = 0, {}
    for b, L in enumerate(plan["lens"]):
        g, s = plan["gid"][b], plan["share"][b]
        need += -(-L // P) - s
        if s and g not in first:
            first[g] = None
            need += s
    total = need if num_pages is None else num_pages(need)
    ids = list(range(total))
    rng.shuffle(ids)
    at, lists, shared = 0, [], {}
    for b, L in enumerate(plan["lens"]):
        g, s, n = plan["gid"][b], plan["share"][b], -(-L // P)
        if g not in shared:
            shared[g] = ids[at:at + s]
            at += s
        lists.append(shared[g] + ids[at:at + n - s])
        at += n - s
    return lists, ids[at:], total


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def _pool(case, layers, num_pages, gen):
    shape = (layers, num_pages, case["hkv"], case["page"], case["d"])
    out = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        x.normal_(generator=gen)
        if case.get("fp8"):
            # codes of N(0, 1) values under a scale that maps about 5 to the largest code
            x = torch.cat([(x[:, i:i + 256].float() * (448.0 / 5.0)).clamp(-448.0, 448.0)
                           .to(torch.float8_e4m3fn).view(torch.uint8)
                           for i in range(0, num_pages, 256)], dim=1)
        out.append(x if case.get("layers", 1) > 1 or case["op"] in ("fork", "compact") else x[0])
    return out


def _scales(case, gen):
    return [(0.8 + 0.4 * torch.rand(case["hkv"], generator=gen, device=DEV)) * (5.0 / 448.0)
            for _ in range(2)]


def _table(lists, lens, free, num_pages, max_seqs, max_pages):
    """A page table's buffer; the library's scratch behind the lists is left as it is found."""
    t = np.zeros(16 + max_seqs * (8 + max_pages) + num_pages * 4, dtype=np.int32)
    lens_at, list_at = HEADER, HEADER + max_seqs
    rc_at = list_at + max_seqs * max_pages
    fl_at = rc_at + num_pages
    t[0] = len(free)
    t[lens_at:lens_at + len(lens)] = lens
    t[list_at:rc_at] = -1
    for s, pages in enumerate(lists):
        t[list_at + s * max_pages:list_at + s * max_pages + len(pages)] = pages
        np.add.at(t, rc_at + np.asarray(pages, dtype=np.int64), 1)
    t[fl_at:fl_at + len(free)] = free
    return torch.from_numpy(t).to(DEV), fl_at + num_pages


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, P = case["op"], case["page"]
    plan = _plan(case, seed)
    rng = plan["rng"]
    if op == "shared":
        lists, _, total = _pages(plan, P, lambda need: need + 3)
        B, q_len = case["batch"], case["q_len"]
        k, v = _pool(case, 1, total, gen)
        s = dict(k_pages=k, v_pages=v,
                 kv_indptr=_i32(np.concatenate([[0], np.cumsum(plan["lens"])])),
                 page_indptr=_i32(np.concatenate([[0], np.cumsum([len(x) for x in lists])])),
                 page_indices=_i32([p for x in lists for p in x]),
                 group_indptr=_i32(plan["group"]), prefix_lens=_i32(plan["prefix"]),
                 q_len=q_len, max_prefix=max(plan["prefix"]), max_suffix=max(plan["suffix"]),
                 max_kv=max(plan["lens"]), window=case["window"])
        s["q"] = torch.empty((B * q_len, case["hq"], case["d"]), dtype=torch.bfloat16,
                             device=DEV).normal_(generator=gen)
        s["sinks"] = torch.rand(case["hq"], generator=gen, device=DEV) * 4.0 - 2.0
        if case["fp8"]:
            s["k_scale"], s["v_scale"] = _scales(case, gen)
        return dict(case, **s)
    if op == "append":
        n = case["n"]
        new = [plan["sizes"].randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        top = case["len_hi"] + case["new_hi"]
        extra = sum(-(-x // P) + 1 for x in new) + 5
        lists, free, total = _pages(plan, P, lambda need: need + extra)
        max_pages = -(-top // P) + -(-case["new_hi"] // P) + 2
        table, used = _table(lists, plan["lens"], free, total, n + 3, max_pages)
        ids = list(range(n))
        rng.shuffle(ids)
        k, v = _pool(case, 1, total, gen)
        T = sum(new)
        # K and V are slices of one fused projection's rows [q | k | v]
        width = (case["hq"] + 2 * case["hkv"]) * case["d"]
        qkv = torch.empty((T, width), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        k_new = qkv[:, case["hq"] * case["d"]:(case["hq"] + case["hkv"]) * case["d"]]
        v_new = qkv[:, (case["hq"] + case["hkv"]) * case["d"]:]
        s = dict(k_pages=k, v_pages=v, k_new=k_new.view(T, case["hkv"], case["d"]),
                 v_new=v_new.view(T, case["hkv"], case["d"]),
                 cu_new=_i32(np.concatenate([[0], np.cumsum(new)])), total_new=T,
                 kv_indptr=torch.zeros(n + 1, dtype=torch.int32, device=DEV),
                 page_indptr=torch.zeros(n + 1, dtype=torch.int32, device=DEV),
                 page_indices=torch.zeros(n * max_pages, dtype=torch.int32, device=DEV))
        if case["fp8"]:
            s["k_scale"], s["v_scale"] = _scales(case, gen)
    elif op == "fork":
        par, ch = case["parents"], case["children"]
        n = par * (ch + 1)
        lists, free, total = _pages(plan, P, lambda need: need + 2 * n + 5)
        max_pages = -(-case["len_hi"] // P) + 4
        table, used = _table(lists, plan["lens"], free, total, n + 2, max_pages)
        dst = list(range(par, n))
        ids = list(range(n))
        rng.shuffle(dst)
        rng.shuffle(ids)
        k, v = _pool(case, case["layers"], total, gen)
        s = dict(k_pages=k, v_pages=v, src=_i32([i % par for i in range(par * ch)]), dst=_i32(dst),
                 cu_new=_i32(range(n + 1)), total_new=n)
    elif op == "truncate":
        held = case["held"]
        lists, free, total = _pages(plan, P, lambda need: need + need // 10 + 5)
        max_pages = -(-case["len_hi"] // P) + 1
        table, used = _table(lists, plan["lens"], free, total, held, max_pages)
        ids = rng.sample(range(held), case["n"])
        new = [max(0, plan["lens"][i] - rng.randint(case["drop_lo"], case["drop_hi"])) for i in ids]
        s = dict(new_lens=_i32(new))
    else:
        held = case["held"]
        lists, free, total = _pages(plan, P, lambda need: int(need * (1 + case["spare"])) + 1)
        max_pages = -(-case["len_hi"] // P) + 1
        table, used = _table(lists, plan["lens"], free, total, held, max_pages)
        ids = [0]
        k, v = _pool(case, case["layers"], total, gen)
        s = dict(k_pages=k, v_pages=v)
    max_seqs = {"append": case.get("n", 0) + 3, "fork": len(plan["lens"]) * (case.get("children", 0) + 1) + 2}.get(
        op, case.get("held", 0))
    return dict(case, table=table, table0=table[:used].clone(), used=used, num_pages=total,
                max_seqs=max_seqs, max_pages=max_pages, ids=_i32(ids), **s)


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _views(s):
    a = HEADER + s["max_seqs"]
    b = a + s["max_seqs"] * s["max_pages"]
    c = b + s["num_pages"]
    t = s["table"]
    return dict(free_count=t[0:1], seq_lens=t[HEADER:a],
                page_list=t[a:b].view(s["max_seqs"], s["max_pages"]), refcount=t[b:c],
                free_list=t[c:c + s["num_pages"]])


def _plain_shared(s):
    q, P, G = s["q"], s["page"], s["hq"] // s["hkv"]
    hkv, d, ql = s["hkv"], s["d"], s["q_len"]
    lens = (s["kv_indptr"][1:] - s["kv_indptr"][:-1]).long()
    B = lens.numel()
    npg = -(-s["max_kv"] // P)
    have = (s["page_indptr"][1:] - s["page_indptr"][:-1]).long()
    e = torch.minimum(torch.arange(npg, device=q.device)[None, :], have[:, None] - 1)
    pages = s["page_indices"][s["page_indptr"][:-1].long()[:, None] + e].long()

    def keys(pool, scale):
        if s["fp8"]:
            x = pool[pages].view(torch.float8_e4m3fn).float() * scale[None, None, :, None, None]
        else:
            x = pool[pages].float()
        return x.permute(0, 2, 1, 3, 4).reshape(B, hkv, npg * P, d)

    k = keys(s["k_pages"], s.get("k_scale"))
    qf = q.float().view(B, ql, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, ql * G, d)
    l = torch.matmul(qf, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    del k
    pos = lens[:, None] - ql + torch.arange(ql, device=q.device)[None, :]
    j = torch.arange(npg * P, device=q.device)
    seen = j[None, None, :] <= pos[:, :, None]
    if s["window"] > 0:
        seen &= j[None, None, :] > pos[:, :, None] - s["window"]
    l.view(B, hkv, ql, G, -1).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    sink = s["sinks"].view(hkv, 1, G).expand(hkv, ql, G).reshape(1, hkv, ql * G)
    m = torch.maximum(l.amax(-1), sink)
    l.sub_(m[..., None]).exp_()
    den = l.sum(-1) + torch.exp(sink - m)
    v = keys(s["v_pages"], s.get("v_scale"))
    o = torch.matmul(l, v) / den[..., None]
    o = o.view(B, hkv, ql, G, d).permute(0, 2, 1, 3, 4).reshape(B * ql, s["hq"], d)
    lse = (m + den.log()).view(B, hkv, ql, G).permute(0, 2, 1, 3).reshape(B * ql, s["hq"])
    return o.to(torch.bfloat16), lse


def _plain_reserve(s, t):
    """Room for cu_new's tokens at the ends of the sequences `ids`; the slot of each token."""
    P, N = s["page"], s["num_pages"]
    dev = s["table"].device
    ids, cu = s["ids"].long(), s["cu_new"].long()
    n = ids.numel()
    new, L = cu[1:] - cu[:-1], t["seq_lens"][ids].long()
    have, want = (L + P - 1) // P, (L + new + P - 1) // P
    tail = t["page_list"][ids, (have - 1).clamp(min=0)].long().clamp(min=0)
    i = torch.arange(n, device=dev)
    shared = (L % P > 0) & (new > 0) & (t["refcount"][tail] > 1)
    writers = torch.zeros(N, dtype=torch.int32, device=dev).scatter_add_(0, tail, shared.int())
    first = torch.full((N,), n, device=dev).scatter_reduce_(
        0, tail, torch.where(shared, i, n), "amin")
    # the last holder of a page writes in place: the first writer, if every holder writes
    cow = shared & ~((writers[tail] == t["refcount"][tail]) & (first[tail] == i))
    need = want - have + cow
    off = need.cumsum(0) - need
    c = t["free_count"].long()
    dst = t["free_list"][(c - 1 - off).clamp(min=0)].long()
    # a copied page takes the rows in use
    pick = cow.nonzero().view(-1)
    frm, to = tail[pick], dst[pick]
    take = (torch.arange(P, device=dev)[None, :] < (L % P)[pick, None])[:, None, :, None]
    for pool in (s["k_pages"], s["v_pages"]):
        p5 = pool if pool.dim() == 5 else pool[None]
        p5[:, to] = torch.where(take, p5[:, frm], p5[:, to])
    most = s.get("new_hi", 1)   # new tokens of a sequence
    j = torch.arange(-(-most // P) + 1, device=dev)[None, :]
    valid = j < (want - have)[:, None]
    page = t["free_list"][(c - 1 - (off + cow)[:, None] - j).clamp(min=0)].long()
    t["refcount"].scatter_add_(0, tail, -cow.int())
    t["refcount"].scatter_add_(0, dst, cow.int())
    t["refcount"].scatter_add_(0, page.view(-1), valid.int().view(-1))
    at = t["page_list"][ids[:, None], have[:, None] + j]
    t["page_list"][ids[:, None], have[:, None] + j] = torch.where(valid, page.int(), at)
    at = t["page_list"][ids, (have - 1).clamp(min=0)]
    t["page_list"][ids, (have - 1).clamp(min=0)] = torch.where(cow, dst.int(), at)
    t["seq_lens"][ids] = (L + new).int()
    t["free_count"].sub_(need.sum().int())
    tok = torch.arange(s["total_new"], device=dev)
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = L[b] + tok - cu[b]
    return (t["page_list"][ids[b], pos // P].long() * P + pos % P).int()


def _plain_append(s, t):
    slots = _plain_reserve(s, t)
    P, ids = s["page"], s["ids"].long()
    at = slots.long()
    for pool, new, scale in ((s["k_pages"], s["k_new"], s.get("k_scale")),
                             (s["v_pages"], s["v_new"], s.get("v_scale"))):
        if s["fp8"]:
            x = (new.float() / scale[None, :, None]).clamp(-448.0, 448.0)
            new = x.to(torch.float8_e4m3fn).view(torch.uint8)
        pool[at // P, :, at % P] = new
    lens = t["seq_lens"][ids]
    have = (lens + P - 1) // P
    s["kv_indptr"][1:] = lens.cumsum(0)
    s["page_indptr"][1:] = have.cumsum(0)
    e = torch.arange(s["max_pages"], device=lens.device)[None, :]
    # entries past a list's end write its own last page once more
    e = torch.minimum(e, have[:, None].long() - 1).clamp(min=0)
    to = s["page_indptr"][:-1].long()[:, None] + e
    s["page_indices"][to.view(-1)] = t["page_list"][ids[:, None], e].view(-1)
    return slots


def _plain_fork(s, t):
    src, dst = s["src"].long(), s["dst"].long()
    pages = t["page_list"][src]
    t["page_list"][dst] = pages
    t["seq_lens"][dst] = t["seq_lens"][src]
    t["refcount"].scatter_add_(0, pages.clamp(min=0).long().view(-1), (pages >= 0).int().view(-1))
    return _plain_reserve(s, t)


def _plain_truncate(s, t):
    P, N, M = s["page"], s["num_pages"], s["max_pages"]
    ids, new = s["ids"].long(), s["new_lens"].long()
    dev = new.device
    L = t["seq_lens"][ids].long()
    e = torch.arange(M, device=dev)[None, :]
    drop = (e >= ((new + P - 1) // P)[:, None]) & (e < ((L + P - 1) // P)[:, None])
    pages = t["page_list"][ids]
    p = pages.long().clamp(min=0).view(-1)
    t["refcount"].scatter_add_(0, p, -drop.int().view(-1))
    pos = torch.arange(p.numel(), device=dev)
    gone = drop.view(-1)
    first = torch.full((N,), p.numel(), device=dev).scatter_reduce_(
        0, p, torch.where(gone, pos, p.numel()), "amin")
    push = gone & (t["refcount"][p] == 0) & (first[p] == pos)
    K, rank = push.sum(), push.cumsum(0) - 1
    room = torch.cat([t["free_list"], t["free_list"][:1]])
    room.scatter_(0, torch.where(push, t["free_count"].long() + K - 1 - rank, N), p.int())
    t["free_list"].copy_(room[:N])
    t["free_count"].add_(K.int())
    t["page_list"][ids] = torch.where(drop, -1, pages)
    t["seq_lens"][ids] = new.int()


def _plain_compact(s, t):
    N = s["num_pages"]
    rc = t["refcount"].clone()
    ar = torch.arange(N, device=rc.device)
    live = rc > 0
    kept = live.sum()
    hole, mover = ~live & (ar < kept), live & (ar >= kept)
    to, frm = hole.nonzero().view(-1), mover.nonzero().view(-1)
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, to] = pool[:, frm]
    page_map = torch.where(live, ar, -1)
    page_map[frm] = to
    t["refcount"].zero_()
    t["refcount"][page_map[live]] = rc[live]
    pages = t["page_list"]
    t["page_list"].copy_(torch.where(pages >= 0, page_map[pages.long().clamp(min=0)].int(), -1))
    t["free_list"].copy_(torch.where(ar < N - kept, (N - 1 - ar).int(), t["free_list"]))
    t["free_count"].copy_((N - kept).int().view(1))
    return page_map.int()


# ----------------------------------------------------------------------------
def _values(s, pool):
    return pool.view(torch.float8_e4m3fn) if s.get("fp8") else pool


def run(s):
    op = s["op"]
    if own:
        import gqa_attention_softmax_gb300 as sa
    if op == "shared":
        if own and s["fp8"]:
            out, lse = sa.sinkattn_decode_shared_paged_fp8(
                s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["kv_indptr"],
                s["page_indptr"], s["page_indices"], s["group_indptr"], s["prefix_lens"],
                s["sinks"], s["q_len"], s["max_prefix"], s["max_suffix"], window=s["window"])
        elif own:
            out, lse = sa.sinkattn_decode_shared_paged(
                s["q"], s["k_pages"], s["v_pages"], s["kv_indptr"], s["page_indptr"],
                s["page_indices"], s["group_indptr"], s["prefix_lens"], s["sinks"], s["q_len"],
                s["max_prefix"], s["max_suffix"], window=s["window"])
        else:
            out, lse = _plain_shared(s)
        return {"out": out, "lse": lse}
    # the table's operators work in place: each pass starts from the table that was prepared
    # (the pages that a pass writes are free in it, or get the same values again)
    s["table"][:s["used"]].copy_(s["table0"])
    res = {}
    if own:
        table = sa.PageTable(s["table"], s["num_pages"], s["page"], s["max_seqs"], s["max_pages"])
        if op == "append":
            slots = sa.sinkattn_pages_reserve(table, s["ids"], s["cu_new"], s["total_new"],
                                              s["k_pages"], s["v_pages"])
            if s["fp8"]:
                sa.sinkattn_append_paged_fp8(s["k_new"], s["v_new"], slots, s["k_scale"],
                                             s["v_scale"], s["k_pages"], s["v_pages"])
            else:
                sa.sinkattn_append_paged(s["k_new"], s["v_new"], slots, s["k_pages"], s["v_pages"])
            sa.sinkattn_pages_lists(table, s["ids"], s["kv_indptr"], s["page_indptr"],
                                    s["page_indices"])
            res["slots"] = slots
        elif op == "fork":
            sa.sinkattn_pages_fork(table, s["src"], s["dst"])
            res["slots"] = sa.sinkattn_pages_reserve(table, s["ids"], s["cu_new"], s["total_new"],
                                                     s["k_pages"], s["v_pages"])
        elif op == "truncate":
            sa.sinkattn_pages_truncate(table, s["ids"], s["new_lens"])
        else:
            res["page_map"] = sa.sinkattn_pages_compact(table, s["k_pages"], s["v_pages"])
    else:
        t = _views(s)
        if op == "append":
            res["slots"] = _plain_append(s, t)
        elif op == "fork":
            res["slots"] = _plain_fork(s, t)
        elif op == "truncate":
            _plain_truncate(s, t)
        else:
            res["page_map"] = _plain_compact(s, t)
    # the whole table without the library's scratch
    res["table"] = s["table"][HEADER:s["used"]]
    res["free_count"] = s["table"][0:1]
    if op == "append":
        res.update(kv_indptr=s["kv_indptr"], page_indptr=s["page_indptr"],
                   page_indices=s["page_indices"])
    if "k_pages" in s:
        res.update(k_pages=_values(s, s["k_pages"]), v_pages=_values(s, s["v_pages"]))
    return res


# ----------------------------------------------------------------------------
def work(case):
    """Bytes and operations of one pass, for lengths at the middle of their ranges."""
    P, d, hkv, hq, op = case["page"], case["d"], case["hkv"], case["hq"], case["op"]
    el = 1 if case.get("fp8") else 2
    row = 2 * hkv * d * el   # K and V of one token
    if op == "shared":
        B, q, ng = case["batch"], case["q_len"], case["groups"]
        suffix = (case["suffix_lo"] + case["suffix_hi"]) / 2
        first = case["prefix"] // P * P
        # the first group has the whole prefix, the others about half of it, one of them none
        mean = first if ng == 1 else first * (1 + 0.5 * (ng - 1 - (ng > 2))) / ng
        keys, seen = mean * ng + B * suffix, mean + suffix
        if case["window"]:
            seen = min(seen, case["window"])
            keys = min(keys, B * seen)
        io = B * q * hq * (2 * d * 2 + 4) + B * (mean + suffix) / P * 4
        return {"bytes": keys * row + io, "flops": 4.0 * B * q * hq * seen * d}
    mid = (case["len_lo"] + case["len_hi"]) / 2
    if op == "append":
        T = case["n"] * (case["new_lo"] + case["new_hi"]) / 2
        lists = case["n"] * (mid / P + 4) * 4 * 2
        return {"bytes": T * (2 * hkv * d * 2 + row + 4) + lists + T / P * 12, "flops": 0.0}
    if op == "fork":
        n = case["parents"] * case["children"]
        half = (P - 1) / 2
        return {"bytes": n * (mid / P) * 12 + case["layers"] * n * half * row * 2 + n * 32, "flops": 0.0}
    if op == "truncate":
        drop = min(mid, (case["drop_lo"] + case["drop_hi"]) / 2)
        return {"bytes": case["n"] * (16 + drop / P * 16), "flops": 0.0}
    # live pages of the sequences (of eight that share a prompt, half of it is held once)
    live = case["held"] * mid / P * (1 - 0.5 * 7 / 8)
    total = live * (1 + case["spare"])
    moved = (total - live) * live / total   # live pages above the kept ones, spread evenly
    return {"bytes": moved * P * row * case["layers"] * 2 + total * 16 + live * 16, "flops": 0.0}


def exact(case, seed):
    s = prepare(case, seed)
    op, P = case["op"], case["page"]
    if op == "append" and case["fp8"]:
        # the nearest e4m3 value of x / scale, to even at ties, from the format's definition
        s0 = dict(s)
        slots = _plain_reserve(dict(s0), _views(s0)).long().cpu()
        found = {}
        for name, new, scale in (("k_pages", s["k_new"], s["k_scale"]),
                                 ("v_pages", s["v_new"], s["v_scale"])):
            pool = s[name].view(torch.float8_e4m3fn).double().cpu()
            x = new.double().cpu() / scale.double().cpu()[None, :, None]
            x = x.clamp(-448.0, 448.0)
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            pool[slots // P, :, slots % P] = torch.round(x / step) * step
            found[name] = pool
        return found
    if op != "shared":
        return None
    G, ql, d = case["hq"] // case["hkv"], case["q_len"], case["d"]
    lens = (s["kv_indptr"][1:] - s["kv_indptr"][:-1]).tolist()
    ptr = s["page_indptr"].tolist()
    outs, lses = [], []
    for b, L in enumerate(lens):
        pages = s["page_indices"][ptr[b]:ptr[b + 1]].long()

        def rows(name, scale):
            x = s[name][pages]
            x = x.view(torch.float8_e4m3fn).double() if case["fp8"] else x.double()
            x = x.transpose(0, 1).reshape(case["hkv"], -1, d)[:, :L]
            return x * s[scale].double()[:, None, None] if case["fp8"] else x

        k, v = rows("k_pages", "k_scale"), rows("v_pages", "v_scale")
        q = s["q"][b * ql:(b + 1) * ql].double()                     # [ql, Hq, d]
        q = q.view(ql, case["hkv"], G, d).transpose(0, 1).reshape(case["hkv"], ql * G, d)
        l = (q @ k.transpose(1, 2)) / math.sqrt(d)
        pos = (L - ql + torch.arange(ql, device=DEV)).repeat_interleave(G)
        j = torch.arange(L, device=DEV)
        hidden = j[None, :] > pos[:, None]
        if case["window"]:
            hidden |= j[None, :] <= pos[:, None] - case["window"]
        l = l.masked_fill(hidden[None], -math.inf)
        sink = s["sinks"].double().view(case["hkv"], 1, G).expand(-1, ql, -1).reshape(case["hkv"], ql * G, 1)
        every = torch.cat([l, sink], dim=2)
        lse = torch.logsumexp(every, dim=2)
        o = torch.exp(l - lse[..., None]) @ v
        outs.append(o.view(case["hkv"], ql, G, d).transpose(0, 1).reshape(ql, case["hq"], d))
        lses.append(lse.view(case["hkv"], ql, G).transpose(0, 1).reshape(ql, case["hq"]))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
