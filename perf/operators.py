"""What is measured of the paged cache and of the attention over a shared prefix.

A paged cache holds K and V in pools [num_pages, kv_heads, page_tokens, head_dim].  A sequence
is a row of page ids (-1 behind its last page) and a length; a page may belong to several
sequences and is free when no row names it.  New pages are always the lowest free ones, in the
order of the call's list.  Four kinds of cases:

  attend  exact attention of nq queries per head and sequence; the first prefix tokens are the
          pages of one sequence, common to the whole batch, the others each sequence's own
  beam    a step of a beam search or of parallel sampling: the losing sequences are freed, their
          slots fork from the winners, and every fork appends its next tokens
  prompt  sequences are freed, get their prompts' rows appended, and are gathered into the dense
          [n, kv_heads, capacity, head_dim] cache that a tree is built over
  move    a saved table is restored, sequences are copied, the originals freed, and the pool is
          compacted
"""
from __future__ import annotations

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # three short chats on one short instruction, fp32: the smallest call, all latency
        _attend("attend_tiny_f32", F32, F32, 3, 2, 1, 64, 16, 64, 1, 40, 1, False),
        # sixteen samples of an fp32 model on a shared context that fills no whole tile
        _attend("attend_ragged_f32", F32, F32, 16, 8, 2, 128, 16, 1008, 1, 700, 1, False),
        # a batch of unrelated sequences, nothing shared, odd batch and lengths
        _attend("attend_own_bf16", BF16, BF16, 33, 32, 8, 128, 32, 0, 1, 4000, 1, False),
        # four draft tokens per sequence verified at once over a 32K document, fp32 outputs
        _attend("attend_verify_32k", BF16, F32, 8, 32, 8, 128, 64, 32768, 4, 500, 4, True),
        # 64 answers on one 128K document
        _attend("attend_share_128k", BF16, BF16, 64, 32, 8, 128, 64, 131072, 1, 1000, 1, False),
        # 16 answers on a 1M-token cache with 64 query heads
        _attend("attend_share_1m", BF16, BF16, 16, 64, 8, 128, 64, 1048576, 1, 300, 1, False),
        # a beam step of a small model, pages of 8 tokens
        _beam("beam_small_f32", F32, 2, 64, 8, 3, 5, 70, 90, 1),
        # 63 samples forked from one 128K document; each adds a token
        _beam("beam_fork_128k", BF16, 8, 128, 16, 1, 63, 131065, 131065, 1),
        # ragged prompts into pages and from there into a tree's dense cache
        _prompt("prompt_ragged", BF16, 8, 128, 32, 9, 1, 8000, 8192),
        # a few short fp32 prompts
        _prompt("prompt_short_f32", F32, 1, 64, 16, 4, 3, 250, 256),
        # four 32K sequences move to the bottom of a 128K-token pool
        _move("move_32k", BF16, 8, 128, 64, 4, 30000, 32768),
        # many short sequences in small pages
        _move("move_short", BF16, 2, 64, 8, 40, 1, 900),
    ]


def _attend(name, kv, out, batch, q_heads, kv_heads, d, page, prefix, lo, hi, nq, causal):
    c = dict(kind="attend", kv=kv, out=out, batch=batch, q_heads=q_heads, kv_heads=kv_heads, d=d, page=page,
             prefix=prefix, lo=lo, hi=hi, nq=nq, causal=causal)
    return dict(c, name=name) if name else c


def _beam(name, kv, kv_heads, d, page, parents, children, lo, hi, new):
    c = dict(kind="beam", kv=kv, kv_heads=kv_heads, d=d, page=page, parents=parents, children=children, lo=lo,
             hi=hi, new=new)
    return dict(c, name=name) if name else c


def _prompt(name, kv, kv_heads, d, page, n, lo, hi, capacity):
    c = dict(kind="prompt", kv=kv, kv_heads=kv_heads, d=d, page=page, n=n, lo=lo, hi=hi, capacity=capacity)
    return dict(c, name=name) if name else c


def _move(name, kv, kv_heads, d, page, n, lo, hi):
    c = dict(kind="move", kv=kv, kv_heads=kv_heads, d=d, page=page, n=n, lo=lo, hi=hi)
    return dict(c, name=name) if name else c


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["attend", "attend", "attend", "beam", "prompt", "move"])
    kv = rng.choice([BF16, BF16, F32])
    d, page = rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    if kind == "attend":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
        nq = rng.choice([1, 1, 1, 2, 4, 7])
        if kv == F32:
            kv_heads, batch, hi, prefix = min(kv_heads, 2), log(1, 24), log(1, 600), log(1, 4000)
        else:
            batch, hi, prefix = log(1, 70), log(1, 3000), log(1, 130000)
        prefix = 0 if rng.random() < 0.2 else -(-prefix // page) * page
        out = F32 if kv == F32 or rng.random() < 0.25 else BF16
        return _attend(None, kv, out, batch, kv_heads * group, kv_heads, d, page, prefix, rng.randint(1, hi), hi,
                       nq, nq > 1 and rng.random() < 0.7)
    if kind == "beam":
        hi = log(1, 100000)
        return _beam(None, kv, kv_heads, d, page, log(1, 8), log(1, 60), rng.randint(1, hi), hi,
                     rng.choice([1, 1, 2, 5]))
    if kind == "prompt":
        hi = log(1, 8000)
        return _prompt(None, kv, kv_heads, d, page, log(1, 9), rng.randint(1, hi), hi, hi + rng.randint(0, 200))
    hi = log(1, 20000)
    return _move(None, kv, kv_heads, d, page, log(1, 3 if hi > 900 else 40), rng.randint(1, hi), hi)


# ------------------------------------------------------------------ sizes that follow from a case

def _spread(lo, hi, n):
    """n lengths from lo to hi: ragged, and the same for every seed."""
    return [lo + (((i + 1) * 2654435761 % 2 ** 32) * (hi - lo + 1) >> 32) for i in range(n)]


def _pages(tokens, page):
    return -(-tokens // page)


def _sizes(c):
    """Lengths by slot, slots, pages a slot may hold, and pages of the pool."""
    page = c["page"]
    if c["kind"] == "attend":
        lens = [c["prefix"] + x for x in _spread(c["lo"], c["hi"], c["batch"])]
        width = _pages(max(lens), page)
        return lens, c["batch"], width, c["prefix"] // page + sum(_pages(x - c["prefix"], page) for x in lens) + 5
    if c["kind"] == "beam":
        lens = _spread(c["lo"], c["hi"], c["parents"])
        width = _pages(max(lens) + c["new"], page)
        more = 1 + _pages(c["new"], page)
        return (lens + [0] * c["children"], c["parents"] + c["children"], width,
                sum(_pages(x, page) for x in lens) + c["children"] * more + 3)
    if c["kind"] == "prompt":
        lens = _spread(c["lo"], c["hi"], c["n"])
        return lens, c["n"], _pages(c["capacity"], page), sum(_pages(x, page) for x in lens) + 7
    lens = _spread(c["lo"], c["hi"], c["n"])
    total = sum(_pages(x, page) for x in lens)
    return lens + [0] * c["n"], 2 * c["n"], _pages(max(lens), page), 2 * total + 4


def work(c):
    d, page = c["d"], c["page"]
    esz = 2 if c["kv"] == BF16 else 4
    row = c["kv_heads"] * d * esz * 2  # K and V of one token
    lens, slots, width, num_pages = _sizes(c)
    if c["kind"] == "attend":
        tokens = c["prefix"] + sum(x - c["prefix"] for x in lens)
        q = c["batch"] * c["q_heads"] * c["nq"] * d
        ids = sum(_pages(x - c["prefix"], page) for x in lens) + c["prefix"] // page
        return {"bytes": tokens * row + q * (esz + (2 if c["out"] == BF16 else 4)) + 4 * (ids + 2 * c["batch"]),
                "flops": 4.0 * d * c["q_heads"] * c["nq"] * sum(lens)}
    if c["kind"] == "beam":
        n, new = c["children"], c["new"]
        src = [lens[i % c["parents"]] for i in range(n)]
        ids = sum(_pages(x + new, page) for x in src)
        tails = sum(x % page for x in {i % c["parents"]: lens[i % c["parents"]] for i in range(n)}.values())
        full = sum(_pages(lens[i], page) for i in range(c["parents"]))
        # rows: each tail read once, written per fork; new rows read and written; page ids: the
        # children's freed and written, the parents' read; reference counts read and written
        return {"bytes": tails * row + sum(x % page for x in src) * row + 2 * n * new * row
                + 4 * (2 * ids + full) + 8 * full, "flops": 0}
    if c["kind"] == "prompt":
        ids = sum(_pages(x, page) for x in lens)
        return {"bytes": 4 * sum(lens) * row + 4 * 6 * ids, "flops": 0}
    total = sum(_pages(x, page) for x in lens)
    # rows copied, then whole pages moved; the table restored, freed and renamed
    return {"bytes": 2 * sum(lens) * row + 2 * total * page * row + 4 * 8 * total, "flops": 0}


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0x5EED0000 + seed)
    lens, slots, width, num_pages = _sizes(c)
    H, d, page, dt = c["kv_heads"], c["d"], c["page"], _DT[c["kv"]]
    s = dict(c, slots=slots, width=width, num_pages=num_pages)
    s["K"] = _normal(gen, num_pages, H, page, d, dtype=dt)
    s["V"] = _normal(gen, num_pages, H, page, d, dtype=dt)
    # a few channels of the keys are much larger than the others
    s["K"] *= torch.exp(0.4 * _normal(gen, d)).to(dt)
    ids = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    if c["kind"] in ("prompt", "move"):
        ids = torch.arange(num_pages, device="cuda", dtype=torch.int32)
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    if c["kind"] != "prompt":
        shared = c["prefix"] // page if c["kind"] == "attend" else 0
        table[:, :shared] = ids[:shared]
        at = shared
        for b, x in enumerate(lens):
            n = _pages(x, page) - shared if x else 0
            table[b, shared:shared + n] = ids[at:at + n]
            at += n
    s["table0"] = table
    s["lens0"] = torch.tensor(lens if c["kind"] != "prompt" else [0] * slots, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["kind"] == "attend":
        s["Q"] = _normal(gen, c["batch"], c["q_heads"], c["nq"], d, dtype=dt)
        s["seqs"] = torch.arange(c["batch"], **i32)
        s["scale"] = d ** -0.5
    elif c["kind"] == "beam":
        n = c["children"]
        s["src"] = torch.tensor([i % c["parents"] for i in range(n)], **i32)
        s["dst"] = torch.arange(c["parents"], slots, **i32)
        s["Kn"] = _normal(gen, n, H, c["new"], d, dtype=dt)
        s["Vn"] = _normal(gen, n, H, c["new"], d, dtype=dt)
    elif c["kind"] == "prompt":
        T = max(lens)
        s["seqs"] = torch.arange(slots, **i32)
        s["counts"] = torch.tensor(lens, **i32)
        s["Kn"] = _normal(gen, slots, H, T, d, dtype=dt)
        s["Vn"] = _normal(gen, slots, H, T, d, dtype=dt)
        s["Kd"] = torch.zeros(slots, H, c["capacity"], d, dtype=dt, device="cuda")
        s["Vd"] = torch.zeros_like(s["Kd"])
    else:
        s["src"] = torch.arange(c["n"], **i32)
        s["dst"] = torch.arange(c["n"], slots, **i32)
        s["pages_moved"] = sum(_pages(x, page) for x in lens)
    if own:
        from tree_indexed_sparse_build_b200 import zha
        s["pages"] = zha.Pages(H, d, page, num_pages, slots, width, dt)
        s["pages"].load(s["table0"], s["lens0"])
    s["table"], s["lens"] = s["table0"].clone(), s["lens0"].clone()
    s["refs"] = _count(s["table"], num_pages)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    p, K, V = s["pages"], s["K"], s["V"]
    if s["kind"] == "attend":
        return p.attend(s["Q"], K, V, s["scale"], seqs=s["seqs"], prefix_seq=0, prefix_tokens=s["prefix"],
                        causal=s["causal"], out_dtype=_DT[s["out"]])
    if s["kind"] == "beam":
        p.free(s["dst"])
        p.fork(K, V, s["src"], s["dst"])
        p.append(K, V, s["dst"], s["Kn"], s["Vn"])
        return {"K": K, "V": V, "table": p.table, "lens": p.lens, "refs": p.refs}
    if s["kind"] == "prompt":
        p.free(s["seqs"])
        p.append(K, V, s["seqs"], s["Kn"], s["Vn"], s["counts"])
        p.gather(K, V, s["seqs"], s["Kd"], s["Vd"])
        return {"K": K, "V": V, "Kd": s["Kd"], "Vd": s["Vd"], "table": p.table, "lens": p.lens, "refs": p.refs}
    p.load(s["table0"], s["lens0"])
    p.copy(K, V, s["src"], s["dst"])
    p.free(s["src"])
    live = p.compact(K, V)
    return {"K": K, "V": V, "table": p.table, "lens": p.lens, "refs": p.refs, "live": live}


def _run_plain(s):
    if s["kind"] == "attend":
        return _plain_attend(s)
    if s["kind"] == "beam":
        _plain_free(s, s["dst"])
        _plain_fork(s, s["src"], s["dst"])
        _plain_append(s, s["dst"], s["Kn"], s["Vn"], torch.full_like(s["dst"], s["new"]))
    elif s["kind"] == "prompt":
        _plain_free(s, s["seqs"])
        _plain_append(s, s["seqs"], s["Kn"], s["Vn"], s["counts"])
        _plain_gather(s, s["seqs"], s["Kd"], s["Vd"])
        return {"K": s["K"], "V": s["V"], "Kd": s["Kd"], "Vd": s["Vd"], "table": s["table"], "lens": s["lens"],
                "refs": s["refs"]}
    else:
        s["table"].copy_(s["table0"])
        s["lens"].copy_(s["lens0"])
        s["refs"] = _count(s["table"], s["num_pages"])
        _plain_copy(s, s["src"], s["dst"])
        _plain_free(s, s["src"])
        live = _plain_compact(s)
        return {"K": s["K"], "V": s["V"], "table": s["table"], "lens": s["lens"], "refs": s["refs"], "live": live}
    return {"K": s["K"], "V": s["V"], "table": s["table"], "lens": s["lens"], "refs": s["refs"]}


# ------------------------------------------------------------------ plain forms

def _plain_attend(s):
    """softmax(scale q . k) v over the tokens that a query sees, in 32 bits; zeros if it sees none."""
    B, H, nq, d, P, page = s["batch"], s["kv_heads"], s["nq"], s["d"], s["prefix"], s["page"]
    rows = s["q_heads"] // H * nq
    dev = s["Q"].device
    table, lens = s["table"][s["seqs"].long()].long(), s["lens"][s["seqs"].long()].long()
    q = s["Q"].float().reshape(B, H, rows, d)
    sees = lens[:, None].expand(B, nq)
    if s["causal"]:
        sees = sees - (nq - 1 - torch.arange(nq, device=dev))
    sees = sees.repeat(1, rows // nq)[:, None, :, None]  # [B, 1, rows, 1]

    def dense(x, ids):  # [..., n] page ids -> [..., H, n * page, d]
        return x[ids].movedim(-4, -3).flatten(-3, -2).float()

    mine = table[:, P // page:].clamp(min=0)
    scores = torch.matmul(q, dense(s["K"], mine).transpose(-1, -2)) * s["scale"]
    seen = P + torch.arange(scores.shape[-1], device=dev) < sees
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    if P:
        common = table[0, :P // page]
        qs = q.movedim(1, 0).reshape(H, B * rows, d)
        first = torch.matmul(qs, dense(s["K"], common).transpose(-1, -2)).view(H, B, rows, P).movedim(0, 1)
        first = (first * s["scale"]).masked_fill(torch.arange(P, device=dev) >= sees, -math.inf)
        top = torch.maximum(top, first.amax(-1, keepdim=True))
    top = top.masked_fill(sees <= 0, 0.0)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, dense(s["V"], mine).masked_fill(
        (P + torch.arange(p.shape[-1], device=dev) >= lens[:, None])[:, None, :, None], 0.0))
    if P:
        p = torch.exp(first - top)
        total = total + p.sum(-1, keepdim=True)
        p = p.movedim(1, 0).reshape(H, B * rows, P)
        out = out + torch.matmul(p, dense(s["V"], common)).view(H, B, rows, d).movedim(0, 1)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.reshape(B, s["q_heads"], nq, d).to(_DT[s["out"]])


def _count(table, num_pages):
    """How many rows name each page."""
    named = table.reshape(-1)
    refs = torch.zeros(num_pages, dtype=torch.int32, device=table.device)
    return refs.scatter_add_(0, named.clamp(min=0).long(), (named >= 0).to(torch.int32))


def _free_first(s):
    """Page ids with the free ones first, each part ascending."""
    return torch.argsort((s["refs"] > 0).to(torch.uint8), stable=True)


def _add_refs(s, ids, valid, by):
    s["refs"].scatter_add_(0, ids.reshape(-1).clamp(min=0).long(), (valid.to(torch.int32) * by).reshape(-1))


def _plain_free(s, seqs):
    seqs = seqs.long()
    ids = s["table"][seqs]
    _add_refs(s, ids, ids >= 0, -1)
    s["table"][seqs] = -1
    s["lens"][seqs] = 0


def _rows_under(new, old, keep):
    """`new` in the first keep[i] rows of page i, `old` in the others ([n, H, page, d])."""
    r = torch.arange(new.shape[-2], device=new.device)
    return torch.where((r < keep.view(-1, 1))[:, None, :, None], new, old)


def _plain_fork(s, src, dst):
    src, dst, page = src.long(), dst.long(), s["page"]
    lens = s["lens"][src].long()
    full, rest = lens // page, lens % page
    part = rest > 0
    order = _free_first(s)
    taken = part.long().cumsum(0)
    # forks with no partial page stand for pages of their own and leave them as they are
    other = taken[-1] + (~part).long().cumsum(0) - 1
    fresh = order[torch.where(part, taken - 1, other)]
    ids = s["table"][src]
    col = torch.arange(s["width"], device=src.device)
    last = ids.gather(1, full.clamp(max=s["width"] - 1)[:, None])[:, 0].clamp(min=0).long()
    ids = torch.where((col == full[:, None]) & part[:, None], fresh[:, None].to(torch.int32), ids)
    _add_refs(s, ids, ids >= 0, 1)
    s["table"][dst] = ids
    s["lens"][dst] = lens.to(torch.int32)
    for x in (s["K"], s["V"]):
        x[fresh] = _rows_under(x[last], x[fresh], torch.where(part, rest, torch.zeros_like(rest)))


def _plain_append(s, seqs, Kn, Vn, counts):
    seqs, counts, page, H = seqs.long(), counts.long(), s["page"], s["kv_heads"]
    n, T, dev = Kn.shape[0], Kn.shape[2], Kn.device
    lens = s["lens"][seqs].long()
    old = -torch.div(-lens, page, rounding_mode="floor")
    more = -torch.div(-(lens + counts), page, rounding_mode="floor") - old
    start = more.cumsum(0) - more
    order = _free_first(s)
    j = torch.arange(_pages(T, page) + 1, device=dev)
    valid = j < more[:, None]
    ids = order[(start[:, None] + j).clamp(max=s["num_pages"] - 1)].to(torch.int32)
    rows = torch.cat([s["table"][seqs], torch.zeros(n, 1, dtype=torch.int32, device=dev)], 1)
    rows.scatter_(1, torch.where(valid, old[:, None] + j, torch.full_like(ids, s["width"]).long()), ids)
    s["table"][seqs] = rows[:, :-1]
    _add_refs(s, ids, valid, 1)
    s["lens"][seqs] = (lens + counts).to(torch.int32)
    # tokens behind a sequence's count stand for its last one, sequences without any for the longest
    i = torch.where(counts > 0, torch.arange(n, device=dev), counts.argmax())[:, None]
    t = torch.minimum(torch.arange(T, device=dev).expand(n, T), counts[i] - 1)
    at = lens[i] + t
    to = s["table"][seqs[i], at // page].long()
    h = torch.arange(H, device=dev)[:, None]
    to = ((to[:, None] * H + h) * page + (at % page)[:, None]).reshape(-1)
    for x, y in ((s["K"], Kn), (s["V"], Vn)):
        x.view(-1, x.shape[-1])[to] = y[i[:, None], h, t[:, None]].reshape(-1, x.shape[-1])


def _plain_copy(s, src, dst):
    src, dst, page = src.long(), dst.long(), s["page"]
    lens = s["lens"][src].long()
    n = -torch.div(-lens, page, rounding_mode="floor")
    ids = s["table"][src]
    col = torch.arange(s["width"], device=src.device)
    valid = col < n[:, None]
    order = _free_first(s)
    fresh = order[((n.cumsum(0) - n)[:, None] + col).clamp(max=s["num_pages"] - 1)]
    s["table"][dst] = torch.where(valid, fresh, torch.full_like(fresh, -1)).to(torch.int32)
    _add_refs(s, fresh, valid, 1)
    s["lens"][dst] = lens.to(torch.int32)
    # columns behind a sequence's last page stand for that page
    col = torch.minimum(col.expand_as(ids), n[:, None] - 1)
    a, b = ids.gather(1, col).reshape(-1).long(), fresh.gather(1, col).reshape(-1)
    keep = torch.minimum(lens[:, None] - col * page, torch.full_like(col, page)).reshape(-1)
    for x in (s["K"], s["V"]):
        x[b] = _rows_under(x[a], x[b], keep)


def _plain_compact(s):
    used = s["refs"] > 0
    page = torch.arange(s["num_pages"], device=used.device)
    live = used.sum()
    holes = torch.argsort((used | (page >= live)).to(torch.uint8), stable=True)
    stray = torch.argsort((~used | (page < live)).to(torch.uint8), stable=True)
    n = min(s["pages_moved"], s["num_pages"] // 2)  # no more than were freed
    k = torch.arange(n, device=used.device) < (used & (page >= live)).sum()
    holes, stray = holes[:n], stray[:n]
    for x in (s["K"], s["V"]):
        x[holes] = torch.where(k[:, None, None, None], x[stray], x[holes])
    name = page.clone()
    name[stray] = torch.where(k, holes, stray)
    refs = s["refs"].clone()
    refs[holes] = torch.where(k, s["refs"][stray], s["refs"][holes])
    refs[stray] = torch.where(k, torch.zeros_like(s["refs"][stray]), refs[stray])
    s["refs"].copy_(refs)
    s["table"].copy_(torch.where(s["table"] >= 0, name[s["table"].clamp(min=0).long()].to(torch.int32), s["table"]))
    return live.to(torch.int32)


def _plain_gather(s, seqs, Kd, Vd):
    seqs, page, H = seqs.long(), s["page"], s["kv_heads"]
    lens = s["lens"][seqs].long()
    t = torch.arange(Kd.shape[2], device=Kd.device)
    at = s["table"][seqs].clamp(min=0).long().gather(1, (t // page).clamp(max=s["width"] - 1).expand(len(seqs), -1))
    at = (at[:, None] * H + torch.arange(H, device=Kd.device)[:, None]) * page + t % page
    valid = (t < lens[:, None])[:, None, :, None]
    for x, y in ((s["K"], Kd), (s["V"], Vd)):
        y.copy_(torch.where(valid, x.view(-1, x.shape[-1])[at], y))


# ------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    """The attention of each sequence and KV head by itself over the tokens of its own table row, in
    64 bits.  The other kinds move rows and count: they have no computed numbers."""
    if c["kind"] != "attend" or c["batch"] * c["kv_heads"] * (c["prefix"] + c["hi"]) > 2 ** 28:
        return None
    s = prepare(c, seed)
    H, G, nq, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["nq"], c["d"]
    lens, out = s["lens0"].tolist(), torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        pages = s["table0"][b, :_pages(n, c["page"])].long()
        for h in range(H):
            k = s["K"][pages, h].reshape(-1, d)[:n].double()
            v = s["V"][pages, h].reshape(-1, d)[:n].double()
            for i in range(nq) if c["causal"] else [slice(None)]:
                m = n - (nq - 1 - i) if c["causal"] else n
                if m > 0:
                    q = s["Q"][b, h * G:(h + 1) * G, i].double()
                    w = torch.softmax(q @ k[:m].T * s["scale"], -1)
                    out[b, h * G:(h + 1) * G, i] = w @ v[:m]
    return out
