"""What is measured of the dense-attention operators: attention over packed prompts, a paged key/value cache with the
attention of one new token per sequence, and the page table's own steps.

``listed()`` gives the fixed cases, ``draw(rng)`` further ones of the same ranges.  ``run(state)`` is one pass of one
operator: the plain torch form where ``own`` is false, the library's entry point where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # the first prompts of a few short chats, one of them a chunk after cached context: latency counts
        dict(name="prompt_short", op="prompt", dtype="bf16", Hq=16, Hkv=16, d=64, seqs=3, longest=129, context=70),
        # a serving batch around one long document, grouped heads (16,384 tokens and 16 heads of 128: the skewed
        # batch's sequence length and heads)
        dict(name="prompt_long", op="prompt", dtype="bf16", Hq=16, Hkv=4, d=128, seqs=6, longest=16384, context=0),
        # fp32 storage, ragged, as the fp32 recall workload (8 heads of 64)
        dict(name="prompt_f32", op="prompt", dtype="f32", Hq=8, Hkv=4, d=64, seqs=5, longest=2047, context=0),
        # one chat's next token: latency counts
        dict(name="decode_one", op="decode", dtype="bf16", Hq=16, Hkv=16, d=64, page=64, rows=1, longest=1000),
        # a batch of long contexts of very different lengths, grouped heads
        dict(name="decode_batch", op="decode", dtype="bf16", Hq=16, Hkv=4, d=128, page=64, rows=40, longest=65521),
        # fp32 storage, small pages
        dict(name="decode_f32", op="decode", dtype="f32", Hq=8, Hkv=8, d=64, page=16, rows=6, longest=4099),
        # one new token of every sequence into its page
        dict(name="append_token", op="append", dtype="bf16", Hkv=4, d=128, page=64, rows=64, longest=8000, new=1),
        # whole prompts into their pages
        dict(name="append_prompt", op="append", dtype="bf16", Hkv=16, d=128, page=128, rows=7, longest=16384, new=8192),
        # a step of four beams of one sequence, one layer
        dict(name="update_beams", op="update", dtype="bf16", Hkv=16, d=64, page=32, layers=1, rows=4, longest=600,
             pages=256),
        # a batch of sequences forked, continued, cut back and dropped, eight layers
        dict(name="update_batch", op="update", dtype="bf16", Hkv=4, d=128, page=64, layers=8, rows=160, longest=1500,
             pages=4096),
        # a small pool closed up, fp32 storage
        dict(name="compact_small", op="compact", dtype="f32", Hkv=4, d=64, page=16, layers=2, rows=9, longest=400,
             pages=300, moved=11),
        # a long-running pool closed up before its end is given back
        dict(name="compact_large", op="compact", dtype="bf16", Hkv=4, d=128, page=64, layers=4, rows=64, longest=4000,
             pages=6000, moved=700),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "decode", "append", "update", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "prompt":
        group = rng.choice([1, 2, 4, 5, 8])
        Hkv = max(1, min(Hkv, 32 // group))
        longest = _log(rng, 1, 2100 if dtype == "f32" else 9000)
        return dict(op=op, dtype=dtype, Hq=Hkv * group, Hkv=Hkv, d=d, seqs=_log(rng, 1, 24 if longest < 2000 else 6),
                    longest=longest, context=rng.choice([0, 0, _log(rng, 1, 2000)]))
    if op == "decode":
        Hkv = min(Hkv, 8)
        rows = _log(rng, 1, 200)
        longest = _log(rng, 1, min(130000, 1200000 // (rows * Hkv) + 300))
        return dict(op=op, dtype=dtype, Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 16]), Hkv=Hkv, d=d, page=page, rows=rows,
                    longest=longest)
    if op == "append":
        rows = _log(rng, 1, 100)
        longest = _log(rng, 4, 9000 if rows < 20 else 2000)
        return dict(op=op, dtype=dtype, Hkv=Hkv, d=d, page=page, rows=rows, longest=longest,
                    new=rng.choice([1, 1, _log(rng, 1, longest)]))
    rows = _log(rng, 1, 160)
    longest = _log(rng, 1, 1500)
    layers = rng.choice([1, 2, 3, 8])
    need = rows * (-(-longest // page) + 2)
    budget = (4 << 30) // (2 * layers * Hkv * page * d * ES[dtype])
    if op == "update":
        rows = max(1, min(rows, budget // (-(-longest // page) + 2) // 2))
        need = rows * (-(-longest // page) + 2)
        return dict(op=op, dtype=dtype, Hkv=Hkv, d=d, page=page, layers=layers, rows=rows, longest=longest,
                    pages=2 * need + rng.randrange(60))
    rows = max(1, min(rows, budget // (-(-longest // page) + 2) // 2))
    need = rows * (-(-longest // page) + 2)
    return dict(op=op, dtype=dtype, Hkv=Hkv, d=d, page=page, layers=layers, rows=rows, longest=longest,
                pages=2 * need + rng.randrange(60), moved=rng.randrange(1, max(2, rows)))


# --------------------------------------------------------------------------
# the sizes of a case: functions of the case alone, so that work() knows them
# --------------------------------------------------------------------------
def _lengths(n, longest, salt=""):
    """n lengths, the longest first, the others spread over the logarithm of 1 .. longest."""
    r = random.Random("%d/%d/%s" % (n, longest, salt))
    return [longest] + [_log(r, 1, longest) for _ in range(n - 1)]


def _prompt_lengths(c):
    lq = _lengths(c["seqs"], c["longest"])
    lk = [q + (c["context"] if i % 2 == 0 else 0) for i, q in enumerate(lq)]
    return lq, lk


def _append_lengths(c):
    """(lengths after the call, new tokens) of each row."""
    lens = _lengths(c["rows"], c["longest"])
    return lens, [min(n, c["new"]) for n in lens]


def _update_rows(c):
    """Lengths, shared leading pages, parents and growth of a pool step: most rows go on by a token, some are forked,
    some dropped, some cut back as after rejected drafts, one slot takes a new prompt."""
    r = random.Random("update/%d/%d" % (c["rows"], c["longest"]))
    n = c["rows"]
    lens = _lengths(n, c["longest"])
    shared = [0] + [r.choice([0, 0, min(lens[i], lens[i - 1]) // c["page"]]) for i in range(1, n)]
    parents, grow = [], []
    for i in range(n):
        what = r.random()
        p = i if what < 0.4 else r.randrange(n) if what < 0.9 else -1
        parents.append(p)
        grow.append(r.choice([0, 40]) if p < 0 else r.choice([1, 1, 1, 5, 0, -3]))
    return lens, shared, parents, grow


def _copied_pages(c):
    """How many tail pages the step of _update_rows copies, by counting the rows that hold each page in their middle."""
    lens, shared, parents, grow = _update_rows(c)
    page = c["page"]
    ids, nxt = [], 0
    for i, n in enumerate(lens):
        np_ = -(-n // page)
        row = (ids[i - 1][:shared[i]] if i else []) + list(range(nxt, nxt + np_ - shared[i]))
        nxt += np_ - shared[i]
        ids.append(row)
    whole, part = set(), {}
    for p, g in zip(parents, grow):
        if p < 0:
            continue
        base = max(0, min(lens[p], lens[p] + g))
        whole |= set(ids[p][:base // page])
        if base % page:
            k = ids[p][base // page]
            part[k] = part.get(k, 0) + 1
    return sum(v if k in whole else v - 1 for k, v in part.items())


def _width(lens, page, more=0):
    return max(1, max(-(-n // page) for n in lens) + more)


def work(c):
    es, d = ES[c["dtype"]], c["d"]
    if c["op"] == "prompt":
        lq, lk = _prompt_lengths(c)
        pairs = sum(q * k - q * (q - 1) // 2 for q, k in zip(lq, lk))
        return {"bytes": es * d * (2 * sum(lq) * c["Hq"] + 2 * sum(lk) * c["Hkv"]), "flops": 4 * d * c["Hq"] * pairs}
    if c["op"] == "decode":
        lens = _lengths(c["rows"], c["longest"])
        table = 4 * sum(-(-n // c["page"]) for n in lens)
        return {"bytes": 2 * es * d * (sum(lens) * c["Hkv"] + c["rows"] * c["Hq"]) + table,
                "flops": 4 * d * c["Hq"] * sum(lens)}
    if c["op"] == "append":
        new = sum(_append_lengths(c)[1])
        return {"bytes": 4 * new * c["Hkv"] * d * es, "flops": 0}
    page_bytes = 2 * c["layers"] * c["Hkv"] * c["page"] * d * es
    if c["op"] == "update":
        lens, _, parents, grow = _update_rows(c)
        after = [max(0, (lens[p] if p >= 0 else 0) + g) for p, g in zip(parents, grow)]
        tables = 4 * sum(-(-n // c["page"]) for n in lens) + 4 * c["rows"] * _width(lens, c["page"], 2)
        return {"bytes": 2 * page_bytes * _copied_pages(c) + tables + 16 * len(after), "flops": 0}
    lens = _lengths(c["rows"], c["longest"])
    tables = 4 * sum(-(-n // c["page"]) for n in lens) + 4 * c["rows"] * _width(lens, c["page"])
    return {"bytes": 2 * page_bytes * _moved_pages(c) + tables, "flops": 0}


def _moved_pages(c):
    live = sum(-(-n // c["page"]) for n in _lengths(c["rows"], c["longest"]))
    return min(c["moved"], live, c["pages"] - live)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _table(rows, width):
    """[rows, width] int32 from lists of page ids, -1 behind each."""
    t = torch.full((len(rows), width), -1, dtype=torch.int32)
    for i, r in enumerate(rows):
        t[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return t.cuda()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    r = random.Random(seed)
    dt, d = DTYPES[c["dtype"]], c["d"]

    def normal(*shape, sd=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=dt) * sd).contiguous()

    s = {"c": c}
    sizes = dict(Hq=c.get("Hq", c["Hkv"]), Hkv=c["Hkv"], d=d, page=c.get("page", 64), pages=1, layers=1, rows=1,
                 width=1, tokens=1, dtype=c["dtype"])
    if c["op"] == "prompt":
        lq, lk = _prompt_lengths(c)
        # attention logits of a few units, as trained heads have them
        s.update(lq=lq, lk=lk, q=normal(sum(lq), c["Hq"], d, sd=1.5), k=normal(sum(lk), c["Hkv"], d, sd=1.5),
                 v=normal(sum(lk), c["Hkv"], d), cu_q=_ints(_cu(lq)), cu_k=_ints(_cu(lk)))
        s["o"] = torch.empty((sum(lq), c["Hq"] * d), dtype=dt, device="cuda")
        sizes.update(rows=len(lq), tokens=sum(lq))
    else:
        page = c["page"]
        if c["op"] == "append":
            lens, new = _append_lengths(c)
        else:
            lens = _lengths(c["rows"], c["longest"])
        counts = [-(-n // page) for n in lens]
        shared = [0] * len(lens)
        more = 0
        if c["op"] == "update":
            _, shared, parents, grow = _update_rows(c)
            more = 2
        pages = c.get("pages", sum(counts) + 5)
        width = _width(lens, page, more)
        if c["op"] == "compact":
            live, moved = sum(counts), _moved_pages(c)
            ids = r.sample(range(live), live - moved) + r.sample(range(live, pages), moved)
            r.shuffle(ids)
        else:
            ids = r.sample(range(pages), sum(counts) - sum(shared))
        rows, at = [], 0
        for i, n in enumerate(counts):
            take = n - shared[i]
            rows.append((rows[i - 1][:shared[i]] if i else []) + ids[at:at + take])
            at += take
        s.update(lens=_ints(lens), table=_table(rows, width))
        layers = c.get("layers", 1)
        # logits of a few units, and a pool whose unused rows hold what earlier sequences left there
        s["kp"] = normal(layers, pages, c["Hkv"], page, d, sd=1.5)
        s["vp"] = normal(layers, pages, c["Hkv"], page, d)
        sizes.update(page=page, pages=pages, layers=layers, rows=len(lens), width=width)
        if c["op"] == "decode":
            s["q"] = normal(len(lens), c["Hq"], d, sd=1.5)
            s["o"] = torch.empty((len(lens), c["Hq"] * d), dtype=dt, device="cuda")
        elif c["op"] == "append":
            s.update(k=normal(sum(new), c["Hkv"], d, sd=1.5), v=normal(sum(new), c["Hkv"], d), cu=_ints(_cu(new)))
        else:
            s.update(table_out=torch.empty((len(lens), width), dtype=torch.int32, device="cuda"))
            if c["op"] == "update":
                s.update(parents=_ints(parents), grow=_ints(grow), lens_out=torch.empty_like(s["lens"]))
    if own:
        from learned_product_hash_proj_b200 import mono
        s["plan"] = mono.PagedPlan(mono.PagedConfig(**sizes))
        s["ws"] = s["plan"].workspace()
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["c"]["op"]
    if own:
        from learned_product_hash_proj_b200 import mono
        plan, ws = s["plan"], s["ws"]
        if op == "prompt":
            mono.prompt_attend(plan, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["o"], ws)
            return s["o"]
        if op == "decode":
            mono.paged_attend(plan, 0, s["q"], s["table"], s["lens"], s["o"], s["kp"], s["vp"], ws)
            return s["o"]
        if op == "append":
            mono.paged_append(plan, 0, s["k"], s["v"], s["cu"], s["table"], s["lens"], s["kp"], s["vp"], ws)
            return s["kp"], s["vp"]
        if op == "update":
            mono.paged_update(plan, s["table"], s["lens"], s["parents"], s["grow"], s["table_out"], s["lens_out"],
                              s["kp"], s["vp"], ws)
            return s["table_out"], s["lens_out"], s["kp"], s["vp"]
        mono.paged_compact(plan, s["table"], s["lens"], s["table_out"], s["kp"], s["vp"], ws)
        return s["table_out"], s["kp"], s["vp"]
    return {"prompt": _prompt, "decode": _decode, "append": _append, "update": _update, "compact": _compact}[op](s)


def _softmax_(x):
    """In place over the last axis; rows that hold only -inf become zeros."""
    m = x.amax(dim=-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    return x.div_(x.sum(dim=-1, keepdim=True).clamp_min_(1e-37))


def _prompt(s):
    c = s["c"]
    G, Hkv, d = c["Hq"] // c["Hkv"], c["Hkv"], c["d"]
    outs, q0, k0 = [], 0, 0
    for nq, nk in zip(s["lq"], s["lk"]):  # packed sequences of different lengths: one at a time
        q = s["q"][q0:q0 + nq].float().view(nq, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * nq, d)
        k = s["k"][k0:k0 + nk].float().permute(1, 2, 0)
        v = s["v"][k0:k0 + nk].float().permute(1, 0, 2)
        x = torch.matmul(q * d ** -0.5, k).view(Hkv, G, nq, nk)
        ahead = torch.arange(nk, device="cuda") > torch.arange(nk - nq, nk, device="cuda")[:, None]
        p = _softmax_(x.masked_fill_(ahead, -math.inf))
        o = torch.matmul(p.view(Hkv, G * nq, nk), v).view(Hkv, G, nq, d)
        outs.append(o.permute(2, 0, 1, 3).reshape(nq, c["Hq"] * d).to(s["q"].dtype))
        q0, k0 = q0 + nq, k0 + nk
    return torch.cat(outs)


def _decode(s):
    c = s["c"]
    n, width = s["table"].shape
    Hkv, d, G = c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    ids = s["table"].clamp_min(0).long()
    k = s["kp"][0][ids].permute(0, 2, 1, 3, 4).reshape(n, Hkv, width * c["page"], d).float()
    x = torch.matmul(s["q"].float().view(n, Hkv, G, d) * d ** -0.5, k.transpose(2, 3))
    del k
    behind = torch.arange(width * c["page"], device="cuda") >= s["lens"][:, None]
    p = _softmax_(x.masked_fill_(behind[:, None, None], -math.inf))
    v = s["vp"][0][ids].permute(0, 2, 1, 3, 4).reshape(n, Hkv, width * c["page"], d).float()
    return torch.matmul(p, v).reshape(n, c["Hq"] * d).to(s["q"].dtype)


def _append(s):
    N = s["k"].shape[0]
    at = torch.arange(N, device="cuda", dtype=torch.int32)
    row = torch.searchsorted(s["cu"], at, right=True) - 1
    pos = s["lens"][row] - s["cu"][row + 1] + at
    page = s["c"]["page"]
    pid, off = s["table"][row, (pos // page).long()].long(), (pos % page).long()
    s["kp"][0][pid, :, off] = s["k"]
    s["vp"][0][pid, :, off] = s["v"]
    return s["kp"], s["vp"]


def _used_pages(s):
    """[pages] true where a row's table holds the page within the row's length."""
    P, page = s["kp"].shape[1], s["c"]["page"]
    cols = torch.arange(s["table"].shape[1], device="cuda")
    held = cols < (s["lens"][:, None] + page - 1) // page
    used = torch.zeros(P + 1, dtype=torch.bool, device="cuda")
    used[torch.where(held, s["table"], P).long().flatten()] = True
    return used[:P], held, cols


def _update(s):
    page, P = s["c"]["page"], s["kp"].shape[1]
    used, _, cols = _used_pages(s)
    par = s["parents"].long()
    src = par.clamp_min(0)
    before = torch.where(par >= 0, s["lens"][src], 0)
    after = (before + s["grow"]).clamp_min(0)
    base = torch.minimum(before, after)
    old = s["table"][src]
    keep = cols < ((base + page - 1) // page)[:, None]
    part = (base % page != 0)
    tail = old.gather(1, (base // page).long().clamp_max(old.shape[1] - 1)[:, None])[:, 0]
    tail = torch.where(part, tail, P).long()
    # a partly filled page stays with the first row that ends in it, unless another row goes on past it
    whole = torch.zeros(P + 1, dtype=torch.bool, device="cuda")
    whole[torch.where(cols < (base // page)[:, None], old, P).long().flatten()] = True
    index = torch.arange(len(par), device="cuda")
    first = torch.full((P + 1,), len(par), device="cuda").scatter_reduce(0, tail, index, "amin")
    copy = part & (whole[tail] | (first[tail] != index))
    fresh = (cols < ((after + page - 1) // page)[:, None]) & ~keep
    fresh |= copy[:, None] & (cols == (base // page)[:, None])
    free = torch.sort(used.to(torch.int8), stable=True)[1]
    nth = fresh.flatten().cumsum(0).view_as(fresh) - 1
    new = torch.where(nth < (~used).sum(), free[nth.clamp(0, P - 1)], -1).int()
    out = torch.where(fresh, new, torch.where(keep, old, -1))
    at = copy.nonzero()[:, 0]
    dst = out[at, (base // page)[at].long()].long()
    s["kp"][:, dst] = s["kp"][:, tail[at]]
    s["vp"][:, dst] = s["vp"][:, tail[at]]
    return out, after, s["kp"], s["vp"]


def _compact(s):
    used, held, _ = _used_pages(s)
    P = used.shape[0]
    live = used.sum()
    ids = torch.arange(P, device="cuda")
    frm = (used & (ids >= live)).nonzero()[:, 0]
    to = (~used & (ids < live)).nonzero()[:, 0]
    s["kp"][:, to] = s["kp"][:, frm]
    s["vp"][:, to] = s["vp"][:, frm]
    ids[frm] = to
    return torch.where(held, ids[s["table"].clamp_min(0).long()].int(), -1), s["kp"], s["vp"]


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits (tables: in plain Python)
# --------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    return {"prompt": _exact_prompt, "decode": _exact_decode, "append": _exact_append, "update": _exact_update,
            "compact": _exact_compact}[c["op"]](s)


def _attend64(q, k, v, seen):
    """q [n, d], k, v [m, d], seen [n]: row i sees the first seen[i] keys."""
    z = torch.einsum("nd,md->nm", q, k) / math.sqrt(q.shape[1])
    z = torch.where(torch.arange(k.shape[0], device=q.device)[None, :] < seen[:, None], z, -math.inf)
    w = torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True))
    return torch.einsum("nm,md->nd", w, v)


def _exact_prompt(s):
    c = s["c"]
    d = c["d"]
    out = torch.empty((sum(s["lq"]), c["Hq"], d), dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(s["lq"], s["lk"]):
        for h in range(c["Hq"]):
            kv = h // (c["Hq"] // c["Hkv"])
            k, v = s["k"][k0:k0 + nk, kv].double(), s["v"][k0:k0 + nk, kv].double()
            for a in range(0, nq, 4096):
                b = min(nq, a + 4096)
                seen = torch.arange(a, b, device="cuda") + (nk - nq + 1)
                m = nk - nq + b
                out[q0 + a:q0 + b, h] = _attend64(s["q"][q0 + a:q0 + b, h].double(), k[:m], v[:m], seen)
        q0, k0 = q0 + nq, k0 + nk
    return out.view(-1, c["Hq"] * d)


def _exact_decode(s):
    c = s["c"]
    d, Hkv, G = c["d"], c["Hkv"], c["Hq"] // c["Hkv"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    out = torch.empty((len(lens), c["Hq"], d), dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        ids = torch.tensor(table[i][:-(-n // c["page"])], device="cuda")
        seen = torch.full((G,), n, device="cuda")
        for h in range(Hkv):
            k, v = (p[0, ids, h].reshape(-1, d)[:n].double() for p in (s["kp"], s["vp"]))
            out[i, h * G:(h + 1) * G] = _attend64(s["q"][i, h * G:(h + 1) * G].double(), k, v, seen)
    return out.view(len(lens), -1)


def _exact_append(s):
    cu, lens, table, page = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist(), s["c"]["page"]
    kp, vp = s["kp"].double(), s["vp"].double()
    for i, n in enumerate(lens):
        t, pos = cu[i], n - (cu[i + 1] - cu[i])
        while pos < n:  # page by page
            m = min(page - pos % page, n - pos)
            for pool, new in ((kp, s["k"]), (vp, s["v"])):
                pool[0, table[i][pos // page], :, pos % page:pos % page + m] = new[t:t + m].double().transpose(0, 1)
            t, pos = t + m, pos + m
    return kp, vp


def _exact_update(s):
    page, P = s["c"]["page"], s["kp"].shape[1]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    parents, grow = s["parents"].tolist(), s["grow"].tolist()
    held = [row[:-(-n // page)] for row, n in zip(table, lens)]
    used = set(p for row in held for p in row)
    free = [p for p in range(P) if p not in used]
    kept, after = [], []
    for p, g in zip(parents, grow):
        n = lens[p] if p >= 0 else 0
        after.append(max(0, n + g))
        kept.append(min(n, after[-1]))
    past = set(x for p, b in zip(parents, kept) if p >= 0 for x in held[p][:b // page])
    taken, out, moves = set(), [], []
    for p, b, n in zip(parents, kept, after):
        row = held[p][:-(-b // page)] if p >= 0 else []
        if b % page:
            last = row[-1]
            if last in past or last in taken:
                row[-1] = free.pop(0)
                moves.append((last, row[-1]))
            taken.add(last)
        while len(row) < -(-n // page):
            row.append(free.pop(0))
        out.append(row)
    kp, vp = s["kp"].double(), s["vp"].double()
    for a, b in moves:
        kp[:, b] = kp[:, a]
        vp[:, b] = vp[:, a]
    return _table(out, s["table"].shape[1]), _ints(after), kp, vp


def _exact_compact(s):
    page, P = s["c"]["page"], s["kp"].shape[1]
    held = [row[:-(-n // page)] for row, n in zip(s["table"].tolist(), s["lens"].tolist())]
    used = sorted(set(p for row in held for p in row))
    live = len(used)
    inside = set(used)
    to = dict(zip([p for p in used if p >= live], [p for p in range(live) if p not in inside]))
    kp, vp = s["kp"].double(), s["vp"].double()
    for a, b in to.items():
        kp[:, b] = kp[:, a]
        vp[:, b] = vp[:, a]
    return _table([[to.get(p, p) for p in row] for row in held], s["table"].shape[1]), kp, vp
