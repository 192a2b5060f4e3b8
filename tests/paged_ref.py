"""Plain statements of the dense operators for their tests: attention in float64, page tables in Python lists.

``attend64`` also returns how far a kernel may be off.  For a query with weights p_j and values v_j the kernels'
error has these parts (u = 2^-24, half an fp32 step):

* scores: a dot product of d products in fp32, scaled: |error| <= (d + 8) u sum_i |q_i k_ji| scale =: E_j; the weight
  exp(s_j) is off by the factor exp(E_j), and so is the sum it is divided by: 2 E with E = max_j E_j;
* exponentials: 2^-20 covers the rounded exponent (below 128 in magnitude: 128 u = 2^-17 of log2, times ln 2 and u
  again in units of the weight, is inside E for the inputs used here) and a few ulp of the function itself;
* sums of n terms in fp32: n u each, for the output and the divisor;
* rounding of the probabilities before the product with V: `p_round` (2^-8 for one bf16 term, 2^-16 for two, 0 fp32);
all relative to sum_j p_j |v_j|, and the rounding of the stored result, half a step of its type relative to it.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attend64(q, k, v, seen, scale, p_round, out_dtype):
    """q [n, d], k, v [m, d] (float64), row i sees the first seen[i] keys -> (o, tolerance), both [n, d]."""
    n, d = q.shape
    m = k.shape[0]
    if m == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    see = torch.arange(m, device=q.device)[None, :] < seen[:, None]
    kk = torch.where(see.any(0)[:, None], k, 0.0)
    s = (q @ kk.T) * scale
    s = torch.where(see, s, -math.inf)
    top = s.amax(1, keepdim=True)
    w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    w = torch.where(see, w, 0.0)
    p = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    vv = torch.where(see.any(0)[:, None], v, 0.0)
    o = p @ vv
    mass = p @ vv.abs()
    u = 2.0 ** -24
    E = ((q.abs() @ kk.abs().T) * see).amax(1, keepdim=True) * scale * (d + 8) * u
    tol = HALF[out_dtype] * o.abs() + (p_round + 4 * E + 2.0 ** -20 + 2 * m * u) * mass
    return o, tol * (1 + 2.0 ** -7)  # products of the parts


def prompt64(q, k, v, cu_q, cu_k, scale, p_round):
    """Packed prompts: q [N, Hq, d], k, v [M, Hkv, d] -> (o, tol) [N, Hq*d]; rows outside sequences: nan."""
    Hq, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    o = torch.full((q.shape[0], Hq, d), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for s in range(len(cu_q) - 1):
        a, b, c, e = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        seen = (torch.arange(b - a, device=q.device) + 1 + (e - c) - (b - a)).clamp_min(0)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            o[a:b, h], tol[a:b, h] = attend64(q[a:b, h].double(), k[c:e, g].double(), v[c:e, g].double(), seen, scale,
                                              p_round, q.dtype)
    return o.view(-1, Hq * d), tol.view(-1, Hq * d)


def rows_of(pool, ids, page, n):
    """The first n tokens of a row with page ids `ids`, from one layer's pool [pages, Hkv, page, d]: [n, Hkv, d]."""
    if n == 0:
        return pool.new_zeros((0, pool.shape[1], pool.shape[3]))
    x = torch.cat([pool[i].transpose(0, 1) for i in ids], 0)
    return x[:n]


def decode64(q, kp, vp, table, lens, scale, p_round):
    """One token per row: q [n, Hq, d], one layer's pools -> (o, tol) [n, Hq*d]."""
    n, Hq, d = q.shape
    Hkv, page = kp.shape[1], kp.shape[2]
    o = torch.zeros((n, Hq, d), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    G = Hq // Hkv
    for i in range(n):
        L = int(lens[i])
        ids = [int(x) for x in table[i][:-(-L // page)]]
        k, v = (rows_of(p, ids, page, L).double() for p in (kp, vp))
        seen = torch.full((G,), L, device=q.device)
        for g in range(Hkv):
            r = slice(g * G, (g + 1) * G)
            o[i, r], tol[i, r] = attend64(q[i, r].double(), k[:, g], v[:, g], seen, scale, p_round, q.dtype)
    return o.view(n, -1), tol.view(n, -1)


def update_ref(table, lens, parents, grow, pages, page, width):
    """mono_paged_update on lists: (table_out rows padded with -1, lens_out, copies [(from, to)], short)."""
    held = [row[:-(-n // page)] for row, n in zip(table, lens)]
    used = {p for row in held for p in row}
    free = [p for p in range(pages) if p not in used]
    kept, after = [], []
    for p, g in zip(parents, grow):
        n = lens[p] if p >= 0 else 0
        after.append(min(max(0, n + g), width * page))
        kept.append(min(n, after[-1]))
    past = {x for p, b in zip(parents, kept) if p >= 0 for x in held[p][:b // page]}
    ends, out, copies, short = set(), [], [], 0

    def take():
        nonlocal short
        if free:
            return free.pop(0)
        short += 1
        return -1

    for p, b, n in zip(parents, kept, after):
        row = list(held[p][:-(-b // page)]) if p >= 0 else []
        if b % page:
            last = row[-1]
            if last in past or last in ends:
                row[-1] = take()
                if row[-1] >= 0:
                    copies.append((last, row[-1]))
            ends.add(last)
        while len(row) < -(-n // page):
            row.append(take())
        out.append(row + [-1] * (width - len(row)))
    return out, after, copies, short


def compact_ref(table, lens, page, width):
    """mono_paged_compact on lists: (table_out, moves [(from, to)], live)."""
    held = [row[:-(-n // page)] for row, n in zip(table, lens)]
    used = sorted({p for row in held for p in row})
    live, inside = len(used), set(used)
    to = dict(zip([p for p in used if p >= live], [p for p in range(live) if p not in inside]))
    out = [[to.get(p, p) for p in row] + [-1] * (width - len(row)) for row in held]
    return out, sorted(to.items()), live
