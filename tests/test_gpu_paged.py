"""The dense operators on the GPU against plain statements in float64 (attention) and Python lists (page tables)."""
import concurrent.futures
import math
import random
import threading
import types

import pytest
import torch

from learned_product_hash_proj_b200 import mono
from paged_ref import HALF, attend64, compact_ref, decode64, prompt64, rows_of, update_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# rounding of the probabilities before the product with V: one bf16 term (prompt), two (one new token), none (fp32).
# The prompt kernel's exponentials are in part a cubic of relative error 7.5e-5 < 2^-13, which counts twice: in a
# probability and in the sum that divides it.
P_PROMPT = {"bf16": 2.0 ** -8 + 2.0 ** -12, "f32": 0.0}
P_DECODE = {"bf16": 2.0 ** -16, "f32": 0.0}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from learned_product_hash_proj_b200 import build
    build.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(seed, *shape, dtype=torch.float32, sd=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sd).to(dtype)


def cumulative(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def plan_for(dtype, Hq, Hkv, d, **kw):
    return mono.PagedPlan(mono.PagedConfig(Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, **kw))


def assert_within(got, ref, tol, what):
    far = ((got.double() - ref).abs() - tol).max().item() if got.numel() else 0.0
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    assert far <= 0.0, f"{what}: {far:.3e} beyond the tolerance"


# ---------------------------------------------------------------------------
# packed prompts
# ---------------------------------------------------------------------------
PROMPTS = {
    "one_token": ([1], [1]),
    "tile_edges": ([127, 128, 129], [127, 128, 129]),
    "two_tiles": ([255, 256, 257, 1], [255, 256, 257, 1]),
    "empty_between": ([0, 5, 0, 0, 70, 0], [0, 5, 0, 0, 70, 0]),
    "after_context": ([1, 33, 128], [500, 97, 129]),
    "fewer_keys": ([40, 7, 130], [3, 0, 129]),       # the first queries see no key: zeros
    "long": ([1100, 3], [1100, 3]),
    "split_keys": ([640], [640]),                    # fp32: few rows and many keys, several CTAs per tile
    "one_after_many": ([3], [1500]),
    "chunks_after_many": ([5, 200], [5000, 3333]),   # bf16: keys split over the CTAs of a cluster
    # bf16: a group per query tile, with keys of its own
    "short_and_long": ([3] * 40 + [700, 0] + [90] * 21, [3] * 40 + [705, 0] + [400] * 20 + [20]),
    "many_short": ([3, 1, 2, 5, 8, 1, 1, 4] * 12, [3, 1, 2, 5, 8, 1, 1, 4] * 12),
}


def run_prompt(dtype, Hq, Hkv, d, lq, lk, seed, scale=0.0, behind=0, ahead=0, q=None, k=None, v=None, stream=None):
    dt = DT[dtype]
    cq, ck = [ahead + x for x in cumulative(lq)], [ahead + x for x in cumulative(lk)]
    nq, nk = cq[-1] + behind, ck[-1] + behind
    q = normal(seed, nq, Hq, d, dtype=dt, sd=1.5) if q is None else q
    k = normal(seed + 1, nk, Hkv, d, dtype=dt, sd=1.5) if k is None else k
    v = normal(seed + 2, nk, Hkv, d, dtype=dt) if v is None else v
    o = torch.full((nq, Hq * d), 7.0, dtype=dt, device="cuda")
    plan = plan_for(dtype, Hq, Hkv, d, rows=len(lq), tokens=nq, scale=scale)
    ws = plan.workspace()
    mono.prompt_attend(plan, q, k, v, ints(cq), ints(ck), o, ws, stream=stream)
    assert mono.paged_stats(plan, ws, stream=stream)["device_error"] == 0
    return q, k, v, cq, ck, o, plan


@pytest.mark.parametrize("name", list(PROMPTS))
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("f32", 4, 4, 64), ("f32", 6, 2, 128), ("bf16", 4, 4, 64),
                                            ("bf16", 5, 1, 128), ("bf16", 8, 2, 128), ("bf16", 6, 1, 64),
                                            ("bf16", 16, 1, 128), ("bf16", 32, 1, 64)])
def test_prompt(dtype, Hq, Hkv, d, name):
    lq, lk = PROMPTS[name]
    q, k, v, cq, ck, o, _ = run_prompt(dtype, Hq, Hkv, d, lq, lk, seed=11)
    ref, tol = prompt64(q, k, v, cq, ck, d ** -0.5, P_PROMPT[dtype])
    assert_within(o, ref, tol, name)
    if name == "fewer_keys":
        assert (o[:37] == 0).all() and (o[40:47] == 0).all() and (o[47] == 0).all() and (o[48] != 0).any()


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("f32", 4, 1, 64), ("bf16", 8, 2, 128), ("bf16", 6, 6, 64)])
def test_prompt_more_tiles_than_sms(dtype, Hq, Hkv, d):
    # several query tiles per CTA, of very different lengths and not in order of length; keys before the queries
    lq = [1, 700, 2600, 0, 257, 1500, 64, 3, 2049, 128, 900]
    lk = [n + 90 * (i % 3) for i, n in enumerate(lq)]
    q, k, v, cq, ck, o, _ = run_prompt(dtype, Hq, Hkv, d, lq, lk, seed=17)
    ref, tol = prompt64(q, k, v, cq, ck, d ** -0.5, P_PROMPT[dtype])
    assert_within(o, ref, tol, "many tiles")


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_short_tiles_again_and_again(d):
    # many items of one to three key tiles per CTA, where the kernel's warps run furthest ahead of one another: every
    # call gives the same bits, and none runs out of time
    lq = [300] * 40 + [1, 129, 40] * 5
    q, k, v, cq, ck, first, plan = run_prompt("bf16", 32, 8, d, lq, lq, seed=23)
    ws = plan.workspace()
    outs = [torch.empty_like(first) for _ in range(30)]
    for o in outs:
        mono.prompt_attend(plan, q, k, v, ints(cq), ints(ck), o, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0
    assert all(torch.equal(o, first) for o in outs)
    ref, tol = prompt64(q, k, v, cq, ck, d ** -0.5, P_PROMPT["bf16"])
    assert_within(first, ref, tol, "short tiles")


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 4, 128), (12, 4, 64), (64, 4, 128)])
def test_prompt_short_behind_contexts_again_and_again(Hq, Hkv, d):
    # few queries over contexts of very different lengths: key tiles land in another order every time
    lq = [1 + 7 * i % 20 for i in range(64)]
    lk = [n + (0, 0, 100, 1000, 3000)[i % 5] for i, n in enumerate(lq)]
    q, k, v, cq, ck, first, plan = run_prompt("bf16", Hq, Hkv, d, lq, lk, seed=29)
    ws = plan.workspace()
    outs = [torch.empty_like(first) for _ in range(60)]
    for o in outs:
        mono.prompt_attend(plan, q, k, v, ints(cq), ints(ck), o, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0
    assert all(torch.equal(o, first) for o in outs)
    ref, tol = prompt64(q, k, v, cq, ck, d ** -0.5, P_PROMPT["bf16"])
    assert_within(first, ref, tol, "short behind contexts")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_many_sequences(dtype):
    # more sequences than the threads that count their tiles
    lq = [1 + i % 2 for i in range(1300)]
    q, k, v, cq, ck, o, _ = run_prompt(dtype, 1, 1, 64, lq, lq, seed=3)
    first = torch.tensor(cq[:-1], device="cuda")
    assert torch.equal(o[first], v[first, 0])              # a first token sees itself alone
    own = [i for i in range(1300) if lq[i] == 2][::50]
    for i in own:
        ref, tol = prompt64(q[cq[i]:cq[i] + 2], k[cq[i]:cq[i] + 2], v[cq[i]:cq[i] + 2], [0, 2], [0, 2], 64 ** -0.5,
                            P_PROMPT[dtype])
        assert_within(o[cq[i]:cq[i] + 2], ref, tol, f"sequence {i}")


def test_prompt_and_decode_of_nothing():
    plan = plan_for("bf16", 4, 2, 64, page=16, pages=4, rows=3, width=2, tokens=8)
    ws = plan.workspace()
    kp, vp = plan.pools()
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    before = mono.kernel_launches()
    mono.prompt_attend(plan, e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), ints([0, 0]), ints([0, 0]), e(0, 256), ws)
    mono.prompt_attend(plan, e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), ints([0]), ints([0]), e(0, 256), ws)
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    mono.paged_attend(plan, 0, e(0, 4, 64), none, ints([]), e(0, 256), kp, vp, ws)
    mono.paged_append(plan, 0, e(0, 2, 64), e(0, 2, 64), ints([0]), none, ints([]), kp, vp, ws)
    mono.paged_update(plan, none, ints([]), ints([]), ints([]), none.clone(), ints([]), kp, vp, ws)
    mono.paged_compact(plan, none, ints([]), none.clone(), kp, vp, ws)
    assert mono.kernel_launches() == before
    # queries without any key: zeros
    o = torch.full((3, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    mono.prompt_attend(plan, normal(1, 3, 4, 64, dtype=torch.bfloat16), e(0, 2, 64), e(0, 2, 64), ints([0, 3]),
                       ints([0, 0]), o, ws)
    assert (o == 0).all()
    # a plan whose rows have no pages at all
    flat = plan_for("f32", 2, 2, 64, page=16, pages=1, rows=2, width=0)
    ws = flat.workspace()
    kp, vp = flat.pools()
    o = torch.full((2, 128), 7.0, device="cuda")
    no = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    mono.paged_attend(flat, 0, normal(1, 2, 2, 64), no, ints([0, 0]), o, kp, vp, ws)
    assert (o == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_touches_and_reads_its_own_rows_only(dtype):
    # rows before the first and behind the last sequence, and a whole neighbour, hold NaN: they reach nothing else
    lq, d = [70, 131, 9], 64
    cq = [13 + x for x in cumulative(lq)]
    n = cq[-1] + 29
    q, k, v = (normal(s, n, 2, d, dtype=DT[dtype]) for s in (1, 2, 3))
    for t in (q, k, v):
        t[:13] = math.nan
        t[cq[-1]:] = math.nan
        t[cq[1]:cq[2]] = math.nan
    *_, o, _ = run_prompt(dtype, 2, 2, d, lq, lq, seed=0, behind=29, ahead=13, q=q, k=k, v=v)
    assert (o[:13] == 7).all() and (o[cq[-1]:] == 7).all()
    ref, tol = prompt64(q, k, v, cq, cq, d ** -0.5, P_PROMPT[dtype])
    own = [r for s in (0, 2) for r in range(cq[s], cq[s + 1])]
    assert_within(o[own], ref[own], tol[own], "neighbours of a NaN sequence")


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("f32", 2, 1, 64), ("bf16", 4, 1, 128), ("bf16", 4, 1, 64),
                                            ("bf16", 2, 2, 64)])
def test_prompt_masked_values_count_for_nothing(dtype, Hq, Hkv, d):
    # keys that a query does not see yet hold the largest finite values, and scores beyond all others
    n, seen = 300, 170
    q, k, v = (normal(s, n, h, d, dtype=DT[dtype]) for s, h in ((1, Hq), (2, Hkv), (3, Hkv)))
    v[seen:] = torch.finfo(DT[dtype]).max
    k[seen:] *= 100
    o = run_prompt(dtype, Hq, Hkv, d, [n], [n], seed=0, q=q, k=k, v=v)[5]
    ref, tol = prompt64(q[:seen], k[:seen], v[:seen], [0, seen], [0, seen], d ** -0.5, P_PROMPT[dtype])
    assert_within(o[:seen], ref, tol, "masked values")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_large_logits_and_scale(dtype):
    # scores of several hundred with a running maximum that keeps growing, and a scale of the caller's
    lq, d = [300], 128
    q, k, v, cq, ck, o, _ = run_prompt(dtype, 2, 1, d, lq, lq, seed=5, scale=0.5)
    ref, tol = prompt64(q, k, v, cq, ck, 0.5, P_PROMPT[dtype])
    assert_within(o, ref, tol, "scale")
    ramp = torch.linspace(0.1, 6.0, 300, device="cuda")[:, None, None]
    k2 = (torch.ones((300, 1, d), device="cuda") * ramp).to(DT[dtype])
    q2 = torch.ones((300, 2, d), device="cuda", dtype=DT[dtype])
    q, k, v, cq, ck, o, _ = run_prompt(dtype, 2, 1, d, lq, lq, seed=5, q=q2, k=k2)
    ref, tol = prompt64(q, k, v, cq, ck, d ** -0.5, P_PROMPT[dtype])
    assert_within(o, ref, tol, "growing maximum")


# one CTA per item, the list, keys split over a cluster, a group per tile; each with key tiles after the first
@pytest.mark.parametrize("lens", [[(70, 70), (300, 310), (1, 400)], [(900, 900)] * 10 + [(3000, 3100)],
                                  [(5, 5000), (200, 3333)], [(40, 60)] * 75 + [(20, 900)]])
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("scale", [2.0 ** 18, 1e9, 1e30])
def test_prompt_scales_that_leave_one_key(dtype, Hq, Hkv, d, lens, scale):
    # scores are whole numbers, exact in fp32, in random order and each there twice; odd heads see them negated.  All
    # weights but the largest are exactly 0; the mean of its values is off by the rounding of each weight and of the
    # result, as in paged_ref
    dt, G = DT[dtype], Hq // Hkv
    cq, ck = cumulative([a for a, _ in lens]), cumulative([b for _, b in lens])
    g = torch.Generator().manual_seed(len(lens))
    order = torch.cat([torch.stack([torch.randperm(b, generator=g) // 2 for _ in range(Hkv)], 1) for _, b in lens]).cuda()
    k = torch.zeros((ck[-1], Hkv, d), device="cuda")
    k[..., 0], k[..., 1] = (order // 256).float(), (order % 256).float()
    sign = 1.0 - 2.0 * (torch.arange(Hq, device="cuda") % 2)
    q = torch.zeros((cq[-1], Hq, d), device="cuda")
    q[..., 0], q[..., 1] = 256 * sign, sign
    v = normal(3, ck[-1], Hkv, d, dtype=dt)
    o = run_prompt(dtype, Hq, Hkv, d, [a for a, _ in lens], [b for _, b in lens], seed=0, scale=scale, q=q.to(dt),
                   k=k.to(dt), v=v)[5].view(-1, Hq, d)
    for s in range(len(lens)):
        a, b, c, e = cq[s], cq[s + 1], ck[s], ck[s + 1]
        see = torch.arange(e - c, device="cuda") <= torch.arange(b - a, device="cuda")[:, None] + (e - c) - (b - a)
        for h in range(Hq):
            z = torch.where(see, (order[c:e, h // G] * sign[h]).double(), -math.inf)
            w = ((z == z.amax(1, keepdim=True)) & see).double()
            w /= w.sum(1, keepdim=True)
            x = v[c:e, h // G].double()
            ref = w @ x
            tol = HALF[dt] * ref.abs() + (P_PROMPT[dtype] + 2.0 ** -20) * (w @ x.abs())
            assert_within(o[a:b, h], ref, tol, f"sequence {s} head {h}")


@pytest.mark.parametrize("dtype,Hq,Hkv", [("bf16", 8, 2), ("f32", 2, 2), ("f32", 8, 2), ("f32", 10, 1)])
@pytest.mark.parametrize("scale", [2.0 ** 18, 1e9, 1e30])
def test_decode_scales_that_leave_one_key(dtype, Hq, Hkv, scale):
    # as above, over pages: whole-number scores, each twice
    dt, page, lens, G = DT[dtype], 32, [700, 1, 70, 4000], Hq // Hkv
    _, kp, vp, table = make_cache(dtype, Hq, Hkv, 64, page, lens, seed=3)
    plan = plan_for(dtype, Hq, Hkv, 64, page=page, pages=kp.shape[1], rows=len(lens), width=len(table[0]), scale=scale)
    g = torch.Generator().manual_seed(1)
    order = [torch.stack([torch.randperm(n, generator=g) // 2 for _ in range(Hkv)], 1).cuda() for n in lens]
    for ids, x, n in zip(table, order, lens):
        for e in range(-(-n // page)):
            part = x[e * page:(e + 1) * page].T
            kp[0, ids[e], :, :part.shape[1]] = 0
            kp[0, ids[e], :, :part.shape[1], 0] = (part // 256).to(dt)
            kp[0, ids[e], :, :part.shape[1], 1] = (part % 256).to(dt)
    sign = 1.0 - 2.0 * (torch.arange(Hq, device="cuda") % 2)
    q = torch.zeros((len(lens), Hq, 64), device="cuda")
    q[..., 0], q[..., 1] = 256 * sign, sign
    o = torch.full((len(lens), Hq * 64), 7.0, dtype=dt, device="cuda")
    mono.paged_attend(plan, 0, q.to(dt), ints(table), ints(lens), o, kp, vp, plan.workspace())
    o = o.view(-1, Hq, 64)
    for r, n in enumerate(lens):
        v = rows_of(vp[0], table[r][:-(-n // page)], page, n).double()
        for h in range(Hq):
            z = order[r][:, h // G] * sign[h]
            x = v[z == z.max(), h // G]
            ref = x.mean(0)
            tol = HALF[dt] * ref.abs() + (P_DECODE[dtype] + 2.0 ** -20) * x.abs().mean(0)
            assert_within(o[r, h], ref, tol, f"row {r} head {h}")


@pytest.mark.parametrize("lens", [[(70, 70), (300, 310), (1, 400)], [(900, 900)] * 10 + [(3000, 3100)],
                                  [(5, 5000), (200, 3333)], [(40, 60)] * 75 + [(20, 900)]])
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("scale", [1e-30, 3e-46, 1e-300])
def test_prompt_scales_that_leave_all_keys_equal(dtype, Hq, Hkv, d, lens, scale):
    # the mean of the values; the last two scales are below the least that fp32 has
    lq, lk = [a for a, _ in lens], [b for _, b in lens]
    q, k, v, cq, ck, o, _ = run_prompt(dtype, Hq, Hkv, d, lq, lk, seed=31, scale=scale)
    ref, tol = prompt64(q, k, v, cq, ck, scale, P_PROMPT[dtype])
    assert_within(o, ref, tol, "mean")


@pytest.mark.parametrize("dtype,Hq,Hkv", [("bf16", 8, 2), ("f32", 2, 2), ("f32", 8, 2), ("f32", 10, 1)])
@pytest.mark.parametrize("scale", [1e-30, 3e-46, 1e-300])
def test_decode_scales_that_leave_all_keys_equal(dtype, Hq, Hkv, scale):
    lens = [700, 1, 0, 2500, 33]
    _, kp, vp, table = make_cache(dtype, Hq, Hkv, 64, 32, lens, seed=3)
    plan = plan_for(dtype, Hq, Hkv, 64, page=32, pages=kp.shape[1], rows=len(lens), width=len(table[0]), scale=scale)
    q = normal(5, len(lens), Hq, 64, dtype=DT[dtype], sd=1.5)
    o = torch.full((len(lens), Hq * 64), 7.0, dtype=DT[dtype], device="cuda")
    mono.paged_attend(plan, 0, q, ints(table), ints(lens), o, kp, vp, plan.workspace())
    ref, tol = decode64(q, kp[0], vp[0], table, lens, scale, P_DECODE[dtype])
    assert_within(o, ref, tol, "mean")


@pytest.mark.parametrize("lens", [[(70, 70), (300, 310), (1, 400)], [(900, 900)] * 10 + [(3000, 3100)],
                                  [(5, 5000), (200, 3333)], [(40, 60)] * 75 + [(20, 900)]])
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("first", [0, 5, 18])
def test_prompt_scores_that_are_not_finite_show(dtype, Hq, Hkv, d, lens, what, first):
    # one key of each sequence, at other places of a tile from sequence to sequence, gives NaN or infinite scores: the
    # rows that see it are NaN, all others have the bits that they have without it
    dt, G = DT[dtype], Hq // Hkv
    cq, ck = cumulative([a for a, _ in lens]), cumulative([b for _, b in lens])
    q, k, v = (normal(s, n, h, d, dtype=dt) for s, n, h in ((1, cq[-1], Hq), (2, ck[-1], Hkv), (3, ck[-1], Hkv)))
    q[..., 3] = q[..., 3].abs() + 0.5
    run = lambda k: run_prompt(dtype, Hq, Hkv, d, [a for a, _ in lens], [b for _, b in lens], seed=0, q=q, k=k, v=v)[5]
    want = run(k).view(-1, Hq, d)
    k = k.clone()
    hit = torch.zeros((cq[-1], Hq), dtype=torch.bool, device="cuda")
    for s, (lq, lk) in enumerate(lens):
        j, h = (first + 37 * s) % lk, s % Hkv
        k[ck[s] + j, h, 3] = what
        hit[cq[s]:cq[s + 1], h * G:(h + 1) * G] = (torch.arange(lq, device="cuda") + lk - lq >= j)[:, None]
    got = run(k).view(-1, Hq, d)
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("dtype,Hq,Hkv", [("bf16", 8, 2), ("f32", 2, 2), ("f32", 8, 2), ("f32", 10, 1)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_decode_scores_that_are_not_finite_show(dtype, Hq, Hkv, what):
    lens = [700, 1, 70, 2500, 33, 64]
    plan, kp, vp, table = make_cache(dtype, Hq, Hkv, 64, 32, lens, seed=3)
    q = normal(5, len(lens), Hq, 64, dtype=DT[dtype], sd=1.5)
    q[..., 3] = q[..., 3].abs() + 0.5
    outs = []
    for bad in (False, True):
        for r, j in ((0, 690), (1, 0), (3, 5), (4, 18)):
            if bad:
                kp[0, table[r][j // 32], :, j % 32, 3] = what
        o = torch.full((len(lens), Hq * 64), 7.0, dtype=DT[dtype], device="cuda")
        mono.paged_attend(plan, 0, q, ints(table), ints(lens), o, kp, vp, plan.workspace())
        outs.append(o)
    assert torch.isnan(outs[1][[0, 1, 3, 4]]).all() and torch.equal(outs[0][[2, 5]], outs[1][[2, 5]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_bad_cumulative_lengths_stay_inside(dtype):
    # lengths that point outside the packed rows are cut to them
    d = 64
    q, k, v = (normal(s, 50, 2, d, dtype=DT[dtype]) for s in (1, 2, 3))
    o = torch.full((50, 2 * d), 7.0, dtype=DT[dtype], device="cuda")
    plan = plan_for(dtype, 2, 2, d, rows=3, tokens=50)
    ws = plan.workspace()
    mono.prompt_attend(plan, q, k, v, ints([-9, 20, 10, 4000]), ints([0, 20, 20, 4000]), o, ws)
    assert torch.isfinite(o.float()).all()
    assert mono.paged_stats(plan, ws, check=False)["device_error"] in (0, 7)


@pytest.mark.parametrize("dtype,heads", [("f32", 2), ("bf16", 2), ("bf16", 64)])  # 64: by way of the tile list
@pytest.mark.parametrize("cu_q,cu_k,spans", [
    # (queries, keys) of each sequence once its lengths are cut to the 50 packed rows
    ([-9, 20, 30, 4000], [0, 20, 20, 4000], [((0, 20), (0, 20)), ((20, 30), (20, 20)), ((30, 50), (20, 50))]),
    ([0, 30, 20, 20], [0, 30, 20, 20], [((0, 30), (0, 30))]),
    ([4, 30, 30, 40], [-3, 30, 30, 99], [((4, 30), (0, 30)), ((30, 40), (30, 50))]),
    ([60, 70, 80, 90], [0, 20, 30, 50], []),
    ([0, 20, 30, 50], [90, 80, 30, 50], [((0, 20), (50, 50)), ((20, 30), (50, 50)), ((30, 50), (30, 50))])])
def test_prompt_bad_cumulative_lengths_are_cut_to_the_rows(dtype, heads, cu_q, cu_k, spans):
    q, k, v = (normal(s, 50, heads, 64, dtype=DT[dtype]) for s in (1, 2, 3))
    o = torch.full((50, heads * 64), 7.0, dtype=DT[dtype], device="cuda")
    plan = plan_for(dtype, heads, heads, 64, rows=3, tokens=50)
    ws = plan.workspace()
    mono.prompt_attend(plan, q, k, v, ints(cu_q), ints(cu_k), o, ws)
    assert mono.paged_stats(plan, ws, check=False)["device_error"] == 7
    free = torch.ones(50, dtype=torch.bool, device="cuda")
    for (a, b), (c, e) in spans:
        ref, tol = prompt64(q[a:b], k[c:e], v[c:e], [0, b - a], [0, e - c], 0.125, P_PROMPT[dtype])
        assert_within(o[a:b], ref, tol, f"queries {a} to {b}")
        free[a:b] = False
    assert (o[free] == 7).all()


@pytest.mark.parametrize("dtype,heads", [("f32", 2), ("bf16", 2), ("bf16", 64)])  # 64: by way of the tile list
@pytest.mark.parametrize("cu_q,cu_k", [
    ([-9, 20, 30, 50], [0, 20, 30, 50]), ([0, 20, 10, 50], [0, 20, 30, 50]), ([0, 20, 20, 51], [0, 20, 30, 50]),
    ([0, 20, 30, 50], [0, 20, 30, 51]), ([0, 20, 30, 50], [0, 25, 20, 50]), ([0, 20, 30, 50], [-1, 20, 30, 50])])
def test_prompt_bad_cumulative_lengths_are_recorded(dtype, heads, cu_q, cu_k):
    q, k, v = (normal(s, 50, heads, 64, dtype=DT[dtype]) for s in (1, 2, 3))
    o = torch.empty((50, heads * 64), dtype=DT[dtype], device="cuda")
    plan = plan_for(dtype, heads, heads, 64, rows=3, tokens=50)
    ws = plan.workspace()
    mono.prompt_attend(plan, q, k, v, ints(cu_q), ints(cu_k), o, ws)
    assert mono.paged_stats(plan, ws, check=False)["device_error"] == 7
    mono.prompt_attend(plan, q, k, v, ints([3, 20, 20, 49]), ints([1, 1, 30, 50]), o, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0


# one CTA per item; by way of the tile list; keys split over clusters; a group per tile
PROMPT_PATHS = [(*heads, lens) for heads in (("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("f32", 4, 2, 64))
                for lens in ([(70, 70), (300, 310), (1, 400)], [(900, 900)] * 10 + [(3000, 3100)],
                             [(5, 5000), (200, 3333)], [(40, 60)] * 75 + [(20, 900)])]


@pytest.mark.parametrize("dtype,Hq,Hkv,d,lens", PROMPT_PATHS)
def test_prompt_captured_and_replayed(dtype, Hq, Hkv, d, lens):
    # two calls in a row on one workspace, captured; the replay sees the inputs and the lengths of its time
    dt = DT[dtype]
    cq, ck = cumulative([a for a, _ in lens]), cumulative([b for _, b in lens])
    plan = plan_for(dtype, Hq, Hkv, d, rows=len(lens), tokens=cq[-1])
    ws = plan.workspace()
    draw = lambda s: [normal(s + x, n, h, d, dtype=dt)
                      for x, (n, h) in enumerate(((cq[-1], Hq), (ck[-1], Hkv), (ck[-1], Hkv)))]
    sets = [draw(s) for s in (1, 11)]
    fixed = [[torch.empty_like(t) for t in x] for x in sets]
    cus, cuk = ints(cq), ints(ck)
    outs = [torch.empty((cq[-1], Hq * d), dtype=dt, device="cuda") for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for x, o in zip(fixed, outs):
            mono.prompt_attend(plan, *x, cus, cuk, o, ws)
    for turn in range(2):
        if turn:                                                  # a token of the first sequence falls away
            cq = [0] + [c - 1 for c in cq[1:]]
            cus.copy_(ints(cq))
        for a, b in zip(fixed, sets[::1 - 2 * turn]):
            for x, y in zip(a, b):
                x.copy_(y)
        want = []
        for x in fixed:
            o = torch.full_like(outs[0], 7.0)
            mono.prompt_attend(plan, *x, cus, cuk, o, ws)
            want.append(o)
        for o in outs:
            o.fill_(7.0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert mono.paged_stats(plan, ws)["device_error"] == 0


@pytest.mark.parametrize("dtype,Hq,Hkv,d,lens", PROMPT_PATHS)
def test_prompt_on_two_streams_at_once(dtype, Hq, Hkv, d, lens):
    dt = DT[dtype]
    cq, ck = cumulative([a for a, _ in lens]), cumulative([b for _, b in lens])
    plan = plan_for(dtype, Hq, Hkv, d, rows=len(lens), tokens=cq[-1])
    k, v = (normal(s, ck[-1], Hkv, d, dtype=dt) for s in (2, 3))
    qs = [normal(s, cq[-1], Hq, d, dtype=dt) for s in (5, 6)]
    wss = [plan.workspace() for _ in range(2)]
    cus, cuk = ints(cq), ints(ck)
    want = [torch.empty((cq[-1], Hq * d), dtype=dt, device="cuda") for _ in range(2)]
    for q, o in zip(qs, want):
        mono.prompt_attend(plan, q, k, v, cus, cuk, o, wss[0])
    outs = [torch.empty_like(o) for o in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for q, o, ws, st in zip(qs, outs, wss, streams):
            mono.prompt_attend(plan, q, k, v, cus, cuk, o, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all(mono.paged_stats(plan, ws)["device_error"] == 0 for ws in wss)


# ---------------------------------------------------------------------------
# one new token over the paged cache
# ---------------------------------------------------------------------------
def make_cache(dtype, Hq, Hkv, d, page, lens, seed, layers=1, spare=3, width=None, garbage=math.nan):
    """Pools whose rows behind every sequence, and whose unused pages, hold `garbage`; the table in random order."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    width = max(counts + [1]) + 1 if width is None else width
    ids = list(range(pages))
    random.Random(seed).shuffle(ids)
    table, at = [], 0
    for c in counts:
        table.append(ids[at:at + c] + [-1] * (width - c))
        at += c
    plan = plan_for(dtype, Hq, Hkv, d, page=page, pages=pages, layers=layers, rows=len(lens), width=width)
    kp, vp = (torch.full(plan.pool_shape, garbage, dtype=DT[dtype], device="cuda") for _ in range(2))
    for i, n in enumerate(lens):
        for e in range(counts[i]):
            m = min(page, n - e * page)
            for pool, s, sd in ((kp, 2 * seed, 1.5), (vp, 2 * seed + 1, 1.0)):
                pool[:, table[i][e], :, :m] = normal(s + 97 * (i * 1000 + e), layers, Hkv, m, d, dtype=DT[dtype], sd=sd)
    return plan, kp, vp, table


LENS = {
    "edges": [0, 1, 15, 16, 17, 63, 64, 65, 128, 129],
    "one_short": [3],
    "one_long": [4321],
    "ragged": [700, 1, 0, 2500, 33, 31, 0, 999],
    "all_empty": [0, 0, 0],
}


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("dtype,Hq,Hkv,d,page", [
    ("bf16", 4, 4, 64, 16), ("bf16", 8, 2, 128, 64), ("bf16", 5, 1, 128, 128), ("bf16", 32, 2, 64, 32),
    ("bf16", 20, 1, 128, 16), ("bf16", 12, 1, 64, 128),
    ("f32", 3, 3, 64, 16), ("f32", 8, 2, 128, 32), ("f32", 10, 2, 64, 64), ("f32", 17, 1, 128, 128),
    ("f32", 16, 1, 128, 16)])
def test_decode(dtype, Hq, Hkv, d, page, name):
    lens = LENS[name]
    plan, kp, vp, table = make_cache(dtype, Hq, Hkv, d, page, lens, seed=3)
    q = normal(5, len(lens), Hq, d, dtype=DT[dtype], sd=1.5)
    o = torch.full((len(lens), Hq * d), 7.0, dtype=DT[dtype], device="cuda")
    ws = plan.workspace()
    mono.paged_attend(plan, 0, q, ints(table), ints(lens), o, kp, vp, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0
    ref, tol = decode64(q, kp[0], vp[0], table, lens, d ** -0.5, P_DECODE[dtype])
    assert_within(o, ref, tol, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_many_rows_and_layers(dtype):
    # more rows than a CTA has threads, several layers, a workspace that earlier calls left full
    r = random.Random(4)
    lens = [r.choice([0, 1, 40, 64, 90, 300]) for _ in range(333)]
    plan, kp, vp, table = make_cache(dtype, 4, 2, 64, 32, lens, seed=9, layers=3)
    q = normal(5, len(lens), 4, 64, dtype=DT[dtype], sd=1.5)
    ws = plan.workspace()
    ws[256:] = 255
    o = torch.empty((len(lens), 4 * 64), dtype=DT[dtype], device="cuda")
    for layer in (2, 0):
        mono.paged_attend(plan, layer, q, ints(table), ints(lens), o, kp, vp, ws)
        ref, tol = decode64(q, kp[layer], vp[layer], table, lens, 64 ** -0.5, P_DECODE[dtype])
        assert_within(o, ref, tol, f"layer {layer}")


@pytest.mark.parametrize("dtype,Hq,Hkv", [("bf16", 40, 1), ("f32", 2, 2)])
def test_decode_very_many_rows(dtype, Hq, Hkv):
    # more rows than the join counts itself; more than two chunks of query heads
    r = random.Random(4)
    lens = [r.choice([0, 1, 7, 16, 33, 70]) for _ in range(1200)]
    lens[700] = 3000
    plan, kp, vp, table = make_cache(dtype, Hq, Hkv, 64, 32, lens, seed=9)
    q = normal(5, len(lens), Hq, 64, dtype=DT[dtype], sd=1.5)
    ws = plan.workspace()
    o = torch.full((len(lens), Hq * 64), 7.0, dtype=DT[dtype], device="cuda")
    mono.paged_attend(plan, 0, q, ints(table), ints(lens), o, kp, vp, ws)
    pick = [0, 1, 2, 3, 699, 700, 701, 1198, 1199] + list(range(10, 1200, 97))
    ref, tol = decode64(q[pick], kp[0], vp[0], [table[i] for i in pick], [lens[i] for i in pick], 64 ** -0.5,
                        P_DECODE[dtype])
    assert_within(o[pick], ref, tol, "rows")
    assert torch.isfinite(o.float()).all()


def test_decode_on_two_streams_at_once():
    # two calls that overlap on the GPU, each with a workspace of its own
    plan, kp, vp, table = make_cache("bf16", 8, 2, 128, 64, [3000, 70, 2000], seed=2)
    args = (ints(table), ints([3000, 70, 2000]))
    qs = [normal(s, 3, 8, 128, dtype=torch.bfloat16) for s in (5, 6)]
    outs = [torch.empty((3, 1024), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wss = [plan.workspace() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, o, ws, st in zip(qs, outs, wss, streams):
            mono.paged_attend(plan, 0, q, *args, o, kp, vp, ws, stream=st)
    torch.cuda.synchronize()
    for q, o in zip(qs, outs):
        ref, tol = decode64(q, kp[0], vp[0], table, [3000, 70, 2000], 128 ** -0.5, P_DECODE["bf16"])
        assert_within(o, ref, tol, "stream")


def test_decode_twice_gives_the_same_bits():
    plan, kp, vp, table = make_cache("bf16", 8, 2, 128, 64, [5000, 70, 9000], seed=2)
    q = normal(5, 3, 8, 128, dtype=torch.bfloat16)
    ws = plan.workspace()
    outs = []
    for _ in range(2):
        o = torch.empty((3, 1024), dtype=torch.bfloat16, device="cuda")
        mono.paged_attend(plan, 0, q, ints(table), ints([5000, 70, 9000]), o, kp, vp, ws)
        outs.append(o)
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_bad_pages_and_lengths(dtype):
    # a page id outside the pool is not followed: its tokens are absent; lengths are cut to the table
    lens, page = [200, 64, 100], 32
    plan, kp, vp, table = make_cache(dtype, 4, 2, 64, page, lens, seed=6)
    bad = [list(r) for r in table]
    bad[0][2], bad[1][0], bad[1][1] = -1, plan.cfg.pages, 1 << 30
    q = normal(5, 3, 4, 64, dtype=DT[dtype], sd=1.5)
    o = torch.empty((3, 256), dtype=DT[dtype], device="cuda")
    ws = plan.workspace()
    mono.paged_attend(plan, 0, q, ints(bad), ints(lens), o, kp, vp, ws)
    st = mono.paged_stats(plan, ws, check=False)
    assert st["device_error"] == 6 and mono.STATUS[st["status"]] == "MONO_ERR_DEVICE"
    assert mono.paged_stats(plan, ws)["device_error"] == 0          # read once, cleared
    short = [table[0][:2] + table[0][3:], [], table[2]]
    ref, tol = decode64(q, kp[0], vp[0], short, [168, 0, 100], 64 ** -0.5, P_DECODE[dtype])
    assert_within(o, ref, tol, "absent pages")
    mono.paged_attend(plan, 0, q, ints(table), ints([-5, 64, 100]), o, kp, vp, ws)
    assert mono.paged_stats(plan, ws, check=False)["device_error"] == 7
    assert (o[0] == 0).all()


def test_decode_offsets_beyond_32_bits():
    # K and V pools of 2^32 elements each and more: pages at both ends
    d, Hkv, page = 128, 8, 128
    pages = (1 << 32) // (d * Hkv * page) + 3
    plan = plan_for("bf16", 16, Hkv, d, page=page, pages=pages, rows=2, width=3)
    kp, vp = (torch.empty(plan.pool_shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = [[pages - 1, 0, pages - 2], [pages - 3, 1, -1]]
    lens = [300, 129]
    new = [normal(s, sum(lens), Hkv, d, dtype=torch.bfloat16) for s in (1, 2)]
    ws = plan.workspace()
    mono.paged_append(plan, 0, *new, ints(cumulative(lens)), ints(table), ints(lens), kp, vp, ws)
    q = normal(5, 2, 16, d, dtype=torch.bfloat16)
    o = torch.empty((2, 16 * d), dtype=torch.bfloat16, device="cuda")
    mono.paged_attend(plan, 0, q, ints(table), ints(lens), o, kp, vp, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0
    for i, (a, b) in enumerate(((0, 300), (300, 429))):
        for h in range(16):
            ref, tol = attend64(q[i, h:h + 1].double(), new[0][a:b, h // 2].double(), new[1][a:b, h // 2].double(),
                                torch.tensor([b - a], device="cuda"), d ** -0.5, P_DECODE["bf16"], torch.bfloat16)
            assert_within(o[i, h * d:(h + 1) * d], ref[0], tol[0], f"row {i} head {h}")


# ---------------------------------------------------------------------------
# writing into pages
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,Hkv,d,page", [("bf16", 4, 128, 64), ("f32", 3, 64, 16), ("bf16", 1, 64, 128),
                                              ("f32", 16, 128, 32)])
@pytest.mark.parametrize("lens,new", [([5], [5]), ([1, 64, 65, 200, 0], [1, 1, 1, 1, 0]),
                                      ([300, 40, 0, 129, 64], [299, 3, 0, 129, 0]), ([1] * 70, [1] * 70)])
def test_append(dtype, Hkv, d, page, lens, new):
    plan, kp, vp, table = make_cache(dtype, Hkv, Hkv, d, page, lens, seed=8, layers=2, garbage=3.0)
    cu, N = cumulative(new), sum(new)
    k, v = (normal(s, N + 4, Hkv, d, dtype=DT[dtype]) for s in (21, 22))  # four rows behind the last sequence
    want = [kp.clone(), vp.clone()]
    for i, n in enumerate(lens):
        for t in range(new[i]):
            pos = n - new[i] + t
            for w, x in zip(want, (k, v)):
                w[1, table[i][pos // page], :, pos % page] = x[cu[i] + t]
    ws = plan.workspace()
    mono.paged_append(plan, 1, k, v, ints(cu), ints(table), ints(lens), kp, vp, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_append_skips_what_it_cannot_place():
    plan, kp, vp, table = make_cache("bf16", 2, 2, 64, 16, [40, 20, 30], seed=8, garbage=3.0)
    table[0][1], table[1][0] = -1, plan.cfg.pages
    k, v = (normal(s, 90, 2, 64, dtype=torch.bfloat16) for s in (21, 22))
    cu, lens = [0, 40, 60, 90], [40, 20, 10]           # row 2: 30 new tokens, but a length of 10
    want = kp.clone()
    for i, n in enumerate(lens):
        for t in range(cu[i + 1] - cu[i]):
            pos = n - (cu[i + 1] - cu[i]) + t
            if pos >= 0 and 0 <= table[i][pos // 16] < plan.cfg.pages:
                want[0, table[i][pos // 16], :, pos % 16] = k[cu[i] + t]
    ws = plan.workspace()
    mono.paged_append(plan, 0, k, v, ints(cu), ints(table), ints(lens), kp, vp, ws)
    assert mono.paged_stats(plan, ws, check=False)["device_error"] in (6, 7)
    assert torch.equal(kp, want)


@pytest.mark.parametrize("cu", [[-1, 40, 60, 90], [0, 40, 30, 90], [0, 40, 60, 91]])
def test_append_records_bad_cumulative_lengths(cu):
    plan, kp, vp, table = make_cache("bf16", 2, 2, 64, 16, [100, 100, 100], seed=8)
    k, v = (normal(s, 90, 2, 64, dtype=torch.bfloat16) for s in (21, 22))
    ws = plan.workspace()
    mono.paged_append(plan, 0, k, v, ints(cu), ints(table), ints([100, 100, 100]), kp, vp, ws)
    assert mono.paged_stats(plan, ws, check=False)["device_error"] == 7
    mono.paged_append(plan, 0, k, v, ints([2, 40, 40, 88]), ints(table), ints([100, 100, 100]), kp, vp, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0


# ---------------------------------------------------------------------------
# the page table's step and closing the holes
# ---------------------------------------------------------------------------
def do_update(plan, table, lens, parents, grow, kp, vp, ws):
    w = plan.cfg.width
    t_in = ints(table).view(len(lens), w)
    t_out = torch.full((len(parents), w), -9, dtype=torch.int32, device="cuda")
    l_out = torch.full((len(parents),), -9, dtype=torch.int32, device="cuda")
    mono.paged_update(plan, t_in, ints(lens), ints(parents), ints(grow), t_out, l_out, kp, vp, ws)
    return t_out.tolist(), l_out.tolist()


UPDATES = {
    "fork": ([70, 64], [0, 0, 0, 1, 1], [0, 1, 2, 0, 1]),
    "drop_and_new": ([70, 64, 10], [-1, 2, -1], [40, 1, 0]),
    "cut_back": ([70, 64, 33], [0, 1, 2], [-6, -64, -100]),
    "cut_into_a_shared_page": ([100, 100], [0, 0, 0, 1], [-30, 5, -31, -99]),
    "nothing_in": ([], [-1, -1], [5, 0]),
    "exact_pages": ([64, 32], [0, 0, 1, 1], [0, 32, -32, 1]),
}


@pytest.mark.parametrize("name", list(UPDATES))
@pytest.mark.parametrize("page,layers", [(32, 1), (16, 3)])
def test_update(name, page, layers):
    lens, parents, grow = UPDATES[name]
    plan0, kp, vp, table = make_cache("bf16", 2, 2, 64, page, lens or [1], seed=5, layers=layers, spare=40, width=9,
                                      garbage=3.0)
    if not lens:
        table = []
    plan = plan_for("bf16", 2, 2, 64, page=page, pages=plan0.cfg.pages, layers=layers, rows=8, width=9)
    want_t, want_l, copies, short = update_ref(table, lens, parents, grow, plan.cfg.pages, page, 9)
    want = [kp.clone(), vp.clone()]
    for a, b in copies:
        for w in want:
            w[:, b] = w[:, a]
    ws = plan.workspace()
    got_t, got_l = do_update(plan, table, lens, parents, grow, kp, vp, ws)
    st = mono.paged_stats(plan, ws)
    assert got_t == want_t and got_l == want_l
    assert (st["pages_copied"], st["pages_short"]) == (len(copies), short) and short == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_update_many_steps_against_lists():
    # a long run of random steps: the table equals the lists', and no row writes where another one reads
    r = random.Random(12)
    page, width, pages, rows = 16, 12, 700, 40
    plan = plan_for("f32", 1, 1, 64, page=page, pages=pages, rows=rows, width=width)
    kp, vp = plan.pools()
    ws = plan.workspace()
    table, lens = [], []
    for step in range(25):
        n_out = r.randrange(1, rows + 1)
        parents = [r.randrange(-1, len(lens)) for _ in range(n_out)]
        grow = [r.choice([0, 1, 1, 1, 17, -1, -20, 40]) for _ in parents]
        grow = [min(g, width * page - (lens[p] if p >= 0 else 0)) for p, g in zip(parents, grow)]
        want_t, want_l, copies, short = update_ref(table, lens, parents, grow, pages, page, width)
        table_, lens_ = do_update(plan, table, lens, parents, grow, kp, vp, ws)
        assert (table_, lens_) == (want_t, want_l), f"step {step}"
        assert short == 0 and mono.paged_stats(plan, ws)["pages_copied"] == len(copies)
        old = [lens[p] if p >= 0 else 0 for p in parents]
        table, lens = table_, lens_
        for i, (a, b) in enumerate(zip(old, lens)):       # pages that row i is about to write
            for e in range(min(a, b) // page, -(-b // page)):
                assert sum(table[i][e] in row for row in table) == 1 or a >= b
    held = {p for row, n in zip(table, lens) for p in row[:-(-n // page)]}
    want_t, moves, live = compact_ref(table, lens, page, width)
    out = torch.empty((len(lens), width), dtype=torch.int32, device="cuda")
    mono.paged_compact(plan, ints(table), ints(lens), out, kp, vp, ws)
    st = mono.paged_stats(plan, ws)
    assert out.tolist() == want_t and st["pages_held"] == live == len(held) and st["pages_copied"] == len(moves)


@pytest.mark.parametrize("pages,rows,width", [(40001, 60, 30), (3000, 250, 300)])
def test_update_and_compact_of_large_pools_and_tables(pages, rows, width):
    # beyond the sizes that one block plans alone: many pages, or many table entries
    r = random.Random(pages)
    page = 16
    plan = plan_for("f32", 1, 1, 64, page=page, pages=pages, rows=rows, width=width)
    kp, vp = (normal(s, *plan.pool_shape) for s in (1, 2))
    ws = plan.workspace()
    lens = [r.choice([0, 5, 16, 100, 130]) for _ in range(rows)]
    ids = r.sample(range(pages), pages // 2)
    table = [[ids.pop() for _ in range(-(-n // page))] + [-1] * (width - -(-n // page)) for n in lens]
    parents = [r.randrange(-1, rows) for _ in range(rows)]
    grow = [r.choice([0, 1, 20, -7]) for _ in range(rows)]
    want_t, want_l, copies, short = update_ref(table, lens, parents, grow, pages, page, width)
    want = [kp.clone(), vp.clone()]
    for a, b in copies:
        for w in want:
            w[:, b] = w[:, a]
    assert copies and do_update(plan, table, lens, parents, grow, kp, vp, ws) == (want_t, want_l) and short == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert mono.paged_stats(plan, ws)["pages_copied"] == len(copies)
    final_t, moves, live = compact_ref(want_t, want_l, page, width)
    for a, b in moves:
        for w in want:
            w[:, b] = w[:, a]
    out = torch.empty((rows, width), dtype=torch.int32, device="cuda")
    mono.paged_compact(plan, ints(want_t), ints(want_l), out, kp, vp, ws)
    assert out.tolist() == final_t and mono.paged_stats(plan, ws)["pages_held"] == live
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@pytest.mark.parametrize("pages,rows,width", [(120, 20, 12), (40001, 60, 30)])
def test_page_steps_captured_and_replayed(pages, rows, width):
    # a step and a compaction in one graph, planned in one block and with marks in memory, replayed from other tables
    r = random.Random(rows)
    page = 16
    plan = plan_for("f32", 1, 1, 64, page=page, pages=pages, rows=rows, width=width)
    kp, vp = (normal(s, *plan.pool_shape) for s in (1, 2))
    ws = plan.workspace()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    t_in, l_in, par, grow = i32(rows, width), i32(rows), i32(rows), i32(rows)
    t_out, l_out, t_end = i32(rows, width), i32(rows), i32(rows, width)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        mono.paged_update(plan, t_in, l_in, par, grow, t_out, l_out, kp, vp, ws)
        mono.paged_compact(plan, t_out, l_out, t_end, kp, vp, ws)
    for _ in range(3):
        lens = [r.choice([0, 5, 16, 30]) for _ in range(rows)]
        ids = r.sample(range(pages), 2 * rows)
        table = [[ids.pop() for _ in range(-(-n // page))] + [-1] * (width - -(-n // page)) for n in lens]
        parents = [r.randrange(-1, rows) for _ in range(rows)]
        grown = [r.choice([0, 1, 20, -7]) for _ in range(rows)]
        for t, x in ((t_in, table), (l_in, lens), (par, parents), (grow, grown)):
            t.copy_(ints(x))
        want_t, want_l, copies, short = update_ref(table, lens, parents, grown, pages, page, width)
        end_t, moves, live = compact_ref(want_t, want_l, page, width)
        want = [kp.clone(), vp.clone()]
        for w in want:
            for a, b in copies + moves:
                w[:, b] = w[:, a]
        graph.replay()
        assert short == 0 and (t_out.tolist(), l_out.tolist(), t_end.tolist()) == (want_t, want_l, end_t)
        assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
        assert mono.paged_stats(plan, ws)["pages_held"] == live


@pytest.mark.parametrize("step", ["update", "compact"])
def test_page_steps_of_two_host_threads(step):
    # pools of different sizes, both beyond the shared memory that a launch gets unasked; a workspace and a stream each
    page, rows, width, n = 16, 4, 4, 400
    start, errors = threading.Barrier(2, timeout=60), []

    def steps(pages):
        try:
            plan = plan_for("f32", 1, 1, 64, page=page, pages=pages, rows=rows, width=width)
            kp, vp = plan.pools()
            ws, stream = plan.workspace(), torch.cuda.Stream()
            table, lens = ints([[9, 5, -1, -1], [3, -1, -1, -1]]), ints([20, 16])
            parents, grow = ints([0, 1]), ints([1, 1])
            t_out = torch.empty((2, width), dtype=torch.int32, device="cuda")
            l_out = torch.empty((2,), dtype=torch.int32, device="cuda")
            torch.cuda.synchronize()
            start.wait()
            for _ in range(n):
                if step == "update":
                    mono.paged_update(plan, table, lens, parents, grow, t_out, l_out, kp, vp, ws, stream=stream)
                else:
                    mono.paged_compact(plan, table, lens, t_out, kp, vp, ws, stream=stream)
            stream.synchronize()
            want = [[9, 5, -1, -1], [3, 0, -1, -1]] if step == "update" else [[2, 1, -1, -1], [0, -1, -1, -1]]
            assert mono.paged_stats(plan, ws, stream=stream)["device_error"] == 0
            return t_out.tolist(), want
        except Exception as e:  # noqa: BLE001  (shown by the assertion below)
            errors.append(e)

    with concurrent.futures.ThreadPoolExecutor(2) as ex:
        got = list(ex.map(steps, (20000, 9000)))
    assert not errors, errors
    for table, want in got:
        assert table == want


def test_update_without_free_pages_and_with_bad_rows():
    page, width = 16, 4
    plan = plan_for("f32", 1, 1, 64, page=page, pages=4, rows=6, width=width)
    kp, vp = plan.pools()
    ws = plan.workspace()
    table, lens = [[2, 0, -1, -1]], [20]
    got = do_update(plan, table, lens, [0, 0, -1], [1, 1, 40], kp, vp, ws)
    want_t, want_l, copies, short = update_ref(table, lens, [0, 0, -1], [1, 1, 40], 4, page, width)
    assert got == (want_t, want_l) and short == 2
    st = mono.paged_stats(plan, ws, check=False)
    assert (st["device_error"], st["pages_short"], st["pages_copied"], st["pages_held"]) == (8, 2, 1, 2)
    # a parent that does not exist, a length beyond the table, a page id outside the pool
    got = do_update(plan, table, lens, [5, 0], [3, 1000], kp, vp, ws)
    assert got[1] == [3, width * page] and mono.paged_stats(plan, ws, check=False)["device_error"] == 7
    got = do_update(plan, [[2, 99, -1, -1]], lens, [0], [0], kp, vp, ws)
    assert got == ([[2, -1, -1, -1]], [20]) and mono.paged_stats(plan, ws, check=False)["device_error"] == 6


def test_update_asks_for_more_than_31_bits_of_pages():
    # rows that together ask for almost 2^32 pages: the first take the pool's, in order, the others none
    page, width, rows, pages = 16, 262142, 16384, 400000
    plan = plan_for("f32", 1, 1, 64, page=page, pages=pages, rows=rows, width=width)
    kp, vp = plan.pools()
    ws = plan.workspace()
    t_out = torch.full((rows, width), -9, dtype=torch.int32, device="cuda")
    l_out = torch.empty((rows,), dtype=torch.int32, device="cuda")
    none = torch.empty((0, width), dtype=torch.int32, device="cuda")
    mono.paged_update(plan, none, ints([]), ints([-1] * rows), ints([width * page] * rows), t_out, l_out, kp, vp, ws)
    st = mono.paged_stats(plan, ws, check=False)
    assert (st["device_error"], st["pages_held"], st["pages_copied"], st["pages_short"]) == (8, 0, 0, 2 ** 31 - 1)
    assert (l_out == width * page).all()
    first = t_out[:2].flatten()
    assert torch.equal(first[:pages], torch.arange(pages, dtype=torch.int32, device="cuda"))
    assert (first[pages:] == -1).all()
    for r in range(2, rows, 2048):                          # (piece by piece: the table is 17 GB)
        assert (t_out[r:r + 2048] == -1).all()


@pytest.mark.parametrize("dtype,Hkv,d,page", [("bf16", 4, 128, 64), ("f32", 1, 64, 16)])
def test_compact_moves_the_data(dtype, Hkv, d, page):
    lens = [200, 5, 0, 333, 64]
    plan, kp, vp, table = make_cache(dtype, Hkv, Hkv, d, page, lens, seed=31, layers=2, spare=60, garbage=3.0)
    table[1] = table[0][:1] + table[1][1:]                # a shared page
    want_t, moves, live = compact_ref(table, lens, page, plan.cfg.width)
    assert moves
    want = [kp.clone(), vp.clone()]
    for a, b in moves:
        for w in want:
            w[:, b] = w[:, a]
    out = torch.empty((len(lens), plan.cfg.width), dtype=torch.int32, device="cuda")
    ws = plan.workspace()
    mono.paged_compact(plan, ints(table), ints(lens), out, kp, vp, ws)
    assert out.tolist() == want_t
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    st = mono.paged_stats(plan, ws)
    assert st["pages_held"] == live and st["pages_copied"] == len(moves)
    again = torch.empty_like(out)
    mono.paged_compact(plan, out, ints(lens), again, kp, vp, ws)
    assert torch.equal(again, out) and mono.paged_stats(plan, ws)["pages_copied"] == 0


def test_refusals_on_the_gpu():
    plan = plan_for("bf16", 4, 2, 64, page=16, pages=4, layers=2, rows=3, width=2, tokens=8)
    ws = plan.workspace()
    kp, vp = plan.pools()
    e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    t, n = e(2, 2, dt=torch.int32), ints([0, 0])
    good = dict(plan=plan, layer=0, Q=e(2, 4, 64), table=t, lens=n, O=e(2, 256), Kp=kp, Vp=vp, ws=ws)
    mono.paged_attend(**good)
    for change, what in [(dict(Q=e(2, 4, 64, dt=torch.float32)), "Q must be"), (dict(Q=e(2, 3, 64)), "shape"),
                         (dict(Q=e(2, 4, 128)[..., ::2]), "contiguous"), (dict(table=e(2, 3, dt=torch.int32)), "shape"),
                         (dict(lens=e(2, dt=torch.int64)), "lens must be"), (dict(layer=2), "layer"),
                         (dict(layer=-1), "layer"), (dict(Kp=kp[:1]), "shape"), (dict(O=e(2, 4, 64)), "shape"),
                         (dict(ws=ws[:256]), "workspace"), (dict(ws=ws.cpu()), "CUDA tensor")]:
        with pytest.raises(ValueError, match=what):
            mono.paged_attend(**{**good, **change})
    with pytest.raises(mono.MonoError):                     # more rows than the plan's
        mono.paged_attend(**{**good, "Q": e(4, 4, 64), "table": e(4, 2, dt=torch.int32), "lens": ints([0] * 4),
                             "O": e(4, 256)})
    shifted = e(2 * 4 * 64 + 4)[4:].view(2, 4, 64)          # 8 bytes off
    with pytest.raises(mono.MonoError) as err:
        mono.paged_attend(**{**good, "Q": shifted})
    assert mono.STATUS[err.value.status] == "MONO_ERR_ALIGN"
    with pytest.raises(mono.MonoError):                     # in place
        mono.paged_update(plan, t, n, ints([0, 1]), ints([0, 0]), t, ints([0, 0]), kp, vp, ws)
    with pytest.raises(mono.MonoError):
        mono.paged_compact(plan, t, n, t, kp, vp, ws)
    with pytest.raises(mono.MonoError):                     # more query tokens than the plan's
        mono.prompt_attend(plan, e(9, 4, 64), e(9, 2, 64), e(9, 2, 64), ints([0, 9]), ints([0, 9]), e(9, 256), ws)
    torch.cuda.synchronize()
    assert mono.paged_stats(plan, ws)["device_error"] == 0


def test_buffers_that_touch_do_not_overlap():
    # everything that a call reads and writes side by side in one allocation
    plan = plan_for("bf16", 4, 2, 64, page=16, pages=4, layers=2, rows=2, width=4, tokens=64)
    block = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    at = [0]

    def take(shape, dtype):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        at[0] += n
        return block[at[0] - n:at[0]].view(dtype).view(shape)

    ws = take((plan.workspace_bytes,), torch.uint8)
    kp, vp, q, o, k, v, po = (take(s, torch.bfloat16) for s in (
        plan.pool_shape, plan.pool_shape, (2, 4, 64), (2, 256), (37, 2, 64), (37, 2, 64), (37, 256)))
    pq = take((37, 4, 64), torch.bfloat16)
    t0, l0, par, grow, t1, l1, cu = (take(s, torch.int32) for s in ((2, 4), (2,), (2,), (2,), (2, 4), (2,), (3,)))
    for x, seed in ((q, 1), (k, 2), (v, 3), (pq, 4)):
        x.copy_(normal(seed, *x.shape, dtype=torch.bfloat16))
    par.fill_(-1)
    grow.copy_(ints([20, 17]))
    cu.copy_(ints([0, 20, 37]))
    mono.paged_update(plan, t0[:0], l0[:0], par, grow, t1, l1, kp, vp, ws)
    mono.prompt_attend(plan, pq, k, v, cu, cu, po, ws)
    mono.paged_append(plan, 1, k, v, cu, t1, l1, kp, vp, ws)
    mono.paged_attend(plan, 1, q, t1, l1, o, kp, vp, ws)
    mono.paged_compact(plan, t1, l1, t0, kp, vp, ws)
    assert mono.paged_stats(plan, ws)["device_error"] == 0
    assert t1.tolist() == t0.tolist() == [[0, 1, -1, -1], [2, 3, -1, -1]] and l1.tolist() == [20, 17]
    ref, tol = prompt64(pq, k, v, [0, 20, 37], [0, 20, 37], 0.125, P_PROMPT["bf16"])
    assert_within(po, ref, tol, "prompt")
    ref, tol = decode64(q, kp[1], vp[1], t1.tolist(), [20, 17], 0.125, P_DECODE["bf16"])
    assert_within(o, ref, tol, "one token")


def test_quick_way_takes_the_usual_calls_and_no_others():
    from learned_product_hash_proj_b200 import _tensor_args as quick
    plan = plan_for("bf16", 4, 1, 64, page=16, pages=4, layers=2, rows=3, width=1, tokens=8)
    ws = plan.workspace()
    kp, vp = plan.pools()
    e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    q, t, n, o = e(1, 4, 64), e(1, 1, dt=torch.int32), ints([0]), e(1, 256)
    good = [plan.quick, 0, q, t, n, o, kp, vp, ws, None]
    side = torch.cuda.Stream()
    odd = torch.as_strided(e(500), (1, 4, 64), (7, 64, 1))          # one row: its stride does not matter
    assert quick.paged_attend(*good) == 0
    for at, usual in ((2, odd), (9, side.cuda_stream), (9, 0), (8, e(ws.numel() + 5, dt=torch.uint8))):
        assert quick.paged_attend(*good[:at], usual, *good[at + 1:]) == 0
    for at, wrong in ((0, None), (1, 2), (1, -1), (1, True), (2, e(1, 4, 128)[..., ::2]), (2, e(1, 4, 64, dt=torch.float16)),
                      (2, e(1, 4, 64, dt=torch.float32)), (2, q.cpu()), (2, e(2, 4, 64)), (2, e(1, 256)),
                      (3, e(1, 2, dt=torch.int32)), (3, e(1, 1, dt=torch.int64)), (3, e(1, 1, dt=torch.uint8)),
                      (4, e(1, 1, dt=torch.int32)), (6, kp[:1]), (6, kp.transpose(0, 1)), (8, ws[:-1]), (9, 1.5)):
        assert quick.paged_attend(*good[:at], wrong, *good[at + 1:]) is None
    none = e(0, 4, 64).transpose(0, 2).transpose(0, 2)
    assert quick.paged_attend(plan.quick, 0, none, t[:0], n[:0], o[:0], kp, vp, ws, None) == 0
    assert quick.paged_attend(plan.quick, 0, e(4, 4, 64), e(4, 1, dt=torch.int32), ints([0] * 4), e(4, 256), kp, vp, ws,
                              None) == 1                            # more rows than the plan's: the library's own answer
    # what only the checks in Python take
    mono.paged_attend(plan, 0, torch.nn.Parameter(q), t, n, o, kp, vp, ws)
    mono.paged_attend(plan, torch.tensor(1), q, t, n, o, kp, vp, ws, stream=side)
    torch.cuda.synchronize()
    assert mono.paged_stats(plan, ws)["device_error"] == 0


def test_operators_without_the_quick_way(monkeypatch):
    # checked in Python alone: the same results
    lens, page = [70, 1, 33], 16
    plan, kp, vp, table = make_cache("bf16", 4, 2, 64, page, lens, seed=8, garbage=3.0)
    q = normal(5, 3, 4, 64, dtype=torch.bfloat16)
    k, v = (normal(s, 104, 2, 64, dtype=torch.bfloat16) for s in (6, 7))
    pq = normal(8, 104, 4, 64, dtype=torch.bfloat16)
    plan = plan_for("bf16", 4, 2, 64, page=page, pages=plan.cfg.pages, rows=3, width=plan.cfg.width, tokens=104)
    cu, t, n, ws = ints(cumulative(lens)), ints(table), ints(lens), plan.workspace()
    got = []
    for quick in (mono._quick, None):
        if quick is None:
            monkeypatch.setattr(mono, "_quick", types.SimpleNamespace(**{f: lambda *a: None for f in (
                "prompt_attend", "paged_append", "paged_attend", "paged_update", "paged_compact")}))
        o, po = (torch.empty((m, 256), dtype=torch.bfloat16, device="cuda") for m in (3, 104))
        t1, n1, t2 = torch.empty_like(t), torch.empty_like(n), torch.empty_like(t)
        a, b = kp.clone(), vp.clone()
        mono.prompt_attend(plan, pq, k, v, cu, cu, po, ws)
        mono.paged_append(plan, 0, k, v, cu, t, n, a, b, ws)
        mono.paged_attend(plan, 0, q, t, n, o, a, b, ws)
        mono.paged_update(plan, t, n, ints([0, 0, 2]), ints([1, 2, -5]), t1, n1, a, b, ws)
        mono.paged_compact(plan, t1, n1, t2, a, b, ws)
        assert mono.paged_stats(plan, ws)["device_error"] == 0
        got.append((o, po, t1, n1, t2, a, b))
    assert all(torch.equal(x, y) for x, y in zip(*got))


# ---------------------------------------------------------------------------
# together, as a serving loop uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(dtype, captured):
    # prompts in, every sequence forked in two, tokens decoded with one dropped on the way; on a stream of its own,
    # and with the decode step captured once and replayed
    dt, Hq, Hkv, d, page, layers, width = DT[dtype], 6, 2, 64, 16, 2, 14
    lens = [37, 64, 1]
    plan = plan_for(dtype, Hq, Hkv, d, page=page, pages=90, layers=layers, rows=8, width=width, tokens=128)
    kp, vp = plan.pools()
    kp.fill_(math.nan)
    vp.fill_(math.nan)
    ws = plan.workspace()
    scale = d ** -0.5
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n = len(lens)
        none = torch.empty((0, width), dtype=torch.int32, device="cuda")
        table = torch.empty((n, width), dtype=torch.int32, device="cuda")
        ln = torch.empty((n,), dtype=torch.int32, device="cuda")
        mono.paged_update(plan, none, none[:, 0].contiguous(), ints([-1] * n), ints(lens), table, ln, kp, vp, ws)
        cu = ints(cumulative(lens))
        hist = [[] for _ in range(layers)]
        for layer in range(layers):
            q, k, v = (normal(10 * layer + x, sum(lens), h, d, dtype=dt, sd=1.2) for x, h in ((0, Hq), (1, Hkv), (2, Hkv)))
            o = torch.empty((sum(lens), Hq * d), dtype=dt, device="cuda")
            mono.prompt_attend(plan, q, k, v, cu, cu, o, ws)
            mono.paged_append(plan, layer, k, v, cu, table, ln, kp, vp, ws)
            c = cumulative(lens)
            ref, tol = prompt64(q, k, v, c, c, scale, P_PROMPT[dtype])
            assert_within(o, ref, tol, "prompt")
            hist[layer] = [(k[a:b], v[a:b]) for a, b in zip(c, c[1:])]
        # fork: each sequence twice; then steps of one token, buffers fixed so that a step can be captured
        m = 2 * n
        rows = [i // 2 for i in range(m)]
        hist = [[h[i] for i in rows] for h in hist]
        t_a, t_b = (torch.empty((m, width), dtype=torch.int32, device="cuda") for _ in range(2))
        l_a, l_b = (torch.empty((m,), dtype=torch.int32, device="cuda") for _ in range(2))
        mono.paged_update(plan, table, ln, ints(rows), ints([0] * m), t_a, l_a, kp, vp, ws)
        one, cum, who = ints([1] * m), ints(list(range(m + 1))), ints(list(range(m)))
        qs, ks, vs = (torch.empty((layers, m, h, d), dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv))
        os_ = torch.empty((layers, m, Hq * d), dtype=dt, device="cuda")

        def step():
            mono.paged_update(plan, t_a, l_a, who, one, t_b, l_b, kp, vp, ws)
            for layer in range(layers):
                mono.paged_append(plan, layer, ks[layer], vs[layer], cum, t_b, l_b, kp, vp, ws)
                mono.paged_attend(plan, layer, qs[layer], t_b, l_b, os_[layer], kp, vp, ws)
            t_a.copy_(t_b)
            l_a.copy_(l_b)

        graph = None
        for it in range(20):
            for x, (buf, sd) in enumerate(((qs, 1.2), (ks, 1.2), (vs, 1.0))):
                buf.copy_(normal(1000 + 10 * it + x, *buf.shape, dtype=dt, sd=sd))
            if it == 9:                                      # row 3 now continues row 0, whose page it shares
                parents = list(range(m))
                parents[3] = 0
                who.copy_(ints(parents))
            elif it == 10:
                who.copy_(ints(list(range(m))))
            if it == 9:
                hist = [[h[0] if i == 3 else h[i] for i in range(m)] for h in hist]
            if captured and it == 2:
                s.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    step()
            if graph is not None:
                graph.replay()
            else:
                step()
            for layer in range(layers):
                hist[layer] = [(torch.cat([k, ks[layer, i:i + 1]]), torch.cat([v, vs[layer, i:i + 1]]))
                               for i, (k, v) in enumerate(hist[layer])]
                for i, (k, v) in enumerate(hist[layer]):
                    for h in range(Hq):
                        ref, tol = attend64(qs[layer, i, h:h + 1].double(), k[:, h // 3].double(), v[:, h // 3].double(),
                                            torch.tensor([k.shape[0]], device="cuda"), scale, P_DECODE[dtype], dt)
                        assert_within(os_[layer, i, h * d:(h + 1) * d], ref[0], tol[0], f"step {it} row {i} head {h}")
        assert l_a.tolist() == [len(h[0]) for h in hist[0]]
        st = mono.paged_stats(plan, ws)
        assert st["device_error"] == 0
        # the cache holds exactly the history
        for layer in range(layers):
            for i, (k, v) in enumerate(hist[layer]):
                assert torch.equal(rows_of(kp[layer], t_a[i].tolist()[:-(-len(k) // page)], page, len(k)), k)
    torch.cuda.current_stream().wait_stream(s)
