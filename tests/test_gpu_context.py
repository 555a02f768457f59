"""The context on the GPU against the float64 oracle (``oracle.context``).

Tolerances, from the number formats (u(t) = eps / 2 of the type: bf16 2^-8,
fp16 2^-11, fp32 2^-24):
  rope       one rounding to bf16 of a float32 rotation: 2^-8 |y| and, for the
             float32 turns and products, 2^-21 of the pair's norm.
  append     codes are the nearest E4M3 values of a float32 number that is off
             by at most 2^-21 of the pair's norm: equal to the oracle's unless
             that number lies so close to the middle of two codes, and then
             one step off.  Scales are equal.
  attention  per element 2^-8 |o| (the result) + (2^-11 + 2^-18 + 2 d)
             sum w |v|: weights are rounded to float16 (2^-11; those under
             2^-24 of the largest are off by up to 2^-35 of it instead, which
             these inputs' sums stay above; exponentials by polynomial
             are off by up to 2.6e-6 < 2^-18), and a logit
             is off by at most d = (dim + 4) 2^-24 max sum |q k| (float32 sums)
             + 2^-17 max |q| max sum |k| (queries as two E4M3 terms: an
             element under 2^-9 of the largest is off by half the smallest
             E4M3 step, 2^-10, when the largest is in [2^7, 2^8)), which moves
             a weight and the normaliser by that part.
"""
import math

import numpy as np
import pytest

from oracle import context as oc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_canvas_denoising_b200 as dg  # noqa: E402
from block_canvas_denoising_b200 import build as dg_build  # noqa: E402

dg_build.build()


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def bf16(rng, *shape):
    return torch.tensor(rng.standard_normal(shape), dtype=torch.float32).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------------------------------------- plan
def make_plan(rng, held, spare, width, rows):
    """A plan whose pool is in use: pages in random order."""
    used = [-(-h // 64) for h in held]
    pages = sum(used) + spare
    order = rng.permutation(pages)
    plan = dg.ContextPlan(len(held), rows, max(pages, 1), width)
    table = np.full((len(held), width), -7, np.int32)
    at = 0
    for r, u in enumerate(used):
        table[r, :u] = order[at:at + u]
        at += u
    free = np.zeros(plan.pages, np.int32)
    free[:spare] = order[at:at + spare]
    plan.table.copy_(torch.from_numpy(table))
    plan.held.copy_(ints(list(held)))
    plan.free_list.copy_(torch.from_numpy(free))
    plan.free_count.fill_(spare)
    return plan


PLAN_FIELDS = ("table", "held", "free_list", "free_count", "lens", "start", "positions", "slots", "runs", "free_next")


def check_plan(plan, add, release=None, commit=False):
    before = {n: getattr(plan, n).cpu().numpy().copy() for n in PLAN_FIELDS}
    held = before["lens"] if commit else before["held"]
    free = int((before["free_next"] if commit else before["free_count"])[0])
    want = oc.plan(before["table"].tolist(), held.tolist(), before["free_list"].tolist(), free, list(add), release,
                   plan.rows)
    dg.context_plan(plan, ints(list(add)), None if release is None else ints(list(release), torch.uint8), commit)
    torch.cuda.synchronize()
    for n in PLAN_FIELDS:
        got = getattr(plan, n).cpu().numpy()
        assert np.array_equal(got, np.array(want[n]).reshape(got.shape)), n
    assert int(plan.status[0]) == want["status"]
    return want


@pytest.mark.parametrize("B,new,context,leave", [(1, 1, 0, 0), (1, 1, 63, 0), (1, 1, 64, 0), (3, 256, 700, 0),
                                                 (17, 130, 500, 0.3), (256, 5, 300, 0.5), (256, 1, 64, 0),
                                                 (33, 1000, 100, 0.2)])
def test_plan_matches_oracle(B, new, context, leave):
    rng = np.random.default_rng(B * 1000 + new)
    held = rng.integers(0, context + 1, B)
    add = rng.integers(0, new + 1, B)
    add[0] = new
    release = (rng.random(B) < leave).astype(int).tolist() if leave else None
    plan = make_plan(rng, held, int(sum(-(-int(a) // 64) + 1 for a in add)), (context + new) // 64 + 2,
                     int(add.sum()) + 3)
    want = check_plan(plan, add, release)
    assert want["status"] == 0
    check_plan(plan, add, release)  # planned over: the same batch again
    check_plan(plan, (add // 2).tolist())  # and another in its place


def test_plan_commits_batch_after_batch():
    rng = np.random.default_rng(5)
    plan = dg.ContextPlan(4, 600, 60, 20)
    total = np.zeros(4, int)
    for step in range(6):
        add = rng.integers(0, 150, 4)
        release = [0, 0, 0, 0]
        if step == 4:
            release[2] = 1
            total[2] = 0
        want = check_plan(plan, add, release if step == 4 else None, commit=step > 0)
        assert want["status"] == 0
        total += add
        assert want["lens"] == total.tolist()
    pages = [p for r in range(4) for p in want["table"][r][:-(-int(total[r]) // 64)]]
    assert len(set(pages)) == len(pages)
    assert sorted(pages + want["free_list"][:want["free_next"]]) == list(range(60))
    assert dg.context_status(plan) == 0


def test_plan_refuses_whole_batches():
    rng = np.random.default_rng(6)
    for held, spare, add, code in (([10, 100], 1, [200, 60], 2), ([10, 100], 1, [200, 50], 1), ([10, 100], 9, [200, 57], 2),
                                   ([10, 100], 9, [300, 1], 3), ([10, 100], 9, [-1, 3], 3), ([10, 100], 9, [2 ** 31 - 1, 2 ** 31 - 1], 3),
                                   ([0, 0], 0, [1, 0], 1), ([0, 0], 0, [0, 0], 0)):
        plan = make_plan(rng, held, spare, 4, 256)
        want = check_plan(plan, add)
        assert want["status"] == code
        assert dg.context_status(plan) == (10 if code else 0)
        if code:
            assert plan.start.cpu().tolist() == [0, 0, 0]
            check_plan(plan, [1, 0] if spare else [0, 0], commit=True)  # a refused batch commits nothing
    # corrupt state is refused, not followed
    plan = make_plan(rng, [10, 100], 3, 4, 256)
    for field, value in (("free_count", 99), ("free_count", -1), ("held", -5), ("held", 1 << 20)):
        saved = getattr(plan, field).clone()
        getattr(plan, field).fill_(value)
        dg.context_plan(plan, ints([1, 1]), ints([1, 1], torch.uint8))
        assert dg.context_status(plan) == 10
        assert plan.runs[:, 0].max().item() == -1
        getattr(plan, field).copy_(saved)


# ---------------------------------------------------------------------------------------------- rope
@pytest.mark.parametrize("rows,heads,dim,rot,il,scaling,far", [
    (1, 1, 64, 64, False, "none", 10), (5, 3, 128, 128, False, "none", 5000), (5, 3, 128, 128, True, "linear", 5000),
    (700, 2, 64, 48, False, "ntk", 100000), (3, 22, 128, 16, True, "parts", 1 << 20), (601, 5, 128, 64, True, "parts", 2 ** 31 - 1)])
def test_rope_matches_oracle(rows, heads, dim, rot, il, scaling, far):
    rng = np.random.default_rng(rows)
    x = bf16(rng, rows, heads, dim)
    pos = rng.integers(0, far, rows)
    pos[0] = far - 1
    f = dg.RopeFrequencies(rot, scaling=scaling, factor=8.0, interleaved=il)
    want = oc.rope(f64(x), pos, *oc.frequencies(rot, scaling=scaling, factor=8.0), il)
    got = dg.rope(x, ints(pos.tolist()), f)
    pair = np.sqrt(2) * np.abs(f64(x)).max(-1, keepdims=True) * f.magnitude
    assert np.all(np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * pair + 1e-38)
    # in place, and as a view of a fused tensor in another layout: the same bits
    y = x.clone()
    assert dg.rope(y, ints(pos.tolist()), f, out=y) is y and torch.equal(y, got)
    fused = torch.zeros((rows, heads + 3, dim), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:2 + heads] = x
    heads_first = torch.zeros((heads, rows, dim), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    dg.rope(fused[:, 2:2 + heads], ints(pos.tolist()), f, out=heads_first)
    assert torch.equal(heads_first, got) and fused[:, 2 + heads:].abs().max() == 0


def test_rope_leaves_rows_without_a_position():
    x = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 5.0)
    dg.rope(x, ints([3, -1, 4, -1]), dg.RopeFrequencies(64), out=out)
    assert (out[[1, 3]] == 5).all() and not (out[[0, 2]] == 5).any()
    assert dg.rope(x[:0], ints([]), dg.RopeFrequencies(64)).shape == (0, 2, 64)


# ---------------------------------------------------------------------------------------------- append
def cache_values(codes):
    return codes.view(torch.float8_e4m3fn).float().double().cpu().numpy()


def check_append(plan, cache, k, v, rope_args=None, rope_obj=None, seen=None):
    state = {n: (cache_values(getattr(cache, n)), f64(getattr(cache, n + "_scale"))) for n in ("k", "v")}
    runs = plan.runs.cpu().tolist()
    total = int(plan.start[-1])
    pos = plan.positions.cpu().numpy()[:total]
    kk, near = f64(k)[:total], 0.0
    if rope_args is not None:
        f, mag, il = rope_args
        kk = oc.rope(kk, pos, f, mag, il)
        near = 2.0 ** -21 * math.sqrt(2) * mag
    dg.context_append(plan, cache, k, v, rope=rope_obj)
    torch.cuda.synchronize()
    for n, x in (("k", kk), ("v", f64(v)[:total])):
        values, scales = state[n]
        oc.append(values, scales, x, runs)
        assert np.array_equal(f64(getattr(cache, n + "_scale")), scales), n
        got = cache_values(getattr(cache, n))
        if n == "v" or rope_args is None:
            assert np.array_equal(got, values), n
            continue
        off = got != values  # only numbers next to the middle of two codes may differ
        assert off.mean() < 1e-3
        for page, h, s, d in zip(*np.nonzero(off)):
            row = next(r0 + s - o for pg, r0, o, c in runs if pg == page and o <= s < o + c)
            y = x[row, h, d] / scales[page, h]
            tol = near * np.abs(f64(k)[row, h]).max() / scales[page, h]
            a, b = oc.round_e4m3(y - tol), oc.round_e4m3(y + tol)
            assert a != b and got[page, h, s, d] in (a, b)


@pytest.mark.parametrize("dim,heads,il,rot", [(128, 2, False, 128), (64, 3, True, 32), (128, 1, True, 48)])
def test_append_matches_oracle(dim, heads, il, rot):
    rng = np.random.default_rng(dim + rot)
    held = [0, 1, 63, 64, 100, 7]
    add = [1, 64, 2, 129, 0, 50]
    plan = make_plan(rng, held, 20, 8, sum(add) + 9)
    dg.context_plan(plan, ints(add))
    cache = dg.ContextCache(plan.pages, heads, dim)
    codes = rng.integers(0, 256, tuple(cache.k.shape)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0
    cache.k.copy_(torch.from_numpy(codes))
    cache.v.copy_(torch.from_numpy(codes[::-1].copy()))
    cache.k_scale.copy_(torch.from_numpy(2.0 ** rng.integers(-12, 0, tuple(cache.k_scale.shape)).astype(np.float32)))
    cache.v_scale.copy_(torch.from_numpy(2.0 ** rng.integers(-12, 0, tuple(cache.k_scale.shape)).astype(np.float32)))
    qkv = bf16(rng, plan.rows, 3 * heads, dim)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    f, mag = oc.frequencies(rot, scaling="parts", factor=4.0)
    obj = dg.RopeFrequencies(rot, scaling="parts", factor=4.0, interleaved=il)
    check_append(plan, cache, k, v, (f, mag, il), obj)
    snapshot = cache.k.clone(), cache.v.clone()
    dg.context_append(plan, cache, k, v, rope=obj)  # a canvas's next step: the same rows again
    assert torch.equal(snapshot[0], cache.k) and torch.equal(snapshot[1], cache.v)
    check_append(plan, cache, v, k)  # no rotation, bit for bit
    assert dg.context_status(plan) == 0


def test_append_extreme_values():
    rng = np.random.default_rng(3)
    plan = dg.ContextPlan(1, 140, 4, 4)
    dg.context_plan(plan, ints([131]))
    cache = dg.ContextCache(4, 1, 64)
    x = bf16(rng, 140, 1, 64)
    x[:64] = 0
    x[64:128] *= 1e-38
    x[128:] *= 1e36
    check_append(plan, cache, x, x)
    assert cache.k_scale[plan.table[0, 0], 0] == 1 and dg.context_status(plan) == 0
    x[70, 0, 3], x[71, 0, 4], x[72, 0, 5] = math.nan, math.inf, -math.inf
    check_append(plan, cache, x, x)
    assert dg.context_status(plan) == 9 and dg.context_status(plan) == 0  # reported once
    x[135:] = math.nan  # rows behind the last are not read
    x[70:73] = 0
    check_append(plan, cache, x, x)
    assert dg.context_status(plan) == 0


# ---------------------------------------------------------------------------------------------- attention
def random_cache(rng, pages, heads, dim, spread=6):
    cache = dg.ContextCache(pages, heads, dim)
    for n in ("k", "v"):
        x = torch.tensor(rng.standard_normal((pages, heads, 64, dim)), dtype=torch.float32)
        s = torch.tensor(2.0 ** rng.integers(-spread, spread + 1, (pages, heads)), dtype=torch.float32)
        codes = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)  # no NaN code
        scale = (s / 128).float()
        getattr(cache, n).copy_(codes.view(torch.uint8))
        getattr(cache, n + "_scale").copy_(scale)
    return cache


def tokens(plan, cache, r, n):
    """Keys and values of request r's first n tokens, float64."""
    page = plan.table[r].cpu().numpy()[:-(-n // 64)]
    got = []
    for name in ("k", "v"):
        x = cache_values(getattr(cache, name))[page] * f64(getattr(cache, name + "_scale"))[page][..., None, None]
        got.append(x.transpose(0, 2, 1, 3).reshape(-1, cache.heads, cache.dim)[:n])
    return got


def value_scales(plan, cache, r):
    """The scale of each token's values, [tokens of the pages, kv heads]."""
    page = plan.table[r].cpu().numpy()[:-(-int(plan.lens[r]) // 64)]
    return np.repeat(f64(cache.v_scale)[page], 64, axis=0)


def check_attention(plan, cache, q, causal, window=0, scale=None, max_new=0, ws=None, rows_of=None):
    heads, dim = q.shape[1], cache.dim
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((plan.rows, heads), 3.0, device="cuda")
    ws = ws or dg.ContextWorkspace(plan.rows, heads, cache.heads, dim)
    dg.context_attention(plan, cache, q, out, ws, causal=None if causal is None else ints(causal, torch.uint8),
                         window=window, scale=scale, lse=lse, max_new=max_new)
    assert dg.device_status(ws) == 0
    start, lens = plan.start.cpu().tolist(), plan.lens.cpu().tolist()
    s = scale or 1 / math.sqrt(dim)
    o, z = f64(out), f64(lse)
    worst = 0.0
    for r in range(plan.B):
        nq = start[r + 1] - start[r]
        if nq == 0:
            continue
        k, v = tokens(plan, cache, r, lens[r])
        pick = np.arange(nq) if rows_of is None else np.unique(np.clip(rows_of, 0, nq - 1))
        qs = f64(q)[start[r]:start[r + 1]]
        for i in pick:  # one row at a time: rows before it are not there for the oracle
            c = bool(causal and causal[r])
            n = lens[r] - nq + i + 1 if c else lens[r]
            # as the last row of a shorter request (causal), or with its own position
            if c:
                w, lw, mass, size = oc.attention(qs[i:i + 1], k[:n], v[:n], s, True, window)
            else:
                lo = max(0, lens[r] - nq + i - window + 1) if window else 0
                w, lw, mass, size = oc.attention(qs[i:i + 1], k[lo:], v[lo:], s, False, 0)
            # Weights are at least 2^6 at the largest weight times page scale, in
            # float16, whose smallest step is 2^-24: a weight further down is
            # off by 2^-25, 2^-31 of the largest, however small the sum of
            # weights times values is beside it (the largest weight's own value
            # may be a 0).
            first, last = (max(0, n - window) if window else 0, n) if c else (lo, n)
            kk, vv, vs = (np.repeat(t[first:last], heads // cache.heads, axis=1) for t in (k, v, value_scales(plan, cache, r)[:n]))
            share = np.exp(np.einsum("nhd,hd->nh", kk, qs[i]) * s - np.where(np.isinf(lw[0]), 0, lw[0])) * vs
            tail = 2.0 ** -31 * share.max(0, initial=0)[:, None] * (np.abs(vv) / vs[..., None]).sum(0)
            terms = 2.0 ** -17 * s * np.abs(qs[i]).max(-1, keepdims=True) * np.abs(k).sum(-1).max(initial=0)
            d = (dim + 4) * 2.0 ** -24 * size[0][:, None] + terms
            tol = 2.0 ** -8 * np.abs(w[0]) + (2.0 ** -11 + 2.0 ** -18 + 2 * d) * mass[0] + tail + 1e-38
            err = np.abs(o[start[r] + i] - w[0])
            assert np.all(err <= tol), (r, i, float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
            got, want = z[start[r] + i], lw[0]
            inf = np.isinf(want)
            assert np.array_equal(got[inf], want[inf])
            assert np.all(np.abs(got[~inf] - want[~inf]) <= d[~inf, 0] + 2.0 ** -18 + 2.0 ** -20 * np.abs(want[~inf]))
    total = start[-1]
    assert (out[total:] == 3).all() and (lse[total:] == 3).all()  # rows behind the last, as they were
    return out, worst


def setup(rng, held, add, heads, kv, dim, behind=0, spread=6):
    width = max(-(-(h + a) // 64) for h, a in zip(held, add)) + 1
    plan = make_plan(rng, held, sum(-(-a // 64) + 1 for a in add), width, sum(add) + behind)
    dg.context_plan(plan, ints(list(add)))
    cache = random_cache(rng, plan.pages, kv, dim, spread)
    return plan, cache, bf16(rng, plan.rows, heads, dim)


@pytest.mark.parametrize("held,add,heads,kv,dim,causal,window", [
    ([0], [1], 1, 1, 64, [1], 0), ([0], [1], 4, 4, 128, None, 0),
    ([62, 63, 64, 127, 0], [1, 1, 1, 1, 1], 8, 2, 128, [1, 0, 1, 0, 1], 0),
    ([300, 5, 0, 1000], [1, 2, 3, 0], 11, 1, 64, [1, 1, 0, 1], 0),
    ([4000], [1], 16, 4, 128, [1], 0), ([3000, 10, 200], [1, 1, 1], 5, 1, 128, [1, 1, 1], 70),
    ([500, 0, 64], [5, 17, 33], 6, 3, 64, [1, 0, 1], 40), ([100] * 40, [1] * 40, 3, 3, 128, None, 0),
    ([1000], [16], 40, 2, 128, [1], 0)])
def test_attention_few_rows(held, add, heads, kv, dim, causal, window):
    rng = np.random.default_rng(len(held) * 100 + sum(add))
    plan, cache, q = setup(rng, held, add, heads, kv, dim, behind=3)
    check_attention(plan, cache, q, causal, window, max_new=max(add))


@pytest.mark.parametrize("held,add,heads,kv,dim,causal,window", [
    ([700], [256], 4, 2, 128, None, 0), ([700], [256], 4, 2, 64, [1], 0),
    ([0, 129, 33], [200, 256, 1], 6, 2, 128, [1, 0, 1], 0), ([0, 0], [300, 70], 11, 1, 64, [1, 0], 0),
    ([64, 3], [256, 100], 3, 1, 128, [0, 1], 50), ([1000, 0, 5], [130, 0, 1], 8, 1, 64, [1, 1, 0], 300),
    ([3000], [256], 22, 2, 128, None, 0), ([20], [513], 2, 2, 128, [1], 0), ([2], [385], 10, 2, 64, [1], 1)])
def test_attention_many_rows(held, add, heads, kv, dim, causal, window):
    rng = np.random.default_rng(len(held) * 100 + sum(add))
    plan, cache, q = setup(rng, held, add, heads, kv, dim, behind=5)
    rows = np.concatenate([[0, 1, 62, 63, 64, 127, 128, 255, 10 ** 6], rng.integers(0, max(add), 6)])
    check_attention(plan, cache, q, causal, window, rows_of=rows)


def test_attention_rows_that_see_nothing():
    # lengths shortened by the caller: the causal rows before the first token see nothing
    rng = np.random.default_rng(1)
    plan, cache, q = setup(rng, [0, 10], [40, 20], 4, 2, 128)
    for lens, causal in (([5, 30], [1, 1]), ([0, 0], [1, 0]), ([0, 30], [0, 0])):
        plan.lens.copy_(ints(lens))
        for most in (0, 1):
            check = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros((plan.rows, 4), device="cuda")
            ws = dg.ContextWorkspace(plan.rows, 4, 2, 128)
            dg.context_attention(plan, cache, q, check, ws, causal=ints(causal, torch.uint8), lse=lse, max_new=most)
            empty = max(40 - lens[0], 0) if causal[0] else (40 if lens[0] == 0 else 0)
            assert (check[:empty] == 0).all() and torch.isneginf(lse[:empty]).all()
            assert torch.isfinite(check.float()).all() and not (check[empty:40] == 0).all(-1).any()


def test_attention_ignores_what_is_behind_the_last_token():
    # NaN codes in the slots behind each request's last token, and in pages nobody holds
    rng = np.random.default_rng(2)
    for dim, add in ((128, [3, 1]), (64, [3, 1]), (128, [200, 130]), (64, [200, 130])):
        plan, cache, q = setup(rng, [70, 0], add, 4, 2, dim)
        clean, _ = check_attention(plan, cache, q, [0, 1])
        used = set()
        for r, n in enumerate(plan.lens.cpu().tolist()):
            page = plan.table[r].cpu().tolist()[:-(-n // 64)]
            used |= set(page)
            if n % 64:
                cache.k[page[-1], :, n % 64:] = 0x7F
                cache.v[page[-1], :, n % 64:] = 0xFF
        for page in set(range(plan.pages)) - used:
            cache.k[page] = 0x7F
            cache.v[page] = 0x7F
        dirty, _ = check_attention(plan, cache, q, [0, 1])
        assert torch.equal(clean, dirty)


def test_attention_bad_pages_are_not_seen():
    rng = np.random.default_rng(4)
    for add in ([1], [200]):
        plan, cache, q = setup(rng, [300], add, 4, 2, 128)
        good = plan.table.clone()
        ws = dg.ContextWorkspace(plan.rows, 4, 2, 128)
        out = torch.zeros_like(q)
        for bad in (-1, plan.pages, 2 ** 31 - 1, -2 ** 31):
            plan.table.copy_(good)
            plan.table[0, 0] = bad
            dg.context_attention(plan, cache, q, out, ws)
            assert dg.device_status(ws) == 0
            # the same as a request without its first page
            n = int(plan.lens[0])
            plan.table.copy_(good)
            k, v = tokens(plan, cache, 0, n)
            w, _, mass, size = oc.attention(f64(q)[:1], k[64:], v[64:], 128 ** -0.5, False, 0)
            assert np.all(np.abs(f64(out)[:1] - w) <= 2.0 ** -8 * np.abs(w) + 2.0 ** -9 * mass)


def test_attention_queries_that_are_not_finite():
    rng = np.random.default_rng(7)
    for add in ([2, 1], [150, 40]):
        plan, cache, q = setup(rng, [100, 30], add, 4, 2, 128)
        clean, _ = check_attention(plan, cache, q, None)
        q[1, 2, 5], q[add[0], 0, 127] = math.nan, math.inf
        out = torch.zeros_like(q)
        dg.context_attention(plan, cache, q, out, dg.ContextWorkspace(plan.rows, 4, 2, 128))
        mark = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        mark[1, 2] = mark[add[0], 0] = True
        assert torch.isnan(out[mark]).all() and torch.equal(out[~mark], clean[~mark])


def test_attention_queries_of_every_size():
    # rows of zeros, tiny and huge ones next to ordinary ones; a peaked softmax
    rng = np.random.default_rng(8)
    for add in ([5], [140]):
        plan, cache, q = setup(rng, [200], add, 2, 1, 128, spread=0)
        q[0] = 0
        q[1] *= 1e-38
        q[2] *= 2.0 ** -120
        q[3] *= 40
        check_attention(plan, cache, q, None, rows_of=[0, 1, 2, 3, 4])
        q[4] *= 1e30  # logits of 1e30: one key has all the weight
        out = torch.zeros_like(q)
        dg.context_attention(plan, cache, q, out, dg.ContextWorkspace(plan.rows, 2, 1, 128))
        k, v = tokens(plan, cache, 0, int(plan.lens[0]))
        for h in range(2):
            best = int(np.argmax(k[:, 0] @ f64(q)[4, h]))
            assert np.all(np.abs(f64(out)[4, h] - v[best, 0]) <= 2.0 ** -8 * np.abs(v[best, 0]))


def test_attention_value_scales_far_apart():
    rng = np.random.default_rng(9)
    for add in ([4], [130]):
        plan, cache, q = setup(rng, [500], add, 4, 2, 64, spread=20)
        cache.k_scale.fill_(2.0 ** -7)
        check_attention(plan, cache, q, [1], rows_of=np.arange(0, 130, 9))


def test_attention_layouts_and_scale():
    rng = np.random.default_rng(10)
    for add in ([3, 2], [130, 70]):
        plan, cache, q = setup(rng, [90, 10], add, 4, 2, 128, behind=2)
        want, _ = check_attention(plan, cache, q, [1, 0], scale=0.3, rows_of=[0, 1, 2, 64, 129])
        fused = torch.zeros((plan.rows, 9, 128), dtype=torch.bfloat16, device="cuda")
        fused[:, 3:7] = q
        heads_first = torch.full((4, plan.rows, 128), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        ws = dg.ContextWorkspace(plan.rows, 4, 2, 128)
        dg.context_attention(plan, cache, fused[:, 3:7], heads_first, ws, causal=ints([1, 0], torch.bool), scale=0.3)
        assert torch.equal(heads_first, want)


def test_attention_is_the_same_every_time():
    rng = np.random.default_rng(11)
    for held, add, heads, kv in (([9000, 100], [1, 1], 8, 2), ([5000, 70], [256, 256], 4, 1)):
        plan, cache, q = setup(rng, held, add, heads, kv, 128)
        ws = dg.ContextWorkspace(plan.rows, heads, kv, 128)
        outs = []
        for _ in range(20):
            out = torch.zeros_like(q)
            dg.context_attention(plan, cache, q, out, ws)
            outs.append(out)
        assert all(torch.equal(o, outs[0]) for o in outs)


def test_wrong_tensors_are_refused():
    rng = np.random.default_rng(12)
    plan, cache, q = setup(rng, [10], [4], 4, 2, 128)
    ws = dg.ContextWorkspace(plan.rows, 4, 2, 128)
    out = torch.zeros_like(q)
    bad = [q.float(), q[:3], q[:, :, :64], q.cpu(), q[0], torch.zeros((4, 4, 136), dtype=torch.bfloat16, device="cuda")[:, :, 1:129],
           torch.zeros((4, 4, 256), dtype=torch.bfloat16, device="cuda")[:, :, ::2]]
    for x in bad:
        with pytest.raises(dg.DGError):
            dg.context_attention(plan, cache, x, out, ws)
        with pytest.raises(dg.DGError):
            dg.context_append(plan, cache, x, x)
    with pytest.raises(dg.DGError):
        dg.context_attention(plan, cache, q, q, ws)
    with pytest.raises(dg.DGError):
        dg.context_attention(plan, cache, q, out, ws, causal=ints([1]))
    with pytest.raises(dg.DGError):
        dg.context_attention(plan, cache, q, out, ws, lse=torch.zeros(4, 4))
    small = dg.ContextWorkspace(plan.rows, 4, 2, 128)
    small.nbytes = 64
    with pytest.raises(dg.DGError):
        dg.context_attention(plan, cache, q, out, small)
    with pytest.raises(dg.DGError):
        dg.context_plan(plan, ints([1, 2]))
    with pytest.raises(dg.DGError):
        dg.context_plan(plan, ints([1]), release=ints([0]))
    with pytest.raises(dg.DGError):
        dg.rope(q, ints([1, 2, 3]), dg.RopeFrequencies(64))
    with pytest.raises(dg.DGError):
        dg.rope(q, ints([1, 2, 3, 4]), dg.RopeFrequencies(64), out=out[:, :2])


# ---------------------------------------------------------------------------------------------- together
def test_captured_and_replayed():
    # plan, append and attend in one graph: the lengths live on the device, so replays follow them
    rng = np.random.default_rng(13)
    heads, kv, dim = 4, 2, 128
    plan = dg.ContextPlan(2, 8, 30, 10)
    cache = dg.ContextCache(30, kv, dim)
    qkv = bf16(rng, 8, heads + 2 * kv, dim)
    f = dg.RopeFrequencies(dim)
    ws = dg.ContextWorkspace(8, heads, kv, dim)
    add, causal = ints([1, 3]), ints([1, 1], torch.uint8)
    q, out = torch.zeros((8, heads, dim), dtype=torch.bfloat16, device="cuda"), torch.zeros((8, heads, dim), dtype=torch.bfloat16, device="cuda")

    def step(plan, cache, out):
        dg.context_plan(plan, add, commit=True)
        dg.context_append(plan, cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], rope=f)
        dg.rope(qkv[:, :heads], plan.positions, f, out=q)
        dg.context_attention(plan, cache, q, out, ws, causal=causal, max_new=3)
    other = dg.ContextPlan(2, 8, 30, 10), dg.ContextCache(30, kv, dim), torch.zeros_like(out)
    step(*other)  # eager once, before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(plan, cache, out)
    for n in range(1, 60):
        add.copy_(ints([n % 3, 3 - n % 3]))
        graph.replay()
        if n > 1:
            step(*other)
        else:
            other = dg.ContextPlan(2, 8, 30, 10), dg.ContextCache(30, kv, dim), torch.zeros_like(out)
            step(*other)
        assert torch.equal(out, other[2]) and torch.equal(plan.lens, other[0].lens)
        assert torch.equal(cache.k, other[1].k) and torch.equal(cache.v_scale, other[1].v_scale)
    assert dg.context_status(plan) == 0 and dg.device_status(ws) == 0


def test_on_another_stream():
    rng = np.random.default_rng(14)
    plan, cache, q = setup(rng, [700, 3], [256, 1], 4, 2, 128)
    want, _ = check_attention(plan, cache, q, None, rows_of=[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(q, 3.0)
    ws = dg.ContextWorkspace(plan.rows, 4, 2, 128)
    torch.cuda.synchronize()
    dg.context_attention(plan, cache, q, out, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_two_steps_of_generation_together():
    # prompts encoded causally, then a canvas rewritten every step, then committed:
    # what is attended equals what an uncached float64 attention sees, up to the 8-bit cache
    rng = np.random.default_rng(15)
    heads, kv, dim, prompts = 4, 2, 64, [70, 5]
    plan = dg.ContextPlan(2, 512, 24, 12)
    cache = dg.ContextCache(24, kv, dim)
    f = dg.RopeFrequencies(dim, interleaved=True)
    ws = dg.ContextWorkspace(512, heads, kv, dim)

    def layer(add, commit, causal):
        dg.context_plan(plan, ints(add), commit=commit)
        x = bf16(rng, 512, heads + 2 * kv, dim)
        dg.context_append(plan, cache, x[:, heads:heads + kv], x[:, heads + kv:], rope=f)
        q = dg.rope(x[:, :heads], plan.positions, f)
        check_attention(plan, cache, q, causal, ws=ws, rows_of=[0, 1, 69, 128, 255])
        return x
    layer(prompts, False, [1, 1])
    layer([256, 256], True, [0, 0])
    layer([256, 256], False, [0, 0])  # the canvas again: planned over, its slots rewritten
    assert plan.lens.cpu().tolist() == [326, 261]
    layer([256, 256], False, [1, 1])  # encoded
    layer([256, 256], True, [0, 0])   # the next block
    assert plan.lens.cpu().tolist() == [582, 517] and dg.context_status(plan) == 0


def test_attention_under_load_equals_itself():
    # a batch with several pieces of work per SM, many times over and from several streams: every
    # result equals the first bit for bit, and the first the one computed request by request
    rng = np.random.default_rng(16)
    held = rng.integers(200, 1500, 12).tolist()
    plan, cache, q = setup(rng, held, [256] * 12, 11, 1, 128)
    first, _ = check_attention(plan, cache, q, None, rows_of=[0, 77, 255])
    streams = [torch.cuda.Stream() for _ in range(3)]
    work = [(s, dg.ContextWorkspace(plan.rows, 11, 1, 128), torch.zeros_like(q)) for s in streams]
    torch.cuda.synchronize()
    for _ in range(40):
        for s, ws, out in work:
            dg.context_attention(plan, cache, q, out, ws, stream=s)
        torch.cuda.synchronize()
        for s, ws, out in work:
            assert torch.equal(out, first)
            out.zero_()
        torch.cuda.synchronize()
    for _, ws, _ in work:
        assert dg.device_status(ws) == 0


def test_cache_beyond_32_bit_offsets():
    # 70,000 pages of 8 heads x 64 x 128: 4.6 GB of codes each, the request's pages at the far end
    rng = np.random.default_rng(17)
    pages, kv, dim = 70000, 8, 128
    cache = dg.ContextCache(pages, kv, dim)
    small = dg.ContextCache(8, kv, dim)
    for add, most in (([150], 0), ([2], 2)):
        big, ref = dg.ContextPlan(1, 150, pages, 4), dg.ContextPlan(1, 150, 8, 4)
        qkv = bf16(rng, 150, 3 * kv, dim)
        outs = []
        for plan, c in ((big, cache), (ref, small)):
            dg.context_plan(plan, ints(add))  # pages come from the top of the stack
            dg.context_append(plan, c, qkv[:, kv:2 * kv], qkv[:, 2 * kv:])
            out = torch.zeros((150, kv, dim), dtype=torch.bfloat16, device="cuda")
            dg.context_attention(plan, c, qkv[:, :kv], out, dg.ContextWorkspace(150, kv, kv, dim), max_new=most)
            outs.append(out)
        assert int(big.table[0, 0]) == pages - 1 and int(big.slots[0]) == (pages - 1) * 64
        assert torch.equal(outs[0], outs[1]) and outs[0].abs().max() > 0


def test_a_batch_without_rows():
    rng = np.random.default_rng(18)
    plan, cache, q = setup(rng, [10, 100], [5, 3], 4, 2, 128)
    dg.context_plan(plan, ints([0, 0]))
    assert plan.start.cpu().tolist() == [0, 0, 0] and (plan.positions == -1).all() and (plan.runs[:, 0] == -1).all()
    before = cache.k.clone()
    dg.context_append(plan, cache, q[:, :2], q[:, 2:])
    assert torch.equal(before, cache.k)
    for most in (0, 1):
        check_attention(plan, cache, q, [1, 0], max_new=most)


@pytest.mark.parametrize("B,heads,kv,dim", [(256, 3, 3, 64), (256, 2, 1, 128), (3, 64, 64, 64), (2, 99, 3, 128), (1, 320, 5, 64)])
def test_attention_many_requests_and_heads(B, heads, kv, dim):
    rng = np.random.default_rng(B + heads)
    held = rng.integers(0, 150, B).tolist()
    add = [1] * B
    add[0] = 2
    plan, cache, q = setup(rng, held, add, heads, kv, dim)
    causal = rng.integers(0, 2, B).tolist()
    check_attention(plan, cache, q, causal, max_new=2)
    check_attention(plan, cache, q, causal, window=33)


def test_one_workspace_for_many_shapes():
    rng = np.random.default_rng(19)
    ws = None
    for dim, add, heads, kv in ((128, [1, 1], 8, 2), (64, [200, 3], 4, 1), (128, [3, 100], 4, 2), (64, [1, 1], 16, 1), (64, [2, 1], 4, 4)):
        plan, cache, q = setup(rng, [2000, 50], add, heads, kv, dim)
        if ws is None:
            ws = dg.ContextWorkspace(plan.rows, heads, kv, dim)
        elif dg.context_workspace_size(plan.rows, heads, kv, dim) > ws.nbytes:
            continue
        check_attention(plan, cache, q, [1, 0], ws=ws, max_new=max(add), rows_of=[0, 1, 2, 99, 199])


@pytest.mark.parametrize("group,new,dim", [(1, 9, 128), (8, 3, 64), (11, 2, 128), (5, 5, 64), (16, 2, 128), (31, 1, 64),
                                           (32, 1, 128), (1, 32, 64), (1, 33, 128), (11, 3, 64), (33, 1, 128), (8, 4, 128)])
def test_attention_some_rows(group, new, dim):
    # between a handful of rows per kv head and a tile of them, where kernels change
    rng = np.random.default_rng(100 * group + new)
    plan, cache, q = setup(rng, [700, 0, 63], [new, 1, new], 2 * group, 2, dim, behind=2)
    check_attention(plan, cache, q, [0, 1, 1], max_new=new)
    check_attention(plan, cache, q, [1, 0, 0], window=65, max_new=new)


@pytest.mark.parametrize("B,heads,dim", [(40, 8, 128), (256, 8, 64), (40, 7, 64), (200, 5, 128)])
def test_append_many_runs(B, heads, dim):
    # so many pages are touched that a block takes several heads
    rng = np.random.default_rng(B + heads)
    held, add = rng.integers(0, 130, B).tolist(), rng.integers(0, 4, B).tolist()
    plan = make_plan(rng, held, 3 * B, 3, sum(add) + 1)
    dg.context_plan(plan, ints(add))
    cache = random_cache(rng, plan.pages, heads, dim)
    x = bf16(rng, plan.rows, 2 * heads, dim)
    check_append(plan, cache, x[:, :heads], x[:, heads:])
    f, mag = oc.frequencies(dim)
    check_append(plan, cache, x[:, heads:], x[:, :heads], (f, mag, False), dg.RopeFrequencies(dim))


@pytest.mark.parametrize("heads,kv,dim", [(1024, 1, 64), (600, 2, 128), (1024, 1024, 64)])
def test_attention_largest_groups(heads, kv, dim):
    rng = np.random.default_rng(heads + kv)
    plan, cache, q = setup(rng, [70, 0], [2, 1], heads, kv, dim, behind=1)
    check_attention(plan, cache, q, [1, 0], max_new=2)


@pytest.mark.parametrize("rows,heads,dim,rot", [(3700, 3, 128, 48), (3601, 40, 64, 64), (4001, 1, 64, 64), (3650, 1, 128, 16),
                                                (3999, 33, 128, 128), (700, 2, 64, 32)])
def test_rope_many_rows(rows, heads, dim, rot):
    # blocks of every number of rows, the last one not full, some rows left alone
    rng = np.random.default_rng(rows)
    x = bf16(rng, rows, heads, dim)
    pos = rng.integers(0, 100000, rows)
    pos[::7] = -1
    f, mag = oc.frequencies(rot)
    want, kept = oc.rope(f64(x), np.maximum(pos, 0), f, mag, False), x.clone()
    out = torch.full_like(x, 3.0)
    dg.rope(x, ints(pos.tolist()), dg.RopeFrequencies(rot), out=out)
    # a bf16 rounding, and 2^-21 of a pair's length as in the append
    size = np.abs(f64(x)).max(-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * math.sqrt(2) * size
    there = pos >= 0
    assert np.all(np.abs(f64(out) - want)[there] <= tol[there]) and (out[torch.from_numpy(~there).cuda()] == 3).all()
    assert torch.equal(x, kept)
    dg.rope(x, ints(pos.tolist()), dg.RopeFrequencies(rot), out=x)  # in place
    assert torch.equal(x[torch.from_numpy(there).cuda()], out[torch.from_numpy(there).cuda()])
    assert torch.equal(x[torch.from_numpy(~there).cuda()], kept[torch.from_numpy(~there).cuda()])
