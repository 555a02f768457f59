"""Batches that are planned over leave nothing in the held tokens: whatever
provisional rows were appended to a page on the way, its held tokens' codes and
the page's scales are those of the batches that were committed, bit for bit."""
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


def rows_of(rng, rows, heads, dim, size):
    x = rng.standard_normal((rows, 2 * heads, dim)) * size
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()


def values(codes):
    return codes.view(torch.float8_e4m3fn).double().cpu().numpy()


def state_of(cache):
    return {n: (values(getattr(cache, n)), getattr(cache, n + "_scale").double().cpu().numpy()) for n in ("k", "v")}


def append_to(state, plan, x, heads):
    """The oracle's append on a copy of a state."""
    runs, total = plan.runs.cpu().tolist(), int(plan.start[-1])
    x = x.double().cpu().numpy()[:total]
    new = {}
    for n, part in (("k", x[:, :heads]), ("v", x[:, heads:])):
        new[n] = tuple(a.copy() for a in state[n])
        oc.append(*new[n], part, runs)
    return new


def check(plan, cache, want):
    """Tokens up to each request's length, and their pages' scales."""
    for n in ("k", "v"):
        got, scales = values(getattr(cache, n)), getattr(cache, n + "_scale").double().cpu().numpy()
        for r, length in enumerate(plan.lens.cpu().tolist()):
            for j in range(-(-length // 64)):
                page, m = int(plan.table[r, j]), min(64, length - 64 * j)
                assert np.array_equal(scales[page], want[n][1][page]), (n, r, j)
                assert np.array_equal(got[page, :, :m], want[n][0][page, :, :m]), (n, r, j)


def run(plan, cache, x, heads):
    dg.context_append(plan, cache, x[:, :heads], x[:, heads:])


@pytest.mark.parametrize("dim,heads,pages", [(128, 2, 30), (64, 3, 30), (128, 1, 400), (64, 5, 400)])
def test_a_batch_planned_over_leaves_the_held_tokens(dim, heads, pages):
    rng = np.random.default_rng(dim + heads)
    plan, cache = dg.ContextPlan(2, 200, pages, 10), dg.ContextCache(pages, heads, dim)
    dg.context_plan(plan, ints([37, 100]))
    x = rows_of(rng, 200, heads, dim, 0.01)
    held = append_to(state_of(cache), plan, x, heads)
    run(plan, cache, x, heads)
    commit = True
    # large rows, larger ones (twice in a plan too), then small ones again
    for size, times in ((100.0, 1), (3000.0, 1), (10.0, 2), (1e-4, 1), (50.0, 1), (0.01, 1)):
        dg.context_plan(plan, ints([20, 60]), commit=commit)
        commit = False
        x = rows_of(rng, 200, heads, dim, size)
        want = append_to(held, plan, x, heads)
        run(plan, cache, x, heads)
        check(plan, cache, want)
        if times > 1:  # the same plan: the scale grows from where it is
            x = rows_of(rng, 200, heads, dim, 8 * size)
            want = append_to(want, plan, x, heads)
            run(plan, cache, x, heads)
            check(plan, cache, want)
    # the last batch is committed as it stands
    dg.context_plan(plan, ints([1, 0]), commit=True)
    x = rows_of(rng, 200, heads, dim, 500.0)
    want = append_to(want, plan, x, heads)
    run(plan, cache, x, heads)
    check(plan, cache, want)
    assert dg.context_status(plan) == 0


@pytest.mark.parametrize("dim,heads,pages,seed", [(128, 2, 40, 0), (64, 9, 40, 1), (64, 2, 300, 2), (128, 40, 300, 3)])
def test_any_order_of_batches(dim, heads, pages, seed):
    # commits, batches planned over, requests that add nothing or leave, sizes up and down
    rng = np.random.default_rng(seed)
    B, rows = 6, 220
    plan, cache = dg.ContextPlan(B, rows, pages, 12), dg.ContextCache(pages, heads, dim)
    held = after = state_of(cache)
    for step in range(40):
        commit = rng.random() < 0.3
        if commit:
            held = after
        add = (rng.integers(0, 36, B) * (rng.random(B) < 0.7)).tolist()
        release = (rng.random(B) < 0.08).astype(int).tolist() if rng.random() < 0.4 else None
        dg.context_plan(plan, ints(add), None if release is None else ints(release, torch.uint8), commit)
        if dg.context_status(plan) != 0:  # the pool is full: everybody leaves
            dg.context_plan(plan, ints([0] * B), ints([1] * B, torch.uint8))
            after = held
            continue
        x = rows_of(rng, rows, heads, dim, 1.0)
        x[:int(plan.start[-1])] *= torch.tensor(2.0 ** rng.integers(-9, 9, (int(plan.start[-1]), 2 * heads, 1)), device="cuda").to(torch.bfloat16)
        after = append_to(held, plan, x, heads)
        run(plan, cache, x, heads)
        # requests that add nothing are not appended to: what an earlier batch left in their page stays until they are
        busy = [r for r in range(B) if add[r] > 0]
        idle = plan.lens.clone()
        plan_view = idle.cpu().tolist()
        for n in ("k", "v"):
            got, scales = values(getattr(cache, n)), getattr(cache, n + "_scale").double().cpu().numpy()
            for r in busy:
                for j in range(-(-plan_view[r] // 64)):
                    page, m = int(plan.table[r, j]), min(64, plan_view[r] - 64 * j)
                    assert np.array_equal(scales[page], after[n][1][page]), (step, n, r, j)
                    assert np.array_equal(got[page, :, :m], after[n][0][page, :, :m]), (step, n, r, j)


def test_held_tokens_written_by_the_caller_stand():
    # the pages get other contents under the same lengths: nothing from before comes back
    rng = np.random.default_rng(5)
    heads, dim = 2, 128
    for pages in (8, 400):
        plan, cache = dg.ContextPlan(1, 64, pages, 4), dg.ContextCache(pages, heads, dim)
        dg.context_plan(plan, ints([30]))
        run(plan, cache, rows_of(rng, 64, heads, dim, 0.01), heads)
        dg.context_plan(plan, ints([10]), commit=True)
        run(plan, cache, rows_of(rng, 64, heads, dim, 100.0), heads)  # the held codes are rounded again
        page = int(plan.table[0, 0])
        cache.k[page, :, 3, 5] ^= 1       # one code of the held ones
        cache.v_scale[page] *= 2          # and the other side's scale
        want = state_of(cache)
        dg.context_plan(plan, ints([10]))
        x = rows_of(rng, 64, heads, dim, 0.01)
        want = append_to(want, plan, x, heads)
        run(plan, cache, x, heads)
        check(plan, cache, want)


def test_without_a_place_to_keep_them():
    # the earlier behaviour, for callers that hand in no place: the scale only grows
    rng = np.random.default_rng(6)
    heads, dim = 2, 64
    for field in ("kept", "epoch"):
        plan, cache = dg.ContextPlan(1, 64, 8, 4), dg.ContextCache(8, heads, dim)
        if field == "kept":
            cache._c.kept = None
        else:
            plan._c.epoch = None
        dg.context_plan(plan, ints([30]))
        x = rows_of(rng, 64, heads, dim, 0.01)
        want = append_to(state_of(cache), plan, x, heads)
        run(plan, cache, x, heads)
        for size in (100.0, 0.01):
            dg.context_plan(plan, ints([10]), commit=size == 100.0)
            x = rows_of(rng, 64, heads, dim, size)
            want = append_to(want, plan, x, heads)
            run(plan, cache, x, heads)
            check(plan, cache, want)
        assert int(cache.kept.max()) == 0


def test_planned_over_in_a_graph():
    # plan and append captured once: replays count their plans on the device
    rng = np.random.default_rng(7)
    heads, dim = 2, 128
    plan, cache = dg.ContextPlan(2, 40, 300, 6), dg.ContextCache(300, heads, dim)
    dg.context_plan(plan, ints([30, 90]))
    x = rows_of(rng, 40, heads, dim, 0.01)
    prompt = rows_of(rng, 120, heads, dim, 0.01)
    big = dg.ContextPlan(2, 120, 300, 6)
    dg.context_plan(big, ints([30, 90]))
    run(big, cache, prompt, heads)
    for n in ("table", "held", "lens", "free_list", "free_count", "free_next"):
        getattr(plan, n).copy_(getattr(big, n))
    plan.held.copy_(ints([30, 90]))
    plan.free_count.copy_(big.free_next)
    held, add = state_of(cache), ints([10, 20])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.context_plan(plan, add)
        run(plan, cache, x, heads)
    for size in (0.02, 500.0, 0.01, 20.0, 4000.0, 1e-3):
        x.copy_(rows_of(rng, 40, heads, dim, size))
        graph.replay()
        check(plan, cache, append_to(held, plan, x, heads))
    assert dg.context_status(plan) == 0


@pytest.mark.parametrize("dim,heads,rot,il", [(128, 2, 128, False), (64, 9, 48, True), (128, 20, 64, False)])
def test_rotated_keys_are_the_same_behind_a_batch_planned_over(dim, heads, rot, il):
    # the rows' codes too, to the last bit: whether a head's scale was to be taken back or not
    rng = np.random.default_rng(8)
    f = dg.RopeFrequencies(rot, interleaved=il)
    B, rows = 5, 220
    held, add = [37, 100, 1, 63, 130], [40, 30, 64, 1, 20]
    prompt = rows_of(rng, sum(held), heads, dim, 0.01)
    x, large = rows_of(rng, rows, heads, dim, 1.0), rows_of(rng, rows, heads, dim, 300.0)
    got = []
    for batches in ((x,), (large, x), (large, large, x), (x, large, x)):
        plan, cache = dg.ContextPlan(B, max(rows, sum(held)), 40, 6), dg.ContextCache(40, heads, dim)
        dg.context_plan(plan, ints(held))
        p = torch.zeros((plan.rows, 2 * heads, dim), dtype=torch.bfloat16, device="cuda")
        p[:sum(held)] = prompt
        dg.context_append(plan, cache, p[:, :heads], p[:, heads:], rope=f)
        for i, b in enumerate(batches):
            dg.context_plan(plan, ints(add), commit=i == 0)
            p[:rows] = b
            dg.context_append(plan, cache, p[:, :heads], p[:, heads:], rope=f)
        state = []
        for r, n in enumerate(plan.lens.cpu().tolist()):
            page = plan.table[r, :-(-n // 64)].long()
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
                state += [c[page].transpose(1, 2).reshape(-1, heads, dim)[:n], s[page]]
        got.append(state)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("pages", [4, 300])
def test_a_page_that_is_begun_again_has_nothing_of_before(pages):
    # a request's tokens, all but 0 beside a later batch, and the next one's on the same page, all 0 under the same
    # scale: nothing tells the two pages' codes apart
    heads, dim = 2, 64
    plan, cache = dg.ContextPlan(1, 64, pages, 4), dg.ContextCache(pages, heads, dim)
    x = torch.full((64, 2 * heads, dim), 1e-6, dtype=torch.bfloat16, device="cuda")
    dg.context_plan(plan, ints([20]))
    run(plan, cache, x, heads)
    x.fill_(400.0)
    dg.context_plan(plan, ints([5]), commit=True)
    run(plan, cache, x, heads)
    page = int(plan.table[0, 0])
    assert cache.k_scale[page].tolist() == [1.0] * heads and int(cache.k[page, :, :20].max()) == 0
    dg.context_plan(plan, ints([20]), release=ints([1], torch.uint8))
    assert int(plan.table[0, 0]) == page
    x.zero_()
    run(plan, cache, x, heads)
    x.fill_(0.01)
    dg.context_plan(plan, ints([5]), commit=True)
    want = append_to(state_of(cache), plan, x, heads)
    run(plan, cache, x, heads)
    check(plan, cache, want)
    assert int(cache.k[page, :, :20].max()) == 0 and cache.k_scale[page].tolist() == [1.0] * heads
