"""Queries that are not finite give NaN in their own row and head wherever they
see a token -- whichever of a page's tokens those are -- and change nothing else."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_canvas_denoising_b200 as dg  # noqa: E402
from block_canvas_denoising_b200 import build as dg_build  # noqa: E402

dg_build.build()


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def context(held, add, heads, kv, dim, seed):
    """A context whose requests hold tokens of random keys and values, and queries."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, rows = len(held), max(sum(held), sum(add))
    plan, cache = dg.ContextPlan(B, rows, 40, 16), dg.ContextCache(40, kv, dim)
    for commit, n in ((False, held), (True, add)):
        dg.context_plan(plan, ints(n), commit=commit)
        x = torch.randn((rows, 2 * kv, dim), generator=g, device="cuda").to(torch.bfloat16)
        dg.context_append(plan, cache, x[:, :kv], x[:, kv:])
    q = torch.randn((rows, heads, dim), generator=g, device="cuda").to(torch.bfloat16)
    return plan, cache, q


def attend(plan, cache, q, causal, window, most):
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device="cuda")
    ws = dg.ContextWorkspace(plan.rows, q.shape[1], cache.heads, cache.dim)
    dg.context_attention(plan, cache, q, out, ws, causal=ints(causal, torch.uint8), window=window, lse=lse, max_new=most)
    assert dg.device_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("add,most", [([200, 70], 0), ([2, 1], 2)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 2, 7])
def test_every_position_of_a_page(add, most, dim, window):
    # held lengths move the few rows over every position of a page as well
    for shift in range(0, 64, 64 if most == 0 else 3):
        plan, cache, q = context([37 + shift, 130], add, 4, 2, dim, seed=dim + shift)
        rows = sum(add)
        clean, clean_lse = attend(plan, cache, q, [1, 1], window, most)
        assert torch.isfinite(clean[:rows].float()).all()
        for value in (math.nan, math.inf, -math.inf):
            mark = torch.zeros((q.shape[0], 4), dtype=torch.bool, device="cuda")
            bad = q.clone()
            for i in range(rows):
                bad[i, i % 4, (7 * i) % dim] = value
                mark[i, i % 4] = True
            out, lse = attend(plan, cache, bad, [1, 1], window, most)
            assert torch.isnan(out[mark]).all() and torch.isnan(lse[mark]).all(), (shift, value)
            assert torch.equal(out[~mark], clean[~mark]) and torch.equal(lse[~mark], clean_lse[~mark])


@pytest.mark.parametrize("add,most", [([200, 70], 0), ([2, 1], 2)])
def test_rows_that_see_nothing_give_zero(add, most):
    # lengths shortened by the caller, and pages that are not there: not even a query that is not finite sees a token
    plan, cache, q = context([37, 130], add, 4, 2, 128, seed=1)
    rows = sum(add)
    q[:, 1, 3] = math.nan
    table, lens = plan.table.clone(), plan.lens.clone()
    plan.lens.copy_(ints([0, 0]))
    out, lse = attend(plan, cache, q, [1, 0], 0, most)
    assert (out[:rows] == 0).all() and torch.isneginf(lse[:rows]).all()
    plan.lens.copy_(lens)
    plan.table.fill_(-1)
    out, lse = attend(plan, cache, q, [1, 0], 0, most)
    assert (out[:rows] == 0).all() and torch.isneginf(lse[:rows]).all()
    # one page there: rows that see some of it are NaN in that head, the others 0
    plan.table[0, 1] = table[0, 1]
    out, _ = attend(plan, cache, q, [1, 1], 5, most)
    first = 37  # position of row 0
    sees = np.array([any(64 <= p < 128 for p in range(max(first + i - 4, 0), first + i + 1)) for i in range(add[0])])
    got = out[:add[0], 1].float().cpu().numpy()
    assert np.isnan(got[sees]).all() and (got[~sees] == 0).all()
    assert (out[add[0]:rows] == 0).all()
