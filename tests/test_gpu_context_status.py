"""Reports of a context: none is lost behind another, and a generation says of a
key or value that is not finite before the block it belongs to is committed."""
import math

import pytest

import synth
from dg_testlib import to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_canvas_denoising_b200 as dg  # noqa: E402
from block_canvas_denoising_b200 import build as dg_build  # noqa: E402

dg_build.build()
L, B, D, V = 256, 2, 256, 1024


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def test_a_value_is_reported_after_a_refused_plan():
    plan, cache = dg.ContextPlan(1, 100, 2, 8), dg.ContextCache(2, 2, 64)
    x = torch.randn((100, 4, 64), device="cuda").to(torch.bfloat16)
    x[5, 0, 3] = math.inf
    dg.context_plan(plan, ints([60]))
    dg.context_append(plan, cache, x[:, :2], x[:, 2:])
    dg.context_plan(plan, ints([100]), commit=True)  # 160 tokens do not fit two pages
    assert dg.context_status(plan) == 10 and dg.context_status(plan) == 10
    dg.context_plan(plan, ints([60]))
    assert dg.context_status(plan) == 9 and dg.context_status(plan) == 0


def generate(plan, cache, bad, n_blocks=2):
    """Blocks whose producer appends a NaN in the call (block, step) that `bad` names; the calls made."""
    E_bits = synth.embedder_normal(V, D, seed=1)
    params, calls = dg.Params(max_steps=3), []

    def hidden(j, k, canvas, committed, h):
        calls.append((j, k))
        h.copy_(to_dev_bf16(synth.loop_hidden(k, synth.loop_targets(L, V, seed=3, B=B), E_bits, seed=4)))
        x = h.view(B * L, 4, 64).clone()
        if (j, k) == bad:
            x[300, 1, 7] = math.nan
        dg.context_append(plan, cache, x[:, :2], x[:, 2:])
    R = B * L
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    try:
        dg.generate_blocks_context(
            plan, to_dev_bf16(E_bits), hidden, n_blocks, torch.empty((R, D), dtype=torch.bfloat16, device="cuda"),
            i32(n_blocks, R), i32(R), i32(R), torch.zeros(R, dtype=torch.uint8, device="cuda"),
            torch.zeros(R, dtype=torch.float32, device="cuda"), i32(R), i32(R), i32(B), dg.Workspace(B, D, V), params)
    except dg.DGError as err:
        return err.code, calls
    return 0, calls


@pytest.mark.parametrize("bad,held", [((0, 1), 0), ((0, 3), 0), ((1, 0), L), ((1, 3), L)])
def test_a_value_ends_the_generation_before_it_is_committed(bad, held):
    plan, cache = dg.ContextPlan(B, B * L, 40, 20), dg.ContextCache(40, 2, 64)
    code, calls = generate(plan, cache, bad)
    assert code == 9 and plan.held.cpu().tolist() == [held] * B
    assert calls[-1] == (bad[0], 3)  # the block is finished, the next not begun
    assert dg.context_status(plan) == 0  # said once


def test_a_prompt_value_ends_the_generation_at_once():
    plan, cache = dg.ContextPlan(B, B * L, 40, 20), dg.ContextCache(40, 2, 64)
    x = torch.full((B * L, 4, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    dg.context_plan(plan, ints([3, 4]))
    dg.context_append(plan, cache, x[:, :2], x[:, 2:])
    assert generate(plan, cache, None) == (9, [])
    code, calls = generate(plan, cache, None)  # nothing left to say
    assert code == 0 and calls[-1] == (1, 3) and dg.context_status(plan) == 0
