"""Block-by-block generation with a context: the blocks are those of
``generate_blocks`` bit for bit, and whenever the hidden-state producer is
called the plan holds its canvas's slots behind everything committed -- checked
by running a layer of append and attention over them inside the producer."""
import math

import numpy as np
import pytest

import synth
from dg_testlib import to_dev_bf16
from oracle import context as oc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_canvas_denoising_b200 as dg  # noqa: E402
from block_canvas_denoising_b200 import build as dg_build  # noqa: E402

dg_build.build()
L, B, D, V, N_BLOCKS = 256, 2, 256, 1024, 3


def _buffers():
    R = B * L
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(h_buf=torch.empty((R, D), dtype=torch.bfloat16, device="cuda"), blocks=i32(N_BLOCKS, R), canvas=i32(R),
                prev_argmax=i32(R), accept=torch.zeros(R, dtype=torch.uint8, device="cuda"),
                entropy=torch.zeros(R, dtype=torch.float32, device="cuda"), sampled=i32(R), argmax=i32(R), stop=i32(B))


def _hidden(E_bits, layer=None):
    def hidden(j, k, canvas, committed, h):
        y = synth.block_targets(j, committed.cpu().numpy(), L, V, B=B)
        h.copy_(to_dev_bf16(synth.loop_hidden(k, y, E_bits, seed=4 + 1000 * j)))
        if layer is not None:
            layer(j, k, h)
    return hidden


def test_blocks_over_a_context():
    E_bits = synth.embedder_normal(V, D, seed=1)
    E = to_dev_bf16(E_bits)
    prompts = [100, 7]
    plan = dg.ContextPlan(B, B * L, 40, 20)
    heads, kv, dim = 4, 2, 64  # 256 = D wide
    cache = dg.ContextCache(plan.pages, kv, dim)
    f = dg.RopeFrequencies(dim)
    ws_a = dg.ContextWorkspace(plan.rows, heads, kv, dim)
    out = torch.zeros((B * L, heads, dim), dtype=torch.bfloat16, device="cuda")
    dg.context_plan(plan, torch.tensor(prompts, dtype=torch.int32, device="cuda"))
    prompt = torch.randn((B * L, heads, dim), device="cuda").to(torch.bfloat16)
    dg.context_append(plan, cache, prompt[:, :kv], prompt[:, kv:], rope=f)
    calls = []

    def layer(j, k, h):
        held = [p + j * L for p in prompts]
        assert plan.held.cpu().tolist() == held and plan.lens.cpu().tolist() == [n + L for n in held]
        assert plan.start.cpu().tolist() == [0, L, 2 * L]
        x = h.view(B * L, heads, dim)
        dg.context_append(plan, cache, x[:, :kv], x[:, kv:], rope=f)
        q = dg.rope(x, plan.positions, f)
        dg.context_attention(plan, cache, q, out, ws_a, max_new=L)
        r, i = 1, 17  # one row against the oracle
        n = held[r] + L
        page = plan.table[r].cpu().numpy()[:-(-n // 64)]
        kk, vv = ((getattr(cache, m).view(torch.float8_e4m3fn).double() * getattr(cache, m + "_scale").double()[..., None, None])
                  .cpu().numpy()[page].transpose(0, 2, 1, 3).reshape(-1, kv, dim)[:n] for m in ("k", "v"))
        w, _, mass, size = oc.attention(q[r * L + i:r * L + i + 1].cpu().double().numpy(), kk, vv, dim ** -0.5, False, 0)
        err = np.abs(out[r * L + i].cpu().double().numpy() - w[0])
        d = ((dim + 4) * 2.0 ** -24 * size[0][:, None] + 2.0 ** -17 * dim ** -0.5 * np.abs(kk).sum(-1).max() *
             q[r * L + i].abs().amax(-1, keepdim=True).cpu().double().numpy())
        # Beside the bound of test_gpu_context.py: float16 weights go up to 2^10 in steps of 2^-24 at the
        # least, so a weight far below the largest is off by up to 2^-25 / 2^10 = 2^-35 of it, times its
        # code (at most 448) and page scale.  It shows here: in some columns every token with weight has
        # the value 0, and the others' sum is 1e-13.
        tail = 2.0 ** -35 * n * 448 * cache.v_scale[torch.from_numpy(page).long().cuda()].max().item()
        tol = 2.0 ** -8 * np.abs(w[0]) + (2.0 ** -11 + 2.0 ** -18 + 2 * d) * mass[0] + tail
        at = np.unravel_index(np.argmax(err / tol), err.shape)
        assert np.all(err <= tol), (j, k, at, err[at], tol[at], w[0][at], mass[0][at], size[0])
        calls.append((j, k))

    results = []
    for use in (False, True):
        b = _buffers()
        args = (E, _hidden(E_bits, layer if use else None), N_BLOCKS, b["h_buf"], b["blocks"], b["canvas"],
                b["prev_argmax"], b["accept"], b["entropy"], b["sampled"], b["argmax"], b["stop"], dg.Workspace(B, D, V))
        steps = dg.generate_blocks_context(plan, *args) if use else dg.generate_blocks(*args)
        results.append((steps, b["blocks"].cpu().numpy()))
    assert np.array_equal(results[0][0], results[1][0]) and np.array_equal(results[0][1], results[1][1])
    assert {j for j, _ in calls} == set(range(N_BLOCKS))
    # the last block stays provisional until something commits it
    assert plan.held.cpu().tolist() == [p + 2 * L for p in prompts]
    assert dg.context_status(plan) == 0 and dg.device_status(ws_a) == 0
    assert math.isfinite(out.float().abs().max().item())


def test_a_pool_that_is_too_small_ends_the_generation():
    E_bits = synth.embedder_normal(V, D, seed=1)
    plan = dg.ContextPlan(B, B * L, 12, 20)  # one block of 2 x 4 pages, not two
    b = _buffers()
    seen = []
    hidden = _hidden(E_bits, lambda j, k, h: seen.append(j))
    with pytest.raises(dg.DGError) as err:
        dg.generate_blocks_context(plan, to_dev_bf16(E_bits), hidden, N_BLOCKS, b["h_buf"], b["blocks"], b["canvas"],
                                   b["prev_argmax"], b["accept"], b["entropy"], b["sampled"], b["argmax"], b["stop"],
                                   dg.Workspace(B, D, V))
    assert err.value.code == 10 and set(seen) == {0}


def test_context_ops_inside_the_device_loop():
    # the hidden-state graph of the device loop runs a layer over the context
    # every step; the last step's attention equals the same calls made eagerly
    E_bits = synth.embedder_normal(V, D, seed=1)
    E = to_dev_bf16(E_bits)
    y = synth.loop_targets(L, V, seed=3, B=B)
    table = torch.stack([to_dev_bf16(synth.loop_hidden(k, y, E_bits, seed=4)).reshape(-1) for k in range(48)])
    heads, kv, dim = 4, 2, 64
    plan = dg.ContextPlan(B, B * L, 40, 20)
    cache = dg.ContextCache(plan.pages, kv, dim)
    f = dg.RopeFrequencies(dim)
    ws_a = dg.ContextWorkspace(plan.rows, heads, kv, dim)
    out, q = (torch.zeros((B * L, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.context_plan(plan, torch.full((B,), L, dtype=torch.int32, device="cuda"))
    b = _buffers()

    def layer(h, cache, out):
        x = h.view(B * L, heads, dim)
        dg.context_append(plan, cache, x[:, :kv], x[:, kv:], rope=f)
        dg.rope(x, plan.positions, f, out=q)
        dg.context_attention(plan, cache, q, out, ws_a, max_new=L)
    state = dg.LoopState(B)
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        b["h_buf"].view(-1).copy_(torch.index_select(table, 0, state.k.to(torch.int64).clamp(0, 47))[0])
        layer(b["h_buf"], cache, out)
    steps = dg.denoise_loop_graph(E, g, b["h_buf"], b["canvas"], b["prev_argmax"], np.zeros(B, np.uint8), b["accept"],
                                  b["entropy"], b["sampled"], b["argmax"], b["stop"], dg.Workspace(B, D, V), state)
    torch.cuda.synchronize()
    last = int(steps.max()) - 1
    again, cache2 = torch.zeros_like(out), dg.ContextCache(plan.pages, kv, dim)
    layer(table[last].view(B * L, D), cache2, again)
    assert torch.equal(out, again) and out.abs().max() > 0
    assert dg.context_status(plan) == 0 and dg.device_status(ws_a) == 0
