"""What a block leaves in the context: the keys and values of its finished
canvas, encoded causally, code for code as if the finished blocks had been
appended by hand -- whatever the denoising steps appended on the way."""
import numpy as np
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
L, B, D, V, N_BLOCKS = 256, 2, 256, 1024, 3
HEADS, KV, DIM = 4, 2, 64


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


class Layer:
    """One layer over a context: queries, keys and values are looked up by
    token, so the cache says which tokens were encoded, and how."""

    def __init__(self, pages, seed, rows=B * L):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.table = torch.randn((V, HEADS + 2 * KV, DIM), generator=g, device="cuda")
        self.table *= 2.0 ** torch.randint(-3, 4, (V, 1, 1), generator=g, device="cuda")  # tokens differ in size
        self.table = self.table.to(torch.bfloat16)
        self.cache = dg.ContextCache(pages, KV, DIM)
        self.f = dg.RopeFrequencies(DIM)
        self.ws = dg.ContextWorkspace(rows, HEADS, KV, DIM)
        self.out = torch.zeros((rows, HEADS, DIM), dtype=torch.bfloat16, device="cuda")

    def __call__(self, plan, tokens, causal):
        """Append the tokens' keys and values; attend, so that a second layer's depend on the context."""
        x = torch.zeros((plan.rows, HEADS + 2 * KV, DIM), dtype=torch.bfloat16, device="cuda")
        x[:tokens.numel()] = self.table[tokens.long()]
        dg.context_append(plan, self.cache, x[:, HEADS:HEADS + KV], x[:, HEADS + KV:], rope=self.f)
        q = torch.zeros_like(self.out)
        dg.rope(x[:, :HEADS], plan.positions, self.f, out=q)
        dg.context_attention(plan, self.cache, q, self.out, self.ws, causal=ints([causal] * plan.B, torch.uint8), max_new=L)
        return self.out

    def second(self, plan, below, causal):
        """A layer above: its keys and values are the attention's results below."""
        dg.context_append(plan, self.cache, below[:, :KV], below[:, KV:2 * KV], rope=self.f)


def forward(plan, layers, tokens, causal):
    layers[1].second(plan, layers[0](plan, tokens, causal), causal)


def held_values(plan, layer, lens):
    """Codes and scales of each request's first tokens, in order."""
    got = []
    for r, n in enumerate(lens):
        page = plan.table[r, :-(-n // 64)].long()
        for c, s in ((layer.cache.k, layer.cache.k_scale), (layer.cache.v, layer.cache.v_scale)):
            got += [c[page].transpose(1, 2).reshape(-1, KV, DIM)[:n].cpu().numpy(), s[page].cpu().numpy()]
    return got


@pytest.mark.parametrize("prompts", [[128, 64], [100, 7]])
def test_a_block_is_encoded_before_it_is_committed(prompts):
    E_bits = synth.embedder_normal(V, D, seed=1)
    E = to_dev_bf16(E_bits)
    prompt = torch.randint(0, V, (sum(prompts),), device="cuda", dtype=torch.int32)
    plan, layers = dg.ContextPlan(B, B * L, 60, 20), [Layer(60, s) for s in (1, 2)]
    dg.context_plan(plan, ints(prompts))
    forward(plan, layers, prompt, True)
    params, calls = dg.Params(), []

    def hidden(j, k, canvas, committed, h):
        calls.append((j, k))
        forward(plan, layers, canvas, k == params.max_steps)
        if k == params.max_steps:
            h.fill_(float("nan"))  # not read in this call
            return
        y = synth.block_targets(j, committed.cpu().numpy(), L, V, B=B)
        h.copy_(to_dev_bf16(synth.loop_hidden(k, y, E_bits, seed=4 + 1000 * j)))
    R = B * L
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    blocks = i32(N_BLOCKS, R)
    steps = dg.generate_blocks_context(
        plan, E, hidden, N_BLOCKS, torch.empty((R, D), dtype=torch.bfloat16, device="cuda"), blocks, i32(R), i32(R),
        torch.zeros(R, dtype=torch.uint8, device="cuda"), torch.zeros(R, dtype=torch.float32, device="cuda"), i32(R), i32(R),
        i32(B), dg.Workspace(B, D, V), params)
    # the same tokens by hand, causally, on a context of their own
    ref, by_hand = dg.ContextPlan(B, B * L, 60, 20), [Layer(60, s) for s in (1, 2)]
    dg.context_plan(ref, ints(prompts))
    forward(ref, by_hand, prompt, True)
    for j in range(N_BLOCKS):
        dg.context_plan(ref, ints([L] * B), commit=True)
        forward(ref, by_hand, blocks[j], True)
    # the last block is encoded, and provisional until something commits it
    lens = [p + N_BLOCKS * L for p in prompts]
    assert plan.lens.cpu().tolist() == lens and plan.held.cpu().tolist() == [n - L for n in lens]
    for a, b in zip(layers, by_hand):
        for x, y in zip(held_values(plan, a, lens), held_values(ref, b, lens)):
            assert np.array_equal(x, y)
    # every block: its steps in order, then the call that encodes it
    for j in range(N_BLOCKS):
        assert [k for i, k in calls if i == j] == list(range(int(steps[j].max()))) + [params.max_steps]
    assert dg.context_status(plan) == 0 and all(dg.device_status(x.ws) == 0 for x in layers)


def test_an_encoding_that_fails_ends_the_generation():
    E_bits = synth.embedder_normal(V, D, seed=1)
    plan = dg.ContextPlan(B, B * L, 60, 20)
    params, seen = dg.Params(max_steps=3), []

    def hidden(j, k, canvas, committed, h):
        seen.append((j, k))
        if k == params.max_steps:
            raise ValueError("no encoder")
        h.copy_(to_dev_bf16(synth.loop_hidden(k, synth.loop_targets(L, V, seed=3, B=B), E_bits, seed=4)))
    R = B * L
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(dg.DGError) as err:
        dg.generate_blocks_context(
            plan, to_dev_bf16(E_bits), hidden, 2, torch.empty((R, D), dtype=torch.bfloat16, device="cuda"), i32(2, R), i32(R),
            i32(R), torch.zeros(R, dtype=torch.uint8, device="cuda"), torch.zeros(R, dtype=torch.float32, device="cuda"),
            i32(R), i32(R), i32(B), dg.Workspace(B, D, V), params)
    assert err.value.code == 7 and isinstance(err.value.__cause__, ValueError)
    assert seen == [(0, 0), (0, 1), (0, 2), (0, 3)]
    assert plan.held.cpu().tolist() == [0, 0]  # nothing of the block was committed


@pytest.mark.parametrize("where", [(0, 0), (1, 2), (1, 3), "workspace"])
def test_a_block_that_was_not_finished_leaves_no_slots(where):
    # the generation fails in a step, in an encoding, or before its first step; the next one goes on behind the
    # blocks that were finished, not behind slots that nobody encoded
    E_bits = synth.embedder_normal(V, D, seed=1)
    E = to_dev_bf16(E_bits)
    plan, layer = dg.ContextPlan(B, B * L, 60, 20), Layer(60, 1)
    prompts = [100, 7]
    dg.context_plan(plan, ints(prompts))
    prompt = torch.randint(0, V, (sum(prompts),), device="cuda", dtype=torch.int32)
    layer(plan, prompt, True)
    params, fail, seen = dg.Params(max_steps=3), [True], []

    def hidden(j, k, canvas, committed, h):
        if fail[0] and (j, k) == where:
            raise ValueError("stop")
        seen.append(plan.held.cpu().tolist())
        layer(plan, canvas, k == params.max_steps)
        h.copy_(to_dev_bf16(synth.loop_hidden(k, synth.loop_targets(L, V, seed=3, B=B), E_bits, seed=4)))
    R = B * L
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    blocks, ws = i32(2, R), dg.Workspace(B, D, V)

    def run():
        dg.generate_blocks_context(
            plan, E, hidden, 2, torch.zeros((R, D), dtype=torch.bfloat16, device="cuda"), blocks, i32(R), i32(R),
            torch.zeros(R, dtype=torch.uint8, device="cuda"), torch.zeros(R, dtype=torch.float32, device="cuda"), i32(R), i32(R),
            i32(B), ws, params)
    nbytes = ws.nbytes
    if where == "workspace":
        ws.nbytes = 64
    with pytest.raises(dg.DGError) as err:
        run()
    assert err.value.code == (3 if where == "workspace" else 7)
    done = 0 if where == "workspace" else where[0]
    held = [p + done * L for p in prompts]
    assert plan.held.cpu().tolist() == held and plan.lens.cpu().tolist() == held
    finished = blocks[:done].clone()
    ws.nbytes, fail[0] = nbytes, False
    seen.clear()
    run()
    assert seen[0] == held and plan.lens.cpu().tolist() == [n + 2 * L for n in held]
    ref, by_hand = dg.ContextPlan(B, B * L, 60, 20), Layer(60, 1)
    dg.context_plan(ref, ints(prompts))
    by_hand(ref, prompt, True)
    for tokens in (*finished, *blocks):
        dg.context_plan(ref, ints([L] * B), commit=True)
        by_hand(ref, tokens, True)
    for x, y in zip(held_values(plan, layer, plan.lens.tolist()), held_values(ref, by_hand, ref.lens.tolist())):
        assert np.array_equal(x, y)
    assert dg.context_status(plan) == 0
