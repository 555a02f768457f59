"""What a call allocates for its result belongs to the stream it runs on: memory
that the current stream is still using is not handed to another one."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_canvas_denoising_b200 as dg  # noqa: E402
from block_canvas_denoising_b200 import build as dg_build  # noqa: E402

dg_build.build()


def late_fill(nbytes, value):
    """Memory that goes back to the current stream's pool while a fill of it is still queued there."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # nothing else to hand out
    buf = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # some tenth of a second
    buf.fill_(value)
    del buf


def test_rope_makes_its_result_on_its_stream():
    rows, heads, dim = 3000, 8, 128
    x = torch.randn((rows, heads, dim), device="cuda").to(torch.bfloat16)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    f = dg.RopeFrequencies(dim)
    want = dg.rope(x, pos, f)
    side = torch.cuda.Stream()
    for _ in range(3):  # the first calls load what they need, which may wait for the device
        late_fill(x.numel() * 2, 7)
        out = dg.rope(x, pos, f, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del out


def test_workspaces_are_made_on_their_stream():
    side = torch.cuda.Stream()
    sizes = [dg.context_workspace_size(64, 4, 2, 128), dg.workspace_size(1, 256, 1024)]
    for make, n in zip((lambda: dg.ContextWorkspace(64, 4, 2, 128, stream=side),
                        lambda: dg.Workspace(1, 256, 1024, stream=side)), sizes):
        late_fill(n, 255)
        ws = make()
        torch.cuda.synchronize()
        assert dg.device_status(ws) == 0  # the latch and the tickets are 0, not 255s
        assert int(ws.buf[:256].max()) == 0


def test_rope_rows_without_a_position_of_a_new_tensor_are_zero():
    x = torch.randn((70, 3, 64), device="cuda").to(torch.bfloat16)
    pos = torch.arange(70, dtype=torch.int32, device="cuda")
    pos[::3] = -1
    f = dg.RopeFrequencies(64)
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        late = torch.full_like(x, 9.0)
        del late  # the next tensor of this size
        out = dg.rope(x, pos, f, stream=stream)
        torch.cuda.synchronize()
        assert (out[::3] == 0).all() and out[1::3].abs().max() > 0


def test_a_producer_runs_on_the_stream_of_its_steps():
    # it fills h late: steps that did not wait would read the call before's
    import numpy as np
    import synth
    from dg_testlib import to_dev_bf16
    L, B, D, V, n_blocks = 256, 1, 256, 1024, 2
    R = L * B
    E_bits = synth.embedder_normal(V, D, seed=1)
    E = to_dev_bf16(E_bits)
    y = synth.loop_targets(L, V, seed=3, B=B)
    table = [to_dev_bf16(synth.loop_hidden(k, y, E_bits, seed=4)) for k in range(49)]
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(name, stream):
        h = torch.zeros((R, D), dtype=torch.bfloat16, device="cuda")
        blocks, canvas = i32(n_blocks, R), i32(R)
        late = stream is not None

        def hidden(*args):
            k = args[0] if name == "loop" else args[1]
            if late:
                assert torch.cuda.current_stream() == stream
                torch.cuda._sleep(3_000_000)
            h.copy_(table[k])
        outs = (torch.zeros(R, dtype=torch.uint8, device="cuda"), torch.zeros(R, dtype=torch.float32, device="cuda"), i32(R),
                i32(R), i32(B), dg.Workspace(B, D, V))
        torch.cuda.synchronize()
        if name == "loop":
            steps = dg.denoise_loop(E, hidden, h, canvas, i32(R), np.zeros(B, np.uint8), *outs, stream=stream)
            result = canvas
        else:
            args = (E, hidden, n_blocks, h, blocks, canvas, i32(R), *outs)
            if name == "context":
                steps = dg.generate_blocks_context(dg.ContextPlan(B, R, 20, 10), *args, stream=stream)
            else:
                steps = dg.generate_blocks(*args, stream=stream)
            result = blocks
        torch.cuda.synchronize()
        return steps, result
    for name in ("loop", "blocks", "context"):
        want = run(name, None)
        got = run(name, torch.cuda.Stream())
        assert np.array_equal(want[0], got[0]) and torch.equal(want[1], got[1]), name
