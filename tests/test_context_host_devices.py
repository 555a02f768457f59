"""The block driver refuses tensors of another device than its plan's, before it
calls the library (so: without a device)."""
import types

import pytest

import block_canvas_denoising_b200 as dg
from block_canvas_denoising_b200 import build as dg_build

torch = pytest.importorskip("torch")
dg_build.build()

NAMES = ("E", "h_buf", "blocks", "canvas", "prev_argmax", "accept", "entropy", "sampled", "argmax", "stop")


def call(here, there=(), stream=None, e_scale=None):
    """Tensors on device `here`, those named in `there` on another."""
    plan = dg.ContextPlan(1, 256, 8, 8, device=here)
    other = "meta" if here == "cpu" else "cpu"
    made = {n: torch.zeros(1, device=other if n in there else here) for n in (*NAMES, "ws")}
    made["h_buf"], made["E"] = made["h_buf"].view(1, 1), made["E"].view(1, 1)
    ws = types.SimpleNamespace(buf=made["ws"], nbytes=1)
    dg.generate_blocks_context(plan, made["E"], lambda *a: None, 1, *(made[n] for n in NAMES[1:]), ws, e_scale=e_scale,
                               stream=stream)


@pytest.mark.parametrize("name", [*NAMES, "ws"])
def test_a_tensor_of_another_device(name):
    with pytest.raises(dg.DGError) as err:
        call("cpu", (name,))
    assert err.value.code == 1 and ("workspace" if name == "ws" else name) in str(err.value)


def test_scales_and_streams_of_another_device():
    with pytest.raises(dg.DGError) as err:
        call("cpu", e_scale=torch.zeros(1, device="meta"))
    assert err.value.code == 1 and "e_scale" in str(err.value)
    with pytest.raises(dg.DGError) as err:
        call("cpu", stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
    assert err.value.code == 1 and "stream" in str(err.value)
