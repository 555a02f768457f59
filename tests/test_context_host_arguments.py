"""Numbers that the C types cannot hold are refused, not cut: a window of 2^32 + 5
is not one of 5.  All before the library is called (so: without a device)."""
import types

import pytest

import block_canvas_denoising_b200 as dg
from block_canvas_denoising_b200 import build as dg_build

torch = pytest.importorskip("torch")
dg_build.build()


def attend(**kw):
    plan, cache = dg.ContextPlan(1, 4, 8, 8, device="cpu"), dg.ContextCache(8, 2, 64, device="cpu")
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    ws = types.SimpleNamespace(buf=torch.zeros(1, dtype=torch.uint8), nbytes=1)
    dg.context_attention(plan, cache, q, torch.zeros_like(q), ws, **kw)


@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(window=-2 ** 32), dict(max_new=2 ** 32 + 1),
                                dict(scale=1e-50), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))])
def test_attention(kw):
    with pytest.raises(dg.DGError) as err:
        attend(**kw)
    assert err.value.code == 1


@pytest.mark.parametrize("kw", [dict(original_length=2 ** 32 + 4096), dict(rot=2 ** 32 + 64), dict(original_length=2 ** 31)])
def test_frequencies(kw):
    args = dict(rot=64, scaling="parts", factor=8.0, device="cpu")
    args.update(kw)
    with pytest.raises(dg.DGError) as err:
        dg.RopeFrequencies(**args)
    assert err.value.code == 1


def test_sizes():
    with pytest.raises(dg.DGError):
        dg.ContextPlan(1, 4, 8, 2 ** 32 + 8, device="meta")
    with pytest.raises(dg.DGError):
        dg.ContextCache(2 ** 32 + 8, 2, 64, device="meta")
    with pytest.raises(dg.DGError):
        dg.context_workspace_size(2 ** 32 + 16, 4, 2, 128)
