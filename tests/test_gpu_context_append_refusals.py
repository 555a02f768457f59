"""Keys and values that append refuses, one property wrong at a time: each once as
the keys beside good values and once as the values beside good keys."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_canvas_denoising_b200 as dg  # noqa: E402
from block_canvas_denoising_b200 import build as dg_build  # noqa: E402

dg_build.build()
ROWS, KV, DIM = 14, 2, 128


def zeros(*shape, dtype=torch.bfloat16, device="cuda"):
    return torch.zeros(shape, dtype=dtype, device=device)


BAD = [("type", lambda: zeros(ROWS, KV, DIM, dtype=torch.float32), 1), ("half", lambda: zeros(ROWS, KV, DIM, dtype=torch.float16), 1),
       ("device", lambda: zeros(ROWS, KV, DIM, device="cpu"), 1), ("dimensions", lambda: zeros(ROWS, KV * DIM), 1),
       ("rows", lambda: zeros(ROWS - 1, KV, DIM), 2), ("heads", lambda: zeros(ROWS, KV + 1, DIM), 2),
       ("width", lambda: zeros(ROWS, KV, DIM // 2), 2), ("inner stride", lambda: zeros(ROWS, KV, 2 * DIM)[:, :, ::2], 1),
       ("alignment", lambda: zeros(ROWS, KV, DIM + 8)[:, :, 1:DIM + 1], 1), ("head stride", lambda: zeros(ROWS, KV, DIM + 4)[:, :, :DIM], 1),
       ("broadcast rows", lambda: zeros(1, KV, DIM).expand(ROWS, KV, DIM), 1),
       ("broadcast heads", lambda: zeros(ROWS, 1, DIM).expand(ROWS, KV, DIM), 1)]


@pytest.mark.parametrize("name,make,code", BAD, ids=[b[0] for b in BAD])
def test_one_thing_wrong(name, make, code):
    plan, cache = dg.ContextPlan(1, ROWS, 4, 4), dg.ContextCache(4, KV, DIM)
    dg.context_plan(plan, torch.tensor([10], dtype=torch.int32, device="cuda"))
    good = torch.randn((ROWS, KV, DIM), device="cuda").to(torch.bfloat16)
    bad = make()
    for k, v in ((bad, good), (good, bad)):
        with pytest.raises(dg.DGError) as err:
            dg.context_append(plan, cache, k, v)
        assert err.value.code == code
    torch.cuda.synchronize()
    assert int(cache.k.max()) == 0 and int(cache.v.max()) == 0  # nothing was written
    dg.context_append(plan, cache, good, good)  # the good pair is accepted
    torch.cuda.synchronize()
    assert int(cache.k.max()) > 0 and torch.equal(cache.k, cache.v) and dg.context_status(plan) == 0
