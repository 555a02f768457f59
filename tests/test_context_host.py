"""The context on the CPU: the oracle's pieces against independent ones, the
library's host functions, and its refusals (all before any device work)."""
import ctypes
import math

import numpy as np
import pytest

import block_canvas_denoising_b200 as dg
from block_canvas_denoising_b200 import build as dg_build
from oracle import context as oc

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def libdg():
    dg_build.build()
    return dg.lib()


# ---- the oracle ----
def test_oracle_rounding_matches_an_independent_e4m3():
    x = np.concatenate([np.linspace(-500, 500, 4001), oc.E4M3, -oc.E4M3, (oc.E4M3[1:] + oc.E4M3[:-1]) / 2,
                        2.0 ** np.arange(-14, 9), [0.0, 2.0 ** -10, 2.0 ** -10 * 1.0001]])
    want = torch.tensor(np.clip(x, -448, 448), dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oc.round_e4m3(x), want)


@pytest.mark.parametrize("top", [448.0, 448.0000001, 447.99, 1.0, 0.875, 0.8750001, 3e38, 1e-30, 1e-42])
def test_oracle_scale_is_the_least_power_of_two(top):
    s = oc.scale_of(top)
    assert math.log2(s) == int(math.log2(s)) and top <= 448 * s
    assert s == 2.0 ** -100 or top > 448 * s / 2


def test_oracle_rope_keeps_norms_and_relative_positions():
    rng = np.random.default_rng(0)
    for scaling in ("none", "linear", "ntk", "parts"):
        f, mag = oc.frequencies(64, scaling=scaling, factor=8.0)
        for il in (False, True):
            x, y = rng.standard_normal((2, 1, 1, 96))
            for p in (0, 5, 70000):
                a, b = oc.rope(x, [p], f, 1.0, il), oc.rope(y, [p + 11], f, 1.0, il)
                c, d = oc.rope(x, [0], f, 1.0, il), oc.rope(y, [11], f, 1.0, il)
                assert abs(np.linalg.norm(a) - np.linalg.norm(x)) < 1e-12
                assert abs((a * b).sum() - (c * d).sum()) < 1e-9  # only the distance counts
            assert np.allclose(oc.rope(x, [0], f, mag, il)[..., :64], mag * x[..., :64])


def test_oracle_attention_matches_a_direct_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 6, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    for causal in (False, True):
        for window in (0, 3):
            out, lse, _, _ = oc.attention(q, k, v, 0.5, causal, window)
            kk, vv = np.repeat(k, 3, axis=1), np.repeat(v, 3, axis=1)
            z = 0.5 * torch.einsum("ihd,nhd->hin", torch.tensor(q), torch.tensor(kk))
            pos, key = torch.arange(4, 9)[:, None], torch.arange(9)
            hide = (key > pos) if causal else torch.zeros(5, 9, dtype=torch.bool)
            if window:
                hide = hide | (key <= pos - window)
            z = z.masked_fill(hide, -math.inf)
            want = torch.einsum("hin,nhd->ihd", torch.softmax(z, -1), torch.tensor(vv)).numpy()
            assert np.allclose(out, want, atol=1e-12)
            assert np.allclose(lse, torch.logsumexp(z, -1).numpy().T, atol=1e-12)


def test_oracle_plan_by_hand():
    # 2 requests, 6 pages: request 0 holds 65 tokens (2 pages), request 1 none
    p = oc.plan([[4, 2, -1], [-1, -1, -1]], [65, 0], [0, 1, 3, 5, 9, 9], 4, [63, 65], None, 128)
    assert p["table"] == [[4, 2, -1], [5, 3, -1]] and p["free_next"] == 2 and p["free_count"] == 4
    assert p["lens"] == [128, 65] and p["start"] == [0, 63, 128] and p["status"] == 0
    assert p["runs"][:3] == [[2, 0, 1, 63], [5, 63, 0, 64], [3, 127, 0, 1]] and p["runs"][3] == [-1, 0, 0, 0]
    assert p["positions"][:2] == [65, 66] and p["slots"][0] == 2 * 64 + 1 and p["slots"][127] == 3 * 64
    # request 0 leaves: its pages are on top of the stack and taken again
    p = oc.plan([[4, 2, -1], [-1, -1, -1]], [65, 0], [0, 1, 3, 5, 9, 9], 4, [0, 65], [1, 0], 128)
    assert p["table"][1][:2] == [2, 4] and p["free_next"] == 4 and p["held"] == [0, 0]
    for add, code in (([64 * 3, 64], 3), ([100, 100], 2), ([-1, 0], 3)):
        p = oc.plan([[4, 2, -1], [-1, -1, -1]], [65, 0], [0, 1, 3, 5], 4, add, None, 128)
        assert p["status"] == code and p["start"] == [0, 0, 0] and p["lens"] == [65, 0] and p["free_next"] == 4
    assert oc.plan([[4, 2, -1], [-1, -1, -1]], [65, 0], [0, 1, 3, 5], 1, [64, 64], None, 128)["status"] == 1


# ---- the library on the host ----
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts"])
@pytest.mark.parametrize("rot,base,factor,length", [(128, 10000.0, 8.0, 4096), (16, 500000.0, 1.0, 1), (48, 1e6, 32.0, 8192)])
def test_rope_frequencies(libdg, scaling, rot, base, factor, length):
    f, mag = np.zeros(rot // 2), ctypes.c_float()
    code = libdg.dg_rope_frequencies(rot, base, ["none", "linear", "ntk", "parts"].index(scaling), factor, length,
                                     f.ctypes.data_as(ctypes.c_void_p), ctypes.byref(mag))
    want, m = oc.frequencies(rot, base, scaling, factor, length)
    assert code == 0 and np.allclose(f, want, rtol=1e-14, atol=0) and mag.value == np.float32(m)


def test_rope_frequency_refusals(libdg):
    f, mag = np.zeros(64), ctypes.c_float()

    def call(rot=64, base=1e4, scaling=0, factor=1.0, length=4096, out=f.ctypes.data_as(ctypes.c_void_p)):
        return libdg.dg_rope_frequencies(rot, base, scaling, factor, length, out, ctypes.byref(mag))
    assert call() == 0
    assert call(rot=0) == 2 and call(rot=24) == 2 and call(rot=144) == 2
    for bad in (dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(scaling=4), dict(scaling=-1),
                dict(factor=0.5), dict(factor=math.nan), dict(length=0), dict(out=None)):
        assert call(**bad) == 1, bad
    with pytest.raises(dg.DGError):
        dg.RopeFrequencies(64, scaling="other", device="cpu")


FAKE = 4096  # an aligned address that no refused call dereferences


def _ctx(**kw):
    c = dg._Context(2, 256, 8, 4, *([FAKE] * 11))
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _cache(**kw):
    c = dg._Cache(8, 2, 128, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _heads(**kw):
    h = dg._Heads(FAKE, 512, 128)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


BAD_CONTEXTS = [(dict(B=0), 2), (dict(B=257), 2), (dict(rows=0), 2), (dict(rows=1 << 25), 2), (dict(pages=0), 2),
                (dict(max_pages=0), 2), (dict(table=None), 1), (dict(runs=FAKE + 8), 1), (dict(slots=FAKE + 4), 1),
                (dict(status=None), 1), (dict(lens=FAKE + 2), 1)]
BAD_CACHES = [(dict(dim=96), 2), (dict(dim=256), 2), (dict(heads=0), 2), (dict(heads=1025), 2), (dict(pages=9), 2),
              (dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(k_scale=None), 1), (dict(v_scale=FAKE + 2), 1)]
BAD_HEADS = [dict(data=None), dict(data=FAKE + 8), dict(row_stride=500), dict(head_stride=100), dict(row_stride=64),
             dict(head_stride=64), dict(row_stride=-512), dict(head_stride=0)]


def _ref(x):
    return None if x is None else ctypes.byref(x)


def test_plan_refusals(libdg):
    for kw, code in BAD_CONTEXTS:
        assert libdg.dg_context_plan(_ref(_ctx(**kw)), FAKE, None, 0, None) == code, kw
        assert libdg.dg_context_status(_ref(_ctx(**kw)), None) == code, kw
    assert libdg.dg_context_plan(None, FAKE, None, 0, None) == 1
    assert libdg.dg_context_plan(_ref(_ctx()), None, None, 0, None) == 1
    assert libdg.dg_context_plan(_ref(_ctx()), FAKE + 1, None, 0, None) == 1


def test_rope_refusals(libdg):
    good = dg._RopeArgs(64, 0, 1.0, FAKE)

    def call(x=_heads(), out=_heads(data=2 * FAKE), rows=4, heads=4, dim=128, pos=FAKE, rope=good):
        return libdg.dg_rope(_ref(x), _ref(out), rows, heads, dim, pos, _ref(rope), None)
    for kw in BAD_HEADS:
        assert call(x=_heads(**kw)) == 1 and call(out=_heads(**kw)) == 1, kw
    assert call(x=None) == 1 and call(rope=None) == 1 and call(pos=None) == 1 and call(pos=FAKE + 2) == 1
    assert call(rows=-1) == 2 and call(heads=0) == 2 and call(dim=32) == 2
    for r in (dg._RopeArgs(0, 0, 1.0, FAKE), dg._RopeArgs(24, 0, 1.0, FAKE), dg._RopeArgs(144, 0, 1.0, FAKE),
              dg._RopeArgs(64, 0, math.nan, FAKE), dg._RopeArgs(64, 0, math.inf, FAKE), dg._RopeArgs(64, 0, 1.0, None),
              dg._RopeArgs(64, 0, 1.0, FAKE + 4)):
        assert call(rope=r) == 1
    assert call(out=_heads(row_stride=1024)) == 1  # in place with other strides


def test_append_refusals(libdg):
    def call(ctx=_ctx(), cache=_cache(), k=_heads(), v=_heads(), rope=None):
        return libdg.dg_context_append(_ref(ctx), _ref(cache), _ref(k), _ref(v), _ref(rope), None)
    for kw, code in BAD_CONTEXTS:
        assert call(ctx=_ctx(**kw)) == code, kw
    for kw, code in BAD_CACHES:
        assert call(cache=_cache(**kw)) == code, kw
    for kw in BAD_HEADS:
        assert call(k=_heads(**kw)) == 1 and call(v=_heads(**kw)) == 1, kw
    assert call(ctx=None) == 1 and call(cache=None) == 1 and call(k=None) == 1
    assert call(rope=dg._RopeArgs(20, 0, 1.0, FAKE)) == 1
    big = _cache(pages=1 << 24, heads=4)
    assert call(ctx=_ctx(pages=1 << 24), cache=big) == 2  # the cache's rows pass 31 bits


def test_attention_refusals(libdg):
    def call(ctx=_ctx(), cache=_cache(), q=_heads(), out=_heads(data=2 * FAKE), hq=4, scale=0.0, window=0, most=0,
             lse=None):
        return libdg.dg_context_attention(_ref(ctx), _ref(cache), _ref(q), _ref(out), hq, scale, None, window, most, lse,
                                          FAKE, ctypes.c_size_t(1 << 40), None)
    for kw, code in BAD_CONTEXTS:
        assert call(ctx=_ctx(**kw)) == code, kw
    for kw, code in BAD_CACHES:
        assert call(cache=_cache(**kw)) == code, kw
    for kw in BAD_HEADS:
        assert call(q=_heads(**kw)) == 1 and call(out=_heads(**kw)) == 1, kw
    for hq in (0, 1, 3, 4096):
        assert call(hq=hq) == 2, hq
    assert call(out=_heads()) == 1  # out is q
    for kw in (dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(window=-1), dict(most=-1),
               dict(lse=FAKE + 2)):
        assert call(**kw) == 1, kw
    assert libdg.dg_context_workspace_size(0, 4, 2, 128) == 0
    assert libdg.dg_context_workspace_size(16, 3, 2, 128) == 0
    assert libdg.dg_context_workspace_size(16, 4, 2, 80) == 0


def test_block_driver_refusals(libdg):
    shp = dg._Shape(2, 256, 512, 4096, 0)
    prm = dg.Params().c()
    cb = dg._BLOCK_HIDDEN_FN(lambda *a: 0)
    steps = np.zeros(4, np.int32)
    sp = steps.ctypes.data_as(ctypes.c_void_p)

    def call(ctx, add=FAKE):
        return libdg.dg_generate_blocks_context(ctypes.byref(shp), ctypes.byref(prm), FAKE, None, 1, cb, None,
                                                _ref(ctx), add, FAKE, FAKE, sp, *([FAKE] * 7), FAKE,
                                                ctypes.c_size_t(1 << 30), None)
    assert call(None) == 1
    assert call(_ctx(rows=512), add=None) == 1
    assert call(_ctx(rows=511)) == 2 and call(_ctx(B=1, rows=512)) == 2
    assert call(_ctx(rows=512, table=None)) == 1


def test_error_name(libdg):
    assert libdg.dg_error_string(10) != libdg.dg_error_string(99) and dg.STATUS[10] == "DG_ERR_CAPACITY"
