"""The place for held codes on the host: its size and the refusals."""
import ctypes

import pytest

import block_canvas_denoising_b200 as dg
from block_canvas_denoising_b200 import build as dg_build

FAKE = 4096  # an aligned address that no refused call dereferences


@pytest.fixture(scope="module")
def libdg():
    dg_build.build()
    return dg.lib()


def test_kept_size(libdg):
    # a word beside each scale; a page's codes of each head, keys and values, and a tag for each, of at most 256 pages
    for pages, heads, dim, slots in ((1, 1, 64, 1), (40, 3, 128, 40), (256, 8, 128, 256), (70000, 8, 128, 256), (1 << 24, 1024, 64, 256)):
        n = libdg.dg_context_kept_size(pages, heads, dim)
        assert 0 <= n - pages * 2 * heads * 4 - slots * 2 * heads * (64 * dim + 28) < 512
    for bad in ((0, 1, 64), (1, 0, 64), (1, 1025, 64), (1, 1, 96), ((1 << 24) + 1, 1, 64)):
        assert libdg.dg_context_kept_size(*bad) == 0


def test_kept_refusals(libdg):
    def call(epoch=FAKE, kept=FAKE):
        c = dg._Context(2, 256, 8, 4, *([FAKE] * 11), epoch)
        cache = dg._Cache(8, 2, 128, FAKE, FAKE, FAKE, FAKE, kept)
        h = dg._Heads(None, 512, 128)  # refused in any case: nothing is launched
        return (libdg.dg_context_plan(ctypes.byref(c), None if epoch == FAKE else FAKE, None, 0, None),
                libdg.dg_context_append(ctypes.byref(c), ctypes.byref(cache), ctypes.byref(h), ctypes.byref(h), None, None))
    assert call() == (1, 1)
    assert call(epoch=FAKE + 2) == (1, 1)
    for kept in (FAKE + 8, FAKE + 1):
        c, cache = dg._Context(2, 256, 8, 4, *([FAKE] * 11), FAKE), dg._Cache(8, 2, 128, FAKE, FAKE, FAKE, FAKE, kept)
        h = dg._Heads(FAKE, 512, 128)
        assert libdg.dg_context_append(ctypes.byref(c), ctypes.byref(cache), ctypes.byref(h), ctypes.byref(h), None, None) == 1
