"""compact_drafts writes a sequence's new length while warps of others, and of its other heads, still read lengths,
starts, kept and page_table: an `out` that shares memory with one of them is refused, on the host."""
import ctypes
import struct

import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_cache_pages import Drafts, caches, clones, equal, move

KV = struct.Struct("4P9q5i4x")  # moe_kv_cache


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def test_shared_memory_is_refused():
    st = (2 * 16 * 64, 16 * 64, 64)
    kv = KV.pack(256, 512, 0, 0, *st, *st, 32, 16, 1, 0, 4, 16, 2, 64)
    ls = ctypes.cast((ctypes.c_int64 * 3)(8192, 8192, 128), ctypes.c_void_p)

    def call(out, B=3, ld=9, kld=10):
        return moe.lib().moe_compact_drafts(kv, 2, ls, 4096, ld, 4, 1024, 2048, 8192, kld, B, 5, out, None, None)

    for start, n in ((1024, 3), (2048, 4)):
        for at in range(-2, n):
            assert call(start + 4 * at) == 1, (start, at)
    for start, width, ld in ((4096, 4, 9), (8192, 5, 10)):  # rows, and the gaps between them where [B] does not fit
        for at in range(-2, 2 * ld + width):
            free = at % ld >= width and at % ld + 3 <= ld and at < 2 * ld
            assert free or call(start + 4 * at) == 1, (start, at)
    for B in (1,):
        assert call(1024, B) == 1 and call(2048, B) == 1 and call(2052, B) == 1 and call(8192 + 16, B) == 1
    assert call(1026) == 2


@pytest.mark.gpu
def test_an_out_between_rows_is_used():
    d = Drafts([5, 6], [8, 8], [[1, 3, 4], [0, 2]], page=4)
    c = caches(2, d.pages, 2, 4, 64, "bf16")
    room = torch.full((2, 9), 77, dtype=torch.int32, device="cuda")
    room[:, :3] = d.kept_t
    want, got = clones(c), clones(c)
    move(want, d.moves())
    out = room[0, 4:6]
    assert d.run(got, kept=room[:, :3], out=out).data_ptr() == out.data_ptr()
    equal(got, want)
    assert out.tolist() == d.lengths_after() and room[0, 6:].tolist() == [77] * 3 and room[1, :3].tolist() == d.kept_t[1].tolist()
    for out in (room[0, 2:4], room[0, 8:].new_empty(0), d.starts[1:]):
        with pytest.raises((ValueError, moe.MoeError)):
            d.run(got, kept=room[:, :3], out=out)
    one = Drafts([5], [8], [[1]], page=4)
    c = caches(2, one.pages, 2, 4, 64, "bf16")
    with pytest.raises(moe.MoeError):
        one.run(c, out=one.kept_t.view(1))
