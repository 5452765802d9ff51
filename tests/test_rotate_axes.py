"""Rotation by positions with several axes (moe_rotate_append_axes): refusals on the CPU; on the GPU pair by
pair against the one-axis call, of which it is the same arithmetic (bit for bit), and against the formula in
64 bits.

Tolerance against 64 bits, as for the one-axis rotation: less than 2^-21 of (|x| + |y|) before the last
rounding (the angle's fraction of a turn once, sincospi, products and sum), then half a step of the type."""
import math
import struct

import pytest
import torch

import sparse_moe_layer_gb300 as moe

KV = struct.Struct("4P9q5i4x")  # moe_kv_cache
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def test_refusals_on_the_host():
    L = moe.lib()
    kv = KV.pack(256, 512, 0, 0, 2048, 1024, 64, 2048, 1024, 64, 32, 16, 1, 0, 4, 16, 2, 64)

    def call(q=256, pos=256, n=3, ld=9, axes=256, slots=256, inv=256, rot=64, N=9, out=256):
        return L.moe_rotate_append_axes(kv, q, 256, 256, 0, 256, 64, 128, 64, 128, 64, pos, n, ld, axes, slots, inv, rot, 0,
                                        1.0, N, 4, out, 256, 64, None, None)

    for name in ("q", "pos", "axes", "slots", "inv", "out"):
        assert call(**{name: None}) == 1, name
    assert call(n=0) == 1 and call(n=17) == 1 and call(ld=8) == 1 and call(ld=-9) == 1 and call(N=0) == 1
    assert call(axes=258) == 2 and call(pos=260) == 2 and call(rot=72) == 1


gpu = pytest.mark.gpu


def inputs(N, Hq, Hkv, D, dtype, cache, page, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(N, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dtype)
    pages = -(-N // page) + 1
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:N]
    if N > 4:
        slots[2] = -1
    pos = torch.randint(0, 1 << 20, (4, N), generator=g, device="cuda")
    if cache == "e4m3":
        kv = [torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        sc = [torch.zeros(pages, Hkv, page, device="cuda") for _ in range(2)]
    else:
        kv, sc = [torch.zeros(pages, Hkv, page, D, dtype=dtype, device="cuda") for _ in range(2)], [None, None]
    return (qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]), slots, pos, kv, sc


def freq(rot):
    return 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))


def axes_of(rot, A, kind, seed=0):
    n = rot // 2
    if kind == "sections":
        return (torch.arange(n) * A // max(n, 1)).int().cuda()
    if kind == "turns":
        return (torch.arange(n) % A).int().cuda()
    return torch.randint(0, A, (n,), generator=torch.Generator().manual_seed(seed)).int().cuda()


@gpu
@pytest.mark.parametrize("N,Hq,Hkv,D,rot,page", [(1, 8, 2, 64, 64, 16), (5, 3, 3, 80, 16, 7), (777, 20, 4, 96, 48, 24),
                                                 (2100, 16, 2, 128, 128, 64), (33, 4, 1, 256, 256, 8), (9, 4, 2, 64, 0, 16)])
@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, "16"), (torch.float16, "16"), (torch.bfloat16, "e4m3")])
@pytest.mark.parametrize("A,kind,interleaved", [(3, "sections", False), (2, "turns", True), (4, "any", False), (1, "any", True)])
def test_each_pair_turns_as_by_its_own_axis(N, Hq, Hkv, D, rot, page, dtype, cache, A, kind, interleaved):
    qkv, slots, pos, kv, sc = inputs(N, Hq, Hkv, D, dtype, cache, page, seed=N + A)
    pos, axes, f = pos[:A], axes_of(rot, A, kind), freq(rot)
    status = moe.new_status()
    got = moe.rotate_append(*qkv, pos, slots, *kv, f, *sc, interleaved=interleaved, rope_scale=1.25, axes=axes, status=status)
    assert moe.read_device_status(status) == 0
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for a in range(A):
        # by one axis alone, into a 16-bit cache
        k16 = [torch.zeros(x.shape, dtype=dtype, device="cuda") for x in kv]
        q = moe.rotate_append(*qkv, pos[a].contiguous(), slots, *k16, f, interleaved=interleaved, rope_scale=1.25)
        mine = (axes == a).nonzero()[:, 0]
        for part in (first, second):
            assert torch.equal(got[..., part][..., mine], q[..., part][..., mine])
            if cache == "16":
                assert torch.equal(kv[0][..., part][..., mine], k16[0][..., part][..., mine])
        assert torch.equal(got[..., rot:], q[..., rot:])
        if cache == "16":
            assert torch.equal(kv[1], k16[1])
    # against 64 bits
    phase = (pos.double()[axes.long()].t() * f)[:, None]
    x, y = qkv[0][..., first].double(), qkv[0][..., second].double()
    for part, want in ((first, x * phase.cos() - y * phase.sin()), (second, x * phase.sin() + y * phase.cos())):
        want = want * 1.25
        tol = (x.abs() + y.abs()) * 1.25 * 2.0 ** -21 + want.abs() * HALF[dtype] + (2.0 ** -25 if dtype == torch.float16 else 0)
        assert torch.all((got[..., part].double() - want).abs() <= tol)
    if cache == "e4m3":
        x, y = qkv[1][..., first].double(), qkv[1][..., second].double()
        want = qkv[1].double().clone()
        want[..., first] = (x * phase.cos() - y * phase.sin()) * 1.25
        want[..., second] = (x * phase.sin() + y * phase.cos()) * 1.25
        live = slots >= 0
        pg, off = slots[live] // page, slots[live] % page
        s = sc[0][pg, :, off].double()
        top = want[live].abs().amax(-1)
        assert torch.all((s - top / 448).abs() <= top / 448 * (2.0 ** -24 + 2.0 ** -20 * math.sqrt(2)))
        # half a step of e4m3, of the value or of the smallest, and the fp32 error of the value
        value = kv[0][pg, :, off].view(torch.float8_e4m3fn).double() * s[..., None]
        assert torch.all((value - want[live]).abs() <= want[live].abs() * (2.0 ** -4 * 1.001) + s[..., None] * (2.0 ** -10 * 1.001)
                         + top[..., None] * 2.0 ** -20)


@gpu
def test_bad_axes_count_as_the_first_and_are_reported():
    qkv, slots, pos, kv, sc = inputs(6, 4, 2, 64, torch.bfloat16, "16", 16, 3)
    axes = axes_of(64, 3, "turns")
    bad = axes.clone()
    bad[3], bad[7] = -1, 3  # 3 is axis 0 already, 7 was axis 1
    axes[7] = 0
    status = moe.new_status()
    want = moe.rotate_append(*qkv, pos[:3], slots, *[x.clone() for x in kv], freq(64), axes=axes)
    got = moe.rotate_append(*qkv, pos[:3], slots, *kv, freq(64), axes=bad, status=status)
    assert torch.equal(got, want) and moe.read_device_status(status) == 6


@gpu
def test_strided_positions_in_place_and_refusals():
    qkv, slots, pos, kv, sc = inputs(6, 4, 2, 64, torch.bfloat16, "16", 16, 3)
    axes = axes_of(64, 3, "sections")
    wide = torch.zeros(3, 50, dtype=torch.long, device="cuda")
    wide[:, :6] = pos[:3]
    want = moe.rotate_append(*qkv, pos[:3], slots, *kv, freq(64), axes=axes)
    q = qkv[0].clone()
    got = moe.rotate_append(q, *qkv[1:], wide[:, :6], slots, *kv, freq(64), axes=axes, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    for bad in (dict(positions=pos[0]), dict(positions=pos[:3, :5]), dict(positions=pos[:3].int()), dict(axes=axes[:31]),
                dict(axes=axes.long()), dict(positions=pos[:3].t().contiguous().t()), dict(axes=axes.cpu()),
                dict(positions=pos[:0])):
        kw = dict(positions=pos[:3], axes=axes) | bad
        with pytest.raises(ValueError):
            moe.rotate_append(*qkv, kw.pop("positions"), slots, *kv, freq(64), **kw)
