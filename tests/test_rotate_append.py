"""Rotation and paged append (moe_rotate_append): refusals on the CPU, then on
the GPU against the formula in 64 bits, value by value, with every slot that
no token names checked to be untouched.

Tolerance of a rotated value before its last rounding: the angle's fraction of
a turn is rounded once (2^-25 of a turn = 2^-22.3 rad), sincospi is within two
steps (2^-22.5), the scale, two products and the sum round once each (2^-24):
less than 2^-21 of (|x| + |y|) * scale.  The last rounding adds half a step:
2^-8 (bf16) or 2^-11 (fp16) of the value, or half the
type's smallest step (2^-134, 2^-25).
e4m3: 2^-4 of the value, or half its smallest step (2^-10 of a scale); a scale is
rounded to 2^-24 of itself, or half the smallest fp32 step (2^-150)."""
import ctypes
import math
import struct

import pytest
import torch

import sparse_moe_layer_gb300 as moe

KV = struct.Struct("4P9q5i4x")  # moe_kv_cache
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def inv_freq(rot):
    return 150000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))


# ------------------------------------------------------------- on the CPU ----
def kv_bytes(dt=0, P=4, S=16, H=2, D=64, k=256, v=512, ks=0, vs=0, strides=None, sstr=(32, 16, 1)):
    st = strides or (H * S * D, S * D, D)
    return KV.pack(k, v, ks, vs, *st, *st, *sstr, dt, P, S, H, D)


def test_refusals_on_the_host():
    L = moe.lib()

    def call(kv=None, q=256, k=256, v=256, dt=0, st=None, pos=256, slots=256, inv=256, rot=64, N=3, Hq=4, out=256,
             ost=(256, 64), status=None, **cache):
        return L.moe_rotate_append(kv_bytes(**cache) if kv is None else kv, q, k, v, dt,
                                   *(st or (256, 64, 128, 64, 128, 64)), pos, slots, inv, rot, 0, 1.0, N, Hq, out, *ost,
                                   status, None)

    assert L.moe_rotate_append(None, *[256] * 3, 0, 256, 64, 128, 64, 128, 64, 256, 256, 256, 64, 0, 1.0, 3, 4, 256, 256,
                               64, None, None) == 1
    for name in ("q", "k", "v", "pos", "slots", "inv", "out"):
        assert call(**{name: None}) == 1, name
    assert call(kv=kv_bytes(k=0)) == 1 and call(N=0) == 1 and call(Hq=0) == 1 and call(Hq=5000) == 1
    assert call(D=72) == 1 and call(D=0) == 1 and call(D=272) == 1 and call(S=0) == 1 and call(P=0) == 1 and call(H=0) == 1
    assert call(P=1 << 20, S=1 << 11) == 1  # 2^31 slots
    assert call(rot=72) == 1 and call(rot=80) == 1 and call(rot=-16) == 1
    assert call(dt=2) == 2 and call(dt=3) == 2  # fp32, e4m3 inputs
    assert call(kv=kv_bytes(dt=1)) == 2 and call(kv=kv_bytes(dt=2)) == 2 and call(kv=kv_bytes(dt=9)) == 2
    assert call(kv=kv_bytes(dt=3)) == 1  # no scales
    assert call(kv=kv_bytes(dt=3, ks=18, vs=16)) == 2
    assert call(q=264) == 2 and call(out=264) == 2 and call(kv=kv_bytes(k=264)) == 2
    assert call(st=(252, 64, 128, 64, 128, 64)) == 2 and call(st=(256, 64, 128, 64, 128, 65)) == 2
    assert call(st=(256, -64, 128, 64, 128, 64)) == 1
    assert call(kv=kv_bytes(strides=(2048, 1024, 68))) == 2
    assert call(kv=kv_bytes(dt=3, ks=256, vs=256, strides=(2048, 1024, 72))) == 2
    assert call(pos=260) == 2 and call(slots=260) == 2 and call(inv=260) == 2 and call(status=258) == 2


def test_binding_refuses():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="must be CUDA tensors"):
        moe.rotate_append(q, q[:, :2], q[:, :2], i, i, kv, kv, inv_freq(64))


# ------------------------------------------------------------- on the GPU ----
gpu = pytest.mark.gpu


def new_cache(pages, heads, page, D, dtype, nhd, seed=0):
    """Filled k and v caches (and scales); nhd: tokens-major in memory."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (pages, page, heads) if nhd else (pages, heads, page)
    if dtype == "e4m3":
        kv = [torch.randint(0, 120, (*shape, D), dtype=torch.uint8, device="cuda", generator=g) for _ in range(2)]
        sc = [torch.rand(shape, device="cuda", generator=g) for _ in range(2)]
    else:
        kv = [torch.randn((*shape, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2)]
        sc = [None, None]
    t = (lambda x: None if x is None else x.transpose(1, 2)) if nhd else (lambda x: x)
    return t(kv[0]), t(kv[1]), t(sc[0]), t(sc[1])


def rotated(x, positions, inv, rot, interleaved, scale):
    """x in 64 bits -> (rotated, |x| + |y| of each dim's pair; 0 where not rotated)."""
    x = x.double().clone()
    mag = torch.zeros_like(x)
    ang = positions.double()[:, None, None] * inv
    c, s = ang.cos() * scale, ang.sin() * scale
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    xa, xb = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = xa * c - xb * s, xa * s + xb * c
    mag[..., a] = mag[..., b] = (xa.abs() + xb.abs()) * scale
    return x, mag


def within(diff, tol):
    worst = float((diff.abs() / tol).nan_to_num(nan=0.0, posinf=math.inf).max()) if diff.numel() else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the tolerance"


def check(N, Hq, Hkv, D, rot, page, dtype, cache, interleaved=False, nhd=False, scale=1.0, first=0, drop=(), fused=True,
          values=None, in_place=False, extra_pages=2):
    g = torch.Generator(device="cuda").manual_seed(N + D)
    qkv = torch.randn((N, Hq + 2 * Hkv, D), device="cuda", generator=g)
    if values is not None:
        values(qkv)
    qkv = qkv.to(DT[dtype])
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.transpose(0, 1).contiguous().transpose(0, 1), v.contiguous()
    pages = -(-N // page) + extra_pages
    perm = torch.randperm(pages * page, generator=torch.Generator().manual_seed(N))[:N].cuda()
    slots = perm.clone()
    for d in drop:
        slots[d] = -1 - d
    positions = (first + torch.arange(N, device="cuda") * 977 % 50000).long()
    inv = inv_freq(rot).cuda()
    kc, vc, ks, vs = new_cache(pages, Hkv, page, D, cache, nhd)
    before = [None if t is None else t.clone() for t in (kc, vc, ks, vs)]
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    status = moe.new_status()
    out = moe.rotate_append(q, k, v, positions, slots, kc, vc, inv, k_scale=ks, v_scale=vs, interleaved=interleaved,
                            rope_scale=scale, q_out=q if in_place else None, status=status)
    assert moe.read_device_status(status) == 0
    scale32 = float(torch.tensor(scale, dtype=torch.float32))
    tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
    want, mag = rotated(q0, positions, inv, rot, interleaved, scale32)
    within(out.double() - want, mag * 2.0 ** -21 + (want.abs() + mag * 2.0 ** -21) * HALF[dtype] + tiny)
    assert torch.equal(k, k0) and torch.equal(v, v0) and (in_place or torch.equal(q, q0))
    live = slots >= 0
    pg, off = slots[live] // page, slots[live] % page
    named = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    named[pg, off] = True
    for t, b in zip((kc, vc, ks, vs), before):
        if t is not None:
            t, b = t.transpose(1, 2)[~named], b.transpose(1, 2)[~named]  # [slots, heads, ...]
            assert torch.equal(t, b)
    for x, c, sc, turn in ((k0, kc, ks, True), (v0, vc, vs, False)):
        if turn:
            want, mag = rotated(x, positions, inv, rot, interleaved, scale32)
        else:
            want, mag = x.double(), torch.zeros_like(x, dtype=torch.float64)
        want, mag = want[live], mag[live]
        got = c[pg, :, off]
        if cache != "e4m3":
            got = got.double()
            within(got - want, mag * 2.0 ** -21 + (want.abs() + mag * 2.0 ** -21) * HALF[dtype] + tiny)
            if not turn:
                assert torch.equal(got, want)
            continue
        s = sc[pg, :, off].double()
        amax, slack = want.abs().amax(-1), mag.amax(-1) * 2.0 ** -21
        ref = torch.where(amax == 0, 1.0, amax / 448.0)
        within(s - ref, slack / 448.0 + ref * 2.0 ** -24 + 2.0 ** -150)
        val = got.view(torch.float8_e4m3fn).double() * s[..., None]
        tol = (want.abs() + slack[..., None]) * 2.0 ** -4 + s[..., None] * 2.0 ** -10 + 2 * slack[..., None] + 448 * 2.0 ** -150
        within(val - want, tol)
        if not turn and D <= 128:  # unrotated heads: the layer's group quantiser, bit for bit
            rows = want.float().reshape(-1, D).contiguous()
            q8, sx = moe.quantize_rows(rows)
            assert torch.equal(q8[:, :D], got.reshape(-1, D)) and torch.equal(sx[:, 0], sc[pg, :, off].reshape(-1))


@gpu
@pytest.mark.parametrize("D,rot", [(64, 64), (16, 16), (64, 32), (80, 16), (96, 48), (128, 128), (128, 0), (256, 256),
                                   (256, 64), (240, 240)])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dims_types_and_pairs(D, rot, cache, dtype):
    for interleaved in (False, True):
        check(33, 6, 2, D, rot, 16, dtype, dtype if cache == "same" else cache, interleaved=interleaved, scale=1.25,
              drop=(0, 7, 32))


@gpu
@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("nhd", [False, True])
def test_pages_orders_and_counts(page, nhd):
    for N in (1, 2, 5, 130):
        for cache in ("bf16", "e4m3"):
            check(N, 8, 2, 64, 64, page, "bf16", cache, nhd=nhd, drop=(1,) if N > 2 else (), fused=N % 2 == 0)


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (64, 8), (64, 4), (20, 4), (128, 128), (300, 1)])
def test_heads(Hq, Hkv):
    check(9, Hq, Hkv, 64, 64, 16, "bf16", "bf16")
    check(9, Hq, Hkv, 128, 64, 16, "fp16", "e4m3", interleaved=True)


@gpu
def test_large_batches_take_several_tokens_per_block():
    for N in (304, 1000, 5000):
        check(N, 2, 1, 16, 16, 16, "bf16", "bf16", drop=(N - 1,))
        check(N, 4, 1, 64, 64, 16, "fp16", "e4m3", drop=(0, N - 1))


@gpu
def test_far_positions():
    check(65, 4, 2, 64, 64, 16, "fp16", "fp16", first=2_000_000)
    check(65, 4, 2, 128, 128, 16, "fp16", "e4m3", first=10 ** 9, scale=1.3465735902799727)


@gpu
def test_in_place_q():
    check(40, 8, 2, 64, 64, 16, "bf16", "bf16", in_place=True)
    check(40, 8, 2, 96, 48, 16, "fp16", "e4m3", in_place=True, interleaved=True)


@gpu
def test_zero_tiny_and_large_heads_in_e4m3():
    def values(x):
        x[0] = 0.0
        x[1] *= 1e-30
        x[2] *= 1e30
        x[3, :, 1:] = 0.0
        x[4] *= 1e-38

    check(8, 4, 2, 64, 64, 16, "bf16", "e4m3", values=values)
    check(8, 4, 2, 64, 0, 16, "bf16", "e4m3", values=values)


@gpu
def test_slot_past_the_cache_is_refused_on_the_device():
    kc, vc, _, _ = new_cache(3, 2, 16, 64, "bf16", False)
    k0, v0 = kc.clone(), vc.clone()
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    pos = torch.tensor([3, 4], device="cuda")
    status = moe.new_status()
    for bad in (48, 49, 2 ** 31, 2 ** 40):
        slots = torch.tensor([bad, -1], device="cuda")
        out = moe.rotate_append(q, q[:, :2], q[:, 2:], pos, slots, kc, vc, inv_freq(64).cuda(), status=status)
        assert moe.read_device_status(status) == 6 and moe.read_device_status(status) == 0
        assert torch.equal(kc, k0) and torch.equal(vc, v0)
        moe.rotate_append(q, q[:, :2], q[:, 2:], pos, slots, kc, vc, inv_freq(64).cuda())
        torch.cuda.synchronize()
        assert torch.equal(kc, k0) and torch.all(torch.isfinite(out))
    moe.rotate_append(q, q[:, :2], q[:, 2:], pos, torch.tensor([47, -1], device="cuda"), kc, vc, inv_freq(64).cuda(),
                      status=status)
    assert moe.read_device_status(status) == 0
    assert not torch.equal(kc, k0)


@gpu
def test_offsets_beyond_32_bits():
    pages, H, S, D = 40000, 8, 64, 128
    kc = torch.zeros(pages, H, S, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 31
    ks = torch.zeros(pages, H, S, device="cuda")
    vs = torch.zeros_like(ks)
    qkv = torch.randn(3, 16 + 2 * H, D, device="cuda").bfloat16()
    slots = torch.tensor([pages * S - 1, (2 ** 31) // (H * D) + 5, 0], device="cuda")
    pos = torch.arange(3, device="cuda")
    moe.rotate_append(qkv[:, :16], qkv[:, 16:24], qkv[:, 24:], pos, slots, kc, vc, inv_freq(0).cuda(), k_scale=ks,
                      v_scale=vs)
    for x, c, s in ((qkv[:, 16:24], kc, ks), (qkv[:, 24:], vc, vs)):
        q8, sx = moe.quantize_rows(x.float().reshape(-1, D).contiguous())
        assert torch.equal(c[slots // S, :, slots % S].reshape(-1, D), q8)
        assert torch.equal(s[slots // S, :, slots % S].reshape(-1), sx[:, 0])
        assert int((s != 0).sum()) == 3 * H
    del kc, vc, ks, vs
    torch.cuda.empty_cache()


@gpu
def test_graph_replay_and_another_stream():
    kc, vc, _, _ = new_cache(5, 2, 16, 64, "bf16", False)
    qkv = torch.randn(4, 8, 64, device="cuda").bfloat16()
    pos, slots = torch.arange(4, device="cuda"), torch.tensor([3, 70, 21, -1], device="cuda")
    inv = inv_freq(64).cuda()

    def run(kc, vc):
        return moe.rotate_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, slots, kc, vc, inv)

    k2, v2 = kc.clone(), vc.clone()
    run(k2, v2)  # before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(kc, vc)
    qkv.copy_(torch.randn(4, 8, 64, device="cuda"))
    pos.add_(1000)
    slots.copy_(torch.tensor([9, 71, -1, 33], device="cuda"))
    g.replay()
    want = run(k2, v2)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run(kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(again, want)
    live = slots[slots >= 0]
    assert torch.equal(kc[live // 16, :, live % 16], k2[live // 16, :, live % 16])


@gpu
def test_empty_batch_and_shape_refusals():
    kc, vc, _, _ = new_cache(2, 2, 16, 64, "bf16", False)
    z = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert moe.rotate_append(z, z[:, :2], z[:, :2], i, i, kc, vc, inv_freq(64).cuda()).shape == (0, 4, 64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    j = torch.zeros(2, dtype=torch.int64, device="cuda")
    ok = (q, q[:, :2], q[:, 2:], j, j, kc, vc, inv_freq(64).cuda())

    def refuse(match, **swap):
        args = list(ok)
        for at, x in swap.items():
            args[int(at[1:])] = x
        with pytest.raises((ValueError, moe.MoeError), match=match):
            moe.rotate_append(*args)

    refuse("alike", a0=q.float())
    refuse("alike", a1=q[:, :2].half())
    refuse("must be", a1=q)
    refuse("contiguous", a0=q.transpose(1, 2).contiguous().transpose(1, 2))
    refuse("positions", a3=j.int())
    refuse("slots", a4=j[:1])
    refuse("fp64", a7=inv_freq(64).float().cuda())
    refuse("status 1", a7=inv_freq(128).cuda())
    refuse("both be", a6=vc[:, :1])
    refuse("needs k_scale", a5=kc.view(torch.uint8)[..., :64], a6=vc.view(torch.uint8)[..., :64])
    refuse("status 2", a0=torch.zeros(2 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 512].view(2, 4, 64))
