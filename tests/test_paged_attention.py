"""Paged attention of one new token (moe_paged_attention): refusals on the CPU,
then on the GPU against the formula in 64 bits over lengths from none to
thousands, odd sizes, every head grouping, cut and uncut rows, sinks, windows,
garbage in unused places, and bad pages and lengths.

Tolerance of out_d, from what is rounded (h: half a step of a 16-bit type, 2^-8
bf16, 2^-11 fp16; A = sum_t p_t |v_td| with p summing to at most 1):
  scores      fp32 sums of D products, each step at most 2^-23 of scale sum|q k|:
              a factor exp(+-e) on every p_t, e = (D + 8) 2^-23 scale max_t sum|q k_t|,
              twice (numerator and sum)                                  2 e A
  weights     ex2 2^-22, rescaling and the sums over L tokens, 2^-22 each    (L + 64) 2^-22 A
  p to 16 bit h of the product's type (bf16 for a bf16 cache, else fp16)  h A
              fp16 below its normals: half its smallest step, 2^-25, of the largest p,
              times sum_t |v| (e4m3: of the largest value scale)        2^-25 L max|v|
  out         half a step                                                 h |out|"""
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


# ------------------------------------------------------------- on the CPU ----
def kv_bytes(dt=0, P=4, S=16, H=2, D=64, k=256, v=512, ks=0, vs=0, strides=None):
    st = strides or (H * S * D, S * D, D)
    return KV.pack(k, v, ks, vs, *st, *st, H * S, S, 1, dt, P, S, H, D)


def test_refusals_on_the_host():
    L = moe.lib()

    def call(kv=None, q=256, dt=0, qst=(256, 64), table=256, ld=4, width=4, lens=256, B=3, Hq=4, scale=0.125, sinks=None,
             window=0, out=256, ost=(256, 64), ws=256, wsb=1 << 40, status=None, **cache):
        return L.moe_paged_attention(kv_bytes(**cache) if kv is None else kv, q, dt, *qst, table, ld, width, lens, B, Hq,
                                     scale, sinks, window, out, *ost, ws, wsb, status, None)

    for name in ("q", "table", "lens", "out"):
        assert call(**{name: None}) == 1, name
    assert call(width=100, ld=100, ws=None) == 1  # rows that may be cut need a workspace
    assert call(kv=kv_bytes(k=0)) == 1 and call(B=0) == 1 and call(B=65537) == 1 and call(Hq=0) == 1
    assert call(Hq=3) == 1 and call(Hq=4098) == 1  # not a multiple of the key heads; too many
    assert call(D=72) == 1 and call(D=272) == 1 and call(S=0) == 1 and call(H=300) == 1
    assert call(width=0) == 1 and call(ld=3) == 1 and call(width=1 << 28, ld=1 << 28) == 1
    assert call(window=-1) == 1 and call(scale=math.nan) == 1
    assert call(dt=2) == 2 and call(dt=1) == 2 and call(kv=kv_bytes(dt=2)) == 2
    assert call(kv=kv_bytes(dt=3)) == 1
    assert call(q=258) == 2 and call(out=258) == 2 and call(table=258) == 2 and call(lens=258) == 2
    assert call(sinks=258) == 2 and call(status=258) == 2 and call(ws=264) == 2
    assert call(qst=(256, 65)) == 2 and call(ost=(255, 64)) == 2 and call(qst=(-256, 64)) == 1
    assert call(kv=kv_bytes(k=264)) == 2 and call(kv=kv_bytes(strides=(2048, 1024, 68))) == 2
    assert call(width=100, ld=100, wsb=64) == 3
    size = L.moe_attention_workspace_size
    assert size(0, 4, 2, 64, 0, 99) == 0 and size(1, 3, 2, 64, 0, 99) == 0 and size(1, 4, 2, 72, 0, 99) == 0
    assert size(1, 4, 2, 64, 2, 99) == 0 and size(1, 4, 2, 64, 0, 0) == 0
    assert size(1, 4, 2, 64, 0, 99) == 256 and size(1, 4, 2, 64, 3, 99999) > 256


def test_lengths_past_31_bits_are_refused():
    """Token numbers are rounded up to a tile of 32, and a batch's tiles are counted in 32 bits."""
    L = moe.lib()

    def call(B, width, page=16, window=0, ws=None):
        return L.moe_paged_attention(kv_bytes(S=page), 256, 0, 256, 64, 256, width, width, 256, B, 4, 0.125, None, window,
                                     256, 256, 64, ws, 0, None, None)

    assert call(1, (1 << 27) - 1) == 1 and call(1, (1 << 31) - 17, page=1) == 1
    assert call(1, (1 << 27) - 2, ws=256) == 3  # passes, for the workspace to be found too small
    assert call(65536, 1 << 16, ws=256) == 1 and call(65536, 1 << 14, ws=256) == 3


def test_binding_refuses():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be CUDA tensors"):
        moe.paged_attention(q, kv, kv, i[:, None], i, 0.125)


# ------------------------------------------------------------- on the GPU ----
gpu = pytest.mark.gpu


class Case:
    """Sequences in a paged cache whose unused places hold NaN, and page table entries past the
    lengths -1."""

    def __init__(self, lengths, Hq, Hkv, D, page=16, dtype="bf16", cache=None, nhd=False, seed=0, spread=2.0, wide=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        h = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        self.dtype, self.cache, self.Hq, self.Hkv, self.D, self.page = dtype, cache, Hq, Hkv, D, page
        B = len(lengths)
        self.lengths = lengths
        counts = [-(-n // page) for n in lengths]
        pages = sum(counts) + 2
        order = torch.randperm(pages, generator=h).tolist()
        width = max(1, max(counts, default=1)) + wide
        table = torch.full((B, width), -1, dtype=torch.int32)
        used = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(lengths):
            for j in range(counts[b]):
                table[b, j] = order[at]
                used[order[at], :max(0, min(page, n - j * page))] = True
                at += 1
        self.table, self.lens = table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda")
        used = used.cuda()
        shape = (pages, page, Hkv) if nhd else (pages, Hkv, page)
        turn = (lambda x: x.transpose(1, 2)) if nhd else (lambda x: x)
        self.kv, self.sc = [], []
        for _ in range(2):
            x = turn(torch.randn((*shape, D), generator=g, device="cuda"))
            if cache == "e4m3":
                x = x * torch.exp(turn(torch.randn(shape, generator=g, device="cuda")))[..., None]
                s = x.abs().amax(-1) / 448.0
                q = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
                q[~used[:, None].expand(s.shape)] = 0x7F
                s = s.masked_fill(~used[:, None], math.nan)
                self.kv.append(turn(turn(q).contiguous()))
                self.sc.append(turn(turn(s).contiguous()))
            else:
                x = x.to(DT[cache]).masked_fill(~used[:, None, :, None], math.nan)
                self.kv.append(turn(turn(x).contiguous()))
                self.sc.append(None)
        self.q = (spread * torch.randn(B, Hq, D, generator=g, device="cuda")).to(DT[dtype])
        self.sinks = torch.randn(Hq, generator=g, device="cuda")

    def run(self, sinks=False, window=0, scale=None, **kw):
        return moe.paged_attention(kw.pop("q", self.q), *self.kv, self.table, kw.pop("lens", self.lens),
                                   self.D ** -0.5 if scale is None else scale, k_scale=self.sc[0], v_scale=self.sc[1],
                                   sinks=self.sinks if sinks else None, window=window, **kw)

    def values(self, i, b, lo, hi):
        """Keys (0) or values (1) of tokens [lo, hi) of sequence b in 64 bits: [Hkv, tokens, D]."""
        t = torch.arange(lo, hi, device="cuda")
        pg, off = self.table[b].long()[t // self.page], t % self.page
        x = self.kv[i][pg, :, off]
        if self.cache == "e4m3":
            x = x.view(torch.float8_e4m3fn).double() * self.sc[i][pg, :, off].double()[..., None]
        return x.double().transpose(0, 1)

    def check(self, out, sinks=False, window=0, scale=None, q=None):
        q = self.q if q is None else q
        scale = self.D ** -0.5 if scale is None else scale
        G = self.Hq // self.Hkv
        hp, ho = HALF["bf16" if self.cache == "bf16" else "fp16"], HALF[self.dtype]
        worst = 0.0
        assert out.shape == q.shape and out.dtype == q.dtype
        for b, n in enumerate(self.lengths):
            lo = max(0, n - window) if window else 0
            if n == 0:
                assert torch.all(out[b] == 0)
                continue
            k, v = self.values(0, b, lo, n), self.values(1, b, lo, n)
            qb = q[b].double().view(self.Hkv, G, self.D)
            s = (qb @ k.transpose(1, 2)) * scale
            e = (self.D + 8) * 2.0 ** -23 * abs(scale) * (qb.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True)
            if sinks:
                s = torch.cat((s, self.sinks.double().view(self.Hkv, G, 1)), -1)
            p = torch.softmax(s, -1)[..., :n - lo]
            want, A = p @ v, p @ v.abs()
            L = n - lo
            tol = A * (2 * e + (L + 64) * 2.0 ** -22 + hp) + 2.0 ** -25 * (1 + L * v.abs().amax()) + want.abs() * ho
            got = out[b].double().view(self.Hkv, G, self.D)
            assert torch.all(torch.isfinite(got)), b
            worst = max(worst, float(((got - want).abs() / tol).max()))
        assert worst <= 1.0, f"{worst:.3f} of the tolerance"
        return worst

    def both(self, **kw):
        self.check(self.run(**kw), **kw)


CACHES = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")]


@gpu
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 128, 144, 192, 256])
@pytest.mark.parametrize("dtype,cache", CACHES)
def test_dims_and_types(D, dtype, cache):
    Case([0, 1, 2, 15, 16, 17, 31, 33, 100], 8, 2, D, dtype=dtype, cache=cache, seed=D).both(sinks=True)
    Case([0, 700, 1, 129, 0], 8, 2, D, dtype=dtype, cache=cache, seed=D + 1).both()


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (7, 1), (16, 2), (16, 1), (17, 1), (40, 2), (64, 8), (64, 4),
                                    (128, 1)])
def test_head_groups(Hq, Hkv):
    for dtype, cache in CACHES[:3]:
        Case([5, 64, 130, 400], Hq, Hkv, 64, dtype=dtype, cache=cache, seed=Hq).both(sinks=True)
        Case([90, 1], Hq, Hkv, 128, dtype=dtype, cache=cache, seed=Hq).both()


@gpu
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 256])
@pytest.mark.parametrize("nhd", [False, True])
def test_page_sizes_and_orders(page, nhd):
    for dtype, cache in CACHES[:3]:
        for D in (64, 128):
            c = Case([1, 47, 300, 0, 1025], 8, 2, D, page=page, dtype=dtype, cache=cache, nhd=nhd, seed=page)
            c.both(sinks=True)
            c.both(window=100)


@gpu
@pytest.mark.parametrize("dtype,cache", CACHES[:3])
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 128, 129, 1000, 5000])
def test_windows(window, dtype, cache):
    c = Case([0, 1, 16, 99, 100, 101, 128, 400, 1500, 3001], 8, 1, 64, dtype=dtype, cache=cache, seed=window)
    c.both(window=window, sinks=True)
    c.both(window=window)


@gpu
@pytest.mark.parametrize("dtype,cache", CACHES[:3])
def test_one_long_sequence_is_cut_and_joined(dtype, cache):
    for n, Hq, Hkv in ((4097, 8, 1), (20000, 16, 8), (65536 + 13, 4, 4)):
        Case([n], Hq, Hkv, 64, dtype=dtype, cache=cache, seed=n % 97).both(sinks=True)
    Case([30011], 16, 1, 128, page=64, dtype=dtype, cache=cache).both()
    Case([5000], 4, 2, 256, page=64, dtype=dtype, cache=cache).both()


@gpu
@pytest.mark.parametrize("dtype,cache", CACHES[:3])
def test_ragged_batches(dtype, cache):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 600, (300,), generator=g).tolist()
    Case(lens, 16, 8, 64, dtype=dtype, cache=cache).both(sinks=True)  # more rows than runs
    lens = [0] * 100 + [9000] + [1] * 50 + [0, 3000, 0]
    Case(lens, 8, 1, 64, dtype=dtype, cache=cache).both(sinks=True)
    Case([0, 0, 0], 8, 1, 64, dtype=dtype, cache=cache).both(sinks=True)
    Case([0, 0, 0], 8, 1, 64, dtype=dtype, cache=cache, wide=100).both()
    Case([7] * 1000, 8, 2, 64, dtype=dtype, cache=cache, wide=300).both()


@gpu
@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("D", [48, 64, 128, 256])
@pytest.mark.parametrize("B", [39, 76, 100, 160, 330])
def test_many_short_rows(B, D, dtype, cache):
    """Whole rows by CTA and by warp, below, at and past one wave of each: 8 B rows."""
    lens = [(i * 53) % 131 for i in range(B)]
    Case(lens, 16, 8, D, dtype=dtype, cache=cache, seed=B).both(sinks=True)
    c = Case([n + 60 for n in lens], 16, 8, D, dtype=dtype, cache=cache, seed=B)
    c.both(window=33, sinks=True)
    c.both()
    Case(lens, 16, 8, D, dtype=dtype, cache=cache, seed=B, wide=100).both(sinks=True)  # short only by the lengths


@gpu
def test_large_batch_of_slices():
    """More sequences than one per thread: the list is searched by slices."""
    lens = [(i * 37) % 50 for i in range(2500)]
    Case(lens, 2, 1, 64).both()
    Case(lens, 2, 1, 64, wide=60).both(sinks=True)


@gpu
def test_peaked_and_flat_scores():
    for cache in ("bf16", "e4m3"):
        Case([1000, 33], 8, 2, 64, cache=cache, spread=40.0).both(sinks=True)
        Case([1000, 33], 8, 2, 64, cache=cache, spread=0.0).both()
        Case([1000, 33], 8, 2, 64, cache=cache).both(scale=-0.25)
        Case([1000, 33], 8, 2, 64, cache=cache).both(scale=0.0, sinks=True)


@gpu
def test_zero_queries_with_a_scale_of_zero():
    """The scores' factor of such a row stays above 0 (0 times a masked score's -inf is NaN)."""
    for cache in ("bf16", "e4m3"):
        Case([1000, 33], 8, 2, 64, cache=cache, spread=0.0).both(scale=0.0)
        Case([7, 33], 8, 2, 64, cache=cache, spread=0.0).both(scale=-1e-30, sinks=True)


@gpu
def test_extreme_sinks():
    c = Case([0, 1, 50, 3000], 8, 2, 64)
    c.sinks = torch.tensor([-math.inf, 100.0, -100.0, 30.0, 0.0, 1e30, -1e30, 5.0], device="cuda")
    c.both(sinks=True)


@gpu
def test_e4m3_scales_of_all_sizes():
    """Value scales from 2^-60 to 2^60 in one row, and all-zero heads: the accumulator's scale follows."""
    for order in (1, -1):
        c = Case([200, 70], 8, 2, 64, cache="e4m3")
        for b, n in enumerate(c.lengths):
            t = torch.arange(n, device="cuda")
            pg, off = c.table[b].long()[t // 16], t % 16
            c.sc[1][pg, :, off] = (2.0 ** (torch.arange(n, device="cuda") * order % 121 - 60.0))[:, None].expand(n, 2)
            c.sc[0][pg, :, off] *= 2.0 ** ((t % 5) - 2.0)[:, None]
        c.kv[1][c.table[0, 3].long()] = 0
        c.both(sinks=True)
    c = Case([130], 8, 2, 64, cache="e4m3")
    c.q = (c.q.float() * 1e30).bfloat16()
    c.sc[0].mul_(1e-30)
    c.both()


@gpu
def test_strided_q_and_out():
    c = Case([5, 300, 77], 8, 2, 64)
    fused = torch.randn(3, 12, 64, device="cuda").bfloat16()
    q = fused[:, :8]
    out = torch.zeros(3, 10, 64, dtype=torch.bfloat16, device="cuda")
    ws = moe.attention_workspace(3, 8, 2, 64, 100000)
    ws.fill_(0xFF)
    got = c.run(q=q, out=out[:, 1:9], workspace=ws)
    c.check(got, q=q)
    assert torch.all(out[:, 0] == 0) and torch.all(out[:, 9] == 0)
    odd = torch.randn(8, 3, 66, device="cuda").bfloat16().transpose(0, 1)[..., :64]  # heads outermost, rows of 66
    c.check(c.run(q=odd), q=odd)


@gpu
def test_repeated_calls_and_graph_replay_agree():
    c = Case([6000, 0, 1, 800, 77], 16, 2, 64)
    ws = moe.attention_workspace(5, 16, 2, 64, 6000)
    a = c.run(sinks=True, workspace=ws)
    for _ in range(3):
        ws.random_(0, 256)
        assert torch.equal(c.run(sinks=True, workspace=ws), a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.run(sinks=True)
    short = torch.tensor([100, 5, 0, 800, 3], dtype=torch.int32, device="cuda")
    c.table[1] = c.table[0]
    c.lens.copy_(short)
    c.lengths = short.tolist()
    graph.replay()
    torch.cuda.synchronize()
    c.check(out, sinks=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = c.run(sinks=True)
    torch.cuda.synchronize()
    assert torch.equal(other, out)


@gpu
def test_bad_pages_and_lengths_are_left_out_and_reported():
    for cache in ("bf16", "e4m3"):
        c = Case([40, 700], 8, 2, 64, cache=cache, wide=2)
        status = moe.new_status()
        c.check(c.run(status=status))
        assert moe.read_device_status(status) == 0
        pages = c.kv[0].shape[0]
        for bad in (pages, -1, 2 ** 31 - 1, -2 ** 31):
            table = c.table
            c.table = table.clone()
            c.table[0, 2] = bad  # tokens 32..39 of sequence 0
            out = c.run(status=status)
            assert moe.read_device_status(status) == 6 and moe.read_device_status(status) == 0
            c.table = table
            lens = c.lengths
            c.lengths = [32, lens[1]]
            c.check(out)
            c.lengths = lens
        width = c.table.shape[1] * 16
        low = c.run(lens=torch.tensor([-5, 700], dtype=torch.int32, device="cuda"), status=status)
        assert moe.read_device_status(status) == 6 and torch.all(low[0] == 0)
        c.table[0] = c.table[1]
        high = c.run(lens=torch.tensor([width + 1, 700], dtype=torch.int32, device="cuda"), status=status)
        assert moe.read_device_status(status) == 6  # the pages past 700 tokens are -1 as well
        c.lengths = [704, 700]
        assert torch.all(torch.isfinite(high[1]))
        c.lengths = [700, 700]
        c.check(torch.stack((high[1], high[1])), q=torch.stack((c.q[1], c.q[1])))


@gpu
def test_offsets_beyond_32_bits():
    pages, H, S, D = 40000, 8, 64, 128
    c = Case([300, 64], 16, H, D, page=S, cache="e4m3")
    kv = [torch.zeros(pages, H, S, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(pages, H, S, device="cuda") for _ in range(2)]
    assert kv[0].numel() > 2 ** 31
    n = c.kv[0].shape[0]
    for i in range(2):
        kv[i][pages - n:] = c.kv[i]
        sc[i][pages - n:] = c.sc[i]
    c.kv, c.sc = kv, sc
    c.table = torch.where(c.table >= 0, c.table + pages - n, c.table)
    c.both()
    del c, kv, sc
    torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_tokens_appended_are_tokens_read(cache):
    """A decode loop: each step appends its token and attends to all so far, beside attention over the
    rotated tokens kept in 64 bits (16-bit caches hold them rounded: h of each key and value more)."""
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 8
    inv = (150000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    dt = torch.uint8 if cache == "e4m3" else torch.bfloat16
    kc = torch.zeros(30, Hkv, page, D, dtype=dt, device="cuda")
    vc = torch.zeros_like(kc)
    sc = [torch.zeros(30, Hkv, page, device="cuda") for _ in range(2)] if cache == "e4m3" else [None, None]
    table = torch.randperm(30, generator=torch.Generator().manual_seed(3)).int()[:B * 6].view(B, 6).cuda()
    for step in range(45):
        qkv = torch.randn(B, Hq + 2 * Hkv, D, device="cuda").bfloat16()
        pos = torch.full((B,), step, device="cuda")
        slots = table[:, step // page].long() * page + step % page
        q = moe.rotate_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, slots, kc, vc, inv, k_scale=sc[0],
                              v_scale=sc[1])
        lens = torch.full((B,), step + 1, dtype=torch.int32, device="cuda")
        out = moe.paged_attention(q, kc, vc, table, lens, D ** -0.5, k_scale=sc[0], v_scale=sc[1])
    c = Case.__new__(Case)
    c.dtype, c.cache, c.Hq, c.Hkv, c.D, c.page = "bf16", cache, Hq, Hkv, D, page
    c.lengths, c.table, c.kv, c.sc, c.q = [45] * B, table, [kc, vc], sc, q
    c.check(out)


@gpu
def test_shape_refusals():
    c = Case([5, 30], 8, 2, 64)

    def refuse(match, **kw):
        with pytest.raises((ValueError, moe.MoeError), match=match):
            c.run(**kw)

    refuse("its type", q=c.q.half())
    refuse("its type", q=c.q.cpu())
    refuse("must be", q=c.q[..., :48])
    refuse("status 1", q=torch.cat((c.q, c.q), 1)[:, :9].contiguous())
    refuse("lengths", lens=c.lens.long())
    refuse("lengths", lens=c.lens[:1])
    long = Case([5000], 8, 2, 64)
    with pytest.raises(moe.MoeError, match="status 3"):
        long.run(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    refuse("like q", out=torch.empty(2, 8, 64, device="cuda"))
    refuse("status 1", window=-1)
    refuse("status 1", scale=math.nan)
    assert moe.paged_attention(c.q[:0], *c.kv, c.table[:0], c.lens[:0], 0.125).shape == (0, 8, 64)
