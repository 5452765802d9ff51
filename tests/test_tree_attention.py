"""Attention of drafted tokens (moe_tree_attention): refusals on the CPU, then on the GPU against the
formula in 64 bits over trees, chains and stars of 0 to 256 drafts behind contexts from none to
thousands of tokens, odd sizes, every head grouping, sinks, windows, garbage in unused places and masked
keys, bad pages, lengths, starts and parents.

Tolerance of out_d, from what is rounded (h: half a step of a 16-bit type, 2^-8 bf16, 2^-11 fp16;
A = sum_t p_t |v_td| with p summing to at most 1), as for the attention of one token:
  scores      fp32 sums of D products, each step at most 2^-23 of scale sum|q k|: a factor exp(+-e) on
              every p_t, e = (D + 8) 2^-23 scale max_t sum|q k_t|, twice (numerator and sum)      2 e A
  weights     ex2 2^-22, rescaling and the sums over L tokens, 2^-22 each              (L + 64) 2^-22 A
  p to 16 bit h of the product's type (bf16 for a bf16 cache, else fp16)                          h A
              fp16 below its normals: half its smallest step, 2^-25, of the largest p, times
              sum_t |v| (e4m3: of the largest value scale)                             2^-25 L max|v|
  out         half a step                                                                     h |out|"""
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

    def call(kv=None, q=256, dt=0, qst=(256, 64), table=256, ld=4, width=4, lens=256, starts=256, parents=256, N=9, B=3, Hq=4,
             scale=0.125, sinks=None, window=0, out=256, ost=(256, 64), ws=256, wsb=1 << 40, status=None, **cache):
        return L.moe_tree_attention(kv_bytes(**cache) if kv is None else kv, q, dt, *qst, table, ld, width, lens, starts,
                                    parents, N, B, Hq, scale, sinks, window, out, *ost, ws, wsb, status, None)

    for name in ("q", "table", "lens", "starts", "out"):
        assert call(**{name: None}) == 1, name
    assert call(width=100, ld=100, ws=None) == 1  # rows that may be cut need a workspace
    assert call(k=0) == 1 and call(B=0) == 1 and call(B=65537) == 1 and call(N=0) == 1 and call(N=1 << 27) == 1
    assert call(Hq=0) == 1 and call(Hq=3) == 1 and call(Hq=4098) == 1 and call(D=72) == 1 and call(D=272) == 1
    assert call(S=0) == 1 and call(H=300) == 1 and call(width=0) == 1 and call(ld=3) == 1
    assert call(width=1 << 27, ld=1 << 27) == 1 and call(B=1, width=(1 << 27) - 15, wsb=0) == 1
    assert call(B=1, width=(1 << 27) - 16, wsb=0) == 3  # passes, for the workspace to be found too small
    assert call(window=-1) == 1 and call(scale=math.nan) == 1
    assert call(dt=2) == 2 and call(dt=1) == 2 and call(kv=kv_bytes(dt=2)) == 2 and call(kv=kv_bytes(dt=3)) == 1
    assert call(q=264) == 2 and call(out=264) == 2 and call(ws=264) == 2
    for name in ("table", "lens", "starts", "parents", "sinks", "status"):
        assert call(**{name: 258}) == 2, name
    assert call(qst=(256, 65)) == 2 and call(ost=(252, 64)) == 2 and call(qst=(-256, 64)) == 1
    assert call(kv=kv_bytes(k=264)) == 2 and call(kv=kv_bytes(strides=(2048, 1024, 68))) == 2
    assert call(width=100, ld=100, wsb=64) == 3
    size = L.moe_tree_attention_workspace_size
    assert size(0, 1, 4, 2, 64, 0, 99) == 0 and size(3, 0, 4, 2, 64, 0, 99) == 0 and size(3, 1, 3, 2, 64, 0, 99) == 0
    assert size(3, 1, 4, 2, 72, 0, 99) == 0 and size(3, 1, 4, 2, 64, 2, 99) == 0 and size(3, 1, 4, 2, 64, 0, 0) == 0
    assert size(3, 1, 4, 2, 64, 3, 99) == 256 and size(3, 1, 4, 2, 64, 3, 99999) > 256


def test_binding_refuses():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be CUDA tensors"):
        moe.tree_attention(q, kv, kv, i[:, None], i, i, 0.125)


# ------------------------------------------------------------- on the GPU ----
gpu = pytest.mark.gpu


def tree(kind, n, g):
    """Parents of n drafts, as numbers in the sequence."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1 if i == 0 else 0 for i in range(n)]
    if kind == "roots":
        return [-1] * n
    if kind == "binary":
        return [(i + 1) // 2 - 1 for i in range(n)]
    up = [-1]  # random: near ones preferred, a few more roots
    for i in range(1, n):
        up.append(int(torch.randint(max(-1, i - 9), i, (1,), generator=g)))
    return up[:n]


class Case:
    """Sequences with drafts in a paged cache whose unused places hold NaN, and page table entries past
    the lengths -1."""

    def __init__(self, contexts, drafts, Hq, Hkv, D, page=16, dtype="bf16", cache=None, kind="random", nhd=False, seed=0,
                 spread=2.0, wide=0, gap=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        h = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        self.dtype, self.cache, self.Hq, self.Hkv, self.D, self.page = dtype, cache, Hq, Hkv, D, page
        self.contexts, self.drafts, B = contexts, drafts, len(contexts)
        self.lengths = [a + b for a, b in zip(contexts, drafts)]
        self.trees = [tree(kind, n, h) for n in drafts]
        self.parents = None if kind == "none" else torch.tensor(sum(self.trees, []) + [7] * gap, dtype=torch.int32, device="cuda")
        if kind == "none":
            self.trees = [tree("chain", n, h) for n in drafts]
        self.starts = torch.tensor([sum(drafts[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        counts = [-(-n // page) for n in self.lengths]
        pages = sum(counts) + 2
        order = torch.randperm(pages, generator=h)
        width = max(1, max(counts)) + wide
        table = torch.full((B, width), -1, dtype=torch.int32)
        used = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(self.lengths):
            ids = order[at:at + counts[b]]
            table[b, :counts[b]] = ids.int()
            used[ids] = (torch.arange(counts[b] * page) < n).view(-1, page)
            at += counts[b]
        self.table, self.lens = table.cuda(), torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
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
        self.q = (spread * torch.randn(sum(drafts) + gap, Hq, D, generator=g, device="cuda")).to(DT[dtype])
        self.sinks = torch.randn(Hq, generator=g, device="cuda")

    def place(self, b, t):
        """(page, offset) of token t of sequence b."""
        return int(self.table[b, t // self.page]), t % self.page

    def run(self, sinks=False, window=0, scale=None, **kw):
        kw.setdefault("parents", self.parents)
        return moe.tree_attention(kw.pop("q", self.q), *kw.pop("kv", self.kv), kw.pop("table", self.table),
                                  kw.pop("lens", self.lens), kw.pop("starts", self.starts),
                                  self.D ** -0.5 if scale is None else scale, k_scale=self.sc[0], v_scale=self.sc[1],
                                  sinks=self.sinks if sinks else None, window=window, **kw)

    def tokens(self, b):
        """Keys and values [Hkv, length, D] of a sequence in 64 bits, and the value scales."""
        t = torch.arange(self.lengths[b], device="cuda")
        pg, off = self.table[b, t // self.page].long(), t % self.page
        out = []
        for c, s in zip(self.kv, self.sc):
            y = c[pg, :, off]
            y = y.view(torch.float8_e4m3fn).double() * s[pg, :, off].double()[..., None] if self.cache == "e4m3" else y.double()
            out.append(y.transpose(0, 1))
        return out

    def seen(self, b, window, trees=None):
        """[n, length] of what each draft sees."""
        c, n = self.contexts[b], self.drafts[b]
        m = torch.zeros(n, c + n, dtype=torch.bool)
        for i in range(n):
            path, j = [], i
            while j >= 0:
                path.append(j)
                j = (trees or self.trees)[b][j]
            w = window or c + n + 1
            m[i, max(0, c + len(path) - w):c] = True
            m[i, [c + a for a in path[:w]]] = True
        return m.cuda()

    def check(self, out, sinks=False, window=0, scale=None, only=None, trees=None):
        scale = self.D ** -0.5 if scale is None else scale
        G, hp = self.Hq // self.Hkv, HALF["bf16" if self.cache == "bf16" else "fp16"]
        for b, n in enumerate(self.drafts):
            if n == 0 or (only is not None and b not in only):
                continue
            lo = int(self.starts[b])
            k, v = self.tokens(b)
            see = self.seen(b, window, trees)
            q = self.q[lo:lo + n].double().view(n, self.Hkv, G, self.D).permute(1, 2, 0, 3)
            s = (q @ k[:, None].transpose(-1, -2)) * scale  # [Hkv, G, n, L]
            s = s.masked_fill(~see, -math.inf)
            if sinks:
                s = torch.cat((s, self.sinks.double().view(self.Hkv, G, 1, 1).expand(-1, -1, n, 1)), -1)
            p = torch.softmax(s, -1).nan_to_num(0.0)[..., :self.lengths[b]]
            want, A = p @ v[:, None], p @ v[:, None].abs()
            most = ((q.abs() @ k[:, None].abs().transpose(-1, -2)) * abs(scale)).masked_fill(~see, 0.0).amax(-1, keepdim=True)
            L = self.lengths[b]
            tol = A * (2 * (self.D + 8) * 2.0 ** -23 * most + (L + 64) * 2.0 ** -22 + hp) + want.abs() * HALF[self.dtype]
            if self.cache != "bf16":
                tol = tol + 2.0 ** -25 * L * v.abs().amax()
            tol = tol + (2.0 ** -25 if self.dtype == "fp16" else 1e-38)
            got = out[lo:lo + n].double().view(n, self.Hkv, G, self.D).permute(1, 2, 0, 3)
            bad = (got - want).abs() > tol
            assert torch.all(torch.isfinite(got)), f"sequence {b}"
            assert not torch.any(bad), (f"sequence {b}: {int(bad.sum())} of {bad.numel()}, worst "
                                        f"{float(((got - want).abs() / tol).max()):.2f} of the tolerance")


SIZES = [(8, 2, 64, 16, "bf16", "bf16", False), (64, 8, 64, 16, "bf16", "bf16", False), (20, 4, 96, 24, "fp16", "fp16", True),
         (16, 1, 128, 64, "bf16", "e4m3", False), (4, 4, 80, 1, "bf16", "bf16", False), (6, 2, 256, 8, "fp16", "fp16", False),
         (5, 1, 16, 7, "bf16", "e4m3", True), (24, 2, 128, 32, "fp16", "e4m3", False), (32, 4, 128, 128, "bf16", "bf16", False),
         (10, 2, 240, 16, "bf16", "e4m3", False), (8, 8, 64, 16, "fp16", "e4m3", False)]


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,cache,nhd", SIZES)
@pytest.mark.parametrize("contexts,drafts", [([0], [1]), ([90], [6]), ([0, 1, 15, 63, 64], [3, 1, 17, 1, 64]),
                                             ([65, 300, 0, 127, 1000, 5], [7, 0, 0, 2, 33, 12])])
@pytest.mark.parametrize("kind,sinks", [("random", True), ("none", False)])
def test_against_64_bits(Hq, Hkv, D, page, dtype, cache, nhd, contexts, drafts, kind, sinks):
    c = Case(contexts, drafts, Hq, Hkv, D, page, dtype, cache, kind, nhd, wide=3)
    status = moe.new_status()
    c.check(c.run(sinks, status=status), sinks)
    assert moe.read_device_status(status) == 0


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,cache,nhd", [SIZES[i] for i in (1, 2, 3, 5, 7, 10)])
@pytest.mark.parametrize("window", [1, 2, 5, 16, 100, 128, 1000])
@pytest.mark.parametrize("kind", ["random", "chain", "none"])
def test_windows(Hq, Hkv, D, page, dtype, cache, nhd, window, kind):
    c = Case([0, 40, 128, 700, 1500], [9, 1, 40, 64, 5], Hq, Hkv, D, page, dtype, cache, kind, nhd, seed=window)
    # pages before every window are gone
    for b, n in enumerate(c.contexts):
        c.table[b, :max(0, n - window + 1) // page] = -1
    status = moe.new_status()
    out = c.run(True, window, status=status)
    assert moe.read_device_status(status) == 0
    keep = c.table
    c.table = keep.clamp(min=0)  # (the check reads them, and masks them)
    c.check(out, True, window)


@gpu
@pytest.mark.parametrize("kind", ["chain", "none", "star", "roots", "binary", "random"])
@pytest.mark.parametrize("n", [2, 31, 32, 33, 100, 255, 256])
def test_trees_of_every_size(kind, n):
    c = Case([70, 5], [n, 3], 8, 2, 64, kind=kind, seed=n)
    c.check(c.run(True), True)
    c.check(c.run(window=20), window=20)


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,dtype,cache", [(64, 8, 64, "bf16", "bf16"), (64, 4, 128, "bf16", "e4m3"),
                                                  (64, 4, 128, "bf16", "bf16"), (32, 2, 64, "fp16", "e4m3"),
                                                  (16, 1, 112, "fp16", "fp16"), (12, 1, 192, "bf16", "bf16")])
@pytest.mark.parametrize("drafts", [[64, 64], [256, 17], [16, 16], [1, 130]])
def test_many_rows(Hq, Hkv, D, dtype, cache, drafts):
    """Row tiles of one key head: one, two, and several pairs; the last one short."""
    c = Case([333, 1200], drafts, Hq, Hkv, D, dtype=dtype, cache=cache, seed=sum(drafts))
    c.check(c.run(True), True)


@gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("contexts,drafts", [([20000], [5]), ([40000, 3, 9000], [64, 2, 40]), ([8000] * 3, [3] * 3)])
def test_long_contexts_are_cut_and_joined(contexts, drafts, cache):
    c = Case(contexts, drafts, 16, 2, 64, page=64, cache=cache, seed=4)
    out = c.run(True)
    c.check(out, True)
    for _ in range(3):
        assert torch.equal(c.run(True), out)


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,cache", [(8, 1, 64, 16, "bf16", "bf16"), (32, 2, 128, 24, "fp16", "fp16"),
                                                       (16, 4, 128, 64, "bf16", "e4m3"), (6, 2, 80, 7, "fp16", "e4m3"),
                                                       (4, 1, 240, 16, "bf16", "bf16"), (32, 1, 64, 32, "bf16", "e4m3")])
@pytest.mark.parametrize("contexts,drafts", [([5000], [9]), ([900] * 40, [4] * 40), ([1, 9000, 0, 700], [12, 3, 1, 70]),
                                             ([2100] * 12, [20] * 12)])
@pytest.mark.parametrize("window", [0, 3000])
def test_cut_and_whole_items(Hq, Hkv, D, page, dtype, cache, contexts, drafts, window):
    c = Case(contexts, drafts, Hq, Hkv, D, page, dtype, cache, seed=len(contexts))
    out = c.run(True, window)
    c.check(out, True, window)
    assert torch.equal(c.run(True, window), out)


@gpu
def test_many_sequences():
    h = torch.Generator().manual_seed(1)
    ctx = torch.randint(0, 200, (700,), generator=h).tolist()
    n = torch.randint(0, 5, (700,), generator=h).tolist()
    c = Case(ctx, n, 8, 2, 64, seed=3)
    c.check(c.run(True), True)
    c.check(c.run(window=32), window=32)


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30])
@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_scales(scale, cache):
    c = Case([0, 200, 600], [5, 20, 3], 8, 2, 64, dtype="fp16" if cache == "fp16" else "bf16", cache=cache, seed=5)
    c.check(c.run(True, scale=scale), True, scale=scale)


@gpu
@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_rising_scores_move_what_the_sums_are_about(cache):
    """Keys that grow along the context: each tile's scores stand far above the last one's."""
    c = Case([1000], [8], 8, 2, 64, dtype="fp16" if cache == "fp16" else "bf16", cache=cache, seed=6)
    grow = torch.linspace(0.1, 6.0, 1008, device="cuda")
    t = torch.arange(1008, device="cuda")
    pg, off = c.table[0, t // 16].long(), t % 16
    if cache == "e4m3":
        c.sc[0][pg, :, off] *= grow[:, None]
        c.sc[1][pg, :, off] *= grow[:, None] ** 4
    else:
        c.kv[0][pg, :, off] = (c.kv[0][pg, :, off].float() * grow[:, None, None]).to(c.kv[0].dtype)
    c.check(c.run(True), True)


@gpu
def test_e4m3_scales_of_every_kind():
    """Heads of zeros with the scale 1 among small ones, negative and zero scales."""
    c = Case([500, 70], [9, 64], 8, 2, 128, cache="e4m3", seed=7)
    for s in c.sc:
        s.mul_(1e-3)
    c.kv[1][2:5, :, 3] = 0
    c.sc[1][2:5, :, 3] = 1.0
    c.sc[1][7] *= -1
    c.sc[0][8] *= -1
    c.sc[1][9, :, 5] = 0
    c.check(c.run(True), True)


@gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_masked_keys_may_be_anything(cache):
    """NaN and infinite keys of drafts reach only what sees them; rows outside the sequences are left as they were."""
    c = Case([33, 100], [12, 70], 8, 2, 64, cache=cache, kind="binary", seed=8, gap=5)
    want = c.run(True)
    c.check(want, True)
    for b, j in ((0, 3), (1, 2), (1, 40)):
        pg, off = c.place(b, c.contexts[b] + j)
        if cache == "e4m3":
            c.sc[0][pg, :, off] = math.nan if j == 3 else math.inf
        else:
            c.kv[0][pg, :, off] = math.nan if j == 3 else math.inf
    out = torch.full_like(c.q, 9.0)
    assert c.run(True, out=out) is not None
    assert torch.all(out[82:] == 9.0)
    clean = [i for i in range(12) if not c.seen(0, 0)[i, 33 + 3]]
    clean += [12 + i for i in range(70) if not c.seen(1, 0)[i, 100 + 2] and not c.seen(1, 0)[i, 100 + 40]]
    assert len(clean) > 30 and torch.equal(out[clean], want[clean])
    assert not torch.all(torch.isfinite(out[[3, 14, 52]]))


@gpu
@pytest.mark.parametrize("window", [0, 64])
@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_one_draft_is_the_next_token(cache, window):
    """Within both operators' tolerance of each other."""
    c = Case([0, 5, 63, 500, 3000], [1] * 5, 16, 2, 64, dtype="fp16" if cache == "fp16" else "bf16", cache=cache, kind="roots")
    one = moe.paged_attention(c.q, *c.kv, c.table, c.lens, 0.125, k_scale=c.sc[0], v_scale=c.sc[1], sinks=c.sinks, window=window)
    c.check(one, True, window)
    c.check(c.run(True, window), True, window)


@gpu
def test_bad_pages_lengths_starts_and_parents():
    c = Case([40, 50, 60], [5, 6, 7], 8, 2, 64, seed=9)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    status = moe.new_status()
    # starts: the sequence is left out (in the first, the last sequence has rows 3 to 9)
    for starts, others in (([0, 5, 3, 10], []), ([-1, 5, 11, 18], [1, 2]), ([0, 5, 11, 19], [0, 1]), ([0, 5, 11, 1 << 30], [0, 1])):
        out = torch.full_like(c.q, 9.0)
        c.run(True, starts=i(starts), out=out, status=status)
        assert moe.read_device_status(status) == 6
        c.check(out, True, only=others)
        left = slice(10, 18) if not others else slice(0, 5) if 0 not in others else slice(11, 18)
        assert torch.all(out[left] == 9.0)
    many = Case([5, 5], [257, 2], 8, 2, 64, seed=1)
    out = torch.full_like(many.q, 9.0)
    many.run(out=out, status=status)
    assert moe.read_device_status(status) == 6 and torch.all(out[:257] == 9.0)
    many.check(out, only=[1])
    # lengths: past the table, and fewer tokens than drafts
    most = c.table.shape[1] * 16
    for lens, b, n in (([45, 56, most + 100], 2, most), ([45, 56, (1 << 31) - 1], 2, most), ([3, 56, 67], 0, 3), ([-5, 56, 67], 0, 0)):
        out = c.run(True, lens=i(lens), status=status)
        assert moe.read_device_status(status) == 6
        c.check(out, True, only=[s for s in range(3) if s != b])
        if n == 0:
            assert torch.all(out[:5] == 0)
        elif n == 3:  # no context, drafts 0 to 2 are tokens 0 to 2
            d = Case([40, 50, 60], [5, 6, 7], 8, 2, 64, seed=9)
            d.contexts, d.lengths = [0, 50, 60], [5, 56, 67]
            seen = d.seen(0, 0)
            seen[:, 3:] = False
            d.seen = lambda *a: seen
            d.check(out, True, only=[0])
    # parents: not before their draft
    up = c.parents.clone()
    up[2], up[8], up[14] = 2, 1 << 20, -7
    out = c.run(True, parents=up, status=status)
    assert moe.read_device_status(status) == 6
    trees = [list(t) for t in c.trees]
    trees[0][2] = trees[1][3] = trees[2][3] = -1
    c.check(out, True, trees=trees)
    # a page out of range: its tokens are left out
    bad = c.table.clone()
    bad[1, 1] = 1 << 29
    out = c.run(True, table=bad, status=status)
    assert moe.read_device_status(status) == 6
    see = c.seen(1, 0)
    see[:, 16:32] = False
    c.seen = lambda *a: see
    c.check(out, True, only=[1])


@gpu
def test_gpu_refusals():
    c = Case([40, 50], [5, 6], 8, 2, 64, seed=9)
    for bad in (dict(q=c.q.float()), dict(q=c.q.half()), dict(q=c.q[0]), dict(lens=c.lens.long()), dict(starts=c.starts[:2]),
                dict(parents=c.parents[:5]), dict(parents=c.parents.long()), dict(table=c.table[:1]), dict(table=c.table.t()),
                dict(out=c.q.float()), dict(out=c.q[:5]), dict(workspace=c.q), dict(lens=c.lens.cpu()), dict(status=c.q),
                dict(q=c.q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            c.run(**bad)
    with pytest.raises(moe.MoeError):
        c.run(window=-1)
    long = Case([1000], [2], 8, 2, 64, seed=9)
    with pytest.raises(moe.MoeError):
        long.run(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.tree_attention_workspace(0, 1, 8, 2, 64, 100)
    e = torch.zeros(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    assert c.run(q=e, parents=None).shape == (0, 8, 64)


@gpu
def test_strided_views_and_given_buffers():
    c = Case([40, 500], [5, 60], 8, 2, 64, seed=10)
    want = c.run(True)
    wide = torch.zeros(65, 14, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = c.q
    out = torch.zeros(65, 10, 72, dtype=torch.bfloat16, device="cuda")[:, 1:9, :64]
    table = torch.full((2, 90), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    ws = moe.tree_attention_workspace(65, 2, 8, 2, 64, 90 * 16)
    got = c.run(True, q=wide[:, 3:11], out=out, table=table[:, :c.table.shape[1]], workspace=ws.fill_(255))
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
    one = Case([70], [1], 1, 1, 64, seed=1)
    one.check(one.run())


@gpu
def test_far_cache_offsets():
    """Pages past 2^32 bytes."""
    pages = 33000
    k = torch.zeros(pages, 8, 64, 128, dtype=torch.bfloat16, device="cuda")
    assert (pages - 5) * k.stride(0) * 2 > 1 << 32
    c = Case([200], [9], 16, 8, 128, page=64, seed=2)
    n = c.kv[0].shape[0]
    v = torch.zeros_like(k)
    k[-n:], v[-n:] = c.kv
    want = c.run(True)
    got = c.run(True, kv=[k, v], table=torch.where(c.table >= 0, c.table + pages - n, -1))
    assert torch.equal(got, want)


@gpu
def test_captured_graphs_and_a_side_stream():
    """Two graphs with a workspace each, replayed at the same time, on lengths and trees that change between replays."""
    cases = [Case([3000, 40], [20, 7], 16, 2, 64, seed=s) for s in (1, 2)]
    wants = [c.run(True) for c in cases]
    graphs, kept, outs, streams = [], [], [], [torch.cuda.Stream() for _ in cases]
    for c, st in zip(cases, streams):
        ws, out = moe.tree_attention_workspace(27, 2, 16, 2, 64, c.table.shape[1] * 16), torch.zeros_like(c.q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(True, out=out, workspace=ws)
        graphs.append(graph)
        kept.append(ws)  # a graph holds no tensor that was made before its capture
        outs.append(out)
    for _ in range(5):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert torch.equal(out, want)
    a, b = cases
    a.parents.copy_(b.parents)
    graphs[0].replay()
    torch.cuda.synchronize()
    a.check(outs[0], True, trees=b.trees)
    got = a.run(True, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(got, outs[0])
