"""Moves within a paged cache of several layers (moe_copy_pages, moe_compact_drafts): refusals on the
CPU, then on the GPU against the same moves made value by value, with every place that no move names
checked to be untouched.  Values are moved, not computed: everything is compared bit for bit."""
import ctypes
import struct

import pytest
import torch

import sparse_moe_layer_gb300 as moe

KV = struct.Struct("4P9q5i4x")  # moe_kv_cache
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.uint8}


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


# ------------------------------------------------------------- on the CPU ----
def kv_bytes(dt=0, P=4, S=16, H=2, D=64, k=256, v=512, ks=0, vs=0, strides=None):
    st = strides or (H * S * D, S * D, D)
    return KV.pack(k, v, ks, vs, *st, *st, H * S, S, 1, dt, P, S, H, D)


def strides(*s):
    return ctypes.cast((ctypes.c_int64 * 3)(*s), ctypes.c_void_p)


def test_copy_refusals_on_the_host():
    L = moe.lib()

    def call(kv=None, layers=2, ls=(8192, 8192, 128), src=256, dst=256, tokens=None, N=3, status=None, **cache):
        return L.moe_copy_pages(kv_bytes(**cache) if kv is None else kv, layers, strides(*ls) if ls else None, src, dst,
                                tokens, N, status, None)

    for name in ("src", "dst"):
        assert call(**{name: None}) == 1, name
    assert L.moe_copy_pages(None, 1, None, 256, 256, None, 1, None, None) == 1
    assert call(k=0) == 1 and call(D=72) == 1 and call(N=0) == 1 and call(N=-1) == 1
    assert call(layers=0) == 1 and call(layers=65537) == 1 and call(ls=None) == 1
    assert call(ls=(-8192, 8192, 0)) == 1 and call(ls=(8192, 8196, 0)) == 2 and call(ls=(8200, 8192, 7), N=0) == 1
    assert call(N=(1 << 31) - 1, layers=2) == 1  # more CTAs than a launch has
    assert call(src=258) == 2 and call(dst=257) == 2 and call(tokens=258) == 2 and call(status=258) == 2
    assert call(dt=2) == 2 and call(dt=3) == 1 and call(dt=3, ks=256, vs=256, ls=(8192, 8192, -4)) == 1


def test_compact_refusals_on_the_host():
    L = moe.lib()

    def call(kv=None, layers=2, ls=(8192, 8192, 128), table=256, ld=4, width=4, lens=256, starts=256, kept=256, kld=5, B=3,
             K=5, out=512, status=None, **cache):
        return L.moe_compact_drafts(kv_bytes(**cache) if kv is None else kv, layers, strides(*ls) if ls else None, table, ld,
                                    width, lens, starts, kept, kld, B, K, out, status, None)

    for name in ("table", "lens", "starts", "kept", "out"):
        assert call(**{name: None}) == 1, name
    assert call(k=0) == 1 and call(B=0) == 1 and call(B=65537) == 1 and call(K=0) == 1 and call(width=0) == 1
    assert call(ld=3) == 1 and call(kld=4) == 1 and call(width=1 << 28, ld=1 << 28) == 1
    assert call(out=256) == 1  # the lengths themselves
    assert call(layers=0) == 1 and call(ls=None) == 1 and call(ls=(8192, 8196, 0)) == 2
    for name in ("table", "lens", "starts", "kept", "out", "status"):
        assert call(**{name: 258}) == 2, name


def test_binding_refuses():
    kv = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for c in (kv, kv[None]):
        with pytest.raises(ValueError, match="must be CUDA tensors"):
            moe.copy_pages(c, c, i, i)
        with pytest.raises(ValueError, match="must be CUDA tensors"):
            moe.compact_drafts(c, c, i[:, None], i, i, i[:, None])


# ------------------------------------------------------------- on the GPU ----
gpu = pytest.mark.gpu


def caches(layers, pages, H, page, D, kind, nhd=False, pad=0, seed=0):
    """[k, v, k_scale, v_scale]; layers 0: without that dim; nhd: tokens-major pages; pad: values
    between heads (or tokens) that belong to no place."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lead = (layers,) if layers else ()
    at = (*lead, pages, page, H) if nhd else (*lead, pages, H, page)
    made = []
    for _ in range(2):
        if kind == "e4m3":
            x = torch.randint(0, 256, (*at, D + pad), dtype=torch.uint8, device="cuda", generator=g)
        else:
            x = torch.randn(*at, D + pad, device="cuda", generator=g).to(TYPES[kind])
        x = x[..., :D]
        made.append(x.transpose(-3, -2) if nhd else x)
    for _ in range(2):
        s = torch.randn(at, device="cuda", generator=g)
        made.append(None if kind != "e4m3" else s.transpose(-2, -1) if nhd else s)
    return made


def clones(c):
    """Copies in the same layout, gaps included."""
    out = []
    for x in c:
        if x is None:
            out.append(None)
            continue
        base = x._base if x._base is not None else x
        out.append(base.clone().as_strided(x.shape, x.stride(), x.storage_offset()))
    return out


def equal(a, b):
    for x, y in zip(a, b):
        if x is not None:
            whole = [(t._base if t._base is not None else t).contiguous().view(torch.uint8) for t in (x, y)]
            assert torch.equal(*whole)


def move(c, moves):
    """moves (page, place, page, place): all read, then written."""
    a, o, b, u = (torch.tensor(x, device="cuda") for x in zip(*moves)) if moves else [torch.zeros(0, dtype=torch.long)] * 4
    for i, x in enumerate(c):
        if x is None or not moves:
            continue
        y = x if x.dim() == (5 if i < 2 else 4) else x[None]
        y[:, b, :, u] = y[:, a, :, o].clone()


LAYOUTS = [(0, 2, 16, 64, "bf16", False, 0), (3, 8, 16, 64, "bf16", False, 0), (2, 3, 24, 96, "fp16", True, 8),
           (5, 4, 64, 128, "e4m3", False, 16), (1, 1, 1, 16, "e4m3", False, 0), (2, 5, 7, 256, "fp16", False, 0),
           (3, 2, 8, 80, "e4m3", True, 0)]


@gpu
@pytest.mark.parametrize("layers,H,page,D,kind,nhd,pad", LAYOUTS)
@pytest.mark.parametrize("N,part", [(1, False), (5, True), (40, False), (33, True)])
def test_copies(layers, H, page, D, kind, nhd, pad, N, part):
    h = torch.Generator().manual_seed(N)
    c = caches(layers, 2 * N + 2, H, page, D, kind, nhd, pad)
    want, got = clones(c), clones(c)
    order = torch.randperm(2 * N + 2, generator=h).int()
    src, dst = order[:N].clone(), order[N:2 * N].clone()
    tokens = torch.randint(0, page + 1, (N,), generator=h, dtype=torch.int32) if part else None
    if N > 8:  # padding
        src[3], dst[4] = -1, -5
    moves = [(a, o, b, o) for i, (a, b) in enumerate(zip(src.tolist(), dst.tolist())) if a >= 0 and b >= 0
             for o in range(page if tokens is None else int(tokens[i]))]
    move(want, moves)
    status = moe.new_status()
    assert moe.copy_pages(got[0], got[1], src.cuda(), dst.cuda(), tokens=None if tokens is None else tokens.cuda(),
                          k_scale=got[2], v_scale=got[3], status=status) is None
    equal(got, want)
    assert moe.read_device_status(status) == 0


@gpu
def test_copy_leaves_out_bad_pages_and_bounds_counts():
    c = caches(2, 8, 2, 16, 64, "e4m3")
    for src, dst, tokens in (([0, 1], [2, 8], [3, 3]), ([0, 1 << 30], [2, 3], [3, 3])):
        want, got = clones(c), clones(c)
        move(want, [(0, o, 2, o) for o in range(3)])
        status = moe.new_status()
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        moe.copy_pages(got[0], got[1], i(src), i(dst), i(tokens), got[2], got[3], status=status)
        equal(got, want)
        assert moe.read_device_status(status) == 6
    want, got = clones(c), clones(c)
    move(want, [(1, o, 3, o) for o in range(16)])  # -4: none of page 0; 17: all of page 1
    moe.copy_pages(got[0], got[1], i([0, 1]), i([2, 3]), i([-4, 17]), got[2], got[3], status=status)
    equal(got, want)
    assert moe.read_device_status(status) == 6
    moe.copy_pages(got[0], got[1], i([]), i([]), k_scale=got[2], v_scale=got[3])
    equal(got, want)


class Drafts:
    """Sequences of a paged cache whose last tokens are drafts, and which of them are kept."""

    def __init__(self, contexts, drafts, kept, page, wide=0, seed=0):
        h = torch.Generator().manual_seed(seed)
        self.page, self.contexts, self.drafts, self.kept = page, contexts, drafts, kept
        lengths = [a + b for a, b in zip(contexts, drafts)]
        counts = [-(-n // page) for n in lengths]
        self.pages = sum(counts) + 2
        order = torch.randperm(self.pages, generator=h).tolist()
        self.table = torch.full((len(lengths), max(1, max(counts)) + wide), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table_t = self.table.cuda()
        K = max(1, max(len(k) for k in kept))
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.lens = i(lengths)
        self.starts = i([sum(drafts[:b]) for b in range(len(drafts) + 1)])
        self.kept_t = i([list(k) + [-1] * (K - len(k)) for k in kept])

    def moves(self):
        out = []
        for b, kept in enumerate(self.kept):
            row, c = self.table[b].tolist(), self.contexts[b]
            out += [(row[(c + f) // self.page], (c + f) % self.page, row[(c + t) // self.page], (c + t) % self.page)
                    for t, f in enumerate(kept)]
        return out

    def lengths_after(self):
        return [c + len(k) for c, k in zip(self.contexts, self.kept)]

    def run(self, c, **kw):
        return moe.compact_drafts(c[0], c[1], kw.pop("table", self.table_t), kw.pop("lens", self.lens),
                                  kw.pop("starts", self.starts), kw.pop("kept", self.kept_t), k_scale=c[2], v_scale=c[3], **kw)


def ragged(B, seed, most=40):
    h = torch.Generator().manual_seed(seed)
    contexts, drafts, kept = [], [], []
    for b in range(B):
        n = int(torch.randint(0, most + 1, (1,), generator=h))
        k = int(torch.randint(0, n + 1, (1,), generator=h))
        contexts.append(int(torch.randint(0, 90, (1,), generator=h)))
        drafts.append(n)
        kept.append(sorted(torch.randperm(n, generator=h)[:k].tolist()))
    return contexts, drafts, kept


@gpu
@pytest.mark.parametrize("layers,H,page,D,kind,nhd,pad", LAYOUTS)
@pytest.mark.parametrize("B", [1, 3, 17])
def test_compacts(layers, H, page, D, kind, nhd, pad, B):
    d = Drafts(*ragged(B, seed=B), page=page, wide=2)
    c = caches(layers, d.pages, H, page, D, kind, nhd, pad)
    want, got = clones(c), clones(c)
    move(want, d.moves())
    status = moe.new_status()
    n = d.run(got, status=status)
    equal(got, want)
    assert n.dtype == torch.int32 and n.tolist() == d.lengths_after()
    assert moe.read_device_status(status) == 0


@gpu
@pytest.mark.parametrize("kept", [[], [0], [255], list(range(256)), list(range(1, 256)), list(range(0, 256, 2)),
                                  list(range(100)) + list(range(150, 256)), [31, 32, 33, 64, 65, 200]])
def test_compacts_long_lists(kept):
    d = Drafts([13], [256], [kept], page=16)
    c = caches(9, d.pages, 2, 16, 64, "bf16")
    want, got = clones(c), clones(c)
    move(want, d.moves())
    out = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    assert d.run(got, out=out) is not None and out.tolist() == [13 + len(kept)]
    equal(got, want)


@gpu
@pytest.mark.parametrize("given,counts", [([2, 1, 3, -1], 1), ([0, 4, 9, 3], 2), ([3, 3, 5, 6], 1), ([1, 2, 8, 9], 2),
                                          ([-1, 2, 3, 4], 0), ([1 << 30, 0, 1, 2], 0)])
def test_lists_end_at_what_is_no_ascending_draft(given, counts):
    """Eight drafts: what stands before the first bad entry is kept."""
    d = Drafts([5], [8], [given[:counts]], page=4)
    c = caches(2, d.pages, 2, 4, 64, "fp16")
    want, got = clones(c), clones(c)
    move(want, d.moves())
    status = moe.new_status()
    n = d.run(got, kept=torch.tensor([given], dtype=torch.int32, device="cuda"), status=status)
    equal(got, want)
    assert n.tolist() == [5 + counts]
    assert moe.read_device_status(status) == (0 if given[counts] == -1 else 6)


@gpu
def test_sequences_that_do_not_fit_stay():
    d = Drafts([5, 6, 7], [8, 8, 8], [[1, 3]] * 3, page=4)
    c = caches(2, d.pages, 2, 4, 64, "fp16")
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    status = moe.new_status()
    most = d.table.shape[1] * 4
    for lens, starts, stays in (([13, 7, 15], [0, 8, 16, 24], 1), ([13, most + 1, 15], [0, 8, 16, 24], 1),
                                ([13, 14, 15], [0, 8, 16, 9], 2), ([13, 14, 15], [-3, 5, 13, 21], 0)):
        want, got = clones(c), clones(c)
        moves = d.moves()
        del moves[2 * stays:2 * stays + 2]
        move(want, moves)
        n = d.run(got, lens=i(lens), starts=i(starts), status=status)
        equal(got, want)
        assert n.tolist() == [lens[b] if b == stays else [7, 8, 9][b] for b in range(3)]
        assert moe.read_device_status(status) == 6
    bad = d.table.clone()
    bad[1, (6 + 1) // 4] = 1 << 20  # draft 1 of sequence 1 stays, its place among the kept too
    want, got = clones(c), clones(c)
    moves = [m for m in d.moves() if m[0] != int(d.table[1, 1]) and m[2] != int(d.table[1, 1])]
    move(want, moves)
    n = d.run(got, table=bad.cuda(), status=status)
    equal(got, want)
    assert n.tolist() == [7, 8, 9] and moe.read_device_status(status) == 6


@gpu
def test_gpu_refusals():
    d = Drafts([5, 6], [8, 8], [[1, 3]] * 2, page=4)
    c = caches(2, d.pages, 2, 4, 64, "e4m3")
    with pytest.raises(ValueError, match="out cannot be lengths"):
        d.run(c, out=d.lens)
    with pytest.raises(ValueError, match="starts must be"):
        d.run(c, starts=d.starts[:2])
    with pytest.raises(ValueError, match="kept must be"):
        d.run(c, kept=d.kept_t.long())
    with pytest.raises(ValueError, match="page_table must be"):
        d.run(c, table=d.table[0].cuda())
    with pytest.raises(ValueError, match="needs k_scale and v_scale"):
        d.run([c[0], c[1], c[2], None])
    with pytest.raises(ValueError):
        d.run([c[0], c[1][:1], c[2], c[3]])
    with pytest.raises(ValueError):
        d.run([c[0], c[1], c[2], c[3][0]])
    with pytest.raises(ValueError, match="equal strides"):
        d.run([c[0], c[1], c[2], c[3].expand(2, -1, -1, -1)[:1].expand_as(c[3])])
    with pytest.raises(ValueError, match="contiguous"):
        d.run([c[0].transpose(3, 4), c[1].transpose(3, 4), c[2], c[3]])
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(src=i.long()), dict(src=i[:, None]), dict(dst=i[:1]), dict(tokens=i[:1]), dict(dst=i.cpu())):
        kw = dict(src=i, dst=i + 1) | bad
        with pytest.raises(ValueError):
            moe.copy_pages(c[0], c[1], kw.pop("src"), kw.pop("dst"), k_scale=c[2], v_scale=c[3], **kw)
    with pytest.raises(moe.MoeError):
        moe.copy_pages(c[0][..., 8:24], c[1][..., 8:24], i, i + 1, k_scale=c[2], v_scale=c[3])  # not 16-byte aligned


@gpu
def test_long_cache_offsets_pass_32_bits():
    """Pages whose bytes lie past 2^32 from the first, and layers too."""
    pages, page = 2800, 128
    k = torch.zeros(3, pages, 8, page, 256, dtype=torch.bfloat16, device="cuda")  # 4.4 GB
    v = k.clone()
    far = pages - 1
    k[:, 3] = torch.randn(3, 8, page, 256, device="cuda").bfloat16()
    v[:, 3] = torch.randn(3, 8, page, 256, device="cuda").bfloat16()
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    assert (2 * pages + far) * k.stride(1) * 2 > 1 << 32
    moe.copy_pages(k, v, i([3]), i([far]))
    assert torch.equal(k[:, far], k[:, 3]) and torch.equal(v[:, far], v[:, 3])
    assert int(k.view(torch.int16)[:, 4:far].count_nonzero()) == 0
    table = i([[far, 3]])
    n = moe.compact_drafts(k, v, table, i([2 * page]), i([0, page]), i([[5, 100]]))
    assert n.tolist() == [page + 2]
    assert torch.equal(k[:, 3, :, 0], k[:, far, :, 5]) and torch.equal(v[:, 3, :, 1], v[:, far, :, 100])


@gpu
def test_captured_and_replayed():
    """A graph of both moves replays on new contents; two graphs share nothing."""
    d = Drafts([5, 30], [8, 8], [[1, 3], [0, 2, 7]], page=4)
    c = caches(3, d.pages + 4, 2, 4, 64, "e4m3")
    got = clones(c)
    src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([d.pages], [d.pages + 2]))
    out = torch.empty(2, dtype=torch.int32, device="cuda")

    def both():
        d.run(got, out=out)
        moe.copy_pages(got[0], got[1], src, dst, k_scale=got[2], v_scale=got[3])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (1, 2):
        new = caches(3, d.pages + 4, 2, 4, 64, "e4m3", seed=seed)
        want = clones(new)
        move(want, d.moves() + [(d.pages, o, d.pages + 2, o) for o in range(4)])
        for a, b in zip(got, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        equal(got, want)
        assert out.tolist() == d.lengths_after()
