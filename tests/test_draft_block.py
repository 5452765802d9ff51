"""Steps of drafted tokens (DraftBlock of examples/decode_block.py): rotate_append,
tree_attention, compact_drafts and copy_pages together, eager and as a CUDA graph; and the
new operators on streams other than the current one."""
import importlib.util
import os

import pytest
import torch

import sparse_moe_layer_gb300 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(H=256, I=256, E=8, top_k=2, q_heads=8, kv_heads=2, head_dim=64, page=8)
PARENTS = [-1, 0, 0, 1, 1, 2, -1, 6, 3]
PATHS = [[0, 1, 3, 8], [6, 7], [0, 2, 5], [0], []]  # of five sequences


@pytest.fixture(scope="module")
def example():
    moe.build()
    spec = importlib.util.spec_from_file_location("decode_block", os.path.join(ROOT, "examples", "decode_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def kept_of(paths):
    most = max(len(p) for p in paths)
    return torch.tensor([p + [-1] * (most - len(p)) for p in paths], dtype=torch.int32, device="cuda")


def tokens(b, i):
    """What the cache holds of sequence i: raw keys, values (and scales) of its tokens."""
    t = torch.arange(int(b.lengths[i]), device="cuda")
    pg, off = b.table[i, t // b.page].long(), t % b.page
    return [c[pg, :, off] for c in (b.k, b.v, b.ks, b.vs) if c is not None]


def check(b, q, out, window):
    """The attention of a step against 64 bits: two roundings of bf16 (probabilities, output; fp16 probabilities
    in an e4m3 cache are finer) and the fp32 score error, far below them here."""
    n = len(PARENTS)
    for i in range(b.B):
        raw, L = tokens(b, i), int(b.lengths[i])
        kv = [x.double() for x in raw] if len(raw) == 2 else [
            x.view(torch.float8_e4m3fn).double() * s.double()[..., None] for x, s in zip(raw[:2], raw[2:])]
        k, v = (x.transpose(0, 1).repeat_interleave(4, 0) for x in kv)  # [Hq, L, D]
        see = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        c = L - n
        for d in range(n):
            path, a = [], d
            while a >= 0:
                path.append(a)
                a = PARENTS[a]
            w = window or L + 1
            see[d, max(0, c + len(path) - w):c] = True
            see[d, [c + a for a in path[:w]]] = True
        s = (q[i * n:(i + 1) * n].double().transpose(0, 1) @ k.transpose(1, 2)) * 64 ** -0.5
        s = s.masked_fill(~see, float("-inf"))
        p = torch.softmax(torch.cat((s, b.sinks.double().view(-1, 1, 1).expand(-1, n, 1)), -1), -1)[..., :-1]
        want = (p @ v).transpose(0, 1)
        tol = (p @ v.abs()).transpose(0, 1) * 2.0 ** -8 * 1.02 + want.abs() * 2.0 ** -8
        assert torch.all((out[i * n:(i + 1) * n].double() - want).abs() <= tol), i


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 16])
def test_steps_against_64_bits(example, cache, window):
    n = len(PARENTS)
    b = example.DraftBlock(5, 37, 4 * 5 + n, PARENTS, cache=cache, window=window, **SIZES)
    g = torch.Generator().manual_seed(3)
    for step in range(5):
        before = b.lengths.tolist()
        held = [tokens(b, i) for i in range(5)]
        q, out = b.attention(torch.randn(5 * n, 256, generator=g).cuda().bfloat16())
        assert b.lengths.tolist() == [x + n for x in before]
        check(b, q, out, window)
        drafts = [[x[before[i]:] for x in tokens(b, i)] for i in range(5)]
        paths = [PATHS[(i + step) % 5] for i in range(5)]
        b.keep(kept_of(paths))
        assert b.lengths.tolist() == [x + len(p) for x, p in zip(before, paths)]
        for i in range(5):
            for now, was, new in zip(tokens(b, i), held[i], drafts[i]):
                assert torch.equal(now, torch.cat((was, new[paths[i]])))
        if step == 2:  # sequences 0 and 3 go on from where 4 and 1 are
            b.fork(torch.tensor([4, 1], device="cuda"), torch.tensor([0, 3], device="cuda"))
            assert b.lengths[0] == b.lengths[4] and b.lengths[3] == b.lengths[1]
            for i, j in ((0, 4), (3, 1)):
                assert all(torch.equal(x, y) for x, y in zip(tokens(b, i), tokens(b, j)))
                full = int(b.lengths[i]) // b.page
                assert torch.equal(b.table[i, :full], b.table[j, :full]) and b.table[i, full] != b.table[j, full]
    assert moe.read_device_status(b.status) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_graphed_steps_equal_eager_steps(example, cache):
    n, kept = len(PARENTS), kept_of(PATHS)
    a, b = (example.DraftBlock(5, 300, 5 * 4 + n, PARENTS, cache=cache, **SIZES) for _ in range(2))
    x = torch.randn(5 * n, 256, device="cuda").bfloat16()
    static, out, graph = b.graphed(x)
    assert b.lengths.tolist() == [300] * 5
    for _ in range(5):
        want = a.step(x)
        a.keep(kept)
        static.copy_(x)
        graph.replay()
        b.keep(kept)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.all(torch.isfinite(want))
        assert torch.equal(a.k, b.k) and torch.equal(a.lengths, b.lengths)
        x = example.norm(want)
    for blk in (a, b):
        assert moe.read_device_status(blk.status) == 0 and moe.read_device_status(blk.moe_ws) == 0


def test_one_draft_is_a_decode_step(example):
    """A step of one draft, kept, against the decode step: the same cache, attention within two roundings of each."""
    a = example.DecodeBlock(5, 37, 8, **SIZES)
    b = example.DraftBlock(5, 37, 8, [-1], **SIZES)
    for _ in range(4):
        x = torch.randn(5, 256, device="cuda").bfloat16()
        (qa, oa), (qb, ob) = a.attention(x), b.attention(x)
        b.keep(torch.zeros(5, 1, dtype=torch.int32, device="cuda"))
        assert torch.equal(qa, qb) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.lengths, b.lengths)
        assert torch.all(torch.isfinite(oa)) and torch.all(torch.isfinite(ob))
        # each rounds probabilities, whose sum is at most 1, and its output, by 2^-8 at most
        tol = 2 * 2.0 ** -8 * (a.v.double().abs().amax() * 1.02 + oa.double().abs())
        assert torch.all((oa.double() - ob.double()).abs() <= tol)


def test_command(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["decode_block.py", "--batch", "3", "--context", "70", "--steps", "2", "--drafts", "6"])
    example.main()
    assert "3 of them kept" in capsys.readouterr().out


# ---------------------------------------------------------------- streams ----
def calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    cache = [normal(400, 2, 16, 64), normal(400, 2, 16, 64)]
    table = torch.arange(400, device="cuda", dtype=torch.int32).view(2, 200)
    lens = torch.tensor([3200, 1500], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 9, 14], dtype=torch.int32, device="cuda")
    kept = torch.tensor([[1, 4, 8], [0, 3, -1]], dtype=torch.int32, device="cuda")
    src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([3, 9], [398, 399]))
    q = normal(14, 8, 64)
    qkv = normal(300, 12, 64)
    pos = torch.arange(600, device="cuda").view(2, 300)
    freq = (1e4 ** -torch.arange(32, device="cuda", dtype=torch.float64).div(32))
    axes = torch.arange(32, device="cuda", dtype=torch.int32) % 2

    def copied(s):
        mine = [c.clone() for c in cache]
        torch.cuda.synchronize()
        moe.copy_pages(*mine, src, dst, stream=s)
        (s or torch.cuda.current_stream()).synchronize()
        return mine[0]

    return {
        "tree_attention": lambda s: moe.tree_attention(q, *cache, table, lens, starts, 0.125, stream=s),
        "compact_drafts": lambda s: moe.compact_drafts(*cache, table, lens, starts, kept, stream=s),
        "rotate_append": lambda s: moe.rotate_append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], pos, pos[0],
                                                     *[c.clone() for c in cache], freq, axes=axes, stream=s),
        "copy_pages": copied,
    }


@pytest.mark.parametrize("name", ["tree_attention", "compact_drafts", "rotate_append"])
def test_dropped_results_are_not_written_over_other_memory(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call(None)
    call(side)  # first use of the stream
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # ~10 ms: the call is still waiting when its result is dropped
    got = call(side)
    shape, dtype = got.shape, got.dtype
    del got
    mine = [torch.full(shape, 7, dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.all(m == 7) for m in mine)
    got = call(side)
    side.synchronize()
    assert torch.equal(got, want)


def test_pages_copied_on_another_stream():
    call = calls()["copy_pages"]
    assert torch.equal(call(None), call(torch.cuda.Stream()))
