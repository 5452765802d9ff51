"""Forks of a draft block's sequences (DraftBlock.fork of examples/decode_block.py), one after another: no sequence
writes on a page that another one names.  On the CPU the page table and the copies alone; on the GPU with steps."""
import importlib.util
import os
import random

import pytest
import torch

import sparse_moe_layer_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("decode_block", os.path.join(ROOT, "examples", "decode_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Sequences:
    """A block's table, lengths and a cache [pages, 1, page, 1] of numbers on the CPU, and what each sequence should hold."""

    def __init__(self, m, lengths, pages, page):
        B = len(lengths)
        b = object.__new__(m.DraftBlock)
        b.B, b.page = B, page
        b.table = torch.arange(B * pages, dtype=torch.int32).view(B, pages)
        b.lengths = torch.zeros(B, dtype=torch.int32)
        b.k, b.v = torch.zeros(B * pages, 1, page, 1), torch.zeros(B * pages, 1, page, 1)
        b.ks = b.vs = b.status = None
        self.b, self.want, self.next = b, [[] for _ in lengths], 1
        for i, n in enumerate(lengths):
            self.append(i, n)

    def append(self, i, n):
        b = self.b
        for t in range(len(self.want[i]), len(self.want[i]) + n):
            b.k[b.table[i, t // b.page], 0, t % b.page] = self.next
            self.want[i].append(self.next)
            self.next += 1
        b.lengths[i] += n

    def fork(self, src, dst):
        self.b.fork(torch.tensor(src), torch.tensor(dst))
        for i, j in zip(src, dst):
            self.want[j] = list(self.want[i])

    def check(self):
        b = self.b
        for i, want in enumerate(self.want):
            assert b.lengths[i] == len(want)
            t = torch.arange(len(want))
            assert b.k[b.table[i, t // b.page].long(), 0, t % b.page, 0].tolist() == want, i
        assert b.table.min() >= 0 and b.table.max() < b.k.shape[0]


def copy_pages(k, v, src, dst, tokens, k_scale=None, v_scale=None, status=None):
    for a, b, n in zip(src.tolist(), dst.tolist(), tokens.tolist()):
        for c in (k, v):
            c[b, :, :n] = c[a, :, :n]


@pytest.fixture
def example(monkeypatch):
    m = load()
    monkeypatch.setattr(m.moe, "copy_pages", copy_pages)
    return m


def test_a_lender_becomes_a_fork(example):
    s = Sequences(example, [16, 44, 20], 8, 8)
    s.fork([1], [0])
    s.check()
    s.fork([2], [1])  # sequence 0 still reads the pages that 1 had
    s.check()
    for i in (1, 0, 2):
        s.append(i, 15)
    s.check()


def test_a_fork_forks_again_from_a_shorter_sequence(example):
    s = Sequences(example, [16, 60, 20], 10, 8)
    s.fork([1], [0])
    s.fork([2], [0])
    s.check()
    for i in (0, 1, 2):
        s.append(i, 13)
    s.check()


@pytest.mark.parametrize("seed", range(20))
def test_forks_at_random(example, seed):
    """Beams: several sequences a call, some from one source, full pages and empty sequences among them."""
    r = random.Random(seed)
    B, pages, page = r.randint(2, 7), r.randint(1, 12), r.choice([1, 4, 8])
    s = Sequences(example, [r.randint(0, pages * page) for _ in range(B)], pages, page)
    for _ in range(30):
        dst = r.sample(range(B), r.randint(1, B - 1))
        src = [r.choice([i for i in range(B) if i not in dst]) for _ in dst]
        s.fork(src, dst)
        s.check()
        for i in range(B):
            n = r.randint(0, min(pages * page - len(s.want[i]), 2 * page))
            s.append(i, n)
            lost = r.randint(0, n)  # as a step's rejected drafts
            s.want[i] = s.want[i][:len(s.want[i]) - lost]
            s.b.lengths[i] -= lost
            s.check()


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_steps_of_forked_sequences_leave_the_others_alone(cache):
    moe.build()
    m = load()
    n, parents = 5, [-1, 0, 0, 1, 3]
    b = m.DraftBlock(4, 37, 60, parents, H=256, I=256, E=8, top_k=2, q_heads=8, kv_heads=2, head_dim=64, page=8, cache=cache)
    paths = [[0, 1, 3, 4], [0], [0, 2], []]

    def held(i):
        t = torch.arange(int(b.lengths[i]), device="cuda")
        pg, off = b.table[i, t // b.page].long(), t % b.page
        return [c[pg, :, off] for c in (b.k, b.v, b.ks, b.vs) if c is not None]

    g = torch.Generator().manual_seed(1)
    for step, (src, dst) in enumerate([([0], [1]), ([2], [0]), ([3, 3], [0, 1]), ([1], [3]), ([0], [2]), ([3, 2], [1, 0])]):
        before = [held(i) for i in range(4)]
        b.fork(torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda"))
        now = list(range(4))
        for i, j in zip(src, dst):
            now[j] = i
        before = [before[now[i]] for i in range(4)]
        b.attention(torch.randn(4 * n, 256, generator=g).cuda().bfloat16())
        kept = [paths[(i + step) % 4] for i in range(4)]
        b.keep(torch.tensor([p + [-1] * (4 - len(p)) for p in kept], dtype=torch.int32, device="cuda"))
        for i in range(4):
            for x, y in zip(held(i), before[i]):
                assert len(x) == len(y) + len(kept[i]) and torch.equal(x[:len(y)], y), (step, i)
    assert moe.read_device_status(b.status) == 0
