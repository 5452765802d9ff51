"""Measured cases of the operators for drafted tokens, forked pages and positions with several axes.

tree_attention   attention of a tree (or a chain) of drafted tokens per sequence over a paged cache
compact_drafts   the drafts that were kept move up in the cache, in all layers at once
copy_pages       pages of all layers copied, whole or their first places: forks and moves
rotate_append    rotation by positions with several axes (time, height, width), appended to a paged cache

`run` computes an operator in its plain torch form, or, where `own` is set, with the package's kernels;
`exact` computes it from its definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases ----
def _tree(B, fewest, most, shortest, longest, Hq, Hkv, D, page, dtype, cache, sinks, window, chain, nhd):
    return dict(op="tree", B=B, fewest=fewest, most=most, shortest=shortest, longest=longest, Hq=Hq, Hkv=Hkv, D=D,
                page=page, dtype=dtype, cache=cache, sinks=sinks, window=window, chain=chain, nhd=nhd)


def _compact(B, drafts, keep, L, Hkv, D, page, cache, nhd):
    return dict(op="compact", B=B, drafts=drafts, keep=keep, L=L, Hkv=Hkv, D=D, page=page, cache=cache, nhd=nhd)


def _copy(N, partial, L, Hkv, D, page, cache, nhd):
    return dict(op="copy", N=N, partial=partial, L=L, Hkv=Hkv, D=D, page=page, cache=cache, nhd=nhd)


def _axes(N, Hq, Hkv, D, rot, page, dtype, cache, interleaved, sections, frame, nhd):
    return dict(op="axes", N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rot, page=page, dtype=dtype, cache=cache, interleaved=interleaved,
                sections=sections, frame=frame, nhd=nhd)


def listed():
    return [
        # one short sequence with a small tree: latency
        dict(name="tree_one_short", **_tree(1, 6, 6, 90, 90, 64, 8, 64, 16, "bf16", "bf16", True, 0, False, False)),
        # a batch of very different lengths, a chain of four tokens each, with sinks
        dict(name="tree_chain_64", **_tree(64, 4, 4, 1, 16384, 64, 8, 64, 16, "bf16", "bf16", True, 0, True, False)),
        # sliding-window layers of a large batch, trees of up to eight
        dict(name="tree_window_256", **_tree(256, 1, 8, 200, 2000, 64, 8, 64, 16, "bf16", "bf16", True, 128, False, False)),
        # wide trees: sixty-four drafts of each sequence on eight query heads a key
        dict(name="tree_wide_32", **_tree(32, 48, 64, 2000, 8192, 64, 8, 64, 16, "bf16", "bf16", False, 0, False, False)),
        # a few very long sequences in an e4m3 cache, sixteen heads to a key
        dict(name="tree_long_e4m3", **_tree(4, 16, 16, 100000, 131072, 64, 4, 128, 64, "bf16", "e4m3", False, 0, False, False)),
        # odd: ragged trees, five heads to a key, pages of 24, tokens-major pages
        dict(name="tree_odd_fp16", **_tree(9, 1, 37, 0, 3000, 20, 4, 96, 24, "fp16", "fp16", True, 0, False, True)),
        # one sequence's kept drafts in every layer: latency
        dict(name="compact_one", **_compact(1, 8, 4, 24, 8, 64, 16, "bf16", False)),
        # a batch's kept drafts, e4m3 cache
        dict(name="compact_128_e4m3", **_compact(128, 24, 7, 36, 4, 128, 64, "e4m3", False)),
        # sixty-four sequences forked: the used places of their last pages
        dict(name="copy_fork_64", **_copy(64, True, 24, 8, 64, 16, "bf16", False)),
        # pages moved together after many sequences ended, whole, e4m3 cache
        dict(name="copy_move_256", **_copy(256, False, 36, 4, 128, 64, "e4m3", False)),
        # a video prompt's chunk: time, height and width
        dict(name="axes_chunk_8192", **_axes(8192, 64, 8, 128, 128, 16, "bf16", "bf16", False, "16,24,24", 1024, False)),
        # an odd image: half of each head turned in neighbouring pairs, e4m3 cache
        dict(name="axes_odd_e4m3", **_axes(1025, 20, 4, 96, 48, 24, "fp16", "e4m3", True, "8,8,8", 1025, True)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "compact", "copy", "axes"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 64, 80, 96, 128, 128])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    nhd = rng.random() < 0.3
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, "e4m3"])
    if op == "tree":
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16] if Hkv <= 4 else [1, 2, 4, 5, 8])
        longest = _log(rng, 1, 131072)
        most = _log(rng, 1, 64)
        # at most the keys and values, and the products, of the largest listed cases
        size = longest * Hkv * D * 2 * (1 if cache == "e4m3" else 2)
        flops = 4 * most * Hq * (longest + most) * D
        B = _log(rng, 1, max(1, min(256, 4 * 131072 * 4 * 128 * 2 // size, 32 * 4 * 64 * 64 * 8192 * 64 // flops)))
        shortest = rng.choice([0, 1, longest, rng.randint(0, longest)])
        return _tree(B, rng.choice([0, 1, most, rng.randint(1, most)]), most, shortest, longest, Hq, Hkv, D, page, dtype,
                     cache, rng.random() < 0.5, rng.choice([0, 0, 0, 100, 128, 1000]), rng.random() < 0.3, nhd)
    if op == "axes":
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        rot = 16 * rng.randint(1, D // 16)
        first = rng.randint(0, rot // 2)
        second = rng.randint(0, rot // 2 - first)
        return _axes(_log(rng, 1, 8192), Hq, Hkv, D, rot, page, dtype, cache, rng.random() < 0.4,
                     "%d,%d,%d" % (first, second, rot // 2 - first - second), _log(rng, 1, 4096), nhd)
    L = rng.choice([1, 2, 12, 24, 36])
    # at most the bytes of the largest listed cases
    one = L * Hkv * D * page * 2 * (1 if cache == "e4m3" else 2)
    if op == "compact":
        drafts = _log(rng, 1, 64)
        pages = -(-(50 + drafts) // page) + 1
        B = _log(rng, 1, max(1, min(256, 128 * 2 * 36 * 4 * 128 * 64 * 2 // (one * pages))))
        return _compact(B, drafts, rng.randint(1, min(drafts, 8)), L, Hkv, D, page, cache, nhd)
    N = _log(rng, 1, max(1, min(4096, 256 * 36 * 4 * 128 * 64 * 2 // one)))
    return _copy(N, rng.random() < 0.5, L, Hkv, D, page, cache, nhd)


# ------------------------------------------------------------------ inputs ----
def _caches(c, shape, normal):
    """k and v [*shape, D], shape (layers,) pages, heads, page: 16-bit values, or e4m3 codes with their scales
    (absolute maximum of a token's head = 448 codes); heads-major in memory, or views of tokens-major pages."""
    kv, sc = [], []
    for _ in range(2):
        at = (*shape[:-2], shape[-1], shape[-2]) if c["nhd"] else shape
        x = normal(*at, c["D"], dtype=torch.bfloat16 if c["cache"] == "e4m3" else DTYPES[c["cache"]])
        s = None
        if c["cache"] == "e4m3":
            s = x.abs().amax(-1).float() / 448.0
            x = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        if c["nhd"]:
            x = x.transpose(-3, -2)
            s = None if s is None else s.transpose(-2, -1)
        kv.append(x)
        sc.append(s)
    return dict(k_cache=kv[0], v_cache=kv[1], k_scale=sc[0], v_scale=sc[1])


def _spread(lo, hi, n, h):
    """n numbers spread evenly over [lo, hi], hi among them, in random order."""
    return (hi - (hi - lo) * torch.arange(n) // max(1, n - 1))[torch.randperm(n, generator=h)]


def _table(lengths, page, h, spare=1):
    """Page ids in random order, entries past a sequence's last page -1; and the number of pages."""
    counts = (lengths + page - 1) // page
    num = int(counts.sum()) + spare
    order = torch.randperm(num, generator=h)
    at = torch.arange(max(1, int(counts.max())))
    place = ((counts.cumsum(0) - counts)[:, None] + at).clamp(max=num - 1)
    return torch.where(at < counts[:, None], order[place], -1).int(), num


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    if c["op"] == "tree":
        B = c["B"]
        drafts, context = _spread(c["fewest"], c["most"], B, h), _spread(c["shortest"], c["longest"], B, h)
        lengths = context + drafts  # the drafts' keys and values are in the cache
        starts = torch.cat((torch.zeros(1, dtype=torch.long), drafts.cumsum(0)))
        # the likeliest continuation first, as a chain, then alternatives to any token before them
        i = torch.cat([torch.arange(n) for n in drafts.tolist()])
        parents = torch.where(i < 6, i - 1, (torch.rand(len(i), generator=h) * i).long())
        table, num = _table(lengths, page, h)
        return dict(c, q=(2.0 * normal(len(i), c["Hq"], D)).to(DTYPES[c["dtype"]]), **_caches(c, (num, Hkv, page), normal),
                    page_table=table.cuda(), lengths=lengths.int().cuda(), starts=starts.int().cuda(),
                    parents=None if c["chain"] else parents.int().cuda(), sinks=normal(c["Hq"]) if c["sinks"] else None)
    if c["op"] == "compact":
        B, n, K = c["B"], c["drafts"], c["keep"]
        context = _spread(20, 50, B, h)
        lengths = context + n
        # a prefix of the chain that the first K drafts are, then alternatives in ascending order; -1 ends
        count = torch.randint(1, K + 1, (B,), generator=h)
        prefix = (torch.rand(B, generator=h) * (count + 1)).long().clamp(min=1)
        others = torch.rand(B, n, generator=h).masked_fill(torch.arange(n) < K, 2.0).sort(1).indices[:, :K]
        at = torch.arange(K)
        if n < 2 * K:  # no room for alternatives: the chain is kept
            prefix = count
        kept = torch.where(at < prefix[:, None], at, others)
        kept = torch.where(at < count[:, None], kept, n).sort(1).values
        kept = torch.where(at < count[:, None], kept, -1)
        table, num = _table(lengths, page, h)
        starts = torch.arange(B + 1) * n
        return dict(c, **_caches(c, (c["L"], num, Hkv, page), normal), page_table=table.cuda(), lengths=lengths.int().cuda(),
                    starts=starts.int().cuda(), kept=kept.int().cuda())
    if c["op"] == "copy":
        N = c["N"]
        order = torch.randperm(2 * N + 3, generator=h).int()
        tokens = torch.randint(1, page + 1, (N,), generator=h, dtype=torch.int32).cuda() if c["partial"] else None
        return dict(c, **_caches(c, (c["L"], 2 * N + 3, Hkv, page), normal), src=order[:N].cuda(), dst=order[N:2 * N].cuda(),
                    tokens=tokens)
    # frames of a video: time, and height and width within a frame about as high as wide
    N, Hq, frame = c["N"], c["Hq"], c["frame"]
    qkv = normal(N, Hq + 2 * Hkv, D).to(DTYPES[c["dtype"]])  # q, k, v are views of one fused projection
    n = torch.arange(N)
    wide = max(1, int(math.sqrt(frame)))
    positions = 100 + torch.stack((n // frame, n % frame // wide, n % frame % wide))
    axes = torch.repeat_interleave(torch.arange(3), torch.tensor([int(x) for x in c["sections"].split(",")]))
    num = -(-N // page) + 3
    order = torch.randperm(num, generator=h)
    slots = order[(n + 1) // page] * page + (n + 1) % page  # the first slot of the first page is taken
    if N > 8:
        slots[torch.randint(0, N, (N // 64 + 1,), generator=h)] = -1
    inv_freq = 1e6 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
    return dict(c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], positions=positions.cuda(), slots=slots.cuda(),
                **_caches(c, (num, Hkv, page), normal), inv_freq=inv_freq.cuda(), axes=axes.int().cuda())


# --------------------------------------------------------------------- run ----
def run(state):
    return {"tree": _run_tree, "compact": _run_compact, "copy": _run_copy, "axes": _run_axes}[state["op"]](state)


def _run_tree(s):
    D, Hq, Hkv, B, page = s["D"], s["Hq"], s["Hkv"], s["B"], s["page"]
    if own:
        import sparse_moe_layer_gb300 as moe
        return moe.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], s["starts"], D ** -0.5,
                                  parents=s["parents"], k_scale=s["k_scale"], v_scale=s["v_scale"], sinks=s["sinks"],
                                  window=s["window"])
    n, most, G = s["q"].shape[0], s["most"], Hq // Hkv
    starts, length = s["starts"].long(), s["lengths"].long()
    drafts = starts[1:] - starts[:-1]
    first = length - drafts
    i = torch.arange(most, device="cuda")
    real = i < drafts[:, None]
    row = (starts[:-1, None] + i).clamp(max=n - 1)
    # ancestors: (1 - P)^-1, with P the matrix of parents
    parent = i - 1 if s["parents"] is None else torch.where(real, s["parents"].long()[row], -1)
    up = (parent.expand(B, -1)[..., None] == i).float()
    eye = torch.eye(most, device="cuda").expand(B, -1, -1)
    above = torch.linalg.solve_triangular(eye - up, eye, upper=False, unitriangular=True)
    depth = above.sum(-1).long() - 1
    near = depth[..., None] - depth[:, None] < (s["window"] or 1 << 30)
    above = (above > 0.5) & near & real[..., None] & real[:, None]
    # the tokens that any draft of a sequence can see
    span = s["page_table"].shape[1] * page
    if s["window"] > 0:
        span = min(span, s["window"] - 1 + most)
    t = (length[:, None] - span).clamp(min=0) + torch.arange(span, device="cuda")
    there = t < length[:, None]
    pages = s["page_table"].long().gather(1, torch.where(there, t // page, 0)).clamp(min=0)

    def gather(cache, scale):
        x = cache if scale is None else cache.view(torch.float8_e4m3fn)
        x = x[pages, :, t % page].float()  # [B, span, Hkv, D]
        if scale is not None:
            x = x * scale[pages, :, t % page][..., None]
        return x.masked_fill(~there[..., None, None], 0.0).transpose(1, 2)

    j = (t - first[:, None]).clamp(0, most - 1)
    seen = above.gather(2, j[:, None].expand(-1, most, -1))
    past = t[:, None] < first[:, None, None]
    if s["window"] > 0:
        past = past & (t[:, None] > (first[:, None] + depth)[..., None] - s["window"])
    seen = torch.where(t[:, None] < first[:, None, None], past, seen) & (there[:, None] & real[..., None])  # [B, most, span]
    q = s["q"].float()[row].view(B, most, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, most * G, D)
    sc = ((q @ gather(s["k_cache"], s["k_scale"]).transpose(-1, -2)) * D ** -0.5).view(B, Hkv, most, G, span)
    sc = sc.masked_fill(~seen[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    sink = None
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, 1, G, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m)
    z = p.sum(-1, keepdim=True)
    if sink is not None:
        z = z + torch.exp(sink - m)
    o = (p.view(B, Hkv, most * G, span) @ gather(s["v_cache"], s["v_scale"])).view(B, Hkv, most, G, D) / torch.where(z == 0, 1.0, z)
    return o.permute(0, 2, 1, 3, 4).reshape(B, most, Hq, D)[real].to(s["q"].dtype)


def _outputs(s, **more):
    """The updated cache; e4m3 codes as the type whose values they stand for."""
    if s["k_scale"] is None:
        return dict(more, k_cache=s["k_cache"], v_cache=s["v_cache"])
    return dict(more, k_cache=s["k_cache"].view(torch.float8_e4m3fn), v_cache=s["v_cache"].view(torch.float8_e4m3fn),
                k_scale=s["k_scale"], v_scale=s["v_scale"])


def _run_compact(s):
    if own:
        import sparse_moe_layer_gb300 as moe
        lengths = moe.compact_drafts(s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], s["starts"], s["kept"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return _outputs(s, lengths=lengths)
    page, kept = s["page"], s["kept"].long()
    first = s["lengths"].long() - (s["starts"][1:] - s["starts"][:-1])
    live = kept >= 0
    old = first[:, None] + kept.clamp(min=0)
    new = first[:, None] + torch.arange(kept.shape[1], device="cuda")
    table = s["page_table"].long()
    src, dst = table.gather(1, old // page)[live], table.gather(1, torch.where(live, new // page, 0))[live]
    at, to = (old % page)[live], (new % page)[live]

    def move(cache, scale):
        cache[:, dst, :, to] = cache[:, src, :, at]
        if scale is not None:
            scale[:, dst, :, to] = scale[:, src, :, at]

    move(s["k_cache"], s["k_scale"])
    move(s["v_cache"], s["v_scale"])
    return _outputs(s, lengths=(first + live.sum(1)).int())


def _run_copy(s):
    if own:
        import sparse_moe_layer_gb300 as moe
        moe.copy_pages(s["k_cache"], s["v_cache"], s["src"], s["dst"], tokens=s["tokens"], k_scale=s["k_scale"],
                       v_scale=s["v_scale"])
        return _outputs(s)
    src, dst = s["src"].long(), s["dst"].long()
    at = None
    if s["tokens"] is not None:
        used = torch.arange(s["page"], device="cuda") < s["tokens"][:, None]
        src, dst = (x[:, None].expand_as(used)[used] for x in (src, dst))
        at = torch.arange(s["page"], device="cuda").expand_as(used)[used]

    def copy(x):
        if at is None:
            x[:, dst] = x[:, src]
        else:
            x[:, dst, :, at] = x[:, src, :, at]

    copy(s["k_cache"])
    copy(s["v_cache"])
    if s["k_scale"] is not None:
        copy(s["k_scale"])
        copy(s["v_scale"])
    return _outputs(s)


def _run_axes(s):
    if own:
        import sparse_moe_layer_gb300 as moe
        q = moe.rotate_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"], s["inv_freq"],
                              k_scale=s["k_scale"], v_scale=s["v_scale"], interleaved=s["interleaved"], axes=s["axes"])
        return _outputs(s, q=q)
    rot, page = s["rot"], s["page"]
    angle = s["positions"].double()[s["axes"].long()].t() * s["inv_freq"]  # far positions: angles in 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x):
        x = x.float()
        r = x[..., :rot]
        if s["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((y, x[..., rot:]), -1)

    live = s["slots"] >= 0
    to, at = s["slots"][live] // page, s["slots"][live] % page

    def append(x, cache, scale):
        x = x[live]
        if scale is None:
            cache[to, :, at] = x.to(cache.dtype)
        else:
            amax = x.abs().amax(-1)
            sc = torch.where(amax == 0, 1.0, amax / 448.0)
            cache[to, :, at] = (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[to, :, at] = sc

    append(rotate(s["k"]), s["k_cache"], s["k_scale"])
    append(s["v"].float(), s["v_cache"], s["v_scale"])
    return _outputs(s, q=rotate(s["q"]).to(s["q"].dtype))


# ------------------------------------------------------------------- bytes ----
def work(case):
    c = case
    one = 1 if c["cache"] == "e4m3" else 2
    token = 2 * c["Hkv"] * (c["D"] * one + (4 if one == 1 else 0))  # bytes of its keys and values in a layer
    if c["op"] == "axes":
        N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
        return {"bytes": N * (2 * (2 * Hq + 2 * Hkv) * D + token + 32) + 6 * c["rot"], "flops": 3 * N * (Hq + Hkv) * c["rot"]}
    if c["op"] == "copy":
        return {"bytes": c["N"] * (2 * c["L"] * token * ((c["page"] + 1) / 2 if c["partial"] else c["page"]) + 8), "flops": 0}
    if c["op"] == "compact":
        # the kept tokens that are not in their place yet: of a mean of (K + 1) / 2 kept, about a half
        moved = (c["keep"] + 1) / 4 if c["drafts"] >= 2 * c["keep"] else 0
        return {"bytes": c["B"] * (2 * c["L"] * token * moved + 4 * c["keep"] + 16), "flops": 0}
    # contexts and numbers of drafts are spread evenly between their bounds
    B = c["B"]
    drafts = B * (c["fewest"] + c["most"]) / 2 if B > 1 else c["most"]
    seen = B * _mean_seen(c) if B > 1 else min(c["longest"], c["window"] or c["longest"])
    products = drafts * (seen / B + 1)  # the drafts' own ancestors are a few more
    return {"bytes": (seen + drafts) * (token + 4 / c["page"]) + 4 * drafts * c["Hq"] * c["D"],
            "flops": 4 * products * c["Hq"] * c["D"]}


def _mean_seen(c):
    """Mean of min(context, window) for a context uniform over [shortest, longest]."""
    a, b, w = c["shortest"], c["longest"], c["window"] or c["longest"]
    if w >= b:
        return (a + b) / 2
    if w <= a:
        return float(w)
    low = (w - a) * (a + w - 1) / 2  # the sum of the contexts below the window
    return (low + (b - w + 1) * w) / (b - a + 1)


# ------------------------------------------------------------------- exact ----
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    D, page, Hkv = c["D"], c["page"], c["Hkv"]

    def value(name):
        x = s[name + "_cache"]
        return x.view(torch.float8_e4m3fn).to(torch.float64) if c["cache"] == "e4m3" else x.to(torch.float64)

    if c["op"] in ("compact", "copy"):
        # moved places keep their bits: a list of (from page, place, to page, place)
        moves = []
        got = {}
        if c["op"] == "copy":
            count = s["tokens"].tolist() if s["tokens"] is not None else [page] * c["N"]
            for a, b, n in zip(s["src"].tolist(), s["dst"].tolist(), count):
                moves += [(a, o, b, o) for o in range(n)]
        else:
            table, lengths = s["page_table"].tolist(), []
            for row, n, path in zip(table, s["lengths"].tolist(), s["kept"].tolist()):
                path = [p for p in path if p >= 0]
                c0 = n - c["drafts"]
                for to, p in enumerate(path):
                    moves.append((row[(c0 + p) // page], (c0 + p) % page, row[(c0 + to) // page], (c0 + to) % page))
                lengths.append(c0 + len(path))
            got["lengths"] = torch.tensor(lengths, dtype=torch.int32)
        a, o, b, u = (torch.tensor(x, device="cuda") for x in zip(*moves))
        for name in ("k", "v"):
            x = s[name + "_cache"]
            x[:, b, :, u] = x[:, a, :, o].clone()
            got[name + "_cache"] = x.view(torch.float8_e4m3fn) if c["cache"] == "e4m3" else x
            if c["cache"] == "e4m3":
                y = s[name + "_scale"]
                y[:, b, :, u] = y[:, a, :, o].clone()
                got[name + "_scale"] = y
        return got

    if c["op"] == "axes":
        rot = c["rot"]
        which = s["axes"].tolist()
        phase = torch.stack([s["positions"][a].to(torch.float64) * f for a, f in zip(which, s["inv_freq"].tolist())], 1)
        turn = torch.polar(torch.ones_like(phase), phase)[:, None, :]
        first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"]
                         else (slice(0, rot // 2), slice(rot // 2, rot)))

        def turned(x):
            y = x.to(torch.float64).clone()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        got = {"q": turned(s["q"])}
        dest = s["slots"].cpu()
        keep = torch.nonzero(dest >= 0)[:, 0]
        pg, off = (dest[keep] // page).cuda(), (dest[keep] % page).cuda()
        for name, x in (("k", turned(s["k"])), ("v", s["v"].to(torch.float64))):
            x = x[keep.cuda()]
            if c["cache"] == "e4m3":
                got[name + "_cache"] = None  # the codes are what the rounding makes of the values
                sc = s[name + "_scale"].to(torch.float64)
                top = x.abs().max(-1).values
                sc[pg, :, off] = torch.where(top == 0, 1.0, top / 448.0)
                got[name + "_scale"] = sc
            else:
                new = value(name)
                new[pg, :, off] = x
                got[name + "_cache"] = new
        return got

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G = c["Hq"] // Hkv
    starts, lengths, table = s["starts"].tolist(), s["lengths"].tolist(), s["page_table"].cpu()
    parents = None if s["parents"] is None else s["parents"].tolist()
    keys, values = s["k_cache"], s["v_cache"]
    for b, length in enumerate(lengths):
        lo, n = starts[b], starts[b + 1] - starts[b]
        if n == 0:
            continue
        c0 = length - n
        # what each draft sees of the drafts, and from which token on, by walking to the root
        tail = torch.zeros(n, n, dtype=torch.bool)
        since = torch.zeros(n, dtype=torch.long)
        for i in range(n):
            path, j = [], i
            while j >= 0:
                path.append(j)
                j = j - 1 if parents is None else parents[lo + j]
            w = c["window"] or length + 1
            tail[i, path[:w]] = True
            since[i] = max(0, c0 + len(path) - w)
        start = int(since.min())
        t = torch.arange(start, length)
        pg, off = table[b, t // page].long().cuda(), (t % page).cuda()
        kv = []
        for name, x in (("k", keys), ("v", values)):
            x = x[pg, :, off]
            if c["cache"] == "e4m3":
                x = x.view(torch.float8_e4m3fn).to(torch.float64) * s[name + "_scale"][pg, :, off].to(torch.float64)[..., None]
            kv.append(x.to(torch.float64).permute(1, 0, 2))  # [Hkv, tokens, D]
        mask = torch.cat((t[None, :max(0, c0 - start)] >= since[:, None], tail[:, max(0, start - c0):]), 1).cuda()
        q = s["q"][lo:lo + n].to(torch.float64).reshape(n, Hkv, G, D).permute(1, 2, 0, 3)
        for h in range(Hkv):
            a = (q[h].reshape(G * n, D) @ kv[0][h].t()).reshape(G, n, -1) / math.sqrt(D)
            a = torch.where(mask, a, -math.inf)
            if s["sinks"] is not None:
                a = torch.cat((a, s["sinks"][h * G:(h + 1) * G].to(torch.float64)[:, None, None].expand(G, n, 1)), 2)
            p = torch.softmax(a, 2)[..., :len(t)]
            out[lo:lo + n, h * G:(h + 1) * G] = (p.reshape(G * n, -1) @ kv[1][h]).reshape(G, n, D).transpose(0, 1)
    return out
