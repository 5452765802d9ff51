"""Measured cases of the decoder-block operators that stand before the expert GEMMs.

route_experts    expert choice from router logits: softmax or sigmoid scores, balance bias, groups, top-k
rotate_append    rotation of q and k by position, keys and values appended to a paged cache (16-bit or e4m3)
paged_attention  attention of one new token per sequence over that cache: grouped heads, sinks, window

`run` computes an operator in its plain torch form, or, where `own` is set, with the package's kernels;
`exact` computes it from its definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases ----
def _route(T, E, k, dtype, score, bias, groups, top_groups, group_top, renormalize, scale):
    return dict(op="route", T=T, E=E, k=k, dtype=dtype, score=score, bias=bias, groups=groups, top_groups=top_groups,
                group_top=group_top, renormalize=renormalize, scale=scale)


def _append(N, Hq, Hkv, D, rot, page, dtype, cache, interleaved, rope_scale, first, nhd):
    return dict(op="append", N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rot, page=page, dtype=dtype, cache=cache,
                interleaved=interleaved, rope_scale=rope_scale, first=first, nhd=nhd)


def _attend(B, Hq, Hkv, D, shortest, longest, page, dtype, cache, sinks, window, nhd):
    return dict(op="attend", B=B, Hq=Hq, Hkv=Hkv, D=D, shortest=shortest, longest=longest, page=page, dtype=dtype,
                cache=cache, sinks=sinks, window=window, nhd=nhd)


def listed():
    return [
        # one generated token through a 32-expert layer: latency
        dict(name="route_one_token", **_route(1, 32, 4, "bf16", "softmax", False, 1, 1, 1, True, 1.0)),
        # a decode batch through a 128-expert layer, logits kept in 32 bits
        dict(name="route_decode_256", **_route(256, 128, 4, "fp32", "softmax", False, 1, 1, 1, True, 1.0)),
        # a prompt chunk, 256 experts in 8 groups, sigmoid scores with a balance bias
        dict(name="route_chunk_grouped", **_route(16384, 256, 8, "fp32", "sigmoid", True, 8, 4, 2, True, 2.5)),
        # an odd chunk of an odd expert count, weights left as scores over all experts
        dict(name="route_odd_softmax", **_route(3001, 160, 6, "bf16", "softmax", False, 8, 3, 1, False, 16.0)),
        # one new token of one sequence: latency
        dict(name="append_one_token", **_append(1, 64, 8, 64, 64, 16, "bf16", "bf16", False, 1.3465735902799727, 999, False)),
        # a decode batch, one token of each sequence
        dict(name="append_decode_256", **_append(256, 64, 8, 64, 64, 16, "bf16", "bf16", False, 1.3465735902799727, 70000, False)),
        # a prompt chunk into an e4m3 cache, four key-value heads
        dict(name="append_chunk_e4m3", **_append(8192, 64, 4, 128, 128, 64, "bf16", "e4m3", False, 1.0, 0, False)),
        # an odd chunk: half of each head rotated in neighbouring pairs, pages of 24, tokens-major pages
        dict(name="append_odd_partial", **_append(777, 20, 4, 96, 48, 24, "fp16", "fp16", True, 1.0, 5, True)),
        # one short sequence: latency
        dict(name="attend_one_short", **_attend(1, 64, 8, 64, 90, 90, 16, "bf16", "bf16", True, 0, False)),
        # a decode batch of very different lengths, with sinks
        dict(name="attend_ragged_64", **_attend(64, 64, 8, 64, 1, 16384, 16, "bf16", "bf16", True, 0, False)),
        # the same batch's sliding-window layers
        dict(name="attend_window_256", **_attend(256, 64, 8, 64, 200, 8192, 16, "bf16", "bf16", True, 128, False)),
        # a few very long sequences in an e4m3 cache, 16 heads to a key
        dict(name="attend_long_e4m3", **_attend(4, 64, 4, 128, 100000, 131072, 64, "bf16", "e4m3", False, 0, False)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "append", "attend"])
    if op == "route":
        T = _log(rng, 1, 16384)
        k = rng.randint(1, 8)
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, -(-8 // groups)), 256 // groups)
        top_groups = rng.randint(min(groups, -(-k * groups // E)), groups)
        score = rng.choice(["softmax", "sigmoid"])
        return _route(T, E, k, rng.choice(["bf16", "fp16", "fp32"]), score, rng.random() < 0.5, groups, top_groups,
                      rng.choice([1, 2]), rng.random() < 0.6, rng.choice([1.0, 2.5]))
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16] if Hkv <= 4 else [1, 2, 4, 5, 8])
    D = rng.choice([64, 64, 80, 96, 128, 128])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, "e4m3"])
    nhd = rng.random() < 0.3
    if op == "append":
        rot = 16 * rng.randint(1, D // 16)
        return _append(_log(rng, 1, 8192), Hq, Hkv, D, rot, page, dtype, cache, rng.random() < 0.4,
                       rng.choice([1.0, 1.25]), _log(rng, 1, 500000) - 1, nhd)
    longest = _log(rng, 1, 131072)
    # at most the key-value bytes of the largest listed case
    per = longest * Hkv * D * 2 * (1 if cache == "e4m3" else 2)
    B = _log(rng, 1, max(1, min(256, 4 * 131072 * 4 * 128 * 2 // per)))
    shortest = rng.choice([0, 1, longest, rng.randint(0, longest)])
    window = rng.choice([0, 0, 0, 100, 128, 1000])
    return _attend(B, Hq, Hkv, D, shortest, longest, page, dtype, cache, rng.random() < 0.5, window, nhd)


# ------------------------------------------------------------------ inputs ----
def _inv_freq(rot):
    return 150000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _pages(num_pages, c, values):
    """A cache tensor [pages, heads, page, D]: heads-major in memory, or a view of tokens-major pages."""
    if c["nhd"]:
        return values(num_pages, c["page"], c["Hkv"]).transpose(1, 2)
    return values(num_pages, c["Hkv"], c["page"])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    if c["op"] == "route":
        # logits of a trained router: spread of about 1.5; the balance bias moves scores by a few hundredths
        s = dict(c, logits=(1.5 * normal(c["T"], c["E"])).to(DTYPES[c["dtype"]]), bias=None)
        if c["bias"]:
            s["bias"] = 0.05 * normal(c["E"])
        return s

    dt = DTYPES[c["dtype"]]
    e4m3 = c["cache"] == "e4m3"
    D, Hq, Hkv, page = c["D"], c["Hq"], c["Hkv"], c["page"]

    def cache_of(num_pages):
        """16-bit values, or e4m3 codes with their scales (absolute maximum of a token's head = 448 codes)."""
        if not e4m3:
            return _pages(num_pages, c, lambda *s: normal(*s, D, dtype=dt)), None
        v = _pages(num_pages, c, lambda *s: normal(*s, D, dtype=torch.bfloat16))
        sc = (v.abs().amax(-1).float() / 448.0).contiguous()
        return (v / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), sc

    if c["op"] == "append":
        N = c["N"]
        # q, k, v are views of one fused projection; a few tokens of the batch are padding (slot -1)
        qkv = normal(N, Hq + 2 * Hkv, D).to(dt)
        num_pages = -(-N // page) + 3
        order = torch.randperm(num_pages, generator=h)
        spot = torch.arange(N) + 1  # the first slot of the first page is taken
        slots = order[spot // page] * page + spot % page
        if N > 8:
            slots[torch.randint(0, N, (N // 64 + 1,), generator=h)] = -1
        positions = c["first"] + torch.arange(N)
        kc, ks = cache_of(num_pages)
        vc, vs = cache_of(num_pages)
        return dict(c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], positions=positions.cuda(),
                    slots=slots.cuda(), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, inv_freq=_inv_freq(c["rot"]).cuda())

    B = c["B"]
    lengths = torch.randint(c["shortest"], c["longest"] + 1, (B,), generator=h, dtype=torch.int32)
    lengths[int(torch.randint(0, B, (1,), generator=h))] = c["longest"]
    counts = (lengths.long() + page - 1) // page
    num_pages = int(counts.sum()) + 1
    order = torch.randperm(num_pages, generator=h).int()
    # page ids in random order; entries past a sequence's last page are not set
    width = max(1, int(counts.max()))
    at = torch.arange(width)
    table = torch.where(at < counts[:, None], order[torch.clamp((counts.cumsum(0) - counts)[:, None] + at, max=num_pages - 1)], -1)
    kc, ks = cache_of(num_pages)
    vc, vs = cache_of(num_pages)
    return dict(c, q=(2.0 * normal(B, Hq, D)).to(dt), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                page_table=table.int().cuda(), lengths=lengths.cuda(), sinks=normal(Hq) if c["sinks"] else None)


# --------------------------------------------------------------------- run ----
def run(state):
    s = state
    if s["op"] == "route":
        return _run_route(s)
    return _run_append(s) if s["op"] == "append" else _run_attend(s)


def _run_route(s):
    if own:
        import sparse_moe_layer_gb300 as moe
        idx, w = moe.route_experts(s["logits"], s["k"], score=s["score"], bias=s["bias"], groups=s["groups"],
                                   top_groups=s["top_groups"], group_top=s["group_top"], renormalize=s["renormalize"],
                                   scale=s["scale"])
        return {"idx": idx, "w": w}
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    lg = s["logits"].double()  # choices next to a border are made in 64 bits
    score = torch.softmax(lg, -1) if s["score"] == "softmax" else torch.sigmoid(lg)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        part = choice.view(T, G, E // G)
        best = part.topk(s["group_top"], -1).values.sum(-1) if E // G >= s["group_top"] else part.sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :s["top_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=lg.device).scatter_(1, kept, True)
        choice = part.masked_fill(~open_[..., None], -math.inf).view(T, E)
    idx = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :k].sort(dim=-1).values
    w = score.gather(1, idx).float()
    if s["renormalize"]:
        w = w / (w.sum(-1, keepdim=True) + 1e-20)
    return {"idx": idx.int(), "w": w * s["scale"]}


def _append_outputs(s, q):
    """Rotated q and the updated cache; e4m3 codes as the type whose values they stand for."""
    if s["k_scale"] is None:
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"q": q, "k_cache": s["k_cache"].view(torch.float8_e4m3fn), "v_cache": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _run_append(s):
    if own:
        import sparse_moe_layer_gb300 as moe
        q = moe.rotate_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                              s["inv_freq"], k_scale=s["k_scale"], v_scale=s["v_scale"], interleaved=s["interleaved"],
                              rope_scale=s["rope_scale"])
        return _append_outputs(s, q)
    rot, page = s["rot"], s["page"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]  # far positions: angles in 64 bits
    cos = (angle.cos() * s["rope_scale"]).float()[:, None]
    sin = (angle.sin() * s["rope_scale"]).float()[:, None]

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
            sc = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
            cache[to, :, at] = (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[to, :, at] = sc

    append(rotate(s["k"]), s["k_cache"], s["k_scale"])
    append(s["v"].float(), s["v_cache"], s["v_scale"])
    return _append_outputs(s, rotate(s["q"]).to(s["q"].dtype))


def _run_attend(s):
    D, Hq, Hkv, B, page = s["D"], s["Hq"], s["Hkv"], s["B"], s["page"]
    if own:
        import sparse_moe_layer_gb300 as moe
        return moe.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], D ** -0.5,
                                   k_scale=s["k_scale"], v_scale=s["v_scale"], sinks=s["sinks"], window=s["window"])
    n = s["lengths"].long()[:, None]
    span = s["page_table"].shape[1] * page
    if s["window"] > 0:  # only the window's positions
        span = min(span, s["window"])
        t = (n - span).clamp(min=0) + torch.arange(span, device="cuda")
    else:
        t = torch.arange(span, device="cuda").expand(B, -1)
    seen = t < n
    pages = s["page_table"].long().gather(1, torch.where(seen, t // page, torch.zeros_like(t))).clamp(min=0)

    def gather(cache, scale):
        x = cache if scale is None else cache.view(torch.float8_e4m3fn)
        x = x[pages, :, t % page].float()  # [B, L, Hkv, D]
        if scale is not None:
            x = x * scale[pages, :, t % page][..., None]
        return x.masked_fill(~seen[..., None, None], 0.0).transpose(1, 2)

    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    sc = (q @ gather(s["k_cache"], s["k_scale"]).transpose(-1, -2)) * D ** -0.5
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    sink = None
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, Hq // Hkv, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    z = p.sum(-1, keepdim=True)
    if sink is not None:
        z = z + torch.exp(sink - m)
    o = (p @ gather(s["v_cache"], s["v_scale"])) / torch.where(z == 0, torch.ones_like(z), z)
    return o.view(B, Hq, D).to(s["q"].dtype)


# ------------------------------------------------------------------- bytes ----
def work(case):
    c = case
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        return {"bytes": T * E * (4 if c["dtype"] == "fp32" else 2) + 4 * E * c["bias"] + 8 * T * c["k"],
                "flops": 5 * T * E}
    one = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
        return {"bytes": N * (2 * (2 * Hq + 2 * Hkv) * D + 2 * Hkv * D * one + 16 + (8 * Hkv if one == 1 else 0)) + 4 * c["rot"],
                "flops": 3 * N * (Hq + Hkv) * c["rot"]}
    # lengths are uniform between the shortest and the longest; one is the longest
    mean = _mean_seen(c)
    tokens = mean * (c["B"] - 1) + min(c["longest"], c["window"] or c["longest"])
    return {"bytes": tokens * c["Hkv"] * 2 * (c["D"] * one + (4 if one == 1 else 0)) + 4 * c["B"] * c["Hq"] * c["D"]
            + 4 * tokens / c["page"],
            "flops": 4 * tokens * c["Hq"] * c["D"]}


def _mean_seen(c):
    """Mean of min(length, window) for a length uniform over [shortest, longest]."""
    a, b, w = c["shortest"], c["longest"], c["window"] or c["longest"]
    if w >= b:
        return (a + b) / 2
    if w <= a:
        return float(w)
    low = (w - a) * (a + w - 1) / 2  # the sum of the lengths below the window
    return (low + (b - w + 1) * w) / (b - a + 1)


# ------------------------------------------------------------------- exact ----
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        # rank by counting: an expert is chosen if fewer than k stand before it
        x = s["logits"].to(torch.float64)
        if c["score"] == "softmax":
            e = torch.exp(x - x.max(1, keepdim=True).values)
            p = e / e.sum(1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-x))
        v = p + (s["bias"].to(torch.float64) if s["bias"] is not None else 0.0)
        T, E, k, G = c["T"], c["E"], c["k"], c["groups"]

        def before(a):
            """[rows, n] -> how many entries of the row stand before each."""
            n = a.shape[1]
            out = torch.zeros(a.shape, dtype=torch.int64, device=a.device)
            for j in range(n):
                one = a[:, j:j + 1]
                out += (one > a) | ((one == a) & (j < torch.arange(n, device=a.device)))
            return out

        if G > 1:
            members = v.reshape(T, G, E // G)
            rank = before(members.reshape(T * G, E // G)).reshape(members.shape)
            total = (members * (rank < c["group_top"])).sum(2)
            good = before(total) < c["top_groups"]
            v = torch.where(good.repeat_interleave(E // G, 1), v, torch.full_like(v, -math.inf))
        chosen = before(v) < k
        idx = chosen.nonzero()[:, 1].reshape(T, k)
        w = p[chosen].reshape(T, k)
        if c["renormalize"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return {"idx": idx.to(torch.int32), "w": w * c["scale"]}

    D, page, Hkv = c["D"], c["page"], c["Hkv"]
    if c["op"] == "append":
        rot = c["rot"]
        phase = torch.outer(s["positions"].to(torch.float64), s["inv_freq"])
        turn = torch.polar(torch.full_like(phase, c["rope_scale"]), phase)[:, None, :]
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
        pg, off = dest[keep] // page, dest[keep] % page
        for name, x in (("k", turned(s["k"])), ("v", s["v"].to(torch.float64))):
            x = x[keep.cuda()]
            old, sc = s[name + "_cache"], s[name + "_scale"]
            if sc is None:
                new = old.to(torch.float64)
                new[pg.cuda(), :, off.cuda()] = x
            else:
                new = None  # the codes are what the rounding makes of the values
                sc = sc.to(torch.float64)
                top = x.abs().max(-1).values
                sc[pg.cuda(), :, off.cuda()] = torch.where(top == 0, 1.0, top / 448.0)
                got[name + "_scale"] = sc
            got[name + "_cache"] = new
        return got

    out = torch.zeros(c["B"], c["Hq"], D, dtype=torch.float64, device="cuda")
    group = c["Hq"] // Hkv
    lengths, table = s["lengths"].tolist(), s["page_table"].cpu()
    for b, n in enumerate(lengths):
        start = max(0, n - c["window"]) if c["window"] > 0 else 0
        if n <= 0:
            continue
        t = torch.arange(start, n)
        pg, off = table[b, t // page].long().cuda(), (t % page).cuda()
        kv = []
        for name in ("k", "v"):
            x = s[name + "_cache"]
            if c["cache"] == "e4m3":
                x = x.view(torch.float8_e4m3fn)[pg, :, off].to(torch.float64)
                x = x * s[name + "_scale"][pg, :, off].to(torch.float64)[..., None]
            else:
                x = x[pg, :, off].to(torch.float64)
            kv.append(x.permute(1, 0, 2))  # [Hkv, tokens, D]
        a = torch.bmm(s["q"][b].to(torch.float64).reshape(Hkv, group, D), kv[0].transpose(1, 2)) / math.sqrt(D)
        if s["sinks"] is not None:
            a = torch.cat((a, s["sinks"].to(torch.float64).reshape(Hkv, group, 1)), 2)
        p = torch.softmax(a, 2)[..., :n - start]
        out[b] = torch.bmm(p, kv[1]).reshape(c["Hq"], D)
    return out
