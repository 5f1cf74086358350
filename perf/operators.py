"""Cases for the operators around the attention of a serving step, with their plain forms.

  norm_rope  the rows of one QKV projection -> position-rotated, normalised
             queries and keys and the values, head by head
             (``gqa.qk_norm_rope``)
  tree       a tree of drafted tokens attends over a cache and over its own
             ancestors (``gqa.decode_tree``)
  commit     the accepted path of that tree enters the cache
             (``gqa.tree_commit``)
  scored     the last rows of a sequence attend over the cache, and what each
             cell was given is added up (``gqa.decode_scored``)
  evict      the cells that were given least leave the cache
             (``gqa.cache_evict``)

``run`` computes them in elementary float32 torch operations (float64 for
rotation angles) where ``own`` is false, and calls the library where it is
true.  ``exact`` states the same results in float64, apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = {"op": op, "dtype": "bf16"}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One generated token for each of 8 running sequences: latency counts.
        _case("norm_rope step B8", "norm_rope", B=8, T=1, Hq=32, Hkv=8, d=128, rot=128,
              norm=True, axes=1, cyclic=False, interleaved=False, far=8000, theta=1e6),
        # A batch of odd-length image and text prompts, three position axes.
        _case("norm_rope 3 axes T1021 f32", "norm_rope", dtype="f32", B=4, T=1021, Hq=8, Hkv=2, d=64, rot=64,
              norm=True, axes=3, cyclic=False, interleaved=False, far=1021, theta=1e4),
        # One long prompt before its prefill.
        _case("norm_rope prompt T32768", "norm_rope", B=1, T=32768, Hq=32, Hkv=8, d=128, rot=128,
              norm=True, axes=1, cyclic=False, interleaved=False, far=0, theta=1e6),
        # A single conversation verifying a small draft: latency counts.
        _case("tree B1 n1000 t8", "tree", B=1, Hq=8, Hkv=2, d=64, C=1088, lo=1000, hi=1000,
              t=8, pad=0, window=-1),
        # A batch of ordinary trees over caches of about 8000 cells.
        _case("tree B8 n8000 t26", "tree", B=8, Hq=32, Hkv=8, d=128, C=8064, lo=7900, hi=8000,
              t=26, pad=3, window=-1),
        # Many sequences of all lengths that share one KV head, wide trees.
        _case("tree MQA ragged t63", "tree", B=64, Hq=8, Hkv=1, d=128, C=8256, lo=1, hi=8192,
              t=63, pad=9, window=-1),
        # The accepted tokens of those trees enter the cache.
        _case("commit B8 t26", "commit", B=8, Hkv=8, d=128, C=192, lo=20, hi=180, t=26, P=6),
        _case("commit B64 t63", "commit", B=64, Hkv=8, d=128, C=320, lo=1, hi=300, t=63, P=12),
        # A decode step that keeps account of which cells are still looked at.
        _case("scored B8 n8000", "scored", B=8, Hq=32, Hkv=8, d=128, C=8064, lo=8001, hi=8001, t=1),
        # The last 32 rows of a long prompt look back over all of it.
        _case("scored n32768 t32", "scored", B=1, Hq=32, Hkv=8, d=128, C=32768, lo=32768, hi=32768,
              t=32),
        # Running sequences fall back to half their cells.
        _case("evict B8 8000 to 4096", "evict", B=8, Hkv=8, d=128, C=8064, lo=7900, hi=8001,
              budget=4096, recent=512),
        # A long prompt's cache shrinks into a small one.
        _case("evict 32768 to 4096", "evict", B=1, Hkv=8, d=128, C=32768, lo=32768, hi=32768,
              budget=4096, recent=256),
    ]


def _log(rng, lo, hi):
    """A whole number from [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "tree", "tree", "commit", "scored", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128]) if rng.random() < 0.8 else rng.choice([32, 80, 96, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    small = dtype == "f32" or d not in (64, 128)  # these cost more for the same sizes
    if op == "norm_rope":
        B = _log(rng, 1, 16)
        T = _log(rng, 1, max(1, min(32768, (1 << 26) // (B * (Hq + 2 * Hkv) * d))))
        rot = d if rng.random() < 0.7 else d // 2
        axes = rng.choice([1, 1, 3])
        return _case(None, op, dtype=dtype, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, rot=rot,
                     norm=rng.random() < 0.8, axes=axes, cyclic=axes > 1 and rng.random() < 0.5,
                     interleaved=rng.random() < 0.4, far=_log(rng, 1, 1000000),
                     theta=rng.choice([1e4, 1e6]))
    if op == "commit":
        t = _log(rng, 1, 128)
        P = _log(rng, 1, min(t, 16))
        hi = _log(rng, 1, 500)
        return _case(None, op, dtype=dtype, B=_log(rng, 1, 64), Hkv=Hkv, d=d, C=hi + P, lo=rng.randint(0, hi),
                     hi=hi, t=t, P=P)
    if op == "tree":
        t = _log(rng, 1, 64 if small else 128)
        B = _log(rng, 1, 4 if small else 32)
        most = max(64, min(2000 if small else 32768, (1 << 31) // (B * Hq * t * 64)))
        hi = _log(rng, 16, most)
        return _case(None, op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, d=d, C=hi + t, lo=rng.randint(0, hi), hi=hi,
                     t=t, pad=rng.randint(0, t // 4), window=-1 if rng.random() < 0.7 else _log(rng, 1, hi))
    if op == "scored":
        t = rng.choice([1, 1, _log(rng, 2, 32)])
        B = _log(rng, 1, 4 if small else 32)
        hi = t + _log(rng, 16, max(64, min(2000 if small else 32768, (1 << 30) // (B * Hq * t * 64))))
        return _case(None, op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, d=d, C=hi + rng.randint(0, 70),
                     lo=rng.randint(t, hi), hi=hi, t=t)
    B = _log(rng, 1, 32)
    hi = _log(rng, 16, max(64, min(32768, (1 << 26) // (B * Hkv * d))))
    budget = _log(rng, 1, hi)
    return _case(None, op, dtype=dtype, B=B, Hkv=Hkv, d=d, C=hi + rng.randint(0, 70), lo=rng.randint(0, hi),
                 hi=hi, budget=budget, recent=rng.randint(0, budget))


def _lengths(c):
    """Lengths over [lo, hi], the same for every seed; the longest is hi."""
    lo, hi = c["lo"], c["hi"]
    return [hi - int((hi - lo) * ((0.6180339887 * b) % 1.0)) for b in range(c["B"])]


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm_rope":
        x = c["B"] * c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        return {"bytes": 2 * x * e + 4 * c["axes"] * c["B"] * c["T"], "flops": 8 * x}
    lens = _lengths(c)
    lane = c["Hkv"] * c["d"]  # values of K (or V) in one cell
    if c["op"] == "commit":
        rows = sum(_accepted(c))
        return {"bytes": 4 * rows * lane * e + 4 * c["B"] * (c["P"] + 3), "flops": 0}
    if c["op"] == "evict":
        kept = sum(min(n, c["budget"]) for n in lens)
        return {"bytes": 4 * kept * lane * e + c["Hkv"] * 4 * (sum(lens) + 2 * kept), "flops": 0}
    rows = c["B"] * c["Hq"] * c["t"] * c["d"]
    if c["op"] == "tree":
        w = c["window"]
        cells = [n if w < 0 else min(n, w - 1) for n in lens]
        read = sum(n if w < 0 else min(n, w + c["t"]) for n in lens) + c["B"] * c["t"]
        return {"bytes": (2 * rows + 2 * read * lane) * e + 4 * c["B"] * c["t"],
                "flops": 4 * c["Hq"] * c["d"] * c["t"] * (sum(cells) + c["B"])}
    return {"bytes": (2 * rows + 2 * sum(lens) * lane) * e + 8 * c["Hkv"] * sum(lens),
            "flops": 4 * c["Hq"] * c["d"] * c["t"] * sum(lens)}


# ------------------------------------------------------------------ inputs
def _accepted(c):
    """Accepted tokens of each sequence (at least the root)."""
    return [1 + (7 * b + 2) % c["P"] for b in range(c["B"])]


def _trees(B, t, pad, gen):
    """Parents of B trees of t nodes in drafting order: -1 a root, -2 padding
    behind a tree of fewer nodes."""
    u = torch.rand(B, t, generator=gen)
    i = torch.arange(t)
    lo = torch.clamp(torch.div(i, 4, rounding_mode="floor") - 2, min=-1)
    par = torch.clamp(lo + (u * (i - lo)).long(), max=i - 1)
    par[:, 0] = -1
    for b in range(B):
        k = (b * 5) % (pad + 1)
        if k:
            par[b, t - k:] = -2
    return par.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    gc = torch.Generator()
    gc.manual_seed(int(seed) + 1)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    B, d = c["B"], c["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dt)

    s = {"case": c}
    if c["op"] == "norm_rope":
        T, H = c["T"], c["Hq"] + 2 * c["Hkv"]
        s["qkv"] = normal(B, T, H * d)
        s["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt) if c["norm"] else None
        s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt) if c["norm"] else None
        half = c["rot"] // 2
        s["inv_freq"] = (float(c["theta"]) ** (-torch.arange(half, dtype=torch.float64) / half)).to(
            device=DEV, dtype=torch.float32)
        start = torch.randint(0, c["far"] + 1, (c["axes"], B, 1), generator=g, device=DEV)
        step = torch.arange(T, device=DEV).expand(c["axes"], B, T)
        if c["axes"] > 1:  # frames, rows and columns of a picture 32 wide
            k = torch.arange(T, device=DEV)
            step = torch.stack([k // 1024, (k // 32) % 32, k % 32])[:, None].expand(3, B, T)
        s["pos"] = (start + step).to(torch.int32).contiguous()
        if c["cyclic"]:
            ax = [i % c["axes"] for i in range(half)]
        else:
            ax = [min(c["axes"] - 1, (i * (c["axes"] + 1)) // max(1, half)) for i in range(half)]
        s["axes"] = ax
        s["axis_of"] = torch.tensor(ax, device=DEV)
        s["q"] = torch.empty(B, c["Hq"], T, d, device=DEV, dtype=dt)
        s["k"] = torch.empty(B, c["Hkv"], T, d, device=DEV, dtype=dt)
        s["v"] = torch.empty(B, c["Hkv"], T, d, device=DEV, dtype=dt)
        return s

    Hkv, C = c["Hkv"], c["C"]
    s["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
    s["kc"], s["vc"] = normal(B, Hkv, C, d), normal(B, Hkv, C, d)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if c["op"] in ("tree", "scored"):
        s["q"] = normal(B, c["Hq"], c["t"], d)
        s["o"] = torch.empty_like(s["q"])
    if c["op"] in ("tree", "commit"):
        s["kd"], s["vd"] = normal(B, Hkv, c["t"], d), normal(B, Hkv, c["t"], d)
    if c["op"] == "tree":
        s["parents"] = _trees(B, c["t"], c["pad"], gc).to(DEV)
    elif c["op"] == "commit":
        acc = _accepted(c)
        path = torch.full((B, c["P"]), -1, dtype=torch.int32)
        for b in range(B):
            path[b, :acc[b]] = torch.randperm(c["t"], generator=gc)[:acc[b]].sort().values.to(torch.int32)
        s["path"] = path.to(DEV)
        s["acc"] = torch.tensor(acc, dtype=torch.int32, device=DEV)
        s["lens_out"] = torch.zeros_like(s["lens"])
    elif c["op"] == "scored":
        s["w"] = torch.zeros(B, Hkv, C, device=DEV)
    elif c["op"] == "evict":
        # accumulated weights: a heavy tail, and cells that never got any
        u = torch.rand(B, Hkv, C, generator=g, device=DEV)
        s["w"] = torch.where(u < 0.05, torch.zeros_like(u), 0.01 * u / (1.0001 - u))
        m = c["budget"]
        s["ko"], s["vo"] = torch.zeros(B, Hkv, m, d, device=DEV, dtype=dt), torch.zeros(B, Hkv, m, d, device=DEV, dtype=dt)
        s["wo"] = torch.zeros(B, Hkv, m, device=DEV)
        s["kept"] = torch.zeros(B, Hkv, m, dtype=torch.int32, device=DEV)
        s["lens_out"] = torch.zeros_like(s["lens"])
    if own and c["op"] in ("tree", "scored"):
        from grouped_query_attention_03_b200 import gqa
        make = gqa.decode_tree_workspace if c["op"] == "tree" else gqa.decode_scored_workspace
        s["ws"] = make(s["q"], s["kc"])
    return s


# -------------------------------------------------------------- plain forms
def _plain_norm_rope(s):
    c = s["case"]
    B, T, Hq, Hkv, d, half = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["rot"] // 2
    x = s["qkv"].view(B, T, Hq + 2 * Hkv, d)
    ang = s["pos"].double()[s["axis_of"]].permute(1, 2, 0) * s["inv_freq"].double()  # [B,T,half]
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]

    def one(y, w):
        y = y.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        a, rest = y[..., :2 * half], y[..., 2 * half:]
        if c["interleaved"]:
            u, v = a[..., 0::2], a[..., 1::2]
            a = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
        else:
            u, v = a[..., :half], a[..., half:]
            a = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
        return torch.cat([a, rest], -1).transpose(1, 2).contiguous().to(x.dtype)

    return {"q": one(x[:, :, :Hq], s["qw"]), "k": one(x[:, :, Hq:Hq + Hkv], s["kw"]),
            "v": x[:, :, Hq + Hkv:].transpose(1, 2).contiguous()}


def _attend(s, permitted, k, v):
    """softmax(scale q k^T) over the permitted keys, and its mix of v; rows
    that may read nothing are zero.  permitted [B,1,t,keys]."""
    c = s["case"]
    B, Hq, Hkv, t, d = c["B"], c["Hq"], c["Hkv"], c["t"], c["d"]
    q = s["q"].float().view(B, Hkv, (Hq // Hkv) * t, d)
    x = (q @ k.float().transpose(-1, -2) * d ** -0.5).view(B, Hkv, Hq // Hkv, t, -1)
    x = x.masked_fill(~permitted[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = (p.view(B, Hkv, -1, p.shape[-1]) @ v.float()).view(B, Hq, t, d)
    return o.to(s["q"].dtype), p


def _plain_tree(s):
    c = s["case"]
    t, w = c["t"], c["window"]
    par = s["parents"].long()
    seen = torch.eye(t, device=DEV).expand(c["B"], t, t)
    up = (par[:, :, None] == torch.arange(t, device=DEV)).float()
    for _ in range(max(1, t - 1).bit_length()):  # ancestors up to 2^k steps above
        seen = ((seen + up @ seen) > 0).float()
        up = up @ up
    live = par > -2
    depth = seen.sum(-1) - 1
    anc = (seen > 0) & live[:, :, None]
    n = s["lens"].long()[:, None, None]
    cell = torch.arange(c["C"], device=DEV)[None, None]
    old = ((cell < n) & live[:, :, None]).expand(-1, t, -1)
    if w > 0:
        at = n + depth[:, :, None]
        old = old & (cell > at - w)
        anc = anc & (depth[:, None, :] > depth[:, :, None] - w)
    permitted = torch.cat([old, anc], -1)[:, None]
    k, v = torch.cat([s["kc"], s["kd"]], 2), torch.cat([s["vc"], s["vd"]], 2)
    return {"o": _attend(s, permitted, k, v)[0]}


def _plain_commit(s):
    c = s["case"]
    j = torch.arange(c["P"], device=DEV)
    use = (j[None] < s["acc"][:, None])[:, None, :, None]
    shape = (c["B"], c["Hkv"], c["P"], c["d"])
    src = s["path"].long().clamp(min=0)[:, None, :, None].expand(shape)
    dst = (s["lens"].long()[:, None] + j)[:, None, :, None].expand(shape)
    for cache, new in ((s["kc"], s["kd"]), (s["vc"], s["vd"])):
        cache.scatter_(2, dst, torch.where(use, new.gather(2, src), cache.gather(2, dst)))
    s["lens_out"].copy_(s["lens"] + s["acc"])
    return {"k": s["kc"], "v": s["vc"], "lens": s["lens_out"]}


def _plain_scored(s):
    c = s["case"]
    n = s["lens"].long()[:, None, None]
    at = n - c["t"] + torch.arange(c["t"], device=DEV)[None, :, None]
    permitted = (torch.arange(c["C"], device=DEV)[None, None] <= at)[:, None]
    o, p = _attend(s, permitted, s["kc"], s["vc"])
    s["w"] += p.sum((2, 3))
    return {"o": o, "w": s["w"]}


def _plain_evict(s):
    c = s["case"]
    m = c["budget"]
    n = s["lens"].long()[:, None, None]
    cell = torch.arange(c["C"], device=DEV)[None, None]
    x = torch.where(cell >= n - c["recent"], math.inf, s["w"].double())
    x = torch.where(cell >= n, -math.inf, x)
    best = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :m]
    i = torch.arange(m, device=DEV)[None, None]
    best = torch.where(i < n, best, c["C"]).sort(-1).values
    use = i < torch.clamp(n, max=m)
    src = best.clamp(max=c["C"] - 1)
    rows = src[..., None].expand(-1, -1, -1, c["d"])
    for out, cache in ((s["ko"], s["kc"]), (s["vo"], s["vc"])):
        out.copy_(torch.where(use[..., None], cache.gather(2, rows), out))
    s["wo"].copy_(torch.where(use, s["w"].gather(2, src), 0.0))
    s["kept"].copy_(torch.where(use, src, -1))
    s["lens_out"].copy_(torch.clamp(s["lens"], max=m))
    return {"k": s["ko"], "v": s["vo"], "w": s["wo"], "kept": s["kept"], "lens": s["lens_out"]}


# ------------------------------------------------------------ library calls
def _own(s):
    from grouped_query_attention_03_b200 import gqa
    c = s["case"]
    if c["op"] == "norm_rope":
        q, k, v = gqa.qk_norm_rope(s["qkv"], c["Hq"], c["Hkv"], c["d"], q_weight=s["qw"], k_weight=s["kw"],
                                   inv_freq=s["inv_freq"], positions=s["pos"], axes=s["axes"],
                                   interleaved=c["interleaved"], eps=EPS, out=(s["q"], s["k"], s["v"]))
        return {"q": q, "k": k, "v": v}
    if c["op"] == "tree":
        o = gqa.decode_tree(s["q"], s["kc"], s["vc"], s["kd"], s["vd"], s["parents"], s["lens"],
                            window=None if c["window"] < 0 else c["window"], out=s["o"],
                            workspace=s["ws"], status=s["status"])
        return {"o": o}
    if c["op"] == "commit":
        gqa.tree_commit(s["kc"], s["vc"], s["kd"], s["vd"], s["path"], s["acc"], s["lens"],
                        lens_out=s["lens_out"], status=s["status"])
        return {"k": s["kc"], "v": s["vc"], "lens": s["lens_out"]}
    if c["op"] == "scored":
        o = gqa.decode_scored(s["q"], s["kc"], s["vc"], s["w"], s["lens"], out=s["o"],
                              workspace=s["ws"], status=s["status"])
        return {"o": o, "w": s["w"]}
    gqa.cache_evict(s["kc"], s["vc"], s["w"], s["lens"], c["budget"], c["recent"], kept=s["kept"],
                    k_out=s["ko"], v_out=s["vo"], weights_out=s["wo"], lens_out=s["lens_out"],
                    status=s["status"])
    return {"k": s["ko"], "v": s["vo"], "w": s["wo"], "kept": s["kept"], "lens": s["lens_out"]}


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "tree": _plain_tree, "commit": _plain_commit,
            "scored": _plain_scored, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exactly
def exact(case, seed):
    """The definitions in float64, one sequence (and head) at a time.  What is
    only moved or counted has no computed value: None."""
    c = case
    if c["op"] in ("commit", "evict"):
        return None
    s = prepare(c, seed)
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    r = Hq // Hkv
    if c["op"] == "norm_rope":
        T, half = c["T"], c["rot"] // 2
        x = s["qkv"].view(B, T, Hq + 2 * Hkv, d)
        out = {"q": torch.empty(B, Hq, T, d, device=DEV, dtype=torch.float64),
               "k": torch.empty(B, Hkv, T, d, device=DEV, dtype=torch.float64), "v": None}
        first = [2 * i if c["interleaved"] else i for i in range(half)]
        second = [2 * i + 1 if c["interleaved"] else half + i for i in range(half)]
        turn = torch.stack([s["pos"][a] for a in s["axes"]], -1).double() * s["inv_freq"].double()
        for h in range(Hq + Hkv):
            y = x[:, :, h].double()
            w = s["qw"] if h < Hq else s["kw"]
            if w is not None:
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + EPS) * w.double()
            z = torch.polar(torch.ones_like(turn), turn) * torch.complex(y[..., first], y[..., second])
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            if h < Hq:
                out["q"][:, h] = y
            else:
                out["k"][:, h - Hq] = y
        return out
    t = c["t"]
    o = torch.zeros(B, Hq, t, d, device=DEV, dtype=torch.float64)
    w = torch.zeros(B, Hkv, c["C"], device=DEV, dtype=torch.float64)
    lens = _lengths(c)
    par = s["parents"].tolist() if c["op"] == "tree" else None
    for b in range(B):
        n = lens[b]
        if c["op"] == "tree":
            bias = torch.full((t, n + t), -math.inf, dtype=torch.float64)
            for i in range(t):
                if par[b][i] == -2:
                    continue
                line, a = [], i
                while a >= 0:
                    line.append(a)
                    a = par[b][a]
                reach = len(line) if c["window"] < 0 else c["window"]  # cells that count
                for a in line[:reach]:
                    bias[i, n + a] = 0
                lo = 0 if c["window"] < 0 else max(0, n + len(line) - c["window"])
                bias[i, lo:n] = 0
            bias = bias.to(DEV)
            k = torch.cat([s["kc"][b, :, :n], s["kd"][b]], 1)
            v = torch.cat([s["vc"][b, :, :n], s["vd"][b]], 1)
        else:
            row = torch.arange(t, device=DEV)[:, None] + n - t
            bias = torch.where(torch.arange(n, device=DEV)[None] <= row, 0.0, -math.inf).double()
            k, v = s["kc"][b, :, :n], s["vc"][b, :, :n]
        for h in range(Hq):
            x = s["q"][b, h].double() @ k[h // r].double().T / math.sqrt(d) + bias
            p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
            o[b, h] = p @ v[h // r].double()
            if c["op"] == "scored":
                w[b, h // r, :n] += p.sum(0)
    return {"o": o} if c["op"] == "tree" else {"o": o, "w": w}
