"""The operators of a video world model's layer around the packed KV cache, as measurable cases.

A layer step norms and rotates its queries and keys (``norm_rope``), writes the keys and values of
the frames being generated into each branch's pages (``append``), attends over the packed history
that all branches share followed by each branch's own pages (``shared``), and attends to an
encoder's states (``cross``).  ``run`` computes a case either in elementary torch operations, 32 bits
wide (``own`` false), or through the library's entry points (``own`` true).

Sizes follow the layers of ``qwm_synth.CONFIGS``: 12 or 40 heads of 128 channels (or 64), frames of
880, 1560 or 3600 tokens, histories of up to 37440 tokens.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
SCALINGS = ("none", "linear", "ntk", "parts")


# ------------------------------------------------------------------------------- cases
def _rope(name, **kw):
    case = dict(kind="norm_rope", tokens=1, heads=40, kv_heads=40, head_dim=128, rot_dim=128, layout="interleaved",
                axes=1, scaling="none", factor=1.0, norm=True, far=0)
    case.update(kw)
    return dict(case, name=name) if name else case


def _append(name, **kw):
    case = dict(kind="append", branches=8, tokens=880, ragged=True, heads=12, head_dim=128, page=64, held=880,
                rot_dim=128, layout="half", norm=True)
    case.update(kw)
    return dict(case, name=name) if name else case


def _shared(name, **kw):
    case = dict(kind="shared", branches=8, tokens=1, ragged=False, heads=40, group_heads=1, head_dim=128, centroids=256,
                group=32, rank=8, history=37440, frame=1560, own=1560, page=64, causal=False)
    case.update(kw)
    return dict(case, name=name) if name else case


def _cross(name, **kw):
    case = dict(kind="cross", batch=1, tokens=1560, ragged=False, heads=40, kv_heads=40, head_dim=128, states=512,
                short=False, empty=False)
    case.update(kw)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one 480p frame's queries and keys: time, height and width axes, norms on
        _rope("rope frame", tokens=1560, axes=3),
        # one generated token far behind the trained range, frequencies scaled by parts, no norm
        _rope("rope token", tokens=1, heads=12, kv_heads=12, layout="half", scaling="parts", factor=8.0, norm=False,
              far=200000),
        # a whole history's prompt with shared key heads, half of each head rotated
        _rope("rope prompt", tokens=9361, heads=40, kv_heads=8, rot_dim=64, layout="half", scaling="ntk", factor=4.0),
        # eight branches of the small layer append ragged frames behind one earlier frame
        _append("append frames"),
        # one token of each of 64 branches of the 480p layer into small pages
        _append("append tokens", branches=64, tokens=1, ragged=False, heads=40, page=16, held=1559, layout="interleaved"),
        # one query token per branch over the whole 480p history and up to a frame of its own
        _shared("shared tokens", branches=8, tokens=1),
        # four ragged, causal pieces of a small-layer frame over the small layer's history
        _shared("shared pieces", branches=4, tokens=220, ragged=True, heads=12, history=7919, frame=880, own=501, page=16,
                causal=True),
        # two whole frames of the 480p layer generated from one history
        _shared("shared frames", branches=2, tokens=1560),
        # a 480p frame against a padded text encoding of 512 states
        _cross("cross frame"),
        # a few query rows of small heads against short ragged encodings, one of them empty
        _cross("cross rows", batch=5, tokens=7, ragged=True, heads=12, kv_heads=4, head_dim=64, states=77, short=True,
               empty=True),
        # four 720p frames against ragged encodings of image and text states
        _cross("cross frames", batch=4, tokens=3600, ragged=True, states=769, short=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def _query_heads(rng, kv):
    """As many query heads as key heads, or a multiple of them, at most 40."""
    return kv * rng.choice([1, 1] + [g for g in (3, 5) if g * kv <= 40])


def draw(rng):
    kind = rng.choice(("norm_rope", "append", "shared", "cross"))
    d = rng.choice((64, 128, 128))
    if kind == "norm_rope":
        kv = rng.choice((1, 4, 8, 12, 40))
        scaling = rng.choice(SCALINGS)
        return _rope(None, tokens=_spread(rng, 1, 9361), heads=_query_heads(rng, kv), kv_heads=kv, head_dim=d,
                     rot_dim=rng.randrange(2, d // 16 + 1) * 16, layout=rng.choice(("interleaved", "half")),
                     axes=rng.choice((1, 1, 3)), scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 8.0)),
                     norm=rng.random() < 0.7, far=rng.choice((0, 4096, 1000000)))
    if kind == "append":
        b = _spread(rng, 1, 64)
        return _append(None, branches=b, tokens=_spread(rng, 1, max(1, 7040 // b)), ragged=rng.random() < 0.5,
                       heads=rng.choice((1, 4, 12)), head_dim=d, page=rng.choice((16, 32, 64, 128, 256)), held=_spread(rng, 1, 1560),
                       rot_dim=rng.randrange(0, d // 16 + 1) * 16, layout=rng.choice(("interleaved", "half")),
                       norm=rng.random() < 0.5)
    if kind == "shared":
        b, h, g = _spread(rng, 1, 64), rng.choice((1, 4, 12, 40)), rng.choice((1, 1, 2))
        group = rng.choice((16, 32))
        t = _spread(rng, 1, 37440)
        # at most the rows of the largest listed case
        return _shared(None, branches=b, tokens=_spread(rng, 1, max(1, min(1560, 1560 * 2 // (b * g)))), ragged=rng.random() < 0.5,
                       heads=h, group_heads=g, head_dim=d, centroids=rng.choice((16, 256, 512)), group=group,
                       rank=rng.choice((0, 4, 8, 16)), history=t, frame=rng.choice((880, 1560)),
                       own=_spread(rng, 1, 1560), page=rng.choice((16, 64, 128)), causal=rng.random() < 0.4)
    kv = rng.choice((1, 4, 12, 40))
    b = _spread(rng, 1, 32)
    return _cross(None, batch=b, tokens=_spread(rng, 1, max(1, min(3600, 14400 // b))), ragged=rng.random() < 0.5,
                  heads=_query_heads(rng, kv), kv_heads=kv, head_dim=d, states=_spread(rng, 1, 769),
                  short=rng.random() < 0.5, empty=rng.random() < 0.2)


# ------------------------------------------------------------------------------- lengths
def _lengths(n, most, ragged, step=37):
    """n lengths of at most `most` (the first is `most`); ragged ones fall and return in uneven steps."""
    return [max(1, most - (step * i * i + 11 * i) % most) if ragged else most for i in range(n)]


def _offsets(lengths):
    return [sum(lengths[:i]) for i in range(len(lengths) + 1)]


def _state_lengths(case):
    lens = _lengths(case["batch"], case["states"], case["short"], 29)
    return [0 if case["empty"] and i == case["batch"] // 2 and case["batch"] > 1 else n for i, n in enumerate(lens)]


def _own_lengths(case):
    """Keys of each branch, the new tokens among them."""
    q = _lengths(case["branches"], case["tokens"], case["ragged"])
    return [max(a, b) for a, b in zip(q, _lengths(case["branches"], max(case["own"], case["tokens"]), True, 13))]


# ------------------------------------------------------------------------------- work
def work(case):
    k, d = case["kind"], case["head_dim"]
    if k == "norm_rope":
        el = case["tokens"] * (case["heads"] + case["kv_heads"]) * d
        return {"bytes": 4 * el + 4 * case["axes"] * case["tokens"], "flops": 7 * el}
    if k == "append":
        el = sum(_lengths(case["branches"], case["tokens"], case["ragged"])) * case["heads"] * d
        return {"bytes": 8 * el, "flops": 7 * el}
    if k == "shared":
        h, g, r = case["heads"], case["group_heads"], case["rank"]
        q = _lengths(case["branches"], case["tokens"], case["ragged"])
        kv = _own_lengths(case)
        packed = 2 * (d // 4 + 4 * (d // case["group"]) + (1 if case["centroids"] <= 256 else 2)) + r + 2
        pairs = sum(a * case["history"] + (a * b - a * (a - 1) // 2 if case["causal"] else a * b) for a, b in zip(q, kv))
        return {"bytes": h * (packed * case["history"] + 4 * d * sum(kv) + 4 * d * g * sum(q)) + 4 * h * g * sum(q),
                "flops": 4 * d * h * g * pairs}
    q = _lengths(case["batch"], case["tokens"], case["ragged"])
    s = _state_lengths(case)
    return {"bytes": 4 * d * (case["heads"] * sum(q) + case["kv_heads"] * sum(s)) + 4 * case["heads"] * sum(q),
            "flops": 4 * d * case["heads"] * sum(a * b for a, b in zip(q, s))}


# ------------------------------------------------------------------------------- inputs
def _axis_dims(rot_dim, axes):
    """Channels of each position axis: even, the first axis takes what does not divide."""
    each = rot_dim // (2 * axes) * 2
    return [rot_dim - each * (axes - 1)] + [each] * (axes - 1)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _whole(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _rope_arguments(case):
    return dict(head_dim=case["head_dim"], rot_dim=case["rot_dim"], layout=case["layout"], theta=10000.0,
                axis_dims=_axis_dims(case["rot_dim"], case.get("axes", 1)), scaling=case.get("scaling", "none"),
                factor=case.get("factor", 1.0), orig_len=4096, beta_fast=32.0, beta_slow=1.0)


def _pages(gen, case, lengths, filled):
    """A pool of pages in a shuffled order, and the table of each sequence's pages."""
    h, d, p = case["heads"], case["head_dim"], case["page"]
    width = -(-max(lengths) // p)
    n = len(lengths) * width + 3
    table = torch.randperm(n, generator=gen, device="cuda")[: len(lengths) * width].to(torch.int32).view(len(lengths), width)
    # free places of a pool hold what was there before
    make = _normal if filled else (lambda g, *shape: torch.zeros(shape, device="cuda"))
    return make(gen, n, h, p, d).to(BF16), make(gen, n, h, p, d).to(BF16), table.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, d = case["kind"], case["head_dim"]
    s = {"case": case}
    if kind == "norm_rope":
        n, hq, hk = case["tokens"], case["heads"], case["kv_heads"]
        # the fused projection's rows: queries, keys and values side by side
        rows = _normal(gen, n, hq + 2 * hk, d) * (0.5 + torch.rand(1, hq + 2 * hk, d, generator=gen, device="cuda"))
        s["qkv"] = rows.to(BF16)
        s["q"], s["k"] = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk]
        side = max(1, math.isqrt(n))
        at = torch.arange(n, device="cuda")
        grid = [at // (side * 4) + case["far"], at // 4 % side, at % 4] if case["axes"] == 3 else [at + case["far"]]
        s["pos"] = torch.stack(grid).to(torch.int32)
        s["wq"], s["wk"] = ((1 + 0.2 * _normal(gen, d)).to(BF16) if case["norm"] else None for _ in range(2))
    elif kind == "append":
        h, q = case["heads"], _lengths(case["branches"], case["tokens"], case["ragged"])
        held = _lengths(case["branches"], case["held"], True, 53)
        s["K"], s["V"], s["table"] = _pages(gen, case, [a + b for a, b in zip(q, held)], False)
        rows = _normal(gen, sum(q), 2, h, d).to(BF16)
        s["k"], s["v"] = rows[:, 0], rows[:, 1]
        s["cu"], s["start"] = _whole(_offsets(q)), _whole(held)
        s["pos"] = _whole([[b + i for a, b in zip(q, held) for i in range(a)]])
        s["wk"] = (1 + 0.2 * _normal(gen, d)).to(BF16) if case["norm"] else None
    elif kind == "shared":
        q, kv = _lengths(case["branches"], case["tokens"], case["ragged"]), _own_lengths(case)
        s["packed"] = _packed_history(gen, case)
        s["K"], s["V"], s["table"] = _pages(gen, case, kv, True)
        s["q"] = _normal(gen, sum(q), case["heads"] * case["group_heads"], d).to(BF16)
        s["cu"], s["kv"], s["most"], s["most_kv"] = _whole(_offsets(q)), _whole(kv), max(q), max(kv)
    else:
        q, kv = _lengths(case["batch"], case["tokens"], case["ragged"]), _state_lengths(case)
        s["q"] = _normal(gen, sum(q), case["heads"], d).to(BF16)
        # the encoder's projection, padded to the longest: keys and values side by side
        s["kvs"] = _normal(gen, case["batch"], case["states"], 2, case["kv_heads"], d).to(BF16)
        s["cu"], s["kv"], s["most"], s["most_kv"] = _whole(_offsets(q)), _whole(kv), max(q), case["states"]
        s["start"] = _whole([i * case["states"] for i in range(case["batch"])])
    if own:
        s["handle"] = _handle(case, s)
    return s


def _packed_history(gen, case):
    """The packed fields of `history` tokens: codes, group parameters, centroids, coefficients and versions."""
    h, d, c, r, t = case["heads"], case["head_dim"], case["centroids"], case["rank"], case["history"]
    ng = d // case["group"]
    tcap = -(-t // 128) * 128
    frames = -(-t // case["frame"])
    rand = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731
    whole = lambda most, *shape: torch.randint(0, most, shape, generator=gen, device="cuda")  # noqa: E731

    def side():
        step = 0.3 + 0.4 * rand(h, tcap, ng)
        return {"codes": whole(256, h, tcap, d // 4).to(torch.uint8),
                "params": torch.stack([-1.5 * step + 0.1 * rand(h, tcap, ng), step], -1).to(torch.float16),
                "idx": whole(c, h, tcap).to(torch.uint8 if c <= 256 else torch.int16)}

    loud = torch.where(torch.arange(d, device="cuda") % 16 == 5, 4.0, 1.0)
    at = torch.arange(tcap, device="cuda") // case["frame"]
    return {"k": side(), "v": side(), "tcap": tcap, "frames": frames,
            "cent_k": (_normal(gen, 2, h, c, d) * loud).to(BF16), "cent_v": _normal(gen, 2, h, c, d).to(BF16),
            "coef": (whole(255, h, tcap, max(r, 1)) - 127).to(torch.int8)[..., :r].contiguous(),
            "cscale": (0.002 + 0.01 * rand(h, tcap)).to(torch.float16),
            "basis": _normal(gen, frames, h, d, max(r, 1)) / math.sqrt(d),
            "tokver": at.clamp(max=frames - 1).to(torch.int16),
            "centver": (at >= (frames + 1) // 2).to(torch.int16)}


def _handle(case, s):
    """What a program keeps between calls of the library: the rotation, the pages' handle, the restored cache."""
    import bit_kv_cache_23_b200 as lib
    kind = case["kind"]
    if kind == "norm_rope":
        return lib.qwm_rope_init(**_rope_arguments(case))
    if kind == "append":
        return lib.PagedKV(s["K"], s["V"]), (lib.qwm_rope_init(**_rope_arguments(case)) if case["rot_dim"] else None)
    if kind == "shared":
        p = s["packed"]
        cache = lib.QuantKVCache(case["heads"], case["head_dim"], case["centroids"], case["group"], 4, case["rank"],
                                 case["history"], max_versions=p["frames"], max_cent_versions=2)
        fields = {"k_codes": p["k"]["codes"], "k_params": p["k"]["params"], "k_idx": p["k"]["idx"], "k_coef": p["coef"],
                  "k_cscale": p["cscale"], "v_codes": p["v"]["codes"], "v_params": p["v"]["params"], "v_idx": p["v"]["idx"],
                  "cent_k": p["cent_k"], "cent_v": p["cent_v"], "basis": p["basis"], "tokver": p["tokver"],
                  "centver": p["centver"]}
        for name, value in fields.items():
            if value.numel():
                cache.buffers[name][: value.numel() * value.element_size()].copy_(value.reshape(-1).view(torch.uint8))
        cache.c.len, cache.c.has_centroids = case["history"], 1
        cache.c.n_versions, cache.c.cur_version = p["frames"], p["frames"] - 1
        cache.c.n_cent_versions, cache.c.cur_cent_version = 2, 1
        return cache, lib.PagedKV(s["K"], s["V"])
    return lib


# ------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        h = s["handle"]
        if kind == "norm_rope":
            from bit_kv_cache_23_b200 import qwm_norm_rope
            return qwm_norm_rope(h, s["q"], s["k"], s["pos"], s["wq"], s["wk"])
        if kind == "append":
            h[0].append(s["table"], s["cu"], s["start"], s["k"], s["v"], rope=h[1],
                        pos=s["pos"] if h[1] is not None else None, k_weight=s["wk"])
            return s["K"], s["V"]
        if kind == "shared":
            lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
            return h[0].attention_shared(s["q"], s["cu"], s["most"], h[1], s["table"], s["kv"], s["most_kv"],
                                         causal=case["causal"], lse=lse), lse
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        kvs = s["kvs"].flatten(0, 1)
        return h.qwm_cross_attention(s["q"], kvs[:, 0], kvs[:, 1], s["cu"], s["start"], s["kv"], s["most"], s["most_kv"],
                                     lse=lse), lse
    if kind == "norm_rope":
        return tuple(_norm_rope(case, x, w, s["pos"]) for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    if kind == "append":
        b, i = _rows(s["cu"], s["k"].shape[0])
        at = s["start"].long()[b] + i
        page = s["table"][b, at // case["page"]].long()
        s["K"][page, :, at % case["page"]] = _norm_rope(case, s["k"], s["wk"], s["pos"])
        s["V"][page, :, at % case["page"]] = s["v"]
        return s["K"], s["V"]
    return _shared_plain(case, s) if kind == "shared" else _cross_plain(case, s)


def _rows(cu, n):
    """The sequence of each of n rows, and the row's place in it."""
    at = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), at, right=True)
    return b, at - cu.long()[b]


def _frequencies(case):
    """64-bit angle per position of each pair, the axis of each pair, and the factor of cos and sin."""
    a = _rope_arguments(case)
    s = a["factor"]
    dims = torch.tensor(a["axis_dims"], dtype=torch.float64, device="cuda")
    axis = torch.repeat_interleave(torch.arange(len(a["axis_dims"]), device="cuda"), (dims / 2).long())
    first = torch.cumsum(dims / 2, 0) - dims / 2
    i, dim = torch.arange(len(axis), device="cuda") - first[axis], dims[axis]
    theta = a["theta"] * s ** (dim / (dim - 2)) if a["scaling"] == "ntk" else torch.full_like(dim, a["theta"])
    f, by = theta ** (-2 * i / dim), 1.0
    if a["scaling"] == "linear":
        f = f / s
    if a["scaling"] == "parts":
        turns = a["orig_len"] * f / (2 * math.pi)
        keep = ((turns - a["beta_slow"]) / (a["beta_fast"] - a["beta_slow"])).clamp(0, 1)
        f, by = keep * f + (1 - keep) * f / s, 0.1 * math.log(s) + 1
    return f, axis, by


def _norm_rope(case, x, w, pos):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    rot = case["rot_dim"]
    if rot == 0:
        return x.to(BF16)
    f, axis, by = _frequencies(case)
    angle = pos.double()[axis].T * f
    cos, sin = ((t * by).float()[:, None] for t in (angle.cos(), angle.sin()))
    head, rest = x[..., :rot], x[..., rot:]
    if case["layout"] == "half":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([head, rest], -1).to(BF16)


def _unpacked(case, p, side, cent):
    """Centroid plus residual of every cached token, [heads][tokens][channels]."""
    h, t, d = case["heads"], case["history"], case["head_dim"]
    codes = (p[side]["codes"][:, :t, :, None] >> torch.arange(0, 8, 2, device="cuda", dtype=torch.uint8)) & 3
    par = p[side]["params"][:, :t].float()
    deq = par[..., :1] + codes.reshape(h, t, -1, case["group"]).float() * par[..., 1:]
    idx = p[side]["idx"][:, :t].long() & (255 if case["centroids"] <= 256 else 65535)
    return cent[p["centver"][:t].long(), torch.arange(h, device="cuda")[:, None], idx].float() + deq.view(h, t, d)


def _history(case, p):
    """K' and V' as the cache's reconstruction defines them: summed wide, rounded once to bf16."""
    h, t, d, r = case["heads"], case["history"], case["head_dim"], case["rank"]
    k, v = _unpacked(case, p, "k", p["cent_k"]), _unpacked(case, p, "v", p["cent_v"])
    if r:
        # each token's coefficients stand in the columns of its basis version
        c = p["coef"][:, :t].float() * p["cscale"][:, :t, None].float()
        wide = torch.zeros(h, t, p["frames"], r, device="cuda")
        wide[:, torch.arange(t, device="cuda"), p["tokver"][:t].long()] = c
        k = k + wide.view(h, t, -1) @ p["basis"].permute(1, 0, 3, 2).reshape(h, -1, d)
    return k.to(BF16).float(), v.to(BF16).float()


def _shared_plain(case, s):
    h, g, d, b = case["heads"], case["group_heads"], case["head_dim"], case["branches"]
    scale, rows = 1 / math.sqrt(d), s["q"].shape[0]
    kp, vp = _history(case, s["packed"])
    q = s["q"].float().view(rows, h, g, d)
    before = torch.einsum("rhgd,htd->hrgt", q, kp) * scale
    # own keys, gathered page by page into [branch][heads][place][channels]
    n = s["table"].shape[1] * case["page"]
    at = torch.arange(n, device="cuda")
    live = (at < s["kv"][:, None])[:, None, :, None]
    k, v = (torch.where(live, x[s["table"].long()].transpose(1, 2).reshape(b, h, n, d).float(), 0) for x in (s["K"], s["V"]))
    br, i = _rows(s["cu"], rows)
    place = torch.arange(s["most"], device="cuda")
    qp = q[(s["cu"][:-1, None].long() + place).clamp(max=rows - 1)]  # [branch][place][heads][group][channels]
    after = torch.einsum("bqhgd,bhtd->bhqgt", qp, k) * scale
    last = s["kv"].long()[:, None] - 1 + place * 0
    if case["causal"]:
        last = (s["kv"] - (s["cu"][1:] - s["cu"][:-1])).long()[:, None] + place
    seen = (at <= torch.minimum(last, s["kv"].long()[:, None] - 1)[..., None])[:, None, :, None]
    after = after.masked_fill(~seen, -math.inf)
    top = torch.maximum(before.amax(-1), after.amax(-1)[br, :, i].transpose(0, 1))  # [heads][rows][group]
    top_own = torch.full(after.shape[:-1], 0.0, device="cuda")
    top_own[br, :, i] = top.transpose(0, 1)
    before, after = before.sub_(top[..., None]).exp_(), after.sub_(top_own[..., None]).exp_()
    total = before.sum(-1) + after.sum(-1)[br, :, i].transpose(0, 1)
    out = torch.einsum("hrgt,htd->hrgd", before, vp)
    out = out + torch.einsum("bhqgt,bhtd->bhqgd", after, v)[br, :, i].transpose(0, 1)
    out = (out / total[..., None]).transpose(0, 1).reshape(rows, h * g, d)
    return out.to(BF16), (top + total.log()).transpose(0, 1).reshape(rows, h * g)


def _cross_plain(case, s):
    b, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]
    rows, g = s["q"].shape[0], case["heads"] // case["kv_heads"]
    br, i = _rows(s["cu"], rows)
    place = torch.arange(s["most"], device="cuda")
    live = (torch.arange(case["states"], device="cuda") < s["kv"][:, None])
    k, v = (torch.where(live[..., None, None], s["kvs"][:, :, j].float(), 0) for j in (0, 1))
    q = s["q"].float().view(rows, hk, g, d)[(s["cu"][:-1, None].long() + place).clamp(max=rows - 1)]
    x = torch.einsum("bqhgd,bthd->bhqgt", q, k) / math.sqrt(d)
    x = x.masked_fill(~live[:, None, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x = (x - top).exp()
    total = x.sum(-1, keepdim=True)
    out = torch.einsum("bhqgt,bthd->bhqgd", x, v) / torch.where(total > 0, total, 1)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    return out[br, :, i].reshape(rows, h, d).to(BF16), lse[br, :, i].reshape(rows, h)


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits, one head (or sequence) at a time."""
    s = prepare(case, seed)
    kind, d = case["kind"], case["head_dim"]
    f64 = torch.float64

    def turned(x, w):
        y = x.to(f64)
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-6) * w.to(f64)
        a, pair = _rope_arguments(case), 0
        for axis, dim in enumerate(a["axis_dims"]):
            for i in range(dim // 2):
                theta = a["theta"]
                if a["scaling"] == "ntk":
                    theta *= a["factor"] ** (dim / (dim - 2))
                f, by = math.pow(theta, -2.0 * i / dim), 1.0
                if a["scaling"] == "linear":
                    f /= a["factor"]
                if a["scaling"] == "parts":
                    t = a["orig_len"] * f / (2 * math.pi)
                    keep = min(1.0, max(0.0, (t - a["beta_slow"]) / (a["beta_fast"] - a["beta_slow"])))
                    f, by = f * (keep + (1 - keep) / a["factor"]), 1 + math.log(a["factor"]) / 10
                at = s["pos"][axis].to(f64)[:, None] * f
                m, n = (pair, pair + case["rot_dim"] // 2) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)
                u, v = y[..., m].clone(), y[..., n].clone()
                y[..., m] = by * (u * torch.cos(at) - v * torch.sin(at))
                y[..., n] = by * (u * torch.sin(at) + v * torch.cos(at))
                pair += 1
        return y

    def attend(q, k, v, hidden=None):
        x = q @ k.T / math.sqrt(d)
        if hidden is not None:
            x[hidden] = -math.inf
        lse = torch.logsumexp(x, -1)
        return torch.exp(x - lse[:, None]) @ v, lse

    if kind == "norm_rope":
        return turned(s["q"], s["wq"]), turned(s["k"], s["wk"])
    if kind == "append":
        k, v, cu, p = s["K"].to(f64), s["V"].to(f64), s["cu"].tolist(), case["page"]
        new, start = turned(s["k"], s["wk"]), s["start"].tolist()
        for b in range(case["branches"]):
            at = torch.arange(cu[b + 1] - cu[b], device="cuda") + start[b]
            page = s["table"][b].long()[torch.div(at, p, rounding_mode="floor")]
            k[page, :, at % p], v[page, :, at % p] = new[cu[b]:cu[b + 1]], s["v"][cu[b]:cu[b + 1]].to(f64)
        return k, v
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=f64, device="cuda")
    if kind == "cross":
        g = case["heads"] // case["kv_heads"]
        for b in range(case["batch"]):
            for h in range(case["heads"] if kv[b] else 0):
                k, v = (s["kvs"][b, : kv[b], j, h // g].to(f64) for j in (0, 1))
                out[cu[b]:cu[b + 1], h], lse[cu[b]:cu[b + 1], h] = attend(s["q"][cu[b]:cu[b + 1], h].to(f64), k, v)
        return out, lse
    p, t, g = s["packed"], case["history"], case["group_heads"]
    ver, cver = p["tokver"][:t].long(), p["centver"][:t].long()
    for h in range(case["heads"]):
        full = []
        for side, cent in (("k", p["cent_k"]), ("v", p["cent_v"])):
            byte = p[side]["codes"][h, :t].long()
            code = torch.stack([byte // 4 ** j % 4 for j in range(4)], -1).view(t, d).to(f64)
            mn, sc = (p[side]["params"][h, :t, :, j].to(f64).repeat_interleave(case["group"], 1) for j in (0, 1))
            idx = p[side]["idx"][h, :t].long() % (256 if case["centroids"] <= 256 else 65536)
            x = cent[cver, h, idx].to(f64) + mn + code * sc
            for j in range(case["rank"] if side == "k" else 0):
                x += p["basis"][ver, h, :, j].to(f64) * (p["coef"][h, :t, j].to(f64) * p["cscale"][h, :t].to(f64))[:, None]
            full.append(x.to(BF16).to(f64))  # the cache is read as bf16
        for b in range(case["branches"]):
            pages = s["table"][b].long()
            k, v = (x[pages, h].reshape(-1, d)[: kv[b]].to(f64) for x in (s["K"], s["V"]))
            k, v = torch.cat([full[0], k]), torch.cat([full[1], v])
            hidden = None
            if case["causal"]:
                n = cu[b + 1] - cu[b]
                hidden = torch.arange(t + kv[b], device="cuda") > t + kv[b] - n + torch.arange(n, device="cuda")[:, None]
            for j in range(h * g, h * g + g):
                out[cu[b]:cu[b + 1], j], lse[cu[b]:cu[b + 1], j] = attend(s["q"][cu[b]:cu[b + 1], j].to(f64), k, v, hidden)
    return out, lse
