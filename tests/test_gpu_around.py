"""The operators around the packed cache (norm and rotation, paged append,
attention over a shared history, cross attention) against plain 64-bit forms."""
import math

import pytest
import torch

import bit_kv_cache_23_b200 as q
from around_util import (BF16, F32, HALF, attend, check, check_lse, frequencies, ints, norm_rope, offsets,
                         randn)

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _fine():
    assert q.qwm_device_status() == 0, "a device wait timed out or an index was clamped"


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("d,rot,layout,axes,scaling,factor,norm,n,hq,hk,far", [
    (128, 128, "interleaved", (44, 42, 42), "none", 1.0, True, 33, 5, 5, 0),
    (128, 128, "half", (128,), "parts", 8.0, False, 1, 12, 12, 200000),
    (128, 64, "half", (64,), "ntk", 4.0, True, 67, 8, 2, 1000000),
    (128, 16, "interleaved", (16,), "linear", 2.0, True, 5, 1, 3, 4096),
    (64, 64, "half", (64,), "none", 1.0, True, 130, 3, 1, 2**31 - 200),
    (64, 48, "half", (16, 16, 16), "ntk", 2.0, False, 17, 7, 7, 0),
    (64, 32, "interleaved", (30, 2), "none", 1.0, False, 9, 33, 1, -5),
    (128, 96, "half", (96,), "none", 1.0, True, 4101, 2, 1, 0),      # four tokens per block, ragged
    (128, 128, "interleaved", (128,), "none", 1.0, False, 1026, 1, 1, 0),
    (64, 0, "half", (0,), "none", 1.0, True, 21, 4, 4, 0),           # norm alone
])
def test_norm_rope(d, rot, layout, axes, scaling, factor, norm, n, hq, hk, far):
    g = _gen(d + n)
    rows = (randn(g, n, hq + hk + 1, d) * 3).to(BF16)   # parts of one projection
    Q, K = rows[:, :hq], rows[:, hq:hq + hk]
    wq, wk = ((1 + randn(g, d)).to(BF16) if norm else None for _ in range(2))
    rope = q.qwm_rope_init(d, rot, layout, axis_dims=axes, scaling=scaling, factor=factor) if rot else None
    pos = torch.stack([torch.arange(n, device="cuda") * (i + 1) + far for i in range(len(axes))]).to(torch.int32)
    pos = pos if far < 2**30 else ints([[far + i for i in range(n)]])
    freqs, gain = frequencies(rot, axes, scaling, factor) if rot else (None, 1.0)
    before = rows.clone()
    got = q.qwm_norm_rope(rope, Q, K, pos if rope else None, wq, wk)
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int16), rows.view(torch.int16)), "an input was written"
    for name, x, w, o in (("Q", Q, wq, got[0]), ("K", K, wk, got[1])):
        want, bound = norm_rope(x, w, pos, freqs, gain, rot, layout)
        check(name, o, want, bound)
    # in place, one side alone, and the same bits again
    both = rows.clone()
    q.qwm_norm_rope(rope, both[:, :hq], both[:, hq:hq + hk], pos if rope else None, wq, wk,
                    Q_out=both[:, :hq], K_out=both[:, hq:hq + hk])
    assert torch.equal(both[:, :hq], got[0]) and torch.equal(both[:, hq:hq + hk], got[1])
    assert torch.equal(both[:, hq + hk:], rows[:, hq + hk:])
    alone = q.qwm_norm_rope(rope, None, K, pos if rope else None, None, wk)
    assert alone[0] is None and torch.equal(alone[1], got[1])


def test_norm_rope_edge_values():
    """A row of zeros stays zero under the norm; no rows at all are no work; without rope and weights
    the rows are copied bit for bit, NaN included."""
    g = _gen(3)
    rope = q.qwm_rope_init(64, 64)
    x = randn(g, 3, 2, 64).to(BF16)
    x[1] = 0
    w = torch.ones(64, dtype=BF16, device="cuda")
    out, _ = q.qwm_norm_rope(rope, x, pos=ints([0, 1, 2]), q_weight=w)
    assert torch.equal(out[1], torch.zeros_like(out[1]))
    none, _ = q.qwm_norm_rope(rope, x[:0], pos=ints([]), q_weight=w)
    assert none.shape == (0, 2, 64)
    x[2, 1, 7] = NAN
    same, _ = q.qwm_norm_rope(None, x)
    assert torch.equal(same.view(torch.int16), x.view(torch.int16))


# ------------------------------------------------------------------ pages
def _table(g, lengths, page, spare=2):
    width = max(1, -(-max(lengths) // page))
    n = len(lengths) * width + spare
    perm = torch.randperm(n, generator=g, device="cuda")[: len(lengths) * width]
    return n, perm.to(torch.int32).view(len(lengths), width).contiguous()


@pytest.mark.parametrize("d,h,page,new,held,rot,layout,norm,behind", [
    (128, 3, 16, (5, 1, 40), (0, 15, 9), 128, "half", True, 0),
    (128, 1, 256, (300, 0, 7), (250, 3, 0), 64, "interleaved", False, 3),
    (64, 5, 64, (1, 1, 1, 1), (63, 64, 0, 127), 64, "half", True, 1),
    (64, 2, 128, (0, 0, 2100), (1, 2, 100), 0, "half", False, 0),
])
def test_paged_append(d, h, page, new, held, rot, layout, norm, behind):
    g = _gen(page + d)
    n = sum(new) + behind
    n_pages, table = _table(g, [a + b for a, b in zip(new, held)], page)
    kv = q.PagedKV(randn(g, n_pages, h, page, d).to(BF16), randn(g, n_pages, h, page, d).to(BF16))
    want_k, want_v = kv.K.double(), kv.V.clone()
    rows = randn(g, n, 2, h, d).to(BF16)
    K, V = rows[:, 0], rows[:, 1]
    w = (1 + randn(g, d)).to(BF16) if norm else None
    rope = q.qwm_rope_init(d, rot, layout) if rot else None
    pos = torch.randint(0, 5000, (1, n), generator=g, device="cuda").to(torch.int32) if rot else None
    kv.append(table, ints(offsets(new)), ints(held), K, V, rope, pos, w)
    _fine()
    freqs, gain = frequencies(rot, (rot,), "none", 1.0) if rot else (None, 1.0)
    turned, tol = norm_rope(K, w, pos, freqs, gain, rot, layout)
    if not rot and not norm:
        tol = torch.zeros_like(tol)
    bound = torch.zeros_like(want_k)
    cu = offsets(new)
    for b in range(len(new)):
        for i in range(new[b]):
            p = held[b] + i
            at = int(table[b, p // page])
            want_k[at, :, p % page], bound[at, :, p % page] = turned[cu[b] + i], tol[cu[b] + i]
            want_v[at, :, p % page] = V[cu[b] + i]
    check("K", kv.K, want_k, bound)   # places that no row goes to: bound 0
    assert torch.equal(kv.V, want_v)


def test_paged_append_bad_pages_and_offsets():
    """Page numbers outside the pool and positions outside the table drop their rows, write nothing
    else, and are reported once."""
    g = _gen(9)
    kv = q.PagedKV(randn(g, 4, 2, 16, 64).to(BF16), randn(g, 4, 2, 16, 64).to(BF16))
    before = kv.K.clone(), kv.V.clone()
    K, V = randn(g, 40, 2, 64).to(BF16), randn(g, 40, 2, 64).to(BF16)
    assert q.qwm_device_status() == 0
    for table, cu, start in (([[4, 5]], [0, 20], [0]), ([[-1, 2**31 - 1]], [0, 20], [0]),
                             ([[0, 1]], [0, 40], [32]), ([[0, 1]], [0, 5], [-100])):
        kv.append(ints(table), ints(cu), ints(start), K, V)
        assert q.qwm_device_status() == 2
        assert q.qwm_device_status() == 0
        assert torch.equal(kv.K, before[0]) and torch.equal(kv.V, before[1])
    kv.append(ints([[0, 1]]), ints([50, 60]), ints([0]), K, V)   # every row is before the first sequence
    assert q.qwm_device_status() == 0
    assert torch.equal(kv.K, before[0]) and torch.equal(kv.V, before[1])


# ------------------------------------------------------------------ shared history
def _cache(g, H, d, T, C=16, G=16, r=4, frames=3):
    """A cache of T tokens appended in frames, with a basis version and (from the second on) a table
    version of their own."""
    c = q.QuantKVCache(H, d, C, G, 4, r, max(T, 1), max_versions=frames + 1, max_cent_versions=2)
    cuts = [T * f // frames for f in range(frames + 1)]
    for f in range(frames if T else 0):
        n = cuts[f + 1] - cuts[f]
        K, V = randn(g, max(n, C), H, d).to(BF16), randn(g, max(n, C), H, d).to(BF16)
        if f < 2:
            c.build_centroids(K, V, iters=1)
        c.update_query_stats(randn(g, 16, H, d).to(BF16))
        if n:
            c.append_kv(K[:n].contiguous(), V[:n].contiguous())
    assert c.len == T
    return c


def _shared_case(d, H, g_heads, T, new, own, page, causal, seed, poison=True, C=16, G=16, r=4):
    g = _gen(seed)
    c = _cache(g, H, d, T, C, G, r)
    Kp, Vp = c.reconstruct() if T else (torch.empty(H, 0, d, device="cuda"),) * 2
    n_pages, table = _table(g, own, page)
    K, V = (randn(g, n_pages, H, page, d).to(BF16) for _ in range(2))
    rows = [(K[t.long()].transpose(0, 1).reshape(H, -1, d)[:, :n].clone(),
             V[t.long()].transpose(0, 1).reshape(H, -1, d)[:, :n].clone()) for t, n in zip(table, own)]
    if poison:   # what lies behind a sequence's end, and in pages of no sequence
        used = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
        for t, n in zip(table, own):
            for p in range(n):
                used[int(t[p // page]), p % page] = True
        for x in (K, V):
            x.transpose(1, 2)[~used] = NAN
    n = sum(new) + 2   # two rows of no sequence
    Hq = H * g_heads
    qkv = randn(g, n, Hq + 1, d).to(BF16)
    return c, Kp, Vp, rows, q.PagedKV(K, V), table, qkv[:, :Hq], ints(offsets(new)), ints(own)


def _shared_want(Kp, Vp, rows, Q, new, own, causal, g_heads):
    n, Hq, d = Q.shape
    out = torch.zeros(n, Hq, d, dtype=torch.float64, device="cuda")
    bound, lse = torch.zeros_like(out), torch.zeros(n, Hq, dtype=torch.float64, device="cuda")
    lb = torch.zeros_like(lse)
    cu = offsets(new)
    T = Kp.shape[1]
    for b, (k, v) in enumerate(rows):
        seen = None
        if causal:
            at = torch.arange(T + own[b], device="cuda")
            last = T + own[b] - new[b] + torch.arange(new[b], device="cuda")
            seen = (at <= last[:, None]) | (at < T)
        s = slice(cu[b], cu[b + 1])
        for h in range(Hq):
            kh = h // g_heads
            out[s, h], bound[s, h], lse[s, h], lb[s, h] = attend(
                Q[s, h], torch.cat([Kp[kh], k[kh]]), torch.cat([Vp[kh], v[kh]]), 1 / math.sqrt(d), seen)
    return out, bound, lse, lb


@pytest.mark.parametrize("d,H,gh,T,new,own,page,causal", [
    (128, 2, 1, 300, (1, 1, 1), (1, 130, 64), 16, False),             # single tokens, ragged pages
    (128, 3, 2, 1000, (70, 1, 33), (70, 5, 200), 64, True),           # causal pieces, shared key heads
    (128, 1, 1, 129, (300,), (257,), 128, False),                     # one branch, two row blocks
    (64, 2, 1, 513, (7, 0, 9), (100, 0, 9), 32, True),                # a branch of no rows
    (64, 1, 4, 5, (3, 2), (0, 17), 16, False),                        # a branch of no own keys
    (128, 2, 1, 0, (4, 3), (129, 0), 16, False),                      # no history: empty rows
    (64, 1, 2, 0, (5,), (3,), 256, True),                             # causal rows before the first key
    (128, 1, 1, 2500, (260, 129), (1, 300), 16, True),                # more than one row block, split ranges
    (128, 4, 1, 40, (2,) * 70, (3,) * 70, 16, False),                 # many short branches
    (128, 4, 1, 2000, (1,) * 100, (5, 0, 33, 1) * 25, 16, False),     # the history apart from the branches' keys
    (64, 3, 2, 1500, (2, 0, 1, 3) * 30, (70, 9, 1, 3) * 30, 32, True),
    (128, 2, 2, 57610, (2, 3), (40, 7), 16, True),                    # few rows of shared key heads, long history
    (64, 2, 3, 57605, (1, 0, 1), (0, 5, 130), 32, False),
])
def test_attention_shared(d, H, gh, T, new, own, page, causal):
    c, Kp, Vp, rows, kv, table, Q, cu, lens = _shared_case(d, H, gh, T, new, own, page, causal, 11 + T)
    n, Hq = Q.shape[:2]
    want, bound, wl, lb = _shared_want(Kp, Vp, rows, Q, new, own, causal, gh)
    least, full = q.qwm_attention_shared_workspace(c.c, n, Hq, len(new), max(new), max(own))
    live = sum(new)
    for size in {least, full}:
        O = torch.full((n, Hq, d), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((n, Hq), 5.0, device="cuda")
        ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        got = c.attention_shared(Q, cu, max(new), kv, table, lens, max(own), causal=causal, O=O, lse=lse,
                                 workspace=ws)
        assert got is O
        _fine()
        check("O", O[:live], want[:live], bound[:live])
        check_lse("lse", lse[:live], wl[:live], lb[:live])
        assert (O[live:] == 7.0).all() and (lse[live:] == 5.0).all(), "rows of no sequence were written"


@pytest.mark.parametrize("C,G,r,d,T", [
    (16, 16, 0, 128, 701), (300, 32, 16, 128, 701), (300, 32, 8, 64, 701), (16, 32, 5, 64, 701),
    (4, 16, 8, 128, 9601), (4, 32, 16, 64, 9600), (8, 16, 0, 128, 19001),   # long runs: staged tables
])
def test_shared_history_is_the_reconstruction(C, G, r, d, T):
    """The unpacked history, read back from the workspace, which ends with it (keys, then values), is the
    bf16 cache that the reconstruction returns.  Values, and keys without compensation, are equal bit for
    bit.  The compensation's r products are summed in another order: with S = |c + mn + code sc| + sum |U c8
    cs| each of the two sums is off by at most E = (r + 4) 2^-24 S before its one rounding, so the results
    differ by 2 E and a bf16 step (at most 2^-7 of the larger), and they differ at all only where a border
    between two bf16 values (2^-8 |K'| apart at least) lies within 2 E: for a share 2 E / (2^-8 |K'|) of
    such elements, which is small unless the compensation cancels the rest."""
    c, Kp, Vp, rows, kv, table, Q, cu, lens = _shared_case(d, 2, 1, T, (70,), (20,), 16, False, 5, C=C, G=G, r=r)
    full = q.qwm_attention_shared_workspace(c.c, Q.shape[0], 2, 1, 70, 20)[1]
    ws = torch.zeros(full, dtype=torch.uint8, device="cuda")
    c.attention_shared(Q, cu, 70, kv, table, lens, 20, workspace=ws)
    _fine()
    n = 2 * T * d
    tail = ws[full - 4 * n:].view(torch.int16)
    assert torch.equal(tail[n:].view(2, T, d), Vp.view(torch.int16))
    got, want = tail[:n].view(BF16).view(2, T, d).double(), Kp.double()
    if r == 0:
        assert torch.equal(tail[:n].view(2, T, d), Kp.view(torch.int16))
        return
    U, ver = c.view("basis").double().abs(), c.view("tokver")[:T].long()
    c8, cs = c.view("k_coef")[:, :T].double().abs(), c.view("k_cscale").view(torch.float16)[:, :T].double().abs()
    comp = torch.stack([torch.einsum("tdr,tr->td", U[ver, h], c8[h]) * cs[h][:, None] for h in range(2)])
    both = 2 * (r + 4) * F32 * (want.abs() + 2 * comp)
    off = (got - want).abs()
    assert (off <= both + 2 * HALF * torch.maximum(got.abs(), want.abs())).all(), off.max()
    share = (both / (HALF * want.abs().clamp_min(1e-30))).clamp_max(1.0)
    assert (off > 0).sum() <= share.sum(), ((off > 0).sum(), share.sum())


@pytest.mark.parametrize("H,C,G,r,d,T,rows", [
    (3, 256, 32, 8, 128, 4000, 8),     # both tables in shared memory; keys of two basis versions in one tile
    (3, 300, 32, 8, 128, 1000, 16),    # tables read through the cache, 16-bit centroid numbers
    (3, 512, 16, 3, 64, 1500, 32),
    (3, 40, 16, 8, 128, 129, 1),       # a chunk of one key
    (3, 16, 32, 1, 64, 1, 5),          # a single key
    (3, 64, 32, 0, 128, 777, 17),      # no compensation
    (3, 64, 32, 9, 128, 777, 17),      # an odd rank above 8
    (3, 256, 16, 16, 128, 700, 3),     # the largest rank and tables that shared memory takes
    (3, 512, 16, 16, 64, 700, 16),
    (3, 512, 32, 12, 128, 700, 16),
    # as many tiles as the few-row kernel wants (four for every warp of the GPU, below 7200)
    (2, 256, 16, 16, 128, 57601, 3),
    (2, 256, 32, 8, 128, 57609, 16),
    (2, 256, 32, 8, 128, 57609, 17),   # a row more than it takes
    (2, 300, 32, 8, 128, 57600, 16),
    (1, 512, 16, 3, 64, 115231, 7),
    (2, 512, 16, 12, 64, 57623, 1),
    (5, 64, 32, 0, 128, 23057, 5),
    (100, 40, 16, 5, 128, 1153, 2),    # a block's run of tiles crosses heads
    (1200, 16, 32, 8, 64, 96, 16),     # many heads in a block's run, a table and basis for each
    (3700, 16, 16, 4, 64, 17, 1),      # a whole tile and one key per head
])
def test_few_rows_over_the_history(H, C, G, r, d, T, rows):
    """Against the unpacked history (test_shared_history_is_the_reconstruction holds it to the
    reconstruction), which the same decoder makes: where the compensation's order of sums lets a key
    element fall to the other side of a border, a step of 2^-7 |K'|, a score moves by 2^-7 |K'| |q| / sqrt(d),
    0.004 at |K'| = 2 and |q| = 2, d = 64, and the log-sum-exp of 96 keys by a 96th of that, 4e-5 and more
    with the key's weight: of the order of the bounds, which count no such steps."""
    g = _gen(C + T)
    c = _cache(g, H, d, T, C, G, r)
    full = q.qwm_attention_shared_workspace(c.c, 17, H, 1, 17, 0)[1]
    ws = torch.empty(full, dtype=torch.uint8, device="cuda")
    c.attention_shared(torch.zeros(17, H, d, dtype=BF16, device="cuda"), ints([0, 17]), 17, workspace=ws)
    Kp, Vp = ws[full - 4 * H * T * d:].view(BF16).view(2, H, T, d)
    Q = randn(g, rows, H, d).to(BF16)
    lse = torch.empty(rows, H, device="cuda")
    O = c.attention_shared(Q, ints([0, rows]), rows, lse=lse)
    _fine()
    for h in range(H) if H <= 5 else range(0, H, H // 50):
        want, bound, wl, lb = attend(Q[:, h], Kp[h], Vp[h], 1 / math.sqrt(d))
        check("O", O[:, h], want, bound)
        check_lse("lse", lse[:, h], wl, lb)
    assert torch.equal(O, c.attention_shared(Q, ints([0, rows]), rows))   # the same bits again


def test_shared_history_alone_is_qwm_attention():
    """Without pages the call is qwm_attention (both read the same bf16 cache); a longer max_q than
    needed changes nothing, a shorter one leaves the rows behind it out."""
    c, Kp, Vp, rows, kv, table, Q, cu, lens = _shared_case(128, 2, 1, 900, (5, 9), (1, 1), 16, False, 21)
    want, bound, wl, lb = _shared_want(Kp, Vp, [(k[:, :0], v[:, :0]) for k, v in rows], Q, (5, 9), (0, 0), False, 1)
    O = c.attention_shared(Q, cu, 100)
    check("O", O[:14], want[:14], bound[:14])
    other = c.attention(Q.contiguous())
    check("attention", other[:14], want[:14], 2 * bound[:14])
    short = torch.full_like(O, 7.0)
    c.attention_shared(Q, cu, 6, O=short)
    _fine()
    check("short", short[:11], want[:11], bound[:11])
    assert (short[11:] == 7.0).all()


@pytest.mark.parametrize("T,new", [(300, (130, 140)), (0, (3, 5)), (200, (2, 3))])
def test_shared_bounds_below_the_lengths(T, new):
    """max_kv below a branch's keys leaves the keys behind it out, max_q the rows; the causal limit still
    counts from the branch's true length."""
    own, most_q, most_kv = (150, 160), min(new), 100
    c, Kp, Vp, rows, kv, table, Q, cu, lens = _shared_case(64, 2, 1, T, new, own, 16, True, 41)
    O, lse = torch.full_like(Q, 7.0).contiguous(), torch.full(Q.shape[:2], 5.0, device="cuda")
    c.attention_shared(Q, cu, most_q, kv, table, lens, most_kv, causal=True, O=O, lse=lse)
    _fine()
    at = torch.arange(T + most_kv, device="cuda")
    for b in range(2):
        s = slice(sum(new[:b]), sum(new[:b]) + most_q)
        last = T + own[b] - new[b] + torch.arange(most_q, device="cuda")
        for h in range(2):
            k, v = (torch.cat([x[h], y[h][:most_kv]]) for x, y in zip((Kp, Vp), rows[b]))
            want, bound, wl, lb = attend(Q[s, h], k, v, 1 / 8, (at <= last[:, None]) | (at < T))
            check("O", O[s, h], want, bound)
            check_lse("lse", lse[s, h], wl, lb)
    left = slice(new[0] + most_q, None)
    assert (O[left] == 7.0).all() and (lse[left] == 5.0).all()


def test_shared_bad_device_arrays():
    """Page numbers, lengths and offsets outside their buffers are clamped and reported."""
    c, Kp, Vp, rows, kv, table, Q, cu, lens = _shared_case(64, 1, 1, 100, (4, 4), (20, 20), 16, False, 31)
    assert q.qwm_device_status() == 0
    for bad_table, bad_cu, bad_len in ((table + 1000, cu, lens), (table * 0 - 1, cu, lens),
                                       (table, cu, ints([20, 10**9])), (table, cu, ints([-3, 20])),
                                       (table, ints([0, 4, 10**6]), lens), (table, ints([0, -4, 8]), lens)):
        c.attention_shared(Q, bad_cu, 8, kv, bad_table, bad_len, 32)
        assert q.qwm_device_status() == 2
        assert q.qwm_device_status() == 0


# ------------------------------------------------------------------ cross attention
@pytest.mark.parametrize("d,Hk,gh,new,states,padded,split", [
    (128, 2, 1, (1, 3), (1, 77), True, True),
    (128, 1, 3, (200, 57, 0), (129, 0, 300), True, True),     # an empty encoding, a batch entry of no rows
    (64, 3, 1, (7, 7, 7), (512, 128, 127), False, True),
    (64, 1, 5, (300,), (1500,), False, True),                 # key ranges split
    (64, 1, 5, (300,), (1500,), False, False),                # the same in one range (no workspace)
    (128, 4, 1, (513,), (1025,), True, True),
    (128, 1, 1, (1,), (5000,), False, True),                  # one row, many ranges
    (128, 12, 1, (8,), (16300,), False, False),               # few rows, bound by memory: many laps of the ring
    (64, 16, 1, (3, 1), (16300, 9000), False, False),
])
def test_cross_attention(d, Hk, gh, new, states, padded, split):
    g = _gen(d + sum(states))
    most = max(states)
    start = [most * i for i in range(len(states))] if padded else offsets(states)[:-1]
    n_kv = most * len(states) if padded else sum(states)
    kvs = randn(g, n_kv, 2, Hk, d).to(BF16)
    used = torch.zeros(n_kv, dtype=torch.bool, device="cuda")
    for s, n in zip(start, states):
        used[s:s + n] = True
    kvs[~used] = NAN   # padding
    n, Hq = sum(new) + 1, Hk * gh
    Q = randn(g, n, Hq, d).to(BF16)
    O = torch.full((n, Hq, d), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((n, Hq), 5.0, device="cuda")
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    q.qwm_cross_attention(Q, kvs[:, 0], kvs[:, 1], ints(offsets(new)), ints(start), ints(list(states)), max(new),
                          most, O=O, lse=lse, workspace=ws)
    _fine()
    cu = offsets(new)
    for b in range(len(new)):
        for h in range(Hq):
            k, v = (kvs[start[b]:start[b] + states[b], j, h // gh] for j in (0, 1))
            want, bound, wl, lb = attend(Q[cu[b]:cu[b + 1], h], k, v, 1 / math.sqrt(d))
            check("O", O[cu[b]:cu[b + 1], h], want, bound)
            check_lse("lse", lse[cu[b]:cu[b + 1], h], wl, lb)
    assert (O[-1] == 7.0).all() and (lse[-1] == 5.0).all(), "a row of no sequence was written"


def test_cross_attention_bad_device_arrays():
    g = _gen(1)
    Q, kv = randn(g, 6, 1, 64).to(BF16), randn(g, 50, 1, 64).to(BF16)
    assert q.qwm_device_status() == 0
    for start, n in ((60, 3), (-2, 3), (40, 20), (2**31 - 1, 2**31 - 1), (0, -1)):
        q.qwm_cross_attention(Q, kv, kv, ints([0, 6]), ints([start]), ints([n]), 6, 60)
        assert q.qwm_device_status() == 2


@pytest.mark.parametrize("new,states,split", [((130,), (200,), False), ((3,), (5000,), True)])
def test_a_nan_query_stays_in_its_row(new, states, split):
    """A NaN in one query row gives NaN (O and lse) there, and leaves the other rows' bits alone; in one
    key range and in several."""
    g = _gen(41)
    Q, kv = randn(g, new[0], 2, 128).to(BF16), randn(g, states[0], 2, 128).to(BF16)
    sizes = q.qwm_cross_attention_workspace(2, 2, 128, new[0], 1, new[0], states[0])
    assert (sizes[1] > 0) == split
    args = ints([0, new[0]]), ints([0]), ints(list(states)), new[0], states[0]
    lse, bad = (torch.empty(new[0], 2, device="cuda") for _ in range(2))
    O = q.qwm_cross_attention(Q, kv, kv, *args, lse=lse)
    Q[1, 1, 5] = NAN
    P = q.qwm_cross_attention(Q, kv, kv, *args, lse=bad)
    _fine()
    assert P[1, 1].isnan().all() and bad[1, 1].isnan()
    P[1, 1], bad[1, 1] = O[1, 1], lse[1, 1]
    assert torch.equal(P, O) and torch.equal(bad, lse)


def test_large_scores_and_scale():
    """Scores up to +-2000: the running maximum moves, no weight overflows; an explicit scale."""
    g = _gen(77)
    Q, K, V = (randn(g, n, 1, 128) for n in (40, 700, 700))
    K = K * torch.linspace(0.1, 12, 700, device="cuda")[:, None, None]
    Q, K, V = (Q * 4).to(BF16), K.to(BF16), V.to(BF16)
    lse = torch.empty(40, 1, device="cuda")
    O = q.qwm_cross_attention(Q, K, V, ints([0, 40]), ints([0]), ints([700]), 40, 700, lse=lse, scale=1.0)
    _fine()
    want, bound, wl, lb = attend(Q[:, 0], K[:, 0], V[:, 0], 1.0)
    check("O", O[:, 0], want, bound)
    check_lse("lse", lse[:, 0], wl, lb)


# ------------------------------------------------------------------ a layer step
def test_layer_step_in_a_graph():
    """Two branches of one history: norm and rotation, append to pages, attention over history and
    pages, cross attention; on a side stream, captured once and replayed on new rows, against the
    same calls made eagerly and against the 64-bit forms."""
    H, d, T, page, new, held = 3, 128, 400, 16, (20, 31), (5, 0)
    g = _gen(123)
    c = _cache(g, H, d, T)
    own = [a + b for a, b in zip(new, held)]
    n_pages, table = _table(g, own, page)
    kv = q.PagedKV(torch.zeros(n_pages, H, page, d, dtype=BF16, device="cuda"),
                   torch.zeros(n_pages, H, page, d, dtype=BF16, device="cuda"))
    n = sum(new)
    qkv = torch.empty(n, 3 * H, d, dtype=BF16, device="cuda")
    enc = randn(g, 90, 2, H, d).to(BF16)
    w = (1 + 0.3 * randn(g, d)).to(BF16)
    rope = q.qwm_rope_init(d, 128, "interleaved", axis_dims=(44, 42, 42))
    pos = torch.randint(0, 900, (3, n), generator=g, device="cuda").to(torch.int32)
    cu, start, lens, es, en = ints(offsets(new)), ints(list(held)), ints(own), ints([0, 40]), ints([40, 50])

    def step(stream=None):
        Q, _ = q.qwm_norm_rope(rope, qkv[:, :H], None, pos, w, stream=stream)
        kv.append(table, cu, start, qkv[:, H:2 * H], qkv[:, 2 * H:], rope, pos, w, stream=stream)
        O = c.attention_shared(Q, cu, max(new), kv, table, lens, max(own), causal=True, stream=stream)
        return Q, O, q.qwm_cross_attention(O, enc[:, 0], enc[:, 1], cu, es, en, max(new), 50, stream=stream)

    qkv.copy_(randn(g, n, 3 * H, d).to(BF16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in (1, 2):
        qkv.copy_(randn(_gen(seed), n, 3 * H, d).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in kept]
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        eager = step(stream=other)   # tensors of the current stream, work on another
        other.synchronize()
        for a, b in zip(replayed, eager):
            assert torch.equal(a, b)
        _fine()
        freqs, gain = frequencies(128, (44, 42, 42), "none", 1.0)
        want, bound = norm_rope(qkv[:, :H], w, pos, freqs, gain, 128, "interleaved")
        check("Q", replayed[0], want, bound)
        Kp, Vp = c.reconstruct()
        rows = [tuple(x[t.long()].transpose(0, 1).reshape(H, -1, d)[:, :m] for x in (kv.K, kv.V))
                for t, m in zip(table, own)]
        out, tol, _, _ = _shared_want(Kp, Vp, rows, replayed[0], new, own, True, 1)
        check("O", replayed[1], out, tol)
        cb = offsets(new)
        for b, (s, m) in enumerate(((0, 40), (40, 50))):
            for h in range(H):
                x = attend(replayed[1][cb[b]:cb[b + 1], h], enc[s:s + m, 0, h], enc[s:s + m, 1, h], 1 / math.sqrt(d))
                check("cross", replayed[2][cb[b]:cb[b + 1], h], x[0], x[1])


def test_replay_with_other_lengths():
    """One captured call serves other lengths and rows per branch up to its bounds: the device arrays are
    read at each replay."""
    c, Kp, Vp, rows, kv, table, Q, cu, lens = _shared_case(128, 2, 1, 300, (9, 6), (80, 50), 16, True, 3, poison=False)
    n = Q.shape[0]
    O = torch.zeros(n, 2, 128, dtype=BF16, device="cuda")
    lse = torch.zeros(n, 2, device="cuda")
    ws = torch.empty(q.qwm_attention_shared_workspace(c.c, n, 2, 2, 12, 90)[1], dtype=torch.uint8, device="cuda")

    def call():
        c.attention_shared(Q, cu, 12, kv, table, lens, 80, causal=True, O=O, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new, own in (((9, 6), (80, 50)), ((3, 12), (17, 12)), ((0, 1), (0, 1)), ((1, 1), (64, 33))):
        cu.copy_(ints(offsets(new)))
        lens.copy_(ints(list(own)))
        graph.replay()
        _fine()
        part = [(k[:, :m], v[:, :m]) for (k, v), m in zip(rows, own)]
        want, bound, wl, lb = _shared_want(Kp, Vp, part, Q, new, own, True, 1)
        live = sum(new)
        check("O", O[:live], want[:live], bound[:live])
        check_lse("lse", lse[:live], wl[:live], lb[:live])


def test_two_calls_at_once():
    """Calls on two streams at once, each with a workspace of its own, give what they give alone."""
    cases = [_shared_case(128, 2, 1, 900, (40, 40), (70, 20), 16, True, seed) for seed in (1, 2)]
    g = _gen(5)
    x, enc = randn(g, 300, 2, 128).to(BF16), randn(g, 2500, 2, 128).to(BF16)
    args = ints([0, 300]), ints([0]), ints([2500]), 300, 2500

    def shared(i, stream=None):
        c, _, _, _, kv, table, Q, cu, lens = cases[i]
        return c.attention_shared(Q[:80], cu, 40, kv, table, lens, 70, causal=True, stream=stream)

    alone = shared(0), shared(1), q.qwm_cross_attention(x, enc, enc, *args)
    _fine()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = (shared(0, streams[0]), shared(1, streams[1]),
               q.qwm_cross_attention(x, enc, enc, *args, stream=streams[2]))
        for s in streams:
            s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, got))
    _fine()


def test_branches_that_share_pages():
    """Two branches whose tables begin with the same pages (a common prefix), and one page named twice in
    a table: pages are only read."""
    g = _gen(8)
    c = _cache(g, 2, 64, 100)
    Kp, Vp = c.reconstruct()
    kv = q.PagedKV(randn(g, 5, 2, 32, 64).to(BF16), randn(g, 5, 2, 32, 64).to(BF16))
    table = ints([[3, 1, 1], [3, 1, 4]])
    own, new = (80, 96), (2, 3)
    rows = [(kv.K[t.long()].transpose(0, 1).reshape(2, -1, 64)[:, :m],
             kv.V[t.long()].transpose(0, 1).reshape(2, -1, 64)[:, :m]) for t, m in zip(table, own)]
    Q = randn(g, 5, 2, 64).to(BF16)
    O = c.attention_shared(Q, ints([0, 2, 5]), 3, kv, table, ints(list(own)), 96)
    _fine()
    want, bound, _, _ = _shared_want(Kp, Vp, rows, Q, new, own, False, 1)
    check("O", O, want, bound)


def test_many_sequences():
    """65535 sequences, most of them empty, in append and in both attentions."""
    g = _gen(21)
    n_seq, live = 65535, (0, 77, 40000, 65534)
    cu = torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda")
    for b in live:
        cu[b + 1:] += 1
    K, V, Q = (randn(g, 4, 1, 64).to(BF16) for _ in range(3))
    kv = q.PagedKV(torch.zeros(4, 1, 16, 64, dtype=BF16, device="cuda"), torch.zeros(4, 1, 16, 64, dtype=BF16, device="cuda"))
    table = torch.full((n_seq, 1), -1, dtype=torch.int32, device="cuda")
    start, lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda"), torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    for i, b in enumerate(live):
        table[b], start[b], lens[b] = i, 2 * i, 2 * i + 1
    kv.append(table, cu, start, K, V)
    for i in range(4):
        assert torch.equal(kv.K[i, :, 2 * i], K[i]) and torch.equal(kv.V[i, :, 2 * i], V[i])
    c = _cache(g, 1, 64, 50)
    Kp, Vp = c.reconstruct()
    O = c.attention_shared(Q, cu, 1, kv, table, lens, 16)
    X = q.qwm_cross_attention(Q, kv.K.view(64, 1, 64), kv.V.view(64, 1, 64), cu, start, lens, 1, 16)
    _fine()
    for i in range(4):
        k, v = kv.K[i, 0, :2 * i + 1], kv.V[i, 0, :2 * i + 1]
        want, bound, _, _ = attend(Q[i], torch.cat([Kp[0], k]), torch.cat([Vp[0], v]), 0.125)
        check("shared", O[i], want, bound)
        k, v = (x.view(64, 64)[2 * i:4 * i + 1] for x in (kv.K, kv.V))
        want, bound, _, _ = attend(Q[i], k, v, 0.125)
        check("cross", X[i], want, bound)


def _small_calls():
    """Calls of each operator that allocates, by stream."""
    c, _, _, _, kv, table, Q, cu, lens = _shared_case(128, 2, 1, 900, (40, 40), (70, 20), 16, True, 7)
    g = _gen(5)
    x, enc = randn(g, 300, 2, 128).to(BF16), randn(g, 2500, 2, 128).to(BF16)
    args = ints([0, 300]), ints([0]), ints([2500]), 300, 2500
    w = (1 + randn(g, 128)).to(BF16)
    sizes = {"rope": 0, "shared": q.qwm_attention_shared_workspace(c.c, 80, 2, 2, 40, 70)[1],
             "cross": q.qwm_cross_attention_workspace(2, 2, 128, 300, 1, 300, 2500)[1]}
    calls = {"rope": lambda s: q.qwm_norm_rope(None, x, q_weight=w, stream=s)[0],
             "shared": lambda s: c.attention_shared(Q[:80], cu, 40, kv, table, lens, 70, causal=True, stream=s),
             "cross": lambda s: q.qwm_cross_attention(x, enc, enc, *args, stream=s)}
    return calls, sizes


@pytest.mark.parametrize("name", ["rope", "shared", "cross"])
def test_a_call_on_another_stream_leaves_freed_memory_alone(name):
    """Blocks that were freed while the current stream's work still reads them are not what a call on
    another stream, which does not wait for that work, writes to."""
    calls, sizes = _small_calls()
    alone = calls[name](None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls[name](side)   # (the other stream's pool has blocks of these sizes from here on)
    g = _gen(6)
    for raw in (False, True):
        read = [torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8)
                for n in (alone.numel() * 2, sizes[name]) if n]
        want = [t.clone() for t in read]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)   # about 0.06 s
        kept = [t.clone() for t in read]
        del read
        got = calls[name](side.cuda_stream if raw else side)
        side.synchronize()
        assert torch.equal(got, alone)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_a_call_here_beside_one_on_another_stream():
    """A call on the current stream, whose workspace is free again while it still runs, and one on a
    stream that does not wait for it."""
    calls, _ = _small_calls()
    alone = {name: call(None) for name, call in calls.items()}
    side = torch.cuda.Stream()
    for _ in range(5):
        for here, there in (("shared", "shared"), ("cross", "shared"), ("shared", "cross"), ("rope", "cross")):
            side.wait_stream(torch.cuda.current_stream())
            a, b = calls[here](None), calls[there](side)
            side.synchronize()
            assert torch.equal(a, alone[here]) and torch.equal(b, alone[there])
    _fine()


def test_cache_calls_on_another_stream_leave_freed_memory_alone():
    """The same of the calls on the packed cache that return tensors, and of a new cache."""
    g = _gen(9)
    c = _cache(g, 2, 128, 300)
    Q = randn(g, 40, 2, 128).to(BF16)
    K = randn(g, 300, 2, 128).to(BF16)
    calls = (lambda s: [c.attention(Q, stream=s)], lambda s: [c.attention_ext(Q, stream=s)],
             lambda s: c.reconstruct(stream=s), lambda s: c.top1_shift(Q, K, stream=s),
             lambda s: list(q.QuantKVCache(2, 128, 16, 16, 4, 4, 300, stream=s).buffers.values()))
    side = torch.cuda.Stream()
    for call in calls:
        alone = call(None)
        torch.cuda.synchronize()
        read = [torch.randint(0, 256, (t.numel() * t.element_size(),), generator=g, device="cuda",
                              dtype=torch.uint8) for t in alone]
        want = [t.clone() for t in read]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        kept = [t.clone() for t in read]
        del read
        got = call(side)
        side.synchronize()
        if call is not calls[-1]:
            assert all(torch.equal(a, b) for a, b in zip(got, alone))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 64), (128, 16), (64, 16), (64, 48)])
def test_channels_that_are_not_rotated_stay_alone(d, rot, layout):
    """Behind rot_dim a channel without a norm leaves as it came, NaN, infinities and the sign of zero
    included, whatever its neighbours hold; with a norm an infinity, which makes its own channel NaN
    (inf / inf), leaves the others 0.  Rotated channels and an append's keys alike."""
    g = _gen(d + rot)
    n, rest = 9, d - rot
    x = randn(g, n, 2, d).to(BF16)
    special = torch.tensor([NAN, math.inf, -math.inf, -0.0, 0.0, -1.0, 3e38, -3e38], device="cuda").to(BF16)
    for i in range(1, n):   # row 0 has no special values
        for h in range(2):
            at = torch.randperm(rest, generator=g, device="cuda")[:5] + rot
            x[i, h, at] = special[torch.randint(0, 8, (5,), generator=g, device="cuda")]
    clean = x.clone()
    clean[..., rot:] = 1.0
    rope, pos = q.qwm_rope_init(d, rot, layout), ints(list(range(100, 100 + n)))
    out, _ = q.qwm_norm_rope(rope, x, pos=pos)
    assert torch.equal(out[..., rot:].isnan(), x[..., rot:].isnan())
    live = ~x[..., rot:].isnan()
    assert torch.equal(out[..., rot:].view(torch.int16)[live], x[..., rot:].view(torch.int16)[live])
    want, _ = q.qwm_norm_rope(rope, clean, pos=pos)
    assert torch.equal(out[..., :rot], want[..., :rot])
    kv = q.PagedKV(*(torch.zeros(1, 2, 16, d, dtype=BF16, device="cuda") for _ in range(2)))
    kv.append(ints([[0]]), ints([0, n]), ints([0]), x, x, rope, pos)
    assert torch.equal(kv.K[0, :, :n].transpose(0, 1).contiguous().view(torch.int16), out.view(torch.int16))
    x = clean
    x[:, :, rot + 5] = math.inf
    out, _ = q.qwm_norm_rope(rope, x, pos=pos, q_weight=torch.ones(d, dtype=BF16, device="cuda"))
    assert out[:, :, rot + 5].isnan().all()
    out[:, :, rot + 5] = 0
    assert (out == 0).all()


def test_shared_without_a_bound_of_keys():
    """max_kv left out: all of a branch's keys, as with the bound that the tables give."""
    c, Kp, Vp, rows, kv, table, Q, cu, lens = _shared_case(64, 2, 1, 300, (3, 2), (40, 17), 16, True, 51)
    lse = torch.empty(7, 2, device="cuda")
    O = c.attention_shared(Q, cu, 3, kv, table, lens, causal=True, lse=lse)
    _fine()
    want, bound, wl, lb = _shared_want(Kp, Vp, rows, Q, (3, 2), (40, 17), True, 1)
    check("O", O[:5], want[:5], bound[:5])
    check_lse("lse", lse[:5], wl[:5], lb[:5])


def test_calls_with_a_stream_in_a_graph():
    """Calls that name their stream, the capturing one and one that was forked from it, captured and
    replayed over memory that other work has used since."""
    calls, _ = _small_calls()
    alone = {name: call(None) for name, call in calls.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        kept = [(name, call(s)) for name, call in calls.items() for s in (here, side)]
        here.wait_stream(side)
    for _ in range(3):
        for _, t in kept:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, alone[name]) for name, t in kept)
    _fine()
