"""Attention of branches over a shared packed history, held to the packed fields themselves: K' and V'
are rebuilt in 64 bits from the cache's buffers, and the reconstruction is one of the histories that the
attention may have read."""
import math

import pytest
import torch

import bit_kv_cache_23_b200 as q
from around_util import BF16, F32, HALF, attend, check, check_lse, ints, randn
from test_gpu_around import _cache, _fine, _gen

pytestmark = pytest.mark.gpu


def _history(c, h):
    """(lowest, highest) bf16 values, in 64 bits, that K' and V' of head h can have.

    Before its rounding to bf16 an element is x = (c + mn + code sc) + cs sum_i U_i c8_i within E, S =
    |c| + |mn| + |code sc| + cs sum_i |U_i c8_i|, F = 2^-24:
    - a sum of r products by the tensor core, with U in three parts: 3 r terms, each cut off below the
      largest at two roundings at most, 6 r F S; one after another in fp32 it is 2 r F S;
    - the product with cs, the three sums and U's last part (2^-27): 8 F S;
    - mn is shifted by 4^(4 - i) sc (i: place in the code byte) and back: the rounding of that
      difference, computed as it is.
    E counts all of them; where bf16(x - E) = bf16(x + E) the element is that value.  Values, and keys
    at rank 0, are two fp32 operations, t = mn + code sc rounded once and c + t rounded once, whatever
    the order of the rest: x is that result (sums of a few bits, which often lie on a border between two
    bf16 values), and E is 0 where the shift is exact, else the shift's rounding and two more."""
    r, d, T, G = c.cfg.rank, c.cfg.head_dim, c.len, c.cfg.group
    shift = 4.0 ** (4 - torch.arange(d, device="cuda") % 4)
    out = []
    for side in ("k", "v"):
        byte = c.view(side + "_codes")[h, :T].long()
        code = torch.stack([byte >> s & 3 for s in (0, 2, 4, 6)], -1).view(T, d).double()
        mn, sc = c.view(side + "_params").view(torch.float16)[h, :T].double().repeat_interleave(G, 1).unbind(-1)
        idx = c.view(side + "_idx")[h, :T].long() & 0xffff
        ver = c.view("centver")[:T].long()
        cent = torch.stack([c.view("cent_" + side, v)[h] for v in range(c.cfg.max_cent_versions)]).view(BF16)
        cent = cent[ver, idx].double()
        S = cent.abs() + mn.abs() + code * sc.abs()
        x = (cent + (mn + code * sc).float().double()).float().double()   # (exact in 64 bits before each rounding)
        E = ((mn - sc * shift).float().double() - (mn - sc * shift)).abs()
        if side == "k" and r > 0:
            x = cent + mn + code * sc
            coef = c.view("k_coef")[h, :T].double()
            cs = c.view("k_cscale").view(torch.float16)[h, :T, None].double()
            U, tv = c.view("basis")[:, h].double(), c.view("tokver")[:T].long()
            for v in tv.unique().tolist():
                at = tv == v
                x[at] += coef[at] @ U[v].T * cs[at]
                S[at] += coef[at].abs() @ U[v].T.abs() * cs[at].abs()
            E += (6 * r + 8) * F32 * S
        else:
            E = torch.where(E > 0, E + 2 * F32 * S, 0)
        out += [(x - E).to(BF16).double(), (x + E).to(BF16).double()]
    return out


def _check_head(c, h, Kp, Vp, Q, O, lse):
    """One head's rows against the attention over the reconstruction (Kp, Vp).  The attention's own
    history lies between the same bounds, so a score is off by at most ds_t = scale sum_c |q_c| (highest -
    lowest K'_tc); then a weight p_t becomes at most p_t e^(ds_t + ell), ell = ln sum_t p_t e^(ds_t), which
    also bounds the log-sum-exp, and O moves by sum_t p_t ((e^(ds_t + ell) - 1) |v_t| + e^(ds_t + ell)
    (highest - lowest V'_t))."""
    k0, k1, v0, v1 = _history(c, h)
    for name, x, low, high in (("K'", Kp, k0, k1), ("V'", Vp, v0, v1)):
        assert ((low <= x.double()) & (x.double() <= high)).all(), f"{name} of the reconstruction"
    scale = 1 / math.sqrt(c.cfg.head_dim)
    want, bound, wl, lb = attend(Q, Kp, Vp, scale)
    q64, k, v = Q.double(), Kp.double(), Vp.double()
    ds = q64.abs() @ (k1 - k0).T * scale
    p = torch.softmax(q64 @ k.T * scale, 1)
    ell = (p * ds.exp()).sum(1).log()
    grown = p * (ds + ell[:, None]).exp()
    extra = (grown - p) @ v.abs() + grown @ (v1 - v0)
    more = (ds.amax(1) + ell).exp()   # (the bound's own weights may be larger by this)
    check("O", O, want, bound * more[:, None] + extra)
    check_lse("lse", lse, wl, lb * more + ell)
    # so the extra is a small share: the check would see a wrong key
    assert extra.mean() <= HALF * v.abs().mean(), (extra.mean(), v.abs().mean())


CASES = [   # heads, centroids, group, rank, head_dim, tokens, rows, path
    (3, 16, 32, 1, 64, 1, 5, "unpacked"),          # a single key
    (3, 40, 16, 8, 128, 129, 1, "unpacked"),
    (3, 256, 32, 8, 128, 4000, 8, "unpacked"),
    (3, 300, 32, 8, 128, 1000, 16, "unpacked"),    # 16-bit centroid numbers
    (3, 512, 16, 3, 64, 1500, 32, "unpacked"),
    (3, 64, 32, 0, 128, 777, 17, "unpacked"),      # no compensation
    (3, 64, 32, 9, 128, 777, 17, "unpacked"),      # an odd rank above 8
    (3, 256, 16, 16, 128, 700, 3, "unpacked"),
    (3, 512, 16, 16, 64, 700, 16, "unpacked"),
    (3, 512, 32, 12, 128, 700, 16, "unpacked"),
    # staged tables in the unpacking: 32 keys per centroid in a block's run
    (4, 4, 16, 16, 128, 9601, 17, "unpacked"),
    (4, 8, 32, 8, 128, 9601, 17, "unpacked"),
    (4, 4, 16, 8, 64, 9601, 17, "unpacked"),
    (4, 4, 32, 16, 64, 9601, 17, "unpacked"),
    (4, 32, 16, 16, 128, 40000, 17, "unpacked"),
    (32, 256, 32, 16, 128, 38001, 17, "unpacked"),
    # decoded into the products: up to 16 rows, four tiles for every warp of the GPU (below 7200)
    (2, 256, 16, 16, 128, 57601, 3, "rows"),
    (2, 256, 32, 8, 128, 57609, 16, "rows"),
    (2, 300, 32, 8, 128, 57600, 16, "rows"),       # tables read through the cache, 16-bit numbers
    (2, 300, 32, 16, 128, 57609, 16, "rows"),      # the same with a rank above 8
    (3, 512, 16, 12, 128, 38401, 1, "rows"),
    (1, 512, 16, 3, 64, 115231, 7, "rows"),
    (2, 512, 16, 12, 64, 57623, 1, "rows"),
    (5, 64, 32, 0, 128, 23057, 5, "rows"),
    (100, 40, 16, 5, 128, 1153, 2, "rows"),        # a block's run of tiles crosses heads
    (1200, 16, 32, 8, 64, 96, 16, "rows"),
    (3700, 16, 16, 4, 64, 17, 1, "rows"),
]


@pytest.mark.parametrize("H,C,G,r,d,T,rows,path", CASES)
def test_history_from_the_packed_fields(H, C, G, r, d, T, rows, path):
    g = _gen(C + T + 1)
    c = _cache(g, H, d, T, C, G, r)
    Kp, Vp = c.reconstruct()
    Q = randn(g, rows, H, d).to(BF16)
    least, full = q.qwm_attention_shared_workspace(c.c, rows, H, 1, rows, 0)
    head = 4 * T * d   # of one head unpacked; the workspace then holds one at least
    assert full - least == (head * (H - 1) if path == "unpacked" else 0) and (H > 1 or full < head)
    lse = torch.empty(rows, H, device="cuda")
    O = c.attention_shared(Q, ints([0, rows]), rows, lse=lse)
    _fine()
    for h in range(H) if H <= 5 else range(0, H, -(-H // 20)):
        _check_head(c, h, Kp[h], Vp[h], Q[:, h], O[:, h], lse[:, h])


def test_a_kept_branch_is_committed():
    """Keys normed and rotated once go to a branch's pages and, when the branch is kept, to the packed
    history: the pages hold those rows, and the history grows by them."""
    g = _gen(61)
    H, d, new = 2, 64, 40
    c = q.QuantKVCache(H, d, 16, 16, 4, 4, 200)
    first = randn(g, 2, 100, H, d).to(BF16)
    c.build_centroids(*first)
    c.update_query_stats(randn(g, 16, H, d).to(BF16))
    c.append_kv(*first)
    qkv = randn(g, 2 * new, 3 * H, d).to(BF16)
    w = (1 + 0.3 * randn(g, d)).to(BF16)
    rope, pos = q.qwm_rope_init(d, d), torch.arange(2 * new, device="cuda", dtype=torch.int32) % new + 100
    kv = q.PagedKV(*(torch.zeros(6, H, 16, d, dtype=BF16, device="cuda") for _ in range(2)))
    table, cu = ints([[5, 0, 3], [1, 2, 4]]), ints([0, new, 2 * new])
    _, K = q.qwm_norm_rope(rope, None, qkv[:, H:2 * H], pos, k_weight=w)
    kv.append(table, cu, ints([0, 0]), K, qkv[:, 2 * H:])
    rows = slice(new, 2 * new)   # the second branch is kept
    c.append_kv(K[rows].contiguous(), qkv[rows, 2 * H:].contiguous())
    _fine()
    assert c.len == 100 + new
    paged = kv.K[table[1].long()].transpose(0, 1).reshape(H, -1, d)[:, :new]
    assert torch.equal(paged, K[rows].transpose(0, 1))
    Q = randn(g, 5, H, d).to(BF16)
    Kp, Vp = c.reconstruct()
    lse = torch.empty(5, H, device="cuda")
    O = c.attention_shared(Q, ints([0, 5]), 5, lse=lse)
    for h in range(H):
        _check_head(c, h, Kp[h], Vp[h], Q[:, h], O[:, h], lse[:, h])
