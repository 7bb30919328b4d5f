"""Plain 64-bit forms of the operators around the packed cache, and the error
bounds that their tests hold the kernels to."""
import math

import torch

BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2        # one rounding to bf16: 2^-8 relative
F32 = torch.finfo(torch.float32).eps / 2  # one rounding to fp32: 2^-24 relative


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets(lengths):
    return [sum(lengths[:i]) for i in range(len(lengths) + 1)]


def frequencies(rot, axis_dims, scaling, factor, theta=10000.0, orig=4096.0, fast=32.0, slow=1.0):
    """(frequency, axis) of each pair and the gain, from the formulas."""
    out = []
    for axis, dim in enumerate(axis_dims):
        for i in range(dim // 2):
            base = theta * factor ** (dim / (dim - 2)) if scaling == "ntk" else theta
            f = base ** (-2 * i / dim)
            if scaling == "linear":
                f /= factor
            if scaling == "parts":
                keep = min(1.0, max(0.0, (orig * f / (2 * math.pi) - slow) / (fast - slow)))
                f = keep * f + (1 - keep) * f / factor
            out.append((f, axis))
    assert len(out) == rot // 2
    return out, 1 + 0.1 * math.log(factor) if scaling == "parts" else 1.0


def norm_rope(x, w, pos, freqs, gain, rot, layout, eps=1e-6):
    """(result, bound) in 64 bits of the norm and rotation of x [n][h][d]."""
    y = x.double()
    d = y.shape[-1]
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    out, size = y.clone(), y.abs()
    for p, (f, axis) in enumerate(freqs if rot else []):
        a, b = (p, p + rot // 2) if layout == "half" else (2 * p, 2 * p + 1)
        t = (pos[axis].double() * f)[:, None]
        out[..., a] = gain * (y[..., a] * t.cos() - y[..., b] * t.sin())
        out[..., b] = gain * (y[..., a] * t.sin() + y[..., b] * t.cos())
        size[..., a] = size[..., b] = gain * (y[..., a].abs() + y[..., b].abs())
    # fp32 before the one rounding: mean (log2 d + 8 roundings), root, weight, gain, two
    # products and a sum: below 32 roundings; the angle's reduction to fp32 (half a step of
    # [2, 4): 2^-23) and sincosf (2 steps: 2^-23) count 2^-22 together = 4 roundings
    return out, HALF * out.abs() + (32 + 4) * F32 * size * (1 + HALF)


def attend(q, k, v, scale, seen=None):
    """(out, bound, lse, bound) in 64 bits: q [n][d] over k, v [t][d]; seen: [n][t] or None.

    Weights p are rounded to bf16 (HALF relative each, so HALF times the weighted mean of |v|),
    scores carry d products and sums in fp32 (tensor-core sums may truncate: two roundings each),
    2^x is good to 2^-22, and the sums over t keys are fp32."""
    q, k, v = q.double(), k.double(), v.double()
    n, t = q.shape[0], k.shape[0]
    if t == 0:
        z = torch.zeros(n, v.shape[1], dtype=torch.float64, device=q.device)
        inf = torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
        return z, z, inf, torch.zeros_like(inf)
    s = q @ k.T * scale
    ds = 2 * q.shape[1] * F32 * (q.abs() @ k.abs().T * scale).amax(1)
    if seen is not None:
        s = s.masked_fill(~seen, -math.inf)
    top = s.amax(1)
    live = top > -math.inf
    top0 = torch.where(live, top, 0)
    p = (s - top0[:, None]).exp()
    l = p.sum(1)
    ls = torch.where(live, l, 1)
    out, mean = p @ v / ls[:, None], p @ v.abs() / ls[:, None]
    # the exponent is formed as score times log2 e minus the reference: roundings of both
    ds = ds + 8 * F32 * (1 + s.masked_fill(s == -math.inf, 0).abs().amax(1))
    rel = HALF + 2 * ds + (2 * t + 64) * F32
    bound = HALF * out.abs() + rel[:, None] * mean * (1 + 2 * HALF)
    lse = torch.where(live, top0 + ls.log(), -math.inf)
    return out, bound, lse, 2 * ds + (t + 64) * F32 + 4 * F32 * top0.abs()


def check(name, got, want, bound):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst {err[bad].max():.3g} " \
                          f"(bound {bound[bad].min():.3g}) first at {bad.nonzero()[0].tolist()}"


def check_lse(name, got, want, bound):
    dead = want == -math.inf
    assert torch.equal(dead, got.double() == -math.inf), f"{name}: lse of rows without keys"
    check(name, got[~dead], want[~dead], bound[~dead])
