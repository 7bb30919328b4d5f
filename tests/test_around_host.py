"""Host-side checks of the operators around the packed cache (no GPU needed):
invalid calls return the documented status before touching the device, the
binding's structures match the header, and workspaces follow the sizes."""
import ctypes
import math
import os
import subprocess
import tempfile

import pytest
import torch

import bit_kv_cache_23_b200 as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x200000)
ODD = ctypes.c_void_p(0x200004)


def _rope(**kw):
    return q.qwm_rope_init(**dict(dict(head_dim=128, rot_dim=128), **kw))


def test_structures_match_the_header():
    src = r'''
#include <stddef.h>
#include <stdio.h>
#include "qwm.h"
#define F(T, f) printf(#T "." #f " %zu\n", offsetof(T, f))
int main(void) {
  printf("qwm_rope %zu\nqwm_pages %zu\n", sizeof(qwm_rope), sizeof(qwm_pages));
  F(qwm_rope, head_dim); F(qwm_rope, rot_dim); F(qwm_rope, layout); F(qwm_rope, n_axes);
  F(qwm_rope, axis_dim); F(qwm_rope, magic); F(qwm_rope, gain); F(qwm_rope, freq);
  F(qwm_pages, K); F(qwm_pages, V); F(qwm_pages, n_pages); F(qwm_pages, heads);
  F(qwm_pages, head_dim); F(qwm_pages, page_size); F(qwm_pages, reserved);
  printf("half %d\ninterleaved %d\nnone %d\nlinear %d\nntk %d\nparts %d\n", QWM_ROPE_HALF,
         QWM_ROPE_INTERLEAVED, QWM_ROPE_SCALE_NONE, QWM_ROPE_SCALE_LINEAR, QWM_ROPE_SCALE_NTK,
         QWM_ROPE_SCALE_PARTS);
  return 0;
}
'''
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "p.c"), os.path.join(td, "p")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        out = dict(line.split() for line in subprocess.check_output([exe], text=True).splitlines())
    for name in ("qwm_rope", "qwm_pages"):
        st = getattr(q, name)
        assert int(out[name]) == ctypes.sizeof(st)
        for f, _ in st._fields_:
            assert int(out[f"{name}.{f}"]) == getattr(st, f).offset, f
    for table in (q.ROPE_LAYOUTS, q.ROPE_SCALINGS):
        for name, value in table.items():
            assert int(out[name]) == value


def test_rope_frequencies():
    r = _rope(axis_dims=(44, 42, 42), layout="interleaved")
    want = [10000.0 ** (-2 * i / n) for n in (44, 42, 42) for i in range(n // 2)]
    assert all(math.isclose(a, b, rel_tol=1e-14) for a, b in zip(r.freq, want)) and r.gain == 1.0
    r = _rope(scaling="parts", factor=8.0)
    assert math.isclose(r.gain, 1 + 0.1 * math.log(8), rel_tol=1e-15)
    assert r.freq[0] == 1.0                                             # 652 turns: kept
    assert math.isclose(r.freq[63], 10000.0 ** (-126 / 128) / 8, rel_tol=1e-14)   # below one turn: divided
    assert math.isclose(_rope(scaling="ntk", factor=4.0).freq[63], (10000.0 * 4 ** (128 / 126)) ** (-126 / 128),
                        rel_tol=1e-13)
    assert math.isclose(_rope(scaling="linear", factor=4.0).freq[5], 10000.0 ** (-10 / 128) / 4, rel_tol=1e-14)


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=144), dict(theta=1.0), dict(theta=math.nan),
    dict(factor=0.5), dict(factor=math.inf), dict(axis_dims=(64, 63, 1)), dict(axis_dims=(64, 32)),
    dict(axis_dims=(32, 32, 32, 32)), dict(axis_dims=()), dict(axis_dims=(126, 2), scaling="ntk"),
    dict(axis_dims=(130, -2)), dict(scaling="parts", orig_len=0.0), dict(scaling="parts", beta_fast=1.0),
    dict(scaling="parts", beta_slow=-1.0), dict(head_dim=64, rot_dim=128)])
def test_rope_refusals(bad):
    with pytest.raises(q.QwmError) as e:
        _rope(**bad)
    assert e.value.status == 1


def test_rope_unknown_names():
    with pytest.raises(ValueError):
        _rope(layout="other")
    with pytest.raises(ValueError):
        _rope(scaling="other")


def _norm_rope(**kw):
    r = _rope()
    a = dict(rope=ctypes.addressof(r), d=128, n=4, Q=P, ldq=256, hq=2, wq=None, Qo=ctypes.c_void_p(0x300000), ldqo=256,
             K=P, ldk=128, hk=1, wk=None, Ko=ctypes.c_void_p(0x400000), ldko=128, pos=P, ldpos=4, eps=1e-6)
    a.update(kw)
    return q.lib().qwm_norm_rope(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(d=96), 1), (dict(d=64), 1), (dict(n=-1), 1), (dict(n=2**31), 1), (dict(Q=None), 1), (dict(Qo=None), 1),
    (dict(ldq=248), 1), (dict(ldq=260), 1), (dict(ldqo=248), 1), (dict(ldk=0), 1), (dict(pos=None), 1),
    (dict(ldpos=3), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(hq=-1), 1), (dict(hk=70000), 1),
    (dict(Qo=P, ldqo=264), 1), (dict(Q=ODD), 2), (dict(Ko=ODD), 2), (dict(wq=ODD), 2),
    (dict(pos=ctypes.c_void_p(0x200002)), 2), (dict(n=0), 0), (dict(hq=0, hk=0), 0),
])
def test_norm_rope_arguments(bad, status):
    assert _norm_rope(**bad) == status


def test_norm_rope_needs_an_initialised_rope():
    assert _norm_rope(rope=ctypes.addressof(q.qwm_rope(head_dim=128, rot_dim=128))) == 1


def _pages(**kw):
    return q.qwm_pages(**dict(dict(K=0x200000, V=0x300000, n_pages=8, heads=2, head_dim=64, page_size=16, reserved=0), **kw))


BAD_PAGES = [dict(K=None), dict(V=None), dict(n_pages=0), dict(n_pages=2**31), dict(heads=0), dict(head_dim=96),
             dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(reserved=1)]


def _append(pages=None, **kw):
    a = dict(p=ctypes.byref(_pages(**(pages or {}))), table=P, n_seq=2, width=3, cu=P, start=P, K=P, ldk=128, V=P, ldv=128,
             n=4, rope=None, pos=None, ldpos=4, wk=None, eps=0.0)
    a.update(kw)
    return q.lib().qwm_paged_append(*a.values(), None)


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_append_bad_pages(bad):
    assert _append(pages=bad) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(p=None), 1), (dict(table=None), 1), (dict(n_seq=0), 1), (dict(width=0), 1), (dict(cu=None), 1),
    (dict(start=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(ldk=120), 1), (dict(ldv=132), 1), (dict(n=-1), 1),
    (dict(eps=-1.0), 1), (dict(K=ODD), 2), (dict(V=ODD), 2), (dict(wk=ODD), 2), (dict(cu=ctypes.c_void_p(0x200002)), 2),
    (dict(n=0), 0)])
def test_append_arguments(bad, status):
    assert _append(**bad) == status


def test_append_rope_of_another_head_dim():
    r = _rope()
    assert _append(rope=ctypes.addressof(r), pos=P) == 1


def _cache(**kw):
    c = q.qwm_cache()
    c.cfg = q.qwm_config(heads=2, head_dim=64, n_centroids=16, group=16, n_cand=4, rank=4, max_versions=4, flags=0,
                         max_cent_versions=1, max_queries=0, max_tokens=1000)
    c.tcap = 1024
    for i in range(q.NBUF):
        c.buf.ptr[i] = 0x100000 + 256 * i * 4096
    c.magic, c.n_versions, c.has_centroids, c.len = 0x51574D31, 1, 1, 1000
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _shared(cache=None, pool=None, **kw):
    pg = _pages(**(pool or {}))
    a = dict(c=ctypes.byref(_cache(**(cache or {}))), Q=P, ldq=256, n_q=8, hq=4, cu=P, n_seq=2, max_q=4,
             pages=ctypes.addressof(pg), table=P, width=3, kv_len=P, max_kv=40, causal=1, scale=0.0, O=P, lse=None,
             ws=ctypes.c_void_p(0x40000000), ws_bytes=1 << 30)
    a.update(kw)
    return q.lib().qwm_attention_shared(*a.values(), None)


@pytest.mark.parametrize("bad", BAD_PAGES + [dict(heads=4), dict(head_dim=128)])
def test_shared_bad_pages(bad):
    assert _shared(pool=bad) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(c=None), 1), (dict(Q=None), 1), (dict(O=None), 1), (dict(cu=None), 1), (dict(hq=3), 1), (dict(hq=0), 1),
    (dict(ldq=248), 1), (dict(ldq=260), 1), (dict(n_q=-1), 1), (dict(n_seq=0), 1), (dict(n_seq=65536), 1),
    (dict(max_q=-1), 1), (dict(max_kv=-1), 1), (dict(max_kv=2**30 + 1), 1), (dict(n_q=2**30), 1), (dict(pages=None), 1), (dict(table=None), 1),
    (dict(kv_len=None), 1), (dict(width=0), 1), (dict(Q=ODD), 2), (dict(O=ODD), 2), (dict(lse=ctypes.c_void_p(0x200002)), 2),
    (dict(ws=ctypes.c_void_p(0x40000010)), 2), (dict(ws=None), 3), (dict(ws_bytes=1000), 3),
    (dict(cache=dict(has_centroids=0)), 4), (dict(cache=dict(magic=0)), 1), (dict(n_q=0), 0), (dict(max_q=0), 0)])
def test_shared_arguments(bad, status):
    assert _shared(**bad) == status


def test_shared_workspace_sizes():
    c = _cache()
    least, full = q.qwm_attention_shared_workspace(c, 80, 4, 2, 40, 40)
    assert full - least == 1000 * 64 * 4      # one of the two heads, keys and values
    assert _shared(n_q=80, max_q=40, ws_bytes=least - 1) == 3
    long = _cache(len=57600)   # few rows over a long history: nothing is unpacked
    few = q.qwm_attention_shared_workspace(long, 8, 4, 2, 4, 40)
    assert few[0] == few[1] and _shared(cache=dict(len=57600), ws_bytes=few[0] - 1) == 3
    empty = _cache(len=0)
    least, full = q.qwm_attention_shared_workspace(empty, 8, 4, 2, 4, 40)
    assert least == full
    with pytest.raises(q.QwmError):
        q.qwm_attention_shared_workspace(c, 8, 5, 2, 4, 40)


def _cross(**kw):
    a = dict(Q=P, ldq=256, n_q=8, hq=4, K=P, ldk=128, V=P, ldv=128, n_kv=100, hk=2, d=64, cu=P, start=P, len=P, n_seq=2,
             max_q=4, max_kv=50, scale=0.0, O=P, lse=None, ws=None, ws_bytes=0)
    a.update(kw)
    return q.lib().qwm_cross_attention(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(Q=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(O=None), 1), (dict(cu=None), 1), (dict(start=None), 1),
    (dict(len=None), 1), (dict(hq=3), 1), (dict(hk=0), 1), (dict(d=96), 1), (dict(d=128), 1), (dict(ldk=120), 1),
    (dict(ldv=130), 1), (dict(n_kv=-1), 1), (dict(n_kv=2**30 + 1), 1), (dict(n_q=2**30), 1), (dict(n_seq=0), 1), (dict(max_q=-1), 1), (dict(n_q=-1), 1), (dict(Q=ODD), 2),
    (dict(K=ODD), 2), (dict(ws=ctypes.c_void_p(0x40000010)), 2), (dict(n_q=0), 0), (dict(max_q=0), 0)])
def test_cross_arguments(bad, status):
    assert _cross(**bad) == status


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    rope = _rope(head_dim=64, rot_dim=64)
    with pytest.raises(ValueError):   # no CPU path exists
        q.qwm_norm_rope(rope, x, x, i)
    with pytest.raises(ValueError):
        q.qwm_cross_attention(x, x, x, i, i, i, 4, 4)
    with pytest.raises(ValueError):
        q.PagedKV(x[None], x[None])
    with pytest.raises(ValueError):
        q.qwm_norm_rope(rope, None, None)


# ------------------------------------------------------------------ the binding, without a GPU
class _Device:
    """Stands in for the GPU beneath the binding: CPU tensors pass its checks, launches are kept
    instead of made, and every allocation is kept with the stream that was current."""

    def __init__(self, monkeypatch):
        self.streams, self.made, self.launches = ["current"], [], []
        empty, empty_like = torch.empty, torch.empty_like

        def on(stream):
            device = self

            class Context:
                def __enter__(self):
                    device.streams.append(stream)

                def __exit__(self, *error):
                    device.streams.pop()

            return Context()

        def allocated(make):
            def call(*a, **kw):
                kw.pop("device", None)
                self.made.append(self.streams[-1])
                return make(*a, **kw)
            return call

        for at, name, value in (
                (torch, "empty", allocated(empty)), (torch, "empty_like", allocated(empty_like)),
                (torch.cuda, "stream", on), (torch.cuda, "current_stream", lambda *a: self.streams[-1]),
                (torch.cuda, "ExternalStream", lambda handle, device=None: ("raw", handle)),
                (torch.Tensor, "record_stream", lambda *a: None),
                (q, "_device_of", lambda t, name: t.get_device()), (q, "_raw_stream", lambda *a: 0),
                (q, "_launch", lambda name, index, *a: self.launches.append((name, a))),
                (q, "_shared_full", lambda *a: 4096), (q, "_cross_full", lambda *a: 4096)):
            monkeypatch.setattr(at, name, value)


class _Stream:
    cuda_stream = 64


@pytest.mark.parametrize("stream,where", [(_Stream, _Stream), (128, ("raw", 128)), (None, "current")])
def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch, stream, where):
    """Outputs and workspaces come from the pool of the stream that the call runs on: in the current
    stream's pool lie blocks whose last use is still queued there."""
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    cache = _cache()
    device = _Device(monkeypatch)
    q.qwm_norm_rope(None, x, x, stream=stream)
    assert device.made == [where] * 2
    q.qwm_attention_shared(cache, x, i, 4, stream=stream)
    assert device.made[2:] == [where] * 2
    q.qwm_cross_attention(x, x, x, i, i[:2], i[:2], 4, 4, stream=stream)
    assert device.made[4:] == [where] * 2
    assert [name for name, _ in device.launches] == ["qwm_norm_rope", "qwm_attention_shared", "qwm_cross_attention"]


@pytest.mark.parametrize("stream,where", [(_Stream, _Stream), (128, ("raw", 128)), (None, "current")])
def test_what_the_cache_calls_allocate_belongs_to_their_stream(monkeypatch, stream, where):
    """The same of the calls on the packed cache, and of the cache's buffers, which its first call writes."""

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = _cache()
    sizes = q.qwm_cache_sizes(cache.cfg)
    device = _Device(monkeypatch)
    monkeypatch.setattr(q, "lib", Library)
    monkeypatch.setattr(q, "qwm_cache_sizes", lambda cfg: sizes)
    monkeypatch.setattr(q, "_dev_ptr", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(q, "_stream", lambda *a: 0)
    for count, call in ((1, lambda: q.qwm_attention(cache, x, stream=stream)),
                        (1, lambda: q.qwm_attention_ext(cache, x, stream=stream)),
                        (2, lambda: q.qwm_reconstruct(cache, 0, 5, "cuda", stream=stream)),
                        (2, lambda: q.qwm_top1_shift(cache, x, x, stream=stream)),
                        (q.NBUF, lambda: q.QuantKVCache(2, 64, 16, 16, 4, 4, 1000, stream=stream))):
        device.made.clear()
        call()
        assert device.made == [where] * count


def test_pages_without_a_bound_are_attended_to_whole(monkeypatch):
    """max_kv left out bounds nothing: it is what the tables can hold; a table or lengths without pages,
    which would be left out without a word, are refused."""
    x, cu = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    table, lens = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, pages = _cache(), _pages()
    device = _Device(monkeypatch)

    def bound(*a, **kw):
        device.launches.clear()
        q.qwm_attention_shared(cache, x, cu, 4, *a, **kw)
        return device.launches[0][1][12]

    assert bound(pages, table, lens) == 5 * 16
    assert bound(pages, table, lens, 7) == 7
    assert bound(pages, table, lens, max_kv=0) == 0
    assert bound() == 0
    for kw in (dict(table=table), dict(kv_len=lens), dict(pages=pages), dict(pages=pages, table=table)):
        with pytest.raises(ValueError):
            bound(**kw)


def test_more_rows_than_a_launch_takes_are_an_invalid_argument():
    """Rows times blocks of 64 heads (of queries and keys, or keys and values) end at 2^31 - 1; the call
    says so itself, not the launch."""
    many = dict(n=2**30, ldpos=2**30)
    assert _norm_rope(**many) == 1
    assert _norm_rope(n=2**31 - 1, ldpos=2**31, hq=1, hk=1) == 1
    assert _append(n=2**30) == 1
    assert _append(n=2**24, pages=dict(heads=4096, n_pages=1), ldk=4096 * 64, ldv=4096 * 64) == 1
