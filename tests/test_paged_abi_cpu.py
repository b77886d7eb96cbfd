"""Host side of the calls on a paged cache: refusals before any kernel,
workspace sizes, rotation tables.  CPU only: no call here reaches a kernel."""
import ctypes
import math

import numpy as np
import pytest
import torch

import decode_fathom_plan_b200 as fp
from decode_fathom_plan_b200 import build as fbuild
from tests import paged_oracle as po

FAKE = 0x10000      # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fp.load_library()


def cache(**kw):
    c = fp.fathom_kv_cache(FAKE, FAKE, 8 * 16 * 128, 16 * 128, 128, 64, 16, 8, 128, fp.FATHOM_BF16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rows(heads=8, dtype=fp.FATHOM_BF16, **kw):
    r = fp.fathom_rows(FAKE, heads * 128, 128, heads, dtype)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def table(**kw):
    t = fp.fathom_rotary(FAKE, 128, 0, 1.0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("kind,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
@pytest.mark.parametrize("rd", [4, 64, 128])
def test_rotation_tables(lib, kind, factor, rd):
    code = fp.RotaryTable._SCALINGS[kind]
    got, mag = fp.fathom_rotary_turns(rd, 1e6, code, factor, 32768, 32.0, 1.0)
    freq, want_mag = po.turns(rd, 1e6, kind, factor, 32768, 32.0, 1.0)
    assert np.allclose(got.numpy() * 2 * math.pi, freq, rtol=1e-12, atol=0)
    assert abs(mag - want_mag) <= 2.0 ** -24 * want_mag


@pytest.mark.parametrize("args", [(0,), (3,), (-2,), (64, 0.0), (64, -1.0), (64, math.inf),
                                  (64, 1e4, 4), (64, 1e4, -1), (64, 1e4, 1, 0.5),
                                  (64, 1e4, 1, math.nan), (2, 1e4, 2, 2.0), (64, 1e4, 3, 2.0, 0),
                                  (64, 1e4, 3, 2.0, 4096, 1.0, 1.0)])
def test_bad_rotation_tables_are_refused(lib, args):
    with pytest.raises(fp.FathomError):
        fp.fathom_rotary_turns(*args)


def norm_rope(lib, T=4, d=128, pos=FAKE, rot=None, wq=0, wk=0, eps=1e-6, q=None, qo=None, k=None, ko=None):
    ref = lambda x: None if x is None else ctypes.byref(x)   # noqa: E731
    return lib.fathom_qk_norm_rope(T, d, pos, ref(rot), wq, wk, eps, ref(q), ref(qo), ref(k), ref(ko), 0)


def test_norm_rope_refusals(lib):
    r = rows()
    bad = fp.FATHOM_ERR_INVALID_ARG
    assert norm_rope(lib) == bad                                     # neither q nor k
    assert norm_rope(lib, q=r) == bad                                # q without q_out
    assert norm_rope(lib, q=r, qo=r, ko=r) == bad
    assert norm_rope(lib, q=r, qo=rows(heads=4)) == bad
    assert norm_rope(lib, q=r, qo=r, k=rows(dtype=fp.FATHOM_F16), ko=r) == bad
    assert norm_rope(lib, q=r, qo=r, wk=FAKE) == bad                 # a weight of rows that are not there
    assert norm_rope(lib, T=-1, q=r, qo=r) == bad
    for d in (0, 16, 48, 288):
        assert norm_rope(lib, d=d, q=r, qo=r) == bad
    for eps in (-1.0, math.inf, math.nan):
        assert norm_rope(lib, eps=eps, q=r, qo=r) == bad
    assert norm_rope(lib, pos=0, rot=table(), q=r, qo=r) == bad
    for kw in (dict(turns=0), dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130),
               dict(interleaved=2), dict(magnitude=math.inf), dict(turns=FAKE + 4)):
        assert norm_rope(lib, rot=table(**kw), q=r, qo=r) == bad
    for kw in (dict(data=0), dict(data=FAKE + 1), dict(n_heads=0), dict(dtype=3), dict(dtype=-1)):
        assert norm_rope(lib, q=rows(**kw), qo=r) == bad
    assert norm_rope(lib, T=0, q=r, qo=r, rot=table()) == fp.FATHOM_OK   # nothing to do


BAD_CACHES = [dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(page_size=4), dict(page_size=24),
              dict(page_size=2048), dict(n_pages=0), dict(n_kv_heads=0), dict(head_dim=48),
              dict(head_dim=288), dict(dtype=fp.FATHOM_F32), dict(page_stride=-8),
              dict(token_stride=132), dict(head_stride=4), dict(token_stride=136), dict(k=FAKE + 16),
              dict(v=FAKE + 16), dict(page_stride=8 * 128 * 16 + 8)]


def append(lib, c=None, T=4, k=None, v=None, seq=FAKE, pos=FAKE, pt=FAKE, n=2, stride=8, rot=None,
           eps=1e-6):
    c, k, v = c or cache(), k or rows(), v or rows()
    return lib.fathom_append_kv(ctypes.byref(c), T, ctypes.byref(k), ctypes.byref(v), seq, pos, pt, n,
                                stride, None if rot is None else ctypes.byref(rot), 0, eps, 0)


def test_append_refusals(lib):
    # the cache's addresses are asked for last: with no GPU (or as here none of
    # its memory) even a well-formed call is refused, so each refusal is its own
    # only up to that; a bad one must not get further
    bad = fp.FATHOM_ERR_INVALID_ARG
    for kw in BAD_CACHES:
        assert append(lib, cache(**kw)) == bad
    for kw in (dict(T=-1), dict(seq=0), dict(pos=0), dict(pt=0), dict(n=0), dict(stride=0),
               dict(k=rows(heads=4)), dict(v=rows(heads=4)), dict(k=rows(dtype=fp.FATHOM_F32)),
               dict(rot=table(rotary_dim=256)), dict(eps=-1.0), dict(T=0, c=cache())):
        assert append(lib, **kw) == bad


def attention(lib, c=None, q=None, out=None, pt=FAKE, stride=64, sl=FAKE, n=2, max_len=1000,
              prefix=0, scale=0.1, cap=0.0, ws=FAKE, nb=1 << 30):
    c, q, out = c or cache(), q or rows(32), out or rows(32)
    return lib.fathom_paged_attention(ctypes.byref(c), ctypes.byref(q), pt, stride, sl, n, max_len,
                                      prefix, scale, cap, 0, ctypes.byref(out), ws, nb, 0)


def sparse(lib, c=None, q=None, out=None, idx=FAKE, k=64, pt=FAKE, stride=64, sl=FAKE, n=2, scale=0.1,
           cap=0.0, ws=FAKE, nb=1 << 30):
    c, q, out = c or cache(), q or rows(32), out or rows(32)
    return lib.fathom_sparse_attention_paged(ctypes.byref(c), ctypes.byref(q), idx, k, pt, stride, sl,
                                             n, scale, cap, 0, ctypes.byref(out), ws, nb, 0)


def test_attention_refusals(lib):
    bad = fp.FATHOM_ERR_INVALID_ARG
    for call in (attention, sparse):
        for kw in BAD_CACHES:
            assert call(lib, cache(**kw)) == bad
        for kw in (dict(pt=0), dict(stride=0), dict(sl=0), dict(n=0), dict(n=65536),
                   dict(scale=math.nan), dict(cap=-1.0), dict(cap=math.inf),
                   dict(q=rows(32, fp.FATHOM_F16)), dict(out=rows(32, fp.FATHOM_F32)),
                   dict(q=rows(30), out=rows(30)), dict(q=rows(72), out=rows(72)),
                   dict(out=rows(16)), dict(q=rows(32, data=FAKE + 2)),
                   dict(q=rows(32, token_stride=4100)), dict(out=rows(32, head_stride=132))):
            assert call(lib, **kw) == bad
    for kw in (dict(max_len=0), dict(max_len=1025), dict(prefix=-16), dict(prefix=8),
               dict(prefix=1008)):
        assert attention(lib, **kw) == bad
    for kw in (dict(idx=0), dict(k=0)):
        assert sparse(lib, **kw) == bad


def test_attention_refusals_beside_a_call_that_lacks_only_its_workspace(lib):
    bad, lacking = fp.FATHOM_ERR_INVALID_ARG, fp.FATHOM_ERR_WORKSPACE
    for call, kw in ((attention, dict(max_len=1000)), (sparse, dict(k=4096))):
        def at(**more):
            return call(lib, **{**kw, "ws": 0, **more})
        assert at() == lacking
        for cap in (1e-30, 50.0, 16384.0):
            assert at(cap=cap) == lacking
        for cap in (-1e-30, 16385.0, 3e38, math.inf, math.nan, 1e-40):
            assert at(cap=cap) == bad
        for scale in (math.inf, math.nan, 3e38, -3e38):
            assert at(scale=scale) == bad
        for scale in (1e38, 0.0, -0.1):
            assert at(scale=scale) == lacking
        assert at(cap=1.0, scale=2e38) == bad
        for c in (dict(token_stride=136), dict(head_stride=136), dict(page_stride=136), dict(head_dim=48)):
            assert at(c=cache(**c)) == bad
        for r in (dict(token_stride=4100), dict(head_stride=132), dict(data=FAKE + 8)):
            assert at(q=rows(32, **r)) == bad and at(out=rows(32, **r)) == bad
        for r in (dict(token_stride=4104), dict(head_stride=136), dict(data=FAKE + 16)):
            assert at(q=rows(32, **r), out=rows(32, **r)) == lacking
    c = cache()
    assert fp.fathom_paged_attention_workspace_bytes(c, 2, 4, 1000) > 0
    for kw in (dict(token_stride=136), dict(head_stride=136), dict(page_stride=136)):
        assert fp.fathom_paged_attention_workspace_bytes(cache(**kw), 2, 4, 1000) == 0


def test_workspace_sizes(lib):
    c = cache()
    size = fp.fathom_paged_attention_workspace_bytes
    assert size(c, 1, 4, 131072) > 0
    assert size(c, 64, 4, 34816, 32768) > size(c, 1, 4, 34816, 32768) > 0
    for bad in ((0, 4, 100, 0), (1, 0, 100, 0), (1, 9, 100, 0), (1, 4, 0, 0), (1, 4, 100, -16),
                (1, 4, 100, 8), (1, 4, 100, 112), (65536, 4, 100, 0)):
        assert size(c, *bad) == 0
    assert size(cache(page_size=12), 1, 4, 100) == 0
    size = fp.fathom_sparse_attention_paged_workspace_bytes
    assert size(1, 32, 128, 2048) >= 32 * 16 * 130 * 4
    for bad in ((0, 32, 128, 64), (1, 0, 128, 64), (1, 32, 100, 64), (1, 32, 128, 0)):
        assert size(*bad) == 0


def test_binding_refuses_what_the_call_would_misread(lib):
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fp.fathom_qk_norm_rope(x, None, None, x, None)             # host rows
    with pytest.raises(ValueError):
        fp.fathom_qk_norm_rope(None, None, None, None, None)
    with pytest.raises(ValueError):
        fp.fathom_qk_norm_rope(x, None, None, None, None)          # q without q_out
    with pytest.raises(ValueError):
        fp.fathom_append_kv(cache(), x, x[:2], None, None, None)   # v of fewer tokens
    with pytest.raises(ValueError):
        fp.fathom_append_kv(cache(head_dim=64), x, x, None, None, None)
    with pytest.raises(ValueError):
        fp.PagedKV.from_tensors(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64))   # not pinned
    with pytest.raises(ValueError):
        fp.PagedKV.from_tensors(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 8, 64))
    with pytest.raises(ValueError):
        fp.RotaryTable(64, 128)
    with pytest.raises(ValueError):
        fp.RotaryTable(64, scaling="other")
