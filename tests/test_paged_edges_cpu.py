"""Host side of the calls on a paged cache at the edges of what their documentation allows.  CPU only:
no call here reaches a kernel."""
import ctypes
import math

import numpy as np
import pytest

import decode_fathom_plan_b200 as fp
from decode_fathom_plan_b200 import build as fbuild


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fp.load_library()


def test_wait_limit_is_kept_and_given_back(lib):
    before = fp.fathom_set_wait_limit(7)
    assert before == 500000000
    assert fp.fathom_set_wait_limit(2 ** 64 - 1) == 7
    assert fp.fathom_set_wait_limit(before) == 2 ** 64 - 1


# ------------------------------------------- one workspace for a batch and every smaller one
FAKE = 0x10000      # aligned, never dereferenced


def cache(H, d, page=16):
    return fp.fathom_kv_cache(FAKE, FAKE, H * page * d, page * d, d, 1 << 20, page, H, d, fp.FATHOM_BF16)


def rows(heads, d):
    return fp.fathom_rows(FAKE, heads * d, d, heads, fp.FATHOM_BF16)


def attention_lacks(lib, H, G, d, n, max_len, prefix, nb):
    """Whether a call finds its workspace of nb bytes too small (its cache is refused after that)."""
    c, q = cache(H, d), rows(H * G, d)
    rc = lib.fathom_paged_attention(ctypes.byref(c), ctypes.byref(q), FAKE, 1 << 20, FAKE, n, max_len, prefix, 0.1,
                                    0.0, 0, ctypes.byref(q), FAKE, nb, 0)
    assert rc in (fp.FATHOM_ERR_WORKSPACE, fp.FATHOM_ERR_INVALID_ARG)
    return rc == fp.FATHOM_ERR_WORKSPACE


def sparse_lacks(lib, H, G, d, n, k, nb):
    c, q = cache(H, d), rows(H * G, d)
    rc = lib.fathom_sparse_attention_paged(ctypes.byref(c), ctypes.byref(q), FAKE, k, FAKE, 1 << 20, FAKE, n, 0.1,
                                           0.0, 0, ctypes.byref(q), FAKE, nb, 0)
    assert rc in (fp.FATHOM_ERR_WORKSPACE, fp.FATHOM_ERR_INVALID_ARG)
    return rc == fp.FATHOM_ERR_WORKSPACE


@pytest.mark.parametrize("H,G,d,most,max_len,prefix", [
    (8, 4, 128, 40, 34816, 32768), (8, 4, 128, 64, 34816, 32768), (4, 5, 128, 23, 5309, 5008),
    (1, 1, 64, 700, 9000, 8192), (2, 8, 256, 90, 4096, 4096), (8, 8, 128, 321, 2100, 2048),
    (1, 7, 32, 2000, 66000, 65536), (8, 4, 128, 33, 1000, 0), (3, 3, 192, 130, 700, 640)])
def test_attention_workspace_serves_every_smaller_batch(lib, H, G, d, most, max_len, prefix):
    size = fp.fathom_paged_attention_workspace_bytes
    c = cache(H, d)
    nb = size(c, most, G, max_len, prefix)
    last = 0
    for n in range(1, most + 1):
        assert not attention_lacks(lib, H, G, d, n, max_len, prefix, nb), n
        mine = size(c, n, G, max_len, prefix)
        assert last <= mine <= nb and not attention_lacks(lib, H, G, d, n, max_len, prefix, mine)
        last = mine
    # and smaller prefixes and bounds of the lengths, no prefix at all among them
    for n in {1, most // 2, most - 1, most} - {0}:
        for part in (0, 16, prefix // 3 // 16 * 16, max(0, prefix - 16), prefix):
            for longest in {max(1, part), max(part, max_len // 2), max_len}:
                if part <= min(prefix, longest):
                    assert not attention_lacks(lib, H, G, d, n, longest, part, nb), (n, part, longest)
                    assert size(c, n, G, longest, part) <= nb


@pytest.mark.parametrize("H,G,d,most,k", [(8, 4, 128, 64, 2048), (8, 4, 128, 64, 512), (1, 1, 32, 3000, 700),
                                          (2, 7, 256, 40, 4096), (8, 8, 96, 100, 128), (1, 3, 64, 900, 129)])
def test_sparse_workspace_serves_every_smaller_batch(lib, H, G, d, most, k):
    size = fp.fathom_sparse_attention_paged_workspace_bytes
    nb = size(most, H * G, d, k)
    last = 0
    for n in range(1, most + 1):
        assert not sparse_lacks(lib, H, G, d, n, k, nb), n
        mine = size(n, H * G, d, k)
        assert last <= mine <= nb and not sparse_lacks(lib, H, G, d, n, k, mine)
        last = mine
        for fewer in (1, 64, 129, 257, 385, 513, k // 3, k // 2, k - 1):
            if 1 <= fewer < k:
                assert not sparse_lacks(lib, H, G, d, n, fewer, nb), (n, fewer)
                assert size(n, H * G, d, fewer) <= nb


def test_a_valid_size_is_never_zero(lib):
    for k in (1, 64, 128):
        assert fp.fathom_sparse_attention_paged_workspace_bytes(1, 1, 32, k) > 0
    assert fp.fathom_sparse_attention_paged_workspace_bytes(1, 1, 32, 0) == 0
    assert fp.fathom_paged_attention_workspace_bytes(cache(1, 32), 1, 1, 1) > 0


# -------------------------------------------------------------- lengths near the end of 32 bits
def test_bounds_of_the_lengths_that_a_key_number_cannot_pass_are_refused(lib):
    """Key numbers are int32 and run up to a block past the last key."""
    c, q, most = cache(1, 32), rows(1, 32), 2 ** 31 - 2 ** 16

    def call(max_len, prefix=0):
        return lib.fathom_paged_attention(ctypes.byref(c), ctypes.byref(q), FAKE, 1 << 27, FAKE, 1, max_len, prefix,
                                          0.1, 0.0, 0, ctypes.byref(q), 0, 0, 0)

    size = fp.fathom_paged_attention_workspace_bytes
    for heads, longest in ((65535, 2 ** 21 - 64), (128, 2 ** 30 - 128)):      # blocks of 64 of all KV heads
        many, h = cache(heads, 32), rows(heads, 32)
        for n, rc in ((longest, fp.FATHOM_ERR_WORKSPACE), (longest + 2 ** 12, fp.FATHOM_ERR_INVALID_ARG)):
            assert lib.fathom_paged_attention(ctypes.byref(many), ctypes.byref(h), FAKE, 1 << 27, FAKE, 1, n, 0, 0.1,
                                              0.0, 0, ctypes.byref(h), 0, 0, 0) == rc
            assert (size(many, 1, 1, n) > 0) == (rc == fp.FATHOM_ERR_WORKSPACE)
    assert call(most) == call(most, most) == fp.FATHOM_ERR_WORKSPACE and size(c, 1, 1, most, most) > 0
    for longer in (most + 1, 2 ** 31 - 1):
        assert call(longer) == call(longer, most) == fp.FATHOM_ERR_INVALID_ARG
        assert size(c, 1, 1, longer) == size(c, 1, 1, longer, 16) == 0


# ------------------------------------------------------------------ rotation over pair numbers
def yarn_index(rd, base, factor, length, fast, slow):
    """Radians per position, pair by pair from the formula."""
    def number(turns):          # of the pair that turns so often over the original context
        return rd * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
    low, high = max(math.floor(number(fast)), 0), min(math.ceil(number(slow)), rd - 1)
    if low == high:
        high += 0.001
    out = []
    for i in range(rd // 2):
        stretched = min(max((i - low) / (high - low), 0.0), 1.0)
        f = base ** (-2 * i / rd)
        out.append(f / factor * stretched + f * (1 - stretched))
    return np.array(out), low, high


@pytest.mark.parametrize("rd,base,factor,length,fast,slow", [
    (128, 1e6, 8.0, 32768, 32.0, 1.0), (64, 1e4, 40.0, 4096, 32.0, 1.0), (128, 5e5, 4.0, 8192, 16.0, 2.0),
    (2, 1e4, 2.0, 4096, 32.0, 1.0), (128, 1e4, 2.0, 16, 32.0, 1.0), (128, 1e4, 2.0, 10 ** 9, 32.0, 1.0),
    (96, 1e6, 1.0, 32768, 32.0, 1.0)])
def test_yarn_over_pair_numbers(lib, rd, base, factor, length, fast, slow):
    code = fp.RotaryTable._SCALINGS["yarn_index"]
    got, mag = fp.fathom_rotary_turns(rd, base, code, factor, length, fast, slow)
    want, _, _ = yarn_index(rd, base, factor, length, fast, slow)
    assert np.allclose(got.numpy() * 2 * math.pi, want, rtol=1e-12, atol=0)
    assert abs(mag - (0.1 * math.log(factor) + 1)) <= 2.0 ** -23


def test_yarn_over_pair_numbers_worked_by_hand(lib):
    """128 channels, base 1e6, 32768, betas 32 and 1: n(32) = 128*ln(162.97)/27.63 = 23.6 and
    n(1) = 128*ln(5215.2)/27.63 = 39.6, so pair 31 is 8/17 of the way from 23 to 40."""
    got, _ = fp.fathom_rotary_turns(128, 1e6, fp.FATHOM_ROTARY_YARN_INDEX, 8.0, 32768, 32.0, 1.0)
    f = 1e6 ** (-np.arange(0, 128, 2) / 128)
    ratio = got.numpy() * 2 * math.pi / f
    assert np.allclose(ratio[[0, 23, 31, 40, 63]], [1, 1, 9 / 17 + 8 / 17 / 8, 1 / 8, 1 / 8], rtol=1e-12)
    assert yarn_index(128, 1e6, 8.0, 32768, 32.0, 1.0)[1:] == (23, 40)


@pytest.mark.parametrize("args", [(64, 1.0, 4, 2.0, 4096, 32.0, 1.0), (64, 0.5, 4, 2.0, 4096, 32.0, 1.0),
                                  (64, 1e4, 4, 2.0, 4096, 32.0, 0.0), (64, 1e4, 4, 2.0, 4096, 32.0, -1.0),
                                  (64, 1e4, 4, 2.0, 0, 32.0, 1.0), (64, 1e4, 4, 0.5, 4096, 32.0, 1.0),
                                  (64, 1e4, 4, 2.0, 4096, 1.0, 1.0), (64, 1e4, 4, 2.0, 1, 32.0, 1.0),
                                  (64, 2.0, 4, 2.0, 10 ** 9, 32.0, 1.0), (64, 1e4, 5, 2.0, 4096, 32.0, 1.0)])
def test_bad_yarn_over_pair_numbers_is_refused(lib, args):
    with pytest.raises(fp.FathomError):
        fp.fathom_rotary_turns(*args)


@pytest.mark.parametrize("freq", [[], [1.0] * 33, [[1.0]], [math.nan], [1.0, math.inf]])
def test_bad_frequencies_are_refused(freq):
    with pytest.raises(ValueError):
        fp.RotaryTable.from_frequencies(freq, 64)
    with pytest.raises(ValueError):
        fp.RotaryTable.from_frequencies([1.0], 64, magnitude=math.inf)


# -------------------------------------------------------------------------- the native module
def test_module_is_rebuilt_for_another_torch(lib, monkeypatch):
    assert fbuild.binding_up_to_date() and not fbuild.binding_lacks()
    monkeypatch.setattr(fbuild, "torch_mark", lambda: b"built for torch 0.0.0;")
    assert not fbuild.binding_up_to_date()


@pytest.mark.parametrize("lack", ["torch", "headers", "compiler"])
def test_library_is_built_where_the_module_cannot_be(lib, monkeypatch, tmp_path, capsys, lack):
    from torch.utils import cpp_extension
    stale = tmp_path / "_binding.so"
    stale.write_bytes(b"of another torch")
    monkeypatch.setattr(fbuild, "BINDING", str(stale))
    if lack == "torch":
        monkeypatch.setattr(fbuild, "torch_mark", lambda: b"")
        stale.unlink()
    elif lack == "headers":
        monkeypatch.setattr(cpp_extension, "include_paths", lambda *a, **k: [str(tmp_path)])
    else:
        monkeypatch.setenv("CXX", "no-such-compiler")
    assert fbuild.build() == fbuild.LIB
    assert "is not built" in capsys.readouterr().err
    assert not stale.exists()
