"""Host side of the calls on a paged cache at the edges of what their documentation allows.  CPU only:
no call here reaches a kernel."""
import ctypes

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
