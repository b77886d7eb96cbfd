"""Calls on a paged cache against plain float64 forms: norm and rotation of
heads, paged append, attention with and without a shared prefix, attention
over selected keys, and a decode step that runs them with the key scan."""
import math

import numpy as np
import pytest
import torch

import decode_fathom_plan_b200 as fp
from tests import paged_oracle as po

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp.load_library()
    torch.cuda.set_device(0)
    fp.fathom_last_device_status()


def status():
    return fp.fathom_last_device_status()


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def check(got, want, tol, what=""):
    got = po.f64(got)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.3g} of the "
                           f"tolerance at {np.argwhere(bad)[:3].tolist()}: {got[bad][:3]} for {want[bad][:3]}")


# ------------------------------------------------------------- norm and rotation
ROPE = [
    # T, hq, hkv, d, dtype, k_out, rotary_dim, interleaved, scaling, factor, norm, first position
    (1, 32, 8, 128, BF16, BF16, 128, False, "none", 1.0, True, 131071),
    (3, 4, 1, 32, F16, F32, 32, True, "linear", 4.0, True, 0),
    (7, 6, 2, 64, BF16, F32, 32, False, "yarn", 8.0, False, 1 << 20),
    (5, 3, 3, 96, F16, F16, 96, False, "ntk", 2.0, True, 40000),
    (33, 2, 1, 160, BF16, F16, 80, True, "none", 1.0, True, 7),
    (2, 8, 1, 192, F32, F32, 192, False, "yarn", 4.0, True, 1 << 30),
    (9, 1, 1, 224, F16, BF16, 16, True, "none", 1.0, False, 5),
    (4, 5, 2, 256, BF16, BF16, 256, False, "none", 1.0, True, 1000),
    (6, 2, 2, 64, F16, F16, 10, False, "none", 1.0, True, 99),      # pairs one at a time
    (6, 2, 2, 256, BF16, F32, 250, True, "none", 1.0, True, 99),
    (2000, 5, 2, 64, BF16, F32, 64, False, "none", 1.0, True, 0),   # tiles of tokens
    (1027, 3, 1, 96, F16, F16, 48, True, "linear", 2.0, True, 3),
    (300, 32, 8, 128, F32, F32, 128, False, "none", 1.0, True, 100),
]


@pytest.mark.parametrize("T,hq,hk,d,dtype,kdtype,rd,inter,scaling,factor,norm,first", ROPE)
def test_norm_rope(T, hq, hk, d, dtype, kdtype, rd, inter, scaling, factor, norm, first):
    seed = T + d + rd
    qkv = randn([T, hq + 2 * hk, d], dtype, seed, 3.0).cuda()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    qw, kw = ((1 + 0.3 * randn([d], F32, seed + i)).to(dtype).cuda() if norm else None for i in (1, 2))
    pos = (first + 3 * torch.arange(T)).to(torch.int32).cuda()
    tab = fp.RotaryTable(d, rd, 1e6, inter, scaling, factor, 32768)
    q_out = torch.full([T, hq, d], math.nan, dtype=dtype, device="cuda")
    k_out = torch.full([hk, T, d], math.nan, dtype=kdtype, device="cuda").transpose(0, 1)
    fp.fathom_qk_norm_rope(q, k, pos, q_out, k_out, tab, qw, kw)
    freq, mag = po.turns(rd, 1e6, scaling, factor, 32768)
    for x, w, out, what in ((q, qw, q_out, "q"), (k, kw, k_out, "k")):
        y, size = po.norm_rope(po.f64(x), pos.cpu().numpy().astype(np.float64),
                               None if w is None else po.f64(w), 1e-6, freq, mag, inter)
        check(out, y, po.norm_rope_tolerance(y, size, out.dtype), what)
    assert status() == fp.FATHOM_OK


@pytest.mark.parametrize("shift", [0, 1, 4])
def test_norm_rope_unaligned_rows_in_place_and_one_sided(shift):
    T, h, d = 5, 3, 64
    base = torch.zeros(T * h * d + 16, dtype=BF16, device="cuda")
    x = base[shift:shift + T * h * d].view(T, h, d)
    src = randn([T, h, d], BF16, 5)
    x.copy_(src)
    w = torch.ones(d + 8, dtype=BF16, device="cuda")[shift % 2:shift % 2 + d]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    tab = fp.RotaryTable(d)
    fp.fathom_qk_norm_rope(None, x, pos, None, x, tab, None, w)
    y, size = po.norm_rope(po.f64(src), np.arange(T, dtype=np.float64), np.ones(d), 1e-6, po.turns(d)[0])
    check(x, y, po.norm_rope_tolerance(y, size, BF16))
    assert (base[:shift] == 0).all() and (base[shift + T * h * d:] == 0).all()


def test_norm_rope_of_positions_below_zero_and_at_the_end_of_the_range():
    pos = torch.tensor([-1, -7, -2 ** 31, 2 ** 31 - 1, 0, 1 << 24], dtype=torch.int32, device="cuda")
    for d, inter in ((128, False), (96, True)):
        x = randn([6, 2, d], F32, 4).cuda()
        guard = torch.full([6 * 2 * d + 64], 7.0, device="cuda")
        out = guard[:6 * 2 * d].view(6, 2, d)
        fp.fathom_qk_norm_rope(x, None, pos, out, None, fp.RotaryTable(d, base=1e6, interleaved=inter))
        p = pos.cpu().numpy().astype(np.float64)
        y, size = po.norm_rope(po.f64(x), p, None, 1e-6, po.turns(d, 1e6)[0], 1.0, inter)
        # the reference's own angle is a float64 product of some 2^31 radians: 2^-22 of a radian
        check(out, y, po.norm_rope_tolerance(y, size, F32) + 2.0 ** -21 * size)
        assert (guard[6 * 2 * d:] == 7.0).all()


def test_norm_rope_without_rotation_or_norm():
    x = randn([4, 2, 96], F16, 1).cuda()
    out = torch.empty([4, 2, 96], dtype=F32, device="cuda")
    fp.fathom_qk_norm_rope(x, None, None, out, None)
    assert torch.equal(out, x.float())
    w = randn([96], F16, 2).cuda()
    fp.fathom_qk_norm_rope(x, None, None, out, None, q_weight=w)
    y, size = po.norm_rope(po.f64(x), None, po.f64(w))
    check(out, y, po.norm_rope_tolerance(y, size, F32))
    zero = torch.zeros([1, 1, 96], dtype=F16, device="cuda")      # a norm of nothing is nothing
    fp.fathom_qk_norm_rope(zero, None, None, out[:1, :1], None, q_weight=w)
    assert (out[:1, :1] == 0).all()
    fp.fathom_qk_norm_rope(x[:0], None, None, out[:0], None)      # no tokens
    y, size = po.norm_rope(po.f64(x), None, po.f64(w))
    assert status() == fp.FATHOM_OK


def test_norm_rope_keeps_infinities_and_nan_in_their_heads():
    x = randn([2, 3, 64], BF16, 8).cuda()
    x[0, 1, 5] = math.nan
    x[1, 2, 7] = math.inf
    w = torch.ones(64, dtype=BF16, device="cuda")
    out = torch.empty_like(x)
    fp.fathom_qk_norm_rope(x, None, torch.arange(2, dtype=torch.int32, device="cuda"), out, None,
                           fp.RotaryTable(64), w)
    fine = torch.isfinite(out).all(-1)
    assert fine.tolist() == [[True, False, True], [True, True, False]]


# ------------------------------------------------------------------------ append
def make_pool(pages, H, page, d, dtype, token_major, fill=math.nan, residency="device"):
    kv = fp.PagedKV(pages, page, H, d, dtype, "token_major" if token_major else "head_major", residency)
    kv.k.fill_(fill)
    kv.v.fill_(fill)
    return kv


APPEND = [
    # tokens per sequence, first positions, H, d, in, cache, page, token_major, rotary_dim, interleaved, norm
    ([1, 1, 1], [0, 7, 16], 8, 128, BF16, BF16, 16, False, 128, False, True),
    ([5, 0, 17, 1], [0, 3, 8, 31], 2, 64, F16, F16, 8, True, 32, True, False),
    ([40], [100], 1, 32, F32, BF16, 32, False, 32, False, True),
    ([9, 30], [1000, 2], 3, 96, BF16, F16, 128, True, 18, False, True),
    ([700, 600], [0, 13], 2, 256, F16, F16, 64, False, 256, True, True),
    ([1200, 3], [5, 0], 4, 192, BF16, BF16, 1024, False, 96, False, False),
]


@pytest.mark.parametrize("counts,firsts,H,d,dtype,cdtype,page,tm,rd,inter,norm", APPEND)
@pytest.mark.parametrize("residency", ["device", "host_mapped"])
def test_append(counts, firsts, H, d, dtype, cdtype, page, tm, rd, inter, norm, residency):
    rng = np.random.default_rng(sum(counts) + d)
    need = [-(-(f + c) // page) for f, c in zip(firsts, counts)]
    pages = sum(need) + 2
    perm = rng.permutation(pages).astype(np.int32)
    tab = np.full((len(counts), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        tab[b, :n] = perm[at:at + n]
        at += n
    seq = np.concatenate([np.full(c, b) for b, c in enumerate(counts)] + [np.full(3, -1)]).astype(np.int32)
    pos = np.concatenate([f + np.arange(c) for f, c in zip(firsts, counts)] + [[-5, 0, 1 << 30]]).astype(np.int32)
    order = rng.permutation(len(seq))
    seq, pos = seq[order], pos[order]
    T = len(seq)
    k, v = randn([H, T, d], dtype, d, 2.0).cuda().transpose(0, 1), randn([T, H, d], dtype, d + 1).cuda()
    w = (1 + 0.3 * randn([d], F32, 3)).to(dtype).cuda() if norm else None
    kv = make_pool(pages, H, page, d, cdtype, tm, 3.0, residency)
    rot = fp.RotaryTable(d, rd, 1e5, inter)
    fp.fathom_append_kv(kv.desc, k, v, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                        torch.from_numpy(tab).cuda(), rot, w)
    torch.cuda.synchronize()
    assert status() == fp.FATHOM_OK
    y, size = po.norm_rope(po.f64(k), pos.astype(np.float64), None if w is None else po.f64(w), 1e-6,
                           po.turns(rd, 1e5)[0], 1.0, inter)
    tol = po.norm_rope_tolerance(y, size, cdtype)
    want_k, want_v = np.full(kv.k.shape, 3.0), np.full(kv.k.shape, 3.0)
    tol_k = np.zeros(kv.k.shape)
    for t in range(T):
        if seq[t] >= 0:
            p, s = tab[seq[t], pos[t] // page], pos[t] % page
            want_k[p, :, s], tol_k[p, :, s] = y[t], tol[t]
            want_v[p, :, s] = po.f64(v[t].to(cdtype))
    check(kv.k, want_k, tol_k, "keys")
    assert np.array_equal(po.f64(kv.v), want_v)


@pytest.mark.parametrize("seq,pos,page0", [(2, 0, 0), (0, -1, 0), (0, 32, 0), (0, 2 ** 31 - 1, 0),
                                           (0, 3, 9), (0, 3, -1), (0, 3, -2 ** 31)])
def test_append_refuses_what_the_device_sees(seq, pos, page0):
    kv = make_pool(4, 2, 16, 64, BF16, False, 1.0)
    tab = torch.tensor([[page0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    x = randn([2, 2, 64], BF16, 1).cuda()
    fp.fathom_append_kv(kv.desc, x, x, torch.tensor([seq, 1], dtype=torch.int32, device="cuda"),
                        torch.tensor([pos, 5], dtype=torch.int32, device="cuda"), tab)
    assert status() == fp.FATHOM_ERR_INVALID_ARG and status() == fp.FATHOM_OK
    assert torch.equal(kv.k[2, :, 5], x[1]) and torch.equal(kv.v[2, :, 5], x[1])   # the good token
    kv.k[2, :, 5] = kv.v[2, :, 5] = 1.0
    assert (kv.k == 1.0).all() and (kv.v == 1.0).all()                             # nothing else


# --------------------------------------------------------------------- attention
class Batch:
    """Sequences of given lengths over scattered pages; every slot that no sequence holds is NaN."""

    def __init__(self, lens, prefix, H, G, d, page, dtype, tm, seed, key_scale=1.0, spare=1, residency="device"):
        rng = np.random.default_rng(seed)
        self.lens, self.prefix, self.H, self.G, self.d, self.page, self.dtype = lens, prefix, H, G, d, page, dtype
        shared = prefix // page
        need = [max(0, -(-(n - prefix) // page)) for n in lens]
        pages = shared + sum(need) + spare
        perm = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), shared + max(need + [1]) + 1), -7, np.int32)
        self.table[:, :shared] = perm[:shared]
        at = shared
        for b, n in enumerate(need):
            self.table[b, shared:shared + n] = perm[at:at + n]
            at += n
        k = randn([pages, H, page, d], dtype, seed, key_scale)
        v = randn([pages, H, page, d], dtype, seed + 1)
        used = np.zeros((pages, page), bool)
        for b, n in enumerate(lens):
            j = np.arange(n if n else 0)
            used[self.table[b, j // page], j % page] = True
        if prefix:
            used[perm[:shared]] = True
        dead = torch.from_numpy(~used)[:, None, :, None]
        k, v = k.masked_fill(dead, math.nan), v.masked_fill(dead, math.nan)
        self.kv = make_pool(pages, H, page, d, dtype, tm, residency=residency)
        self.kv.k.copy_(k)
        self.kv.v.copy_(v)
        self.k64, self.v64 = po.f64(k), po.f64(v)
        self.q = randn([len(lens), H * G, d], dtype, seed + 2).cuda()
        self.out = torch.full_like(self.q, math.nan)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.table_t = torch.from_numpy(self.table).cuda()
        self.scale = 1.0 / math.sqrt(d)

    def slopes(self):
        n = self.H * self.G
        return 2.0 ** (-8.0 * torch.arange(1, n + 1, dtype=torch.float32) / n)

    def attention(self, max_len=None, cap=0.0, slopes=None, ws=None, stream=None):
        max_len = max_len or max(self.lens + [1])
        need = fp.fathom_paged_attention_workspace_bytes(self.kv.desc, len(self.lens), self.G, max_len, self.prefix)
        self.ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda") if ws is None else ws
        fp.fathom_paged_attention(self.kv.desc, self.q, self.table_t, self.lens_t, max_len, self.out, self.ws,
                                  self.scale, self.prefix, cap, slopes, stream)

    def expect(self, cap=0.0, slopes=None, rows=None, idx=None, round_p=True):
        """(out, tolerance) of the given rows (all)."""
        hq = self.H * self.G
        want, tol = np.zeros((len(self.lens), hq, self.d)), np.zeros((len(self.lens), hq, self.d))
        sl = np.zeros(hq) if slopes is None else po.f64(slopes)
        q = po.f64(self.q)
        step = po.HALF_STEP[self.dtype] if round_p else 0.0
        tiny = po.TINY[self.dtype] * 2.0 ** 8 if round_p else 0.0
        for b in range(len(self.lens)):
            for i in range(hq):
                if rows is not None and (b, i) not in rows:
                    continue
                j = np.arange(self.lens[b]) if idx is None else idx[b, i][idx[b, i] >= 0]
                ks = po.gather(self.k64, self.table[b], j, i // self.G, self.page)
                vs = po.gather(self.v64, self.table[b], j, i // self.G, self.page)
                o, e = po.attend(q[b, i], ks, vs, self.lens[b] - 1 - j, self.scale, cap, sl[i], step, tiny)
                want[b, i], tol[b, i] = o, e + po.HALF_STEP[self.dtype] * np.abs(o) * 1.01 + \
                    po.TINY[self.dtype] + 1e-30
        return want, tol


ATTENTION = [
    # lens, prefix, H, G, d, page, dtype, token_major, cap, slopes
    ([1], 0, 1, 1, 32, 8, BF16, False, 0.0, False),
    ([0, 2, 15, 16, 17], 0, 2, 4, 128, 16, BF16, False, 0.0, False),
    ([64, 65, 63], 0, 2, 3, 64, 8, F16, True, 0.0, False),
    ([1000, 1, 513], 0, 8, 4, 128, 16, BF16, False, 0.0, True),
    ([2000], 0, 2, 8, 96, 128, F16, False, 30.0, False),
    ([5, 300], 0, 1, 7, 160, 32, BF16, True, 50.0, True),
    ([129, 0], 0, 2, 2, 192, 16, F16, False, 0.0, True),
    ([700, 31], 0, 1, 5, 224, 64, BF16, False, 0.0, False),
    ([257, 1024], 0, 2, 8, 256, 16, F16, True, 20.0, False),
    ([3000, 17, 0, 1], 0, 2, 8, 64, 1024, BF16, False, 0.0, False),
    # a shared prefix: rows of a KV head from 1 to over 256, tails of nothing and more
    ([16], 16, 1, 1, 128, 16, BF16, False, 0.0, False),
    ([130, 128, 0, 145], 128, 2, 4, 128, 16, BF16, False, 0.0, False),
    ([8, 9, 12], 8, 1, 2, 64, 8, F16, True, 0.0, True),
    ([200, 193, 192], 192, 2, 8, 64, 64, BF16, False, 30.0, False),
    ([1000 + i for i in range(33)], 992, 1, 4, 128, 32, BF16, False, 0.0, False),
    ([520 + 3 * i for i in range(40)], 512, 1, 7, 128, 16, F16, True, 0.0, True),
    ([300 + i for i in range(20)], 296, 2, 5, 96, 8, BF16, False, 50.0, True),
    ([400 + 7 * i for i in range(9)], 400, 1, 8, 32, 16, F16, False, 0.0, False),
    ([2050, 2049, 0, 2048, 2500], 2048, 2, 6, 256, 16, BF16, False, 0.0, False),
    ([640 + i for i in range(35)], 640, 1, 4, 160, 128, F16, False, 0.0, True),
    ([1152 + i for i in range(17)], 1152, 1, 8, 192, 16, BF16, True, 20.0, False),
    ([64] * 70, 64, 1, 8, 64, 64, F16, False, 0.0, False),
]


@pytest.mark.parametrize("lens,prefix,H,G,d,page,dtype,tm,cap,slopes", ATTENTION)
def test_attention(lens, prefix, H, G, d, page, dtype, tm, cap, slopes):
    b = Batch(lens, prefix, H, G, d, page, dtype, tm, 11 + d + len(lens))
    sl = b.slopes().cuda() if slopes else None
    b.attention(cap=cap, slopes=sl)
    want, tol = b.expect(cap, sl)
    check(b.out, want, tol)
    assert status() == fp.FATHOM_OK
    first = b.out.clone()
    b.out.fill_(math.nan)
    b.attention(cap=cap, slopes=sl)
    assert torch.equal(b.out, first)          # the same sums in the same order
    # a wider bound than the longest sequence changes the split, not the result
    if max(lens):
        b.table_t = torch.nn.functional.pad(b.table_t, (0, 4096 // page), value=-9)
        b.attention(max_len=max(lens) + 3000, cap=cap, slopes=sl)
        check(b.out, want, tol)
        assert status() == fp.FATHOM_OK


def few_rows(b, n=12):
    """Some rows of a batch, the first, the last and the borders of 128-row blocks among them."""
    hq = b.H * b.G
    every = [(s, i) for s in range(len(b.lens)) for i in range(hq)]
    per = 128 // b.G                                    # sequences of a block
    border = [(s, i) for k in (1, 2, 3) for s in (k * per - 1, k * per) if s < len(b.lens) for i in (0, hq - 1)]
    rng = np.random.default_rng(n)
    return set(border + [every[0], every[-1]] + [every[j] for j in rng.choice(len(every), min(n, len(every)), replace=False)])


def check_rows(b, rows, cap=0.0, slopes=None):
    want, tol = b.expect(cap, slopes, rows=rows)
    at = tuple(np.array(sorted(rows)).T)
    check(b.out.cpu()[at], want[at], tol[at])


# prefixes whose repeated reads, 4 bytes * d * H * prefix * (sequences - 1), pass 8 MB: multiplied
# with the queries of all sequences at once
SHARED = [
    # lens, prefix, H, G, d, page, dtype, token_major, cap, slopes
    ([2100, 2049], 2048, 8, 1, 128, 16, BF16, False, 0.0, False),
    ([1000 + i for i in range(33)], 992, 2, 4, 128, 32, BF16, False, 0.0, False),
    ([512 + 3 * i for i in range(40)], 512, 1, 7, 128, 16, F16, True, 0.0, True),
    ([512] * 70, 512, 1, 8, 64, 64, F16, False, 0.0, False),
    ([1160 + i for i in range(20)], 1160, 2, 5, 96, 8, BF16, False, 50.0, True),
    ([4112 + 7 * i for i in range(9)], 4112, 2, 8, 32, 16, F16, False, 0.0, False),
    ([2050, 2049, 0, 2048, 2500], 2048, 2, 6, 256, 16, BF16, False, 0.0, False),
    ([640 + i for i in range(35)], 640, 1, 4, 160, 128, F16, False, 0.0, True),
    ([1152 + i for i in range(17)], 1152, 1, 8, 192, 16, BF16, True, 20.0, False),
    ([1024 + 500 * (i % 2) for i in range(12)], 1024, 1, 3, 224, 1024, F16, False, 0.0, False),
    ([136 + i % 5 for i in range(130)], 136, 1, 1, 128, 8, BF16, False, 0.0, True),
    ([8200, 0, 8192], 8192, 8, 2, 64, 16, BF16, True, 0.0, False),
    ([4096 + 11 * i for i in range(40)], 4096, 8, 4, 128, 256, BF16, False, 0.0, False),
    ([33000, 32768], 32768, 1, 8, 128, 16, F16, False, 30.0, True),
    ([16384 + i for i in range(3)], 16384, 4, 2, 256, 32, F16, False, 0.0, False),
]


@pytest.mark.parametrize("lens,prefix,H,G,d,page,dtype,tm,cap,slopes", SHARED)
def test_shared_prefix(lens, prefix, H, G, d, page, dtype, tm, cap, slopes):
    assert 4 * d * H * prefix * (len(lens) - 1) >= 8 << 20
    b = Batch(lens, prefix, H, G, d, page, dtype, tm, 31 + d + len(lens))
    sl = b.slopes().cuda() if slopes else None
    b.attention(cap=cap, slopes=sl)
    rows = few_rows(b)
    check_rows(b, rows, cap, sl)
    assert status() == fp.FATHOM_OK
    for s, n in enumerate(lens):
        assert n or (b.out[s] == 0).all()
    first = b.out.clone()
    for _ in range(4):
        b.out.fill_(math.nan)
        b.attention(cap=cap, slopes=sl)
        assert torch.equal(b.out, first)
    # the same batch with nothing said of the prefix: each sequence reads it for itself
    b.prefix = 0
    b.attention(cap=cap, slopes=sl)
    check_rows(b, rows, cap, sl)
    if max(lens) + 3000 < 40000:
        b.prefix = prefix
        b.table_t = torch.nn.functional.pad(b.table_t, (0, -(-3000 // page)), value=-9)
        b.attention(max_len=max(lens) + 3000, cap=cap, slopes=sl)
        check_rows(b, rows, cap, sl)
        assert status() == fp.FATHOM_OK


@pytest.mark.parametrize("page", [16, 128])
def test_shared_prefix_beside_many_own_keys(page):
    """Slots of a CTA that run apart from each other: the sums of every call are those of the first."""
    b = Batch([20000 + 4000 - 17 * i for i in range(15)], 20000 // page * page, 3, 2, 128, page, BF16, False, 77)
    b.attention()
    check_rows(b, few_rows(b, 6))
    first = b.out.clone()
    for _ in range(300):
        outs = []
        for _ in range(8):
            b.attention(ws=b.ws)
            outs.append(b.out.clone())
        assert all(torch.equal(o, first) for o in outs)
    assert status() == fp.FATHOM_OK


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (2, 256)])
def test_shared_prefix_of_growing_scores(dtype, G, d):
    """Every step of every slot renews its maximum and rescales its sums."""
    n, prefix, H = 16500, 16384, 8 if d < 256 else 4
    b = Batch([n, n - 7], prefix, H, G, d, 16, dtype, False, 3)
    ramp = torch.linspace(0.5, 24.0, n).to(dtype).cuda()
    for s, m in enumerate(b.lens):
        j = np.arange(m)
        pg, at = torch.from_numpy(b.table[s, j // 16]).long().cuda(), torch.from_numpy(j % 16).cuda()
        b.kv.k[pg, :, at] = ramp[:m, None, None].expand(m, H, d).contiguous()
    b.q.fill_(1.0)
    b.k64 = po.f64(b.kv.k)
    b.attention()
    check_rows(b, few_rows(b, 4))
    # and a scale below zero, under which they fall
    b.scale = -b.scale
    b.attention()
    for s, i in sorted(few_rows(b, 2)):
        ks, vs = (po.gather(p, b.table[s], np.arange(b.lens[s]), i // G, 16) for p in (b.k64, b.v64))
        q = po.f64(b.q)[s, i]
        want, err = po.attend(-q, ks, vs, np.zeros(b.lens[s]), -b.scale, p_step=po.HALF_STEP[dtype],
                              p_tiny=po.TINY[dtype] * 2.0 ** 8)
        check(b.out[s, i], want, err + po.HALF_STEP[dtype] * np.abs(want) * 1.01 + po.TINY[dtype])


def test_shared_prefix_refusals_on_the_device():
    b = Batch([2100, 2060, 2090], 2048, 8, 2, 64, 16, F16, False, 9)
    good = b.table_t.clone()
    b.attention()
    rows = few_rows(b)
    check_rows(b, rows)
    clean = b.out.clone()
    b.lens_t[1] = 2047                              # inside the prefix
    b.attention()
    assert status() == fp.FATHOM_ERR_INVALID_ARG
    assert (b.out[1] == 0).all() and torch.equal(b.out[[0, 2]], clean[[0, 2]])
    b.lens_t[1] = 2060
    for page in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1, b.kv.k.shape[0]):
        b.table_t[:, 77] = page
        b.attention()
        assert status() == fp.FATHOM_ERR_INVALID_ARG
        assert torch.isfinite(b.out).all()
        b.table_t.copy_(good)
    b.kv.v[b.table[0, 5], 3, 2, 7] = math.inf        # one value of a prefix key: its channel of its head
    b.attention()
    inf = ~torch.isfinite(b.out)
    assert inf[:, 6:8, 7].all() and not inf[:, :6].any() and not inf[:, 8:].any()
    assert not inf[:, 6:8, :7].any() and not inf[:, 6:8, 8:].any()
    assert status() == fp.FATHOM_OK


def test_shared_prefix_captured_and_on_two_streams():
    bs = [Batch([2300 + i, 2200, 2048, 0], 2048, 8, 2, 64, 16, BF16, False, 40 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in bs]
    for b in bs:
        b.table_t = torch.nn.functional.pad(b.table_t, (0, 10), value=-9)
        b.space = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        b.attention(max_len=2400, ws=b.space)
    torch.cuda.synchronize()
    graphs = []
    for b, s in zip(bs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            g.capture_begin()
            b.attention(max_len=2400, ws=b.space)
            g.capture_end()
        graphs.append(g)
    for r in range(3):
        for b in bs:
            b.lens = [2049 + 30 * r, 0, 2300, 2048]
            b.lens_t.copy_(torch.tensor(b.lens, dtype=torch.int32))
            b.table_t[:, 128:] = b.table_t[:1, 128:]            # all read the first one's own pages
            b.q.copy_(randn(list(b.q.shape), BF16, 90 + r))
            b.out.fill_(math.nan)
        torch.cuda.synchronize()
        for _ in range(4):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for b in bs:
            b.table = b.table_t.cpu().numpy()
            b.lens = [2049 + 30 * r, 0, 2300, 2048]
            check_rows(b, few_rows(b))
        assert status() == fp.FATHOM_OK


@pytest.mark.parametrize("prefix", [0, 512])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_of_sharp_and_growing_scores(prefix, dtype):
    """Scores of hundreds, each tile above the last: every tile renews the maximum."""
    n, d = 1500, 128
    b = Batch([n] * 3, prefix, 2, 4, d, 16, dtype, False, 3)
    ramp = torch.linspace(0.5, 24.0, n).to(dtype)
    for s in range(3):
        j = np.arange(n)
        pg, at = torch.from_numpy(b.table[s, j // 16]).long(), torch.from_numpy(j % 16)
        b.kv.k[pg.cuda(), :, at.cuda()] = ramp[:, None, None].expand(n, 2, d).contiguous().cuda()
    b.q.fill_(1.0)
    b.k64 = po.f64(b.kv.k)
    b.attention()
    want, tol = b.expect()
    check(b.out, want, tol)


def test_attention_keeps_nan_and_infinities_of_read_rows_to_their_sequence():
    b = Batch([40, 50, 60], 0, 1, 4, 64, 16, BF16, False, 5)
    b.kv.v[b.table[1, 2], 0, 3] = math.inf          # key 35 of sequence 1
    b.kv.k[b.table[2, 1], 0, 0] = math.nan          # key 16 of sequence 2
    b.attention()
    assert torch.isfinite(b.out[0]).all()
    assert not torch.isfinite(b.out[1]).any()
    assert torch.isnan(b.out[2]).all()


@pytest.mark.parametrize("lens,prefix", [([5, -1, 7], 0), ([5, 200, 7], 0), ([70, 30, 80], 64)])
def test_attention_refuses_bad_lengths(lens, prefix):
    fine = [n if i != 1 else max(prefix, 1) for i, n in enumerate(lens)]
    b = Batch(fine, prefix, 1, 2, 64, 16, F16, False, 9)
    b.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    b.table_t = torch.nn.functional.pad(b.table_t, (0, 96 // 16), value=-9)    # room for 96 keys
    b.attention(max_len=96)
    assert status() == fp.FATHOM_ERR_INVALID_ARG
    want, tol = b.expect()
    want[1], tol[1] = 0.0, 0.0
    check(b.out, want, tol)


@pytest.mark.parametrize("page", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("prefix", [0, 64])
def test_attention_never_follows_a_bad_page(page, prefix):
    b = Batch([100, 120], prefix, 1, 2, 64, 16, BF16, False, 4)
    b.table_t[0, 5] = page                      # keys 80..95 of sequence 0
    if prefix:
        b.table_t[:, 2] = page                  # and 32..47 of the prefix
    b.attention()
    assert status() == fp.FATHOM_ERR_INVALID_ARG
    assert torch.isfinite(b.out).all()
    if not prefix:
        want, tol = b.expect()
        check(b.out[1:], want[1:], tol[1:])
        keep = np.r_[0:80, 96:100][None, None].repeat(2, 0).repeat(2, 1)
        want, tol = b.expect(idx=keep, rows={(0, 0), (0, 1)})
        check(b.out[:1], want[:1], tol[:1])


def test_attention_strided_rows_and_offsets_past_32_bits():
    """Query rows inside a projection, and a cache whose pages lie over 2^32 elements apart."""
    H, G, d, page, n = 2, 4, 128, 16, 60
    b = Batch([n, 33], 0, H, G, d, page, BF16, False, 6)
    far = 1 << 28                                        # elements between pages
    pages = 20
    pool = torch.empty(2, pages * far // 2, dtype=BF16, device="cuda")   # overlapping k and v halves are apart
    k = pool[0].as_strided([pages // 2, H, page, d], [far, page * d, d, 1])
    v = pool[1].as_strided([pages // 2, H, page, d], [far, page * d, d, 1])
    assert (pages // 2 - 1) * far > 1 << 31
    kv = fp.PagedKV.from_tensors(k, v)
    n_p = b.kv.k.shape[0]
    place = torch.randperm(pages // 2)[:n_p]
    place[0] = pages // 2 - 1
    place = torch.unique(place)
    while len(place) < n_p:
        place = torch.unique(torch.cat([place, torch.randint(0, pages // 2, [1])]))
    for i, p in enumerate(place.tolist()):
        k[p].copy_(b.kv.k[i])
        v[p].copy_(b.kv.v[i])
    tab = np.where(b.table >= 0, place.numpy()[np.clip(b.table, 0, n_p - 1)], -1).astype(np.int32)
    wide = torch.zeros(2, H * G + 5, d + 8, dtype=BF16, device="cuda")
    q = wide[:, 2:2 + H * G, :d]
    q.copy_(b.q)
    out = torch.zeros(H * G, 2, d, dtype=BF16, device="cuda").transpose(0, 1)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    fp.fathom_paged_attention(kv.desc, q, torch.from_numpy(tab).cuda(), b.lens_t, n, out, ws, b.scale)
    want, tol = b.expect()
    check(out, want, tol)
    idx = np.tile(np.arange(n, dtype=np.int32), (2, H * G, 1))
    idx[1, :, 33:] = -1
    fp.fathom_sparse_attention_paged(kv.desc, q, torch.from_numpy(idx).cuda(), torch.from_numpy(tab).cuda(),
                                     b.lens_t, out, ws, b.scale)
    check(out, want, tol)
    assert status() == fp.FATHOM_OK


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 16384.0])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_smallest_and_largest_caps(cap, dtype):
    """Bounds as everywhere: 2^-21 of the cap for a score."""
    own = Batch([300, 5], 0, 2, 4, 64, 16, dtype, False, 11)
    own.attention(cap=cap)
    want, tol = own.expect(cap)
    check(own.out, want, tol)
    idx = np.full((2, 8, 300), -1, np.int32)
    for b, n in enumerate(own.lens):
        idx[b, :, :n] = np.arange(n)
    need = fp.fathom_sparse_attention_paged_workspace_bytes(2, 8, 64, 300)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    fp.fathom_sparse_attention_paged(own.kv.desc, own.q, torch.from_numpy(idx).cuda(), own.table_t, own.lens_t,
                                     own.out, ws, own.scale, cap)
    want, tol = own.expect(cap, idx=idx, round_p=False)
    check(own.out, want, tol)
    shared = Batch([2048 + i for i in range(9)], 2048, 2, 4, 64, 16, dtype, False, 12)
    assert 8 * 2048 * 2 * 64 * 4 >= 8 << 20
    shared.attention(cap=cap)
    check_rows(shared, {(0, 0), (3, 5), (8, 7)}, cap)
    assert status() == fp.FATHOM_OK


def test_attention_refuses_a_cache_in_host_memory():
    b = Batch([100], 0, 1, 2, 64, 16, BF16, False, 4, residency="host_mapped")
    with pytest.raises(fp.FathomError) as e:
        b.attention()
    assert e.value.status == fp.FATHOM_ERR_INVALID_ARG


@pytest.mark.parametrize("prefix", [0, 2048])
def test_attention_writes_only_its_output_rows(prefix):
    b = Batch([prefix + 70, 0, prefix + 1], prefix, 8, 2, 96, 16, F16, False, 4)
    wide = torch.full([3, 18, 104], 5.0, dtype=F16, device="cuda")
    b.out = wide[:, 1:17, :96]
    b.attention()
    want, tol = b.expect()
    check(b.out, want, tol)
    b.out.fill_(5.0)
    assert (wide == 5.0).all()


def test_attention_workspace_too_small_is_refused():
    b = Batch([1000], 0, 1, 2, 64, 16, BF16, False, 4)
    need = fp.fathom_paged_attention_workspace_bytes(b.kv.desc, 1, 2, 1000)
    assert need > 0
    with pytest.raises(fp.FathomError) as e:
        b.attention(ws=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == fp.FATHOM_ERR_WORKSPACE
    guard = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    b.attention(ws=guard[:need])
    torch.cuda.synchronize()
    assert (guard[need:] == 0xA5).all()


# --------------------------------------------------------- selected keys, in pages
SPARSE = [
    # lens, H, G, d, page, dtype, token_major, k, cap, slopes, residency
    ([4096], 8, 4, 128, 16, BF16, False, 500, 0.0, False, "device"),
    ([1, 40, 0], 1, 1, 32, 8, F16, True, 3, 0.0, False, "device"),
    ([300, 2000], 2, 3, 64, 64, BF16, False, 129, 30.0, True, "host_mapped"),
    ([90, 17], 2, 8, 96, 32, F16, True, 64, 0.0, True, "device"),
    ([1000], 1, 5, 160, 16, F16, False, 300, 20.0, False, "device"),
    ([700, 650], 1, 2, 192, 128, BF16, False, 128, 0.0, False, "host_mapped"),
    ([333], 2, 7, 224, 8, BF16, True, 333, 0.0, True, "device"),
    ([2048, 9], 2, 4, 256, 16, F16, False, 1025, 50.0, False, "device"),
]


@pytest.mark.parametrize("lens,H,G,d,page,dtype,tm,k,cap,slopes,residency", SPARSE)
def test_sparse(lens, H, G, d, page, dtype, tm, k, cap, slopes, residency):
    b = Batch(lens, 0, H, G, d, page, dtype, tm, 21 + d, residency=residency)
    rng = np.random.default_rng(k)
    idx = np.full((len(lens), H * G, k), -1, np.int32)
    for s, n in enumerate(lens):
        for i in range(H * G):
            m = min(n, k) - (i % 3 if n > 3 else 0)
            at = np.sort(rng.choice(k, m, replace=False))       # padding anywhere in the list
            idx[s, i, at] = rng.choice(n, m, replace=False) if n else 0
    if lens[0] > 4:
        idx[0, 0] = -1                                          # an empty list
        idx[0, -1, :2] = 3                                      # a key twice
    sl = b.slopes().cuda() if slopes else None
    need = fp.fathom_sparse_attention_paged_workspace_bytes(len(lens), H * G, d, k)
    guard = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    fp.fathom_sparse_attention_paged(b.kv.desc, b.q, torch.from_numpy(idx).cuda(), b.table_t, b.lens_t, b.out,
                                     guard[:need], b.scale, cap, sl)
    want, tol = b.expect(cap, sl, idx=idx, round_p=False)
    check(b.out, want, tol)
    assert status() == fp.FATHOM_OK and (guard[need:] == 0xA5).all()


def test_sparse_refuses_bad_keys_and_pages():
    b = Batch([100, 50], 0, 1, 2, 64, 16, BF16, False, 2)
    idx = np.tile(np.arange(20, dtype=np.int32), (2, 2, 1))
    for bad in (100, -2, 2 ** 31 - 1, -2 ** 31):
        one = idx.copy()
        one[0, 1, 7] = bad
        keep = idx.copy()
        keep[0, 1, 7] = -1
        ws = torch.empty(16, dtype=torch.uint8, device="cuda")
        fp.fathom_sparse_attention_paged(b.kv.desc, b.q, torch.from_numpy(one).cuda(), b.table_t, b.lens_t,
                                         b.out, ws, b.scale)
        assert status() == fp.FATHOM_ERR_INVALID_ARG
        want, tol = b.expect(idx=keep, round_p=False)
        check(b.out, want, tol)
    b.table_t[0, 1] = 99
    fp.fathom_sparse_attention_paged(b.kv.desc, b.q, torch.from_numpy(idx).cuda(), b.table_t, b.lens_t, b.out,
                                     ws, b.scale)
    assert status() == fp.FATHOM_ERR_INVALID_ARG
    keep = np.where(idx >= 16, -1, idx)
    keep[1] = idx[1]
    want, tol = b.expect(idx=keep, round_p=False)
    check(b.out, want, tol)


# -------------------------------------------------------------------- used together
def test_decode_steps_with_the_scan():
    """A prompt and four decode steps of one layer: norm and rotation, paged append, key index append,
    plan, scan, and attention over the scan's selection; then over all keys."""
    H, G, d, page, n0, steps, k = 2, 4, 128, 16, 3000, 4, 256
    hq = H * G
    rot = fp.RotaryTable(d, base=1e6)
    qw, kw = ((1 + 0.2 * randn([d], F32, i)).to(BF16).cuda() for i in (1, 2))
    T = n0 + steps
    qkv = randn([T, hq + 2 * H, d], BF16, 3).cuda()
    qr, kr, vr = qkv[:, :hq], qkv[:, hq:hq + H], qkv[:, hq + H:]
    kv = make_pool(T // page + 2, H, page, d, BF16, False)
    tab = torch.randperm(T // page + 1, dtype=torch.int32)[None].cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    ix = fp.KeyIndex(H, G, n0, d, capacity=T)

    def keys32(a, b):
        out = torch.empty([H, b - a, d], device="cuda")
        fp.fathom_qk_norm_rope(None, kr[a:b], pos[a:b], None, out.transpose(0, 1), rot, None, kw)
        fp.fathom_append_kv(kv.desc, kr[a:b], vr[a:b], seq[a:b], pos[a:b], tab, rot, kw)
        return out

    ix.pack(keys32(0, n0))
    buf = fp.ScanBuffers(ix, k)
    budget = torch.full([hq], 4 * d, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    y, size = po.norm_rope(po.f64(kr), np.arange(T, dtype=np.float64), po.f64(kw), 1e-6, po.turns(d, 1e6)[0])
    pool_k, pool_v, table = None, None, tab.cpu().numpy()[0]
    for s in range(steps):
        t = n0 + s
        ix.append(keys32(t, t + 1))
        q = torch.empty([1, hq, d], dtype=BF16, device="cuda")
        fp.fathom_qk_norm_rope(qr[t:t + 1], None, pos[t:t + 1], q, None, rot, qw)
        fp.plan_and_scan(ix, q.view(hq, d).view(torch.int16), budget, buf)
        n = torch.full([1], t + 1, dtype=torch.int32, device="cuda")
        out, dense = torch.empty_like(q), torch.empty_like(q)
        fp.fathom_sparse_attention_paged(kv.desc, q, buf.idx[None], tab, n, out, ws, d ** -0.5)
        fp.fathom_paged_attention(kv.desc, q, tab, n, T, dense, ws, d ** -0.5)
        assert status() == fp.FATHOM_OK
        idx, q64 = buf.idx.cpu().numpy(), po.f64(q)[0]
        pool_k, pool_v = po.f64(kv.k), po.f64(kv.v)
        all_j = np.arange(t + 1)
        rows = pool_k[table[all_j // page], :, all_j % page]
        check(torch.from_numpy(rows), y[:t + 1], po.norm_rope_tolerance(y, size, BF16)[:t + 1], "cache")
        for i in range(hq):
            for o, j, step in ((out, idx[i], 0.0), (dense, all_j, po.HALF_STEP[BF16])):
                ks, vs = (po.gather(p, table, j, i // G, page) for p in (pool_k, pool_v))
                want, err = po.attend(q64[i], ks, vs, t - j, d ** -0.5, p_step=step)
                check(o[0, i], want, err + po.HALF_STEP[BF16] * np.abs(want) * 1.01)


@pytest.mark.parametrize("prefix", [0, 256])
def test_captured_step_replays_on_new_inputs(prefix):
    """One graph of append and attention, replayed while lengths, positions, rows and pages change."""
    H, G, d, page, n_seq, longest = 2, 4, 64, 16, 3, 400
    b = Batch([prefix + 40, prefix + 1, prefix + 33], prefix, H, G, d, page, BF16, False, 7, spare=80)
    # room to grow: unused pages of the pool behind each sequence's own
    free = [p for p in range(b.kv.k.shape[0]) if p not in set(b.table[b.table >= 0].tolist())]
    table = np.full((n_seq, longest // page), -1, np.int32)
    table[:, :b.table.shape[1]] = b.table
    for s in range(n_seq):
        for c in range(longest // page):
            if table[s, c] < 0:
                table[s, c] = free.pop() if free else 0
    b.table, b.table_t = table, torch.from_numpy(table).cuda()
    k, v = torch.zeros([n_seq, H, d], dtype=BF16, device="cuda"), torch.zeros([n_seq, H, d], dtype=BF16, device="cuda")
    seq, pos = torch.arange(n_seq, dtype=torch.int32, device="cuda"), torch.zeros(n_seq, dtype=torch.int32, device="cuda")

    def step():
        fp.fathom_append_kv(b.kv.desc, k, v, seq, pos, b.table_t)
        b.attention(max_len=longest, ws=ws)

    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    pos.copy_(b.lens_t - 1)
    k.copy_(torch.stack([b.kv.k[table[s, (n - 1) // page], :, (n - 1) % page] for s, n in enumerate(b.lens)]))
    v.copy_(torch.stack([b.kv.v[table[s, (n - 1) // page], :, (n - 1) % page] for s, n in enumerate(b.lens)]))
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin()
        step()
        graph.capture_end()
    for r in range(3):
        b.lens = [n + 1 for n in b.lens]
        b.lens_t.copy_(torch.tensor(b.lens, dtype=torch.int32))
        pos.copy_(b.lens_t - 1)
        k.copy_(randn([n_seq, H, d], BF16, 50 + r))
        v.copy_(randn([n_seq, H, d], BF16, 60 + r))
        b.q.copy_(randn(list(b.q.shape), BF16, 70 + r))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.k64, b.v64 = po.f64(b.kv.k), po.f64(b.kv.v)
        want, tol = b.expect()
        check(b.out, want, tol)
        assert status() == fp.FATHOM_OK


def test_calls_on_two_streams_with_their_own_workspaces():
    bs = [Batch([900 + i, 1500], 512, 2, 4, 128, 16, BF16, False, 30 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(bs, streams):
            b.attention(stream=s, ws=getattr(b, "ws", None))
    torch.cuda.synchronize()
    for b in bs:
        want, tol = b.expect()
        check(b.out, want, tol)
